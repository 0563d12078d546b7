// bf16 rows to dense fp32 rows and back, for the calls of few values that run on fp32 operands.
#include "kda_device.h"
#include "kda_gdn.h"

namespace kda {
namespace gdn {
namespace {

// One launch converts up to four tensors: blockIdx.y picks the tensor, a thread one 16-byte piece of bf16.
template <bool WIDEN>
__global__ void __launch_bounds__(256) convert_kernel(ConvertParams p) {
    const ConvertRows t = p.t[blockIdx.y];
    const int64_t per = t.cols / 8;
    int64_t first = 0, n = t.rows * per;
    if (p.cu) {
        const int a = min(max(p.cu[0], 0), p.T), b = min(max(p.cu[p.num_seqs], a), p.T);
        first = a * per;
        n = b * per;
    }
    for (int64_t i = first + (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per, c = i % per * 8;
        uint16_t *b = static_cast<uint16_t *>(t.bf16) + row * t.ld + c;
        float *f = static_cast<float *>(t.f32) + row * t.cols + c;
        if constexpr (WIDEN) {
            IoTraits<float>::store4(f, IoTraits<uint16_t>::load4(b));
            IoTraits<float>::store4(f + 4, IoTraits<uint16_t>::load4(b + 4));
        } else {
            IoTraits<uint16_t>::store4(b, IoTraits<float>::load4(f));
            IoTraits<uint16_t>::store4(b + 4, IoTraits<float>::load4(f + 4));
        }
    }
}

}  // namespace

hipError_t launch_convert(bool widen, const ConvertParams &p, hipStream_t stream) {
    int64_t most = 0;
    for (int i = 0; i < p.n; ++i) most = p.t[i].rows * (p.t[i].cols / 8) > most ? p.t[i].rows * (p.t[i].cols / 8) : most;
    if (most <= 0) return hipSuccess;
    const int64_t blocks = (most + 255) / 256;
    const dim3 grid((unsigned)(blocks < 1024 ? blocks : 1024), (unsigned)p.n);
    if (widen) hipLaunchKernelGGL((convert_kernel<true>), grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((convert_kernel<false>), grid, dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace gdn
}  // namespace kda
