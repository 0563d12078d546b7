// Gradients of the output epilogue (Kimi Linear summary page, section "Kimi Linear model
// composition"; the reading of the forward is out = o * r * w * sigmoid(z), r = (mean(o^2) + eps)^-1/2,
// for every (token, head) row of d values).  With hat = o r, s = sigmoid(z) and dn = dy w s:
//
//     do = r (dn - hat mean(dn hat))      dz = dy hat w s (1 - s)      dw = sum over rows of dy hat s
//
// Bound: HBM (reads o, z and dy once, writes do and dz once).  As in the forward, a lane holds one
// 16-byte segment of a row and the lanes of a row sum over it with lane shuffles.  Every workgroup
// walks its share of the rows and keeps its part of dw in registers (fp32: at most rows / (blocks *
// rows per pass) terms per lane), adds it up over its lanes in LDS and writes one partial row; a
// second kernel adds the partial rows in fp64 in a fixed order, so dw repeats bit for bit.  A call
// that one workgroup covers writes dw itself.
//
// 262,144 rows of 128 in bf16: 72 us (4.65 TB/s of the 4.8 that a large copy reaches), 62 of them the
// gradients and 6 the sum of the partial rows (2,048 of them, eight loads in flight per lane; one: 12).
#include "kda_device.h"
#include "kda_internal.h"
#include "kda_seg.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 2048;  // eight workgroups per CU

template <typename IO, int D>
constexpr int rows_per_pass() {
    return kThreads / (D / Seg<IO>::N);
}

template <typename IO, int D>
__global__ void __launch_bounds__(kThreads) norm_gate_bwd_kernel(int64_t rows, float eps, const IO *__restrict__ o,
                                                                 const IO *__restrict__ z,
                                                                 const float *__restrict__ weight,
                                                                 const IO *__restrict__ dy, IO *d_o, IO *d_z,
                                                                 float *__restrict__ dw) {
    constexpr int N = Seg<IO>::N, LPR = D / N, RPP = rows_per_pass<IO, D>();
    __shared__ float part[RPP][D];
    const int lr = threadIdx.x % LPR, rr = threadIdx.x / LPR;
    float w[N], acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        w[i] = weight[lr * N + i];
        acc[i] = 0.f;
    }
    for (int64_t row = (int64_t)blockIdx.x * RPP + rr; row < rows; row += (int64_t)gridDim.x * RPP) {
        const int64_t at = row * D + lr * N;
        float x[N], g[N], y[N];
        Seg<IO>::load(o + at, x);
        Seg<IO>::load(z + at, g);
        Seg<IO>::load(dy + at, y);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int off = LPR / 2; off >= 1; off >>= 1) ss += __shfl_xor(ss, off);
        const float r = 1.0f / sqrtf(ss * (1.0f / D) + eps);
        float dn[N], dot = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            // s and 1 - s from one exponential of -|z| <= 0, without overflow or cancellation
            const float e = __builtin_amdgcn_exp2f(-1.44269504f * fabsf(g[i])), u = __builtin_amdgcn_rcpf(1.0f + e);
            const float big = u, small = e * u, s = g[i] >= 0.f ? big : small;
            x[i] *= r;
            const float ys = y[i] * s;
            acc[i] = fmaf(ys, x[i], acc[i]);
            dn[i] = ys * w[i];
            dot = fmaf(dn[i], x[i], dot);
            g[i] = dn[i] * x[i] * (g[i] >= 0.f ? small : big);
        }
#pragma unroll
        for (int off = LPR / 2; off >= 1; off >>= 1) dot += __shfl_xor(dot, off);
        dot *= 1.0f / D;
#pragma unroll
        for (int i = 0; i < N; ++i) dn[i] = r * fmaf(-x[i], dot, dn[i]);
        Seg<IO>::store(d_o + at, dn);
        Seg<IO>::store(d_z + at, g);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) part[rr][lr * N + i] = acc[i];
    __syncthreads();
    if (threadIdx.x < D) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < RPP; ++i) s += part[i][threadIdx.x];
        dw[(int64_t)blockIdx.x * D + threadIdx.x] = s;
    }
}

// dw = sum of `blocks` partial rows: a workgroup owns 16 columns, 64 lanes of rows each, a lane's rows eight
// loads at a time
template <int D>
__global__ void __launch_bounds__(1024) norm_gate_dw_kernel(int blocks, const float *__restrict__ part,
                                                            float *__restrict__ dw) {
    __shared__ double sum[64][16];
    const int c = threadIdx.x & 15, r = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
    double s = 0.0;
    for (int i0 = r; i0 < blocks; i0 += 64 * 8) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + 64 * j;
            x[j] = part[(int64_t)min(i, blocks - 1) * D + col];
            if (i >= blocks) x[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) s += x[j];
    }
    sum[r][c] = s;
    __syncthreads();
    for (int h = 32; h >= 1; h >>= 1) {
        if (r < h) sum[r][c] += sum[r + h][c];
        __syncthreads();
    }
    if (r == 0) dw[col] = (float)sum[0][c];
}

template <typename IO, int D>
hipError_t launch(int64_t rows, float eps, const void *o, const void *z, const float *w, const void *dy, void *d_o,
                  void *d_z, float *dw, float *part, int blocks, hipStream_t stream) {
    hipLaunchKernelGGL((norm_gate_bwd_kernel<IO, D>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, rows, eps,
                       static_cast<const IO *>(o), static_cast<const IO *>(z), w, static_cast<const IO *>(dy),
                       static_cast<IO *>(d_o), static_cast<IO *>(d_z), blocks > 1 ? part : dw);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || blocks == 1) return e;
    hipLaunchKernelGGL((norm_gate_dw_kernel<D>), dim3(D / 16), dim3(1024), 0, stream, blocks, part, dw);
    return hipGetLastError();
}

}  // namespace

// One workgroup also where there are no rows: it writes dw = 0.
int norm_gate_bwd_blocks(kda_dtype_t io, int64_t rows, int d) {
    const int64_t rpp = kThreads / (d / (io == KDA_BF16 ? 8 : 4));
    const int64_t b = rows / rpp + (rows % rpp != 0);
    return (int)(b < 1 ? 1 : b > kMaxBlocks ? kMaxBlocks : b);
}

hipError_t launch_norm_gate_bwd(kda_dtype_t io, int64_t rows, int d, float eps, const void *o, const void *z,
                                const float *w, const void *dy, void *d_o, void *d_z, float *dw, float *part,
                                hipStream_t stream) {
    const int blocks = norm_gate_bwd_blocks(io, rows, d);
    if (io == KDA_BF16)
        return d == 64 ? launch<uint16_t, 64>(rows, eps, o, z, w, dy, d_o, d_z, dw, part, blocks, stream)
                       : launch<uint16_t, 128>(rows, eps, o, z, w, dy, d_o, d_z, dw, part, blocks, stream);
    return d == 64 ? launch<float, 64>(rows, eps, o, z, w, dy, d_o, d_z, dw, part, blocks, stream)
                   : launch<float, 128>(rows, eps, o, z, w, dy, d_o, d_z, dw, part, blocks, stream);
}

}  // namespace kda
