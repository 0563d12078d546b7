// Rotary positions of queries and keys, or (sign -1) their gradients: pairs of a head's leading channels turned by
// position * frequency.
//
// Bound: HBM, each value is read and written once.  A thread owns 8 pairs (16 channels) of a token and turns them in
// HP heads, so that the angles (about 30 instructions a pair, some in 64 bits) are worked out once for them; the
// threads of a wave lie along a head and then along the heads, whose loads are all issued first.
//
// bf16, 16,384 tokens: 16 + 8 heads of 128, slices of one projection, 42 us a call (4.8 TB/s; the kernel 34); 32 + 8 heads, half
// of the channels copied, 64 us (5.3 TB/s).  A copy reaches 4.9.
#include "kda_paged.h"
#include "kda_rope.h"

namespace kda {
namespace paged {
namespace {

// Heads per thread: four, so that the angles cost less than the transfer, or one where four would leave lanes of
// the chip without work (256 CUs x 2,048 threads).
constexpr int kHeads = 4;
int64_t items_of(int64_t tokens, int32_t heads, int32_t d, int hp) {
    return tokens * ((heads + hp - 1) / hp) * (d / 16);
}
int heads_per_thread(int64_t tokens, int32_t heads, int32_t d) {
    return items_of(tokens, heads, d, kHeads) >= 256 * 2048 ? kHeads : 1;
}

template <typename IO, int D, int HP>
__global__ void __launch_bounds__(256) rope_kernel(RopeParams p) {
    constexpr unsigned U = D / 16;
    const unsigned heads = p.Hq + p.Hk, groups = (heads + HP - 1) / HP;
    const unsigned idx = blockIdx.x * 256u + threadIdx.x;
    const int u = idx % U;
    const unsigned r = idx / U, hg = r % groups;
    const int64_t t = r / groups;
    if (t >= p.tokens) return;
    const bool turned = 16 * u < p.rot;
    Turn turn;
    if (turned) turn.set(p.positions ? p.positions[t] : (int)(t % p.T), p.freq, u, p.amplitude, p.sign);
    const int a0 = run0(u, p.rot, p.interleaved), b0 = run1(u, p.rot, p.interleaved);
    Eight<IO> a[HP], b[HP];
#pragma unroll
    for (int i = 0; i < HP; ++i) {
        const unsigned h = hg + i * groups;
        if (h >= heads) continue;
        const IO *x = h < (unsigned)p.Hq ? static_cast<const IO *>(p.q) + t * p.ldq + h * D
                                         : static_cast<const IO *>(p.k) + t * p.ldk + (h - p.Hq) * D;
        a[i].load(x + a0);
        b[i].load(x + b0);
    }
#pragma unroll
    for (int i = 0; i < HP; ++i) {
        const unsigned h = hg + i * groups;
        if (h >= heads) continue;
        if (turned) turn.apply(a[i], b[i], p.interleaved);
        IO *y = h < (unsigned)p.Hq ? static_cast<IO *>(p.q_out) + t * p.ldqo + h * D
                                   : static_cast<IO *>(p.k_out) + t * p.ldko + (h - p.Hq) * D;
        a[i].store(y + a0);
        b[i].store(y + b0);
    }
}

template <typename IO, int D>
hipError_t launch(const RopeParams &p, hipStream_t stream) {
    const int hp = heads_per_thread(p.tokens, p.Hq + p.Hk, D);
    const int64_t items = items_of(p.tokens, p.Hq + p.Hk, D, hp);
    if (items <= 0) return hipSuccess;
    const dim3 grid((unsigned)((items + 255) / 256));
    if (hp == kHeads)
        hipLaunchKernelGGL((rope_kernel<IO, D, kHeads>), grid, dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((rope_kernel<IO, D, 1>), grid, dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace

int64_t rope_items(int64_t tokens, int32_t heads, int32_t d) {
    return items_of(tokens, heads, d, heads_per_thread(tokens, heads, d));
}

hipError_t launch_rope(bool bf16, const RopeParams &p, hipStream_t stream) {
    if (bf16) return p.d == 128 ? launch<uint16_t, 128>(p, stream) : launch<uint16_t, 64>(p, stream);
    return p.d == 128 ? launch<float, 128>(p, stream) : launch<float, 64>(p, stream);
}

}  // namespace paged
}  // namespace kda
