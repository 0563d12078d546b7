// Joins the segments of a walk that was split over its length.  (Gradients: the same with M transposed, from the
// last segment to the first, H from a reverse walk of each segment.)  A chunk takes the state S to
// (e^{G_C} I - ..) S + .., a linear map, so a whole segment takes it to M S + H.  One scan over the segments
// side by side gives H (from a zero state) and M (from the identity and no values); this kernel then walks
// the few segments, S <- M_p S + H_p, and leaves the state entering each of them where H_p was.
//
// One workgroup owns (sequence, value head, 16 columns), each wave a row tile.  M_p (64 KB at d_k = 128) and
// H_p are read straight into operands, a segment ahead; S goes through LDS, transposed.  All in fp32.
// 65,536 tokens x 8 heads of 128 x 128, 8 segments: 20 us of 874 (the maps 507, the forward on the segments
// 330; one walk 2,389).
#include "kda_device.h"
#include "kda_gdn.h"

namespace kda {
namespace gdn {
namespace {

template <int DK, bool REV>
__global__ void __launch_bounds__(4 * DK) gdn_join_kernel(JoinParams p) {
    constexpr int KT = DK / 16, LD = DK + 4;
    __shared__ __attribute__((aligned(16))) float St[2][16 * LD];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, q4 = lane >> 4, row = 16 * wave + 4 * q4;
    const int ntile = p.dv / 16, col = (int)(blockIdx.x % ntile) * 16 + l16;
    const int64_t chain = blockIdx.x / ntile;  // sequence * Hv + value head
    const int64_t b = chain / p.Hv, h = chain % p.Hv;
    f32x4 S = zero4();
    auto load0 = [&](auto *src) {
#pragma unroll
        for (int j = 0; j < 4; ++j) S[j] = elem_f32(src[(chain * DK + row + j) * p.dv + col]);
    };
    if (p.s0 && p.state_bf16) load0(static_cast<const uint16_t *>(p.s0));
    else if (p.s0) load0(static_cast<const float *>(p.s0));
    // the maps of segment s: a row tile of M and a tile of H
    struct Maps {
        Frag<false> m[KT];
        f32x4 h;
    };
    auto at = [&](int s) { return (b * p.segs + (REV ? p.segs - 1 - s : s)) * p.Hv + h; };
    auto load = [&](Maps &x, int s) {
        const float *M = p.m + at(s) * DK * DK + (REV ? 4 * q4 * DK + 16 * wave + l16 : (16 * wave + l16) * DK + 4 * q4);
        const float *H = p.h + (at(s) * DK + row) * p.dv + col;
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            if constexpr (REV) {
                const float *m = M + 16 * t * DK;
                x.m[t].v = make_float4(m[0], m[DK], m[2 * DK], m[3 * DK]);
            } else {
                x.m[t].v = *reinterpret_cast<const float4 *>(M + 16 * t);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) x.h[j] = H[(int64_t)j * p.dv];
    };
    auto put = [&](int s) {
        float *H = p.h + (at(s) * DK + row) * p.dv + col;
#pragma unroll
        for (int j = 0; j < 4; ++j) H[(int64_t)j * p.dv] = S[j];
    };
    auto step = [&](Maps &now, Maps &next, int s) {
        float *x = St[s & 1];
        *reinterpret_cast<f32x4 *>(x + l16 * LD + row) = S;
        if (s + 2 < p.segs) load(next, s + 1);
        __syncthreads();
        put(s);
        S = now.h;
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            Frag<false> f;
            f.v = *reinterpret_cast<const float4 *>(x + l16 * LD + 16 * t + 4 * q4);
            mma16(S, now.m[t], f);
        }
        mfma_settle(S);
    };
    Maps a, c;
    load(a, 0);
    int s = 0;
    for (; s + 2 < p.segs; s += 2) {
        step(a, c, s);
        step(c, a, s + 1);
    }
    if (s + 1 < p.segs) step(a, c, s++);
    put(s);
}

}  // namespace

hipError_t launch_join(const JoinParams &p, hipStream_t stream) {
    const int64_t blocks = (int64_t)p.batch * p.Hv * (p.dv / 16);
    if (blocks <= 0) return hipSuccess;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3((unsigned)(4 * p.dk)), 0, stream, p);
        return hipGetLastError();
    };
    if (p.dk == 64) return p.reverse ? go(gdn_join_kernel<64, true>) : go(gdn_join_kernel<64, false>);
    return p.reverse ? go(gdn_join_kernel<128, true>) : go(gdn_join_kernel<128, false>);
}

}  // namespace gdn
}  // namespace kda
