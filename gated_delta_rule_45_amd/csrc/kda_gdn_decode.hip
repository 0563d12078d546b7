// Gated delta rule, recurrent form on a pool of state slots: one or a few new tokens per sequence,
// states updated in place (Kimi Linear summary page, "From linear attention to Gated DeltaNet": the
// scalar-gate delta rule; the fixed-size state takes the place of a growing key-value cache).
//
//     S <- e^g S;  u = beta (v - S^T k);  S <- S + k u^T;  o = scale S^T q
//
// Bound: HBM, each state is read and written once per call whatever the token count.  The state's
// columns do not meet, so one wave owns 32 columns of one (sequence, value head): a lane holds 16 bytes
// (W columns) of each of d_k / RG rows, in fp32 registers over all its tokens.  S^T k and S^T q of the decayed
// state are summed in one pass and one exchange between the RG row groups (o = S'^T q + (q.k) u), in
// registers: a wave needs no LDS and no barrier.  The next token's inputs are loaded while the current
// one is computed.  All arithmetic is fp32; a bf16 state is rounded once, at the end.
//
// 32 heads of 128 x 128 (bf16 q, k, v): 256 sequences, one token, fp32 states 188 us (5.8 TB/s), bf16 states
// 106 us (5.1 TB/s); 96 sequences, 4 tokens, bf16 states 58 us (3.5 TB/s: here the arithmetic of four
// tokens, about 350 instructions each, costs as much as the transfer; exchanging through LDS 69 us).
#include <type_traits>

#include "kda_device.h"
#include "kda_gdn.h"

namespace kda {
namespace gdn {
namespace {

constexpr int kCols = 32;

template <typename T, int N>
struct Vals {
    static constexpr int kPer = 16 / sizeof(T);  // elements of a 16-byte load
    u32x4 w[(N + kPer - 1) / kPer];
    __device__ __forceinline__ void load(const T *p) {
        static_assert(N % kPer == 0 || 2 * N == kPer);
        if constexpr (N < kPer) {
            const uint2 x = *reinterpret_cast<const uint2 *>(p);
            w[0] = u32x4{x.x, x.y, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < N / kPer; ++i) w[i] = reinterpret_cast<const u32x4 *>(p)[i];
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(T) == 2) {
            const unsigned x = w[i / 8][(i % 8) / 2];
            return i & 1 ? bf16_hi(x) : bf16_lo(x);
        } else {
            return __uint_as_float(w[i / 4][i % 4]);
        }
    }
};

__device__ __forceinline__ float load_gate1(const void *p, int64_t at, int bf16) {
    return bf16 ? bf16_to_f32(static_cast<const uint16_t *>(p)[at]) : static_cast<const float *>(p)[at];
}

// x and y summed over the halves of a wave, the sum of x in the lower one and that of y in the upper one;
// then the same for the 16-lane rows of each half; and the ways back.
__device__ __forceinline__ float fold32(float x, float y) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float fold16(float x, float y) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ void unfold32(float z, float &x, float &y) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(z), __float_as_uint(z), false, false);
    x = __uint_as_float(r[0]);
    y = __uint_as_float(r[1]);
}
__device__ __forceinline__ void unfold16(float z, float &x, float &y) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(z), __float_as_uint(z), false, false);
    x = __uint_as_float(r[0]);
    y = __uint_as_float(r[1]);
}
template <int ROR>
__device__ __forceinline__ float add_turned(float x) {  // + the lane ROR further in its row of 16
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x120 + ROR, 0xf, 0xf, true));
}
// Sums over the lanes that differ in their row group (lane / CG), in every lane.
template <int CG>
__device__ __forceinline__ float sum_row(float x) {
    x = add_turned<8>(x);
    if constexpr (CG == 4) x = add_turned<4>(x);
    return x;
}
template <int W, int CG>
__device__ __forceinline__ void sum_groups(float (&a)[W], float (&b)[W], float &c) {
#pragma unroll
    for (int j = 0; j < W; j += 2) {
        const float s = sum_row<CG>(fold16(fold32(a[j], b[j]), fold32(a[j + 1], b[j + 1])));
        float x, y;
        unfold16(s, x, y);
        unfold32(x, a[j], b[j]);
        unfold32(y, a[j + 1], b[j + 1]);
    }
    c = fold32(c, c);
    c = sum_row<CG>(fold16(c, c));
}

template <typename T, int W>
__device__ __forceinline__ void load_w(float (&x)[W], const T *p) {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
        const float4 v = IoTraits<T>::load4(p + i);
        x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
    }
}

template <typename IO, typename ST, int DK>
__global__ void __launch_bounds__(256) gdn_decode_kernel(DecodeParams p) {
    constexpr int W = 16 / sizeof(ST), CG = kCols / W, RG = 64 / CG, R = DK / RG;
    const int lane = threadIdx.x & 63, rg = lane / CG, cg = lane % CG;
    const int ntile = p.dv / kCols;
    const int64_t item = (int64_t)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6);
    if (item >= (int64_t)p.num_seqs * p.Hv * ntile) return;
    const int tile = (int)(item % ntile), h = (int)(item / ntile % p.Hv);
    const int n = (int)(item / ntile / p.Hv);
    const int hk = h / (p.Hv / p.Hk);
    const int64_t slot = p.slots ? p.slots[n] : n;
    if (slot < 0 || slot >= p.num_slots) return;  // a padded row: its state and its outputs stay as they are
    int64_t t0;
    int len;
    if (p.cu) {
        const int a = min(max(p.cu[n], 0), p.T), b = min(max(p.cu[n + 1], a), p.T);
        t0 = a;
        len = b - a;
    } else {
        t0 = (int64_t)n * p.T;
        len = p.T;
    }
    if (len <= 0) return;
    const int col = tile * kCols + W * cg;
    const IO *q = static_cast<const IO *>(p.q) + t0 * p.ldq + hk * DK + rg * R;
    const IO *k = static_cast<const IO *>(p.k) + t0 * p.ldk + hk * DK + rg * R;
    const IO *v = static_cast<const IO *>(p.v) + t0 * p.ldv + (int64_t)h * p.dv + col;
    IO *o = static_cast<IO *>(p.out) + (t0 * p.Hv + h) * p.dv + col;
    ST *st = static_cast<ST *>(p.state) + ((slot * p.Hv + h) * DK + rg * R) * p.dv + col;

    float S[R][W];
#pragma unroll
    for (int m = 0; m < R; ++m) {
        // a wave's rows of a bf16 state are half a cache line: kept, as the next wave reads the other half
        const u32x4 *at = reinterpret_cast<const u32x4 *>(st + m * p.dv);
        const u32x4 x = W == 4 ? __builtin_nontemporal_load(at) : *at;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (W == 4) {
                S[m][i] = __uint_as_float(x[i]);
            } else {
                S[m][2 * i] = bf16_lo(x[i]);
                S[m][2 * i + 1] = bf16_hi(x[i]);
            }
        }
    }
    Vals<IO, R> kn, qn;
    kn.load(k);
    qn.load(q);
    float vn[W];
    load_w(vn, v);
    float gn = load_gate1(p.g, t0 * p.Hv + h, p.gate_bf16), bn = load_gate1(p.beta, t0 * p.Hv + h, p.gate_bf16);
#pragma unroll 1
    for (int t = 0; t < len; ++t) {
        const Vals<IO, R> kc = kn, qc = qn;
        float vc[W];
#pragma unroll
        for (int j = 0; j < W; ++j) vc[j] = vn[j];
        const float a = expf(gn), beta = bn;
        if (t + 1 < len) {
            k += p.ldk;
            q += p.ldq;
            v += p.ldv;
            kn.load(k);
            qn.load(q);
            load_w(vn, v);
            const int64_t at = (t0 + t + 1) * p.Hv + h;
            gn = load_gate1(p.g, at, p.gate_bf16);
            bn = load_gate1(p.beta, at, p.gate_bf16);
        }
        float pk[W], pq[W], qk = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) pk[j] = pq[j] = 0.f;
#pragma unroll
        for (int m = 0; m < R; ++m) {
            const float km = kc[m], qm = qc[m];
#pragma unroll
            for (int j = 0; j < W; ++j) {
                S[m][j] *= a;
                pk[j] = fmaf(km, S[m][j], pk[j]);
                pq[j] = fmaf(qm, S[m][j], pq[j]);
            }
            qk = fmaf(qm, km, qk);
        }
        sum_groups<W, CG>(pk, pq, qk);
        float u[W], y[W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            u[j] = beta * (vc[j] - pk[j]);
            y[j] = p.scale * fmaf(qk, u[j], pq[j]);
        }
#pragma unroll
        for (int m = 0; m < R; ++m) {
            const float km = kc[m];
#pragma unroll
            for (int j = 0; j < W; ++j) S[m][j] = fmaf(km, u[j], S[m][j]);
        }
        if (rg == 0) {
#pragma unroll
            for (int j = 0; j < W; j += 4)
                IoTraits<IO>::store4(o + (int64_t)t * p.Hv * p.dv + j, make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]));
        }
    }
#pragma unroll
    for (int m = 0; m < R; ++m) {
        if constexpr (W == 4) {
            __builtin_nontemporal_store(f32x4{S[m][0], S[m][1], S[m][2], S[m][3]}, reinterpret_cast<f32x4 *>(st + m * p.dv));
        } else {
            IoTraits<ST>::store4(st + m * p.dv, make_float4(S[m][0], S[m][1], S[m][2], S[m][3]));
            IoTraits<ST>::store4(st + m * p.dv + 4, make_float4(S[m][4], S[m][5], S[m][6], S[m][7]));
        }
    }
}

template <typename IO, typename ST, int DK>
hipError_t launch(const DecodeParams &p, hipStream_t stream) {
    const int64_t items = (int64_t)p.num_seqs * p.Hv * (p.dv / kCols);
    if (items <= 0) return hipSuccess;
    hipLaunchKernelGGL((gdn_decode_kernel<IO, ST, DK>), dim3((unsigned)((items + 3) / 4)), dim3(256), 0, stream, p);
    return hipGetLastError();
}
template <typename IO>
hipError_t launch_io(const DecodeParams &p, hipStream_t s) {
    if (p.dk == 64) return p.state_bf16 ? launch<IO, uint16_t, 64>(p, s) : launch<IO, float, 64>(p, s);
    return p.state_bf16 ? launch<IO, uint16_t, 128>(p, s) : launch<IO, float, 128>(p, s);
}

}  // namespace

hipError_t launch_decode(bool io_bf16, const DecodeParams &p, hipStream_t stream) {
    return io_bf16 ? launch_io<uint16_t>(p, stream) : launch_io<float>(p, stream);
}

}  // namespace gdn
}  // namespace kda
