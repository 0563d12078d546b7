// Gated delta rule, recurrent form on a pool of state slots: one or a few new tokens per sequence,
// states updated in place (Kimi Linear summary page, "From linear attention to Gated DeltaNet": the
// scalar-gate delta rule; the fixed-size state takes the place of a growing key-value cache).
//
//     S <- e^g S;  u = beta (v - S^T k);  S <- S + k u^T;  o = scale S^T q
//
// Bound: HBM, each state is read and written once per call whatever the token count.  The state's
// columns do not meet, so one wave owns 32 columns of one (sequence, value head): lane (rg, cg) holds
// rows d_k / 8 * rg .. and columns 4 cg .. + 3 in registers over all its tokens.  S^T k and S^T q of
// the decayed state are summed in one pass and one exchange between the 8 row groups (o = S'^T q +
// (q.k) u), so a wave needs no LDS and no barrier.  The next token's inputs are loaded while the
// current one is computed.  All arithmetic is fp32; a bf16 state is rounded once, at the end.
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

template <typename IO, typename ST, int DK>
__global__ void __launch_bounds__(256) gdn_decode_kernel(DecodeParams p) {
    constexpr int R = DK / 8;
    const int lane = threadIdx.x & 63, rg = lane >> 3, cg = lane & 7;
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
    const int col = tile * kCols + 4 * cg;
    const IO *q = static_cast<const IO *>(p.q) + t0 * p.ldq + hk * DK + rg * R;
    const IO *k = static_cast<const IO *>(p.k) + t0 * p.ldk + hk * DK + rg * R;
    const IO *v = static_cast<const IO *>(p.v) + t0 * p.ldv + (int64_t)h * p.dv + col;
    IO *o = static_cast<IO *>(p.out) + (t0 * p.Hv + h) * p.dv + col;
    ST *st = static_cast<ST *>(p.state) + ((slot * p.Hv + h) * DK + rg * R) * p.dv + col;

    f32x4 S[R];
#pragma unroll
    for (int m = 0; m < R; ++m) {
        if constexpr (sizeof(ST) == 4) {
            S[m] = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(st + m * p.dv));
        } else {
            const float4 x = IoTraits<ST>::load4(st + m * p.dv);
            S[m] = f32x4{x.x, x.y, x.z, x.w};
        }
    }
    Vals<IO, R> kn, qn;
    kn.load(k);
    qn.load(q);
    float4 vn = IoTraits<IO>::load4(v);
    float gn = load_gate1(p.g, t0 * p.Hv + h, p.gate_bf16), bn = load_gate1(p.beta, t0 * p.Hv + h, p.gate_bf16);
#pragma unroll 1
    for (int t = 0; t < len; ++t) {
        const Vals<IO, R> kc = kn, qc = qn;
        const float4 vc = vn;
        const float a = expf(gn), beta = bn;
        if (t + 1 < len) {
            k += p.ldk;
            q += p.ldq;
            v += p.ldv;
            kn.load(k);
            qn.load(q);
            vn = IoTraits<IO>::load4(v);
            const int64_t at = (t0 + t + 1) * p.Hv + h;
            gn = load_gate1(p.g, at, p.gate_bf16);
            bn = load_gate1(p.beta, at, p.gate_bf16);
        }
        f32x4 pk = zero4(), pq = zero4();
        float qk = 0.f;
#pragma unroll
        for (int m = 0; m < R; ++m) {
            const float km = kc[m], qm = qc[m];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                S[m][j] *= a;
                pk[j] = fmaf(km, S[m][j], pk[j]);
                pq[j] = fmaf(qm, S[m][j], pq[j]);
            }
            qk = fmaf(qm, km, qk);
        }
#pragma unroll
        for (int off = 8; off < 64; off <<= 1) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                pk[j] += __shfl_xor(pk[j], off);
                pq[j] += __shfl_xor(pq[j], off);
            }
            qk += __shfl_xor(qk, off);
        }
        const float vv[4] = {vc.x, vc.y, vc.z, vc.w};
        float u[4], y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u[j] = beta * (vv[j] - pk[j]);
            y[j] = p.scale * fmaf(qk, u[j], pq[j]);
        }
#pragma unroll
        for (int m = 0; m < R; ++m) {
            const float km = kc[m];
#pragma unroll
            for (int j = 0; j < 4; ++j) S[m][j] = fmaf(km, u[j], S[m][j]);
        }
        if (rg == 0) IoTraits<IO>::store4(o + (int64_t)t * p.Hv * p.dv, make_float4(y[0], y[1], y[2], y[3]));
    }
#pragma unroll
    for (int m = 0; m < R; ++m) {
        if constexpr (sizeof(ST) == 4) __builtin_nontemporal_store(S[m], reinterpret_cast<f32x4 *>(st + m * p.dv));
        else IoTraits<ST>::store4(st + m * p.dv, make_float4(S[m][0], S[m][1], S[m][2], S[m][3]));
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
