// Gated delta rule with one log-gate per token and value head: the gradients of a chunk, once the
// reverse scan has left dX (= dV) and the gradient dS of the state leaving every chunk, and the keeping
// forward the state S entering it and Z (notation of kda_gdn_scan.h).  Per chunk and value head, with
// W1 = dO Z^T, W2 = dX Z^T, E = scale W1 B o Gam (i >= j), F = -W2 B o Gam (i > j):
//
//     dQ = scale Diag(e^G) dO S^T + E K
//     dK = -Diag(e^G) dX S^T + Diag(beta e^{G_C - G}) Z dS^T + E^T Q + (F + F^T) K
//     t_ij = Gam_ij (scale (Q K^T)_ij W1_ij - (K K^T)_ij W2_ij),   x_i = e^{G_C - G_i} k_i . (dS Z_i)
//     dbeta_j = sum_{i > j} t_ij + scale (q_j . k_j) W1_jj + x_j = W2_jj / beta_j
//     dG_i = sum_{j < i} beta_j t_ij - beta_i sum_{j > i} t_ji + q_i . dQ(state part)_i + k_i . dK(S part)_i - beta_i x_i
//     dG_C += sum_i beta_i x_i + e^{G_C} <S, dS>,   dg = reverse cumulative sum of dG over the chunk
//
// dX_j is beta_j times a vector, so the quotient has no cancellation where the sums have (repeated keys: error
// of dbeta 7e-2 of its norm by the sums, 3e-2 so).  The sums serve |beta| < 2^-64, so every beta has its
// gradient: there dX nears the smallest normal number, where it loses its bits (beta = 1e-38: dbeta half off)
// or is 0.  Repeated keys cancel only as far as beta is near 1.  The diagonal, where the gate cancels, is left
// out of dG rather than added and subtracted.
//
// One workgroup owns (chunk, key head) and walks the value heads that share it, so that dQ and dK are
// summed over them in registers, in a fixed order.  Two waves own the 16 tokens of row tile r, one
// half of the channels each: dO, dX and Z rows are operand fragments read straight from memory, dQ^T
// and dK^T stay in accumulators (lane = token, so the gates are lane scalars and 8 consecutive channels
// leave as 16 bytes).  S, dS, then Z with E and F + F^T take turns in one 32 KB LDS buffer beside K and Q.
//
// Roundings to bf16 (bf16 io only): what the scans leave (S, dS, Z, dX) and E and F + F^T, each once, as operands;
// W1, W2, the sums and the gates' gradients are fp32.  Each adds about as much, in squares, as the outputs' own rounding
// (error of the gradients 2.4 to 4.0e-3 of their norm, 1.7e-3 of it their own).  A second term of Z, dX, E and F
// would double these products and want operand registers that the kernel has not left.
//
// Measured, 4 x 4,096 tokens x 16 heads, d = 128, bf16: 245 us, 0.76 GB of HBM traffic, so 3.1 TB/s, the waves
// waiting 61 % of their time and the matrix units busy 8 %: bound by the latency of a workgroup's chain of
// loads, products and barriers (16 us), with one workgroup of 8 waves per CU at 256 registers.  Four waves with
// all channels each spilled (356 us); two workgroups per CU at 128 registers spill too (430 to 570 us); dO and
// dX loaded twice instead of kept 277 us; dS and Z loaded ahead at the start 255 us.
#pragma once

#include "kda_gdn_scan.h"

namespace kda {
namespace gdn {

// Rows as row_off lays them out, the slots of rows 16 apart exchanged too: the four groups of 4 rows, 8
// apart, of a transposed read then meet 4 deep instead of 8 in the banks.  (Not in the scan, whose
// addresses differ by constants from row tile to row tile only without it.)
template <int RB>
__device__ __forceinline__ int mix_off(int row, int byte) {
    return RB >= 256 ? row_off<RB>(row, byte) ^ (row >> 4 & 3) << 6 : row_off<RB>(row, byte);
}
template <bool BF, int RB>
__device__ __forceinline__ Frag2<BF> mix_frag(const char *base, int row, int e0) {
    Frag2<BF> f;
    if constexpr (BF) {
        const uint4 w = *reinterpret_cast<const uint4 *>(base + mix_off<RB>(row, 2 * e0));
        f.a.v = make_uint2(w.x, w.y);
        f.b.v = make_uint2(w.z, w.w);
    } else {
        f.a.v = *reinterpret_cast<const float4 *>(base + mix_off<RB>(row, 4 * e0));
        f.b.v = *reinterpret_cast<const float4 *>(base + mix_off<RB>(row, 4 * e0 + 16));
    }
    return f;
}

// As col_frag, the contraction over 8 consecutive rows per lane: 32 u + 8 q4 ..
template <bool BF, int RB>
__device__ __forceinline__ Frag2<BF> col_frag8(const char *base, int ct, int u, int l16, int q4) {
    Frag2<BF> f;
    if constexpr (BF) {
        const int byte = 16 * (4 * (ct >> 1) + (l16 & 3)) + 8 * (ct & 1);
        const int r0 = 32 * u + 8 * q4 + (l16 >> 2);
        f.a = read_tr4x16(base + mix_off<RB>(r0, byte));
        f.b = read_tr4x16(base + mix_off<RB>(r0 + 4, byte));
    } else {
        const int byte = 4 * state_channel(ct, l16 >> 2, l16 & 3);
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = *reinterpret_cast<const float *>(base + mix_off<RB>(32 * u + 8 * q4 + j, byte));
        f.a = make_frag<BF>(x[0], x[1], x[2], x[3]);
        f.b = make_frag<BF>(x[4], x[5], x[6], x[7]);
    }
    return f;
}
// Column 16 c + l16 of a stored [rows][cols] matrix, rows 32 u + 8 q4 ..
template <bool BF, int RB>
__device__ __forceinline__ Frag2<BF> plain_col_frag8(const char *base, int c, int u, int l16, int q4) {
    Frag2<BF> f;
    const int r0 = 32 * u + 8 * q4;
    if constexpr (BF) {
        const int byte = 2 * (16 * c + 4 * (l16 & 3));
        f.a = read_tr4x16(base + mix_off<RB>(r0 + (l16 >> 2), byte));
        f.b = read_tr4x16(base + mix_off<RB>(r0 + 4 + (l16 >> 2), byte));
    } else {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = *reinterpret_cast<const float *>(base + mix_off<RB>(r0 + j, 4 * (16 * c + l16)));
        f.a = make_frag<BF>(x[0], x[1], x[2], x[3]);
        f.b = make_frag<BF>(x[4], x[5], x[6], x[7]);
    }
    return f;
}
// Eight consecutive values of a row in memory (zero for a row past the end).
template <bool BF>
__device__ __forceinline__ Frag2<BF> mem_frag(const void *p, int64_t at, bool valid) {
    Frag2<BF> f;
    if constexpr (BF) {
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (valid) w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at);
        f.a.v = make_uint2(w.x, w.y);
        f.b.v = make_uint2(w.z, w.w);
    } else {
        f.a.v = f.b.v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (valid) {
            f.a.v = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
            f.b.v = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at + 4);
        }
    }
    return f;
}
// The same fragment to a row in LDS.
template <bool BF, int RB>
__device__ __forceinline__ void row_put_frag(char *base, int row, int e0, const Frag2<BF> &f) {
    if constexpr (BF) {
        *reinterpret_cast<uint4 *>(base + mix_off<RB>(row, 2 * e0)) = make_uint4(f.a.v.x, f.a.v.y, f.b.v.x, f.b.v.y);
    } else {
        *reinterpret_cast<float4 *>(base + mix_off<RB>(row, 4 * e0)) = f.a.v;
        *reinterpret_cast<float4 *>(base + mix_off<RB>(row, 4 * e0 + 16)) = f.b.v;
    }
}
// Eight consecutive fp32 values to memory.
template <bool BF, typename IO>
__device__ __forceinline__ void put_row8(IO *p, const f32x4 &a, const f32x4 &b) {
    if constexpr (BF) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                                   pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3]));
    } else {
        *reinterpret_cast<f32x4 *>(p) = a;
        *reinterpret_cast<f32x4 *>(p + 4) = b;
    }
}
__device__ __forceinline__ float dot4(const f32x4 &x, const f32x4 &y, float s) {
#pragma unroll
    for (int j = 0; j < 4; ++j) s = fmaf(x[j], y[j], s);
    return s;
}
template <bool BF>
__device__ __forceinline__ float dot16(const u32x4 &x, const u32x4 &y, float s) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (BF) {
            s = fmaf(bf16_lo(x[j]), bf16_lo(y[j]), s);
            s = fmaf(bf16_hi(x[j]), bf16_hi(y[j]), s);
        } else {
            s = fmaf(__uint_as_float(x[j]), __uint_as_float(y[j]), s);
        }
    }
    return s;
}

template <bool BF, int DK, int DV>
struct GradLds {
    static constexpr int E = BF ? 2 : 4, C = BF ? kChunkBf16 : kChunkF32, RT = C / 16, NT = 128 * RT;
    static constexpr int RB = DK * E, ZRB = DV * E, MRB = C * E;
    static constexpr int KB = C * RB, SB = DV * RB, ZB = C * ZRB, MB = C * MRB;
    static constexpr int B0 = 2 * KB, BB = SB > ZB + 2 * MB ? SB : ZB + 2 * MB;
    static constexpr int G0 = B0 + BB;                     // up, down, beta, hi, lo [C]; 12 block factors, resets
    static constexpr int T0 = G0 + 5 * C * 4 + 64;         // column sums [RT][C]
    static constexpr int V0 = T0 + RT * C * 4;             // row terms and x, per channel half, and two diagonals [C]
    static constexpr int D0 = V0 + 6 * C * 4;              // <S, dS> per wave
    static constexpr int kBytes = D0 + 2 * RT * 4;
};

template <bool BF, int DK, int DV>
__global__ void __launch_bounds__((GradLds<BF, DK, DV>::NT), (BF ? 2 : 1)) gdn_grad_kernel(GradParams gp) {
    using L = GradLds<BF, DK, DV>;
    using IO = typename std::conditional<BF, uint16_t, float>::type;
    constexpr int C = L::C, RT = L::RT, K2 = DK / 32, V2 = DV / 32, T2 = K2 / 2;
    __shared__ __attribute__((aligned(16))) char smem[L::kBytes];
    const GdnParams &p = gp.f;
    int tid = threadIdx.x;
    // wave: row tile r, half hf of the channels
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = wave >> 1, hf = wave & 1;
    int l16 = lane & 15, q4 = lane >> 4;
    // the chunk of this slot
    const int64_t slot = blockIdx.x / p.Hk;
    const int hk = (int)(blockIdx.x % p.Hk), rep = p.Hv / p.Hk;
    int64_t tok;
    int clen;
    if (p.cu) {
        // last sequence whose first slot is not behind this one
        int lo = 0, hi = p.num_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (slot_base(min(max(p.cu[mid], 0), p.T), mid, C) <= slot) lo = mid;
            else hi = mid - 1;
        }
        const int a = min(max(p.cu[lo], 0), p.T), b = min(max(p.cu[lo + 1], a), p.T);
        const int64_t c = slot - slot_base(a, lo, C);
        if (c < 0 || c * C >= b - a) return;
        tok = a + c * C;
        clen = (int)min((int64_t)C, b - tok);
    } else {
        const int nch = (p.T + C - 1) / C;
        const int c = (int)(slot % nch);
        tok = slot / nch * p.T + (int64_t)c * C;
        clen = min(C, p.T - c * C);
    }
    char *K = smem, *Q = smem + L::KB, *buf = smem + L::B0;
    char *E1 = buf + L::ZB, *H = E1 + L::MB;
    float *gate = reinterpret_cast<float *>(smem + L::G0), *fac = gate + 5 * C;
    float *colsum = reinterpret_cast<float *>(smem + L::T0);
    float *rowv = reinterpret_cast<float *>(smem + L::V0), *xv = rowv + 2 * C, *diag = xv + 2 * C, *dxz = diag + C;
    float *sds = reinterpret_cast<float *>(smem + L::D0);

    {
        const int row = 16 * r + l16;
        const bool valid = row < clen;
#pragma unroll
        for (int t = 0; t < T2; ++t) {
            const int e0 = 32 * (T2 * hf + t) + 8 * q4;
            row_put_frag<BF, L::RB>(K, row, e0, mem_frag<BF>(p.k, (tok + row) * p.ldk + hk * DK + e0, valid));
            row_put_frag<BF, L::RB>(Q, row, e0, mem_frag<BF>(p.q, (tok + row) * p.ldq + hk * DK + e0, valid));
        }
    }
    f32x4 dq[2 * T2], dk[2 * T2];
#pragma unroll
    for (int i = 0; i < 2 * T2; ++i) dq[i] = dk[i] = zero4();
    // loops over the channel tiles end here, so that the operands of one tile are loaded at a time
    auto tile_end = [] { __builtin_amdgcn_sched_barrier(0); };

#pragma unroll 1
    for (int g = 0; g < rep; ++g) {
        const int h = hk * rep + g;
        // addresses are formed anew for every head rather than kept in (or spilled from) registers
        asm volatile("" : "+v"(l16), "+v"(q4), "+v"(tid));
        const int row = 16 * r + l16;
        const bool valid = row < clen;
        const int64_t vrow = ((tok + row) * p.Hv + h) * DV;
        Frag2<BF> dof[V2], dxf[V2], zf[V2];
#pragma unroll
        for (int u = 0; u < V2; ++u) {
            dof[u] = mem_frag<BF>(p.v, vrow + 32 * u + 8 * q4, valid);
            dxf[u] = mem_frag<BF>(gp.dx, vrow + 32 * u + 8 * q4, valid);
        }
        constexpr int NP = L::SB / 16 / L::NT;
        const int64_t sat = (slot * p.Hv + h) * (int64_t)L::SB;
        const u32x4 *sp = reinterpret_cast<const u32x4 *>(static_cast<const char *>(gp.hs) + sat);
        const u32x4 *dp = reinterpret_cast<const u32x4 *>(static_cast<const char *>(gp.dhs) + sat);
        auto state_at = [&](int i) {
            const int piece = i * L::NT + tid;
            return reinterpret_cast<u32x4 *>(buf + mix_off<L::RB>(piece / (L::RB / 16), piece % (L::RB / 16) * 16));
        };
        {
            u32x4 sv[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i) sv[i] = sp[i * L::NT + tid];
            if (g > 0) __syncthreads();  // the last head's reads of the buffer
#pragma unroll
            for (int i = 0; i < NP; ++i) *state_at(i) = sv[i];
        }
        if (wave == 0) {
            Walk w;
            w.tok0 = tok;
            w.len = clen;
            w.h = h;
            const RawGate raw = load_gate<C>(p, w, 0, lane);
            const Gates gt = make_gates<C>(raw, lane);
            const uint64_t resets = __ballot(raw.g <= kNoGate);
            if (lane < C) {
                gate[lane] = gt.up;
                gate[C + lane] = gt.down;
                gate[2 * C + lane] = gt.beta;
                gate[3 * C + lane] = gt.hi;
                gate[4 * C + lane] = gt.lo;
                if ((lane & 15) == 0) {
                    fac[lane >> 4] = gt.f[0];
                    fac[4 + (lane >> 4)] = gt.f[1];
                }
                if (lane == 0) {
#pragma unroll
                    for (int i = 2; i < 6; ++i) fac[6 + i] = gt.f[i];
                    *reinterpret_cast<uint64_t *>(fac + 12) = resets;
                }
            }
        }
        __syncthreads();
        const float up = gate[row], bet = gate[2 * C + row];
        const float eG = up * fac[r], eB = gate[C + row] * fac[4 + r];
        // the parts through the state entering the chunk
        float rowsum = 0.f, xk = 0.f;
#pragma unroll
        for (int t = 0; t < T2; ++t) {
            const int e0 = 32 * (T2 * hf + t) + 8 * q4;
            const Frag2<BF> kr = mix_frag<BF, L::RB>(K, row, e0), qr = mix_frag<BF, L::RB>(Q, row, e0);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f32x4 r1 = zero4(), r2 = zero4();
#pragma unroll
                for (int u = 0; u < V2; ++u) {
                    const Frag2<BF> a = col_frag8<BF, L::RB>(buf, 2 * (T2 * hf + t) + i, u, l16, q4);
                    mma<BF>(r1, a, dof[u]);
                    mma<BF>(r2, a, dxf[u]);
                }
                r1 = r1 * (eG * p.scale);
                r2 = r2 * -eG;
                rowsum = dot4(frag_f32<BF>(i ? qr.b : qr.a), r1, rowsum);
                rowsum = dot4(frag_f32<BF>(i ? kr.b : kr.a), r2, rowsum);
                dq[2 * t + i] = dq[2 * t + i] + r1;
                dk[2 * t + i] = dk[2 * t + i] + r2;
                tile_end();
            }
        }
        // dS takes the place of S; a thread stores where it stored before and meets its pieces of S there
        float ss = 0.f;
        {
            u32x4 dv[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i) dv[i] = dp[i * L::NT + tid];
#pragma unroll
            for (int u = 0; u < V2; ++u) zf[u] = mem_frag<BF>(gp.zs, vrow + 32 * u + 8 * q4, valid);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                u32x4 *at = state_at(i);
                ss = dot16<BF>(*at, dv[i], ss);
                *at = dv[i];
            }
        }
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) ss += __shfl_xor(ss, off);
        if (lane == 0) sds[wave] = ss;
        __syncthreads();
        // the part through the state leaving it
#pragma unroll
        for (int t = 0; t < T2; ++t) {
            const Frag2<BF> kr = mix_frag<BF, L::RB>(K, row, 32 * (T2 * hf + t) + 8 * q4);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f32x4 r3 = zero4();
#pragma unroll
                for (int u = 0; u < V2; ++u)
                    mma<BF>(r3, col_frag8<BF, L::RB>(buf, 2 * (T2 * hf + t) + i, u, l16, q4), zf[u]);
                r3 = r3 * eB;
                xk = dot4(frag_f32<BF>(i ? kr.b : kr.a), r3, xk);
                dk[2 * t + i] = dk[2 * t + i] + r3 * bet;
                tile_end();
            }
        }
        __syncthreads();
        // inside the chunk: Z to LDS, then the 16 x 16 tiles of row tile r, shared between its two waves
#pragma unroll
        for (int u = 0; u < V2; ++u)
            if ((u & 1) == hf) row_put_frag<BF, L::ZRB>(buf, row, 32 * u + 8 * q4, zf[u]);
        __syncthreads();
#pragma unroll 1
        for (int c = hf; c <= r; c += 2) {
            f32x4 kk = zero4(), qk = zero4(), w1 = zero4(), w2 = zero4();
#pragma unroll
            for (int t = 0; t < K2; ++t) {
                const Frag2<BF> kc = mix_frag<BF, L::RB>(K, 16 * c + l16, 32 * t + 8 * q4);
                mma<BF>(kk, kc, mix_frag<BF, L::RB>(K, row, 32 * t + 8 * q4));
                mma<BF>(qk, kc, mix_frag<BF, L::RB>(Q, row, 32 * t + 8 * q4));
            }
            tile_end();
#pragma unroll
            for (int u = 0; u < V2; ++u) {
                const Frag2<BF> zc = mix_frag<BF, L::ZRB>(buf, 16 * c + l16, 32 * u + 8 * q4);
                mma<BF>(w1, zc, dof[u]);
                mma<BF>(w2, zc, dxf[u]);
            }
            const int j0 = 16 * c + 4 * q4;
            f32x4 gam;
            if (c == r) {
                const f32x4 h4 = load_f4(gate + 3 * C + j0), l4 = load_f4(gate + 4 * C + j0);
                const float ho = gate[3 * C + row], lo = gate[4 * C + row];
#pragma unroll
                for (int e = 0; e < 4; ++e) gam[e] = row >= j0 + e ? fast_exp2((ho - h4[e]) + (lo - l4[e])) : 0.f;
            } else {
                const float f = r - c == 1 ? 1.f : fac[8 + (r - c == 3 ? 2 : c)];
                gam = load_f4(gate + C + j0) * (up * f);
            }
            const f32x4 b4 = load_f4(gate + 2 * C + j0);
            mfma_settle(kk, qk);
            mfma_settle(w1, w2);
            f32x4 e1, f1, t;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float a = p.scale * w1[e] * gam[e], b = -w2[e] * gam[e];
                const bool strict = c < r || row > j0 + e;
                e1[e] = a * b4[e];
                f1[e] = strict ? b * b4[e] : 0.f;
                t[e] = qk[e] * a;
                if (c == r && row == j0 + e) {
                    diag[row] = t[e];
                    dxz[row] = w2[e];
                }
                t[e] = strict ? fmaf(kk[e], b, t[e]) : 0.f;
                rowsum = fmaf(b4[e], t[e], rowsum);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) t[e] = scan16_add(t[e]);  // over the tile's rows: the last of 16 lanes has it
            if (l16 == 15) *reinterpret_cast<f32x4 *>(colsum + r * C + j0) = t;
            row_put4<BF, L::MRB>(E1, row, j0, e1[0], e1[1], e1[2], e1[3]);
            row_put4<BF, L::MRB>(H, row, j0, f1[0], f1[1], f1[2], f1[3]);
            wave_lds_sync();
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c < r || row > j0 + e) row_put1<BF, L::MRB>(H, j0 + e, row, f1[e]);
            wave_lds_sync();
        }
        if ((r & 1) == 0 && hf == 0) row_put4<BF, L::MRB>(E1, row, 16 * (r + 1) + 4 * q4, 0.f, 0.f, 0.f, 0.f);
        rowsum += __shfl_xor(rowsum, 16);
        rowsum += __shfl_xor(rowsum, 32);
        xk += __shfl_xor(xk, 16);
        xk += __shfl_xor(xk, 32);
        if (q4 == 0) {
            rowv[hf * C + row] = rowsum;
            xv[hf * C + row] = xk;
        }
        __syncthreads();
        Frag2<BF> er[RT / 2], hr[RT / 2], ec[RT / 2];
#pragma unroll
        for (int u = 0; u < RT / 2; ++u) {
            er[u] = row_frag<BF, L::MRB>(E1, row, 32 * u + 8 * q4);
            hr[u] = row_frag<BF, L::MRB>(H, row, 32 * u + 8 * q4);
            ec[u] = plain_col_frag8<BF, L::MRB>(E1, r, u, l16, q4);
        }
        // row tiles of the first 32 tokens need E's columns there, those of the second its rows there
        auto products = [&](auto second) {
            constexpr int R2 = decltype(second)::value;
#pragma unroll
            for (int i = 0; i < 2 * T2; ++i) {
                const int ct = 2 * T2 * hf + i;
#pragma unroll
                for (int u = 0; u < RT / 2; ++u) {
                    const Frag2<BF> kt = col_frag8<BF, L::RB>(K, ct, u, l16, q4);
                    if (u <= R2) mma<BF>(dq[i], kt, er[u]);
                    mma<BF>(dk[i], kt, hr[u]);
                    if (u >= R2) mma<BF>(dk[i], col_frag8<BF, L::RB>(Q, ct, u, l16, q4), ec[u]);
                }
                tile_end();
            }
        };
        if (RT > 2 && r >= 2) products(std::integral_constant<int, 1>{});
        else products(std::integral_constant<int, 0>{});
#pragma unroll
        for (int i = 0; i < 2 * T2; ++i) mfma_settle(dq[i], dk[i]);
        if (wave == 0) {
            // gates' gradients, lane = token
            float dG = 0.f, db = 0.f, bx = 0.f;
            if (lane < C) {
                float cs = 0.f;
                for (int rr = lane >> 4; rr < RT; ++rr) cs += colsum[rr * C + lane];
                const float b = gate[2 * C + lane], x = xv[lane] + xv[C + lane];
                db = fabsf(b) < 0x1p-64f ? cs + diag[lane] + x : dxz[lane] / b;
                bx = b * x;
                dG = rowv[lane] + rowv[C + lane] - b * cs - bx;
            }
            float end = bx;
#pragma unroll
            for (int off = 32; off >= 1; off >>= 1) end += __shfl_xor(end, off);
            float sd = 0.f;
            for (int i = 0; i < 2 * RT; ++i) sd += sds[i];
            if (lane == C - 1) dG += fmaf(fac[11], sd, end);
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const float o = __shfl_down(dG, off);
                dG += lane + off < 64 ? o : 0.f;
            }
            // at a gate that is as good as e^g = 0 the sum cancels: 0 rather than what is left of it (a NaN stays)
            if (*reinterpret_cast<const uint64_t *>(fac + 12) >> lane & 1) dG *= 0.f;
            if (lane < clen) {
                const int64_t at = (tok + lane) * p.Hv + h;
                if (p.gate_bf16) {
                    static_cast<uint16_t *>(gp.dg)[at] = f32_to_bf16(dG);
                    static_cast<uint16_t *>(gp.dbeta)[at] = f32_to_bf16(db);
                } else {
                    static_cast<float *>(gp.dg)[at] = dG;
                    static_cast<float *>(gp.dbeta)[at] = db;
                }
            }
        }
    }
    const int row = 16 * r + l16;
    if (row < clen) {
        const int64_t at = ((tok + row) * p.Hk + hk) * DK + 32 * T2 * hf + 8 * q4;
        IO *oq = static_cast<IO *>(gp.dq) + at, *ok = static_cast<IO *>(gp.dk) + at;
#pragma unroll
        for (int t = 0; t < T2; ++t) {
            put_row8<BF>(oq + 32 * t, dq[2 * t], dq[2 * t + 1]);
            put_row8<BF>(ok + 32 * t, dk[2 * t], dk[2 * t + 1]);
        }
    }
}

template <bool BF>
hipError_t launch_grad(const GradParams &gp, hipStream_t stream) {
    const GdnParams &p = gp.f;
    const int64_t blocks = gp.slots * p.Hk;
    if (blocks <= 0) return hipSuccess;
#define GDN_GRAD(DK_, DV_)                                                                              \
    if (p.dk == DK_ && p.dv == DV_) {                                                                   \
        hipLaunchKernelGGL((gdn_grad_kernel<BF, DK_, DV_>), dim3((unsigned)blocks),                     \
                           dim3((GradLds<BF, DK_, DV_>::NT)), 0, stream, gp);                           \
        return hipGetLastError();                                                                       \
    }
    GDN_GRAD(64, 64)
    GDN_GRAD(64, 128)
    GDN_GRAD(128, 64)
    GDN_GRAD(128, 128)
#undef GDN_GRAD
    return hipErrorInvalidConfiguration;
}

}  // namespace gdn
}  // namespace kda
