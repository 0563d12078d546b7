// Gated delta rule with one log-gate per token and value head: the kernel that walks a sequence's
// chunks.  Source of the method: Kimi Linear summary page, "From linear attention to Gated
// DeltaNet" (the scalar-gate delta rule) and "Chunkwise parallel algorithm".
//
// Mathematics, per (sequence, value head) and chunk of C tokens, G the in-chunk cumulative log gate,
// S the state entering the chunk, B = Diag(beta), Gam_ij = e^{G_i - G_j}:
//
//     M = strictly_lower(K K^T o Gam)           P = lower(Q K^T o Gam)
//     X = V - Diag(e^G) K S                     Z = (I + M B)^{-1} X        Y = B Z
//     O = scale (Diag(e^G) Q S + P Y)           S <- e^{G_C} S + K^T Diag(e^{G_C - G}) Y
//
// and backwards (dS the gradient of the state leaving the chunk):
//
//     dY = scale P^T dO + Diag(e^{G_C - G}) K dS        dX = (I + M B)^{-T} B dY = dV
//     dS <- e^{G_C} dS + scale Q^T Diag(e^G) dO - K^T Diag(e^G) dX
//
// A scalar gate leaves K and Q themselves as the operands of every product (its factors are row
// scalings of accumulators), so nothing has to be prepared per chunk in memory: one kernel stages
// K, Q and the value tile of a chunk in LDS and does everything else from there.  Beta multiplies
// columns of M, so no division by beta appears in the gradients and beta = 0 is exact.
//
// One workgroup owns (sequence, value head, CT state columns); three groups of waves run side by
// side, one chunk apart, with two barriers per chunk:
//   copy wave      global -> LDS loads of chunk s + 2, no registers in between;
//   producer waves chunk s + 1: K K^T and Q K^T (lower 16 x 16 tiles), the decays, then the inverse
//                  of every 32 x 32 diagonal block of I + M B (two 16 x 16 blocks by substitution,
//                  joined by two fp32 matrix products), and the gates of chunk s + 2;
//   chain waves    chunk s: 16 state columns each, the fp32 state in accumulator registers.
// The 64-token inverse is never formed: the second 32 tokens are solved after the first ones'
// result is subtracted (one more product on the chain, but two levels of block products and their
// roundings less per chunk).
//
// Roundings to bf16 (bf16 io only; fp32 io runs the same code on fp32 operands and 32-token
// chunks): the operands of the products that are not inputs (S, X, Z, Y, the strictly lower part of
// the inverse, M B and P).  The unit diagonal of the inverse is applied in fp32, sums and the state
// are fp32, cumulative gates fp64 (their differences stay exact behind a strong gate).
#pragma once

#include <type_traits>

#include "kda_device.h"
#include "kda_gdn.h"

namespace kda {
namespace gdn {

enum { kFwd = 0, kKeep = 1, kRev = 2 };

typedef __attribute__((ext_vector_type(4))) short s16x4;

// Two 16-wide k tiles of one operand (the pair an mma32 takes).
template <bool BF>
struct Frag2 {
    Frag<BF> a, b;
};
template <bool BF>
__device__ __forceinline__ void mma(f32x4 &acc, const Frag2<BF> &x, const Frag2<BF> &y) {
    mma32(acc, x.a, x.b, y.a, y.b);
}

// Position of index i (0..31) in a stored row of 32 contraction indices: a lane's eight values
// (4 q4 + j of both 16-wide tiles) sit next to each other.
__device__ __forceinline__ constexpr int kpos(int i) { return 8 * ((i >> 2) & 3) + 4 * (i >> 4) + (i & 3); }

// Rows of operand values in LDS, RB bytes each, 16-byte slots exchanged within a row so that 16 rows
// read at one slot spread over the 64 banks.
template <int RB>
__device__ __forceinline__ int slot_key(int row) {
    if constexpr (RB >= 256) return row & 15;
    else if constexpr (RB == 128) return (row >> 1) & 7;
    else return (row >> 2) & 3;
}
template <int RB>
__device__ __forceinline__ int row_off(int row, int byte) {
    return row * RB + ((((byte >> 4) ^ slot_key<RB>(row)) << 4) | (byte & 15));
}

// A lane's eight values at element offset e0 (a multiple of 8) of a row.
template <bool BF, int RB>
__device__ __forceinline__ Frag2<BF> row_frag(const char *base, int row, int e0) {
    Frag2<BF> f;
    if constexpr (BF) {
        const uint4 w = *reinterpret_cast<const uint4 *>(base + row_off<RB>(row, 2 * e0));
        f.a.v = make_uint2(w.x, w.y);
        f.b.v = make_uint2(w.z, w.w);
    } else {
        f.a.v = *reinterpret_cast<const float4 *>(base + row_off<RB>(row, 4 * e0));
        f.b.v = *reinterpret_cast<const float4 *>(base + row_off<RB>(row, 4 * e0 + 16));
    }
    return f;
}
// Four values stored at element offset e0 (a multiple of 4) of a row.
template <bool BF, int RB>
__device__ __forceinline__ void row_put4(char *base, int row, int e0, float a, float b, float c, float d) {
    const Frag<BF> f = make_frag<BF>(a, b, c, d);
    if constexpr (BF) *reinterpret_cast<uint2 *>(base + row_off<RB>(row, 2 * e0)) = f.v;
    else *reinterpret_cast<float4 *>(base + row_off<RB>(row, 4 * e0)) = f.v;
}
template <bool BF, int RB>
__device__ __forceinline__ void row_put1(char *base, int row, int e, float a) {
    if constexpr (BF) *reinterpret_cast<uint16_t *>(base + row_off<RB>(row, 2 * e)) = f32_to_bf16(a);
    else *reinterpret_cast<float *>(base + row_off<RB>(row, 4 * e)) = a;
}
// Four rows of 16 bf16 values, transposed: each group of 16 lanes reads a 4 x 16 block (lane l the four
// values of row l / 4, columns 4 (l % 4) .. + 3 at p) and receives column l, rows 0..3.
__device__ __forceinline__ Frag<true> read_tr4x16(const char *p) {
    Frag<true> f;
    const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)p);
    f.v = __builtin_bit_cast(uint2, v);
    return f;
}

// Channels of accumulator tile ct of a state: its row m is channel 32 (ct / 2) + 8 (m / 4) +
// 4 (ct % 2) + m % 4, so the tiles 2 t and 2 t + 1 of a lane are eight consecutive channels, the
// ones row_frag reads from a row of K or Q.
__device__ __forceinline__ int state_channel(int ct, int q4, int j) { return 32 * (ct >> 1) + 8 * q4 + 4 * (ct & 1) + j; }

// Transposed operand: rows are the channels of tile ct, contraction over the 32 tokens from 32 u.
template <bool BF, int RB>
__device__ __forceinline__ Frag2<BF> col_frag(const char *base, int ct, int u, int l16, int q4) {
    Frag2<BF> f;
    if constexpr (BF) {
        const int byte = 16 * (4 * (ct >> 1) + (l16 & 3)) + 8 * (ct & 1);
        const int r0 = 32 * u + 4 * q4 + (l16 >> 2);
        f.a = read_tr4x16(base + row_off<RB>(r0, byte));
        f.b = read_tr4x16(base + row_off<RB>(r0 + 16, byte));
    } else {
        const int byte = 4 * state_channel(ct, l16 >> 2, l16 & 3);
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = *reinterpret_cast<const float *>(base + row_off<RB>(32 * u + 16 * (j >> 2) + 4 * q4 + (j & 3), byte));
        f.a = make_frag<BF>(x[0], x[1], x[2], x[3]);
        f.b = make_frag<BF>(x[4], x[5], x[6], x[7]);
    }
    return f;
}

// LDS of one workgroup.
template <bool BF, int DK, int CT, int MODE>
struct Lds {
    static constexpr int E = BF ? 2 : 4;
    static constexpr int C = BF ? kChunkBf16 : kChunkF32;
    static constexpr int RT = C / 16, NBLK = C / 32, NCW = CT / 16;
    static constexpr int PW0 = NCW, CPW = NCW + 3;  // first producer wave, copy wave
    static constexpr int NT = 64 * (NCW + 4);
    static constexpr int RB = DK * E, VRB = CT * E, PRB = C * E, NRB = 32 * E;
    static constexpr int KB = C * RB, QB = MODE == kKeep ? 0 : KB, VB = C * VRB, SB = KB + QB + VB;
    static constexpr int NBUF = 3;
    static constexpr int LS = 36;  // row stride of the fp32 blocks (floats)
    static constexpr int P0 = NBUF * SB;
    static constexpr int PB = MODE == kKeep ? 0 : C * PRB;
    static constexpr int N0 = P0 + 2 * PB, NB = 32 * NRB;
    static constexpr int L0 = N0 + 2 * NBLK * NB, LB = NBLK > 1 ? NB : 0;
    static constexpr int F0 = L0 + 2 * LB, FB = 32 * LS * 4;
    static constexpr int G0 = F0 + NBLK * FB;             // G of one chunk, fp64, log2 units
    static constexpr int A0 = G0 + 8 * C, AB = 3 * C * 4 + 16;  // e^G, e^{G_C - G}, beta, e^{G_C}
    static constexpr int kBytes = A0 + 3 * AB;
    static_assert(kBytes <= 160 * 1024, "LDS of a CU");
};

// The sequence a workgroup works on.
struct Walk {
    int n, hk, h, col0, len, nch;
    int64_t tok0, slot0;
};

template <int C, int CT>
__device__ __forceinline__ Walk walk_of(const GdnParams &p) {
    Walk w;
    const int ntile = p.dv / CT, rep = p.Hv / p.Hk;
    // the tiles and the value heads that share a key head run next to each other on one XCD
    const SeqItem it = seq_item(blockIdx.x, p.num_seqs, p.Hk, rep * ntile, nullptr);
    w.n = it.n;
    w.hk = it.h;
    w.h = it.h * rep + it.tile / ntile;
    w.col0 = (it.tile % ntile) * CT;
    if (p.cu) {
        // offsets outside the tokens are cut off rather than followed
        const int a = min(max(p.cu[w.n], 0), p.T), b = min(max(p.cu[w.n + 1], a), p.T);
        w.tok0 = a;
        w.len = b - a;
        w.slot0 = slot_base(a, w.n, C);
    } else {
        w.tok0 = (int64_t)w.n * p.T;
        w.len = p.T;
        w.slot0 = (int64_t)w.n * ((p.T + C - 1) / C);
    }
    w.nch = (w.len + C - 1) / C;
    return w;
}

// Copy wave: chunk j's rows of K, Q and the value tile straight into LDS, 1 KB per instruction; rows past
// the end of the sequence re-read its last row (their beta is 0, so they change nothing).
template <bool BF, int DK, int CT, int MODE>
__device__ __forceinline__ void stage_chunk(const GdnParams &p, const Walk &w, int j, char *dst, int lane) {
    using L = Lds<BF, DK, CT, MODE>;
    const int clen = min(L::C, w.len - j * L::C);
    const int64_t t0 = w.tok0 + (int64_t)j * L::C;
    constexpr int SPR = L::RB / 16, VSPR = L::VRB / 16;
#pragma unroll 1
    for (int part = 0; part < (MODE == kKeep ? 1 : 2); ++part) {
        const char *src = static_cast<const char *>(part ? p.q : p.k) +
                          (t0 * (part ? p.ldq : p.ldk) + (int64_t)w.hk * DK) * L::E;
        const int64_t ld = (part ? p.ldq : p.ldk) * L::E;
#pragma unroll
        for (int i = 0; i < L::KB / 1024; ++i) {
            const int piece = 64 * i + lane, row = piece / SPR, slot = piece % SPR;
            load_lds16(src + min(row, clen - 1) * ld + ((slot ^ slot_key<L::RB>(row)) << 4), dst + part * L::KB + i * 1024);
        }
    }
    const char *src = static_cast<const char *>(p.v) + (t0 * p.ldv + (int64_t)w.h * p.dv + w.col0) * L::E;
#pragma unroll
    for (int i = 0; i < L::VB / 1024; ++i) {
        const int piece = 64 * i + lane, row = piece / VSPR;
        load_lds16(src + min(row, clen - 1) * p.ldv * L::E + (piece % VSPR) * 16, dst + L::KB + L::QB + i * 1024);
    }
}

// One producer's 16 x 16 tiles of row block r: the decayed K K^T (scaled by beta into M B) and Q K^T.
// Forward: rows of the stored matrices are the tokens i that are solved for; reverse: transposed.
template <bool BF, int DK, int CT, int MODE>
__device__ __forceinline__ void make_tiles(char *smem, int r, int buf, int par, int abuf, float scale, int l16, int q4) {
    using L = Lds<BF, DK, CT, MODE>;
    constexpr bool REV = MODE == kRev, HASQ = MODE != kKeep;
    const char *K = smem + buf * L::SB, *Q = K + L::KB;
    char *P = smem + L::P0 + par * L::PB;
    char *Lba = smem + L::L0 + par * L::LB;
    float *Lf = reinterpret_cast<float *>(smem + L::F0);
    const double *G = reinterpret_cast<const double *>(smem + L::G0);
    const float *beta = reinterpret_cast<const float *>(smem + L::A0 + abuf * L::AB) + 2 * L::C;
    Frag2<BF> kr[DK / 32], qr[DK / 32];
#pragma unroll
    for (int t = 0; t < DK / 32; ++t) {
        kr[t] = row_frag<BF, L::RB>(K, 16 * r + l16, 32 * t + 8 * q4);
        if constexpr (HASQ) qr[t] = row_frag<BF, L::RB>(Q, 16 * r + l16, 32 * t + 8 * q4);
    }
#pragma unroll 1
    for (int c = 0; c <= r; ++c) {
        f32x4 kk = zero4(), qk = zero4();
#pragma unroll
        for (int t = 0; t < DK / 32; ++t) {
            const Frag2<BF> kc = row_frag<BF, L::RB>(K, 16 * c + l16, 32 * t + 8 * q4);
            if constexpr (REV) {
                mma<BF>(kk, kr[t], kc);
                mma<BF>(qk, qr[t], kc);
            } else {
                mma<BF>(kk, kc, kr[t]);
                if constexpr (HASQ) mma<BF>(qk, kc, qr[t]);
            }
        }
        // a lane's entries: forward (i, j) = (16 r + l16, 16 c + 4 q4 + e), reverse (16 r + 4 q4 + e, 16 c + l16)
        const int own = REV ? 16 * c + l16 : 16 * r + l16, four = (REV ? 16 * r : 16 * c) + 4 * q4;
        const double Go = G[own];
        const float4 bf = *reinterpret_cast<const float4 *>(beta + four);
        const float bo = beta[own], b4[4] = {bf.x, bf.y, bf.z, bf.w};
        float m[4], pp[4];
        mfma_settle(kk, qk);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = REV ? four + e : own, jj = REV ? own : four + e;
            const double d = REV ? G[four + e] - Go : Go - G[four + e];
            const float gam = i >= jj ? fast_exp2((float)d) : 0.f;
            m[e] = i > jj ? kk[e] * gam * (REV ? bo : b4[e]) : 0.f;
            pp[e] = qk[e] * gam * (REV ? scale : 1.f);
        }
        if constexpr (HASQ) row_put4<BF, L::PRB>(P, own, (four & ~31) + kpos(four & 31), pp[0], pp[1], pp[2], pp[3]);
        if ((r >> 1) == (c >> 1)) {
            float *dst = Lf + (r >> 1) * 32 * L::LS;
            if constexpr (REV) {
#pragma unroll
                for (int e = 0; e < 4; ++e) dst[((four + e) & 31) * L::LS + (own & 31)] = m[e];
            } else {
                *reinterpret_cast<float4 *>(dst + (own & 31) * L::LS + (four & 31)) = make_float4(m[0], m[1], m[2], m[3]);
            }
        } else {
            row_put4<BF, L::NRB>(Lba, own & 31, kpos(four & 31), -m[0], -m[1], -m[2], -m[3]);
        }
    }
}

// The inverse of one 32 x 32 diagonal block of I + M B, minus the identity (reverse: transposed).
// Lane (sub, col) solves column col of the 16 x 16 diagonal block sub by forward substitution; the block
// below the diagonal is -N11 (L10 N00).
template <bool BF, int DK, int CT, int MODE>
__device__ __forceinline__ void invert_block(char *smem, int blk, int par, int lane) {
    using L = Lds<BF, DK, CT, MODE>;
    constexpr bool REV = MODE == kRev;
    const int l16 = lane & 15, q4 = lane >> 4, sub = q4 & 1;
    float *Lb = reinterpret_cast<float *>(smem + L::F0) + blk * 32 * L::LS;
    char *N = smem + L::N0 + (par * L::NBLK + blk) * L::NB;
    float x[16];
    const float *Ld = Lb + 16 * sub * L::LS + 16 * sub;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float s = i == l16 ? 1.f : 0.f;
#pragma unroll
        for (int j4 = 0; j4 < (i + 3) / 4; ++j4) {
            const float4 l4 = *reinterpret_cast<const float4 *>(Ld + i * L::LS + 4 * j4);
            const float lr[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * j4 + j < i) s = fmaf(-lr[j], x[4 * j4 + j], s);
        }
        x[i] = s;
    }
    wave_lds_sync();
    // columns of both inverses to LDS: block 0 into the unused upper right block, block 1 over the upper left
    // one, which has been read
    if (lane < 32) {
        float *dst = Lb + l16 * L::LS + (sub ? 0 : 16);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4 *>(dst + 4 * i) = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        if constexpr (REV) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = 4 * i + j == l16 ? 0.f : x[4 * i + j];
                row_put4<BF, L::NRB>(N, 16 * sub + l16, 8 * i + 4 * sub, y[0], y[1], y[2], y[3]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                row_put1<BF, L::NRB>(N, 16 * sub + i, kpos(16 * sub + l16), i == l16 ? 0.f : x[i]);
        }
    }
    wave_lds_sync();
    Frag<false> l10, n00, n11;
    l10.v = *reinterpret_cast<const float4 *>(Lb + (16 + l16) * L::LS + 4 * q4);
    n00.v = *reinterpret_cast<const float4 *>(Lb + l16 * L::LS + 16 + 4 * q4);
    const float *c11 = Lb + 4 * q4 * L::LS + l16;
    n11 = make_frag<false>(c11[0], c11[L::LS], c11[2 * L::LS], c11[3 * L::LS]);
    f32x4 t = zero4(), n10 = zero4();
    mma16(t, l10, n00);
    mfma_settle(t);
    mma16(n10, n11, frag_from_acc<false>(t, -1.f));
    mfma_settle(n10);
    if constexpr (REV) {
        row_put4<BF, L::NRB>(N, l16, kpos(16 + 4 * q4), n10[0], n10[1], n10[2], n10[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) row_put1<BF, L::NRB>(N, 16 + 4 * q4 + j, kpos(l16), n10[j]);
    }
    wave_lds_sync();
}

// One token's gate and beta (lane = token of the chunk), zero past the end.
struct RawGate {
    float g, b;
};
template <int C>
__device__ __forceinline__ RawGate load_gate(const GdnParams &p, const Walk &w, int j, int lane) {
    RawGate r{0.f, 0.f};
    const int t = j * C + lane;
    if (lane < C && t < w.len) {
        const int64_t at = (w.tok0 + t) * p.Hv + w.h;
        if (p.gate_bf16) {
            r.g = bf16_to_f32(static_cast<const uint16_t *>(p.g)[at]);
            r.b = bf16_to_f32(static_cast<const uint16_t *>(p.beta)[at]);
        } else {
            r.g = static_cast<const float *>(p.g)[at];
            r.b = static_cast<const float *>(p.beta)[at];
        }
    }
    return r;
}
// Cumulative gate of the chunk in fp64 (log2 units; a gate below -1e4 is as good as e^g = 0 and keeps the
// differences finite).
__device__ __forceinline__ double gate_scan(float g, int lane) {
    double s = (double)fmaxf(g, -1e4f) * 1.4426950408889634;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double o = __shfl_up(s, d);
        s += lane >= d ? o : 0.0;
    }
    return s;
}
template <bool BF, int DK, int CT, int MODE>
__device__ __forceinline__ void put_gates(char *smem, int abuf, const RawGate &r, int lane) {
    using L = Lds<BF, DK, CT, MODE>;
    const double s = gate_scan(r.g, lane), end = __shfl(s, L::C - 1);
    float *a = reinterpret_cast<float *>(smem + L::A0 + abuf * L::AB);
    if (lane < L::C) {
        reinterpret_cast<double *>(smem + L::G0)[lane] = s;
        a[lane] = fast_exp2((float)s);
        a[L::C + lane] = fast_exp2((float)(end - s));
        a[2 * L::C + lane] = r.b;
        if (lane == 0) a[3 * L::C] = fast_exp2((float)end);
    }
}

// Four consecutive tokens (16 rt + 4 q4 ..) of a wave's column l16 of the value tile.
template <bool BF, int VRB>
__device__ __forceinline__ Frag<BF> value_frag(const char *V, int wv, int rt, int l16, int q4) {
    if constexpr (BF) {
        return read_tr4x16(V + (16 * rt + 4 * q4 + (l16 >> 2)) * VRB + (16 * wv + 4 * (l16 & 3)) * 2);
    } else {
        const float *p = reinterpret_cast<const float *>(V + (16 * rt + 4 * q4) * VRB) + 16 * wv + l16;
        return make_frag<BF>(p[0], p[VRB / 4], p[2 * (VRB / 4)], p[3 * (VRB / 4)]);
    }
}
template <bool BF>
__device__ __forceinline__ f32x4 frag_f32(const Frag<BF> &f) {
    if constexpr (BF) return f32x4{bf16_lo(f.v.x), bf16_hi(f.v.x), bf16_lo(f.v.y), bf16_hi(f.v.y)};
    else return f32x4{f.v.x, f.v.y, f.v.z, f.v.w};
}
__device__ __forceinline__ f32x4 load_f4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }

// A wave's C x 16 result (accumulator layout, fp32) to rows of a [tokens, Hv, dv] tensor: through the wave's
// own columns of the value tile, which it has read, so that rows leave as 16-byte pieces.
template <bool BF, int VRB, int RT>
__device__ __forceinline__ void put_value_rows(char *V, void *dst, int64_t ld, int wv, const f32x4 (&x)[RT], int clen,
                                               int lane) {
    using IO = typename std::conditional<BF, uint16_t, float>::type;
    constexpr int E = sizeof(IO), SEG = 16 * E / 16;  // 16-byte pieces of a row of 16 columns
    const int l16 = lane & 15, q4 = lane >> 4;
    char *base = V + 16 * wv * E;
    wave_lds_sync();
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            IoTraits<IO>::store1(reinterpret_cast<IO *>(base + (16 * rt + 4 * q4 + j) * VRB) + l16, x[rt][j]);
    wave_lds_sync();
#pragma unroll
    for (int i = 0; i < 16 * RT * SEG / 64; ++i) {
        const int piece = 64 * i + lane, row = piece / SEG, s = piece % SEG;
        const u32x4 v = *reinterpret_cast<const u32x4 *>(base + row * VRB + s * 16);
        if (row < clen) *reinterpret_cast<u32x4 *>(static_cast<char *>(dst) + (row * ld + 16 * wv) * E + s * 16) = v;
    }
    wave_lds_sync();
}

template <bool BF, int DK, int CT, int MODE>
__global__ void __launch_bounds__((Lds<BF, DK, CT, MODE>::NT)) gdn_scan_kernel(GdnParams p) {
    using L = Lds<BF, DK, CT, MODE>;
    using IO = typename std::conditional<BF, uint16_t, float>::type;
    constexpr int C = L::C, RT = L::RT, KT = DK / 16, K2 = DK / 32;
    constexpr bool REV = MODE == kRev;
    __shared__ __attribute__((aligned(16))) char smem[L::kBytes];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, q4 = lane >> 4;
    const Walk w = walk_of<C, CT>(p);
    const int nch = w.nch;
    // step s works on chunk ci(s); the reverse scan walks from the last chunk to the first
    auto ci = [&](int s) { return REV ? nch - 1 - s : s; };

    if (nch > 0) {  // the tiles above the diagonal are read and never written
        for (int i = threadIdx.x * 16; i < L::F0 - L::P0; i += L::NT * 16)
            *reinterpret_cast<uint4 *>(smem + L::P0 + i) = make_uint4(0u, 0u, 0u, 0u);
    }

    if (wave == L::CPW) {
        // ------------------------------------------------------------------ copy wave
        if (nch == 0) return;
        auto stage = [&](int s) { stage_chunk<BF, DK, CT, MODE>(p, w, ci(s), smem + (s % L::NBUF) * L::SB, lane); };
        stage(0);
        if (nch > 1) stage(1);
        wait_vmcnt<0>();
        __syncthreads();  // chunk 0 (and 1) in LDS, gates of chunk 0
        __syncthreads();  // tiles of chunk 0
        __syncthreads();  // inverse of chunk 0, gates of chunk 1
        for (int s = 0; s < nch; ++s) {
            if (s + 2 < nch) stage(s + 2);
            __syncthreads();  // A
            wait_vmcnt<0>();
            __syncthreads();  // B
        }
        return;
    }
    if (wave >= L::PW0) {
        // ------------------------------------------------------------------ producer waves
        if (nch == 0) return;
        const int pw = wave - L::PW0;
        RawGate raw{0.f, 0.f};
        if (pw == 2) {
            raw = load_gate<C>(p, w, ci(0), lane);
            put_gates<BF, DK, CT, MODE>(smem, 0, raw, lane);
            if (nch > 1) raw = load_gate<C>(p, w, ci(1), lane);
        }
        auto tiles = [&](int s) {
            const int buf = s % L::NBUF, par = s & 1, ab = s % 3;
            if constexpr (RT == 4) {
                make_tiles<BF, DK, CT, MODE>(smem, pw == 0 ? 3 : pw == 1 ? 2 : 1, buf, par, ab, p.scale, l16, q4);
                if (pw == 2) make_tiles<BF, DK, CT, MODE>(smem, 0, buf, par, ab, p.scale, l16, q4);
            } else if (pw < 2) {
                make_tiles<BF, DK, CT, MODE>(smem, pw, buf, par, ab, p.scale, l16, q4);
            }
        };
        auto finish = [&](int s) {  // the inverse of chunk s, the gates of chunk s + 1
            if (pw < L::NBLK) invert_block<BF, DK, CT, MODE>(smem, pw, s & 1, lane);
            if (pw == 2 && s + 1 < nch) {
                put_gates<BF, DK, CT, MODE>(smem, (s + 1) % 3, raw, lane);
                if (s + 2 < nch) raw = load_gate<C>(p, w, ci(s + 2), lane);
            }
        };
        __syncthreads();
        tiles(0);
        __syncthreads();
        finish(0);
        __syncthreads();
        for (int s = 0; s < nch; ++s) {
            if (s + 1 < nch) tiles(s + 1);
            __syncthreads();  // A
            if (s + 1 < nch) finish(s + 1);
            __syncthreads();  // B
        }
        return;
    }

    // ------------------------------------------------------------------ chain waves
    const int col = w.col0 + 16 * wave + l16;
    const int64_t sbase = ((int64_t)w.n * p.Hv + w.h) * DK * p.dv + col;
    f32x4 S[KT];
#pragma unroll
    for (int ct = 0; ct < KT; ++ct)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t at = sbase + (int64_t)state_channel(ct, q4, j) * p.dv;
            S[ct][j] = !p.s0 ? 0.f
                       : p.state_bf16 ? bf16_to_f32(static_cast<const uint16_t *>(p.s0)[at])
                                      : static_cast<const float *>(p.s0)[at];
        }
    if (nch > 0) {
        __syncthreads();
        __syncthreads();
        __syncthreads();
    }
#pragma unroll 1
    for (int s = 0; s < nch; ++s) {
        const int c = ci(s), clen = min(C, w.len - c * C);
        const int64_t tok = w.tok0 + (int64_t)c * C;
        char *K = smem + (s % L::NBUF) * L::SB, *Q = K + L::KB, *V = K + L::KB + L::QB;
        const char *P = smem + L::P0 + (s & 1) * L::PB;
        const char *N = smem + L::N0 + (s & 1) * L::NBLK * L::NB, *Lba = smem + L::L0 + (s & 1) * L::LB;
        const float *eG = reinterpret_cast<const float *>(smem + L::A0 + (s % 3) * L::AB);
        const float *eB = eG + C, *beta = eG + 2 * C;
        const float eC = eG[3 * C];
        Frag2<BF> Sb[K2];
#pragma unroll
        for (int t = 0; t < K2; ++t) Sb[t] = {frag_from_acc<BF>(S[2 * t]), frag_from_acc<BF>(S[2 * t + 1])};
        if constexpr (MODE != kFwd) {
            // the state entering (reverse: the gradient of the state leaving) the chunk, [dv][d_k]
            IO *dst = static_cast<IO *>(p.hs) + (((w.slot0 + c) * p.Hv + w.h) * p.dv + col) * DK + 8 * q4;
#pragma unroll
            for (int t = 0; t < K2; ++t) {
                if constexpr (BF) {
                    *reinterpret_cast<uint4 *>(dst + 32 * t) =
                        make_uint4(Sb[t].a.v.x, Sb[t].a.v.y, Sb[t].b.v.x, Sb[t].b.v.y);
                } else {
                    *reinterpret_cast<float4 *>(dst + 32 * t) = Sb[t].a.v;
                    *reinterpret_cast<float4 *>(dst + 32 * t + 4) = Sb[t].b.v;
                }
            }
        }
        f32x4 x[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            x[rt] = zero4();
#pragma unroll
            for (int t = 0; t < K2; ++t) mma<BF>(x[rt], row_frag<BF, L::RB>(K, 16 * rt + l16, 32 * t + 8 * q4), Sb[t]);
        }
        Frag<BF> vf[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) vf[rt] = value_frag<BF, L::VRB>(V, wave, rt, l16, q4);

        if constexpr (!REV) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const f32x4 e = load_f4(eG + 16 * rt + 4 * q4), v = frag_f32<BF>(vf[rt]);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[rt][j] = fmaf(-e[j], x[rt][j], v[j]);
            }
            // Z, 32 tokens at a time
#pragma unroll
            for (int b = 0; b < L::NBLK; ++b) {
                if (b > 0) {
                    const Frag2<BF> za = {frag_from_acc<BF>(x[0]), frag_from_acc<BF>(x[1])};
#pragma unroll
                    for (int h = 0; h < 2; ++h) mma<BF>(x[2 + h], row_frag<BF, L::NRB>(Lba, 16 * h + l16, 8 * q4), za);
                }
                const Frag2<BF> xb = {frag_from_acc<BF>(x[2 * b]), frag_from_acc<BF>(x[2 * b + 1])};
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    mma<BF>(x[2 * b + h], row_frag<BF, L::NRB>(N + b * L::NB, 16 * h + l16, 8 * q4), xb);
            }
            __syncthreads();  // A
            Frag2<BF> yp[RT / 2], ys[RT / 2];
#pragma unroll
            for (int u = 0; u < RT / 2; ++u) {
                f32x4 a[2], d[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int rt = 2 * u + h;
                    const f32x4 bt = load_f4(beta + 16 * rt + 4 * q4), e = load_f4(eB + 16 * rt + 4 * q4);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        a[h][j] = bt[j] * x[rt][j];
                        d[h][j] = e[j] * a[h][j];
                    }
                }
                yp[u] = {frag_from_acc<BF>(a[0]), frag_from_acc<BF>(a[1])};
                ys[u] = {frag_from_acc<BF>(d[0]), frag_from_acc<BF>(d[1])};
            }
#pragma unroll
            for (int ct = 0; ct < KT; ++ct) {
#pragma unroll
                for (int j = 0; j < 4; ++j) S[ct][j] *= eC;
#pragma unroll
                for (int u = 0; u < RT / 2; ++u) mma<BF>(S[ct], col_frag<BF, L::RB>(K, ct, u, l16, q4), ys[u]);
            }
            if constexpr (MODE == kFwd) {
                // O^T tiles: a lane holds four consecutive columns of one token
                IO *out = static_cast<IO *>(p.out) + (tok * p.Hv + w.h) * p.dv + w.col0 + 16 * wave + 4 * q4;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    f32x4 o = zero4();
#pragma unroll
                    for (int t = 0; t < K2; ++t)
                        mma<BF>(o, Sb[t], row_frag<BF, L::RB>(Q, 16 * rt + l16, 32 * t + 8 * q4));
                    const float e = eG[16 * rt + l16];
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] *= e;
#pragma unroll
                    for (int u = 0; u <= rt / 2; ++u)
                        mma<BF>(o, yp[u], row_frag<BF, L::PRB>(P, 16 * rt + l16, 32 * u + 8 * q4));
                    mfma_settle(o);
                    if (16 * rt + l16 < clen)
                        IoTraits<IO>::store4(out + (int64_t)(16 * rt + l16) * p.Hv * p.dv,
                                             make_float4(o[0] * p.scale, o[1] * p.scale, o[2] * p.scale, o[3] * p.scale));
                }
            } else {
                put_value_rows<BF, L::VRB, RT>(V, static_cast<IO *>(p.zs) + (tok * p.Hv + w.h) * p.dv + w.col0,
                                               (int64_t)p.Hv * p.dv, wave, x, clen, lane);
            }
        } else {
            // rows past the end of the sequence were staged from its last row: no gradient there
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const f32x4 v = frag_f32<BF>(vf[rt]);
                f32x4 m;
#pragma unroll
                for (int j = 0; j < 4; ++j) m[j] = 16 * rt + 4 * q4 + j < clen ? v[j] : 0.f;
                vf[rt] = frag_from_acc<BF>(m);
            }
            // dY = Diag(e^{G_C - G}) K dS + scale P^T dO, times beta
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const f32x4 e = load_f4(eB + 16 * rt + 4 * q4), bt = load_f4(beta + 16 * rt + 4 * q4);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[rt][j] *= e[j];
#pragma unroll
                for (int u = rt / 2; u < RT / 2; ++u)
                    mma<BF>(x[rt], row_frag<BF, L::PRB>(P, 16 * rt + l16, 32 * u + 8 * q4), Frag2<BF>{vf[2 * u], vf[2 * u + 1]});
                mfma_settle(x[rt]);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[rt][j] *= bt[j];
            }
            // dX, the last 32 tokens first
#pragma unroll
            for (int b = L::NBLK - 1; b >= 0; --b) {
                if (b < L::NBLK - 1) {
                    const Frag2<BF> xb = {frag_from_acc<BF>(x[2 * b + 2]), frag_from_acc<BF>(x[2 * b + 3])};
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        mma<BF>(x[2 * b + h], row_frag<BF, L::NRB>(Lba, 16 * h + l16, 8 * q4), xb);
                }
                const Frag2<BF> zb = {frag_from_acc<BF>(x[2 * b]), frag_from_acc<BF>(x[2 * b + 1])};
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    mma<BF>(x[2 * b + h], row_frag<BF, L::NRB>(N + b * L::NB, 16 * h + l16, 8 * q4), zb);
            }
            __syncthreads();  // A
            Frag2<BF> dq[RT / 2], dx[RT / 2];
#pragma unroll
            for (int u = 0; u < RT / 2; ++u) {
                f32x4 a[2], d[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int rt = 2 * u + h;
                    const f32x4 e = load_f4(eG + 16 * rt + 4 * q4), v = frag_f32<BF>(vf[rt]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        a[h][j] = p.scale * e[j] * v[j];
                        d[h][j] = -e[j] * x[rt][j];
                    }
                }
                dq[u] = {frag_from_acc<BF>(a[0]), frag_from_acc<BF>(a[1])};
                dx[u] = {frag_from_acc<BF>(d[0]), frag_from_acc<BF>(d[1])};
            }
#pragma unroll
            for (int ct = 0; ct < KT; ++ct) {
#pragma unroll
                for (int j = 0; j < 4; ++j) S[ct][j] *= eC;
#pragma unroll
                for (int u = 0; u < RT / 2; ++u) {
                    mma<BF>(S[ct], col_frag<BF, L::RB>(Q, ct, u, l16, q4), dq[u]);
                    mma<BF>(S[ct], col_frag<BF, L::RB>(K, ct, u, l16, q4), dx[u]);
                }
            }
            put_value_rows<BF, L::VRB, RT>(V, static_cast<IO *>(p.out) + (tok * p.Hv + w.h) * p.dv + w.col0,
                                           (int64_t)p.Hv * p.dv, wave, x, clen, lane);
        }
#pragma unroll
        for (int ct = 0; ct < KT; ct += 2) mfma_settle(S[ct], S[ct + 1]);
        __syncthreads();  // B
    }
    if (p.sf) {
#pragma unroll
        for (int ct = 0; ct < KT; ++ct)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t at = sbase + (int64_t)state_channel(ct, q4, j) * p.dv;
                if (p.state_bf16) static_cast<uint16_t *>(p.sf)[at] = f32_to_bf16(S[ct][j]);
                else static_cast<float *>(p.sf)[at] = S[ct][j];
            }
    }
}

}  // namespace gdn
}  // namespace kda
