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
// columns of M, so that nothing here is divided by beta and beta = 0 is exact.
//
// One workgroup owns (sequence, value head, CT state columns); groups of waves run side by side, up to
// two chunks apart, with two barriers per chunk:
//   copy wave     global -> LDS loads of chunk s + 2, no registers in between;
//   block waves   chunk s + 1: the lower 16 x 16 tiles of K K^T and Q K^T with their decays, the inverse
//                 of every 32 x 32 diagonal block of I + M B (two 16 x 16 blocks by substitution, joined
//                 by two fp32 matrix products), and the gates of chunk s + 2;
//   chain waves   chunk s: 16 state columns each, the fp32 state in accumulator registers;
//   output        chunk s (forward): O from the state and Y that the chain wave of the same columns hands
//                 over in LDS at the step's middle barrier, by the waves that made Q K^T before it.
// The 64-token inverse is never formed: the second 32 tokens are solved after the first ones'
// result is subtracted (one more product on the chain, but two levels of block products and their
// roundings less per chunk).
//
// Roundings to bf16 (bf16 io only; fp32 io runs the same code on fp32 operands and 32-token chunks): the
// operands of the products that are not inputs (S, X, Z, Y, the strictly lower part of the inverse,
// M B and P).  The forward takes P and Y as two bf16 terms in P Y, a product of waves that have the time:
// error of the output 1.8e-3 of its norm with ordinary decays, 1.7e-3 of it the output's own rounding, where one
// term gives 2.9e-3, in the same time; up to 2.6e-3 with long memories, whose state is rounded as an operand
// in every chunk.  X, Z and K^T Y with two terms as well would cost the chain 0.3 us a chunk for what is then
// 1.7e-3 with ordinary decays.  The unit diagonal of the inverse is applied in fp32, sums and the state
// are fp32, cumulative gates fp64 (their differences stay exact behind a strong gate).
//
// Registers: every mode at d_k = 128 is near the 256 that eight waves leave a lane (bf16 forward 252, reverse 251),
// and two are over: the keeping forward in bf16 and the reverse walk in fp32 keep 12 bytes a lane in scratch.
#pragma once

#include <type_traits>

#include "kda_device.h"
#include "kda_gdn.h"

namespace kda {
namespace gdn {

__device__ __forceinline__ f32x4 load_f4(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }

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

// The rounding error of a bf16 operand, as an operand: hi + lo has 16 bits of each value.
__device__ __forceinline__ Frag<true> frag_lo(const f32x4 &x, const Frag<true> &hi) {
    return make_frag<true>(x[0] - bf16_lo(hi.v.x), x[1] - bf16_hi(hi.v.x), x[2] - bf16_lo(hi.v.y), x[3] - bf16_hi(hi.v.y));
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
    static constexpr int RT = C / 16, NBLK = C / 32;
    // Waves (wave i runs on SIMD i % 4, so that a chain wave shares its SIMD with an output wave, whose main work
    // falls into the other phase): 0, 1 chain; 2, 3 the diagonal blocks of K K^T and their inverses; 4, 5 the blocks
    // of Q K^T, then the output; 6 the block below the diagonal, and the gates; 7 copies.
    static constexpr int NCW = 2, KW0 = 2, QW0 = 4, GW = 6, CPW = 7, NT = 512;
    static constexpr int NOW = MODE == kFwd ? NCW : 0;
    static_assert(CT == 16 * NCW, "a chain wave owns 16 columns");
    static constexpr int RB = DK * E, VRB = CT * E, PRB = C * E, NRB = 32 * E;
    static constexpr int KB = C * RB, QB = MODE == kKeep ? 0 : KB, VB = C * VRB, SB = KB + QB + VB;
    static constexpr int NBUF = 3;
    static constexpr int LS = 36;  // row stride of the fp32 blocks (floats)
    // P, two buffers: forward in bf16 the two terms of one chunk's, else two chunks'
    static constexpr bool PLO = BF && MODE == kFwd;
    static constexpr int P0 = NBUF * SB;
    static constexpr int PB = MODE == kKeep ? 0 : C * PRB;
    static constexpr int N0 = P0 + 2 * PB, NB = 32 * NRB;
    static constexpr int L0 = N0 + 2 * NBLK * NB, LB = NBLK > 1 ? NB : 0;
    static constexpr int F0 = L0 + 2 * LB, FB = 32 * LS * 4;
    static constexpr int G0 = F0 + NBLK * FB;  // G from its 16 tokens' start, log2 units, as two floats
    static constexpr int A0 = G0 + 8 * C, AB = 3 * C * 4 + 64;  // gate factors of one chunk (put_gates)
    // from a chain wave to its output wave: the state's operand fragments and Y's
    static constexpr int H0 = A0 + 3 * AB, HS = DK / 32 * 32 * E * 16, HB = HS + RT / 2 * 32 * E * 16;
    static constexpr int kBytes = H0 + NOW * HB;
    static_assert(kBytes <= 160 * 1024, "LDS of a CU");
};

// The sequence a workgroup works on.
struct Walk {
    int n, hk, h, col0, len, nch;
    bool ident;  // columns of the identity instead of values
    int64_t tok0, slot0;
};

// The sequence of rank r by chunks, most chunks first (ties by index): every thread ranks one sequence.
// Workgroups start in id order, so the longest chains start first and the short ones fill the end.  Up to
// kRanked sequences; with more of them the tail is short anyway.
constexpr int kRanked = 256;
template <int C>
__device__ __forceinline__ int ranked_sequence(const GdnParams &p, int r, int *lds) {
    const int i = threadIdx.x, N = p.num_seqs;
    auto chunks = [&](int j) { return (p.cu[j + 1] - p.cu[j] + C - 1) / C; };
    const int own = i < N ? chunks(i) : 0;
    if (i < kRanked) lds[1 + i] = own;
    __syncthreads();
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < N; ++j) {
        const int c = lds[1 + j];
        rank += c > own || (c == own && j < i);
    }
    if (i < N && rank == r) lds[0] = i;
    __syncthreads();
    const int n = lds[0];
    __syncthreads();
    return n;
}

template <int C, int CT>
__device__ __forceinline__ Walk walk_of(const GdnParams &p, char *smem) {
    Walk w;
    const int ntile = (p.dv + (p.sm ? p.dk : 0)) / CT, rep = p.Hv / p.Hk;
    // the tiles and the value heads that share a key head run next to each other on one XCD
    const SeqItem it = seq_item(blockIdx.x, p.num_seqs, p.Hk, rep * ntile, nullptr);
    w.n = it.n;
    if (p.cu && p.num_seqs > 1 && p.num_seqs <= kRanked)
        w.n = __builtin_amdgcn_readfirstlane(ranked_sequence<C>(p, it.n, reinterpret_cast<int *>(smem)));
    w.hk = it.h;
    w.h = it.h * rep + it.tile / ntile;
    w.col0 = (it.tile % ntile) * CT;
    w.ident = w.col0 >= p.dv;
    if (w.ident) w.col0 -= p.dv;
    if (p.segs) {
        const int seq = w.n / p.seg_run, seg = p.seg_first + w.n % p.seg_run, at = seg * p.seg_len;
        w.n = seq * p.segs + seg;
        w.tok0 = (int64_t)seq * p.T + at;
        w.len = min(p.seg_len, p.T - at);
        w.slot0 = (int64_t)seq * ((p.T + C - 1) / C) + at / C;
    } else if (p.cu) {
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
    const char *src = static_cast<const char *>(p.v) + (t0 * p.ldv + (int64_t)w.h * p.dv + (w.ident ? 0 : w.col0)) * L::E;
#pragma unroll
    for (int i = 0; i < L::VB / 1024; ++i) {
        const int piece = 64 * i + lane, row = piece / VSPR;
        load_lds16(src + min(row, clen - 1) * p.ldv * L::E + (piece % VSPR) * 16, dst + L::KB + L::QB + i * 1024);
    }
}

// Loads above this line are issued before anything below it (left alone, the compiler pairs every LDS read
// with its product and waits for each: 4.1 -> 2.8 us per chunk with the waits spread out).  fp32 operands
// take twice the registers and keep the compiler's order.
template <bool BF>
__device__ __forceinline__ void issue_loads() {
    if constexpr (BF) __builtin_amdgcn_sched_barrier(0);
}

// Decays inside diagonal tile r of the chunk whose cumulative gates are in LDS, as a lane's entries of make_tiles.
template <bool BF, int DK, int CT, int MODE>
__device__ __forceinline__ f32x4 diag_decay(const char *smem, int r, int l16, int q4) {
    using L = Lds<BF, DK, CT, MODE>;
    const float *Gh = reinterpret_cast<const float *>(smem + L::G0) + 16 * r, *Gl = Gh + L::C;
    const float ho = Gh[l16], lo = Gl[l16];
    const f32x4 h4 = load_f4(Gh + 4 * q4), l4 = load_f4(Gl + 4 * q4);
    f32x4 gam;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const bool low = MODE == kRev ? 4 * q4 + e >= l16 : l16 >= 4 * q4 + e;
        const float d = (ho - h4[e]) + (lo - l4[e]);
        gam[e] = low ? fast_exp2(MODE == kRev ? -d : d) : 0.f;
    }
    return gam;
}

// Decay of tile (r, c) as a lane's four entries: forward (i, j) = (16 r + l16, 16 c + 4 q4 + e), reverse
// (16 r + 4 q4 + e, 16 c + l16).  Below the diagonal it is a product of three stored factors, all at most 1
// (row token from its tile's start, between the tiles, column token to its tile's end); inside a
// diagonal tile it is formed from differences of the cumulative gates, kept as two floats.
template <bool BF, int DK, int CT, int MODE>
__device__ __forceinline__ f32x4 tile_decay(const char *smem, const float *gate, int r, int c, int l16, int q4) {
    using L = Lds<BF, DK, CT, MODE>;
    constexpr bool REV = MODE == kRev;
    if (r == c) return diag_decay<BF, DK, CT, MODE>(smem, r, l16, q4);
    const float *up = gate + 16 * r, *down = gate + L::C + 16 * c, *between = gate + 3 * L::C + 8;
    const float f = r - c == 1 ? 1.f : between[r - c == 3 ? 2 : c];
    return load_f4((REV ? up : down) + 4 * q4) * ((REV ? down : up)[l16] * f);
}

// A wave's 16 x 16 tiles of the 32 x 32 block (RB, CB) of M B: the decayed K K^T, its columns scaled by beta.
// Forward: rows of the stored matrices are the tokens i that are solved for; reverse: transposed.
template <bool BF, int DK, int CT, int MODE, int RB, int CB>
__device__ __forceinline__ void make_tiles(char *smem, int buf, int par, int abuf, int l16, int q4) {
    using L = Lds<BF, DK, CT, MODE>;
    constexpr bool REV = MODE == kRev, DIAG = RB == CB;
    const char *K = smem + buf * L::SB;
    const float *gate = reinterpret_cast<const float *>(smem + L::A0 + abuf * L::AB), *beta = gate + 2 * L::C;
    Frag2<BF> kr[2][DK / 32], kc[2][DK / 32];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int t = 0; t < DK / 32; ++t) {
            kr[i][t] = row_frag<BF, L::RB>(K, 32 * RB + 16 * i + l16, 32 * t + 8 * q4);
            if constexpr (!DIAG) kc[i][t] = row_frag<BF, L::RB>(K, 32 * CB + 16 * i + l16, 32 * t + 8 * q4);
        }
    f32x4 gam[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float *bj = beta + 16 * (2 * CB + j);
        const f32x4 bet = REV ? f32x4{bj[l16], bj[l16], bj[l16], bj[l16]} : load_f4(bj + 4 * q4);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (2 * CB + j <= 2 * RB + i)
                gam[i][j] = tile_decay<BF, DK, CT, MODE>(smem, gate, 2 * RB + i, 2 * CB + j, l16, q4) * bet;
    }
    issue_loads<BF>();
    f32x4 kk[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) kk[i][j] = zero4();
#pragma unroll
    for (int t = 0; t < DK / 32; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (2 * CB + j > 2 * RB + i) continue;
                const Frag2<BF> y = DIAG ? kr[j][t] : kc[j][t];
                if constexpr (REV) mma<BF>(kk[i][j], kr[i][t], y);
                else mma<BF>(kk[i][j], y, kr[i][t]);
            }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = 2 * RB + i, c = 2 * CB + j;
            if (c > r) continue;
            const int own = REV ? 16 * c + l16 : 16 * r + l16, four = (REV ? 16 * r : 16 * c) + 4 * q4;
            f32x4 m = kk[i][j] * gam[i][j];
            if constexpr (DIAG) {
                if (c == r) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) m[e] = own == four + e ? 0.f : m[e];
                }
                float *dst = reinterpret_cast<float *>(smem + L::F0) + RB * 32 * L::LS;
                if constexpr (REV) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) dst[((four + e) & 31) * L::LS + (own & 31)] = m[e];
                } else {
                    *reinterpret_cast<f32x4 *>(dst + (own & 31) * L::LS + (four & 31)) = m;
                }
            } else {
                row_put4<BF, L::NRB>(smem + L::L0 + par * L::LB, own & 31, kpos(four & 31), -m[0], -m[1], -m[2], -m[3]);
            }
        }
}

// The tiles of P of wave W of three.  64 tokens: (0,0) (1,0) (1,1) (2,0), then (2,1) (2,2) (3,2) (3,3), and (3,0)
// (3,1) by the wave below the diagonal; 32 tokens: all by the first.
template <int RT, int W>
__device__ __forceinline__ constexpr bool owns_tile(int r, int c) {
    if (c > r || RT == 2) return c <= r && W == 0;
    return W == (r == 3 && c < 2 ? 2 : r < 2 || (r == 2 && c == 0) ? 0 : 1);
}
// Forward: P, in bf16 as two terms, with the diagonal tiles' decays in diag; reverse: scale P^T.
template <bool BF, int DK, int CT, int MODE, int W>
__device__ __forceinline__ void make_p(char *smem, int buf, int par, int abuf, float scale, const f32x4 (&diag)[2],
                                       int l16, int q4) {
    using L = Lds<BF, DK, CT, MODE>;
    constexpr bool REV = MODE == kRev;
    constexpr int RT = L::RT, R0 = W == 0 ? 0 : W + 1, R1 = W == 0 ? (RT == 2 ? 2 : 3) : 4;  // its rows and
    constexpr int C0 = W == 1 ? 1 : 0, C1 = W == 1 ? 4 : 2;                                  // columns of tiles
    const char *K = smem + buf * L::SB, *Q = K + L::KB;
    char *P = smem + L::P0 + par * L::PB;
    const float *gate = reinterpret_cast<const float *>(smem + L::A0 + abuf * L::AB);
    Frag2<BF> qr[R1 - R0][DK / 32], kc[C1][DK / 32];
    f32x4 gam[R1 - R0][C1], acc[R1 - R0][C1];
#pragma unroll
    for (int t = 0; t < DK / 32; ++t) {
#pragma unroll
        for (int r = R0; r < R1; ++r) qr[r - R0][t] = row_frag<BF, L::RB>(Q, 16 * r + l16, 32 * t + 8 * q4);
#pragma unroll
        for (int c = C0; c < C1; ++c) kc[c][t] = row_frag<BF, L::RB>(K, 16 * c + l16, 32 * t + 8 * q4);
    }
#pragma unroll
    for (int r = R0; r < R1; ++r)
#pragma unroll
        for (int c = C0; c < C1; ++c)
            if (owns_tile<RT, W>(r, c)) {
                gam[r - R0][c] = r == c && MODE == kFwd ? diag[r & 1]
                                                        : tile_decay<BF, DK, CT, MODE>(smem, gate, r, c, l16, q4);
                acc[r - R0][c] = zero4();
            }
    issue_loads<BF>();
#pragma unroll
    for (int t = 0; t < DK / 32; ++t)
#pragma unroll
        for (int r = R0; r < R1; ++r)
#pragma unroll
            for (int c = C0; c < C1; ++c)
                if (owns_tile<RT, W>(r, c)) {
                    if constexpr (REV) mma<BF>(acc[r - R0][c], qr[r - R0][t], kc[c][t]);
                    else mma<BF>(acc[r - R0][c], kc[c][t], qr[r - R0][t]);
                }
#pragma unroll
    for (int r = R0; r < R1; ++r)
#pragma unroll
        for (int c = C0; c < C1; ++c) {
            if (!owns_tile<RT, W>(r, c)) continue;
            const int own = REV ? 16 * c + l16 : 16 * r + l16, four = (REV ? 16 * r : 16 * c) + 4 * q4;
            const int at = (four & ~31) + kpos(four & 31);
            f32x4 m = acc[r - R0][c] * gam[r - R0][c];
            if constexpr (REV) m = m * scale;
            row_put4<BF, L::PRB>(P, own, at, m[0], m[1], m[2], m[3]);
            if constexpr (L::PLO) {
                const Frag<true> lo = frag_lo(m, frag_from_acc<true>(m));
                *reinterpret_cast<uint2 *>(P + L::PB + row_off<L::PRB>(own, 2 * at)) = lo.v;
            }
        }
}

// Four rank-1 terms of a substitution inside rows of 16 lanes, other lanes' values read through DPP.
// s_nop 1: a DPP operand must not have been written by the two instructions before.
// rows: n[c] += m * (n[c] of lane J), c = 0..3
template <int J>
__device__ __forceinline__ void bcast_rows4(float *n, float m) {
    asm("s_nop 1\n\t"
        "v_fmac_f32_dpp %0, %0, %4 row_newbcast:%5 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %1, %1, %4 row_newbcast:%5 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %2, %2, %4 row_newbcast:%5 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %3, %3, %4 row_newbcast:%5 row_mask:0xf bank_mask:0xf"
        : "+v"(n[0]), "+v"(n[1]), "+v"(n[2]), "+v"(n[3])
        : "v"(m), "n"(J));
}
// columns: x += n[j] * (m[j] of lane I), j = 0..3
template <int I>
__device__ __forceinline__ void bcast_cols4(float &x, const float *n, const float *m) {
    asm("s_nop 1\n\t"
        "v_fmac_f32_dpp %0, %5, %1 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %6, %2 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %7, %3 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %8, %4 row_newbcast:%9 row_mask:0xf bank_mask:0xf"
        : "+v"(x)
        : "v"(n[0]), "v"(n[1]), "v"(n[2]), "v"(n[3]), "v"(m[0]), "v"(m[1]), "v"(m[2]), "v"(m[3]), "n"(I));
}
// A 16 x 16 x 16 fp32 product in two independent halves.
__device__ __forceinline__ f32x4 product16(const Frag<false> &a, const Frag<false> &b) {
    f32x4 x = zero4(), y = zero4();
    x = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v.x, b.v.x, x, 0, 0, 0);
    y = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v.y, b.v.y, y, 0, 0, 0);
    x = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v.z, b.v.z, x, 0, 0, 0);
    y = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v.w, b.v.w, y, 0, 0, 0);
    return x + y;
}
// Eight columns of row l16 of (I + L)^-1 from nl, row l16 of the strictly lower -L: row j, once it is solved, is
// taken off every later row (nl is zero in the others).  n[0..3] are columns that row j can have for every j,
// n[4..7] columns from 8 on.
template <int J>
__device__ __forceinline__ void solve_rows(float (&n)[8], const float (&nl)[16]) {
    if constexpr (J < 15) {
        bcast_rows4<J>(n, nl[J]);
        if constexpr (J >= 8) bcast_rows4<J>(n + 4, nl[J]);
        solve_rows<J + 1>(n, nl);
    }
}
// Column l16 of (I + L)^-1, the rows of -L held by the lanes.
template <int I>
__device__ __forceinline__ void solve_cols(float (&n)[16], const float (&nl)[16]) {
    if constexpr (I < 16) {
        float x = n[I];
        n[I] = 0.f;  // not yet a term of its own row
#pragma unroll
        for (int j = 0; j < I; j += 4) bcast_cols4<I>(x, n + j, nl + j);
        n[I] = x;
        solve_cols<I + 1>(n, nl);
    }
}

// The inverse of one 32 x 32 diagonal block of I + M B, minus the identity (reverse: transposed), by the wave
// that made its tiles, in two parts on both sides of the step's middle barrier: two 16 x 16 diagonal blocks by forward substitution in registers (lanes of 16
// exchange values through DPP, about 8 cycles a term), and -N11 (L10 N00) below them.  Forward: a lane
// has one row and eight columns (0-3 and 12-15, or 4-7 and 8-11); reverse: one column, half of which it
// stores.
struct Inverse {
    float n[8];
    Frag<false> l10;
};
template <bool BF, int DK, int CT, int MODE>
__device__ __forceinline__ void solve_diagonals(Inverse &inv, char *smem, int blk, int lane) {
    using L = Lds<BF, DK, CT, MODE>;
    constexpr bool REV = MODE == kRev;
    const int l16 = lane & 15, q4 = lane >> 4, sub = q4 & 1, half = q4 >> 1;
    const int c0 = half ? 4 : 0, c1 = half ? 8 : 12;
    float *Lb = reinterpret_cast<float *>(smem + L::F0) + blk * 32 * L::LS;
    const float *Ld = Lb + (16 * sub + l16) * L::LS + 16 * sub;
    float nl[16];
    auto &n = inv.n;
    wave_lds_sync();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x4 v = load_f4(Ld + 4 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) nl[4 * i + j] = -v[j];
    }
    inv.l10.v = *reinterpret_cast<const float4 *>(Lb + (16 + l16) * L::LS + 4 * q4);
    if constexpr (REV) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = i == l16 ? 1.f : 0.f;
        solve_cols<1>(x, nl);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            n[j] = half ? x[4 + j] : x[j];
            n[4 + j] = half ? x[8 + j] : x[12 + j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            n[j] = c0 + j == l16 ? 1.f : 0.f;
            n[4 + j] = c1 + j == l16 ? 1.f : 0.f;
        }
        solve_rows<0>(n, nl);
    }
    wave_lds_sync();
    // both inverses to LDS: block 0 into the unused upper right block, block 1 over the upper left one, which has
    // been read
    float *dst = Lb + l16 * L::LS + (sub ? 0 : 16);
    *reinterpret_cast<float4 *>(dst + c0) = make_float4(n[0], n[1], n[2], n[3]);
    *reinterpret_cast<float4 *>(dst + c1) = make_float4(n[4], n[5], n[6], n[7]);
    wave_lds_sync();
}
template <bool BF, int DK, int CT, int MODE>
__device__ __forceinline__ void join_inverse(const Inverse &inv, char *smem, int blk, int par, int lane) {
    using L = Lds<BF, DK, CT, MODE>;
    constexpr bool REV = MODE == kRev;
    const int l16 = lane & 15, q4 = lane >> 4, sub = q4 & 1, half = q4 >> 1;
    const int c0 = half ? 4 : 0, c1 = half ? 8 : 12;
    const float *Lb = reinterpret_cast<const float *>(smem + L::F0) + blk * 32 * L::LS;
    char *N = smem + L::N0 + (par * L::NBLK + blk) * L::NB;
    const auto &n = inv.n;
    // forward: T = L10 N00, then N10 = -N11 T with rows of N11 as A; its transpose (the operands exchanged) puts
    // four columns of a row of N10 in a lane.  Reverse: the stored rows are columns of the inverses.
    const float *s00 = Lb + 16, *s11 = Lb;
    Frag<false> n00, n11;
    if constexpr (REV) {
        n00.v = *reinterpret_cast<const float4 *>(s00 + l16 * L::LS + 4 * q4);  // N00[4 q4 + j][l16]
        n11 = make_frag<false>(s11[4 * q4 * L::LS + l16], s11[(4 * q4 + 1) * L::LS + l16],
                               s11[(4 * q4 + 2) * L::LS + l16], s11[(4 * q4 + 3) * L::LS + l16]);  // N11[l16][..]
    } else {
        n00 = make_frag<false>(s00[4 * q4 * L::LS + l16], s00[(4 * q4 + 1) * L::LS + l16],
                               s00[(4 * q4 + 2) * L::LS + l16], s00[(4 * q4 + 3) * L::LS + l16]);
        n11.v = *reinterpret_cast<const float4 *>(s11 + l16 * L::LS + 4 * q4);
    }
    issue_loads<BF>();
    const f32x4 t = product16(inv.l10, n00);
    float y[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        y[j] = c0 + j == l16 ? 0.f : n[j];
        y[4 + j] = c1 + j == l16 ? 0.f : n[4 + j];
    }
    row_put4<BF, L::NRB>(N, 16 * sub + l16, kpos(16 * sub + c0), y[0], y[1], y[2], y[3]);
    row_put4<BF, L::NRB>(N, 16 * sub + l16, kpos(16 * sub + c1), y[4], y[5], y[6], y[7]);
    const Frag<false> mt = frag_from_acc<false>(t, -1.f);
    // reverse: N10[4 q4 + j][l16], forward: N10^T[4 q4 + j][l16]
    const f32x4 n10 = REV ? product16(n11, mt) : product16(mt, n11);
    row_put4<BF, L::NRB>(N, (REV ? 0 : 16) + l16, kpos((REV ? 16 : 0) + 4 * q4), n10[0], n10[1], n10[2], n10[3]);
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
// differences finite; a NaN is below nothing and stays one).
constexpr float kNoGate = -1e4f;
__device__ __forceinline__ double lane_value(double x, int lane) {
    const long long b = __double_as_longlong(x);
    const unsigned lo = __builtin_amdgcn_readlane((int)b, lane), hi = __builtin_amdgcn_readlane((int)(b >> 32), lane);
    return __longlong_as_double((long long)hi << 32 | lo);
}
template <int N>
__device__ __forceinline__ double row_shr64(double x) {
    const long long b = __double_as_longlong(x);
    const unsigned lo = __builtin_amdgcn_update_dpp(0, (int)b, 0x110 + N, 0xf, 0xf, true);
    const unsigned hi = __builtin_amdgcn_update_dpp(0, (int)(b >> 32), 0x110 + N, 0xf, 0xf, true);
    return __longlong_as_double((long long)hi << 32 | lo);
}
struct GateScan {
    double s, end[5];  // the lane's cumulative gate; those at the starts of the four 16-token blocks and at the end
};
__device__ __forceinline__ GateScan gate_scan(float g) {
    GateScan r;
    double s = (double)(g < kNoGate ? kNoGate : g) * 1.4426950408889634;
    s += row_shr64<1>(s);
    s += row_shr64<2>(s);
    s += row_shr64<4>(s);
    s += row_shr64<8>(s);
    r.end[0] = 0.0;
#pragma unroll
    for (int b = 0; b < 4; ++b) r.end[b + 1] = r.end[b] + lane_value(s, 16 * b + 15);
    r.s = s;
    return r;
}
// A chunk's gate factors (all at most 1 for g <= 0), lane = token: up = e^{G - G(end of the previous 16
// tokens)}, down = e^{G(end of its 16 tokens) - G}, beta; then per block e^{G} of its start and
// e^{G_C - G} of its end, the decays between non-neighbouring blocks (2,0), (3,1), (3,0), and e^{G_C}.
struct Gates {
    float up, down, beta, hi, lo, f[6];  // f: block start and end, (2,0), (3,1), (3,0), whole chunk
};
template <int C>
__device__ __forceinline__ Gates make_gates(const RawGate &r, int lane) {
    const GateScan sc = gate_scan(r.g);
    const int blk = lane >> 4;
    const double start = blk == 0 ? 0.0 : blk == 1 ? sc.end[1] : blk == 2 ? sc.end[2] : sc.end[3];
    const double own_end = blk == 0 ? sc.end[1] : blk == 1 ? sc.end[2] : blk == 2 ? sc.end[3] : sc.end[4];
    const double end = sc.end[C / 16];
    Gates g;
    g.hi = (float)sc.s;
    g.lo = (float)(sc.s - g.hi);
    g.up = fast_exp2(g.hi);
    g.down = fast_exp2((float)(own_end - start - sc.s));
    g.beta = r.b;
    g.f[0] = fast_exp2((float)start);
    g.f[1] = fast_exp2((float)(end - own_end));
    g.f[2] = fast_exp2((float)(sc.end[2] - sc.end[1]));
    g.f[3] = fast_exp2((float)(sc.end[3] - sc.end[2]));
    g.f[4] = fast_exp2((float)(sc.end[3] - sc.end[1]));
    g.f[5] = fast_exp2((float)end);
    return g;
}
template <bool BF, int DK, int CT, int MODE>
__device__ __forceinline__ void put_gates(char *smem, int abuf, const Gates &g, int lane) {
    using L = Lds<BF, DK, CT, MODE>;
    float *a = reinterpret_cast<float *>(smem + L::A0 + abuf * L::AB), *G = reinterpret_cast<float *>(smem + L::G0);
    if (lane < L::C) {
        G[lane] = g.hi;
        G[L::C + lane] = g.lo;
        a[lane] = g.up;
        a[L::C + lane] = g.down;
        a[2 * L::C + lane] = g.beta;
        float *f = a + 3 * L::C;
        if ((lane & 15) == 0) {
            f[lane >> 4] = g.f[0];
            f[4 + (lane >> 4)] = g.f[1];
        }
        if (lane == 0) {
#pragma unroll
            for (int i = 2; i < 6; ++i) f[6 + i] = g.f[i];
        }
    }
}

// The gates of the chunks to come: in the second phase of step s those of chunk s + 2, made a step before, are
// stored (in the first phase the tile waves read the cumulative gates of chunk s + 1) and those of
// chunk s + 3 made.
template <bool BF, int DK, int CT, int MODE>
struct GateMaker {
    using L = Lds<BF, DK, CT, MODE>;
    const GdnParams &p;
    const Walk &w;
    char *smem;
    int lane;
    RawGate raw{0.f, 0.f}, first[3];
    Gates g{};
    // chunk 0's gates stored, chunk 1's made; chunk 2's are on their way
    __device__ __forceinline__ void begin() {
#pragma unroll
        for (int s = 0; s < 3; ++s)
            if (s < w.nch) first[s] = load_gate<L::C>(p, w, chunk(s), lane);
        g = make_gates<L::C>(first[0], lane);
        put(0);
        if (w.nch > 1) g = make_gates<L::C>(first[1], lane);
        raw = first[2];
    }
    __device__ __forceinline__ int chunk(int s) const { return MODE == kRev ? w.nch - 1 - s : s; }
    __device__ __forceinline__ void load(int s) {
        if (s < w.nch) raw = load_gate<L::C>(p, w, chunk(s), lane);
    }
    __device__ __forceinline__ void make(int s) {  // chunk s, whose raw gates have been loaded
        if (s < w.nch) g = make_gates<L::C>(raw, lane);
        load(s + 1);
        __builtin_amdgcn_sched_barrier(0);
    }
    __device__ __forceinline__ void put(int s) {
        if (s < w.nch) put_gates<BF, DK, CT, MODE>(smem, s % 3, g, lane);
    }
};

// One operand fragment pair per lane, handed from wave to wave.
template <bool BF>
__device__ __forceinline__ void hand_put(char *base, int i, int lane, const Frag2<BF> &f) {
    if constexpr (BF) {
        *reinterpret_cast<uint4 *>(base + (i * 64 + lane) * 16) = make_uint4(f.a.v.x, f.a.v.y, f.b.v.x, f.b.v.y);
    } else {
        *reinterpret_cast<float4 *>(base + (2 * i * 64 + lane) * 16) = f.a.v;
        *reinterpret_cast<float4 *>(base + ((2 * i + 1) * 64 + lane) * 16) = f.b.v;
    }
}
template <bool BF>
__device__ __forceinline__ Frag2<BF> hand_get(const char *base, int i, int lane) {
    Frag2<BF> f;
    if constexpr (BF) {
        const uint4 w = *reinterpret_cast<const uint4 *>(base + (i * 64 + lane) * 16);
        f.a.v = make_uint2(w.x, w.y);
        f.b.v = make_uint2(w.z, w.w);
    } else {
        f.a.v = *reinterpret_cast<const float4 *>(base + (2 * i * 64 + lane) * 16);
        f.b.v = *reinterpret_cast<const float4 *>(base + ((2 * i + 1) * 64 + lane) * 16);
    }
    return f;
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
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, q4 = lane >> 4;
    const Walk w = walk_of<C, CT>(p, smem);
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
#define GDN_TILES(RB_, CB_) make_tiles<BF, DK, CT, MODE, RB_, CB_>(smem, s % L::NBUF, s & 1, s % 3, l16, q4)
    if (wave >= L::QW0 && wave < L::QW0 + 2) {
        // ------------------------------------------------------------------ Q K^T and output waves
        if (nch == 0) return;
        const int cw = wave - L::QW0;
        // forward: P of the step's own chunk, the decays of its diagonal tiles formed a step ahead (the cumulative
        // gates in LDS are the next chunk's by then); reverse: P^T of the next chunk
        f32x4 diag[2];
        auto tiles = [&](int s) {
            if constexpr (MODE != kKeep) {
                const int par = MODE == kFwd ? 0 : s & 1;
                if (cw == 0) make_p<BF, DK, CT, MODE, 0>(smem, s % L::NBUF, par, s % 3, p.scale, diag, l16, q4);
                if constexpr (L::NBLK == 2) {
                    if (cw == 1) make_p<BF, DK, CT, MODE, 1>(smem, s % L::NBUF, par, s % 3, p.scale, diag, l16, q4);
                }
            }
        };
        auto next_diag = [&] {
            if (MODE == kFwd && cw < L::NBLK) {
#pragma unroll
                for (int i = 0; i < 2; ++i) diag[i] = diag_decay<BF, DK, CT, MODE>(smem, 2 * cw + i, l16, q4);
            }
        };
        __syncthreads();
        if (MODE == kFwd) next_diag();
        else tiles(0);
        __syncthreads();
        __syncthreads();
#pragma unroll 1
        for (int s = 0; s < nch; ++s) {
            if (MODE == kFwd) {
                tiles(s);
                if (s + 1 < nch) next_diag();
            } else if (s + 1 < nch) {
                tiles(s + 1);
            }
            __syncthreads();  // A
            if constexpr (MODE == kFwd) {
                const int clen = min(C, w.len - s * C);

                const char *hand = smem + L::H0 + cw * L::HB;
                [[maybe_unused]] const char *ylo = smem + (s % L::NBUF) * L::SB + L::KB + L::QB + cw * (L::VB / 2);
                const char *Q = smem + (s % L::NBUF) * L::SB + L::KB, *P = smem + L::P0;
                const float *gate = reinterpret_cast<const float *>(smem + L::A0 + (s % 3) * L::AB);
                IO *out = static_cast<IO *>(p.out) + ((w.tok0 + (int64_t)s * C) * p.Hv + w.h) * p.dv + w.col0 + 16 * cw + 4 * q4;
                Frag2<BF> qf[RT][K2], pf[RT][RT / 2];
                float e[RT];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
                    for (int t = 0; t < K2; ++t) qf[rt][t] = row_frag<BF, L::RB>(Q, 16 * rt + l16, 32 * t + 8 * q4);
#pragma unroll
                    for (int u = 0; u <= rt / 2; ++u) pf[rt][u] = row_frag<BF, L::PRB>(P, 16 * rt + l16, 32 * u + 8 * q4);
                    e[rt] = gate[16 * rt + l16] * gate[3 * C + rt];
                }
                Frag2<BF> sb[K2], yp[RT / 2], yl[RT / 2];
#pragma unroll
                for (int t = 0; t < K2; ++t) sb[t] = hand_get<BF>(hand, t, lane);
#pragma unroll
                for (int u = 0; u < RT / 2; ++u) {
                yp[u] = hand_get<BF>(hand + L::HS, u, lane);
                if constexpr (L::PLO) yl[u] = hand_get<BF>(ylo, u, lane);
            }
                issue_loads<BF>();
                // O^T tiles: a lane holds four consecutive columns of one token
                f32x4 o[RT];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) o[rt] = zero4();
#pragma unroll
                for (int t = 0; t < K2; ++t)
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) mma<BF>(o[rt], sb[t], qf[rt][t]);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) o[rt] = o[rt] * e[rt];
#pragma unroll
                for (int u = 0; u < RT / 2; ++u)
#pragma unroll
                    for (int rt = 2 * u; rt < RT; ++rt) {
                        mma<BF>(o[rt], yp[u], pf[rt][u]);
                        if constexpr (L::PLO) {
                            mma<BF>(o[rt], yp[u], row_frag<BF, L::PRB>(P + L::PB, 16 * rt + l16, 32 * u + 8 * q4));
                            mma<BF>(o[rt], yl[u], pf[rt][u]);
                        }
                    }
#pragma unroll
                for (int rt = 0; rt < RT; rt += 2) mfma_settle(o[rt], o[rt + 1]);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
                    if (16 * rt + l16 < clen)
                        IoTraits<IO>::store4(out + (int64_t)(16 * rt + l16) * p.Hv * p.dv,
                                             make_float4(o[rt][0] * p.scale, o[rt][1] * p.scale, o[rt][2] * p.scale,
                                                         o[rt][3] * p.scale));
            }
            __syncthreads();  // B
        }
        return;
    }
    if (wave == L::GW) {
        // ------------------------------------------------------------------ block below the diagonal, gates
        if (nch == 0) return;
        GateMaker<BF, DK, CT, MODE> gm{p, w, smem, lane};
        gm.begin();
        const f32x4 none[2] = {zero4(), zero4()};
        auto tiles = [&](int s) {
            if constexpr (L::NBLK == 2) GDN_TILES(1, 0);
        };
        auto p_tiles = [&](int s) {
            if constexpr (L::NBLK == 2 && MODE != kKeep)
                make_p<BF, DK, CT, MODE, 2>(smem, s % L::NBUF, MODE == kFwd ? 0 : s & 1, s % 3, p.scale, none, l16, q4);
        };
        __syncthreads();
        tiles(0);
        if (MODE == kRev) p_tiles(0);
        __syncthreads();
        gm.put(1);
        gm.make(2);
        __syncthreads();
#pragma unroll 1
        for (int s = 0; s < nch; ++s) {
            if (MODE == kFwd) p_tiles(s);
            if (s + 1 < nch) {
                tiles(s + 1);
                if (MODE == kRev) p_tiles(s + 1);
            }
            __syncthreads();  // A
            gm.put(s + 2);
            gm.make(s + 3);
            __syncthreads();  // B
        }
        return;
    }
    if (wave >= L::KW0) {
        // ------------------------------------------------------------------ diagonal blocks and their inverses
        if (nch == 0) return;
        const int blk = wave - L::KW0;
        Inverse inv;
        auto tiles = [&](int s) {
            if (blk == 0) GDN_TILES(0, 0);
            if constexpr (L::NBLK == 2) {
                if (blk == 1) GDN_TILES(1, 1);
            }
            if (blk < L::NBLK) solve_diagonals<BF, DK, CT, MODE>(inv, smem, blk, lane);
        };
        auto join = [&](int s) {
            if (blk < L::NBLK) join_inverse<BF, DK, CT, MODE>(inv, smem, blk, s & 1, lane);
        };
        __syncthreads();
        tiles(0);
        __syncthreads();
        join(0);
        __syncthreads();
#pragma unroll 1
        for (int s = 0; s < nch; ++s) {
            if (s + 1 < nch) tiles(s + 1);
            __syncthreads();  // A
            if (s + 1 < nch) join(s + 1);
            __syncthreads();  // B
        }
        return;
    }
#undef GDN_TILES

    // ------------------------------------------------------------------ chain waves
    __builtin_amdgcn_s_setprio(2);  // the chain is what every other wave waits for
    const int col = w.col0 + 16 * wave + l16;
    // the state's place: rows of `width` columns
    const int width = w.ident ? DK : p.dv;
    const int64_t sbase = ((int64_t)w.n * p.Hv + w.h) * DK * width + col;
    f32x4 S[KT];
    // one branch around all the loads: one per value would wait for each (10 us of a workgroup's start)
    auto load_state = [&](auto *src) {
#pragma unroll
        for (int ct = 0; ct < KT; ++ct)
#pragma unroll
            for (int j = 0; j < 4; ++j) S[ct][j] = elem_f32(src[sbase + (int64_t)state_channel(ct, q4, j) * width]);
    };
    if (w.ident || !p.s0) {
#pragma unroll
        for (int ct = 0; ct < KT; ++ct)
#pragma unroll
            for (int j = 0; j < 4; ++j) S[ct][j] = w.ident && state_channel(ct, q4, j) == col ? 1.f : 0.f;
    } else if (p.s0_bf16) {
        load_state(static_cast<const uint16_t *>(p.s0));
    } else {
        load_state(static_cast<const float *>(p.s0));
    }
    // K's and the values' fragments of a chunk are read before the barrier that opens its step: they have been in
    // LDS for a step by then.  In the forward each chain wave stores over half of both waves' values (the second terms
    // of Y) before the step's middle barrier, so a barrier must stand between these reads and its step: B of
    // the step before, and for chunk 0, which the first opening barrier puts in LDS, the third.
    Frag2<BF> kf[RT][K2];
    Frag<BF> vf[RT];
    auto fetch = [&](int s) {
        const char *K = smem + (s % L::NBUF) * L::SB, *V = K + L::KB + L::QB;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
            for (int t = 0; t < K2; ++t) kf[rt][t] = row_frag<BF, L::RB>(K, 16 * rt + l16, 32 * t + 8 * q4);
            vf[rt] = value_frag<BF, L::VRB>(V, wave, rt, l16, q4);
            if (MODE == kKeep && w.ident) vf[rt] = make_frag<BF>(0.f, 0.f, 0.f, 0.f);
        }
    };
    // (not in reverse, which has no registers left for them, and where a wave stores over its own columns only)
    if (nch > 0) {
        __syncthreads();
        if (!REV) fetch(0);
        __syncthreads();
        __syncthreads();
    }
#pragma unroll 1
    for (int s = 0; s < nch; ++s) {
        const int c = ci(s), clen = min(C, w.len - c * C);
        const int64_t tok = w.tok0 + (int64_t)c * C;
        char *K = smem + (s % L::NBUF) * L::SB, *V = K + L::KB + L::QB;
        [[maybe_unused]] const char *Q = K + L::KB;
        [[maybe_unused]] char *hand = smem + L::H0 + wave * L::HB;
        [[maybe_unused]] const char *P = smem + L::P0 + (s & 1) * L::PB;
        const char *N = smem + L::N0 + (s & 1) * L::NBLK * L::NB, *Lba = smem + L::L0 + (s & 1) * L::LB;
        const float *gate = reinterpret_cast<const float *>(smem + L::A0 + (s % 3) * L::AB), *beta = gate + 2 * C;
        const float eC = gate[3 * C + 11];
        auto eG = [&](int rt) { return load_f4(gate + 16 * rt + 4 * q4) * gate[3 * C + rt]; };          // e^G
        auto eB = [&](int rt) { return load_f4(gate + C + 16 * rt + 4 * q4) * gate[3 * C + 4 + rt]; };  // e^{G_C - G}
        Frag2<BF> Sb[K2];
#pragma unroll
        for (int t = 0; t < K2; ++t) Sb[t] = {frag_from_acc<BF>(S[2 * t]), frag_from_acc<BF>(S[2 * t + 1])};
        if constexpr (MODE == kFwd) {
#pragma unroll
            for (int t = 0; t < K2; ++t) hand_put<BF>(hand, t, lane, Sb[t]);
        } else if (p.hs) {
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
        if constexpr (REV) fetch(s);
        // the inverse blocks and M B between them
        Frag2<BF> nf[L::NBLK][2], lf[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int b = 0; b < L::NBLK; ++b) nf[b][h] = row_frag<BF, L::NRB>(N + b * L::NB, 16 * h + l16, 8 * q4);
            if constexpr (L::NBLK > 1) lf[h] = row_frag<BF, L::NRB>(Lba, 16 * h + l16, 8 * q4);
        }
        issue_loads<BF>();
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) x[rt] = zero4();
#pragma unroll
        for (int t = 0; t < K2; ++t)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) mma<BF>(x[rt], kf[rt][t], Sb[t]);
        if constexpr (!REV) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const f32x4 e = eG(rt), v = frag_f32<BF>(vf[rt]);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[rt][j] = fmaf(-e[j], x[rt][j], v[j]);
            }
            // Z, 32 tokens at a time
#pragma unroll
            for (int b = 0; b < L::NBLK; ++b) {
                if (b > 0) {
                    const Frag2<BF> za = {frag_from_acc<BF>(x[0]), frag_from_acc<BF>(x[1])};
#pragma unroll
                    for (int h = 0; h < 2; ++h) mma<BF>(x[2 + h], lf[h], za);
                }
                const Frag2<BF> xb = {frag_from_acc<BF>(x[2 * b]), frag_from_acc<BF>(x[2 * b + 1])};
#pragma unroll
                for (int h = 0; h < 2; ++h) mma<BF>(x[2 * b + h], nf[b][h], xb);
            }
            Frag2<BF> ys[RT / 2];
#pragma unroll
            for (int u = 0; u < RT / 2; ++u) {
                f32x4 a[2], d[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int rt = 2 * u + h;
                    const f32x4 bt = load_f4(beta + 16 * rt + 4 * q4), e = eB(rt);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        a[h][j] = bt[j] * x[rt][j];
                        d[h][j] = e[j] * a[h][j];
                    }
                }
                if constexpr (MODE == kFwd) {
                    const Frag2<BF> yp = {frag_from_acc<BF>(a[0]), frag_from_acc<BF>(a[1])};
                    hand_put<BF>(hand + L::HS, u, lane, yp);
                    // the second term goes where the chunk's values were, which both chain waves have read before
                    // the barrier that opened this step
                    if constexpr (BF)
                        hand_put<BF>(V + wave * (L::VB / 2), u, lane, Frag2<BF>{frag_lo(a[0], yp.a), frag_lo(a[1], yp.b)});
                }
                ys[u] = {frag_from_acc<BF>(d[0]), frag_from_acc<BF>(d[1])};
            }
            issue_loads<BF>();
            Frag2<BF> kt[KT][RT / 2];
#pragma unroll
            for (int ct = 0; ct < KT; ++ct)
#pragma unroll
                for (int u = 0; u < RT / 2; ++u) kt[ct][u] = col_frag<BF, L::RB>(K, ct, u, l16, q4);
            __syncthreads();  // A
#pragma unroll
            for (int ct = 0; ct < KT; ++ct) S[ct] = S[ct] * eC;
#pragma unroll
            for (int u = 0; u < RT / 2; ++u)
#pragma unroll
                for (int ct = 0; ct < KT; ++ct) mma<BF>(S[ct], kt[ct][u], ys[u]);
            if (MODE == kKeep && p.zs)
                put_value_rows<BF, L::VRB, RT>(V, static_cast<IO *>(p.zs) + (tok * p.Hv + w.h) * p.dv + w.col0,
                                               (int64_t)p.Hv * p.dv, wave, x, clen, lane);
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
                const f32x4 e = eB(rt);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[rt][j] *= e[j];
            }
            Frag2<BF> pf[RT][RT / 2];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int u = rt / 2; u < RT / 2; ++u) pf[rt][u] = row_frag<BF, L::PRB>(P, 16 * rt + l16, 32 * u + 8 * q4);
            issue_loads<BF>();
#pragma unroll
            for (int u = 0; u < RT / 2; ++u)
#pragma unroll
                for (int rt = 0; rt < 2 * u + 2; ++rt) mma<BF>(x[rt], pf[rt][u], Frag2<BF>{vf[2 * u], vf[2 * u + 1]});
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const f32x4 bt = load_f4(beta + 16 * rt + 4 * q4);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[rt][j] *= bt[j];
            }
            // dX, the last 32 tokens first
#pragma unroll
            for (int b = L::NBLK - 1; b >= 0; --b) {
                if (b < L::NBLK - 1) {
                    const Frag2<BF> xb = {frag_from_acc<BF>(x[2 * b + 2]), frag_from_acc<BF>(x[2 * b + 3])};
#pragma unroll
                    for (int h = 0; h < 2; ++h) mma<BF>(x[2 * b + h], lf[h], xb);
                }
                const Frag2<BF> zb = {frag_from_acc<BF>(x[2 * b]), frag_from_acc<BF>(x[2 * b + 1])};
#pragma unroll
                for (int h = 0; h < 2; ++h) mma<BF>(x[2 * b + h], nf[b][h], zb);
            }
            Frag2<BF> dx[RT / 2];
            {
                issue_loads<BF>();
                Frag2<BF> qt[KT][RT / 2], dq[RT / 2];
#pragma unroll
                for (int ct = 0; ct < KT; ++ct)
#pragma unroll
                    for (int u = 0; u < RT / 2; ++u) qt[ct][u] = col_frag<BF, L::RB>(Q, ct, u, l16, q4);
#pragma unroll
                for (int u = 0; u < RT / 2; ++u) {
                    f32x4 a[2], d[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int rt = 2 * u + h;
                        const f32x4 e = eG(rt);
                        a[h] = frag_f32<BF>(vf[rt]) * e * p.scale;
                        d[h] = -x[rt] * e;
                    }
                    dq[u] = {frag_from_acc<BF>(a[0]), frag_from_acc<BF>(a[1])};
                    dx[u] = {frag_from_acc<BF>(d[0]), frag_from_acc<BF>(d[1])};
                }
                issue_loads<BF>();
#pragma unroll
                for (int ct = 0; ct < KT; ++ct) S[ct] = S[ct] * eC;
#pragma unroll
                for (int u = 0; u < RT / 2; ++u)
#pragma unroll
                    for (int ct = 0; ct < KT; ++ct) mma<BF>(S[ct], qt[ct][u], dq[u]);
            }
            issue_loads<BF>();
            Frag2<BF> kt[KT][RT / 2];
#pragma unroll
            for (int ct = 0; ct < KT; ++ct)
#pragma unroll
                for (int u = 0; u < RT / 2; ++u) kt[ct][u] = col_frag<BF, L::RB>(K, ct, u, l16, q4);
            __syncthreads();  // A
#pragma unroll
            for (int u = 0; u < RT / 2; ++u)
#pragma unroll
                for (int ct = 0; ct < KT; ++ct) mma<BF>(S[ct], kt[ct][u], dx[u]);
            if (p.out)
                put_value_rows<BF, L::VRB, RT>(V, static_cast<IO *>(p.out) + (tok * p.Hv + w.h) * p.dv + w.col0,
                                           (int64_t)p.Hv * p.dv, wave, x, clen, lane);
        }
#pragma unroll
        for (int ct = 0; ct < KT; ct += 2) mfma_settle(S[ct], S[ct + 1]);
        issue_loads<BF>();
        if (!REV && s + 1 < nch) fetch(s + 1);
        __syncthreads();  // B
    }
    const bool part = p.segs && !p.maps;  // a sequence's state is that of the last segment walked
    if ((p.sf || w.ident) && (!part || w.n % p.segs == (MODE == kRev ? 0 : p.segs - 1))) {
        // formed anew: otherwise the 64-bit addresses of the first loads stay in registers over the whole walk
        int q4b = q4;
        asm volatile("" : "+v"(q4b));
        const int64_t at = part ? ((int64_t)(w.n / p.segs) * p.Hv + w.h) * DK * width + col : sbase;
        auto store_state = [&](auto *dst, auto convert) {
#pragma unroll
            for (int ct = 0; ct < KT; ++ct)
#pragma unroll
                for (int j = 0; j < 4; ++j) dst[at + (int64_t)state_channel(ct, q4b, j) * width] = convert(S[ct][j]);
        };
        if (w.ident) store_state(p.sm, [](float x) { return x; });
        else if (p.sf_bf16) store_state(static_cast<uint16_t *>(p.sf), [](float x) { return f32_to_bf16(x); });
        else store_state(static_cast<float *>(p.sf), [](float x) { return x; });
    }
}

}  // namespace gdn
}  // namespace kda
