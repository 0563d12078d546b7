// Attention of a few rows over a paged cache: single and drafted tokens of bf16 calls, all fp32 calls; and the kernel
// that joins the parts of long rows of cells.
//
// One pass over the cells with a running maximum m and sum l per row:  p_j = 2^(s_j - m),  o = sum p_j v_j / l.
//
// A tile is 16 rows (tokens x heads that share a key head), the width of the matrix instruction; a sequence has one or a few.  Four waves take the
// 32-cell quarters of each 128-cell block by themselves and are added at the end, so nothing is staged in LDS and
// the loop has no barrier: with few rows each cell is used once per wave, and the kernel is bound by the cache's bytes.
// fp32 calls with many rows are bound by the fp32 matrix instruction and by reading each cell once per 16 rows.
//
// Layouts (lane = 16 g + c).  S^T = K Q^T leaves lane (g, c) the scores of row c for cells 4 g + j of each 16: a lane holds
// 8 cells of one row, the contraction slots of the next product (which may come in any order), so P feeds O^T = V^T P^T
// from the registers it was computed in, statistics are per lane (cells meet across g twice a block, for m only), and
// the rescaling factor of a row belongs to the lane that holds the row's sums.  V^T needs 8 cells of one column in a
// lane: a lane loads d_v / 16 columns of its 8 cells (a cell's row is one run over 16 lanes) and pairs them up with
// byte permutes, one per two values.
//
// Measured (bf16, 32 query and 8 key heads of 128): 64 ragged contexts of up to 8,192 cells 202 us (5.4 TB/s of the cache), one
// of 131,072 cells 97 us (5.6 TB/s), 96 sequences of 4 tokens, 16 query heads and a window of 1,024 cells 72 us
// (5.6 TB/s); fp32, 4 x 1,024 tokens behind 4,096 cells, 16 heads: 1.8 ms (87 TFLOP/s of the 154 of a large product).
// fp32 of the ragged batch 447 us (4.9 TB/s), of the drafted one 149 (5.5 TB/s); its error is 2.5e-7 to 4.2e-7 of the output's norm,
// with the score's scale folded into the exponent of the hardware's exponential.
// Values are loaded past the caches' usual order, as nothing reads them twice: 216 -> 200 us for the ragged batch;
// keys, whose 128-byte lines are read by halves, gain nothing from it (204).
#include "kda_paged_work.h"

namespace kda {
namespace paged {
namespace {

constexpr int kM = 16, kKB = 128;

__device__ __forceinline__ float max_groups(float x) {  // over the lanes that differ in g
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// mfma_settle for all of a wave's sums: one wait, and every sum passes behind it.
template <int N>
__device__ __forceinline__ void settle(f32x4 (&o)[N]) {
    mfma_settle(o[0]);
#pragma unroll
    for (int i = 1; i < N; ++i) asm volatile("" : "+v"(o[i]));
}

// The keys, queries and values of a wave in either type.
template <typename IO, int DK, int DV>
struct Ops;

template <int DK, int DV>
struct Ops<uint16_t, DK, DV> {
    static constexpr int KK = DK / 32, VW = DV / 16;
    using Row = __attribute__((ext_vector_type(VW / 2))) unsigned;
    u32x4 q[KK], k[2][KK];
    Row v[8];
    __device__ __forceinline__ void load_q(const uint16_t *row, int g, bool live, bool flip) {
#pragma unroll
        for (int i = 0; i < KK; ++i) {
            q[i] = live ? *reinterpret_cast<const u32x4 *>(row + 32 * i + 8 * g) : u32x4{0, 0, 0, 0};
            if (flip) q[i] ^= 0x80008000u;
        }
    }
    // (base: the wave's, offset: a lane's, in 32 bits)
    __device__ __forceinline__ void load_k(int s, const char *base, unsigned offset) {
#pragma unroll
        for (int i = 0; i < KK; ++i) k[s][i] = *reinterpret_cast<const u32x4 *>(base + offset + 64 * i);
    }
    __device__ __forceinline__ void load_v(int j, const char *base, unsigned offset) {
        v[j] = __builtin_nontemporal_load(reinterpret_cast<const Row *>(base + offset));
    }
    __device__ __forceinline__ void clear_v(int j) { v[j] = Row(0u); }
    __device__ __forceinline__ bool odd_v(int j) const {  // infinities or NaN among them
        bool bad = false;
#pragma unroll
        for (int i = 0; i < VW / 2; ++i)
            bad |= (v[j][i] & 0x7f80u) == 0x7f80u || (v[j][i] & 0x7f800000u) == 0x7f800000u;
        return bad;
    }
    __device__ __forceinline__ f32x4 scores(int s) const {
        f32x4 a = zero4();
#pragma unroll
        for (int i = 0; i < KK; ++i)
            a = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k[s][i]), __builtin_bit_cast(bf16x8, q[i]), a,
                                                        0, 0, 0);
        return a;
    }
    __device__ __forceinline__ void add(f32x4 (&o)[VW], const float (&p)[8]) const {
        // p as two bf16 terms: one would add its rounding to the output's (2.3e-3 of the norm instead of 1.7e-3), and the
        // second product costs nothing beside the cache's bytes (204.2 us either way for the ragged batch).  The first is p cut
        // off and the second not quite the rest, so that both are above 0 where p is: an infinite value stays infinite.
        u32x4 hi, lo;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            hi[d] = __builtin_amdgcn_perm(__float_as_uint(p[2 * d + 1]), __float_as_uint(p[2 * d]), 0x07060302u);
            lo[d] = pack_bf16x2(fmaf(p[2 * d], 0x1p-60f, p[2 * d] - bf16_lo(hi[d])),
                                fmaf(p[2 * d + 1], 0x1p-60f, p[2 * d + 1] - bf16_hi(hi[d])));
        }
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            u32x4 a;
#pragma unroll
            for (int d = 0; d < 4; ++d)
                a[d] = __builtin_amdgcn_perm(v[2 * d + 1][i / 2], v[2 * d][i / 2], i & 1 ? 0x07060302u : 0x05040100u);
            o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, hi), o[i], 0, 0, 0);
            o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, lo), o[i], 0, 0, 0);
        }
    }
};

template <int DK, int DV>
struct Ops<float, DK, DV> {
    static constexpr int KK = DK / 16, VW = DV / 16;
    f32x4 q[KK], k[2][KK], v[8][VW / 4];
    __device__ __forceinline__ void load_q(const float *row, int g, bool live, bool flip) {
#pragma unroll
        for (int i = 0; i < KK; ++i) {
            q[i] = live ? *reinterpret_cast<const f32x4 *>(row + 16 * i + 4 * g) : zero4();
            if (flip) q[i] = -q[i];
        }
    }
    __device__ __forceinline__ void load_k(int s, const char *base, unsigned offset) {
#pragma unroll
        for (int i = 0; i < KK; ++i) k[s][i] = *reinterpret_cast<const f32x4 *>(base + offset + 64 * i);
    }
    __device__ __forceinline__ void load_v(int j, const char *base, unsigned offset) {
#pragma unroll
        for (int i = 0; i < VW / 4; ++i) v[j][i] = *reinterpret_cast<const f32x4 *>(base + offset + 16 * i);
    }
    __device__ __forceinline__ void clear_v(int j) {
#pragma unroll
        for (int i = 0; i < VW / 4; ++i) v[j][i] = zero4();
    }
    __device__ __forceinline__ bool odd_v(int j) const {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < VW; ++i) bad |= (__float_as_uint(v[j][i / 4][i % 4]) & 0x7f800000u) == 0x7f800000u;
        return bad;
    }
    __device__ __forceinline__ f32x4 scores(int s) const {
        f32x4 a = zero4();
#pragma unroll
        for (int i = 0; i < KK; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) a = __builtin_amdgcn_mfma_f32_16x16x4f32(k[s][i][e], q[i][e], a, 0, 0, 0);
        return a;
    }
    __device__ __forceinline__ void add(f32x4 (&o)[VW], const float (&p)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < VW; ++i) o[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(v[j][i / 4][i % 4], p[j], o[i], 0, 0, 0);
    }
};

// A wave's walk over its 16-cell groups: pages are looked up 64 groups at a time, a lane each, so that the loads of
// keys and values do not wait for a table entry each.
struct Pages {
    int entry;  // of group `lane` from the last refill on; -1: no page
    __device__ __forceinline__ void refill(const Cache &c, int n, int b, int wave, int lane, int hi, int b1) {
        const int bb = b + (lane >> 1), cell = bb * kKB + 32 * wave + 16 * (lane & 1);
        entry = -1;
        if (bb < b1 && cell < hi) {
            entry = c.table[n * c.table_ld + (cell >> c.page_shift)];
            if (entry >= c.num_pages) entry = -1;
        }
    }
    __device__ __forceinline__ int get(int i) const { return __builtin_amdgcn_readlane(entry, i & 63); }
};

// WG: workgroups that share a CU.
template <typename IO, int DK, int DV, int WG>
__global__ void __launch_bounds__(256, WG) attn_rows_kernel(AttnParams p) {
    constexpr int VW = DV / 16, PAD = DV + 4;
    __shared__ union {
        PlanLds plan;
        struct {
            float o[4][kM][PAD], m[4][kM], l[4][kM];
        } sum;
    } lds;
    Work w;
    if (!find_work<256>(p, kM, kKB, w, lds.plan)) return;
    const Cache &c = p.c;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4,
              col = lane & 15;

    Ops<IO, DK, DV> x;
    const int row = w.row0 + min(col, w.rows - 1);  // this lane's row
    const int token = p.by_G.by(row);
    const IO *q = static_cast<const IO *>(p.q) + (w.seq.t0 + token) * p.ldq + (w.head * p.G + (row - token * p.G)) * DK;
    x.load_q(q, g, col < w.rows, p.flip);
    const int pos = w.pos(row, p.by_G), from = w.first(pos, p.window);
    // cells that every row of the tile sees
    const int all_lo = w.first(w.pos(w.row0 + w.rows - 1, p.by_G), p.window), all_hi = min(w.pos(w.row0, p.by_G) + 1, w.cells);
    const bool ragged = all_lo != w.lo || all_hi != w.hi;  // rows see different cells
    const char *kp = reinterpret_cast<const char *>(static_cast<const IO *>(c.k) + w.head * c.k_head);
    const char *vp = reinterpret_cast<const char *>(static_cast<const IO *>(c.v) + w.head * c.v_head);
    const unsigned k_cell = (unsigned)c.k_cell * sizeof(IO), v_cell = (unsigned)c.v_cell * sizeof(IO);  // bytes
    const unsigned k_off = col * k_cell + 16 * g, v_off = 4 * g * v_cell + VW * sizeof(IO) * col;        // a lane's
    const int mask = (1 << c.page_shift) - 1;

    f32x4 o[VW];
#pragma unroll
    for (int i = 0; i < VW; ++i) o[i] = zero4();
    float m = -INFINITY, l = 0.f;
    OddBlocks odd_blocks;

    Pages pages;
    auto load_k = [&](int i, int b) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int page = pages.get(2 * i + s), cell = b * kKB + 32 * wave + 16 * s;
            const char *at = page < 0 ? kp : kp + page * c.k_page * (int64_t)sizeof(IO) + (uint64_t)((unsigned)(cell & mask) * k_cell);
            x.load_k(s, at, k_off);
        }
    };
    // this wave's quarters of the first and the last block may be out of sight
    const int b0 = w.b0 * kKB + 32 * wave + 32 > w.lo ? w.b0 : w.b0 + 1, b1 = (w.b1 - 1) * kKB + 32 * wave < w.hi ? w.b1 : w.b1 - 1;
    pages.refill(c, w.n, b0, wave, lane, w.hi, b1);
    if (b0 < b1) load_k(0, b0);
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        const int i = (b - b0) & 31, cell0 = b * kKB + 32 * wave;
        const int page0 = pages.get(2 * i), page1 = pages.get(2 * i + 1);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int page = s ? page1 : page0;
            const char *at =
                page < 0 ? vp : vp + page * c.v_page * (int64_t)sizeof(IO) + (uint64_t)((unsigned)((cell0 + 16 * s) & mask) * v_cell);
#pragma unroll
            for (int j = 0; j < 4; ++j) x.load_v(4 * s + j, at, v_off + j * v_cell);
        }
        f32x4 s0 = x.scores(0), s1 = x.scores(1);
        mfma_settle(s0, s1);
        // the next block's keys
        if (i == 31) pages.refill(c, w.n, b + 1, wave, lane, w.hi, b1);
        if (b + 1 < b1) load_k(i + 1, b + 1);
        const bool edge = page0 < 0 || page1 < 0 || cell0 < all_lo || cell0 + 32 > all_hi;
        const bool part = ragged && (cell0 < all_lo || cell0 + 32 > all_hi);  // some rows see what others do not
        bool odd = false;
        if (edge) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int cell = cell0 + (j < 4 ? 0 : 16) + 4 * g + (j & 3);
                const bool there = (j < 4 ? page0 : page1) >= 0 && cell < w.cells;
                if (!there || cell > pos || cell < from) (j < 4 ? s0 : s1)[j & 3] = -INFINITY;
                if (!there || cell >= w.hi || cell < w.lo) x.clear_v(j);
                if (part) odd |= x.odd_v(j);
            }
        }
        float t = fmaxf(fmaxf(fmaxf(s0[0], s0[1]), fmaxf(s0[2], s0[3])), fmaxf(fmaxf(s1[0], s1[1]), fmaxf(s1[2], s1[3])));
        t = max_groups(t) * p.scale;
        // the maximum is let run ahead by up to 2^8 before the sums are rescaled
        if (__any(t > m + 8.f)) {
            const float m1 = fmaxf(m, t), r = m1 == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - m1);
            m = m1;
            l *= r;
#pragma unroll
            for (int k = 0; k < VW; ++k) o[k] *= r;
        }
        const float base = m == -INFINITY ? 0.f : m;
        float e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            e[j] = __builtin_amdgcn_exp2f(fmaf(j < 4 ? s0[j & 3] : s1[j & 3], p.scale, -base));
            l += e[j];
        }
        if (__builtin_expect(part && __any(odd), 0)) {
            const int side = cell0 + 32 > all_hi;  // (at most two blocks at either end of a window: 16 rows are 16 tokens at most)
            odd_blocks.add(side, b);
        } else {
            x.add(o, e);
        }
        settle(o);
    }

    // Blocks with infinities or NaN in cells that some rows see and others do not: a weight of 0 does not hide them, so each row
    // adds only the cells that it sees, from memory.
#pragma unroll 1
    for (int i = 0; i < OddBlocks::kMost; ++i) {
        const int odd_block = odd_blocks.get(i);
        if (odd_block < 0) continue;
        const int cell0 = odd_block * kKB + 32 * wave;
#pragma unroll 1
        for (int cell = cell0; cell < cell0 + 32; ++cell) {
            const int page = cell < w.hi ? c.table[w.n * c.table_ld + (cell >> c.page_shift)] : -1;
            if (page < 0 || page >= c.num_pages || cell > pos || cell < from) continue;
            const IO *kr = reinterpret_cast<const IO *>(kp) + page * c.k_page + (cell & mask) * c.k_cell;
            const IO *vr = reinterpret_cast<const IO *>(vp) + page * c.v_page + (cell & mask) * c.v_cell;
            float z = 0.f;
#pragma unroll 1
            for (int j = 0; j < DK; ++j) z = fmaf(IoTraits<IO>::load1(q + j), IoTraits<IO>::load1(kr + j), z);
            const float weight = __builtin_amdgcn_exp2f(fmaf(p.flip ? -z : z, p.scale, -m));
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int y = 0; y < VW; ++y) o[y][r] = fmaf(weight, IoTraits<IO>::load1(vr + VW * (4 * g + r) + y), o[y][r]);
        }
    }

    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    __syncthreads();  // the plan's LDS has been read
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < VW; i += 4)
            *reinterpret_cast<f32x4 *>(&lds.sum.o[wave][col][VW * (4 * g + r) + i]) =
                f32x4{o[i][r], o[i + 1][r], o[i + 2][r], o[i + 3][r]};
    if (g == 0) {
        lds.sum.m[wave][col] = m;
        lds.sum.l[wave][col] = l;
    }
    __syncthreads();
    const int out = tid >> 4, c16 = tid & 15;
    float top = -INFINITY, sum = 0.f, y[VW];
#pragma unroll
    for (int k = 0; k < 4; ++k) top = fmaxf(top, lds.sum.m[k][out]);
#pragma unroll
    for (int i = 0; i < VW; ++i) y[i] = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float r = top == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(lds.sum.m[k][out] - top);
        sum = fmaf(lds.sum.l[k][out], r, sum);
#pragma unroll
        for (int i = 0; i < VW; ++i) y[i] = fmaf(lds.sum.o[k][out][VW * c16 + i], r, y[i]);
    }
    put_row<IO, DV, kM>(p, w, out, c16, y, top, sum);
}

// Joins the splits of a tile (4 us, of which the launch is most).  Bound: the latency of reading them, so a row's splits go to
// 256 / (RJ * DV / 4) groups of threads side by side, RJ rows at a time.  There is a workgroup for every RB rows of the most tiles there can be: one row where a
// few tiles have 16; four where there are many of them, and 32 of 256, since then mostly no tile is split, or in two, and what the
// workgroups cost is their number (131,072 of them 40 us; four rows instead of one for 64 ragged contexts: 204.5 -> 200.7 us).
template <typename IO, int DV, int RJ, int RB>
__global__ void __launch_bounds__(256) attn_join_kernel(AttnParams p, int M) {
    constexpr int LPR = DV / 4, SG = 256 / (RJ * LPR);
    static_assert(SG >= 1 && RB % RJ == 0);
    const int per = M / RB;
    const int64_t tile = blockIdx.x / (unsigned)per;
    const int chunk = blockIdx.x % (unsigned)per;
    if (tile >= (int64_t)p.desc[0] * p.Hk) return;
    const int32_t *d = p.desc + kDesc * (1 + tile);
    const int n = d[0], head = d[1], row0 = d[2], rows = d[3], splits = d[4];
    const int tid = threadIdx.x, lane = tid % LPR, sg = tid / LPR % SG, rj = tid / (LPR * SG);
    // (what no workgroup has written, as offsets that overlap leave it, is no row either)
    if (n < 0 || n >= p.c.num_seqs || head < 0 || head >= p.Hk || row0 < 0 || rows > M || splits < 2 || d[5] < 0 ||
        d[5] > p.slots - splits || chunk * RB >= rows)
        return;
    const Seq s = sequence(p.c, n);
    if (row0 > s.len * p.G - rows) return;
    const int64_t stride = (int64_t)p.Hk * M * (DV + 2);
    const float *part = p.part + ((int64_t)d[5] * p.Hk + head) * M * (DV + 2);
    __shared__ float so[SG][RJ][DV + 4], sm[SG][RJ], sl[SG][RJ];
#pragma unroll 1
    for (int row = chunk * RB + rj; row - rj < min(chunk * RB + RB, rows); row += RJ) {
        float m = -INFINITY, l = 0.f;
        f32x4 o = zero4();
        if (row < rows) {
#pragma unroll 4
            for (int i = sg; i < splits; i += SG) {
                const float *q = part + i * stride;
                const f32x4 v = *reinterpret_cast<const f32x4 *>(q + row * DV + 4 * lane);
                const float ms = q[M * DV + row], ls = q[M * DV + M + row];
                const float m1 = fmaxf(m, ms), base = m1 == -INFINITY ? 0.f : m1;
                const float a = __builtin_amdgcn_exp2f(m - base), b = __builtin_amdgcn_exp2f(ms - base);
                m = m1;
                l = l * a + ls * b;
                o = o * a + v * b;
            }
        }
        if constexpr (SG > 1) {
            if (row - rj > chunk * RB) __syncthreads();  // the last rows' have been read
            *reinterpret_cast<f32x4 *>(&so[sg][rj][4 * lane]) = o;
            if (lane == 0) {
                sm[sg][rj] = m;
                sl[sg][rj] = l;
            }
            __syncthreads();
            if (sg == 0) {
#pragma unroll
                for (int k = 1; k < SG; ++k) m = fmaxf(m, sm[k][rj]);
                const float base = m == -INFINITY ? 0.f : m;
                l = 0.f;
                o = zero4();
#pragma unroll
                for (int k = 0; k < SG; ++k) {
                    const float a = __builtin_amdgcn_exp2f(sm[k][rj] - base);
                    l += sl[k][rj] * a;
                    o += *reinterpret_cast<const f32x4 *>(&so[k][rj][4 * lane]) * a;
                }
            }
        }
        if (row < rows && sg == 0) {
            const int64_t at = out_row(p, s, head, row0 + row);
            const float r = l == 0.f ? 0.f : 1.f / l;
            IoTraits<IO>::store4(static_cast<IO *>(p.out) + at * DV + 4 * lane, make_float4(o[0] * r, o[1] * r, o[2] * r, o[3] * r));
            if (p.lse && lane == 0) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        }
    }
}

template <typename IO, int WG, int WGL>
hipError_t rows(const AttnParams &p, dim3 grid, hipStream_t s) {
    const dim3 block(256);
    if (p.dk == 128 && p.dv == 128) hipLaunchKernelGGL((attn_rows_kernel<IO, 128, 128, WGL>), grid, block, 0, s, p);
    if (p.dk == 128 && p.dv == 64) hipLaunchKernelGGL((attn_rows_kernel<IO, 128, 64, WG>), grid, block, 0, s, p);
    if (p.dk == 64 && p.dv == 128) hipLaunchKernelGGL((attn_rows_kernel<IO, 64, 128, WG>), grid, block, 0, s, p);
    if (p.dk == 64 && p.dv == 64) hipLaunchKernelGGL((attn_rows_kernel<IO, 64, 64, WG>), grid, block, 0, s, p);
    return hipGetLastError();
}

template <typename IO, int RJ, int RB>
hipError_t join(const AttnParams &p, int M, int64_t tiles, hipStream_t s) {
    const dim3 grid((unsigned)(tiles * p.Hk * (M / RB))), block(256);
    if (p.dv == 128)
        hipLaunchKernelGGL((attn_join_kernel<IO, 128, RJ, RB>), grid, block, 0, s, p, M);
    else
        hipLaunchKernelGGL((attn_join_kernel<IO, 64, RJ, RB>), grid, block, 0, s, p, M);
    return hipGetLastError();
}

}  // namespace

// Parts: of at least two blocks of 128 cells in bf16 (a block takes a wave about 1 us, the join 4: with one block a part 512 to
// 4,096 cells of one sequence take 10.0 to 10.3 us instead of 11.1 to 11.6, 256 cells 9.9 instead of
// 9.1: for a lone sequence one would be better from 512 on) and one in fp32, whose
// block takes twice as long (1,002 cells 16.0 -> 13.0 us); for two workgroups per CU: one leaves the ends of ragged batches to few (220
// us instead of 205), three make more parts than the cache's bandwidth needs (131,072 cells: 94 us instead of 89, the
// batch 200).  Three workgroups of the bf16 kernel fit a CU.
AttnTile attn_rows_tile(bool bf16) { return {kM, kKB, bf16 ? 2 : 1, 2, 256}; }

hipError_t launch_attn_rows(bool bf16, bool many, const AttnParams &p, int64_t blocks, hipStream_t stream) {
    if (blocks <= 0) return hipSuccess;
    const dim3 grid((unsigned)blocks);
    if (bf16) return rows<uint16_t, 3, 3>(p, grid, stream);
    return many ? rows<float, 2, 1>(p, grid, stream) : rows<float, 2, 2>(p, grid, stream);
}

hipError_t launch_attn_join(bool bf16, const AttnParams &p, int M, int64_t tiles, hipStream_t stream) {
    if (tiles <= 0) return hipSuccess;
    if (M > kM) return join<uint16_t, 8, 32>(p, M, tiles, stream);
    if (tiles * p.Hk >= 256) return bf16 ? join<uint16_t, 4, 4>(p, M, tiles, stream) : join<float, 4, 4>(p, M, tiles, stream);
    return bf16 ? join<uint16_t, 1, 1>(p, M, tiles, stream) : join<float, 1, 1>(p, M, tiles, stream);
}

}  // namespace paged
}  // namespace kda
