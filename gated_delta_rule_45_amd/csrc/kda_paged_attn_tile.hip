// Attention of many rows over a paged cache (chunks and whole prompts, bf16): tiles of 256 rows.
//
// Bound: the SIMDs' issue of matrix and vector instructions.  Eight waves own 32 rows each and share 64-cell blocks of
// keys and values in LDS; with 2 (d_k + d_v) flops per row and cell a block costs 2,048 cycles of a CU's matrix units, and about as
// many of its vector units for the softmax (an exponential is a quarter-rate instruction), so the two have to run side by
// side: the waves 0-3 and 4-7, one of each on every SIMD, take turns, half an iteration apart: while one group multiplies
// (O += P V of block t, then S = K Q^T of block t + 1), the other starts the loads of later blocks and works out the
// weights of its own.  A barrier ends each half.  Keys are staged three blocks ahead of their use, values two, in rings of four buffers.
//
// Layouts (lane = 32 h + r).  S^T = K Q^T and O^T = V^T P^T as in the kernel for few rows, here as 32 x 32 tiles: a
// lane holds the scores of row r for cells 8 a + 4 h + b of each 32, which are the contraction slots of the next product as they
// are.  V^T comes from LDS through the transposing read (4 cells of one column per lane).  Direct global-to-LDS loads
// place lane l's 16 bytes at 16 l, so rows are scattered over the banks by which bytes a lane fetches: 16-byte
// pieces of keys move by row mod 16 (by half of that where two rows make 256 bytes), 32-byte pieces of values, what 16
// lanes read of a row, by row mod 4: neither then meets a bank twice in the 256 bytes that LDS gives in a cycle.
//
// Weights are rounded to bf16 for their product (error of the output 2.1 to 2.5e-3 of its norm, 1.7e-3 of that its own
// rounding): a second term, as in the kernel for few rows, would add half as many products again.
//
// Measured (32 query and 8 key heads of 128): 4 prompts of 4,096 tokens 565 us, 973 TFLOP/s, and 580 on a second card (a large
// matrix product: 1,378; matrix units busy 46 % of the time, waves waiting 25 %), 6 chunks of 1,024 tokens behind 16,384 cells 1.60 ms, 1,064 TFLOP/s;
// the prompts under a window of 1,024 cells 326 us, 737 TFLOP/s; d_k = d_v = 64: 780 TFLOP/s (the same softmax for half the products).  A half iteration takes 1,600 to 1,700 cycles of
// the 1,024 that its products need.  What it took, on the prompts: products in one run with their LDS reads ten ahead and the
// weights kept before them (678 -> 634 us; weights left to sink between the products: 738; six or fourteen reads ahead: 2 and
// 1 % slower), a bank-free order of the keys (630 -> 615), one base address per load (with one per lane 655, else 600).  Loads
// between the products cost more than they hide (610).  A workgroup's start (plan,
// first blocks) is 10,000 of its 140,000 cycles: one fills a CU, so nothing covers it.
#include <type_traits>

#include "kda_paged_work.h"

namespace kda {
namespace paged {
namespace {

constexpr int kM = 256, kKB = 64, kNT = 512, kRing = 4, kAhead = 10;
typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(2))) unsigned u32x2;

// Position of 16-byte piece c of row r in LDS, and back (both ways are the same exchange).
template <int D>
__device__ __forceinline__ int k_place(int r, int c) { return c ^ (D == 128 ? r & 15 : (r >> 1) & 7); }
template <int D>
__device__ __forceinline__ int v_place(int r, int c) { return c ^ ((D == 128 ? r & 3 : (r >> 1) & 1) << 2); }

// load_lds16 whose end is left to wait_vmcnt and a barrier: the compiler, which cannot tell the buffers of a ring apart, would
// wait for the builtin's loads before every LDS read.  `to`: the wave's address in LDS, for M0, which must be set a cycle
// before.  Nothing here tells the compiler that LDS is written, so that it may move LDS reads of other buffers past it: the
// barriers, which are volatile like this, keep it in its half iteration.
__device__ __forceinline__ unsigned lds_address(const void *p) {
    return __builtin_amdgcn_readfirstlane((unsigned)(uintptr_t)(const __attribute__((address_space(3))) void *)p);
}
__device__ __forceinline__ void load_lds16_async(const void *base, unsigned offset, unsigned to) {  // base: the wave's, offset: a lane's
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %0" ::"s"(base), "v"(offset), "s"(to));
}

template <int DK, int DV>
struct Lds {
    uint16_t k[kRing][kKB * DK], v[kRing][kKB * DV];
    unsigned missing[kRing];  // a byte per 16 cells: page does not exist
    PlanLds plan;
};

template <int DK, int DV>
__global__ void __launch_bounds__(kNT, 1) attn_tile_kernel(AttnParams p) {
    constexpr int KS = DK / 16, DB = DV / 32;                    // steps of a score, column blocks of the output
    constexpr int KC = DK / 8, VC = DV / 8;                      // 16-byte pieces of a row
    constexpr int KI = kKB * KC / kNT, VI = kKB * VC / kNT;      // loads of a wave per block
    constexpr int KR = 64 / KC, VR = 64 / VC;                    // rows of a load
    __shared__ Lds<DK, DV> lds;
    Work w;
    if (!find_work<kNT>(p, kM, kKB, w, lds.plan)) return;
    const Cache &c = p.c;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 31, h = lane >> 5;

    // this wave's rows
    const int wrow = min(wave * 32, w.rows - 1), wlast = min(wave * 32 + 31, w.rows - 1), row = w.row0 + min(wave * 32 + r, w.rows - 1);
    const bool active = wave * 32 < w.rows;
    const int pos = w.pos(row, p.by_G), from = w.first(pos, p.window), last = min(pos, w.cells - 1);
    const int pos0 = w.pos(w.row0 + wrow, p.by_G), pos1 = w.pos(w.row0 + wlast, p.by_G);
    const int see_lo = w.first(pos0, p.window), see_hi = active ? min(pos1 + 1, w.cells) : 0;   // some row
    const int all_lo = w.first(pos1, p.window), all_hi = min(pos0 + 1, w.cells);                // every row
    const int token = p.by_G.by(row);
    const uint16_t *x = static_cast<const uint16_t *>(p.q) + (w.seq.t0 + token) * p.ldq + (w.head * p.G + (row - token * p.G)) * DK;

    // ---- staging
    const char *kp = reinterpret_cast<const char *>(static_cast<const uint16_t *>(c.k) + w.head * c.k_head);
    const char *vp = reinterpret_cast<const char *>(static_cast<const uint16_t *>(c.v) + w.head * c.v_head);
    const __attribute__((address_space(4))) int32_t *table =
        (const __attribute__((address_space(4))) int32_t *)(c.table + w.n * c.table_ld);
    const int mask = (1 << c.page_shift) - 1;
    const int nt = w.b1 - w.b0;
    // A wave loads rows 8 wave .. 8 wave + 7 of every block, of keys and of values: one page.  ek, ev: table entries of
    // the next blocks' loads, read an iteration ahead.
    const int row8 = 8 * wave;
    int ek = -1, ev = -1, e1 = -1;  // of the next keys, the next values, the values before those
    auto look = [&](int t) { return table[min((unsigned)(w.b0 + t) * kKB + row8, (unsigned)w.hi - 1) >> c.page_shift]; };
    unsigned k_off[KI], v_off[VI];  // bytes of a lane's piece from the wave's first cell
#pragma unroll
    for (int i = 0; i < KI; ++i) {
        const int rr = KR * i + lane / KC;
        k_off[i] = (unsigned)(rr * c.k_cell) * 2 + 16 * k_place<DK>(row8 + rr, lane % KC);
    }
#pragma unroll
    for (int i = 0; i < VI; ++i) {
        const int rr = VR * i + lane / VC;
        v_off[i] = (unsigned)(rr * c.v_cell) * 2 + 16 * v_place<DV>(row8 + rr, lane % VC);
    }
    const unsigned k_lds = lds_address(&lds.k[0][row8 * DK]), v_lds = lds_address(&lds.v[0][row8 * DV]);
    const int64_t k_page = c.k_page * 2, v_page = c.v_page * 2;  // bytes
    const unsigned k_cell = (unsigned)c.k_cell * 2, v_cell = (unsigned)c.v_cell * 2;
    // Loads of a wave's rows of block t from page e.  No branch and no address of a lane's own: where the page does not exist they read
    // page 0, behind the last cell what the last page holds there.  Scores of such cells are replaced; values are cleared.
    auto fetch = [&](auto &off, const char *pool, int64_t page, unsigned cell_bytes, int e, int t, unsigned to) {
        constexpr int N = sizeof(off) / sizeof(off[0]);
        const char *base = pool + (int64_t)((unsigned)e < (unsigned)c.num_pages ? e : 0) * page +
                           (uint64_t)(((unsigned)((w.b0 + t) * kKB + row8) & mask) * cell_bytes);
#pragma unroll
        for (int i = 0; i < N; ++i) load_lds16_async(base, off[i], to + 1024 * i);
    };
    auto stage_k = [&](int t) { fetch(k_off, kp, k_page, k_cell, ek, t, k_lds + t % kRing * (kKB * DK * 2)); };
    auto stage_v = [&](int t) { fetch(v_off, vp, v_page, v_cell, ev, t, v_lds + t % kRing * (kKB * DV * 2)); };
    auto mark = [&](int t) {
        if (lane == 0)
            reinterpret_cast<uint8_t *>(&lds.missing[t % kRing])[wave / 2] = (unsigned)ek >= (unsigned)c.num_pages;
    };
    // Zeros over the values of this wave's cells of block t (page e) that are not there or out of every row's sight: a weight of 0
    // would not hide what lies there.
    auto clear = [&](int t, int e) {
        const unsigned cell0 = (unsigned)(w.b0 + t) * kKB + row8;
        if ((unsigned)e < (unsigned)c.num_pages && cell0 >= (unsigned)w.lo && cell0 + 8 <= (unsigned)w.hi) return;
        const unsigned seen = (unsigned)e < (unsigned)c.num_pages ? w.hi - w.lo : 0;
#pragma unroll
        for (int i = 0; i < VI; ++i)
            if (cell0 + VR * i + lane / VC - w.lo >= seen)
                *reinterpret_cast<u32x4 *>(&lds.v[t % kRing][row8 * DV + 512 * i + 8 * lane]) = u32x4{0, 0, 0, 0};
    };

    u32x4 q[KS];
    f32x16 s[2], o[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i) o[i] = f32x16(0.f);
    u32x4 pw[4];
    float m = -INFINITY, l = 0.f;

    auto scores = [&](int t) {  // S^T of block t
        const uint16_t *k = lds.k[t % kRing];
        s[0] = f32x16(0.f);
        s[1] = f32x16(0.f);
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int rr = 32 * b + r;
                const u32x4 x = *reinterpret_cast<const u32x4 *>(k + rr * DK + 8 * k_place<DK>(rr, 2 * i + h));
                s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, q[i]), s[b],
                                                               0, 0, 0);
            }
    };
    auto value = [&](const uint16_t *v, int step, int db) {  // V^T: 32 columns, 16 cells
        u32x4 x;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int rr = 16 * step + 8 * y + 4 * h + (lane & 15) / 4, piece = 4 * db + ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
            const uint16_t *at = v + rr * DV + 8 * v_place<DV>(rr, piece) + 4 * (lane & 1);
            const u32x2 z = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                          (__attribute__((address_space(3))) s16x4 *)at));
            x[2 * y] = z[0];
            x[2 * y + 1] = z[1];
        }
        return x;
    };
    auto add = [&](int t) {  // O^T += V^T P^T of block t
        const uint16_t *v = lds.v[t % kRing];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int b = 0; b < DB; ++b)
                o[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, value(v, i, b)),
                                                               __builtin_bit_cast(bf16x8, pw[i]), o[b], 0, 0, 0);
    };
    auto edge = [&](int t, unsigned missing) {
        const int c0 = (w.b0 + t) * kKB;
        return c0 < all_lo || c0 + kKB > all_hi || missing != 0;
    };
    auto odd = [&](int t) {
        const uint16_t *v = lds.v[t % kRing];
        bool bad = false;
        for (int i = 0; i < kKB * DV / 8 / 64; ++i) {
            const u32x4 x = reinterpret_cast<const u32x4 *>(v)[i * 64 + lane];
#pragma unroll
            for (int y = 0; y < 4; ++y) bad |= (x[y] & 0x7f80u) == 0x7f80u || (x[y] & 0x7f800000u) == 0x7f800000u;
        }
        return __any(bad);
    };
    auto settle = [&]() {
        asm volatile("s_nop 7\n\ts_nop 3" : "+v"(s[0]), "+v"(s[1]));
#pragma unroll
        for (int i = 0; i < DB; ++i) asm volatile("" : "+v"(o[i]));
    };
    auto weights = [&](int t, unsigned missing) {
        if (edge(t, missing)) {
            const int c0 = (w.b0 + t) * kKB + 4 * h, to = last - c0, at = from - c0;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                    const int k = 32 * b + 8 * (y >> 2) + (y & 3);
                    const bool see = (k <= to) & (k >= at);
                    s[b][y] = see ? s[b][y] : -INFINITY;
                }
            if (missing)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int y = 0; y < 16; ++y) s[b][y] = missing >> (8 * (2 * b + (y >> 3))) & 0xff ? -INFINITY : s[b][y];
        }
        float top = fmaxf(s[0][0], s[1][0]);
#pragma unroll
        for (int y = 1; y < 16; ++y) top = fmaxf(fmaxf(top, s[0][y]), s[1][y]);
        const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
        top = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1])) * p.scale;
        // the maximum is let run ahead by up to 2^8 before the sums are rescaled
        if (__any(top > m + 8.f)) {
            const float m1 = fmaxf(m, top), f = m1 == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - m1);
            m = m1;
            l *= f;
#pragma unroll
            for (int b = 0; b < DB; ++b) o[b] *= f;
        }
        const float base = m == -INFINITY ? 0.f : m;
        float sum[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float e[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                e[y] = __builtin_amdgcn_exp2f(fmaf(s[i >> 1][8 * (i & 1) + y], p.scale, -base));
                sum[y & 3] = i == 0 && y < 4 ? e[y] : sum[y & 3] + e[y];
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) pw[i][y] = pack_bf16x2(e[2 * y], e[2 * y + 1]);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    };
    // at most N of this wave's loads are on their way; LDS is touched behind that, not before
    auto landed = [&](auto n) {
        wait_vmcnt<decltype(n)::value>();
        asm volatile("" ::: "memory");
    };
    // this wave's LDS accesses are done, its loads from memory may be on their way (a fence would wait for those too)
    auto barrier = [&]() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };

    if (nt > 0) {
        const int e0 = look(0), e2 = look(2);
        e1 = look(1);
        ek = e0, stage_k(0), mark(0);
        ev = e0, stage_v(0);
        ek = e1, stage_k(1), mark(1);
        ev = e1, stage_v(1);
        ek = e2, stage_k(2), mark(2);
        landed(std::integral_constant<int, 0>());
        clear(0, e0);
        ev = e2;  // of block 2, ek: of block 3
        ek = look(3);
    }
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        q[i] = *reinterpret_cast<const u32x4 *>(x + 16 * i + 8 * h);
        if (p.flip) q[i] ^= 0x80008000u;
    }
    barrier();
    const bool second = wave >= 4;
    if (second) barrier();
    unsigned gone = lds.missing[0];
    if (nt > 0) scores(0);
    settle();
    barrier();
    OddBlocks odd_blocks;
    // (A wave none of whose rows sees a block goes through it all the same, with weights of 0: it has to wait for the others anyway.)
#pragma unroll 1
    for (int t = 0; t < nt; ++t) {
        const unsigned missing = __builtin_amdgcn_readfirstlane(gone);
        gone = lds.missing[(t + 1) % kRing];
        stage_k(t + 3);
        mark(t + 3);
        stage_v(t + 2);
        weights(t, missing);
#pragma unroll
        for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(pw[i]));  // worked out here, not between the products
        asm volatile("" : "+v"(l));
        barrier();
        const int c0 = (w.b0 + t) * kKB;
        bool apart = false;
        if ((c0 < all_lo || c0 + kKB > all_hi) && odd(t)) {
            apart = true;
            if (c0 < see_hi && c0 + kKB > see_lo) {  // (at most two blocks at either end of a window: 32 rows are 32 tokens at most)
                odd_blocks.add(c0 + kKB > all_hi, t);
            }
        }
        if (__builtin_expect(!apart, 1)) {
            // both products in one run, each operand read from LDS kAhead reads before its product (behind the last block the
            // scores are of whatever lies in the ring and are not looked at)
            __builtin_amdgcn_s_setprio(1);
            add(t);
            scores(t + 1);
            __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
            for (int i = 0; i < 4 * DB; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            }
#pragma unroll
            for (int i = 0; i < 2 * KS; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
        } else {
            scores(t + 1);
        }
        settle();
        __builtin_amdgcn_s_setprio(0);
        // the loads that this half iteration started may go on; all others are there for everyone behind the barrier
        landed(std::integral_constant<int, KI + VI>());
        clear(t + 1, e1);
        e1 = ev;
        ev = ek;
        ek = look(t + 4);
        barrier();
    }
    wait_vmcnt<0>();
    if (!second) barrier();

    // Blocks with infinities or NaN in cells that some rows see and others do not: a weight of 0 does not hide them, so each row
    // adds only the cells that it sees, from memory.
#pragma unroll 1
    for (int i = 0; i < OddBlocks::kMost; ++i) {
        const int odd_block = odd_blocks.get(i);
        if (odd_block < 0) continue;
        const int c0 = (w.b0 + odd_block) * kKB;
#pragma unroll 1
        for (int k = 0; k < kKB; ++k) {
            const int cell = c0 + k, e = cell < w.hi ? table[cell >> c.page_shift] : -1;
            if (e < 0 || e >= c.num_pages || cell > last || cell < from) continue;
            const uint16_t *kr = reinterpret_cast<const uint16_t *>(kp) + e * c.k_page + (cell & mask) * c.k_cell;
            const uint16_t *vr = reinterpret_cast<const uint16_t *>(vp) + e * c.v_page + (cell & mask) * c.v_cell;
            float z = 0.f;
#pragma unroll 1
            for (int j = 0; j < DK; ++j) z = fmaf(bf16_to_f32(x[j]), bf16_to_f32(kr[j]), z);
            const float weight = __builtin_amdgcn_exp2f(fmaf(p.flip ? -z : z, p.scale, -m));
#pragma unroll
            for (int b = 0; b < DB; ++b)
#pragma unroll
                for (int y = 0; y < 16; ++y)
                    o[b][y] = fmaf(weight, bf16_to_f32(vr[32 * b + 8 * (y >> 2) + 4 * h + (y & 3)]), o[b][y]);
        }
    }

    l += __shfl_xor(l, 32, 64);
    if (wave * 32 + r >= w.rows) return;
    if (w.splits > 1) {
        float *part = p.part + w.slot * (int64_t)(kM * (DV + 2));
        const int at = wave * 32 + r;
#pragma unroll
        for (int b = 0; b < DB; ++b)
#pragma unroll
            for (int a = 0; a < 4; ++a)
                *reinterpret_cast<f32x4 *>(part + at * DV + 32 * b + 8 * a + 4 * h) =
                    f32x4{o[b][4 * a], o[b][4 * a + 1], o[b][4 * a + 2], o[b][4 * a + 3]};
        if (h == 0) {
            part[kM * DV + at] = m;
            part[kM * DV + kM + at] = l;
        }
        return;
    }
    const int64_t at = out_row(p, w.seq, w.head, row);
    const float f = l == 0.f ? 0.f : 1.f / l;
    uint16_t *y = static_cast<uint16_t *>(p.out) + at * DV + 4 * h;
#pragma unroll
    for (int b = 0; b < DB; ++b)
#pragma unroll
        for (int a = 0; a < 4; ++a)
            IoTraits<uint16_t>::store4(y + 32 * b + 8 * a, make_float4(o[b][4 * a] * f, o[b][4 * a + 1] * f, o[b][4 * a + 2] * f,
                                                                       o[b][4 * a + 3] * f));
    if (p.lse && h == 0) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

// Parts of at least eight blocks, 512 cells: a part's sums (256 rows of d_v fp32) are then small beside its work (1 x 1,024 tokens:
// 40 us, of at least four blocks 52); for two workgroups per CU, although one fills it (one: attention of chunks 664 us instead of 650)
AttnTile attn_tile_tile() { return {kM, kKB, 8, 2, kNT}; }

hipError_t launch_attn_tile(const AttnParams &p, int64_t blocks, hipStream_t s) {
    if (blocks <= 0) return hipSuccess;
    const dim3 grid((unsigned)blocks), block(kNT);
    if (p.dk == 128 && p.dv == 128) hipLaunchKernelGGL((attn_tile_kernel<128, 128>), grid, block, 0, s, p);
    if (p.dk == 128 && p.dv == 64) hipLaunchKernelGGL((attn_tile_kernel<128, 64>), grid, block, 0, s, p);
    if (p.dk == 64 && p.dv == 128) hipLaunchKernelGGL((attn_tile_kernel<64, 128>), grid, block, 0, s, p);
    if (p.dk == 64 && p.dv == 64) hipLaunchKernelGGL((attn_tile_kernel<64, 64>), grid, block, 0, s, p);
    return hipGetLastError();
}

}  // namespace paged
}  // namespace kda
