// Which rows and cells a workgroup of the attention kernels takes.
//
// Lengths are on the device only, and range from one cell to a long document within a batch, so every workgroup
// works out the plan for itself: the blocks of all tiles are summed, cut into parts of c = max(c_min, sum / target)
// blocks (so that about `target` workgroups have equal parts whatever the lengths are), and a prefix sum over the
// sequences finds the part that the workgroup's number stands for.  That costs two passes over the lengths, one load
// each for as many sequences as threads, and needs no launch of its own.  The head is the number's fastest part: workgroups go round robin to the 8 XCDs,
// so that with 8 heads the tiles of a head read its cells through one L2.
#pragma once

#include "kda_device.h"
#include "kda_paged.h"

namespace kda {
namespace paged {

struct Seq {
    int64_t t0;  // first token
    int len;     // new tokens
    int kv;      // cells with them, as given (>= 0)
};
__device__ __forceinline__ Seq sequence(const Cache &c, int n) {
    Seq s;
    if (c.cu) {
        const int a = min(max(c.cu[n], 0), c.T), b = min(max(c.cu[n + 1], a), c.T);
        s.t0 = a;
        s.len = b - a;
    } else {
        s.t0 = (int64_t)n * c.T;
        s.len = c.T;
    }
    s.kv = max(c.lens[n], 0);
    return s;
}

struct Work {
    Seq seq;
    int n, head, row0, rows;  // rows of the tile: row0 .. row0 + rows - 1 of the sequence
    int split, splits;        // this workgroup's part of the tile
    int64_t slot;             // where its sums go, if splits > 1
    int cells, lo, hi;        // cells that exist; those that some row of the tile sees
    int b0, b1;               // blocks of KB cells of this part
    __device__ __forceinline__ int pos(int row, const Div &by_G) const { return seq.kv - seq.len + by_G.by(row); }
    // (a position of -len .. 2^31 - 1: no overflow)
    __device__ __forceinline__ int first(int pos, int window) const {
        return window > 0 && pos >= window ? pos - window + 1 : 0;
    }
};

// Most blocks that a tile of the sequence can see: what its tiles are cut by.
__device__ __forceinline__ int blocks_bound(const AttnParams &p, const Seq &s, int M, int KB, int cells) {
    const int all = (min(s.kv, cells) + KB - 1) / KB;
    if (p.window <= 0) return all;
    const int64_t seen = (int64_t)p.window + p.by_G.by(M - 1) + 1;  // by all tokens of a tile, from some cell of a block
    return (int)min((int64_t)all, (seen + KB - 1) / KB + 1);
}

// Inclusive prefix sum over a wave: rows of 16 lanes, then each row's last lane to the next rows.
__device__ __forceinline__ int wave_scan(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);
    return x;
}
// ceil(a / b) of non-negative numbers; most sums fit 32 bits, whose division is a tenth of the other's
__device__ __forceinline__ long long ceil_div(long long a, int b) {
    a += b - 1;
    return a >> 32 ? a / b : (long long)((unsigned)a / (unsigned)b);
}

constexpr int kPlanWaves = 8;  // at most
struct PlanLds {
    unsigned long long total;
    int sums[kPlanWaves][3];
    int found[6];  // sequence, part within it, splits, first slot, first split tile, split tiles in all
};

// The workgroup's part; false: none.  NT threads, all of them call.
template <int NT>
__device__ __forceinline__ bool find_work(const AttnParams &p, int M, int KB, Work &w, PlanLds &lds) {
    const Cache &c = p.c;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int part = p.by_Hk.by(blockIdx.x);
    w.head = blockIdx.x - part * p.Hk;
    w.cells = c.num_pages > 0 ? c.max_pages << c.page_shift : 0;
    int at, splits, slot0 = 0, tile0 = 0;  // part of its sequence
    if (p.c_min == 0) {
        const int tiles = (c.T * p.G + M - 1) / M;
        w.n = part / tiles;
        at = part % tiles;
        splits = 1;
        if (w.n >= c.num_seqs) return false;
    } else {
        struct Share {
            int rows = 0, blocks = 0;  // of a sequence, rows 0: none of this launch
        };
        auto share = [&](int n) {
            Share x;
            if (n < c.num_seqs) {
                const Seq s = sequence(c, n);
                const int rows = s.len * p.G;
                if (rows >= p.rows_lo && rows <= p.rows_hi) {
                    x.rows = rows;
                    x.blocks = blocks_bound(p, s, M, KB, w.cells);
                }
            }
            return x;
        };
        if (tid == 0) {
            lds.total = 0;
            lds.found[0] = -1;
        }
        const Share mine0 = share(tid);
        unsigned long long cost = (unsigned long long)((mine0.rows + M - 1) / M) * mine0.blocks;
        for (int n = tid + NT; n < c.num_seqs; n += NT) {
            const Share x = share(n);
            cost += (unsigned long long)((x.rows + M - 1) / M) * x.blocks;
        }
        __syncthreads();
        if (cost) atomicAdd(&lds.total, cost);
        __syncthreads();
        const int cut = (int)max((long long)p.c_min, ceil_div((long long)lds.total * p.Hk, p.target));
        int parts = 0, slots = 0, stiles = 0;  // of the sequences so far
        for (int n0 = 0; n0 < c.num_seqs; n0 += NT) {
            const Share x = n0 == 0 ? mine0 : share(n0 + tid);
            const int tiles = (x.rows + M - 1) / M, cuts = x.blocks > cut ? (int)((unsigned)(x.blocks + cut - 1) / (unsigned)cut) : 1;
            const int v[3] = {tiles * cuts, cuts > 1 ? tiles * cuts : 0, cuts > 1 ? tiles : 0};
            int sum[3];
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                sum[i] = wave_scan(v[i]);
                if (lane == 63) lds.sums[wave][i] = sum[i];
            }
            __syncthreads();
            int before[3] = {parts, slots, stiles};
            for (int k = 0; k < NT / 64; ++k) {
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (k < wave) before[i] += lds.sums[k][i];
                parts += lds.sums[k][0];
                slots += lds.sums[k][1];
                stiles += lds.sums[k][2];
            }
            const int mine = part - (before[0] + sum[0] - v[0]);
            if (mine >= 0 && mine < v[0]) {
                lds.found[0] = n0 + tid;
                lds.found[1] = mine;
                lds.found[2] = cuts;
                lds.found[3] = before[1] + sum[1] - v[1];
                lds.found[4] = before[2] + sum[2] - v[2];
            }
            __syncthreads();
            if (part < parts && part > 0) break;  // (part 0 goes on, for the number of split tiles)
        }
        if (blockIdx.x == 0 && tid == 0 && p.desc) p.desc[0] = min(stiles, p.tiles);
        if (lds.found[0] < 0) return false;
        w.n = lds.found[0];
        at = lds.found[1];
        splits = lds.found[2];
        slot0 = lds.found[3];
        tile0 = lds.found[4];
        // offsets that overlap name more rows than the room was made for
        if (splits > 1 && ((int64_t)slot0 + (at / splits + 1) * (int64_t)splits > p.slots || tile0 + at / splits >= p.tiles)) return false;
    }
    w.seq = sequence(c, w.n);
    const int rows = w.seq.len * p.G;
    if (rows < p.rows_lo || rows > p.rows_hi) return false;
    // the last tiles see the most cells: first
    const int tiles = (rows + M - 1) / M, x = splits > 1 ? at / splits : at;
    w.split = at - x * splits;
    w.row0 = (tiles - 1 - x) * M;
    w.rows = min(M, rows - w.row0);
    w.hi = min(w.pos(w.row0 + w.rows - 1, p.by_G) + 1, w.cells);
    w.lo = w.first(w.pos(w.row0, p.by_G), p.window);
    const int first = w.lo / KB, nb = w.hi > w.lo ? (w.hi + KB - 1) / KB - first : 0;
    w.splits = 1;
    if (splits > 1) {
        // this tile may see fewer blocks than the sequence's last: as few parts as they need, of equal length
        const int per = ((nb + splits - 1) / splits + p.c_min - 1) / p.c_min * p.c_min;
        w.splits = max(1, (nb + per - 1) / max(per, 1));
        w.slot = (int64_t)(slot0 + x * splits + w.split) * p.Hk + w.head;
        if (w.split == 0 && tid == 0) {
            int32_t *d = p.desc + kDesc * (1 + (int64_t)(tile0 + x) * p.Hk + w.head);
            d[0] = w.n;
            d[1] = w.head;
            d[2] = w.row0;
            d[3] = w.rows;
            d[4] = w.splits;
            d[5] = (int32_t)(slot0 + x * splits);
        }
        if (w.split >= w.splits) return false;
        w.b0 = first + w.split * per;
        w.b1 = min(w.b0 + per, first + nb);
    } else {
        w.b0 = first;
        w.b1 = first + nb;
    }
    return true;
}

// Blocks that a wave puts off: those at the start and at the end of what its rows see that hold infinities or NaN where some
// rows see and others do not.  A wave's rows are 32 tokens at most, so each end is two blocks at most.
struct OddBlocks {
    static constexpr int kMost = 4;
    int start0 = -1, start1 = -1, end0 = -1, end1 = -1;
    __device__ __forceinline__ void add(bool end, int b) {
        if (end) {
            end1 = end0 < 0 ? end1 : b;
            end0 = end0 < 0 ? b : end0;
        } else {
            start1 = start0 < 0 ? start1 : b;
            start0 = start0 < 0 ? b : start0;
        }
    }
    __device__ __forceinline__ int get(int i) const { return i == 0 ? start0 : i == 1 ? start1 : i == 2 ? end0 : end1; }
};

// Row r of a sequence: its token and head, as an offset in rows of the output.
__device__ __forceinline__ int64_t out_row(const AttnParams &p, const Seq &s, int head, int row) {
    const int t = p.by_G.by(row);
    return (s.t0 + t) * p.Hq + head * p.G + (row - t * p.G);
}

// What a workgroup found for its rows, 16 threads a row (thread tid: row tid / 16, columns VW (tid % 16) ..): the
// weighted sums o, the weights' sum l, their maximum m in powers of two.
template <typename IO, int DV, int M>
__device__ __forceinline__ void put_row(const AttnParams &p, const Work &w, int row, int lane16, const float *o, float m, float l) {
    constexpr int VW = DV / 16;
    if (row >= w.rows) return;
    if (w.splits > 1) {
        float *part = p.part + w.slot * (int64_t)(M * (DV + 2));
#pragma unroll
        for (int i = 0; i < VW; i += 4)
            *reinterpret_cast<f32x4 *>(part + row * DV + VW * lane16 + i) = f32x4{o[i], o[i + 1], o[i + 2], o[i + 3]};
        if (lane16 == 0) {
            part[M * DV + row] = m;
            part[M * DV + M + row] = l;
        }
        return;
    }
    const int64_t at = out_row(p, w.seq, w.head, w.row0 + row);
    const float r = l == 0.f ? 0.f : 1.f / l;  // (a row without cells: 0)
    IO *y = static_cast<IO *>(p.out) + at * DV + VW * lane16;
#pragma unroll
    for (int i = 0; i < VW; i += 4)
        IoTraits<IO>::store4(y + i, make_float4(o[i] * r, o[i + 1] * r, o[i + 2] * r, o[i + 3] * r));
    if (p.lse && lane16 == 0) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace paged
}  // namespace kda
