// Paged key-value cache of the full-attention layers, and rotary positions: declarations shared by the host
// dispatch and the kernel files.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda.h"

namespace kda {
namespace paged {

struct RopeParams {
    const void *q, *k;
    void *q_out, *k_out;
    const int32_t *positions;  // or null: token t of seq_len at t % seq_len
    const float *freq;
    int64_t ldq, ldk, ldqo, ldko;
    int64_t tokens;
    int32_t T, Hq, Hk, d, rot, interleaved;
    float amplitude, sign;     // sign -1: turned back
};
// work-items of a launch for the shape (a multiple of 256)
int64_t rope_items(int64_t tokens, int32_t heads, int32_t d);
hipError_t launch_rope(bool bf16, const RopeParams &p, hipStream_t stream);

// The cache and the batch that meets it.
struct Cache {
    void *k, *v;               // pools; strides in elements
    int64_t k_page, k_head, k_cell, v_page, v_head, v_cell;
    const int32_t *table;      // [num_seqs, max_pages], table_ld entries between sequences
    const int32_t *lens;       // [num_seqs] cells, the new tokens' included
    const int32_t *cu;         // [num_seqs + 1], or null: sequence n is tokens [n T, (n + 1) T)
    int64_t table_ld, num_pages;
    int32_t num_seqs, T, max_pages, page_shift;
};

struct AppendParams {
    Cache c;
    const void *k, *v, *q;     // q may be null
    void *q_out;
    const int32_t *positions;  // or null: the token's cell
    const float *freq;
    int64_t ldk, ldv, ldq, ldqo;
    int64_t tokens;
    int32_t Hq, Hk, dk, dv, rot, interleaved;
    float amplitude;
};
int64_t append_items(int64_t tokens, int32_t heads_q, int32_t heads_kv, int32_t dk, int32_t dv);
hipError_t launch_append(bool bf16, const AppendParams &p, hipStream_t stream);

// Quotients by a number that the host knows, n in 0 .. 2^31 - 1: n mul >> (31 + shift) with 2^shift >= d and
// mul = ceil(2^(31 + shift) / d), exact as n (mul d - 2^(31 + shift)) < 2^(31 + shift).
struct Div {
    uint32_t mul = 0, shift = 0;
    Div() = default;
    explicit Div(uint32_t d) {
        while ((1u << shift) < d) ++shift;
        mul = (uint32_t)((((uint64_t)1 << (31 + shift)) + d - 1) / d);
    }
    __host__ __device__ int by(int n) const { return (int)(((uint64_t)(uint32_t)n * mul) >> (31 + shift)); }
};

// Attention.  A tile is M consecutive (token, head of the group) rows of one sequence and key-value head; its
// cells are cut into blocks of KB, and rows of many blocks into splits that workgroups of their own take.
struct AttnParams {
    Cache c;
    const void *q;
    void *out;
    float *lse;
    int64_t ldq;
    int32_t Hq, Hk, G, dk, dv;
    Div by_G, by_Hk;
    int32_t window;            // 0: none
    float scale;               // |scale| log2(e)
    int32_t flip;              // scale < 0: q enters negated
    // rows of the sequences that a launch takes: other launches take the others
    int32_t rows_lo, rows_hi;
    // splits: parts of at least c_min blocks, about `target` workgroups in all; c_min 0: none is possible and every
    // sequence has the same number of tiles
    int32_t c_min, target;
    int32_t tiles, slots;      // room per head: split tiles, splits of those
    int32_t *desc;             // [0] number of split tiles, then kDesc entries each, per (split tile, head)
    float *part;               // per (split, head): M rows of d_v sums, M maxima, M sums of weights
};
constexpr int kDesc = 8;

// Shape of a kernel's tiles.
struct AttnTile {
    int32_t M, KB, c_min, target_per_cu, threads;
};
AttnTile attn_rows_tile(bool bf16);
// many: fp32 calls of many rows over long contexts, see the host's choice
hipError_t launch_attn_rows(bool bf16, bool many, const AttnParams &p, int64_t blocks, hipStream_t stream);
AttnTile attn_tile_tile();
hipError_t launch_attn_tile(const AttnParams &p, int64_t blocks, hipStream_t stream);  // bf16
// joins the splits of at most `tiles` tiles of M rows per head
hipError_t launch_attn_join(bool bf16, const AttnParams &p, int M, int64_t tiles, hipStream_t stream);

}  // namespace paged
}  // namespace kda
