// Gated delta rule with one log-gate per token and value head: declarations shared by the host
// dispatch and the kernel files.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda.h"

namespace kda {
namespace gdn {

// Tokens per chunk.  bf16: 64, so that the products over a chunk's tokens fill the matrix instruction's
// 32-wide contraction twice; fp32: 32, what three staged chunks of 4-byte K and Q leave of the LDS.
constexpr int kChunkBf16 = 64, kChunkF32 = 32;
inline int chunk_of(int32_t io) { return io == KDA_BF16 ? kChunkBf16 : kChunkF32; }

// First chunk slot of packed sequence n that starts at token `start`: sum_m<n ceil(len_m / C) is at
// most start / C + n, so these bases leave room for every sequence and need no prefix sum.
__host__ __device__ inline int64_t slot_base(int64_t start, int64_t n, int C) { return start / C + n; }

struct GdnParams {
    const void *q, *k;        // [tokens, Hk, d_k], ldq / ldk elements between tokens
    const void *v;            // [tokens, Hv, dv], ldv elements between tokens (reverse scan: d_out)
    const void *g, *beta;     // [tokens, Hv] fp32, or bf16 with gate_bf16
    const void *s0;           // [num_seqs, Hv, d_k, dv] state the walk starts from, or null (zero)
    void *sf;                 // the state it ends with, or null
    const int32_t *cu;        // [num_seqs + 1], or null: sequence n is tokens [n T, (n + 1) T)
    void *out;                // [tokens, Hv, dv] dense: o (forward) or dV (reverse)
    void *hs = nullptr;       // [slots, Hv, dv, d_k] operand type: the state entering each chunk (keeping
                              // forward) or the gradient of the state leaving it (reverse)
    void *zs = nullptr;       // [tokens, Hv, dv] operand type: Z (keeping forward)
    int64_t ldq, ldk, ldv;
    int32_t num_seqs, T, Hk, Hv, dk, dv;
    int32_t gate_bf16;
    int32_t s0_bf16, sf_bf16; // types of s0 and of sf
    float scale;
    // A walk split over its length (segs > 0): "sequence" n is segment seg_first + n % seg_run, of seg_len tokens, of
    // the T tokens n / seg_run; states at s0 are [batch, segs, ..], and only the state that ends the whole
    // walk goes to sf, [batch, ..].  With maps set each segment's goes to sf, [batch, segs, ..], and (keeping
    // forward) d_k more columns, started from the identity and without values, to sm.
    int32_t segs = 0, seg_len = 0, seg_first = 0, seg_run = 0, maps = 0;
    float *sm = nullptr;  // [batch, segs, Hv, d_k, d_k]
};

// Walks every sequence's chunks.  mode: 0 forward, 1 forward that keeps states and Z (no output), 2 reverse.
hipError_t launch_scan_bf16(int mode, const GdnParams &p, hipStream_t stream);
hipError_t launch_scan_f32(int mode, const GdnParams &p, hipStream_t stream);

// Gradients inside the chunks, after a keeping forward and a reverse scan.
struct GradParams {
    GdnParams f;                       // q, k, g, beta, cu, sizes; v = d_out (dense)
    const void *hs, *dhs, *zs, *dx;    // what the scans left: S, dS [slots, Hv, dv, d_k], Z, dX [tokens, Hv, dv]
    void *dq, *dk;                     // [tokens, Hk, d_k] dense
    void *dg, *dbeta;                  // [tokens, Hv] gate type
    int64_t slots;
};
hipError_t launch_grad_bf16(const GradParams &p, hipStream_t stream);
hipError_t launch_grad_f32(const GradParams &p, hipStream_t stream);

// Rows of bf16 values, ld elements apart, and their dense fp32 copy.
struct ConvertRows {
    void *bf16, *f32;
    int64_t rows, cols, ld;  // cols, ld multiples of 8
};
struct ConvertParams {
    ConvertRows t[4];
    int32_t n;
    // a packed batch: only the rows of its sequences, cu[0] .. cu[num_seqs] of T, are written; else null
    const int32_t *cu;
    int32_t num_seqs, T;
};
// widen: bf16 -> fp32, else fp32 -> bf16
hipError_t launch_convert(bool widen, const ConvertParams &p, hipStream_t stream);

// The states entering the segments of split walks (kda_gdn_segments.hip).
struct JoinParams {
    const void *s0;  // [batch, Hv, d_k, dv] fp32 or bf16, or null (zero): what enters the first segment walked
    float *h;        // [batch, segs, Hv, d_k, dv]: H (but of the last segment walked) on entry, the states on return
    const float *m;  // [batch, segs, Hv, d_k, d_k]
    int32_t batch, segs, Hv, dk, dv, state_bf16;
    int32_t reverse; // gradients: from the last segment to the first, M transposed
};
hipError_t launch_join(const JoinParams &p, hipStream_t stream);

struct DecodeParams {
    const void *q, *k, *v;    // as above
    const void *g, *beta;
    void *state;              // [num_slots, Hv, d_k, dv] fp32 or bf16, read and written
    const int32_t *slots;     // [num_seqs] slot of each sequence, or null (sequence n has slot n)
    const int32_t *cu;
    void *out;
    int64_t ldq, ldk, ldv, num_slots;
    int32_t num_seqs, T, Hk, Hv, dk, dv;
    int32_t gate_bf16, state_bf16;
    float scale;
};
hipError_t launch_decode(bool io_bf16, const DecodeParams &p, hipStream_t stream);

}  // namespace gdn
}  // namespace kda
