// Host side of the scalar-gate delta rule: argument checks, launch choices and the C ABI.  As for the other
// entry points the arguments are checked before HIP is touched, so an invalid call returns a status
// without launching anything (and works on machines without a GPU).  Only the gradients' workspace is checked
// after a look at the device, whose number of CUs its size goes by (256 where there is none).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <vector>

#include "kda.h"
#include "kda_args.h"
#include "kda_gdn.h"
#include "kda_internal.h"

namespace {

using namespace kda::args;
using kda::set_error;

// A problem that has passed the checks, with its sizes worked out.
struct Shape {
    int64_t tokens = 0, ldq = 0, ldk = 0, ldv = 0;
    int32_t num_seqs = 0;
    int64_t io = 2, gate = 4, state = 4;      // bytes of an element
    int64_t qk_row = 0, v_row = 0, states = 0;  // elements: a token's rows, all sequences' states
    // bytes from the first to the last element of a strided tensor of `tokens` rows
    int64_t span(int64_t ld, int64_t row) const { return tokens > 0 ? ((tokens - 1) * ld + row) * io : 0; }
};

// Work-items that the scans and decode spend on 32 columns of a (sequence, head).
constexpr int64_t kScanItems = 512, kDecodeItems = 64;

kda_status_t check_shape(const kda_gdn_problem_t *p, bool packed, Shape &s, int64_t items = kScanItems) {
    if (!p) return set_error(KDA_ERR_INVALID_ARGUMENT, "problem is NULL");
    if (p->batch < 0 || p->seq_len < 0 || p->num_heads_k < 1 || p->num_heads_v < 1)
        return set_error(KDA_ERR_INVALID_ARGUMENT, "bad sizes: batch=%d seq_len=%d num_heads_k=%d num_heads_v=%d",
                         p->batch, p->seq_len, p->num_heads_k, p->num_heads_v);
    if (p->num_heads_v % p->num_heads_k != 0)
        return set_error(KDA_ERR_INVALID_ARGUMENT, "num_heads_v %d is not a multiple of num_heads_k %d", p->num_heads_v,
                         p->num_heads_k);
    if (!dtype_ok(p->io_dtype) || !dtype_ok(p->gate_dtype) || !dtype_ok(p->state_dtype))
        return set_error(KDA_ERR_INVALID_ARGUMENT, "io_dtype %d, gate_dtype %d, state_dtype %d: each is KDA_F32 or KDA_BF16",
                         (int)p->io_dtype, (int)p->gate_dtype, (int)p->state_dtype);
    for (int d : {p->head_dim_k, p->head_dim_v})
        if (d != 64 && d != 128)
            return set_error(KDA_ERR_UNSUPPORTED, "head dims d_k=%d d_v=%d: supported are 64 and 128", p->head_dim_k,
                             p->head_dim_v);
    if (!std::isfinite(p->scale)) return set_error(KDA_ERR_INVALID_ARGUMENT, "scale is not finite");
    if (packed) {
        if (p->batch != 1) return set_error(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens needs batch == 1 (got %d)", p->batch);
        if (p->num_seqs < 0) return set_error(KDA_ERR_INVALID_ARGUMENT, "num_seqs %d < 0", p->num_seqs);
    }
    s.num_seqs = packed ? p->num_seqs : p->batch;
    s.tokens = packed ? p->seq_len : (int64_t)p->batch * p->seq_len;
    s.io = bytes_of(p->io_dtype);
    s.gate = bytes_of(p->gate_dtype);
    s.state = bytes_of(p->state_dtype);
    s.qk_row = (int64_t)p->num_heads_k * p->head_dim_k;
    s.v_row = (int64_t)p->num_heads_v * p->head_dim_v;
    const int64_t given[] = {p->stride_q, p->stride_k, p->stride_v};
    const int64_t rows[] = {s.qk_row, s.qk_row, s.v_row};
    int64_t *ld[] = {&s.ldq, &s.ldk, &s.ldv};
    for (int i = 0; i < 3; ++i) {
        *ld[i] = given[i] ? given[i] : rows[i];
        if (*ld[i] < rows[i])
            return set_error(KDA_ERR_INVALID_ARGUMENT, "stride_%c %lld is smaller than a token's %lld elements", "qkv"[i],
                             (long long)*ld[i], (long long)rows[i]);
        if (*ld[i] % (16 / s.io) != 0)
            return set_error(KDA_ERR_INVALID_ARGUMENT, "stride_%c %lld is not a multiple of 16 bytes", "qkv"[i],
                             (long long)*ld[i]);
        if (s.tokens > 0 && *ld[i] > (1LL << 60) / s.tokens) return set_error(KDA_ERR_UNSUPPORTED, "tensor too large");
    }
    // (decode rounds up to workgroups of four waves)
    if ((int64_t)s.num_seqs * p->num_heads_v > (kMostItems - 3 * kDecodeItems) / (items * (p->head_dim_v / 32)))
        return set_error(KDA_ERR_UNSUPPORTED, "too many (sequence, head) pairs: %d x %d", s.num_seqs, p->num_heads_v);
    s.states = (int64_t)s.num_seqs * p->num_heads_v * p->head_dim_k * p->head_dim_v;
    return KDA_OK;
}

kda_status_t check_offsets(const kda_gdn_problem_t *p, const Shape &s, const int32_t *cu, const int32_t *host) {
    return kda::args::check_offsets(p->seq_len, s.num_seqs, cu, host);
}

kda::gdn::GdnParams params_of(const kda_gdn_problem_t *p, const Shape &s, const void *q, const void *k, const void *v,
                              const void *g, const void *beta, const int32_t *cu) {
    kda::gdn::GdnParams r{};
    r.q = q;
    r.k = k;
    r.v = v;
    r.g = g;
    r.beta = beta;
    r.cu = cu;
    r.ldq = s.ldq;
    r.ldk = s.ldk;
    r.ldv = s.ldv;
    r.num_seqs = s.num_seqs;
    r.T = p->seq_len;
    r.Hk = p->num_heads_k;
    r.Hv = p->num_heads_v;
    r.dk = p->head_dim_k;
    r.dv = p->head_dim_v;
    r.gate_bf16 = p->gate_dtype == KDA_BF16;
    r.s0_bf16 = r.sf_bf16 = p->state_dtype == KDA_BF16;
    r.scale = p->scale;
    return r;
}

hipError_t launch_scan(const kda_gdn_problem_t *p, int mode, const kda::gdn::GdnParams &r, hipStream_t s) {
    return p->io_dtype == KDA_BF16 ? kda::gdn::launch_scan_bf16(mode, r, s) : kda::gdn::launch_scan_f32(mode, r, s);
}

// Whether the gradients of a bf16 call are computed on fp32 operands.  Every value has the same error whatever the
// call's size, but over few values the roundings of the products' operands do not average out in the norm (260
// gates: error of dg up to 5.7e-3 of its norm, 3e-3 for thousands of them, about 4e-7 on fp32 operands).  The
// price grows with every chunk of the walk, hence the limit of tokens beside that of gates: d = 128, 256 tokens
// of one head 118 us, 257 on bf16 operands 47; 128 tokens of 4 heads 81, 129 39.
bool bwd_wide(const kda_gdn_problem_t *p, const Shape &s) {
    return p->io_dtype == KDA_BF16 && s.tokens <= 256 && s.tokens * p->num_heads_v <= 512;
}

// Segments of walks that are split over their length: with few (sequence, head) chains most CUs idle while
// each chain's chunks follow one another.  The maps of all segments but the last run side by side
// (d_v + d_k columns), the join walks the segments, and the forward runs on all of them at once.  The
// number of segments is the one with the least time by the model below (us: a chunk of the forward and of
// the maps, each per round of workgroups over the CUs; a segment of the join; the fixed part of the two
// further launches), and the split is taken where that is a tenth less than one walk.  Its constants were measured
// at 128 x 128 with few workgroups.  With one on every CU, as the split may have, a chunk takes a fifth more (2.6
// us forward, 2.0 maps), and at 64 x 64 less (forward 1.8 bf16, 3.4 fp32), so that the choice is not the best one
// everywhere, but it was at no loss for 1 to 32 heads of 64 and 128 around the shortest lengths that are split.
// The gradients split the keeping forward in the same way, and the reverse scan: a segment takes the
// gradient of the state that leaves it to M^T dS + H', H' by one more reverse scan from zero.
// 8 heads of 128 x 128, bf16: one walk against the split 73 / 62 us at 2,048 tokens, 272 / 131 at 8,192,
// 1,070 / 408 at 32,768; at 1,024 tokens 41 / 45, at 32 heads and 8,192 tokens 270 / 376: one walk.
// Gradients, the same heads: 172 / 130 at 2,048 tokens, 646 / 303 at 8,192; at 1,024 97: one walk; fp32 684 / 308
// at 2,048.  Packed batches are not split, for which their segments would have to be listed (one prompt of 65,536
// tokens x 8 heads: 2,440 us packed, 866 as a plain batch of one).
struct Split {
    int32_t segs = 0, seg_len = 0;
    size_t h = 0, bytes = 0;  // offset of M, size
};
Split split_of(const kda_gdn_problem_t *p, const Shape &s, bool packed, int cus, bool bwd) {
    Split r;
    const bool bf = p->io_dtype == KDA_BF16;
    // a chunk of the walks that are split (gradients: the keeping forward and the reverse scan), of the maps
    // and of the reverse scan of the segments
    const double t_walk = bwd ? (bf ? 5.9 : 10.0) : bf ? 2.1 : 5.9, t_map = bf ? 1.7 : 3.4,
                 t_rev = bwd ? (bf ? 3.2 : 6.5) : 0, t_join = bwd ? 2.4 : 1.2, t_fixed = bwd ? 42 : 14;
    const int64_t cols = p->head_dim_v / 32, both = cols + p->head_dim_k / 32, C = kda::gdn::chunk_of(p->io_dtype);
    const int64_t chains = (int64_t)s.num_seqs * p->num_heads_v, chunks = (p->seq_len + C - 1) / C;
    if (packed || chains <= 0) return r;
    double least = 0.9 * t_walk * (double)chunks;
    int64_t per = 0;
    for (int64_t n = 2; n * chains * cols <= cus && 2 * n <= chunks; ++n) {  // one round for the walks themselves
        const int64_t maps = bwd ? n : n - 1, rounds = (maps * chains * both + cus - 1) / cus, len = (chunks + n - 1) / n;
        const double t = (double)len * (t_walk + t_map * (double)rounds + t_rev) + t_join * (double)n + t_fixed;
        if (t < least) {
            least = t;
            per = len;
        }
    }
    if (!per) return r;
    r.segs = (int32_t)((chunks + per - 1) / per);
    r.seg_len = (int32_t)(per * C);
    const size_t n = (size_t)chains * r.segs * p->head_dim_k * sizeof(float);
    r.h = n * p->head_dim_v;
    r.bytes = r.h + n * p->head_dim_k;
    return r;
}

// The `maps` of segments first .. first + run - 1 of the walk r (mode 1 or 2) into h and m, and the states that
// enter every segment into h, as the walk's starting states.
kda_status_t enter_segments(const kda_gdn_problem_t *p, const Split &split, int mode, int first, int run, float *h,
                            const void *s0, kda::gdn::GdnParams &r, hipStream_t hs) {
    const int batch = r.num_seqs;
    r.segs = r.seg_run = split.segs;
    r.seg_len = split.seg_len;
    r.num_seqs = batch * split.segs;
    kda::gdn::GdnParams maps = r;
    maps.maps = 1;
    maps.seg_first = first;
    maps.seg_run = run;
    maps.num_seqs = batch * run;
    maps.s0 = nullptr;
    maps.out = maps.hs = maps.zs = nullptr;
    maps.sf = h;
    maps.sf_bf16 = 0;
    float *m = h + split.h / sizeof(float);
    if (mode == 1) maps.sm = m;
    kda_status_t st = done(launch_scan(p, mode, maps, hs), "kda_gdn segment launch");
    if (st != KDA_OK) return st;
    const kda::gdn::JoinParams join{s0,    h, m, batch, split.segs, p->num_heads_v, p->head_dim_k, p->head_dim_v,
                                    p->state_dtype == KDA_BF16, mode == 2};
    r.s0 = h;
    r.s0_bf16 = 0;
    return done(kda::gdn::launch_join(join, hs), "kda_gdn join launch");
}

// Workspace of the backward: S and dS per chunk slot, Z per token; on fp32 operands also the copies of the
// tensors in bf16 (q, k, v, d_out, dq, dk, dv); where the walks are split, the segments' maps.
struct BwdLayout {
    int64_t slots = 0;
    size_t dhs = 0, zs = 0, copies = 0, qk = 0, vo = 0, maps = 0, bytes = 0;
    Split split;
};
kda_status_t bwd_layout(const kda_gdn_problem_t *p, const Shape &s, bool packed, BwdLayout &b) {
    const bool wide = bwd_wide(p, s);
    const int64_t C = kda::gdn::chunk_of(wide ? KDA_F32 : p->io_dtype), per = (int64_t)p->seq_len / C;
    b.slots = packed ? per + s.num_seqs : (int64_t)s.num_seqs * (per + (p->seq_len % C != 0));
    const int64_t row = s.v_row * (wide ? 4 : s.io);
    // a workgroup of the gradients (8 threads a token) per chunk and key head
    if (b.slots > kMostItems / (8 * C * p->num_heads_k) || b.slots > (1LL << 60) / (row * p->head_dim_k))
        return set_error(KDA_ERR_UNSUPPORTED, "too many chunks");
    auto align = [](int64_t x) { return (size_t)((x + 255) / 256 * 256); };
    b.dhs = align(b.slots * row * p->head_dim_k);
    b.zs = 2 * b.dhs;
    b.copies = b.bytes = b.zs + align(s.tokens * row);
    if (wide) {
        b.qk = align(s.tokens * s.qk_row * 4);
        b.vo = align(s.tokens * s.v_row * 4);
        b.bytes += 4 * b.qk + 3 * b.vo;
    }
    kda_gdn_problem_t run = *p;
    if (wide) run.io_dtype = KDA_F32;
    b.split = split_of(&run, s, packed, current_cus(), true);
    b.maps = b.bytes;
    b.bytes += b.split.bytes;
    return KDA_OK;
}

// Workspace of a problem before it is known whether cu_seqlens will come with it: `need` of the plain batch and,
// where num_seqs > 0 sequences may be packed in one row, the larger of both (without cu_seqlens num_seqs may hold anything).
template <typename Need>
kda_status_t workspace_of(const kda_gdn_problem_t *p, size_t *bytes, Need need) {
    if (!bytes) return set_error(KDA_ERR_INVALID_ARGUMENT, "bytes is NULL");
    *bytes = 0;
    Shape s;
    size_t n = 0, packed = 0;
    kda_status_t st = check_shape(p, false, s);
    if (st == KDA_OK) st = need(s, false, n);
    if (st != KDA_OK) return st;
    if (p->batch == 1 && p->num_seqs > 0) {
        Shape t;
        if (check_shape(p, true, t) == KDA_OK && need(t, true, packed) == KDA_OK) n = std::max(n, packed);
    }
    *bytes = n;
    return done(hipSuccess, "");
}

}  // namespace

extern "C" {

kda_status_t kda_gdn_chunk_fwd(const kda_gdn_problem_t *problem, const void *q, const void *k, const void *v,
                               const void *g, const void *beta, const void *initial_state, const int32_t *cu_seqlens,
                               const int32_t *cu_seqlens_host, void *out, void *final_state, void *workspace,
                               size_t workspace_bytes, void *stream) {
    try {
        Shape s;
        kda_status_t st = check_shape(problem, cu_seqlens != nullptr, s);
        if (st != KDA_OK) return st;
        const int64_t gates = s.tokens * problem->num_heads_v * s.gate;
        const Arg args[] = {
            {"q", q, s.span(s.ldq, s.qk_row), 16, true, false},
            {"k", k, s.span(s.ldk, s.qk_row), 16, true, false},
            {"v", v, s.span(s.ldv, s.v_row), 16, true, false},
            {"g", g, gates, (size_t)s.gate, true, false},
            {"beta", beta, gates, (size_t)s.gate, true, false},
            {"initial_state", initial_state, s.states * s.state, 16, false, false},
            {"final_state", final_state, s.states * s.state, 16, false, true},
            {"out", out, s.tokens * s.v_row * s.io, 16, true, true},
            {"cu_seqlens", cu_seqlens, ((int64_t)s.num_seqs + 1) * 4, 4, false, false},
            {"workspace", workspace, (int64_t)workspace_bytes, 256, false, true},
        };
        st = check_args(args, 5, 6);
        if (st == KDA_OK) st = check_offsets(problem, s, cu_seqlens, cu_seqlens_host);
        if (st != KDA_OK) return st;
        kda::gdn::GdnParams r = params_of(problem, s, q, k, v, g, beta, cu_seqlens);
        r.s0 = initial_state;
        r.sf = final_state;
        r.out = out;
        if (s.num_seqs == 0 || (s.tokens == 0 && !final_state)) return done(hipSuccess, "");
        hipStream_t hs = static_cast<hipStream_t>(stream);
        const Split split = workspace ? split_of(problem, s, cu_seqlens != nullptr, current_cus(), false) : Split();
        if (split.segs > 0 && workspace_bytes >= split.bytes) {
            st = enter_segments(problem, split, 1, 0, split.segs - 1, static_cast<float *>(workspace), initial_state, r, hs);
            if (st != KDA_OK) return st;
        }
        return done(launch_scan(problem, 0, r, hs), "kda_gdn_chunk_fwd launch");
    } catch (...) {
        return set_error(KDA_ERR_HIP, "unexpected exception in argument checks");
    }
}

kda_status_t kda_gdn_chunk_fwd_workspace(const kda_gdn_problem_t *problem, size_t *bytes) {
    return workspace_of(problem, bytes, [&](const Shape &s, bool packed, size_t &n) {
        n = split_of(problem, s, packed, current_cus(), false).bytes;
        return KDA_OK;
    });
}

kda_status_t kda_gdn_chunk_bwd_workspace(const kda_gdn_problem_t *problem, size_t *bytes) {
    return workspace_of(problem, bytes, [&](const Shape &s, bool packed, size_t &n) {
        BwdLayout b;
        const kda_status_t st = bwd_layout(problem, s, packed, b);
        n = b.bytes;
        return st;
    });
}

kda_status_t kda_gdn_chunk_bwd(const kda_gdn_problem_t *problem, const void *q, const void *k, const void *v,
                               const void *g, const void *beta, const void *initial_state, const int32_t *cu_seqlens,
                               const int32_t *cu_seqlens_host, const void *d_out, const void *d_final_state, void *dq,
                               void *dk, void *dv, void *dg, void *dbeta, void *d_initial_state, void *workspace,
                               size_t workspace_bytes, void *stream) {
    try {
        Shape s;
        kda_status_t st = check_shape(problem, cu_seqlens != nullptr, s);
        if (st != KDA_OK) return st;
        const int64_t gates = s.tokens * problem->num_heads_v * s.gate, qk = s.tokens * s.qk_row * s.io,
                      vo = s.tokens * s.v_row * s.io, states = s.states * s.state;
        Arg args[] = {
            {"q", q, s.span(s.ldq, s.qk_row), 16, true, false},
            {"k", k, s.span(s.ldk, s.qk_row), 16, true, false},
            {"v", v, s.span(s.ldv, s.v_row), 16, true, false},
            {"g", g, gates, (size_t)s.gate, true, false},
            {"beta", beta, gates, (size_t)s.gate, true, false},
            {"initial_state", initial_state, states, 16, false, false},
            {"d_out", d_out, vo, 16, true, false},
            {"d_final_state", d_final_state, states, 16, false, false},
            {"cu_seqlens", cu_seqlens, ((int64_t)s.num_seqs + 1) * 4, 4, false, false},
            {"dq", dq, qk, 16, true, true},
            {"dk", dk, qk, 16, true, true},
            {"dv", dv, vo, 16, true, true},
            {"dg", dg, gates, (size_t)s.gate, true, true},
            {"dbeta", dbeta, gates, (size_t)s.gate, true, true},
            {"d_initial_state", d_initial_state, states, 16, false, true},
            {"workspace", workspace, 0, 256, false, true},
        };
        st = check_args(args);
        if (st == KDA_OK) st = check_offsets(problem, s, cu_seqlens, cu_seqlens_host);
        if (st != KDA_OK) return st;
        BwdLayout b;  // asks for the device's CUs
        st = bwd_layout(problem, s, cu_seqlens != nullptr, b);
        args[15].bytes = (int64_t)b.bytes;
        if (st == KDA_OK) st = check_args(args);
        if (st != KDA_OK) return st;
        if (b.bytes > 0 && (!workspace || workspace_bytes < b.bytes))
            return set_error(KDA_ERR_WORKSPACE, "kda_gdn_chunk_bwd needs a 256-byte aligned workspace of %zu bytes (got %zu at %p)",
                             b.bytes, workspace_bytes, workspace);
        if (s.num_seqs == 0 || (s.tokens == 0 && !d_initial_state)) return done(hipSuccess, "");
        hipStream_t hs = static_cast<hipStream_t>(stream);
        char *ws = static_cast<char *>(workspace);
        kda_gdn_problem_t run = *problem;
        kda::gdn::ConvertParams in{}, back{};
        if (bwd_wide(problem, s) && s.tokens > 0) {
            char *at = ws + b.copies;
            auto copy = [&](kda::gdn::ConvertParams &c, const void *p, int64_t cols_, int64_t ld, size_t bytes) {
                c.t[c.n++] = {const_cast<void *>(p), at, s.tokens, cols_, ld};
                void *f = at;
                at += bytes;
                return f;
            };
            q = copy(in, q, s.qk_row, s.ldq, b.qk);
            k = copy(in, k, s.qk_row, s.ldk, b.qk);
            v = copy(in, v, s.v_row, s.ldv, b.vo);
            d_out = copy(in, d_out, s.v_row, s.v_row, b.vo);
            dq = copy(back, dq, s.qk_row, s.qk_row, b.qk);
            dk = copy(back, dk, s.qk_row, s.qk_row, b.qk);
            dv = copy(back, dv, s.v_row, s.v_row, b.vo);
            back.cu = cu_seqlens;  // rows that no sequence owns have no gradients in the copies either
            back.num_seqs = s.num_seqs;
            back.T = problem->seq_len;
            run.io_dtype = KDA_F32;
            s.ldq = s.ldk = s.qk_row;
            s.ldv = s.v_row;
            st = done(kda::gdn::launch_convert(true, in, hs), "kda_gdn_chunk_bwd widening launch");
            if (st != KDA_OK) return st;
        }
        kda::gdn::GdnParams keep = params_of(&run, s, q, k, v, g, beta, cu_seqlens);
        keep.s0 = initial_state;
        keep.hs = ws;
        keep.zs = ws + b.zs;
        kda::gdn::GdnParams rev = params_of(&run, s, q, k, d_out, g, beta, cu_seqlens);
        rev.ldv = s.v_row;
        rev.s0 = d_final_state;
        rev.sf = d_initial_state;
        rev.out = dv;
        rev.hs = ws + b.dhs;
        kda::gdn::GradParams grad{};
        grad.f = rev;  // before the walk is split
        grad.hs = keep.hs;
        grad.dhs = rev.hs;
        grad.zs = keep.zs;
        grad.dx = dv;
        grad.dq = dq;
        grad.dk = dk;
        grad.dg = dg;
        grad.dbeta = dbeta;
        grad.slots = b.slots;
        float *maps = reinterpret_cast<float *>(ws + b.maps);
        if (s.tokens > 0) {
            if (b.split.segs > 0) {
                st = enter_segments(&run, b.split, 1, 0, b.split.segs, maps, initial_state, keep, hs);
                if (st != KDA_OK) return st;
            }
            st = done(launch_scan(&run, 1, keep, hs), "kda_gdn_chunk_bwd forward launch");
            if (st != KDA_OK) return st;
        }
        if (b.split.segs > 0) {  // the segments' M serve again, transposed
            st = enter_segments(&run, b.split, 2, 1, b.split.segs - 1, maps, d_final_state, rev, hs);
            if (st != KDA_OK) return st;
        }
        st = done(launch_scan(&run, 2, rev, hs), "kda_gdn_chunk_bwd reverse launch");
        if (st != KDA_OK || s.tokens == 0) return st;
        st = done(run.io_dtype == KDA_BF16 ? kda::gdn::launch_grad_bf16(grad, hs) : kda::gdn::launch_grad_f32(grad, hs),
                  "kda_gdn_chunk_bwd gradient launch");
        if (st != KDA_OK || back.n == 0) return st;
        return done(kda::gdn::launch_convert(false, back, hs), "kda_gdn_chunk_bwd narrowing launch");
    } catch (...) {
        return set_error(KDA_ERR_HIP, "unexpected exception in argument checks");
    }
}

kda_status_t kda_gdn_decode(const kda_gdn_problem_t *problem, const void *q, const void *k, const void *v,
                            const void *g, const void *beta, void *state, int64_t num_slots, const int32_t *state_slots,
                            const int32_t *state_slots_host, const int32_t *cu_seqlens, const int32_t *cu_seqlens_host,
                            void *out, void *stream) {
    try {
        Shape s;
        kda_status_t st = check_shape(problem, cu_seqlens != nullptr, s, kDecodeItems);
        if (st != KDA_OK) return st;
        if (num_slots < 0 || num_slots > 0x7fffffffLL)
            return set_error(KDA_ERR_INVALID_ARGUMENT, "num_slots %lld out of range", (long long)num_slots);
        if (!state_slots && num_slots < s.num_seqs)
            return set_error(KDA_ERR_INVALID_ARGUMENT, "%d sequences without state_slots need as many slots (got %lld)",
                             s.num_seqs, (long long)num_slots);
        const int64_t gates = s.tokens * problem->num_heads_v * s.gate;
        const int64_t per = (int64_t)problem->num_heads_v * problem->head_dim_k * problem->head_dim_v * s.state;
        if (num_slots > (1LL << 62) / per) return set_error(KDA_ERR_UNSUPPORTED, "state too large");
        const Arg args[] = {
            {"q", q, s.span(s.ldq, s.qk_row), 16, true, false},
            {"k", k, s.span(s.ldk, s.qk_row), 16, true, false},
            {"v", v, s.span(s.ldv, s.v_row), 16, true, false},
            {"g", g, gates, (size_t)s.gate, true, false},
            {"beta", beta, gates, (size_t)s.gate, true, false},
            {"state", state, num_slots * per, 16, true, true},
            {"out", out, s.tokens * s.v_row * s.io, 16, true, true},
            {"state_slots", state_slots, (int64_t)s.num_seqs * 4, 4, false, false},
            {"cu_seqlens", cu_seqlens, ((int64_t)s.num_seqs + 1) * 4, 4, false, false},
        };
        st = check_args(args);
        if (st == KDA_OK) st = check_offsets(problem, s, cu_seqlens, cu_seqlens_host);
        if (st != KDA_OK) return st;
        if (state_slots_host) {
            if (!state_slots) return set_error(KDA_ERR_INVALID_ARGUMENT, "state_slots_host given without state_slots");
            // each slot once: two sequences in one slot would race for it
            std::vector<int32_t> used;
            used.reserve((size_t)s.num_seqs);
            for (int32_t i = 0; i < s.num_seqs; ++i) {
                const int32_t x = state_slots_host[i];
                if (x >= num_slots)
                    return set_error(KDA_ERR_INVALID_ARGUMENT, "state_slots[%d] = %d, there are %lld", i, x, (long long)num_slots);
                if (x >= 0) used.push_back(x);
            }
            std::sort(used.begin(), used.end());
            const auto twice = std::adjacent_find(used.begin(), used.end());
            if (twice != used.end())
                return set_error(KDA_ERR_INVALID_ARGUMENT, "state_slots: two sequences' slots are both %d", *twice);
        }
        if (s.num_seqs == 0 || s.tokens == 0 || num_slots == 0) return done(hipSuccess, "");
        kda::gdn::DecodeParams r{};
        r.q = q;
        r.k = k;
        r.v = v;
        r.g = g;
        r.beta = beta;
        r.state = state;
        r.slots = state_slots;
        r.cu = cu_seqlens;
        r.out = out;
        r.ldq = s.ldq;
        r.ldk = s.ldk;
        r.ldv = s.ldv;
        r.num_slots = num_slots;
        r.num_seqs = s.num_seqs;
        r.T = problem->seq_len;
        r.Hk = problem->num_heads_k;
        r.Hv = problem->num_heads_v;
        r.dk = problem->head_dim_k;
        r.dv = problem->head_dim_v;
        r.gate_bf16 = problem->gate_dtype == KDA_BF16;
        r.state_bf16 = problem->state_dtype == KDA_BF16;
        r.scale = problem->scale;
        return done(kda::gdn::launch_decode(problem->io_dtype == KDA_BF16, r, static_cast<hipStream_t>(stream)),
                    "kda_gdn_decode launch");
    } catch (...) {
        return set_error(KDA_ERR_HIP, "unexpected exception in argument checks");
    }
}

size_t kda_norm_gate_bwd_workspace(int64_t rows, int32_t d, int32_t io_dtype) {
    if (rows < 0 || (d != 64 && d != 128) || !dtype_ok(io_dtype)) return 0;
    const int b = kda::norm_gate_bwd_blocks(io_dtype == KDA_BF16 ? KDA_BF16 : KDA_F32, rows, d);
    return b > 1 ? (size_t)b * d * sizeof(float) : 0;
}

kda_status_t kda_norm_gate_bwd(int64_t rows, int32_t d, int32_t io_dtype, float eps, const void *o, const void *gate,
                               const float *weight, const void *d_out, void *d_o, void *d_gate, float *d_weight,
                               void *workspace, size_t workspace_bytes, void *stream) {
    try {
        if (rows < 0) return set_error(KDA_ERR_INVALID_ARGUMENT, "rows %lld < 0", (long long)rows);
        if (!dtype_ok(io_dtype))
            return set_error(KDA_ERR_INVALID_ARGUMENT, "io_dtype %d is not KDA_F32 or KDA_BF16", (int)io_dtype);
        if (d != 64 && d != 128) return set_error(KDA_ERR_UNSUPPORTED, "d=%d: supported are 64 and 128", d);
        if (!std::isfinite(eps) || eps < 0.f) return set_error(KDA_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
        if (rows > (1LL << 48)) return set_error(KDA_ERR_UNSUPPORTED, "too many rows");
        const int64_t n = rows * d * bytes_of(io_dtype);
        const size_t need = kda_norm_gate_bwd_workspace(rows, d, io_dtype);
        const Arg args[] = {
            {"o", o, n, 16, true, false},
            {"gate", gate, n, 16, true, false},
            {"weight", weight, 4 * d, 16, true, false},
            {"d_out", d_out, n, 16, true, false},
            {"d_o", d_o, n, 16, true, true},
            {"d_gate", d_gate, n, 16, true, true},
            {"d_weight", d_weight, 4 * d, 16, true, true},
            {"workspace", workspace, (int64_t)need, 16, false, true},
        };
        kda_status_t st = check_args(args);
        if (st != KDA_OK) return st;
        if (need > 0 && (!workspace || workspace_bytes < need))
            return set_error(KDA_ERR_WORKSPACE, "kda_norm_gate_bwd needs a workspace of %zu bytes (got %zu at %p)", need,
                             workspace_bytes, workspace);
        return done(kda::launch_norm_gate_bwd(io_dtype == KDA_BF16 ? KDA_BF16 : KDA_F32, rows, d, eps, o, gate, weight,
                                              d_out, d_o, d_gate, d_weight, static_cast<float *>(workspace),
                                              static_cast<hipStream_t>(stream)),
                    "kda_norm_gate_bwd launch");
    } catch (...) {
        return set_error(KDA_ERR_HIP, "unexpected exception in argument checks");
    }
}

}  // extern "C"
