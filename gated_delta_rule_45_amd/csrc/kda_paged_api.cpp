// Host side of rotary positions and of the paged key-value cache: argument checks, launch choices and the C ABI.
// As for the other entry points the arguments are checked before HIP is touched; only the attention's workspace is
// checked after a look at the device, whose number of CUs its size goes by (256 where there is none).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "kda.h"
#include "kda_args.h"
#include "kda_internal.h"
#include "kda_paged.h"

namespace {

using namespace kda::args;
using kda::set_error;

// A strided argument: n runs of `run` bytes, `step` bytes apart (a dense one: n = 1).
struct Runs {
    const char *name;
    const void *p;
    int64_t run, step, n;
    size_t align;
    bool needed, written;
    int twin = -1;   // index of the argument that may be the same runs
    int apart = -1;  // of one that they are compared with elsewhere
    uintptr_t begin() const { return reinterpret_cast<uintptr_t>(p); }
    uintptr_t end() const { return begin() + (uintptr_t)((n - 1) * step + run); }
    bool empty() const { return !p || n <= 0 || run <= 0; }
};

// Whether a byte may be in both: exactly for runs of the same step (slices of one tensor), by their ends otherwise.
bool meet(const Runs &a, const Runs &b) {
    if (a.begin() >= b.end() || b.begin() >= a.end()) return false;
    if (a.n <= 1 || b.n <= 1 || a.step != b.step || a.step <= 0) return true;
    const uintptr_t step = (uintptr_t)a.step;
    const uintptr_t d = b.begin() >= a.begin() ? (b.begin() - a.begin()) % step : (step - (a.begin() - b.begin()) % step) % step;
    return d < (uintptr_t)a.run || d + (uintptr_t)b.run > step;
}

template <int N>
kda_status_t check_runs(const Runs (&a)[N]) {
    for (const Runs &x : a) {
        if (!x.p && x.needed && x.n > 0 && x.run > 0) return set_error(KDA_ERR_INVALID_ARGUMENT, "%s is NULL", x.name);
        if (x.p && !aligned(x.p, x.align))
            return set_error(KDA_ERR_INVALID_ARGUMENT, "%s is not %zu-byte aligned", x.name, x.align);
    }
    for (int i = 0; i < N; ++i) {
        if (!a[i].written || a[i].empty()) continue;
        for (int j = 0; j < N; ++j) {
            if (j == i || a[j].empty() || a[i].apart == j || a[j].apart == i) continue;
            if ((a[i].twin == j || a[j].twin == i) && a[i].p == a[j].p && (a[i].step == a[j].step || a[i].n <= 1)) continue;
            if (meet(a[i], a[j])) return set_error(KDA_ERR_INVALID_ARGUMENT, "%s aliases %s", a[i].name, a[j].name);
        }
    }
    return KDA_OK;
}

constexpr int64_t kMostHeads = 1 << 20;

bool head_dim_ok(int32_t d) { return d == 64 || d == 128; }

// A token stride: given or dense, at least a token's elements, a multiple of 16 bytes, `tokens` of them addressable.
kda_status_t token_stride(const char *name, int64_t given, int64_t row, int64_t elem, int64_t tokens, int64_t &ld) {
    ld = given ? given : row;
    if (ld < row)
        return set_error(KDA_ERR_INVALID_ARGUMENT, "%s %lld is smaller than a token's %lld elements", name, (long long)ld,
                         (long long)row);
    if (ld % (16 / elem) != 0)
        return set_error(KDA_ERR_INVALID_ARGUMENT, "%s %lld is not a multiple of 16 bytes", name, (long long)ld);
    if (tokens > 0 && ld > (1LL << 60) / tokens) return set_error(KDA_ERR_UNSUPPORTED, "tensor too large");
    return KDA_OK;
}

kda_status_t check_rotation(int32_t rot, int32_t interleaved, float amplitude, int32_t d) {
    if (rot < 0 || rot > d || rot % 16 != 0)
        return set_error(KDA_ERR_INVALID_ARGUMENT, "rot_dim %d: a multiple of 16 up to the head's %d is expected", rot, d);
    if (interleaved != 0 && interleaved != 1)
        return set_error(KDA_ERR_INVALID_ARGUMENT, "interleaved is %d, expected 0 or 1", interleaved);
    if (!std::isfinite(amplitude)) return set_error(KDA_ERR_INVALID_ARGUMENT, "amplitude is not finite");
    return KDA_OK;
}

// ------------------------------------------------------------------ paged --
struct Shape {
    int64_t tokens = 0, ldq = 0, ldk = 0, ldv = 0, table_ld = 0;
    int64_t kp[3], vp[3];  // page, head, cell strides
    int64_t io = 2;
    int32_t num_seqs = 0, shift = 0, G = 1;
    int64_t q_row = 0, k_row = 0, v_row = 0;
};

// Strides of a pool: given or dense; no two cells may share memory.
kda_status_t pool_strides(const char *name, const kda_paged_problem_t *p, int64_t elem, int d, const int64_t (&given)[3],
                          int64_t (&out)[3]) {
    const int64_t size[3] = {p->num_pages, p->num_heads_kv, p->page_size};
    if (given[0] == 0 && given[1] == 0 && given[2] == 0) {
        out[2] = d;
        out[1] = out[2] * p->page_size;
        out[0] = out[1] * p->num_heads_kv;
    } else {
        for (int i = 0; i < 3; ++i) out[i] = given[i];
    }
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int a, int b) { return out[a] != out[b] ? out[a] < out[b] : size[a] < size[b]; });
    int64_t inner = d;  // extent of the axes so far
    for (int i : order) {
        if (size[i] <= 1) continue;
        if (out[i] < inner)
            return set_error(KDA_ERR_INVALID_ARGUMENT, "%s: strides %lld, %lld, %lld (page, head, cell) let cells overlap", name,
                             (long long)out[0], (long long)out[1], (long long)out[2]);
        if (out[i] % (16 / elem) != 0)
            return set_error(KDA_ERR_INVALID_ARGUMENT, "%s: stride %lld is not a multiple of 16 bytes", name, (long long)out[i]);
        if (out[i] > (1LL << 58) / size[i]) return set_error(KDA_ERR_UNSUPPORTED, "%s: pool too large", name);
        inner = out[i] * (size[i] - 1) + inner;
    }
    if (out[2] * size[2] > 1LL << 30)  // the kernels reach a head's cells of a page by a 32-bit offset
        return set_error(KDA_ERR_UNSUPPORTED, "%s: %lld cells, %lld elements apart: a head's cells of a page must lie within 2^30 elements",
                         name, (long long)size[2], (long long)out[2]);
    for (int i = 0; i < 3; ++i)
        if (size[i] <= 1) out[i] = 0;
    return KDA_OK;
}
// bytes of one page, from its first to its last element
int64_t page_run(const kda_paged_problem_t *p, const int64_t (&s)[3], int d, int64_t elem) {
    return (s[1] * (p->num_heads_kv - 1) + s[2] * (p->page_size - 1) + d) * elem;
}
// The pool as runs of a page each, or as one run where pages lie inside one another's extent.
Runs pool_runs(const char *name, const void *x, const kda_paged_problem_t *p, const int64_t (&s)[3], int d, int64_t elem,
               bool written) {
    const int64_t run = page_run(p, s, d, elem), step = s[0] * elem;
    if (p->num_pages > 1 && step < run) return {name, x, step * (p->num_pages - 1) + run, 0, 1, 16, true, written};
    return {name, x, run, step, p->num_pages, 16, true, written};
}

// Whether a cell of one pool may share a byte with one of the other, which starts `apart` bytes behind it.  Strides nest
// (pool_strides), so from the widest axis in, cells can only meet for one or two differences of their indexes.  Those are
// followed while the pools have the axis and its stride in common, as slices of one tensor do; behind that a pool's
// remaining axes count as one run.
struct Pool {
    int64_t stride[3], run;  // bytes; stride 0: an axis of one entry, or one that has been followed
};
bool pools_meet(const int64_t (&size)[3], const Pool &a, const Pool &b, int64_t apart) {
    int64_t reach[2];  // bytes from the first to the last
    int widest[2];
    for (int x = 0; x < 2; ++x) {
        const Pool &p = x ? b : a;
        reach[x] = p.run;
        widest[x] = 0;
        for (int i = 0; i < 3; ++i) {
            reach[x] += p.stride[i] * (size[i] - 1);
            if (p.stride[i] > p.stride[widest[x]]) widest[x] = i;
        }
    }
    if (apart >= reach[0] || apart <= -reach[1]) return false;
    const int i = widest[0];
    const int64_t step = a.stride[i];
    if (step == 0 || i != widest[1] || b.stride[i] != step) return true;
    Pool c = a, d = b;
    c.stride[i] = d.stride[i] = 0;
    int64_t more = apart / step;  // indexes that the first is ahead of the second
    if (apart % step < 0) --more;
    for (int64_t n = more; n <= more + 1; ++n)
        if (n < size[i] && -n < size[i] && pools_meet(size, c, d, apart - n * step)) return true;
    return false;
}
kda_status_t check_shape(const kda_paged_problem_t *p, bool packed, Shape &s) {
    if (!p) return set_error(KDA_ERR_INVALID_ARGUMENT, "problem is NULL");
    if (p->batch < 0 || p->seq_len < 0 || p->num_heads_q < 1 || p->num_heads_kv < 1)
        return set_error(KDA_ERR_INVALID_ARGUMENT, "bad sizes: batch=%d seq_len=%d num_heads_q=%d num_heads_kv=%d", p->batch,
                         p->seq_len, p->num_heads_q, p->num_heads_kv);
    if (p->num_heads_q % p->num_heads_kv != 0)
        return set_error(KDA_ERR_INVALID_ARGUMENT, "num_heads_q %d is not a multiple of num_heads_kv %d", p->num_heads_q,
                         p->num_heads_kv);
    if (!dtype_ok(p->io_dtype))
        return set_error(KDA_ERR_INVALID_ARGUMENT, "io_dtype %d is not KDA_F32 or KDA_BF16", (int)p->io_dtype);
    if (!head_dim_ok(p->head_dim_k) || !head_dim_ok(p->head_dim_v))
        return set_error(KDA_ERR_UNSUPPORTED, "head dims d_k=%d d_v=%d: supported are 64 and 128", p->head_dim_k, p->head_dim_v);
    if (p->page_size < 1) return set_error(KDA_ERR_INVALID_ARGUMENT, "page_size %d < 1", p->page_size);
    if (p->page_size < 16 || (p->page_size & (p->page_size - 1)) != 0)
        return set_error(KDA_ERR_UNSUPPORTED, "page_size %d: supported are powers of two from 16 on", p->page_size);
    if (p->max_pages < 0) return set_error(KDA_ERR_INVALID_ARGUMENT, "max_pages %d < 0", p->max_pages);
    if ((int64_t)p->max_pages * p->page_size > 1LL << 30)
        return set_error(KDA_ERR_UNSUPPORTED, "max_pages %d of %d cells: at most 2^30 cells a sequence", p->max_pages, p->page_size);
    if (p->num_pages < 0 || p->num_pages > 0x7fffffffLL)
        return set_error(KDA_ERR_INVALID_ARGUMENT, "num_pages %lld out of range", (long long)p->num_pages);
    if (packed) {
        if (p->batch != 1) return set_error(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens needs batch == 1 (got %d)", p->batch);
        if (p->num_seqs < 0) return set_error(KDA_ERR_INVALID_ARGUMENT, "num_seqs %d < 0", p->num_seqs);
    }
    s.num_seqs = packed ? p->num_seqs : p->batch;
    s.tokens = packed ? p->seq_len : (int64_t)p->batch * p->seq_len;
    s.io = bytes_of(p->io_dtype);
    s.G = p->num_heads_q / p->num_heads_kv;
    if (s.tokens > 0x7fffffffLL || p->num_heads_q > kMostHeads || s.tokens * p->num_heads_q > 0x7fffffffLL)
        return set_error(KDA_ERR_UNSUPPORTED, "too many rows: %lld tokens of %d heads", (long long)s.tokens, p->num_heads_q);
    while ((1 << s.shift) < p->page_size) ++s.shift;
    s.table_ld = p->stride_table ? p->stride_table : p->max_pages;
    if (s.table_ld < p->max_pages || s.table_ld > (1LL << 40))
        return set_error(KDA_ERR_INVALID_ARGUMENT, "stride_table %lld is smaller than max_pages %d", (long long)s.table_ld,
                         p->max_pages);
    s.q_row = (int64_t)p->num_heads_q * p->head_dim_k;
    s.k_row = (int64_t)p->num_heads_kv * p->head_dim_k;
    s.v_row = (int64_t)p->num_heads_kv * p->head_dim_v;
    kda_status_t st = token_stride("stride_q", p->stride_q, s.q_row, s.io, s.tokens, s.ldq);
    if (st == KDA_OK) st = token_stride("stride_k", p->stride_k, s.k_row, s.io, s.tokens, s.ldk);
    if (st == KDA_OK) st = token_stride("stride_v", p->stride_v, s.v_row, s.io, s.tokens, s.ldv);
    const int64_t kg[3] = {p->k_page_stride, p->k_head_stride, p->k_cell_stride},
                  vg[3] = {p->v_page_stride, p->v_head_stride, p->v_cell_stride};
    if (st == KDA_OK) st = pool_strides("k_pages", p, s.io, p->head_dim_k, kg, s.kp);
    if (st == KDA_OK) st = pool_strides("v_pages", p, s.io, p->head_dim_v, vg, s.vp);
    return st;
}

// Keys and values, both to be written, in memory of their own.
kda_status_t check_pools(const kda_paged_problem_t *p, const Shape &s, const void *k, const void *v) {
    if (p->num_pages == 0) return KDA_OK;
    const int64_t size[3] = {p->num_pages, p->num_heads_kv, p->page_size};
    Pool a{{}, p->head_dim_k * s.io}, b{{}, p->head_dim_v * s.io};
    for (int i = 0; i < 3; ++i) {
        a.stride[i] = s.kp[i] * s.io;
        b.stride[i] = s.vp[i] * s.io;
    }
    if (pools_meet(size, a, b, (int64_t)(reinterpret_cast<uintptr_t>(v) - reinterpret_cast<uintptr_t>(k))))
        return set_error(KDA_ERR_INVALID_ARGUMENT, "k_pages aliases v_pages");
    return KDA_OK;
}

Runs table_runs(const kda_paged_problem_t *p, const Shape &s, const int32_t *t) {
    return {"block_table", t, 4LL * p->max_pages, 4 * s.table_ld, s.num_seqs, 4, true, false};
}
Runs dense(const char *name, const void *x, int64_t bytes, size_t align, bool needed, bool written) {
    return {name, x, bytes, 0, 1, align, needed, written};
}

kda::paged::Cache cache_of(const kda_paged_problem_t *p, const Shape &s, const void *k, const void *v, const int32_t *table,
                           const int32_t *lens, const int32_t *cu) {
    kda::paged::Cache c{};
    c.k = const_cast<void *>(k);
    c.v = const_cast<void *>(v);
    c.k_page = s.kp[0], c.k_head = s.kp[1], c.k_cell = s.kp[2];
    c.v_page = s.vp[0], c.v_head = s.vp[1], c.v_cell = s.vp[2];
    c.table = table;
    c.lens = lens;
    c.cu = cu;
    c.table_ld = s.table_ld;
    c.num_pages = p->num_pages;
    c.num_seqs = s.num_seqs;
    c.T = p->seq_len;
    c.max_pages = p->max_pages;
    c.page_shift = s.shift;
    return c;
}

// -------------------------------------------------------------- attention --
using kda::paged::AttnTile;

// Room for the launch that takes sequences of rows_lo to rows_hi rows.
struct Launch {
    AttnTile t{};
    int32_t rows_lo = 1, rows_hi = 0x7fffffff, c_min = 0, target = 0;
    int64_t blocks = 0, tiles = 0, slots = 0;  // workgroups; split tiles and their splits per head
    int64_t most = 0;                          // blocks of a tile, at most
    size_t desc = 0, part = 0;                 // bytes
};

constexpr int64_t kFewBlocks = 16;

// room: bytes of workspace that the launch may take; it cuts its tiles into fewer parts to stay within them.
kda_status_t plan_launch(const kda_paged_problem_t *p, const Shape &s, bool packed, const int32_t *cu_host, int32_t window,
                         int cus, size_t room, Launch &l) {
    const int64_t M = l.t.M, KB = l.t.KB, cells = p->num_pages > 0 ? (int64_t)p->max_pages * p->page_size : 0;
    int64_t tiles = 0;  // of a head, at most
    auto count = [&](int64_t len) { return len * s.G >= l.rows_lo && len * s.G <= l.rows_hi ? (len * s.G + M - 1) / M : 0; };
    if (!packed) {
        tiles = s.num_seqs * count(p->seq_len);
    } else if (cu_host) {
        for (int32_t i = 0; i < s.num_seqs; ++i) tiles += count(cu_host[i + 1] - cu_host[i]);
    } else {
        const int64_t rows = s.tokens * s.G;
        tiles = rows / M + std::min<int64_t>(s.num_seqs, rows / std::max<int64_t>(l.rows_lo, s.G));
    }
    int64_t most = (cells + KB - 1) / KB;  // blocks of a tile, at most
    if (window > 0) most = std::min(most, ((int64_t)window + (M - 1) / s.G + 1 + KB - 1) / KB + 1);
    l.most = most;
    const int64_t Hk = p->num_heads_kv;
    int64_t target = (int64_t)cus * l.t.target_per_cu;
    // No tile is worth splitting: it has few blocks; or they are not many and there are tiles enough; or the blocks of a plain
    // batch's own tokens that its tiles see make parts so long that the kernel would not cut any (without the plan, which costs
    // each workgroup 2 us, and the join, 4 us a call: 4 x 4,096 x 32 heads 577 -> 565 us, 96 x 4 drafted tokens 79 -> 72; for
    // tables about as wide as the batch, as the host knows no lengths).
    // Each of the three holds for every window where it holds without one, and parts of fewer blocks take no more room: so
    // the query, which has no window, counts enough for all of them.
    const bool counted = !packed || cu_host;
    const int64_t own = packed ? 0 : tiles * std::min(most, (std::min<int64_t>(p->seq_len, cells) + KB - 1) / KB);
    if (most <= l.t.c_min || (counted && tiles * Hk >= target && most <= kFewBlocks) || (!packed && own * Hk >= most * target)) {
        l.c_min = packed ? (int32_t)std::max<int64_t>(most, 1) : 0;
        l.blocks = tiles * Hk;
    } else {
        const int64_t each = (most + l.t.c_min - 1) / l.t.c_min;  // parts of a tile, at most
        l.c_min = l.t.c_min;
        for (;; target /= 2) {
            // parts are at least sum / target blocks long: all tiles have at most one part more than target / Hk together; a split
            // tile has more than one part's blocks, hence at most twice as many parts as blocks / part
            l.blocks = std::min(target / Hk + tiles, tiles * each) * Hk;
            l.tiles = std::min(target / Hk, tiles);
            l.slots = std::min(2 * target / Hk, tiles * each);
            if (tiles == 0 || l.slots < 2) l.tiles = l.slots = 0;
            l.desc = (size_t)((1 + l.tiles * Hk) * kda::paged::kDesc * 4 + 255) / 256 * 256;
            l.part = (size_t)(l.slots * Hk * M * (p->head_dim_v + 2) * 4 + 255) / 256 * 256;
            if (l.desc + l.part <= room || target <= 1) break;
        }
        if (l.desc + l.part > room) {  // none: tiles of up to `most` blocks are one part
            l.c_min = (int32_t)std::max<int64_t>(most, 1);
            l.blocks = tiles * Hk;
            l.tiles = l.slots = 0;
            l.desc = l.part = 0;
        }
    }
    l.target = (int32_t)target;
    if (l.blocks > kMostItems / l.t.threads || l.tiles * Hk * M > kMostItems / 256)
        return set_error(KDA_ERR_UNSUPPORTED, "too many rows: %lld workgroups", (long long)l.blocks);
    return KDA_OK;
}

struct AttnPlan {
    Launch part[2];
    bool tile[2] = {false, false};
    int n = 0;
    size_t bytes = 0;
};

// Sequences of few rows go to the kernel for few rows, longer ones of bf16 calls to the one that stages cells in LDS for 256 rows.
// Few: 32, two tiles that read the cells from HBM once (2 sequences of 24 rows over 1,600 cells 25.0 -> 17.7 us, 64 of 32 over
// 100 27.5 -> 16.3; 64 of 36 over 4,000 cells 297, and 315 as few); 64 in calls of few sequences and heads, where the
// other kernel's longer start counts (1 of 64 rows over 30,000 cells, 8 key heads: 78 -> 57; 8 of them over 8,000: 90, 97 as few).
// A packed batch may hold both, and what its offsets do not rule out on the host is launched, but for a batch with no more
// tokens than sequences: the step of one token each that it looks like needs no second launch, and longer sequences among
// empty ones come out the same from the first.
// All rows are few in calls of little work, at most 12 M pairs of (row, key head) and cells that a table has room for (the host
// knows no lengths, so that a table wider than its batch takes this gain away): one round of
// the kernel for few rows is then over before the other one's workgroups have started (1 x 128 tokens over 628 cells,
// 32 / 8 heads: 33 -> 22 us; 3 ragged chunks of up to 700 over 300: 47 -> 21; 64 x 9 over 209: 36 -> 26; beyond,
// 1 x 128 over 4,028: 40 both ways, 8 x 40 over 2,040: 40, 70 as few).
int32_t few_rows(int64_t num_seqs, int64_t heads_kv, int64_t rows, int64_t cells) {
    if (rows * heads_kv <= (12LL << 20) / std::max<int64_t>(cells, 1)) return 0x7fffffff;
    return num_seqs * heads_kv <= 32 ? 64 : 32;
}

kda_status_t plan_attn(const kda_paged_problem_t *p, const Shape &s, bool packed, const int32_t *cu_host, int32_t window, int cus,
                       size_t room, AttnPlan &a) {
    a = AttnPlan{};
    const bool bf16 = p->io_dtype == KDA_BF16;
    const int32_t few = few_rows(s.num_seqs, p->num_heads_kv, s.tokens * s.G, p->num_pages > 0 ? (int64_t)p->max_pages * p->page_size : 0);
    const bool both = bf16 && few < 0x7fffffff && (!packed || cu_host || s.tokens > s.num_seqs);
    for (int tile = 0; tile < (both ? 2 : 1); ++tile) {
        Launch l;
        l.t = tile ? kda::paged::attn_tile_tile() : kda::paged::attn_rows_tile(bf16);
        if (tile) l.rows_lo = few + 1;
        if (both && !tile) l.rows_hi = few;
        const kda_status_t st = plan_launch(p, s, packed, cu_host, window, cus, room, l);
        if (st != KDA_OK) return st;
        if (l.blocks == 0) continue;
        a.bytes = std::max(a.bytes, l.desc + l.part);  // one after the other, in the same room
        a.tile[a.n] = tile;
        a.part[a.n++] = l;
    }
    return KDA_OK;
}

// Room for the problem as a plain batch and, where it can be one, as a packed one, whatever lengths, window and host offsets.
// Only offsets on the host can need more than the plans without a window and without them: in a batch of no more tokens than
// sequences they may show rows for a second launch.  That one stays within this room (or the caller's, if it is larger), rather
// than have every step of single tokens ask for eight times as much (64 sequences over 8,192 cells, 32 / 8 heads of 128: 17 MB,
// 136 with it).
kda_status_t room_of(const kda_paged_problem_t *p, int cus, size_t &room) {
    size_t need = 0;
    for (int packed = 0; packed < 2; ++packed) {
        if (packed && (!p || p->batch != 1 || p->num_seqs <= 0)) break;
        Shape s;
        AttnPlan a;
        kda_status_t st = check_shape(p, packed, s);
        if (st == KDA_OK) st = plan_attn(p, s, packed, nullptr, 0, cus, SIZE_MAX, a);
        if (st != KDA_OK) return st;
        need = std::max(need, a.bytes);
    }
    room = need;
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status_t kda_rope(const kda_rope_problem_t *p, const void *q, const void *k, const int32_t *positions,
                      const float *inv_freq, void *q_out, void *k_out, void *stream) {
    try {
        if (!p) return set_error(KDA_ERR_INVALID_ARGUMENT, "problem is NULL");
        if (p->batch < 0 || p->seq_len < 0 || p->num_heads_q < 1 || p->num_heads_k < 0)
            return set_error(KDA_ERR_INVALID_ARGUMENT, "bad sizes: batch=%d seq_len=%d num_heads_q=%d num_heads_k=%d", p->batch,
                             p->seq_len, p->num_heads_q, p->num_heads_k);
        if (!dtype_ok(p->io_dtype))
            return set_error(KDA_ERR_INVALID_ARGUMENT, "io_dtype %d is not KDA_F32 or KDA_BF16", (int)p->io_dtype);
        if (!head_dim_ok(p->head_dim))
            return set_error(KDA_ERR_UNSUPPORTED, "head_dim %d: supported are 64 and 128", p->head_dim);
        if (p->inverse != 0 && p->inverse != 1)
            return set_error(KDA_ERR_INVALID_ARGUMENT, "inverse is %d, expected 0 or 1", p->inverse);
        kda_status_t st = check_rotation(p->rot_dim, p->interleaved, p->amplitude, p->head_dim);
        if (st != KDA_OK) return st;
        const int64_t tokens = (int64_t)p->batch * p->seq_len, io = bytes_of(p->io_dtype);
        const int64_t q_row = (int64_t)p->num_heads_q * p->head_dim, k_row = (int64_t)p->num_heads_k * p->head_dim;
        int64_t ldq, ldk, ldqo, ldko;
        st = token_stride("stride_q", p->stride_q, q_row, io, tokens, ldq);
        if (st == KDA_OK) st = token_stride("stride_k", p->stride_k, k_row, io, tokens, ldk);
        if (st == KDA_OK) st = token_stride("stride_q_out", p->stride_q_out, q_row, io, tokens, ldqo);
        if (st == KDA_OK) st = token_stride("stride_k_out", p->stride_k_out, k_row, io, tokens, ldko);
        if (st != KDA_OK) return st;
        const int64_t heads = (int64_t)p->num_heads_q + p->num_heads_k;
        if (tokens > 0x7fffffffLL || heads > kMostHeads || kda::paged::rope_items(tokens, (int32_t)heads, p->head_dim) > kMostItems - 255)
            return set_error(KDA_ERR_UNSUPPORTED, "too many rows: %lld tokens of %d + %d heads", (long long)tokens, p->num_heads_q,
                             p->num_heads_k);
        if (p->num_heads_k == 0) k = k_out = nullptr;
        const Runs args[] = {
            {"q", q, q_row * io, ldq * io, tokens, 16, true, false},
            {"k", k, k_row * io, ldk * io, tokens, 16, true, false},
            dense("positions", positions, 4 * tokens, 4, false, false),
            dense("inv_freq", inv_freq, tokens > 0 ? 2LL * p->rot_dim : 0, 4, true, false),
            {"q_out", q_out, q_row * io, ldqo * io, tokens, 16, true, true, 0},
            {"k_out", k_out, k_row * io, ldko * io, tokens, 16, true, true, 1},
        };
        st = check_runs(args);
        if (st != KDA_OK) return st;
        if (tokens == 0) return done(hipSuccess, "");
        kda::paged::RopeParams r{};
        r.q = q, r.k = k, r.q_out = q_out, r.k_out = k_out;
        r.positions = positions;
        r.freq = inv_freq;
        r.ldq = ldq, r.ldk = ldk, r.ldqo = ldqo, r.ldko = ldko;
        r.tokens = tokens;
        r.T = p->seq_len;
        r.Hq = p->num_heads_q;
        r.Hk = p->num_heads_k;
        r.d = p->head_dim;
        r.rot = p->rot_dim;
        r.interleaved = p->interleaved;
        r.amplitude = p->amplitude;
        r.sign = p->inverse ? -1.f : 1.f;
        return done(kda::paged::launch_rope(p->io_dtype == KDA_BF16, r, static_cast<hipStream_t>(stream)), "kda_rope launch");
    } catch (...) {
        return set_error(KDA_ERR_HIP, "unexpected exception in argument checks");
    }
}

kda_status_t kda_rope_frequencies(int32_t rot_dim, double base, int32_t scaling, double factor, int64_t original_len,
                                  double slow, double fast, float *inv_freq_host, float *amplitude_host) {
    try {
        if (rot_dim < 0 || rot_dim % 16 != 0 || rot_dim > 1 << 20)
            return set_error(KDA_ERR_INVALID_ARGUMENT, "rot_dim %d is not a multiple of 16", rot_dim);
        if (!std::isfinite(base) || base <= 1.0) return set_error(KDA_ERR_INVALID_ARGUMENT, "base must be finite and > 1");
        if (scaling < KDA_ROPE_PLAIN || scaling > KDA_ROPE_PARTS)
            return set_error(KDA_ERR_INVALID_ARGUMENT, "scaling %d is none of kda_rope_scaling_t", scaling);
        if (scaling != KDA_ROPE_PLAIN && (!std::isfinite(factor) || factor < 1.0))
            return set_error(KDA_ERR_INVALID_ARGUMENT, "factor must be finite and >= 1");
        if (scaling == KDA_ROPE_PARTS &&
            (original_len < 1 || !std::isfinite(slow) || !std::isfinite(fast) || slow < 0.0 || fast <= slow))
            return set_error(KDA_ERR_INVALID_ARGUMENT, "original_len >= 1 and 0 <= slow < fast are expected");
        if ((rot_dim > 0 && !inv_freq_host) || !amplitude_host)
            return set_error(KDA_ERR_INVALID_ARGUMENT, "inv_freq_host or amplitude_host is NULL");
        if (scaling == KDA_ROPE_BASE && rot_dim > 0) base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
        for (int32_t i = 0; i < rot_dim / 2; ++i) {
            double f = std::pow(base, -2.0 * i / rot_dim);
            if (scaling == KDA_ROPE_LINEAR) f /= factor;
            if (scaling == KDA_ROPE_PARTS) {
                const double turns = (double)original_len * f / 6.283185307179586477;
                const double keep = std::min(1.0, std::max(0.0, (turns - slow) / (fast - slow)));
                f *= keep + (1.0 - keep) / factor;
            }
            inv_freq_host[i] = (float)f;
        }
        *amplitude_host = scaling == KDA_ROPE_PARTS ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
        return done(hipSuccess, "");
    } catch (...) {
        return set_error(KDA_ERR_HIP, "unexpected exception in argument checks");
    }
}

kda_status_t kda_paged_append(const kda_paged_problem_t *p, const void *k, const void *v, const void *q, const kda_rope_t *rope,
                              const int32_t *block_table, const int32_t *kv_lens, const int32_t *cu_seqlens,
                              const int32_t *cu_seqlens_host, void *k_pages, void *v_pages, void *q_out, void *stream) {
    try {
        Shape s;
        kda_status_t st = check_shape(p, cu_seqlens != nullptr, s);
        if (st != KDA_OK) return st;
        if (q && !rope) return set_error(KDA_ERR_INVALID_ARGUMENT, "q is given without rope");
        if (q_out && !q) return set_error(KDA_ERR_INVALID_ARGUMENT, "q_out is given without q");
        if (rope) {
            st = check_rotation(rope->rot_dim, rope->interleaved, rope->amplitude, p->head_dim_k);
            if (st != KDA_OK) return st;
        }
        if (s.tokens > 0 &&
            kda::paged::append_items(s.tokens, q ? p->num_heads_q : 0, p->num_heads_kv, p->head_dim_k, p->head_dim_v) > kMostItems - 255)
            return set_error(KDA_ERR_UNSUPPORTED, "too many rows: %lld tokens", (long long)s.tokens);
        const bool turned = rope && rope->rot_dim > 0;
        const int64_t ldqo = q_out && q_out == q ? s.ldq : s.q_row;
        Runs args[] = {
            {"k", k, s.k_row * s.io, s.ldk * s.io, s.tokens, 16, true, false},
            {"v", v, s.v_row * s.io, s.ldv * s.io, s.tokens, 16, true, false},
            {"q", q, s.q_row * s.io, s.ldq * s.io, s.tokens, 16, false, false},
            {"q_out", q_out, s.q_row * s.io, ldqo * s.io, q ? s.tokens : 0, 16, true, true, 2},
            dense("inv_freq", turned ? rope->inv_freq : nullptr, turned && s.tokens > 0 ? 2LL * rope->rot_dim : 0, 4, true, false),
            dense("positions", rope ? rope->positions : nullptr, 4 * s.tokens, 4, false, false),
            table_runs(p, s, block_table),
            dense("kv_lens", kv_lens, 4LL * s.num_seqs, 4, true, false),
            dense("cu_seqlens", cu_seqlens, 4 * ((int64_t)s.num_seqs + 1), 4, false, false),
            pool_runs("k_pages", k_pages, p, s.kp, p->head_dim_k, s.io, true),
            pool_runs("v_pages", v_pages, p, s.vp, p->head_dim_v, s.io, true),
        };
        args[9].apart = 10;
        st = check_runs(args);
        if (st == KDA_OK) st = check_pools(p, s, k_pages, v_pages);
        if (st == KDA_OK) st = check_offsets(p->seq_len, s.num_seqs, cu_seqlens, cu_seqlens_host);
        if (st != KDA_OK) return st;
        if (s.num_seqs == 0 || s.tokens == 0) return done(hipSuccess, "");
        kda::paged::AppendParams r{};
        r.c = cache_of(p, s, k_pages, v_pages, block_table, kv_lens, cu_seqlens);
        r.k = k, r.v = v, r.q = q;
        r.q_out = q_out;
        r.positions = rope ? rope->positions : nullptr;
        r.freq = rope ? rope->inv_freq : nullptr;
        r.ldk = s.ldk, r.ldv = s.ldv, r.ldq = s.ldq, r.ldqo = ldqo;
        r.tokens = s.tokens;
        r.Hq = p->num_heads_q;
        r.Hk = p->num_heads_kv;
        r.dk = p->head_dim_k;
        r.dv = p->head_dim_v;
        r.rot = rope ? rope->rot_dim : 0;
        r.interleaved = rope ? rope->interleaved : 0;
        r.amplitude = rope ? rope->amplitude : 1.f;
        return done(kda::paged::launch_append(p->io_dtype == KDA_BF16, r, static_cast<hipStream_t>(stream)),
                    "kda_paged_append launch");
    } catch (...) {
        return set_error(KDA_ERR_HIP, "unexpected exception in argument checks");
    }
}

kda_status_t kda_paged_attn_workspace(const kda_paged_problem_t *p, size_t *bytes) {
    if (!bytes) return set_error(KDA_ERR_INVALID_ARGUMENT, "bytes is NULL");
    *bytes = 0;
    try {
        size_t need = 0;
        const kda_status_t st = room_of(p, current_cus(), need);
        if (st != KDA_OK) return st;
        *bytes = need;
        return done(hipSuccess, "");
    } catch (...) {
        return set_error(KDA_ERR_HIP, "unexpected exception in argument checks");
    }
}

kda_status_t kda_paged_attn(const kda_paged_problem_t *p, const void *q, const void *k_pages, const void *v_pages,
                            const int32_t *block_table, const int32_t *kv_lens, const int32_t *cu_seqlens,
                            const int32_t *cu_seqlens_host, float scale, int32_t window, void *out, float *lse, void *workspace,
                            size_t workspace_bytes, void *stream) {
    try {
        Shape s;
        kda_status_t st = check_shape(p, cu_seqlens != nullptr, s);
        if (st != KDA_OK) return st;
        if (!std::isfinite(scale)) return set_error(KDA_ERR_INVALID_ARGUMENT, "scale is not finite");
        if (window < 0) return set_error(KDA_ERR_INVALID_ARGUMENT, "window %d < 0", window);
        const int64_t rows = s.tokens * p->num_heads_q;
        Runs args[] = {
            {"q", q, s.q_row * s.io, s.ldq * s.io, s.tokens, 16, true, false},
            table_runs(p, s, block_table),
            dense("kv_lens", kv_lens, 4LL * s.num_seqs, 4, true, false),
            dense("cu_seqlens", cu_seqlens, 4 * ((int64_t)s.num_seqs + 1), 4, false, false),
            pool_runs("k_pages", k_pages, p, s.kp, p->head_dim_k, s.io, false),
            pool_runs("v_pages", v_pages, p, s.vp, p->head_dim_v, s.io, false),
            dense("out", out, rows * p->head_dim_v * s.io, 16, true, true),
            dense("lse", lse, rows * 4, 4, false, true),
            dense("workspace", workspace, 0, 256, false, true),
        };
        st = check_runs(args);
        if (st == KDA_OK) st = check_offsets(p->seq_len, s.num_seqs, cu_seqlens, cu_seqlens_host);
        if (st != KDA_OK) return st;
        AttnPlan a;
        const int cus = current_cus();
        size_t room = SIZE_MAX;  // (kept where the query refuses the problem: exact offsets may name fewer workgroups than it counts)
        if (cu_seqlens_host && room_of(p, cus, room) == KDA_OK) room = std::max(room, workspace_bytes);
        st = plan_attn(p, s, cu_seqlens != nullptr, cu_seqlens_host, window, cus, room, a);
        if (st != KDA_OK) return st;
        args[8].run = (int64_t)a.bytes;
        st = check_runs(args);
        if (st != KDA_OK) return st;
        if (a.bytes > 0 && (!workspace || workspace_bytes < a.bytes))
            return set_error(KDA_ERR_WORKSPACE, "kda_paged_attn needs a 256-byte aligned workspace of %zu bytes (got %zu at %p)",
                             a.bytes, workspace_bytes, workspace);
        if (s.num_seqs == 0 || s.tokens == 0) return done(hipSuccess, "");
        kda::paged::AttnParams r{};
        r.c = cache_of(p, s, k_pages, v_pages, block_table, kv_lens, cu_seqlens);
        r.q = q;
        r.out = out;
        r.lse = lse;
        r.ldq = s.ldq;
        r.Hq = p->num_heads_q;
        r.Hk = p->num_heads_kv;
        r.G = s.G;
        r.by_G = kda::paged::Div(s.G);
        r.by_Hk = kda::paged::Div(p->num_heads_kv);
        r.dk = p->head_dim_k;
        r.dv = p->head_dim_v;
        r.window = window;
        // the kernels multiply by |scale|, never by 0: a masked score of -inf stays what it is (scores of finite inputs
        // times the least normal number are 0 beside any weight's rounding)
        r.scale = std::min(std::max(std::fabs(scale) * 1.4426950408889634f, 1.17549435e-38f), 3.40282347e38f);
        r.flip = std::signbit(scale);
        const bool bf16 = p->io_dtype == KDA_BF16;
        hipStream_t hs = static_cast<hipStream_t>(stream);
        char *const ws = static_cast<char *>(workspace);
        for (int i = 0; i < a.n; ++i) {
            const Launch &l = a.part[i];
            // fp32 heads of 128: two workgroups of 237 registers on a CU suit single rows and short contexts, whose
            // latency counts (3 x 229 tokens x 32 heads 59 -> 44 us, 59 x 8 tokens over 563 cells 66 -> 56); one of 270, which
            // keeps more loads in flight, many rows over long ones (4 x 512 tokens over 4,608 cells 984 -> 794)
            const bool many = s.tokens * s.G > 16LL * s.num_seqs && l.most > 4;
            r.rows_lo = l.rows_lo;
            r.rows_hi = l.rows_hi;
            r.c_min = l.c_min;
            r.target = l.target;
            r.tiles = (int32_t)l.tiles;
            r.slots = (int32_t)l.slots;
            r.desc = l.desc ? reinterpret_cast<int32_t *>(ws) : nullptr;
            r.part = reinterpret_cast<float *>(ws + l.desc);
            st = done(a.tile[i] ? kda::paged::launch_attn_tile(r, l.blocks, hs) : kda::paged::launch_attn_rows(bf16, many, r, l.blocks, hs),
                      "kda_paged_attn launch");
            if (st == KDA_OK && l.tiles > 0)
                st = done(kda::paged::launch_attn_join(bf16, r, l.t.M, l.tiles, hs), "kda_paged_attn join launch");
            if (st != KDA_OK) return st;
        }
        return done(hipSuccess, "");
    } catch (...) {
        return set_error(KDA_ERR_HIP, "unexpected exception in argument checks");
    }
}

}  // extern "C"
