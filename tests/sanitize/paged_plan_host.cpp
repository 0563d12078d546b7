// What kda_paged_attn plans on the host against what its workgroups make of it on the device, built with AddressSanitizer and
// UndefinedBehaviorSanitizer: launches are taken down here instead of made, and the plan that every workgroup works out (sums of
// blocks, the cut, parts, split tiles) is worked out again from real lengths.  Every row has to be some launch's, every part a
// workgroup's, every split tile and every part of one has to have its room, and all of it has to lie in what the query named.
//
// Exit status 0 when every expectation holds (and no sanitizer report aborted the run).
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "kda.h"
#include "kda_paged.h"

extern "C" hipError_t hipGetDevice(int *) { return hipErrorInvalidValue; }  // (256 CUs)

namespace {

int g_failures = 0, g_checks = 0;
void expect(bool ok, const char *what, int line) {
    ++g_checks;
    if (!ok && ++g_failures < 20) std::fprintf(stderr, "FAILED line %d: %s (last error: %s)\n", line, what, kda_last_error());
}
#define EXPECT(cond) expect((cond), #cond, __LINE__)

struct Taken {
    kda::paged::AttnParams p;
    int M, KB;
    int64_t blocks, join;
};
std::vector<Taken> g_taken;

uint64_t g_rng = 0x2545F4914F6CDD1Dull;
uint64_t next_u64() {  // xorshift64*
    g_rng ^= g_rng >> 12;
    g_rng ^= g_rng << 25;
    g_rng ^= g_rng >> 27;
    return g_rng * 0x9E3779B97F4A7C15ull;
}
int64_t below(int64_t n) { return (int64_t)(next_u64() % (uint64_t)n); }
int64_t spread(int64_t lo, int64_t hi) {  // over the logarithm
    return (int64_t)std::llround(lo * std::pow((double)hi / lo, (next_u64() >> 11) * 0x1p-53));
}
template <typename T, size_t N>
T pick(const T (&a)[N]) {
    return a[next_u64() % N];
}
void *dev(uintptr_t i) { return reinterpret_cast<void *>((i + 1) << 44); }

}  // namespace

namespace kda {
namespace paged {
hipError_t launch_attn_rows(bool bf16, bool, const AttnParams &p, int64_t blocks, hipStream_t) {
    const AttnTile t = attn_rows_tile(bf16);
    g_taken.push_back({p, t.M, t.KB, blocks, 0});
    return hipSuccess;
}
hipError_t launch_attn_tile(const AttnParams &p, int64_t blocks, hipStream_t) {
    const AttnTile t = attn_tile_tile();
    g_taken.push_back({p, t.M, t.KB, blocks, 0});
    return hipSuccess;
}
hipError_t launch_attn_join(bool, const AttnParams &p, int M, int64_t tiles, hipStream_t) {
    EXPECT(!g_taken.empty() && g_taken.back().M == M && g_taken.back().p.desc == p.desc);
    g_taken.back().join = tiles;
    return hipSuccess;
}
hipError_t launch_append(bool, const AppendParams &, hipStream_t) { return hipSuccess; }
}  // namespace paged
}  // namespace kda

namespace {

struct Batch {
    std::vector<int32_t> cu, lens;  // offsets (packed) and cells
};

// One launch against the lengths; rows that it takes are added up.
int check(const Taken &t, const kda_paged_problem_t &pr, const Batch &b, const char *ws, size_t room, std::vector<int> &rows_taken) {
    const kda::paged::AttnParams &p = t.p;
    const kda::paged::Cache &c = p.c;
    const int64_t M = t.M, KB = t.KB, Hk = p.Hk;
    const int64_t cells = c.num_pages > 0 ? (int64_t)c.max_pages << c.page_shift : 0;
    std::vector<int64_t> tiles(c.num_seqs), blocks(c.num_seqs);
    int64_t total = 0;
    for (int n = 0; n < c.num_seqs; ++n) {
        const int64_t len = c.cu ? b.cu[n + 1] - b.cu[n] : c.T, rows = len * p.G;
        if (rows < p.rows_lo || rows > p.rows_hi) continue;
        rows_taken[n] += 1;
        tiles[n] = (rows + M - 1) / M;
        const int64_t all = (std::min<int64_t>(std::max(b.lens[n], 0), cells) + KB - 1) / KB;
        blocks[n] = p.window > 0 ? std::min(all, ((int64_t)p.window + (M - 1) / p.G + 1 + KB - 1) / KB + 1) : all;
        total += tiles[n] * blocks[n];
    }
    int64_t parts = 0, slots = 0, stiles = 0;
    if (p.c_min == 0) {
        EXPECT(!c.cu && !t.join);
        parts = (int64_t)c.num_seqs * (((int64_t)c.T * p.G + M - 1) / M);
    } else {
        EXPECT(p.target >= 1);
        const int64_t cut = std::max<int64_t>(p.c_min, (total * Hk + p.target - 1) / p.target);
        for (int n = 0; n < c.num_seqs; ++n) {
            const int64_t cuts = blocks[n] > cut ? (blocks[n] + cut - 1) / cut : 1;
            parts += tiles[n] * cuts;
            if (cuts > 1) slots += tiles[n] * cuts, stiles += tiles[n];
        }
    }
    EXPECT(parts * Hk <= t.blocks);
    EXPECT(slots <= p.slots && stiles <= p.tiles && stiles <= t.join);
    EXPECT(stiles == 0 || (p.desc && p.part));
    if (p.slots > 0 || p.tiles > 0) {
        const char *desc = reinterpret_cast<const char *>(p.desc), *part = reinterpret_cast<const char *>(p.part);
        EXPECT(desc >= ws && desc + (1 + (int64_t)p.tiles * Hk) * kda::paged::kDesc * 4 <= part);
        EXPECT(part + (int64_t)p.slots * Hk * M * (pr.head_dim_v + 2) * 4 <= ws + room);
        EXPECT(reinterpret_cast<uintptr_t>(part) % 256 == 0);
    } else if (p.desc) {
        EXPECT(reinterpret_cast<const char *>(p.desc) >= ws && reinterpret_cast<const char *>(p.desc + kda::paged::kDesc) <= ws + room);
    }
    return slots > 0;
}

void attention(int n) {
    const int32_t heads[] = {1, 1, 2, 3, 4, 8, 8, 16, 64, 300, 600}, groups[] = {1, 1, 2, 4, 4, 5, 8, 32}, dims[] = {64, 128}, pages[] = {16, 64, 256};
    int split = 0, two = 0, few = 0, tight = 0;
    for (int i = 0; i < n; ++i) {
        kda_paged_problem_t p;
        std::memset(&p, 0, sizeof p);
        const bool packed = below(3) != 0;
        const int64_t seqs = spread(1, 700), tokens = spread(1, 30000);
        p.batch = packed ? 1 : (int32_t)seqs;
        p.seq_len = packed ? (int32_t)tokens : (int32_t)std::max<int64_t>(1, tokens / seqs);
        p.num_seqs = packed ? (int32_t)seqs : 0;
        p.num_heads_kv = pick(heads);
        p.num_heads_q = p.num_heads_kv * pick(groups);
        p.head_dim_k = pick(dims);
        p.head_dim_v = pick(dims);
        p.io_dtype = below(3) ? KDA_BF16 : KDA_F32;
        p.page_size = pick(pages);
        p.max_pages = (int32_t)spread(1, 4000);
        p.num_pages = 1 << 14;
        Batch b;
        const int64_t cells = (int64_t)p.max_pages * p.page_size;
        if (packed) {  // cut at random, or among few of the sequences
            const int64_t kinds = below(3), some = kinds ? seqs : std::min<int64_t>(seqs, 1 + below(4));
            b.cu.assign(seqs + 1, 0);
            for (int64_t t = 0; t < (kinds == 2 ? 0 : tokens); ++t) ++b.cu[1 + (kinds ? below(seqs) : below(some) * (seqs / some))];
            if (kinds == 2) {  // single tokens and the rest in one sequence
                for (int64_t s = 0; s < seqs; ++s) b.cu[1 + s] = s < tokens / 2;
                int64_t used = std::min(seqs, tokens / 2);
                b.cu[seqs] += (int32_t)(tokens - used);
            }
            for (int64_t s = 0; s < seqs; ++s) b.cu[s + 1] += b.cu[s];
            EXPECT(b.cu[seqs] == tokens);
        }
        for (int64_t s = 0; s < seqs; ++s) {
            const int64_t kind = below(4);
            b.lens.push_back((int32_t)(kind == 0 ? below(cells + 100) : kind == 1 ? cells : kind == 2 ? spread(1, cells) : below(40) - 3));
        }
        size_t room = 0;
        const kda_status_t asked = kda_paged_attn_workspace(&p, &room);
        if (asked != KDA_OK) {  // more workgroups than a launch has
            EXPECT(asked == KDA_ERR_UNSUPPORTED && p.num_heads_kv >= 300 && room == 0);
            continue;
        }
        for (int host = 0; host < (packed ? 2 : 1); ++host)
            for (int more = 0; more < 2; ++more) {
                const int32_t window = below(2) ? 0 : (int32_t)spread(1, 2 * cells);
                const size_t given = more ? room * 3 + 5000 : room;
                char *const ws = static_cast<char *>(dev(8));
                g_taken.clear();
                const kda_status_t st = kda_paged_attn(&p, dev(0), dev(1), dev(2), static_cast<int32_t *>(dev(3)), b.lens.data(),
                                                       packed ? b.cu.data() : nullptr, host ? b.cu.data() : nullptr, 1.f, window, dev(4),
                                                       nullptr, given ? ws : nullptr, given, nullptr);
                EXPECT(st == KDA_OK);
                if (st != KDA_OK) continue;
                std::vector<int> rows(seqs, 0);
                for (const Taken &t : g_taken) split += check(t, p, b, ws, given, rows);
                for (int64_t s = 0; s < seqs; ++s) EXPECT(rows[s] == (packed ? b.cu[s + 1] > b.cu[s] : 1));
                two += g_taken.size() > 1;
                few += host && tokens <= seqs && g_taken.size() > 1;
                for (const Taken &t : g_taken) tight += t.p.target < 512 && t.p.c_min > 0;
            }
    }
    std::printf("%d launches split, %d calls of two, %d of them by host offsets alone, %d launches kept within their room\n", split, two, few,
                tight);
    EXPECT(split > n / 4 && two > n / 20 && few > n / 100 && tight > 0);
}

// Pools of any strides, over each other or not: no arithmetic may overflow, whatever the answer.
void pools(int n) {
    const int64_t strides[] = {0, 64, 128, 192, 1 << 10, 1 << 14, (int64_t)1 << 26, (int64_t)1 << 40, (int64_t)1 << 57, INT64_MAX};
    const int64_t counts[] = {0, 1, 2, 1000, INT32_MAX};
    const int32_t offsets[] = {0, 3, 2, 8, 15};  // (decreasing: refused behind the pools)
    int past = 0, met = 0;
    for (int i = 0; i < n; ++i) {
        kda_paged_problem_t p;
        std::memset(&p, 0, sizeof p);
        p.batch = 1;
        p.seq_len = 15;
        p.num_seqs = 4;
        p.num_heads_kv = p.num_heads_q = (int32_t)(1 + below(4));
        p.head_dim_k = below(2) ? 64 : 128;
        p.head_dim_v = below(2) ? 64 : 128;
        p.io_dtype = below(2) ? KDA_BF16 : KDA_F32;
        p.page_size = below(4) ? 16 : 1 << 20;
        p.max_pages = 7;
        p.num_pages = pick(counts);
        p.k_page_stride = pick(strides), p.k_head_stride = pick(strides), p.k_cell_stride = pick(strides);
        p.v_page_stride = p.k_page_stride, p.v_head_stride = p.k_head_stride, p.v_cell_stride = p.k_cell_stride;
        if (below(2)) p.v_head_stride = pick(strides);
        const uintptr_t k = (uintptr_t)1 << 46;
        const uintptr_t v = below(8) ? k + (uintptr_t)(16 * spread(1, (int64_t)1 << 40)) : (uintptr_t)0 - ((uintptr_t)1 << 44);
        const kda_status_t st = kda_paged_append(&p, dev(0), dev(1), nullptr, nullptr, static_cast<int32_t *>(dev(2)),
                                                 static_cast<int32_t *>(dev(3)), static_cast<int32_t *>(dev(4)), offsets,
                                                 reinterpret_cast<void *>(below(2) ? k : v), reinterpret_cast<void *>(below(16) ? v : k), nullptr,
                                                 nullptr);
        EXPECT(st != KDA_OK);
        past += std::strstr(kda_last_error(), "decreases") != nullptr;
        met += std::strstr(kda_last_error(), "k_pages aliases v_pages") != nullptr;
    }
    std::printf("%d pools apart, %d not\n", past, met);
    EXPECT(past > n / 100 && met > n / 100);
}

}  // namespace

int main(int argc, char **argv) {
    const int n = argc > 1 ? std::atoi(argv[1]) : 1000;
    attention(n);
    pools(4 * n);
    std::printf("%d checks, %d failed\n", g_checks, g_failures);
    return g_failures != 0;
}
