// Host-side checks of rotary positions and of the paged cache's entry points, built with AddressSanitizer and
// UndefinedBehaviorSanitizer around their host code.  Every call is refused by validation or describes an empty problem,
// so no kernel is reached; host arrays are allocated at their exact sizes.
//
// Exit status 0 when every expectation holds (and no sanitizer report aborted the run).
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <limits>
#include <memory>
#include <vector>

#include "kda.h"
#include "kda_paged.h"

// Takes the runtime's place: a refused call asks nothing of it.
static int g_device_queries = 0;
extern "C" hipError_t hipGetDevice(int *) {
    ++g_device_queries;
    return hipErrorInvalidValue;
}

namespace {

int g_failures = 0, g_checks = 0;

void expect(bool ok, const char *what, int line) {
    ++g_checks;
    if (!ok) {
        ++g_failures;
        std::fprintf(stderr, "FAILED line %d: %s (last error: %s)\n", line, what, kda_last_error());
    }
}
#define EXPECT(cond) expect((cond), #cond, __LINE__)

// Fake device addresses: aligned, far apart, never dereferenced on the host.
void *dev(uintptr_t i, uintptr_t off = 0) { return reinterpret_cast<void *>((i + 1) << 44 | off); }
template <typename T>
T *dev_of(uintptr_t i) {
    return static_cast<T *>(dev(i));
}

uint64_t g_rng = 0x9E3779B97F4A7C15ull;
uint64_t next_u64() {  // xorshift64*
    g_rng ^= g_rng >> 12;
    g_rng ^= g_rng << 25;
    g_rng ^= g_rng >> 27;
    return g_rng * 0x2545F4914F6CDD1Dull;
}
template <typename T, size_t N>
T pick(const T (&a)[N]) {
    return a[next_u64() % N];
}

struct Args {
    void *q = dev(0), *k = dev(1), *v = dev(2), *out = dev(3), *kp = dev(4), *vp = dev(5), *q_out = nullptr, *ws = dev(6);
    const kda_rope_t *rope = nullptr;
    int32_t *table = dev_of<int32_t>(7), *lens = dev_of<int32_t>(8), *cu = nullptr;
    const int32_t *cu_host = nullptr;
    float *lse = dev_of<float>(9);
    size_t room = ~(size_t)0 >> 1;
    int32_t window = 0;
    float scale = 1.f;
};
kda_status_t append(const kda_paged_problem_t &p, const Args &a) {
    return kda_paged_append(&p, a.k, a.v, a.rope ? a.q : nullptr, a.rope, a.table, a.lens, a.cu, a.cu_host, a.kp, a.vp, a.q_out,
                            nullptr);
}
kda_status_t attn(const kda_paged_problem_t &p, const Args &a) {
    return kda_paged_attn(&p, a.q, a.kp, a.vp, a.table, a.lens, a.cu, a.cu_host, a.scale, a.window, a.out, a.lse, a.ws, a.room,
                          nullptr);
}
kda_paged_problem_t problem() {
    kda_paged_problem_t p;
    std::memset(&p, 0, sizeof p);
    p.batch = 2;
    p.seq_len = 100;
    p.num_heads_q = 4;
    p.num_heads_kv = 2;
    p.head_dim_k = 128;
    p.head_dim_v = 64;
    p.io_dtype = KDA_BF16;
    p.page_size = 16;
    p.max_pages = 100;
    p.num_pages = 300;
    return p;
}

void host_arrays() {
    kda_paged_problem_t p = problem();
    p.batch = 1;
    p.num_seqs = 3;
    Args a;
    a.cu = dev_of<int32_t>(20);
    for (const auto &bad : {std::vector<int32_t>{0, 10, 20, 99}, {0, 30, 20, 100}, {1, 10, 20, 100}, {0, 10, 20, INT32_MIN}}) {
        std::unique_ptr<int32_t[]> cu(new int32_t[bad.size()]);
        std::memcpy(cu.get(), bad.data(), bad.size() * 4);
        a.cu_host = cu.get();
        EXPECT(append(p, a) == KDA_ERR_INVALID_ARGUMENT && attn(p, a) == KDA_ERR_INVALID_ARGUMENT);
    }
    // exact offsets: fewer workgroups than the query's, so its answer is enough; refused for the alignment of q or k
    const int32_t good[] = {0, 1, 1, 100};
    a.cu_host = good;
    a.q = dev(0, 8);
    EXPECT(attn(p, a) == KDA_ERR_INVALID_ARGUMENT && std::strstr(kda_last_error(), "aligned"));
    size_t need = 0;
    p.max_pages = 1 << 20;
    EXPECT(kda_paged_attn_workspace(&p, &need) == KDA_OK && need > 0);
    a = Args();
    a.cu = dev_of<int32_t>(20);
    a.cu_host = good;
    a.ws = nullptr;
    EXPECT(attn(p, a) == KDA_ERR_WORKSPACE);
}

void empty() {
    for (int i = 0; i < 2; ++i) {
        kda_paged_problem_t p = problem();
        (i ? p.batch : p.seq_len) = 0;
        Args a;
        a.q = a.k = a.v = a.out = a.ws = nullptr;
        a.room = 0;
        EXPECT(append(p, a) == KDA_OK && attn(p, a) == KDA_OK);
    }
}

void frequencies() {
    const int32_t dims[] = {INT32_MIN, -16, 0, 8, 16, 48, 128, INT32_MAX}, kinds[] = {-1, 0, 1, 2, 3, 4};
    const double values[] = {-1.0, 0.0, 1.0, 1.5, 32.0, 1e4, 1e308, INFINITY, NAN};
    for (int i = 0; i < 20000; ++i) {
        const int32_t d = pick(dims);
        std::unique_ptr<float[]> f(new float[d > 0 && d <= 128 ? d / 2 : 0]);
        float a = 0;
        const kda_status_t st = kda_rope_frequencies(d, pick(values), pick(kinds), pick(values), (int64_t)next_u64() >> (next_u64() % 64),
                                                     pick(values), pick(values), f.get(), &a);
        EXPECT(st == KDA_OK || st == KDA_ERR_INVALID_ARGUMENT);
        if (st == KDA_OK && d > 0) EXPECT(f[0] >= 0.f && f[0] <= 1.f);
    }
}

void quotients() {
    for (int i = 0; i < 2000000; ++i) {
        const uint32_t d = i < 70000 ? i + 1 : (uint32_t)(next_u64() >> (44 + next_u64() % 20)) % (1u << 20) + 1;
        const kda::paged::Div by(d);
        const int32_t n = (int32_t)(next_u64() >> 33), m = (int32_t)(n / d * d);
        EXPECT(by.by(n) == (int)(n / d) && by.by(m) == (int)(m / d) && (m == 0 || by.by(m - 1) == (int)((m - 1) / d)));
        EXPECT(by.by(INT32_MAX) == (int)(INT32_MAX / d) && by.by(0) == 0);
    }
}

void fuzz(int n) {
    const int32_t sizes[] = {INT32_MIN, -1, 0, 1, 2, 3, 15, 64, 65, 1000, 4096, 65535, 1 << 20, INT32_MAX - 1, INT32_MAX};
    const int32_t heads[] = {0, 1, 2, 4, 8, 32, 96, 1 << 20, INT32_MAX}, dims[] = {64, 64, 128, 128, 64, 128, 96, 0, -64, INT32_MAX};
    const int32_t types[] = {0, 1, 0, 1, 0, 1, 2, -1}, pages[] = {16, 64, 16, 256, 1 << 20, 1 << 30, 8, 0, -16, 48, INT32_MIN};
    const int64_t strides[] = {0, 0, 0, 0, 0, 0, 8, 64, 256, 1 << 14, INT64_MAX, INT64_MIN, (int64_t)1 << 59, (int64_t)1 << 57};
    const int64_t pools[] = {0, 1, 1000, -1, INT32_MAX, (int64_t)INT32_MAX + 1, INT64_MAX};
    const float scales[] = {1.f, 0.f, -3.f, std::numeric_limits<float>::max(), INFINITY, NAN};
    const kda_rope_t turn = {64, 0, 1.f, dev_of<float>(30), nullptr};
    int accepted = 0;
    for (int i = 0; i < n; ++i) {
        kda_paged_problem_t p;
        p.batch = pick(sizes);
        p.seq_len = pick(sizes);
        p.num_seqs = pick(sizes);
        p.num_heads_kv = pick(heads);
        p.num_heads_q = next_u64() & 1 ? p.num_heads_kv : pick(heads);
        p.head_dim_k = pick(dims);
        p.head_dim_v = pick(dims);
        p.io_dtype = pick(types);
        p.page_size = pick(pages);
        p.max_pages = pick(sizes);
        p.num_pages = pick(pools);
        p.stride_table = pick(strides);
        p.stride_q = pick(strides);
        p.stride_k = pick(strides);
        p.stride_v = pick(strides);
        const bool strided = next_u64() & 1;
        for (int64_t *x : {&p.k_page_stride, &p.k_head_stride, &p.k_cell_stride, &p.v_page_stride, &p.v_head_stride, &p.v_cell_stride})
            *x = strided ? pick(strides) : 0;
        if (i & 1) {  // every other one is a sound problem but for a few fields, so that more than the first checks are reached
            const kda_paged_problem_t odd = p;
            p = problem();
            for (int j = 0; j < 3; ++j) switch (next_u64() % 10) {
                    case 0: p.batch = odd.batch; break;
                    case 1: p.seq_len = odd.seq_len; break;
                    case 2: p.num_seqs = odd.num_seqs; break;
                    case 3: p.num_heads_q = odd.num_heads_q; break;
                    case 4: p.head_dim_k = odd.head_dim_k; break;
                    case 5: p.page_size = odd.page_size; break;
                    case 6: p.max_pages = odd.max_pages; break;
                    case 7: p.num_pages = odd.num_pages; break;
                    case 8: p.stride_q = odd.stride_q; break;
                    default: p.k_page_stride = odd.k_page_stride, p.k_head_stride = odd.k_head_stride, p.k_cell_stride = odd.k_cell_stride;
                }
        }
        size_t need = 1;
        const kda_status_t st = kda_paged_attn_workspace(&p, &need);
        EXPECT(st == KDA_OK || need == 0);
        EXPECT(need < (size_t)1 << 40);
        accepted += st == KDA_OK;
        Args a;  // q and v are not aligned: every call is refused, wherever it gets to before
        a.q = dev(0, 8);
        a.v = dev(2, 8);
        a.window = pick(sizes);
        a.scale = pick(scales);
        if (next_u64() & 1) a.cu = dev_of<int32_t>(20);
        if (next_u64() & 1) a.rope = &turn;
        if (next_u64() & 1) a.lse = nullptr;
        const int queries = g_device_queries;
        EXPECT(append(p, a) != KDA_OK && attn(p, a) != KDA_OK);
        EXPECT(g_device_queries == queries);
        kda_rope_problem_t r;
        r.batch = p.batch;
        r.seq_len = p.seq_len;
        r.num_heads_q = p.num_heads_q;
        r.num_heads_k = pick(heads);
        r.head_dim = p.head_dim_k;
        r.io_dtype = p.io_dtype;
        r.rot_dim = pick(dims);
        r.interleaved = pick(types);
        r.inverse = pick(types);
        r.amplitude = a.scale;
        r.stride_q = p.stride_q;
        r.stride_k = p.stride_k;
        r.stride_q_out = p.stride_v;
        r.stride_k_out = pick(strides);
        EXPECT(kda_rope(&r, dev(0, 8), dev(1), nullptr, dev_of<float>(2), dev(3), dev(4), nullptr) != KDA_OK);
        EXPECT(std::strlen(kda_last_error()) > 0);
    }
    EXPECT(n < 1000 || accepted > n / 1000);  // the queries' arithmetic is reached
    std::printf("%d of %d problems accepted by the queries\n", accepted, n);
}

}  // namespace

int main(int argc, char **argv) {
    host_arrays();
    empty();
    frequencies();
    quotients();
    fuzz(argc > 1 ? std::atoi(argv[1]) : 1000);
    std::printf("%d checks, %d failed\n", g_checks, g_failures);
    return g_failures != 0;
}
