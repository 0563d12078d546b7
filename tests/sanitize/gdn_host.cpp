// Host-side checks of the scalar-gate delta rule's entry points and of the epilogue's gradients, built with
// AddressSanitizer and UndefinedBehaviorSanitizer around their host code.  Every call is refused by validation
// or describes an empty problem, so no kernel is reached; host arrays are allocated at their exact sizes.
//
// Exit status 0 when every expectation holds (and no sanitizer report aborted the run).
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <limits>
#include <memory>
#include <new>
#include <vector>

#include "kda.h"

// Takes the runtime's place: a refused call asks nothing of it.
static int g_device_queries = 0;
extern "C" int hipGetDevice(int *) {
    ++g_device_queries;
    return 1;
}

static bool g_no_memory = false;
void *operator new(size_t n) {
    void *p = g_no_memory ? nullptr : std::malloc(n);
    if (!p) throw std::bad_alloc();
    return p;
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, size_t) noexcept { std::free(p); }

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

kda_gdn_problem_t problem() {
    kda_gdn_problem_t p;
    std::memset(&p, 0, sizeof p);
    p.batch = 2;
    p.seq_len = 100;
    p.num_heads_k = 2;
    p.num_heads_v = 4;
    p.head_dim_k = 128;
    p.head_dim_v = 64;
    p.io_dtype = KDA_BF16;
    p.scale = 1.f;
    return p;
}

std::unique_ptr<int32_t[]> host(const std::vector<int32_t> &v) {
    std::unique_ptr<int32_t[]> a(new int32_t[v.size()]);
    for (size_t i = 0; i < v.size(); ++i) a[i] = v[i];
    return a;
}

// Device arguments of the calls, to be bent one at a time.
struct Args {
    void *q = dev(0), *k = dev(1), *v = dev(2), *g = dev(3), *beta = dev(4), *s0 = nullptr, *out = dev(5), *sf = nullptr,
         *d_out = dev(6), *dsf = nullptr, *dq = dev(7), *dk = dev(8), *dv = dev(9), *dg = dev(10), *db = dev(11),
         *ds0 = nullptr, *ws = dev(12), *state = dev(13);
    int32_t *slots = static_cast<int32_t *>(dev(14)), *cu = nullptr;
    const int32_t *cu_host = nullptr, *slots_host = nullptr;
    size_t room = ~(size_t)0 >> 1;
    int64_t num_slots = 1000;
};
kda_status_t fwd(const kda_gdn_problem_t &p, const Args &a) {
    return kda_gdn_chunk_fwd(&p, a.q, a.k, a.v, a.g, a.beta, a.s0, a.cu, a.cu_host, a.out, a.sf, nullptr, 0, nullptr);
}
kda_status_t bwd(const kda_gdn_problem_t &p, const Args &a) {
    return kda_gdn_chunk_bwd(&p, a.q, a.k, a.v, a.g, a.beta, a.s0, a.cu, a.cu_host, a.d_out, a.dsf, a.dq, a.dk, a.dv, a.dg,
                             a.db, a.ds0, a.ws, a.room, nullptr);
}
kda_status_t decode(const kda_gdn_problem_t &p, const Args &a) {
    return kda_gdn_decode(&p, a.q, a.k, a.v, a.g, a.beta, a.state, a.num_slots, a.slots, a.slots_host, a.cu, a.cu_host,
                          a.out, nullptr);
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

void refusals() {
    const kda_gdn_problem_t p = problem();
    Args a;
    a.q = dev(0, 8);
    EXPECT(fwd(p, a) == KDA_ERR_INVALID_ARGUMENT && bwd(p, a) == KDA_ERR_INVALID_ARGUMENT &&
           decode(p, a) == KDA_ERR_INVALID_ARGUMENT);
    a = Args();
    a.ws = nullptr;
    EXPECT(bwd(p, a) == KDA_ERR_WORKSPACE);
    a = Args();
    a.dq = a.dk;
    EXPECT(bwd(p, a) == KDA_ERR_INVALID_ARGUMENT);
    a = Args();
    a.ws = dev(12, 16);
    EXPECT(bwd(p, a) == KDA_ERR_INVALID_ARGUMENT);
    EXPECT(kda_gdn_chunk_fwd_workspace(nullptr, &a.room) == KDA_ERR_INVALID_ARGUMENT && a.room == 0);
    EXPECT(kda_gdn_chunk_bwd_workspace(&p, nullptr) == KDA_ERR_INVALID_ARGUMENT);
}

void host_arrays() {
    kda_gdn_problem_t p = problem();
    p.batch = 1;
    p.num_seqs = 3;
    Args a;
    a.cu = static_cast<int32_t *>(dev(20));
    for (const auto &bad : {std::vector<int32_t>{0, 10, 20, 99}, {0, 30, 20, 100}, {1, 10, 20, 100}, {0, 10, 20, INT32_MIN}}) {
        const auto cu = host(bad);
        a.cu_host = cu.get();
        EXPECT(fwd(p, a) == KDA_ERR_INVALID_ARGUMENT && bwd(p, a) == KDA_ERR_INVALID_ARGUMENT &&
               decode(p, a) == KDA_ERR_INVALID_ARGUMENT);
    }
    p = problem();
    p.batch = 3;
    a = Args();
    for (const auto &bad : {std::vector<int32_t>{5, 7, 5}, {1000, 0, 1}, {INT32_MAX, -1, 2}, {0, 0, -1}}) {
        const auto at = host(bad);
        a.slots_host = at.get();
        EXPECT(decode(p, a) == KDA_ERR_INVALID_ARGUMENT);
    }
}

void out_of_memory() {
    kda_gdn_problem_t p = problem();
    Args a;
    const auto at = host({5, 7});
    a.slots_host = at.get();
    a.q = dev(0, 8);
    EXPECT(decode(p, a) == KDA_ERR_INVALID_ARGUMENT && std::strstr(kda_last_error(), "aligned"));
    a.q = dev(0);
    g_no_memory = true;  // for the list of the slots: what is thrown stays inside, and the message is this call's
    const kda_status_t st = decode(p, a);
    g_no_memory = false;
    EXPECT(st == KDA_ERR_HIP && !std::strstr(kda_last_error(), "aligned") && std::strlen(kda_last_error()) > 0);
}

void empty() {
    for (int i = 0; i < 2; ++i) {
        kda_gdn_problem_t p = problem();
        (i ? p.batch : p.seq_len) = 0;
        Args a;
        a.q = a.k = a.v = a.g = a.beta = a.out = a.d_out = a.dq = a.dk = a.dv = a.dg = a.db = a.ws = nullptr;
        a.room = 0;
        EXPECT(fwd(p, a) == KDA_OK && bwd(p, a) == KDA_OK && decode(p, a) == KDA_OK);
    }
}

void norm() {
    const int64_t rows[] = {-1, 0, 1, 7, 1 << 20, (int64_t)1 << 48, INT64_MAX};
    const int32_t dims[] = {-1, 0, 64, 96, 128, INT32_MAX}, types[] = {-1, 0, 1, 2};
    for (int64_t r : rows)
        for (int32_t d : dims)
            for (int32_t t : types) {
                const size_t need = kda_norm_gate_bwd_workspace(r, d, t);
                const bool good = r >= 0 && (d == 64 || d == 128) && (t == 0 || t == 1);
                EXPECT(good || need == 0);
                EXPECT(kda_norm_gate_bwd(r, d, t, 1e-6f, dev(0, 4), dev(1), static_cast<float *>(dev(2)), dev(3), dev(4),
                                         dev(5), static_cast<float *>(dev(6)), dev(7), need, nullptr) != KDA_OK);
            }
}

void fuzz(int n) {
    const int32_t sizes[] = {INT32_MIN, -1, 0, 1, 2, 3, 15, 64, 65, 1000, 4096, 65535, 1 << 20, INT32_MAX - 1, INT32_MAX};
    const int32_t heads[] = {0, 1, 2, 4, 8, 32, 96, 1 << 20, INT32_MAX}, dims[] = {64, 64, 128, 128, 96, 0, -64, INT32_MAX};
    const int32_t types[] = {0, 1, 0, 1, 0, 1, 2, -1};
    const float scales[] = {1.f, 0.f, -3.f, std::numeric_limits<float>::max(), INFINITY, NAN};
    const int64_t strides[] = {0, 0, 0, 8, 256, 1 << 14, INT64_MAX, INT64_MIN, (int64_t)1 << 59};
    const int64_t slots[] = {0, 1, 1000, -1, INT32_MAX, (int64_t)INT32_MAX + 1, INT64_MAX};
    int accepted = 0;
    for (int i = 0; i < n; ++i) {
        kda_gdn_problem_t p;
        p.batch = pick(sizes);
        p.seq_len = pick(sizes);
        p.num_seqs = pick(sizes);
        p.num_heads_k = pick(heads);
        p.num_heads_v = next_u64() & 1 ? p.num_heads_k : pick(heads);
        p.head_dim_k = pick(dims);
        p.head_dim_v = pick(dims);
        p.io_dtype = pick(types);
        p.gate_dtype = pick(types);
        p.state_dtype = pick(types);
        p.scale = pick(scales);
        p.stride_q = pick(strides);
        p.stride_k = pick(strides);
        p.stride_v = pick(strides);
        size_t need = 1;
        const kda_status_t f = kda_gdn_chunk_fwd_workspace(&p, &need);
        EXPECT(f == KDA_OK || need == 0);
        need = 1;
        const kda_status_t b = kda_gdn_chunk_bwd_workspace(&p, &need);
        EXPECT(b == KDA_OK || need == 0);
        EXPECT(b != KDA_OK || need < (size_t)1 << 63);
        accepted += b == KDA_OK;
        Args a;  // q is not aligned: every call is refused, wherever it gets to before
        a.q = dev(0, 8);
        a.num_slots = pick(slots);
        if (next_u64() & 1) a.cu = static_cast<int32_t *>(dev(20));
        if (next_u64() & 1) a.s0 = dev(21);
        if (next_u64() & 1) a.ds0 = dev(22);
        if (next_u64() & 1) a.slots = nullptr;
        const int queries = g_device_queries;
        EXPECT(fwd(p, a) != KDA_OK && bwd(p, a) != KDA_OK && decode(p, a) != KDA_OK);
        EXPECT(g_device_queries == queries);
        EXPECT(std::strlen(kda_last_error()) > 0);
    }
    EXPECT(n == 0 || g_device_queries > 0);  // by the workspace queries
    EXPECT(n < 1000 || accepted > n / 1000);  // the queries' arithmetic is reached
    std::printf("%d of %d problems accepted by the queries\n", accepted, n);
}

}  // namespace

int main(int argc, char **argv) {
    refusals();
    host_arrays();
    out_of_memory();
    empty();
    norm();
    fuzz(argc > 1 ? std::atoi(argv[1]) : 1000);
    std::printf("%d checks, %d failed\n", g_checks, g_failures);
    return g_failures != 0;
}
