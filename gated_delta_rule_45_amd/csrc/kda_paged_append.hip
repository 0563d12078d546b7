// New tokens' keys and values into the pages of their sequences, keys (and queries) turned by their positions on the
// way: one pass over the projections, where a rotation of its own would write and read q and k once more.
//
// Bound: HBM, each value is read and written once; for a few tokens the latency of a chain of loads (offsets,
// length, page) and of one launch.  Threads own 16 channels as in the rotary kernel; a token's items are first
// its keys and queries, HP heads each where there are many, then its values.
//
// bf16, 132,046 tokens in 64 prompts, 32 query and 8 key heads of 128, half of the channels turned: 610 us (5.3 TB/s; a copy
// reaches 4.9); one token of one sequence 3.5 us in the kernel, 12 with the host's side of the call.
#include "kda_paged.h"
#include "kda_rope.h"

namespace kda {
namespace paged {
namespace {

constexpr int kHeads = 4, kSeqs = 1024;  // offsets searched in LDS up to so many

struct Items {
    unsigned turned_groups, value_groups, turned, all;  // groups of HP heads, items of a token
    __host__ __device__ Items(int Hq, int Hk, int dk, int dv, int hp) {
        turned_groups = (Hq + Hk + hp - 1) / hp;
        value_groups = (Hk + hp - 1) / hp;
        turned = turned_groups * (dk / 16);
        all = turned + value_groups * (dv / 16);
    }
};
int heads_per_thread(int64_t tokens, int32_t Hq, int32_t Hk, int32_t dk, int32_t dv) {
    return tokens * Items(Hq, Hk, dk, dv, kHeads).all >= 256 * 2048 ? kHeads : 1;
}

// Sequence of token t: the last n with cu[n] <= t, found in cu or its copy in LDS.
template <typename P>
__device__ __forceinline__ int find(P cu, int n, int64_t t) {
    int a = 0, b = n;  // cu[a] <= t (as far as anyone knows), cu[b] > t
    while (b - a > 1) {
        const int m = (a + b) / 2;
        if (cu[m] <= t)
            a = m;
        else
            b = m;
    }
    return a;
}

template <typename IO, int HP>
__global__ void __launch_bounds__(256) append_kernel(AppendParams p) {
    __shared__ int32_t cu[kSeqs + 1];
    const Items items(p.q ? p.Hq : 0, p.Hk, p.dk, p.dv, HP);
    const Cache &c = p.c;
    const bool local = c.cu && c.num_seqs <= kSeqs;
    if (local) {
        for (int i = threadIdx.x; i <= c.num_seqs; i += 256) cu[i] = c.cu[i];
        __syncthreads();
    }
    const unsigned idx = blockIdx.x * 256u + threadIdx.x;
    const int64_t t = idx / items.all;
    const unsigned at = idx % items.all;
    if (t >= p.tokens) return;
    int n;
    int64_t from, to;
    if (c.cu) {
        n = local ? find(cu, c.num_seqs, t) : find(c.cu, c.num_seqs, t);
        from = local ? cu[n] : c.cu[n];
        to = local ? cu[n + 1] : c.cu[n + 1];
        to = to < p.tokens ? to : p.tokens;
        if (from < 0) from = 0;
        if (t < from || t >= to) return;  // no sequence's
    } else {
        n = (int)(t / c.T);
        from = (int64_t)n * c.T;
        to = from + c.T;
    }
    const int64_t cell = (int64_t)c.lens[n] - (to - t);
    if (cell < 0) return;  // padding
    const int64_t slot = cell >> c.page_shift;
    int64_t page = slot < c.max_pages ? c.table[n * c.table_ld + slot] : -1;
    if (page >= c.num_pages) page = -1;
    const int64_t in_page = cell & ((1 << c.page_shift) - 1);
    if (at < items.turned) {
        const int U = p.dk / 16, u = at % U;
        const unsigned hg = at / U, heads = p.Hk + (p.q ? p.Hq : 0);
        const bool turned = 16 * u < p.rot;
        Turn turn;
        if (turned) turn.set(p.positions ? p.positions[t] : (int)cell, p.freq, u, p.amplitude, 1.f);
        const int a0 = run0(u, p.rot, p.interleaved), b0 = run1(u, p.rot, p.interleaved);
        Eight<IO> a[HP], b[HP];
#pragma unroll
        for (int i = 0; i < HP; ++i) {
            const unsigned h = hg + i * items.turned_groups;
            if (h >= heads) continue;
            const IO *x = h < (unsigned)p.Hk ? static_cast<const IO *>(p.k) + t * p.ldk + (int64_t)h * p.dk
                                             : static_cast<const IO *>(p.q) + t * p.ldq + (int64_t)(h - p.Hk) * p.dk;
            a[i].load(x + a0);
            b[i].load(x + b0);
        }
#pragma unroll
        for (int i = 0; i < HP; ++i) {
            const unsigned h = hg + i * items.turned_groups;
            if (h >= heads || (h < (unsigned)p.Hk && page < 0)) continue;
            if (turned) turn.apply(a[i], b[i], p.interleaved);
            IO *y = h < (unsigned)p.Hk ? static_cast<IO *>(c.k) + page * c.k_page + h * c.k_head + in_page * c.k_cell
                                       : static_cast<IO *>(p.q_out) + t * p.ldqo + (int64_t)(h - p.Hk) * p.dk;
            a[i].store(y + a0);
            b[i].store(y + b0);
        }
    } else if (page >= 0) {
        const int U = p.dv / 16, u = (at - items.turned) % U;
        const unsigned hg = (at - items.turned) / U;
        Eight<IO> a[HP], b[HP];
#pragma unroll
        for (int i = 0; i < HP; ++i) {
            const unsigned h = hg + i * items.value_groups;
            if (h >= (unsigned)p.Hk) continue;
            const IO *x = static_cast<const IO *>(p.v) + t * p.ldv + (int64_t)h * p.dv + 16 * u;
            a[i].load(x);
            b[i].load(x + 8);
        }
#pragma unroll
        for (int i = 0; i < HP; ++i) {
            const unsigned h = hg + i * items.value_groups;
            if (h >= (unsigned)p.Hk) continue;
            IO *y = static_cast<IO *>(c.v) + page * c.v_page + h * c.v_head + in_page * c.v_cell + 16 * u;
            a[i].store(y);
            b[i].store(y + 8);
        }
    }
}

template <typename IO>
hipError_t launch(const AppendParams &p, hipStream_t stream) {
    const int Hq = p.q ? p.Hq : 0, hp = heads_per_thread(p.tokens, Hq, p.Hk, p.dk, p.dv);
    const int64_t n = p.tokens * Items(Hq, p.Hk, p.dk, p.dv, hp).all;
    if (n <= 0) return hipSuccess;
    const dim3 grid((unsigned)((n + 255) / 256));
    if (hp == kHeads)
        hipLaunchKernelGGL((append_kernel<IO, kHeads>), grid, dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((append_kernel<IO, 1>), grid, dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace

int64_t append_items(int64_t tokens, int32_t Hq, int32_t Hk, int32_t dk, int32_t dv) {
    return tokens * Items(Hq, Hk, dk, dv, heads_per_thread(tokens, Hq, Hk, dk, dv)).all;
}

hipError_t launch_append(bool bf16, const AppendParams &p, hipStream_t stream) {
    return bf16 ? launch<uint16_t>(p, stream) : launch<float>(p, stream);
}

}  // namespace paged
}  // namespace kda
