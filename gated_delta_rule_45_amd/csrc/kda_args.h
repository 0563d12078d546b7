// Argument checks that the host files share: pointers, alignment, overlaps, element types.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda.h"
#include "kda_internal.h"

namespace kda {
namespace args {

inline bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline bool dtype_ok(int32_t t) { return t == KDA_F32 || t == KDA_BF16; }
inline int64_t bytes_of(int32_t t) { return t == KDA_BF16 ? 2 : 4; }

inline kda_status_t done(hipError_t e, const char *what) {
    if (e != hipSuccess) return set_error(KDA_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
    set_error(KDA_OK, "%s", "");
    return KDA_OK;
}

// One tensor argument of a call.
struct Arg {
    const char *name;
    const void *p;
    int64_t bytes;
    size_t align;
    bool needed, written;
};

// Pointers: given, aligned, and no written range meets another one (`twin`: the pair of arguments
// that may be the same buffer).
template <int N>
kda_status_t check_args(const Arg (&a)[N], int twin0 = -1, int twin1 = -1) {
    for (const Arg &x : a) {
        if (!x.p && x.needed && x.bytes > 0) return set_error(KDA_ERR_INVALID_ARGUMENT, "%s is NULL", x.name);
        if (x.p && !aligned(x.p, x.align))
            return set_error(KDA_ERR_INVALID_ARGUMENT, "%s is not %zu-byte aligned", x.name, x.align);
    }
    for (int i = 0; i < N; ++i) {
        if (!a[i].written || !a[i].p || a[i].bytes <= 0) continue;
        const uintptr_t b = reinterpret_cast<uintptr_t>(a[i].p), e = b + (uintptr_t)a[i].bytes;
        for (int j = 0; j < N; ++j) {
            if (j == i || !a[j].p || a[j].bytes <= 0) continue;
            const uintptr_t c = reinterpret_cast<uintptr_t>(a[j].p), f = c + (uintptr_t)a[j].bytes;
            if (b == c && ((i == twin0 && j == twin1) || (i == twin1 && j == twin0))) continue;
            if (b < f && c < e) return set_error(KDA_ERR_INVALID_ARGUMENT, "%s aliases %s", a[i].name, a[j].name);
        }
    }
    return KDA_OK;
}

// Offsets of a packed batch of seq_len tokens, as far as the host sees them.
inline kda_status_t check_offsets(int32_t seq_len, int32_t num_seqs, const int32_t *cu, const int32_t *host) {
    if (!cu) {
        if (host) return set_error(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens_host given without cu_seqlens");
        return KDA_OK;
    }
    if (!aligned(cu, 4)) return set_error(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens is not 4-byte aligned");
    if (!host) return KDA_OK;
    if (host[0] != 0) return set_error(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens[0] = %d, expected 0", host[0]);
    for (int32_t i = 0; i < num_seqs; ++i)
        if (host[i + 1] < host[i])
            return set_error(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens decreases at %d (%d -> %d)", i, host[i], host[i + 1]);
    if (host[num_seqs] != seq_len)
        return set_error(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens[%d] = %d, expected seq_len %d", num_seqs,
                         host[num_seqs], seq_len);
    return KDA_OK;
}

// Work-items of a launch (HIP's limit).
constexpr int64_t kMostItems = 0xffffffffLL;

inline int current_cus() {
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
        return 256;
    return n;
}

}  // namespace args
}  // namespace kda
