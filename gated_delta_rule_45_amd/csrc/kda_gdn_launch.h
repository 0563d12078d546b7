// Launches of the scan kernel for one io type (included by the two kernel files).
#pragma once

#include "kda_gdn_scan.h"

namespace kda {
namespace gdn {

template <bool BF, int DK, int CT, int MODE>
hipError_t launch_one(const GdnParams &p, hipStream_t stream) {
    const int64_t blocks = (int64_t)p.num_seqs * p.Hv * ((p.dv + (p.sm ? p.dk : 0)) / CT);
    if (blocks <= 0) return hipSuccess;
    hipLaunchKernelGGL((gdn_scan_kernel<BF, DK, CT, MODE>), dim3((unsigned)blocks),
                       dim3((Lds<BF, DK, CT, MODE>::NT)), 0, stream, p);
    return hipGetLastError();
}

template <bool BF>
hipError_t launch_scan(int mode, const GdnParams &p, hipStream_t stream) {
#define GDN_CASE(DK_, CT_, M_) \
    if (p.dk == DK_ && mode == M_) return launch_one<BF, DK_, CT_, M_>(p, stream);
#define GDN_MODES(DK_, CT_) GDN_CASE(DK_, CT_, kFwd) GDN_CASE(DK_, CT_, kKeep) GDN_CASE(DK_, CT_, kRev)
    GDN_MODES(64, 32)
    GDN_MODES(128, 32)
#undef GDN_MODES
#undef GDN_CASE
    return hipErrorInvalidConfiguration;
}

}  // namespace gdn
}  // namespace kda
