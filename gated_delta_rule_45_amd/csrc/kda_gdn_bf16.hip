// Scalar-gate delta rule scans for bf16 io.
#include "kda_gdn_launch.h"

namespace kda {
namespace gdn {
hipError_t launch_scan_bf16(int mode, const GdnParams &p, hipStream_t stream) {
    return launch_scan<true>(mode, p, stream);
}
}  // namespace gdn
}  // namespace kda
