// Scalar-gate delta rule scans for fp32 io.
#include "kda_gdn_launch.h"

namespace kda {
namespace gdn {
hipError_t launch_scan_f32(int mode, const GdnParams &p, hipStream_t stream) {
    return launch_scan<false>(mode, p, stream);
}
}  // namespace gdn
}  // namespace kda
