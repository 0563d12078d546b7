// Scalar-gate delta rule gradients for fp32 io.
#include "kda_gdn_grad.h"

namespace kda {
namespace gdn {
hipError_t launch_grad_f32(const GradParams &p, hipStream_t stream) { return launch_grad<false>(p, stream); }
}  // namespace gdn
}  // namespace kda
