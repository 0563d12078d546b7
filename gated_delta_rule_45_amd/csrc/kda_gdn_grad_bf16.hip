// Scalar-gate delta rule gradients for bf16 io.
#include "kda_gdn_grad.h"

namespace kda {
namespace gdn {
hipError_t launch_grad_bf16(const GradParams &p, hipStream_t stream) { return launch_grad<true>(p, stream); }
}  // namespace gdn
}  // namespace kda
