// Routing kernels for f32 logits.
#include "route.cuh"

namespace arn {

RouteKernel route_kernel_f32(int v, RouteBy by) { return route_kernel<float>(v, by); }

}  // namespace arn
