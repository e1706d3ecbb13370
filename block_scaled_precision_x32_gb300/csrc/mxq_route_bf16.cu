// mxq_route_bf16.cu -- the router on bf16 logits.
#include "mxq_route.cuh"

namespace mxq {

cudaError_t launch_route_bf16(bool grad, const RouteArgs& a, cudaStream_t s) { return route_launch<Elt::BF16>(grad, a, s); }

}  // namespace mxq
