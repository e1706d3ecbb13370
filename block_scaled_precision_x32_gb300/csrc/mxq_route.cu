// mxq_route.cu -- the router on fp32 logits, and the choice between the types.
#include "mxq_route.cuh"

namespace mxq {

cudaError_t launch_route_bf16(bool grad, const RouteArgs& a, cudaStream_t s);  // mxq_route_bf16.cu

cudaError_t launch_route(Elt elt, bool grad, const RouteArgs& a, cudaStream_t s) {
    return elt == Elt::BF16 ? launch_route_bf16(grad, a, s) : route_launch<Elt::FP32>(grad, a, s);
}

}  // namespace mxq
