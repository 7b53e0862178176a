// moe_route_tokens with softmax scores: the kernels of router_forward.cuh.
#include "router_forward.cuh"

namespace bsmoe {

cudaError_t launch_route_softmax(int dtype, const RouteArgs& a, int num_sms, cudaStream_t st) {
  return launch_route_kind<false>(dtype, a, num_sms, st);
}

}  // namespace bsmoe
