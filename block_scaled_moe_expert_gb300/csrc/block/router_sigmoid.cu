// moe_route_tokens with sigmoid scores: the kernels of router_forward.cuh.
#include "router_forward.cuh"

namespace bsmoe {

cudaError_t launch_route_sigmoid(int dtype, const RouteArgs& a, int num_sms, cudaStream_t st) {
  return launch_route_kind<true>(dtype, a, num_sms, st);
}

}  // namespace bsmoe
