// Routing kernels for bfloat16 logits (nest_route.cuh), a translation unit of its own so that
// the types compile in parallel.
#include "nest_route.cuh"

namespace nest {

int launch_route_bf16(const RouteArgs &a, int blocks, int threads, void *stream) {
    return launch_route_type<__nv_bfloat16>(a, blocks, threads, stream);
}

int launch_route_backward_bf16(const RouteArgs &a, void *stream) {
    return launch_route_backward_type<__nv_bfloat16>(a, stream);
}

}  // namespace nest
