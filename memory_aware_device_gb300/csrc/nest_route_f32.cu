// Routing kernels for 32-bit logits (nest_route.cuh), a translation unit of its own so that
// the types compile in parallel.
#include "nest_route.cuh"

namespace nest {

int launch_route_f32(const RouteArgs &a, int blocks, int threads, void *stream) {
    return launch_route_type<float>(a, blocks, threads, stream);
}

int launch_route_backward_f32(const RouteArgs &a, void *stream) {
    return launch_route_backward_type<float>(a, stream);
}

}  // namespace nest
