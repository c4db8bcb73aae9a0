// The output head's products in IEEE half precision.
#include "nest_head.cuh"

namespace nest {
namespace head {
int launch_gemm_f16(Product p, const Maps &maps, const GemmArgs &args, int pairs, void *stream) {
    return launch_gemm<__half>(p, maps, args, pairs, stream);
}
}  // namespace head
}  // namespace nest
