// The output head's products in bfloat16.
#include "nest_head.cuh"

namespace nest {
namespace head {
int launch_gemm_bf16(Product p, const Maps &maps, const GemmArgs &args, int pairs, void *stream) {
    return launch_gemm<__nv_bfloat16>(p, maps, args, pairs, stream);
}
}  // namespace head
}  // namespace nest
