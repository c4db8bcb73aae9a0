// The output head's products in bfloat16.
#include "nest_head.cuh"

namespace nest {
namespace head {
int launch_gemm_bf16(Product p, const Maps &maps, const GemmArgs &args, int pairs, void *stream) {
    return launch_gemm<__nv_bfloat16>(p, maps, args, pairs, stream);
}
int gave_up_bf16(int64_t *count, void *stream) { return read_gave_up<__nv_bfloat16>(count, stream); }
}  // namespace head
}  // namespace nest
