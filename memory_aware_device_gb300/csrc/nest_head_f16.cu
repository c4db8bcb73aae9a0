// The output head's products in IEEE half precision.
#include "nest_head.cuh"

namespace nest {
namespace head {
int launch_gemm_f16(Product p, const Maps &maps, const GemmArgs &args, int pairs, void *stream) {
    return launch_gemm<__half>(p, maps, args, pairs, stream);
}
int gave_up_f16(int64_t *count, void *stream) { return read_gave_up<__half>(count, stream); }
}  // namespace head
}  // namespace nest
