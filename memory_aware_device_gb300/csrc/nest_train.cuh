// Shared by the training-step operators (nest_route.cu, nest_optim.cu) and the output head's losses (nest_head.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "../../include/nest_train.h"
#include "nest_internal.cuh"

namespace nest {

constexpr int kSMs = 152;   // of a GB300; grids of at most a few blocks for each

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

inline size_t type_bytes(int32_t t) { return t == NEST_F32 ? 4 : 2; }
inline bool valid_type(int32_t t) { return t == NEST_F32 || t == NEST_BF16 || t == NEST_F16; }
inline bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// fn(T{}) with T the element type t (valid_type holds).
template <typename F>
int with_type(int32_t t, F fn) {
    if (t == NEST_F32) return fn(float{});
    if (t == NEST_BF16) return fn(__nv_bfloat16{});
    return fn(__half{});
}

// Lets KERNEL have up to `bytes` of dynamic shared memory on the current device: asked for once per
// device, as the question costs as much as a launch.
template <auto KERNEL>
int allow(size_t bytes, const char *what) {
    static std::atomic<uint64_t> done{0};
    int device = 0;
    if (const int rc = cuda_status(cudaGetDevice(&device), what)) return rc;
    const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;
    if (done.load(std::memory_order_relaxed) & bit) return NEST_OK;
    const int rc =
        cuda_status(cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes)), what);
    if (!rc) done.fetch_or(bit, std::memory_order_relaxed);
    return rc;
}

// Copies from global to shared memory that the thread waits for later.
template <int BYTES>
__device__ __forceinline__ void copy_ahead(void *to, const void *from) {
    const uint32_t dst = uint32_t(__cvta_generic_to_shared(to));
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(from), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_mark() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LATER>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LATER) : "memory"); }

// Takes a ticket, which is 0 again after `blocks` of them; whether it was the last.  By one thread
// between two barriers of its block: what the block wrote before is seen by the block that
// takes a later ticket.
__device__ __forceinline__ bool last_ticket(uint32_t *ticket, uint32_t blocks) {
    uint32_t before;
    asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;"
                 : "=r"(before)
                 : "l"(ticket), "r"(blocks - 1)
                 : "memory");
    return before == blocks - 1;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace nest
