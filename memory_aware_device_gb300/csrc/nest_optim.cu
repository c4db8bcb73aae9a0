// The optimizer's operators over lists of tensors: gradient norm and AdamW step, with
// moments in 32 or in 8 bits (definitions in nest_train.h).
//
// The packed table holds the tensors' entries and a list of items (tensor, first block);
// an item is up to kItemBlocks blocks of 256 elements of one tensor and is the unit that
// a thread block takes; a warp takes whole blocks of 256.
#include <cmath>
#include <cstring>

#include "nest_train.cuh"

namespace nest {

namespace {

constexpr int kBlock = NEST_OPT_BLOCK;
constexpr int kItemBlocks = 16;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

struct Entry {            // one tensor
    void *weight;
    const void *grad;
    int64_t numel;
    int64_t first;        // its first block in the list's buffers
    float weight_decay, lr_scale;
    int64_t pad;
};
struct Item {
    int32_t tensor, block;   // block: within the tensor
};
static_assert(sizeof(Entry) == 48 && sizeof(Item) == 8, "table layout");

__device__ __forceinline__ const Item *items_of(const void *table, int tensors) {
    return reinterpret_cast<const Item *>(static_cast<const Entry *>(table) + tensors);
}

int64_t blocks_in(int64_t numel) { return (numel + kBlock - 1) / kBlock; }

// A lane's share of a block: elements 8 lane .. 8 lane + 7, in one load of 32 bytes (or 16).
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                 : "l"(p)
                 : "memory");
}
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&x)[8]) {
    static_assert(sizeof(T) == 2, "16-bit type");
    const uint4 q = *reinterpret_cast<const uint4 *>(p);
    const T *h = reinterpret_cast<const T *>(&q);
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = to_f32(h[i]);
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :
                 : "l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&x)[8]) {
    static_assert(sizeof(T) == 2, "16-bit type");
    uint4 q;
    T *h = reinterpret_cast<T *>(&q);
#pragma unroll
    for (int i = 0; i < 8; i++) h[i] = from_f32<T>(x[i]);
    *reinterpret_cast<uint4 *>(p) = q;
}

template <typename T>
__device__ __forceinline__ bool wide(const T *p) {   // every block of the tensor can be loaded by load8
    return (reinterpret_cast<uintptr_t>(p) & (8 * sizeof(T) - 1)) == 0;
}

// The lane's share of the block that starts at p[0], of which `n` elements (1 to 256) exist; the
// others are 0.  A tensor that does not start at a multiple of 8 elements, and a tensor's last
// block, go through the warp's shared memory: 32 neighbours at a time between it and the tensor.
template <typename T>
__device__ __forceinline__ void load_block(const T *p, int n, bool vector, int lane, float *room, float (&x)[8]) {
    if (vector && n >= kBlock) {
        load8(p + 8 * lane, x);
        return;
    }
    T part[8];
#pragma unroll
    for (int i = 0; i < 8; i++) part[i] = lane + 32 * i < n ? p[lane + 32 * i] : from_f32<T>(0.0f);
#pragma unroll
    for (int i = 0; i < 8; i++) room[lane + 32 * i] = to_f32(part[i]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = room[8 * lane + i];
    __syncwarp();
}
template <typename T>
__device__ __forceinline__ void store_block(T *p, int n, bool vector, int lane, float *room, const float (&x)[8]) {
    if (vector && n >= kBlock) {
        store8(p + 8 * lane, x);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; i++) room[8 * lane + i] = x[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; i++)
        if (lane + 32 * i < n) p[lane + 32 * i] = from_f32<T>(room[lane + 32 * i]);
    __syncwarp();
}

// ---- gradient norm ----------------------------------------------------------------

// A sum in 32 bits with the rounding error of every addition added up beside it (Knuth's
// exact sum of two numbers): 64-bit additions are 64 times slower here, and one for every
// item and thread took a quarter of the kernel's time.
struct Sum {
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float x) {
        const float s = hi + x, b = s - hi;
        lo += (hi - (s - b)) + (x - b);
        hi = s;
    }
    __device__ __forceinline__ float value() const { return isfinite(hi) ? hi + lo : hi; }
};

// The block's sum of its threads' values, in thread 0.
__device__ __forceinline__ float block_sum(float v, float *sh) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(threadIdx.x < kWarps ? sh[threadIdx.x] : 0.0f);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_kernel(const void *table, int tensors, int items, float *part) {
    __shared__ float sh[kWarps];
    __shared__ __align__(16) float room[kWarps][kBlock];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Entry *entries = static_cast<const Entry *>(table);
    const Item *list = items_of(table, tensors);
    Sum sum;
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        const Item item = list[it];
        const T *g = static_cast<const T *>(entries[item.tensor].grad);
        const int64_t numel = entries[item.tensor].numel;
        const bool vector = wide(g);
        float s = 0.0f;
#pragma unroll
        for (int b = 0; b < kItemBlocks; b += kWarps) {
            const int64_t at = int64_t(item.block + b + warp) * kBlock, left = numel - at;
            if (left <= 0) break;
            float x[8];
            load_block(g + at, int(left < kBlock ? left : kBlock), vector, lane, room[warp], x);
#pragma unroll
            for (int i = 0; i < 8; i++) s = fmaf(x[i], x[i], s);
        }
        sum.add(s);
    }
    const float s = block_sum(sum.value(), sh);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ void __launch_bounds__(kThreads) norm_finish_kernel(const float *part, int blocks, float max_norm,
                                                               float *out) {
    __shared__ float sh[kWarps];
    pdl_wait();
    pdl_trigger();
    Sum sum;
#pragma unroll 8
    for (int b = threadIdx.x; b < blocks; b += kThreads) sum.add(part[b]);
    const float s = block_sum(sum.value(), sh);
    if (threadIdx.x == 0) {
        const float norm = sqrtf(s);
        out[0] = norm;
        out[1] = isfinite(norm) ? fminf(1.0f, max_norm / (norm + 1e-6f)) : NAN;
    }
}

// ---- moments in 8 bits --------------------------------------------------------------

__host__ __device__ __forceinline__ uint32_t mixed(uint32_t x) {
    x ^= x >> 16;
    x *= 0x9E3779B1u;   // odd, close to 2^32 over the golden ratio
    x ^= x >> 15;
    x *= 0x6A09E667u;   // odd, the fraction of the square root of 2
    return x ^ (x >> 16);
}

__device__ __forceinline__ float power2(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// s of a block from its largest finite magnitude a (as bits): a < 1.75 * 2^s.
__device__ __forceinline__ int shared_exponent(uint32_t a) {
    const int s = int((a + (1u << 21)) >> 23) - 127;
    return max(-100, min(120, s));
}

__device__ __forceinline__ uint32_t finite_bits(float x) {
    const uint32_t a = __float_as_uint(x) & 0x7fffffffu;
    return a < 0x7f800000u ? a : 0u;
}

// Code of y >= 0 with 3 mantissa bits: 16 bits of noise r are added under the last bit
// kept and the rest is cut off.  Exponent field f of a normal code stands for the 32-bit
// exponent field OFFSET + f; under the smallest normal value the code counts steps of
// 1 / small, whose fraction is cut to 16 bits by adding 128 (one unit in the last place of a
// number there is 2^-16) and summed with the noise as an integer.
template <int OFFSET>
__device__ __forceinline__ uint32_t code_of(float y, uint32_t r, float small) {
    const uint32_t normal = (__float_as_uint(y) + (r << 4) - (uint32_t(OFFSET) << 23)) >> 20;
    const uint32_t fixed = (__float_as_uint(__fmaf_rz(y, small, 128.0f)) + r - 0x43000000u) >> 16;
    return __float_as_uint(y) < (uint32_t(OFFSET + 1) << 23) ? fixed : normal;
}

// Codes of a lane's eight pairs of moments; word: the block's noise.  rare: the block holds one
// that is not finite, or whose scale is clipped, and codes are checked against the largest.
template <bool RARE>
__device__ __forceinline__ void encode(const float (&m)[8], const float (&v)[8], int sm, int sv, uint32_t word,
                                       int lane, uint2 &cm, uint2 &cv) {
    const float fm = power2(8 - sm), fv = power2(-1 - sv);
    uint32_t pm[2] = {0, 0}, pv[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; i++) {
        uint32_t x = word + uint32_t(8 * lane + i) * 0x9E3779B1u;
        x ^= x >> 15;
        x *= 0x6A09E667u;
        x ^= x >> 16;
        uint32_t a = code_of<120>(fabsf(m[i]) * fm, x >> 16, 512.0f);
        uint32_t b = code_of<95>(v[i] * fv, x & 0xFFFFu, 0x1p34f);
        if (RARE) {
            a = isfinite(m[i]) ? min(a, 0x7Eu) : 0x7Fu;
            b = isfinite(v[i]) ? min(b, 0xFEu) : 0xFFu;
        }
        a |= (__float_as_uint(m[i]) >> 24) & 0x80u;
        pm[i / 4] |= a << (8 * (i % 4));
        pv[i / 4] |= b << (8 * (i % 4));
    }
    cm = make_uint2(pm[0], pm[1]);
    cv = make_uint2(pv[0], pv[1]);
}

// Two codes with 4 exponent bits as two floats: the hardware's e4m3 conversion (0x7F is NaN there too).
__device__ __forceinline__ float2 pair_of(uint16_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

__device__ __forceinline__ void decode_m(uint2 c, int s, float (&m)[8]) {
    const float f = power2(s - 8);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 y = pair_of(uint16_t((i < 2 ? c.x : c.y) >> (16 * (i & 1))));
        m[2 * i] = y.x * f;
        m[2 * i + 1] = y.y * f;
    }
}

// A code's bits as a 32-bit float are its value with the exponent 95 too small, subnormal codes included.
__device__ __forceinline__ void decode_v(uint2 c, int s, float (&v)[8]) {
    const float f = power2(s + 1);
#pragma unroll
    for (int i = 0; i < 8; i++)
        v[i] = __uint_as_float(((i < 4 ? c.x : c.y) >> (8 * (i & 3)) & 0xFFu) << 20) * 0x1p95f * f;
    if (__vcmpeq4(c.x, 0xFFFFFFFFu) | __vcmpeq4(c.y, 0xFFFFFFFFu)) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (((i < 4 ? c.x : c.y) >> (8 * (i & 3)) & 0xFFu) == 0xFFu) v[i] = NAN;
    }
}

// ---- AdamW --------------------------------------------------------------------------

struct StepArgs {
    const void *table;
    int tensors, items;
    float lr, beta1, beta2, rest1, rest2, eps;
    double beta1d, beta2d;
    uint32_t seed;
    float *master;
    void *m, *v;
    int8_t *m_exp, *v_exp;
    nest_adamw_state *state;
    const float *grad_scale;
};

__device__ __forceinline__ float root_of(float x) {   // relative error 2^-23
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The lane's share of a block of the list's own buffers; past the tensor's end nothing is written.
__device__ __forceinline__ void store_own(float *p, int n, int lane, const float (&x)[8]) {
    if (8 * lane + 8 <= n) {
        store8(p + 8 * lane, x);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; i++)
        if (8 * lane + i < n) p[8 * lane + i] = x[i];
}
__device__ __forceinline__ void store_own(uint8_t *p, int n, int lane, uint2 c) {
    if (8 * lane + 8 <= n) {
        *reinterpret_cast<uint2 *>(p + 8 * lane) = c;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; i++)
        if (8 * lane + i < n) p[8 * lane + i] = uint8_t((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
}

// Magnitudes (as bits) from which a block's codes take the checked path: 1.75 * 2^120, infinity, NaN.
constexpr uint32_t kRare = (uint32_t(120 + 127) << 23) | 0x600000u;

template <typename W, typename G, bool EIGHT>
__global__ void __launch_bounds__(kThreads, 4) adamw_kernel(StepArgs a) {
    constexpr bool kOwnMaster = sizeof(W) == 4;
    __shared__ __align__(16) float room[kWarps][kBlock];
    __shared__ struct {
        float scale, inv1, root2;
        uint32_t start;
    } shared;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Entry *entries = static_cast<const Entry *>(a.table);
    const Item *list = items_of(a.table, a.tensors);
    int it = blockIdx.x;
    Item item = {0, 0};
    if (it < a.items) item = list[it];
    if (threadIdx.x == 0) {   // what all share, by one thread: 64-bit arithmetic is slow
        const nest_adamw_state st = *a.state;
        shared.scale = a.grad_scale ? *a.grad_scale : 1.0f;
        shared.inv1 = 1.0f / float(1.0 - st.beta1_t * a.beta1d);
        shared.root2 = rsqrtf(float(1.0 - st.beta2_t * a.beta2d));
        shared.start = mixed(a.seed ^ mixed(uint32_t(st.step + 1)));
    }
    __syncthreads();
    const float scale = shared.scale, inv1 = shared.inv1, root2 = shared.root2;
    const uint32_t start = shared.start;
    if (!isfinite(scale)) return;
    // says that this block has read the step's state; the last block to say so advances it at
    // its end, when the answer has long arrived
    uint32_t before = 0;
    if (threadIdx.x == 0) {
        __threadfence();
        before = atomicAdd(&a.state->ticket, 1u);
    }
    while (it < a.items) {
        const Entry e = entries[item.tensor];
        it += gridDim.x;
        Item next = {0, 0};
        if (it < a.items) next = list[it];
        W *weight = static_cast<W *>(e.weight);
        const G *grad = static_cast<const G *>(e.grad);
        const bool wide_w = wide(weight), wide_g = wide(grad);
        const float lr = a.lr * e.lr_scale, decay = e.weight_decay;
        for (int b = item.block + warp; b < item.block + kItemBlocks; b += kWarps) {
            const int64_t j0 = int64_t(b) * kBlock, left = e.numel - j0;
            if (left <= 0) break;
            const int n = int(left < kBlock ? left : kBlock);
            const int64_t block = e.first + b, at = block * kBlock;
            float g[8], m[8], v[8], p[8];
            load_block(grad + j0, n, wide_g, lane, room[warp], g);
            if constexpr (kOwnMaster)
                load_block(weight + j0, n, wide_w, lane, room[warp], p);
            else
                load8(a.master + at + 8 * lane, p);   // the list's own buffers hold whole blocks
            if constexpr (EIGHT) {
                const uint2 cm = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.m) + at + 8 * lane);
                const uint2 cv = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.v) + at + 8 * lane);
                decode_m(cm, a.m_exp[block], m);
                decode_v(cv, a.v_exp[block], v);
            } else {
                load8(static_cast<const float *>(a.m) + at + 8 * lane, m);
                load8(static_cast<const float *>(a.v) + at + 8 * lane, v);
            }
            uint32_t top_m = 0, top_v = 0;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float x = g[i] * scale;
                // each product rounded by itself, so that a moment is the same number wherever
                // these formulas are evaluated, and its 8-bit code with it
                m[i] = __fadd_rn(__fmul_rn(m[i], a.beta1), __fmul_rn(x, a.rest1));
                v[i] = __fadd_rn(__fmul_rn(v[i], a.beta2), __fmul_rn(__fmul_rn(x, x), a.rest2));
                p[i] -= lr * (__fdividef(m[i] * inv1, fmaf(root_of(v[i]), root2, a.eps)) + decay * p[i]);
                if (EIGHT && 8 * lane + i < n) {
                    top_m = max(top_m, __float_as_uint(m[i]) & 0x7fffffffu);
                    top_v = max(top_v, __float_as_uint(v[i]) & 0x7fffffffu);
                }
            }
            store_block(weight + j0, n, wide_w, lane, room[warp], p);
            if constexpr (!kOwnMaster) store_own(a.master + at, n, lane, p);
            if constexpr (EIGHT) {
                top_m = __reduce_max_sync(0xffffffffu, top_m);
                top_v = __reduce_max_sync(0xffffffffu, top_v);
                const bool rare = max(top_m, top_v) >= kRare;
                if (rare) {   // the largest finite magnitudes
                    top_m = top_v = 0;
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        if (8 * lane + i < n) {
                            top_m = max(top_m, finite_bits(m[i]));
                            top_v = max(top_v, finite_bits(v[i]));
                        }
                    top_m = __reduce_max_sync(0xffffffffu, top_m);
                    top_v = __reduce_max_sync(0xffffffffu, top_v);
                }
                const int sm = shared_exponent(top_m), sv = shared_exponent(top_v);
                const uint32_t word = mixed(start + uint32_t(block) * 0x9E3779B1u);
                uint2 cm, cv;
                if (rare)
                    encode<true>(m, v, sm, sv, word, lane, cm, cv);
                else
                    encode<false>(m, v, sm, sv, word, lane, cm, cv);
                store_own(static_cast<uint8_t *>(a.m) + at, n, lane, cm);
                store_own(static_cast<uint8_t *>(a.v) + at, n, lane, cv);
                if (lane == 0) {
                    a.m_exp[block] = int8_t(sm);
                    a.v_exp[block] = int8_t(sv);
                }
            } else {
                store_own(static_cast<float *>(a.m) + at, n, lane, m);
                store_own(static_cast<float *>(a.v) + at, n, lane, v);
            }
        }
        item = next;
    }
    if (threadIdx.x == 0 && before == gridDim.x - 1) {
        a.state->beta1_t *= a.beta1d;
        a.state->beta2_t *= a.beta2d;
        a.state->step++;
        a.state->ticket = 0;
    }
}

__global__ void __launch_bounds__(kThreads) values_kernel(int64_t blocks, const uint8_t *m, const uint8_t *v,
                                                          const int8_t *m_exp, const int8_t *v_exp,
                                                          __nv_bfloat16 *m_out, __nv_bfloat16 *v_out) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    for (int64_t b = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> 5; b < blocks; b += int64_t(gridDim.x) * kWarps) {
        const int64_t at = b * kBlock + 8 * lane;
        const uint2 cm = *reinterpret_cast<const uint2 *>(m + at), cv = *reinterpret_cast<const uint2 *>(v + at);
        float x[8];
        decode_m(cm, m_exp[b], x);
        store8(m_out + at, x);
        decode_v(cv, v_exp[b], x);
        store8(v_out + at, x);
    }
}

// ---- host -----------------------------------------------------------------------------

int check_info(const nest_table_info *info) {
    if (!info || info->tensors < 0 || info->blocks < 0 || info->items < 0 || info->items > info->blocks ||
        info->table_bytes < int64_t(sizeof(Entry)) * info->tensors + int64_t(sizeof(Item)) * info->items)
        return NEST_E_INVALID;
    return info->blocks > INT32_MAX ? NEST_E_LIMITS : NEST_OK;
}

int blocks_for(int64_t items) { return int(items < 1 ? 1 : items < kSMs * 8 ? items : kSMs * 8); }

}  // namespace

}  // namespace nest

using namespace nest;

extern "C" {

int nest_table_query(const nest_tensor *t, int32_t n, nest_table_info *out) {
    if (!out || n < 0 || (n && !t)) return NEST_E_INVALID;
    int64_t blocks = 0, items = 0;
    for (int32_t i = 0; i < n; i++) {
        if (t[i].numel < 0 || (t[i].numel && !t[i].grad)) return NEST_E_INVALID;
        if (t[i].numel > int64_t(INT32_MAX) * kBlock) return NEST_E_LIMITS;
        blocks += blocks_in(t[i].numel);
        items += (blocks_in(t[i].numel) + kItemBlocks - 1) / kItemBlocks;
        if (blocks > INT32_MAX) return NEST_E_LIMITS;
    }
    out->table_bytes = int64_t(sizeof(Entry)) * n + int64_t(sizeof(Item)) * items;
    out->blocks = blocks;
    out->items = items;
    out->tensors = n;
    out->reserved = 0;
    return NEST_OK;
}

int nest_table_pack(const nest_tensor *t, int32_t n, const nest_table_info *info, void *table) {
    nest_table_info need;
    if (const int rc = nest_table_query(t, n, &need)) return rc;
    if (!info || need.tensors != info->tensors || need.items != info->items || need.blocks != info->blocks ||
        need.table_bytes != info->table_bytes || (need.table_bytes && !table))
        return NEST_E_INVALID;
    unsigned char *entries = static_cast<unsigned char *>(table), *items = entries + sizeof(Entry) * n;
    int64_t first = 0;
    for (int32_t i = 0; i < n; i++) {
        const Entry e = {t[i].weight, t[i].grad, t[i].numel, first, t[i].weight_decay, t[i].lr_scale, 0};
        std::memcpy(entries + sizeof(Entry) * i, &e, sizeof e);
        const int64_t blocks = blocks_in(t[i].numel);
        for (int64_t b = 0; b < blocks; b += kItemBlocks, items += sizeof(Item)) {
            const Item it = {i, int32_t(b)};
            std::memcpy(items, &it, sizeof it);
        }
        first += blocks;
    }
    return NEST_OK;
}

size_t nest_grad_norm_workspace_size(const nest_table_info *info) {
    if (check_info(info)) return 0;
    return (size_t(blocks_for(info->items)) * 4 + 255) & ~size_t(255);
}

int nest_grad_norm(const nest_table_info *info, const void *table, int32_t grad_type, float max_norm, float *out,
                   void *workspace, size_t ws_bytes, void *stream) {
    if (const int rc = check_info(info)) return rc;
    if (!out || !valid_type(grad_type) || !(max_norm > 0.0f) || (info->items && !table) || !aligned_to(table, 16))
        return NEST_E_INVALID;
    if (!workspace || ws_bytes < nest_grad_norm_workspace_size(info) || !aligned_to(workspace, 256))
        return NEST_E_WORKSPACE;
    const int blocks = blocks_for(info->items);
    float *part = static_cast<float *>(workspace);
    const int rc = with_type(grad_type, [&](auto t) {
        return launch_kernel(norm_kernel<decltype(t)>, dim3(blocks), dim3(kThreads), 0, stream, 1, "norm launch", table,
                             int(info->tensors), int(info->items), part);
    });
    if (rc) return rc;
    return launch_kernel(norm_finish_kernel, dim3(1), dim3(kThreads), 0, stream, 1, "norm finish launch",
                         static_cast<const float *>(part), blocks, max_norm, out);
}

int nest_adamw(const nest_table_info *info, const void *table, const nest_adamw_args *p, void *stream) {
    if (const int rc = check_info(info)) return rc;
    if (!p || !valid_type(p->weight_type) || !valid_type(p->grad_type) || (p->state_bits != 8 && p->state_bits != 32) ||
        !p->state || !aligned_to(p->state, 16) || !aligned_to(table, 16))
        return NEST_E_INVALID;
    if (!(p->beta1 >= 0.0 && p->beta1 < 1.0) || !(p->beta2 >= 0.0 && p->beta2 < 1.0) || !(p->eps >= 0.0) ||
        !std::isfinite(p->lr) || !std::isfinite(p->eps))
        return NEST_E_INVALID;
    if (info->blocks) {
        const bool eight = p->state_bits == 8;
        if (!table || !p->m || !p->v || (p->weight_type != NEST_F32) != (p->master != nullptr) ||
            eight != (p->m_exp != nullptr) || eight != (p->v_exp != nullptr) || !aligned_to(p->m, 256) ||
            !aligned_to(p->v, 256) || !aligned_to(p->master, 256) || !aligned_to(p->m_exp, 256) ||
            !aligned_to(p->v_exp, 256))
            return NEST_E_INVALID;
    }
    const StepArgs a = {table, info->tensors, int(info->items), float(p->lr), float(p->beta1), float(p->beta2),
                        float(1.0 - p->beta1), float(1.0 - p->beta2), float(p->eps), p->beta1, p->beta2, p->seed,
                        p->master, p->m, p->v, p->m_exp, p->v_exp, p->state, p->grad_scale};
    const dim3 grid(blocks_for(info->items));
    return with_type(p->weight_type, [&](auto w) {
        using W = decltype(w);
        return with_type(p->grad_type, [&](auto g) {
            using G = decltype(g);
            return p->state_bits == 8
                       ? launch_kernel(adamw_kernel<W, G, true>, grid, dim3(kThreads), 0, stream, 1, "adamw launch", a)
                       : launch_kernel(adamw_kernel<W, G, false>, grid, dim3(kThreads), 0, stream, 1, "adamw launch", a);
        });
    });
}

int nest_adamw_values(const nest_table_info *info, const void *m, const void *v, const int8_t *m_exp,
                      const int8_t *v_exp, void *m_out, void *v_out, void *stream) {
    if (const int rc = check_info(info)) return rc;
    if (!info->blocks) return NEST_OK;
    if (!m || !v || !m_exp || !v_exp || !m_out || !v_out || !aligned_to(m, 256) || !aligned_to(v, 256) ||
        !aligned_to(m_out, 256) || !aligned_to(v_out, 256))
        return NEST_E_INVALID;
    const int64_t grid_blocks = (info->blocks + kWarps - 1) / kWarps;
    const dim3 grid(unsigned(grid_blocks < kSMs * 8 ? grid_blocks : kSMs * 8));
    return launch_kernel(values_kernel, grid, dim3(kThreads), 0, stream, 1, "adamw values launch", info->blocks,
                         static_cast<const uint8_t *>(m), static_cast<const uint8_t *>(v), m_exp, v_exp,
                         static_cast<__nv_bfloat16 *>(m_out), static_cast<__nv_bfloat16 *>(v_out));
}

}  // extern "C"
