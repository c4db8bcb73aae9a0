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
constexpr int kPerLane = kBlock / 32;

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

// ---- gradient norm ----------------------------------------------------------------

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_kernel(const void *table, int tensors, int items, double *part) {
    __shared__ double sh[kWarps];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Entry *entries = static_cast<const Entry *>(table);
    const Item *list = items_of(table, tensors);
    double sum = 0.0;
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        const Item item = list[it];
        const Entry e = entries[item.tensor];
        const T *g = static_cast<const T *>(e.grad);
        float s = 0.0f;
        for (int b = item.block + warp; b < item.block + kItemBlocks; b += kWarps)
            for (int i = 0; i < kPerLane; i++) {
                const int64_t j = int64_t(b) * kBlock + lane + 32 * i;
                if (j < e.numel) {
                    const float x = to_f32(g[j]);
                    s = fmaf(x, x, s);
                }
            }
        sum += s;
    }
    sum = warp_sum(sum);
    if (lane == 0) sh[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int w = 0; w < kWarps; w++) s += sh[w];
        part[blockIdx.x] = s;
    }
}

__global__ void __launch_bounds__(32) norm_finish_kernel(const double *part, int blocks, float max_norm, float *out) {
    pdl_wait();
    pdl_trigger();
    double s = 0.0;
    for (int b = threadIdx.x; b < blocks; b += 32) s += part[b];
    s = warp_sum(s);
    if (threadIdx.x == 0) {
        const float norm = float(sqrt(s));
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
// exponent field offset + f; under the smallest normal value the code counts steps of 1 / small.
template <int OFFSET>
__device__ __forceinline__ uint32_t code_of(float y, uint32_t r, float small) {
    const uint32_t normal = ((__float_as_uint(y) + (r << 4)) >> 20) - (OFFSET << 3);
    const uint32_t fixed = uint32_t(fmaf(y, small, float(r) * 0x1p-16f));
    return __float_as_uint(y) < (uint32_t(OFFSET + 1) << 23) ? fixed : normal;
}

__device__ __forceinline__ uint8_t encode_m(float m, int s, uint32_t r) {
    const uint32_t sign = (__float_as_uint(m) >> 24) & 0x80u;
    uint32_t c = min(code_of<120>(fabsf(m) * power2(8 - s), r, 512.0f), 0x7Eu);
    if (!isfinite(m)) c = 0x7F;
    return uint8_t(c | sign);
}

__device__ __forceinline__ uint8_t encode_v(float v, int s, uint32_t r) {
    const uint32_t c = min(code_of<95>(v * power2(-1 - s), r, 0x1p34f), 0xFEu);
    return uint8_t(isfinite(v) ? c : 0xFFu);
}

__device__ __forceinline__ float decode_m(uint32_t c, int s) {
    // the code's 7 lower bits as a 32-bit float with the exponent 120 too small
    const float y = __uint_as_float((c & 0x7Fu) << 20) * 0x1p120f * power2(s - 8);
    return (c & 0x7Fu) == 0x7Fu ? NAN : (c & 0x80u) ? -y : y;
}

__device__ __forceinline__ float decode_v(uint32_t c, int s) {
    const float y = __uint_as_float(c << 20) * 0x1p95f * power2(s + 1);
    return c == 0xFFu ? NAN : y;
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

template <typename W, typename G, bool EIGHT>
__global__ void __launch_bounds__(kThreads) adamw_kernel(StepArgs a) {
    constexpr bool kOwnMaster = sizeof(W) == 4;
    pdl_wait();
    pdl_trigger();
    const float scale = a.grad_scale ? *a.grad_scale : 1.0f;
    if (!isfinite(scale)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const double b1t = a.state->beta1_t * a.beta1d, b2t = a.state->beta2_t * a.beta2d;
    const int64_t step = a.state->step + 1;
    const float inv1 = 1.0f / float(1.0 - b1t), root2 = rsqrtf(float(1.0 - b2t));
    const uint32_t start = mixed(a.seed ^ mixed(uint32_t(step)));
    const Entry *entries = static_cast<const Entry *>(a.table);
    const Item *list = items_of(a.table, a.tensors);
    for (int it = blockIdx.x; it < a.items; it += gridDim.x) {
        const Item item = list[it];
        const Entry e = entries[item.tensor];
        const float lr = a.lr * e.lr_scale, decay = e.weight_decay;
        for (int b = item.block + warp; b < item.block + kItemBlocks; b += kWarps) {
            const int64_t j0 = int64_t(b) * kBlock;
            if (j0 >= e.numel) break;
            const int64_t block = e.first + b;
            int sm = 0, sv = 0;
            if constexpr (EIGHT) {
                sm = a.m_exp[block];
                sv = a.v_exp[block];
            }
            float m[kPerLane], v[kPerLane];
            uint32_t top_m = 0, top_v = 0;
#pragma unroll
            for (int i = 0; i < kPerLane; i++) {
                const int pos = lane + 32 * i;
                const int64_t at = block * kBlock + pos;
                m[i] = v[i] = 0.0f;
                if (j0 + pos < e.numel) {
                    const float g = to_f32(static_cast<const G *>(e.grad)[j0 + pos]) * scale;
                    if constexpr (EIGHT) {
                        m[i] = decode_m(static_cast<const uint8_t *>(a.m)[at], sm);
                        v[i] = decode_v(static_cast<const uint8_t *>(a.v)[at], sv);
                    } else {
                        m[i] = static_cast<const float *>(a.m)[at];
                        v[i] = static_cast<const float *>(a.v)[at];
                    }
                    // each product rounded by itself, so that a moment is the same number
                    // wherever these formulas are evaluated, and its 8-bit code with it
                    m[i] = __fadd_rn(__fmul_rn(m[i], a.beta1), __fmul_rn(g, a.rest1));
                    v[i] = __fadd_rn(__fmul_rn(v[i], a.beta2), __fmul_rn(__fmul_rn(g, g), a.rest2));
                    W *w = static_cast<W *>(e.weight) + j0 + pos;
                    float p = kOwnMaster ? to_f32(*w) : a.master[at];
                    p -= lr * (m[i] * inv1 / (sqrtf(v[i]) * root2 + a.eps) + decay * p);
                    if (!kOwnMaster) a.master[at] = p;
                    *w = from_f32<W>(p);
                    if constexpr (EIGHT) {
                        top_m = max(top_m, finite_bits(m[i]));
                        top_v = max(top_v, finite_bits(v[i]));
                    } else {
                        static_cast<float *>(a.m)[at] = m[i];
                        static_cast<float *>(a.v)[at] = v[i];
                    }
                }
            }
            if constexpr (EIGHT) {
                sm = shared_exponent(__reduce_max_sync(0xffffffffu, top_m));
                sv = shared_exponent(__reduce_max_sync(0xffffffffu, top_v));
                const uint32_t noise = mixed(start + uint32_t(block) * 0x9E3779B1u);
#pragma unroll
                for (int i = 0; i < kPerLane; i++) {
                    const int pos = lane + 32 * i;
                    uint32_t x = noise + uint32_t(pos) * 0x9E3779B1u;
                    x ^= x >> 15;
                    x *= 0x6A09E667u;
                    x ^= x >> 16;
                    if (j0 + pos < e.numel) {
                        const int64_t at = block * kBlock + pos;
                        static_cast<uint8_t *>(a.m)[at] = encode_m(m[i], sm, x >> 16);
                        static_cast<uint8_t *>(a.v)[at] = encode_v(v[i], sv, x & 0xFFFFu);
                    }
                }
                if (lane == 0) {
                    a.m_exp[block] = int8_t(sm);
                    a.v_exp[block] = int8_t(sv);
                }
            }
        }
    }
    // the last block to get here has seen every block read the step's state
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(&a.state->ticket, 1u) == gridDim.x - 1) {
            a.state->beta1_t = b1t;
            a.state->beta2_t = b2t;
            a.state->step = step;
            a.state->ticket = 0;
        }
    }
}

__global__ void __launch_bounds__(kThreads) values_kernel(int64_t blocks, const uint8_t *m, const uint8_t *v,
                                                          const int8_t *m_exp, const int8_t *v_exp,
                                                          __nv_bfloat16 *m_out, __nv_bfloat16 *v_out) {
    pdl_wait();
    pdl_trigger();
    for (int64_t at = int64_t(blockIdx.x) * kThreads + threadIdx.x; at < blocks * kBlock;
         at += int64_t(gridDim.x) * kThreads) {
        m_out[at] = __float2bfloat16_rn(decode_m(m[at], m_exp[at / kBlock]));
        v_out[at] = __float2bfloat16_rn(decode_v(v[at], v_exp[at / kBlock]));
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
    return (size_t(blocks_for(info->items)) * 8 + 255) & ~size_t(255);
}

int nest_grad_norm(const nest_table_info *info, const void *table, int32_t grad_type, float max_norm, float *out,
                   void *workspace, size_t ws_bytes, void *stream) {
    if (const int rc = check_info(info)) return rc;
    if (!out || !valid_type(grad_type) || !(max_norm > 0.0f) || (info->items && !table) || !aligned_to(table, 16))
        return NEST_E_INVALID;
    if (!workspace || ws_bytes < nest_grad_norm_workspace_size(info) || !aligned_to(workspace, 256))
        return NEST_E_WORKSPACE;
    const int blocks = blocks_for(info->items);
    double *part = static_cast<double *>(workspace);
    const int rc = with_type(grad_type, [&](auto t) {
        return launch_kernel(norm_kernel<decltype(t)>, dim3(blocks), dim3(kThreads), 0, stream, 1, "norm launch", table,
                             int(info->tensors), int(info->items), part);
    });
    if (rc) return rc;
    return launch_kernel(norm_finish_kernel, dim3(1), dim3(32), 0, stream, 1, "norm finish launch",
                         static_cast<const double *>(part), blocks, max_norm, out);
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
    const dim3 grid(unsigned(info->blocks < kSMs * 16 ? info->blocks : kSMs * 16));
    return launch_kernel(values_kernel, grid, dim3(kThreads), 0, stream, 1, "adamw values launch", info->blocks,
                         static_cast<const uint8_t *>(m), static_cast<const uint8_t *>(v), m_exp, v_exp,
                         static_cast<__nv_bfloat16 *>(m_out), static_cast<__nv_bfloat16 *>(v_out));
}

}  // extern "C"
