// Routing of tokens to experts: softmax gates, the k largest, per-expert counts and the
// balance loss, and the gradient with respect to the logits (definitions in nest_train.h).
//
// Forward: one warp per row holds the row in registers (expert e in lane e % 32), so the
// logits are read once.  The chosen experts come from k rounds of a warp-wide maximum of
// (logit, lower index) keys.  Every warp sums the gates of its rows per expert in
// registers; the block adds its warps in order and writes one partial row of sums and
// counts, and a second kernel adds the blocks' rows in order: no result depends on the
// order in which blocks run.
#include "nest_train.cuh"

namespace nest {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kFinishThreads = 1024;

struct RouteArgs {
    const void *logits;
    const uint8_t *mask;
    int64_t tokens, row_stride, col_stride;
    int experts, k, normalize;
};

// Orders floats as unsigned words (-0 and +0 alike); NaN and minus infinity give 0.
__device__ __forceinline__ uint32_t order_word(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    const uint32_t o = b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
    return x > -INFINITY ? o : 0u;
}

// Loads row t and returns whether it is live; x holds minus infinity past the last expert.
template <typename T, int V>
__device__ __forceinline__ bool load_row(const RouteArgs &a, int64_t t, int lane, float (&x)[V]) {
    if (a.mask && !a.mask[t]) return false;
    const T *row = static_cast<const T *>(a.logits) + t * a.row_stride;
    bool any = false;
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int e = lane + 32 * i;
        x[i] = e < a.experts ? to_f32(row[e * a.col_stride]) : -INFINITY;
        any |= x[i] != -INFINITY;
    }
    return __any_sync(0xffffffffu, any);
}

// p = softmax of the row.  A NaN or an infinite maximum makes every gate NaN.
template <int V>
__device__ __forceinline__ void softmax_row(const RouteArgs &a, int lane, const float (&x)[V], float (&p)[V]) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; i++) top = fmaxf(top, x[i]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; i++) {
        p[i] = lane + 32 * i < a.experts ? __expf(x[i] - top) : 0.0f;
        sum += p[i];
    }
    const float inv = 1.0f / warp_sum(sum);
#pragma unroll
    for (int i = 0; i < V; i++) p[i] = lane + 32 * i < a.experts ? p[i] * inv : 0.0f;
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) route_kernel(RouteArgs a, int32_t *ids, float *weights, float *part_p,
                                                         int32_t *part_c, int32_t *part_n) {
    extern __shared__ unsigned char sh[];
    float *sh_p = reinterpret_cast<float *>(sh);                         // [kWarps][experts]
    int32_t *sh_c = reinterpret_cast<int32_t *>(sh_p + kWarps * a.experts);   // [experts], then live rows
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e <= a.experts; e += kThreads) sh_c[e] = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; i++) acc[i] = 0.0f;
    int live = 0;
    for (int64_t t = int64_t(blockIdx.x) * kWarps + warp; t < a.tokens; t += int64_t(gridDim.x) * kWarps) {
        float x[V], p[V];
        int32_t id = -1;
        float w = 0.0f;
        if (load_row<T, V>(a, t, lane, x)) {
            live++;
            softmax_row<V>(a, lane, x, p);
            uint32_t key[V];
#pragma unroll
            for (int i = 0; i < V; i++) {
                acc[i] += p[i];
                key[i] = order_word(x[i]);
            }
            for (int j = 0; j < a.k; j++) {
                unsigned long long best = 0;
#pragma unroll
                for (int i = 0; i < V; i++) {
                    const unsigned long long c =
                        (static_cast<unsigned long long>(key[i]) << 32) | uint32_t(~(lane + 32 * i));
                    best = c > best ? c : best;
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) {
                    const unsigned long long c = __shfl_xor_sync(0xffffffffu, best, o);
                    best = c > best ? c : best;
                }
                if (!(best >> 32)) break;
                const int e = int(~uint32_t(best));
                float g = 0.0f;
#pragma unroll
                for (int i = 0; i < V; i++)
                    if (lane + 32 * i == e) {
                        g = p[i];
                        key[i] = 0;
                    }
                g = __shfl_sync(0xffffffffu, g, e & 31);
                if (lane == j) {
                    id = e;
                    w = g;
                }
            }
            if (id >= 0) atomicAdd(&sh_c[id], 1);
            if (a.normalize) {
                const float s = warp_sum(w);
                if (id >= 0) w /= s;
            }
        }
        if (lane < a.k) {
            ids[t * a.k + lane] = id;
            weights[t * a.k + lane] = w;
        }
    }
#pragma unroll
    for (int i = 0; i < V; i++)
        if (lane + 32 * i < a.experts) sh_p[warp * a.experts + lane + 32 * i] = acc[i];
    if (lane == 0 && live) atomicAdd(&sh_c[a.experts], live);
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += kThreads) {
        float s = 0.0f;
        for (int w = 0; w < kWarps; w++) s += sh_p[w * a.experts + e];
        part_p[int64_t(blockIdx.x) * a.experts + e] = s;
        part_c[int64_t(blockIdx.x) * a.experts + e] = sh_c[e];
    }
    if (threadIdx.x == 0) part_n[blockIdx.x] = sh_c[a.experts];
}

__global__ void __launch_bounds__(kFinishThreads) route_finish_kernel(int experts, int k, int blocks,
                                                                      const float *part_p, const int32_t *part_c,
                                                                      const int32_t *part_n, int32_t *counts,
                                                                      int32_t *live, float *mean_prob, float *loss) {
    __shared__ double sh_s[kFinishThreads / 32];
    pdl_wait();
    pdl_trigger();
    int n = 0;
    for (int b = 0; b < blocks; b++) n += part_n[b];
    const int e = threadIdx.x;
    double dot = 0.0;
    if (e < experts) {
        float s = 0.0f;
        int c = 0;
        for (int b = 0; b < blocks; b++) {
            s += part_p[int64_t(b) * experts + e];
            c += part_c[int64_t(b) * experts + e];
        }
        const float mean = n ? s / float(n) : 0.0f;
        counts[e] = c;
        mean_prob[e] = mean;
        dot = double(mean) * c;
    }
    dot = warp_sum(dot);
    if ((threadIdx.x & 31) == 0) sh_s[threadIdx.x >> 5] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int w = 0; w < kFinishThreads / 32; w++) s += sh_s[w];
        *live = n;
        *loss = n ? float(s * experts / (double(k) * n)) : 0.0f;
    }
}

// One warp per row; the gates are computed again from the logits, which the row needs
// anyway, so nothing but ids and weights is kept from the forward pass.  The counts
// enter as c[e] - k n / E: a constant in d drops out of the gradient, and without it the
// subtraction of the mean loses no digits.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) route_backward_kernel(RouteArgs a, const int32_t *ids, const float *weights,
                                                                  const int32_t *counts, const int32_t *live,
                                                                  const float *grad_weights, const float *grad_loss,
                                                                  T *grad, int64_t grad_stride) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float n = float(*live);
    const float even = float(a.k) * n / float(a.experts);
    const float f = grad_loss && n > 0.0f ? *grad_loss * float(a.experts) / (float(a.k) * n * n) : 0.0f;
    for (int64_t t = int64_t(blockIdx.x) * kWarps + warp; t < a.tokens; t += int64_t(gridDim.x) * kWarps) {
        float x[V], d[V];
        T *out = grad + t * grad_stride;
        if (!load_row<T, V>(a, t, lane, x)) {
#pragma unroll
            for (int i = 0; i < V; i++)
                if (lane + 32 * i < a.experts) out[lane + 32 * i] = from_f32<T>(0.0f);
            continue;
        }
        float p[V];
        softmax_row<V>(a, lane, x, p);
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int e = lane + 32 * i;
            d[i] = e < a.experts ? f * (float(counts[e]) - even) : 0.0f;
        }
        if (grad_weights) {
            int id = -1;
            float u = 0.0f, w = 0.0f;
            if (lane < a.k) {
                id = ids[t * a.k + lane];
                if (uint32_t(id) >= uint32_t(a.experts)) id = -1;
                if (id >= 0) {
                    u = grad_weights[t * a.k + lane];
                    w = weights[t * a.k + lane];
                }
            }
            if (a.normalize) {
                const float dot = warp_sum(u * w);
                float total = 0.0f;
                for (int j = 0; j < a.k; j++) {
                    const int e = __shfl_sync(0xffffffffu, id, j);
#pragma unroll
                    for (int i = 0; i < V; i++)
                        if (lane + 32 * i == e) total += p[i];
                }
                total = warp_sum(total);
                u = id >= 0 ? (u - dot) / total : 0.0f;
            }
            for (int j = 0; j < a.k; j++) {
                const int e = __shfl_sync(0xffffffffu, id, j);
                const float g = __shfl_sync(0xffffffffu, u, j);
#pragma unroll
                for (int i = 0; i < V; i++)
                    if (lane + 32 * i == e) d[i] += g;
            }
        }
        float mean = 0.0f;
#pragma unroll
        for (int i = 0; i < V; i++) mean += p[i] * d[i];
        mean = warp_sum(mean);
#pragma unroll
        for (int i = 0; i < V; i++)
            if (lane + 32 * i < a.experts) out[lane + 32 * i] = from_f32<T>(p[i] * (d[i] - mean));
    }
}

int check(const nest_route_desc *d) {
    if (!d || d->tokens < 0 || d->row_stride < 0 || d->col_stride < 0 || !valid_type(d->dtype) || d->experts < 1 ||
        d->k < 1 || d->k > d->experts || (d->normalize & ~1))
        return NEST_E_INVALID;
    if (d->experts > 1024 || d->k > 32 || d->tokens > INT32_MAX || d->tokens * d->k > INT32_MAX) return NEST_E_LIMITS;
    return NEST_OK;
}

int blocks_of(const nest_route_desc *d) {
    const int64_t b = (d->tokens + kWarps - 1) / kWarps;
    return int(b < 1 ? 1 : b < kSMs * 4 ? b : kSMs * 4);
}

// fn(integral constant V): the values per lane of a row of `experts`.
template <int V> struct Values { static constexpr int v = V; };
template <typename F>
int with_values(int experts, F fn) {
    if (experts <= 32) return fn(Values<1>{});
    if (experts <= 64) return fn(Values<2>{});
    if (experts <= 128) return fn(Values<4>{});
    if (experts <= 256) return fn(Values<8>{});
    if (experts <= 512) return fn(Values<16>{});
    return fn(Values<32>{});
}

RouteArgs args_of(const nest_route_desc *d, const void *logits, const uint8_t *mask) {
    return {logits, mask, d->tokens, d->row_stride, d->col_stride, d->experts, d->k, d->normalize};
}

}  // namespace

}  // namespace nest

using namespace nest;

extern "C" {

size_t nest_route_workspace_size(const nest_route_desc *d) {
    if (check(d)) return 0;
    return (size_t(blocks_of(d)) * (8 * size_t(d->experts) + 4) + 255) & ~size_t(255);
}

int nest_route(const nest_route_desc *d, const void *logits, const uint8_t *mask, int32_t *ids, float *weights,
               int32_t *counts, int32_t *live, float *mean_prob, float *loss, void *workspace, size_t ws_bytes,
               void *stream) {
    if (const int rc = check(d)) return rc;
    if (!counts || !live || !mean_prob || !loss || (d->tokens && (!logits || !ids || !weights))) return NEST_E_INVALID;
    if (d->tokens && !aligned_to(logits, type_bytes(d->dtype))) return NEST_E_INVALID;
    if (!workspace || ws_bytes < nest_route_workspace_size(d) || !aligned_to(workspace, 256)) return NEST_E_WORKSPACE;
    const int blocks = blocks_of(d);
    float *part_p = static_cast<float *>(workspace);
    int32_t *part_c = reinterpret_cast<int32_t *>(part_p + int64_t(blocks) * d->experts);
    int32_t *part_n = part_c + int64_t(blocks) * d->experts;
    const RouteArgs a = args_of(d, logits, mask);
    const size_t smem = size_t(4) * (kWarps * d->experts + d->experts + 1);
    const int rc = with_type(d->dtype, [&](auto t) {
        using T = decltype(t);
        return with_values(d->experts, [&](auto v) {
            return launch_kernel(route_kernel<T, decltype(v)::v>, dim3(blocks), dim3(kThreads), smem, stream, 1,
                                 "route launch", a, ids, weights, part_p, part_c, part_n);
        });
    });
    if (rc) return rc;
    return launch_kernel(route_finish_kernel, dim3(1), dim3(kFinishThreads), 0, stream, 1, "route finish launch",
                         int(d->experts), int(d->k), blocks, static_cast<const float *>(part_p),
                         static_cast<const int32_t *>(part_c), static_cast<const int32_t *>(part_n), counts, live,
                         mean_prob, loss);
}

int nest_route_backward(const nest_route_desc *d, const void *logits, const uint8_t *mask, const int32_t *ids,
                        const float *weights, const int32_t *counts, const int32_t *live, const float *grad_weights,
                        const float *grad_loss, void *grad_logits, int64_t grad_stride, void *stream) {
    if (const int rc = check(d)) return rc;
    if (grad_stride < d->experts) return NEST_E_INVALID;
    if (!d->tokens) return NEST_OK;
    if (!logits || !ids || !weights || !counts || !live || !grad_logits) return NEST_E_INVALID;
    if (!aligned_to(logits, type_bytes(d->dtype)) || !aligned_to(grad_logits, type_bytes(d->dtype)))
        return NEST_E_INVALID;
    const RouteArgs a = args_of(d, logits, mask);
    const int64_t b = (d->tokens + kWarps - 1) / kWarps;
    return with_type(d->dtype, [&](auto t) {
        using T = decltype(t);
        return with_values(d->experts, [&](auto v) {
            return launch_kernel(route_backward_kernel<T, decltype(v)::v>, dim3(unsigned(b < kSMs * 8 ? b : kSMs * 8)),
                                 dim3(kThreads), 0, stream, 1, "route backward launch", a, ids, weights, counts, live,
                                 grad_weights, grad_loss, static_cast<T *>(grad_logits), grad_stride);
        });
    });
}

}  // extern "C"
