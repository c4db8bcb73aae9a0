// Kernels of the routing operators (definitions in nest_train.h), one instantiation per
// element type in nest_route_f32.cu, nest_route_bf16.cu and nest_route_f16.cu.
//
// A warp takes a row at a time and holds it in registers, so the logits are read once, in
// pieces of up to 32 bytes per lane where alignment allows (VEC); the next row's are under
// way while one is worked on.
//
// Choice of the k largest.  A logit becomes a 32-bit word whose order is that of the logits,
// with its lowest bits replaced by the complement of the expert's index: all words of a row
// differ, and among logits that agree in the bits kept the lower index is the larger word.
// Each lane sorts its words once; then k rounds take the maximum over the lanes' largest words
// with one warp-wide reduction instruction each, and the lane that had it moves its list up.
// 16-bit logits lose nothing to the index.  With 32-bit logits up to 10 bits are lost: one
// more round gives the largest word left, and if two of these neighbours agree in the bits
// kept, or a gate is NaN, the row's choice is made again on whole logits.
//
// Sums.  Every warp adds up the gates of its rows per expert in registers, the block adds its
// warps in order, and the blocks' rows are added in order in 64 bits, so no result depends on
// the order in which blocks run.  Few rows: the whole grid is one cluster, whose blocks read one
// another's sums from shared memory, and the call is one launch.  Otherwise each block writes
// its row of sums to the workspace and a second kernel adds them.
#pragma once

#include <cooperative_groups.h>

#include "nest_train.cuh"

namespace nest {

struct RouteArgs {
    const void *logits;
    const uint8_t *mask;
    int64_t tokens, row_stride, col_stride;
    int experts, k, normalize;
    // forward
    int32_t *ids;
    float *weights;
    float *part_p;      // [blocks][experts], then counts likewise, then live rows; unused when joined
    int32_t *part_c, *part_n;
    int32_t *counts, *live;
    float *mean_prob, *loss;
    int joined;         // the grid is one cluster
    // backward
    const float *grad_weights, *grad_loss;
    void *grad;
    int64_t grad_stride;
    bool vector_grad;
};

// Rows of up to 32 V experts.  Values per lane, block size and blocks per SM that the kernels
// are compiled for: the registers of a row, of the next one and of the sums.
template <int V>
struct RouteShape {
    static constexpr int kWarps = V >= 32 ? 8 : 16;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kPerSm = V <= 8 ? 2 : 1;
};

namespace {

namespace cg = cooperative_groups;

constexpr int kFinishThreads = 1024;
constexpr int kCluster = 8;
constexpr float kLog2e = 1.44269504088896341f;

__device__ __forceinline__ float exp2_of(float x) {   // results below 2^-126 are 0
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float warp_max(float x) {   // NaN counts as nothing
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// Orders floats as unsigned words, -0 and +0 alike; minus infinity becomes kClosed.
constexpr uint32_t kClosed = 0x007FFFFFu;
__device__ __forceinline__ uint32_t order_word(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}

template <int BYTES> struct Piece;
template <> struct Piece<2> { using type = uint16_t; };
template <> struct Piece<4> { using type = uint32_t; };
template <> struct Piece<8> { using type = uint2; };
template <> struct Piece<16> { using type = uint4; };

// Which expert a lane's i-th value is: pieces of C neighbours, one lane's after another's.
template <int V, bool VEC>
struct Place {
    static constexpr int C = VEC ? (V < 8 ? V : 8) : 1;
    static __device__ __forceinline__ int of(int i, int lane) { return (i / C) * (32 * C) + lane * C + i % C; }
};

template <typename T, int N>
__device__ __forceinline__ void load_piece(const T *p, T *to) {
    if constexpr (sizeof(T) * N == 32) {
        uint32_t *w = reinterpret_cast<uint32_t *>(to);
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(p)
                     : "memory");
    } else {
        using P = typename Piece<sizeof(T) * N>::type;
        *reinterpret_cast<P *>(to) = *reinterpret_cast<const P *>(p);
    }
}

template <typename T, int N>
__device__ __forceinline__ void store_piece(T *p, const T *from) {
    if constexpr (sizeof(T) * N == 32) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(from);
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     :
                     : "l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        using P = typename Piece<sizeof(T) * N>::type;
        *reinterpret_cast<P *>(p) = *reinterpret_cast<const P *>(from);
    }
}

// A row as the lane holds it; minus infinity past the last expert.
template <typename T, int V, bool VEC>
__device__ __forceinline__ void fetch_row(const RouteArgs &a, const T *row, int lane, T (&x)[V]) {
    using L = Place<V, VEC>;
#pragma unroll
    for (int i = 0; i < V; i += L::C) {
        const int e = L::of(i, lane);
        if (e < a.experts) {   // VEC: E is a multiple of C
            if constexpr (VEC)
                load_piece<T, L::C>(row + e, x + i);
            else
                x[i] = row[e * a.col_stride];
        } else {
#pragma unroll
            for (int c = 0; c < L::C; c++) x[i + c] = from_f32<T>(-INFINITY);
        }
    }
}

// exp(x - top) over the row's own unit: one multiply-add and an exponential of base 2.  The
// rounding of top * log2(e) is the same factor in every gate of the row and leaves with the
// division by their sum.  A largest value near the type's end would overflow it: then the
// difference is taken first.
struct RowExp {
    float top, shift;
    bool far;
    __device__ __forceinline__ explicit RowExp(float t) : top(t), shift(t * kLog2e), far(fabsf(t) > 1e38f) {}
    __device__ __forceinline__ float operator()(float x) const {
        return exp2_of(far ? (x - top) * kLog2e : fmaf(x, kLog2e, -shift));
    }
};

// Whether a fetched row is live; x, its largest value, e = exp(x - top) and their sum.
template <typename T, int V>
__device__ __forceinline__ bool gates_of(const T (&raw)[V], float (&x)[V], float (&e)[V], float &top, float &sum) {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; i++) {
        x[i] = to_f32(raw[i]);
        top = fmaxf(top, x[i]);
    }
    top = warp_max(top);
    if (!(top > -INFINITY)) {   // closed, unless NaN is in it
        bool nan = false;
#pragma unroll
        for (int i = 0; i < V; i++) nan |= isnan(x[i]);
        if (!__any_sync(0xffffffffu, nan)) return false;
    }
    const RowExp ex(top);
    if (ex.far) {
#pragma unroll
        for (int i = 0; i < V; i++) e[i] = exp2_of((x[i] - top) * kLog2e);
    } else {
#pragma unroll
        for (int i = 0; i < V; i++) e[i] = exp2_of(fmaf(x[i], kLog2e, -ex.shift));
    }
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; i++) sum += e[i];
    sum = warp_sum(sum);
    return true;
}

// The sum over the warp of what only the first 8 lanes (FEW) or any lanes have; the others get it
// only in the second case, or as 0.
template <bool FEW>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = FEW ? 4 : 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sorts w[0 .. V) downwards (V a power of two): Batcher's merging of odd and even parts.
template <int V>
__device__ __forceinline__ void sort_down(uint32_t (&w)[V]) {
#pragma unroll
    for (int p = 1; p < V; p *= 2)
#pragma unroll
        for (int q = p; q > 0; q /= 2)
#pragma unroll
            for (int j = q % p; j < V - q; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; i++)
                    if (i + j + q < V && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const uint32_t hi = max(w[i + j], w[i + j + q]), lo = min(w[i + j], w[i + j + q]);
                        w[i + j] = hi;
                        w[i + j + q] = lo;
                    }
}

// The choice on whole logits, which are read again: lane j gets the j-th chosen expert or -1.
template <typename T, int V>
__device__ __forceinline__ int choose_exactly(const T *row, int64_t col_stride, int experts, int k) {
    const int lane = threadIdx.x & 31;
    uint32_t w[V], taken = 0;
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int e = lane + 32 * i;
        const float x = e < experts ? to_f32(row[e * col_stride]) : -INFINITY;
        w[i] = x > -INFINITY ? order_word(x) : 0u;   // 0 for NaN too
    }
    int id = -1;
#pragma unroll 1
    for (int j = 0; j < k; j++) {
        uint32_t best = 0;
        int at = INT32_MAX;
#pragma unroll
        for (int i = 0; i < V; i++)
            if (w[i] > best && !(taken >> i & 1)) {
                best = w[i];
                at = lane + 32 * i;
            }
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        if (!top) break;
        const int e = __reduce_min_sync(0xffffffffu, best == top ? at : INT32_MAX);
        if ((e & 31) == lane) taken |= 1u << (e >> 5);
        if (lane == j) id = e;
    }
    return id;
}

// Lane j gets the j-th chosen expert of the row or -1.  FEW: k is at most 8.  nan: some gate of
// the row is NaN.
template <typename T, int V, bool VEC, bool FEW>
__device__ __forceinline__ int choose(const RouteArgs &a, const T *row, const float (&x)[V], int lane, bool nan) {
    using L = Place<V, VEC>;
    constexpr uint32_t kIndex = 32 * V - 1;   // the bits that hold the index
    constexpr int kRest = sizeof(T) == 2 ? 0 : 1;   // whether the largest word left is looked at too
    const int k = a.k;
    bool again = nan;
    uint32_t mine = 0;
    if (!again) {
        uint32_t w[V];
#pragma unroll
        for (int i = 0; i < V; i++) w[i] = (order_word(x[i]) & ~kIndex) | (kIndex - L::of(i, lane));
        sort_down<V>(w);
        if constexpr (FEW) {
#pragma unroll
            for (int j = 0; j < 8; j++) {
                if (j >= k) break;
                const uint32_t last = __reduce_max_sync(0xffffffffu, w[0]);
                if (lane == j) mine = last;
                if (w[0] == last) {   // of a list only what the rounds left can reach is moved
                    constexpr int kNone = 0;
                    const int rounds = 8 + kRest - 1 - j;
#pragma unroll
                    for (int i = 0; i < V; i++)
                        if (i < rounds) w[i] = i + 1 < V ? w[i + 1 < V ? i + 1 : i] : kNone;
                }
            }
        } else {
#pragma unroll 1
            for (int j = 0; j < k; j++) {
                const uint32_t last = __reduce_max_sync(0xffffffffu, w[0]);
                if (lane == j) mine = last;
                if (w[0] == last) {
#pragma unroll
                    for (int i = 0; i + 1 < V; i++) w[i] = w[i + 1];
                    w[V - 1] = 0;
                }
            }
        }
        if (kRest) {
            const uint32_t left = __reduce_max_sync(0xffffffffu, w[0]);
            uint32_t next = __shfl_down_sync(0xffffffffu, mine, 1);
            if (lane == k - 1) next = left;
            again = __any_sync(0xffffffffu, lane < k && next > kClosed && ((mine ^ next) & ~kIndex) == 0);
        }
    }
    if (again) return choose_exactly<T, V>(row, a.col_stride, a.experts, k);
    return mine > kClosed ? int(kIndex - (mine & kIndex)) : -1;
}

// Experts first .. first + 31 (lane) summed over `rows` rows of sums and counts by the block's
// warps; warp 0 gets the result in p and c.
template <int WARPS, typename P, typename N>
__device__ __forceinline__ void add_rows(int rows, P part_p, N part_c, double (*sh_p)[32], int32_t (*sh_c)[32],
                                         double &p, int32_t &c) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    p = 0.0;
    c = 0;
    for (int r = warp; r < rows; r += WARPS) {
        p += part_p(r);
        c += part_c(r);
    }
    sh_p[warp][lane] = p;
    sh_c[warp][lane] = c;
    __syncthreads();
    if (warp == 0) {
        p = 0.0;
        c = 0;
        for (int w = 0; w < WARPS; w++) {
            p += sh_p[w][lane];
            c += sh_c[w][lane];
        }
    }
    __syncthreads();
}

// The results from `rows` rows, by the blocks of a cluster: each takes groups of 32 experts.
// row_p(r, e), row_c(r, e): sums and counts; n: live rows.
template <int WARPS, typename P, typename N>
__device__ __forceinline__ void finish(const RouteArgs &a, int rows, P row_p, N row_c, int n) {
    __shared__ double sh_p[WARPS][32];
    __shared__ int32_t sh_c[WARPS][32];
    __shared__ double sh_dot;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = int(cluster.block_rank()), ranks = int(cluster.num_blocks());
    const int lane = threadIdx.x & 31;
    double dot = 0.0;
    for (int first = 32 * rank; first < a.experts; first += 32 * ranks) {
        const int e = first + lane;
        const bool in = e < a.experts;
        double p;
        int32_t c;
        add_rows<WARPS>(rows, [&](int r) { return in ? row_p(r, e) : 0.0f; }, [&](int r) { return in ? row_c(r, e) : 0; },
                 sh_p, sh_c, p, c);
        if (threadIdx.x < 32 && in) {
            const double mean = n ? p / n : 0.0;
            a.counts[e] = c;
            a.mean_prob[e] = float(mean);
            dot += mean * c;
        }
    }
    if (threadIdx.x < 32) {
        dot = warp_sum(dot);
        if (lane == 0) sh_dot = dot;
    }
    cluster.sync();
    if (rank == 0 && threadIdx.x == 0) {
        dot = 0.0;
        for (int r = 0; r < ranks; r++) dot += *cluster.map_shared_rank(&sh_dot, r);
        *a.live = n;
        *a.loss = n ? float(dot * a.experts / (double(a.k) * n)) : 0.0f;
    }
    cluster.sync();   // the others' shared memory is read until here
}

template <typename T, int V, bool VEC, bool FEW>
__global__ void __launch_bounds__(RouteShape<V>::kThreads, RouteShape<V>::kPerSm) route_kernel(RouteArgs a) {
    constexpr int kWarps = RouteShape<V>::kWarps, kThreads = RouteShape<V>::kThreads;
    using L = Place<V, VEC>;
    extern __shared__ unsigned char sh[];
    float *sh_sum = reinterpret_cast<float *>(sh);                            // [kWarps][experts]
    int32_t *sh_count = reinterpret_cast<int32_t *>(sh_sum + kWarps * a.experts);   // [experts], then live rows
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int stride = int(gridDim.x) * kWarps, tokens = int(a.tokens);
    int t = int(blockIdx.x) * kWarps + warp;
    const T *row = static_cast<const T *>(a.logits) + t * a.row_stride;
    const int64_t row_step = stride * a.row_stride;
    int at = t * a.k + lane;             // T k is below 2^31
    const int at_step = stride * a.k;
    T raw[V];
    bool on = t < tokens && !(a.mask && !a.mask[t]);
    if (on) fetch_row<T, V, VEC>(a, row, lane, raw);
    for (int e = threadIdx.x; e <= a.experts; e += kThreads) sh_count[e] = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; i++) acc[i] = 0.0f;
    int live = 0;
#pragma unroll 1
    for (; t < tokens; t += stride, at += at_step) {
        float x[V], e[V], top, sum;
        const bool is_live = on && gates_of<T, V>(raw, x, e, top, sum);
        const T *here = row;
        row += row_step;
        on = t < tokens - stride && !(a.mask && !a.mask[t + stride]);
        if (on) fetch_row<T, V, VEC>(a, row, lane, raw);
        int id = -1;
        float w = 0.0f;
        if (is_live) {
            live++;
            const float inv = __fdividef(1.0f, sum);
#pragma unroll
            for (int i = 0; i < V; i++) acc[i] = fmaf(e[i], inv, acc[i]);
            id = choose<T, V, VEC, FEW>(a, here, x, lane, isnan(sum));
            if (id >= 0) {
                w = RowExp(top)(to_f32(here[id * a.col_stride]));
                atomicAdd(&sh_count[id], 1);
            }
            // in a row with NaN every gate is NaN, also those that are 0 here
            w *= a.normalize && !isnan(sum) ? __fdividef(1.0f, group_sum<FEW>(w)) : inv;
            if (id < 0) w = 0.0f;
        }
        if (lane < a.k) {
            a.ids[at] = id;
            a.weights[at] = w;
        }
    }
#pragma unroll
    for (int i = 0; i < V; i++)
        if (L::of(i, lane) < a.experts) sh_sum[warp * a.experts + L::of(i, lane)] = acc[i];
    if (lane == 0 && live) atomicAdd(&sh_count[a.experts], live);
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += kThreads) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; w++) s += sh_sum[w * a.experts + e];
        if (a.joined) {
            sh_sum[e] = s;   // only this thread reads this column
        } else {
            a.part_p[int64_t(blockIdx.x) * a.experts + e] = s;
            a.part_c[int64_t(blockIdx.x) * a.experts + e] = sh_count[e];
        }
    }
    if (!a.joined) {
        if (threadIdx.x == 0) a.part_n[blockIdx.x] = sh_count[a.experts];
        return;
    }
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    int n = 0;
    for (int r = 0; r < int(gridDim.x); r++) n += *cluster.map_shared_rank(sh_count + a.experts, r);
    finish<kWarps>(a, int(gridDim.x), [&](int r, int e) { return cluster.map_shared_rank(sh_sum, r)[e]; },
           [&](int r, int e) { return cluster.map_shared_rank(sh_count, r)[e]; }, n);
}

// The gradient.  With the weights w that the forward pass wrote, what reaches a chosen logit
// beyond the softmax's own term is w (grad_weight - dot) for normalised gates and
// w grad_weight for plain ones, dot = sum of w grad_weight over the row's chosen; only plain
// gates leave dot in the row's mean.  The counts enter as c - k n / E: a constant in d
// drops out of the gradient, and without it the subtraction of the mean loses no digits.
// The k terms reach their experts' lanes through the warp's row of shared memory.
template <typename T, int V, bool VEC>
__global__ void __launch_bounds__(RouteShape<V>::kThreads, RouteShape<V>::kPerSm) route_backward_kernel(RouteArgs a) {
    constexpr int kWarps = RouteShape<V>::kWarps;
    using L = Place<V, VEC>;
    extern __shared__ unsigned char sh[];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *extra = reinterpret_cast<float *>(sh) + warp * (32 * V);
#pragma unroll
    for (int i = 0; i < V; i++) extra[lane + 32 * i] = 0.0f;
    const float n = float(*a.live), even = float(a.k) * n / float(a.experts);
    const float f = a.grad_loss && n > 0.0f ? *a.grad_loss * float(a.experts) / (float(a.k) * n * n) : 0.0f;
    float own[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int e = L::of(i, lane);
        own[i] = e < a.experts ? f * (float(a.counts[e]) - even) : 0.0f;
    }
    __syncwarp();
    const int64_t stride = int64_t(gridDim.x) * kWarps;
    int64_t t = int64_t(blockIdx.x) * kWarps + warp;
    T raw[V];
    int id = -1;
    float w = 0.0f, u = 0.0f;
    auto fetch = [&](int64_t row) {
        if (row >= a.tokens || (a.mask && !a.mask[row])) return false;
        fetch_row<T, V, VEC>(a, static_cast<const T *>(a.logits) + row * a.row_stride, lane, raw);
        id = -1;
        w = u = 0.0f;
        if (a.grad_weights && lane < a.k) {
            id = a.ids[row * a.k + lane];
            w = a.weights[row * a.k + lane];
            u = a.grad_weights[row * a.k + lane];
            if (uint32_t(id) >= uint32_t(a.experts)) {
                id = -1;
                w = u = 0.0f;
            }
        }
        return true;
    };
    bool on = fetch(t);
    for (; t < a.tokens; t += stride) {
        float x[V], e[V], top, sum;
        const bool is_live = on && gates_of<T, V>(raw, x, e, top, sum);
        const float dot = warp_sum(w * u), term = a.normalize ? w * (u - dot) : w * u;
        const int to = id;
        on = fetch(t + stride);
        T out[V];
        if (is_live) {
            float mean = 0.0f;
#pragma unroll
            for (int i = 0; i < V; i++) mean = fmaf(e[i], own[i], mean);
            const float inv = __fdividef(1.0f, sum);
            mean = warp_sum(mean) * inv;
            if (!a.normalize) mean += dot;
            if (to >= 0) extra[to] = term;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < V; i++)
                out[i] = from_f32<T>(fmaf(e[i] * inv, own[i] - mean, extra[L::of(i, lane)]));
            __syncwarp();
            if (to >= 0) extra[to] = 0.0f;
        } else {
#pragma unroll
            for (int i = 0; i < V; i++) out[i] = from_f32<T>(0.0f);
        }
        T *row = static_cast<T *>(a.grad) + t * a.grad_stride;
#pragma unroll
        for (int i = 0; i < V; i += L::C) {
            const int e0 = L::of(i, lane);
            if (e0 >= a.experts) continue;
            if (VEC && a.vector_grad) {
                store_piece<T, L::C>(row + e0, out + i);
            } else {
#pragma unroll
                for (int c = 0; c < L::C; c++) row[e0 + c] = out[i + c];
            }
        }
    }
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

template <typename T, int V>
bool vector_rows(const RouteArgs &a) {
    constexpr int C = Place<V, true>::C;
    return V > 1 && a.col_stride == 1 && a.experts % C == 0 && a.row_stride % C == 0 &&
           aligned_to(a.logits, C * sizeof(T));
}

}  // namespace

// Launches of one element type (each in its own translation unit).
template <typename T>
int launch_route_type(const RouteArgs &a, int blocks, void *stream) {
    return with_values(a.experts, [&](auto v) {
        constexpr int V = decltype(v)::v;
        using S = RouteShape<V>;
        const size_t smem = size_t(4) * (S::kWarps * a.experts + a.experts + 1);
        const bool vec = vector_rows<T, V>(a), few = a.k <= 8;
        auto kernel = vec ? (few ? route_kernel<T, V, (V > 1), true> : route_kernel<T, V, (V > 1), false>)
                          : (few ? route_kernel<T, V, false, true> : route_kernel<T, V, false, false>);
        return launch_kernel(kernel, dim3(blocks), dim3(S::kThreads), smem, stream, a.joined ? blocks : 1,
                             "route launch", a);
    });
}

template <typename T>
int launch_route_backward_type(RouteArgs a, void *stream) {
    return with_values(a.experts, [&](auto v) {
        constexpr int V = decltype(v)::v;
        using S = RouteShape<V>;
        constexpr int C = Place<V, true>::C;
        a.vector_grad = a.grad_stride % C == 0 && aligned_to(a.grad, C * sizeof(T));
        const size_t smem = size_t(4) * S::kWarps * 32 * V;
        const int64_t b = (a.tokens + S::kWarps - 1) / S::kWarps, most = kSMs * S::kPerSm;
        auto kernel = vector_rows<T, V>(a) ? route_backward_kernel<T, V, (V > 1)> : route_backward_kernel<T, V, false>;
        return launch_kernel(kernel, dim3(unsigned(b < most ? b : most)), dim3(S::kThreads), smem, stream, 1,
                             "route backward launch", a);
    });
}

int launch_route_f32(const RouteArgs &a, int blocks, void *stream);
int launch_route_bf16(const RouteArgs &a, int blocks, void *stream);
int launch_route_f16(const RouteArgs &a, int blocks, void *stream);
int launch_route_backward_f32(const RouteArgs &a, void *stream);
int launch_route_backward_bf16(const RouteArgs &a, void *stream);
int launch_route_backward_f16(const RouteArgs &a, void *stream);

}  // namespace nest
