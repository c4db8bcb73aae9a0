// Entry points of the routing operators: checks, launch shapes and the kernel that adds up
// long rows of sums (the others are in nest_route.cuh).
#include <cooperative_groups.h>

#include "nest_route.cuh"

namespace nest {

namespace {

namespace cg = cooperative_groups;

constexpr int kAddWarps = 32, kCluster = 8;

// The results from the blocks' rows of sums and counts, by the blocks of a cluster: each takes
// groups of 32 experts.  A warp adds every 32nd row, then a warp adds an expert's 32 parts as
// a tree.
__global__ void __launch_bounds__(32 * kAddWarps) route_add_kernel(RouteArgs a, int rows) {
    __shared__ float sh_p[kAddWarps][33], sh_dot[kAddWarps], sh_all[kCluster];
    __shared__ int32_t sh_c[kAddWarps][33];
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();   // every block has started; while the rows are still being written
    pdl_wait();
    pdl_trigger();
    const int rank = int(blockIdx.x), ranks = int(gridDim.x), pitch = row_pitch(a.experts);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int n = 0;
    for (int r = lane; r < rows; r += 32) n += a.part_n[r];
    n = __reduce_add_sync(0xffffffffu, n);
    const float over = n ? 1.0f / float(n) : 0.0f;
    float dot = 0.0f;
    for (int first = 32 * rank; first < a.experts; first += 32 * ranks) {
        float p = 0.0f;
        int32_t c = 0;
        if (first + lane < a.experts) {
#pragma unroll 4
            for (int r = warp; r < rows; r += kAddWarps) {
                const float *row = a.part + int64_t(r) * 2 * pitch + first + lane;
                p += row[0];
                c += __float_as_int(row[pitch]);
            }
        }
        sh_p[warp][lane] = p;
        sh_c[warp][lane] = c;
        __syncthreads();
        p = warp_sum(sh_p[lane][warp]) * over;
        c = __reduce_add_sync(0xffffffffu, sh_c[lane][warp]);
        if (lane == 0 && first + warp < a.experts) {
            a.counts[first + warp] = c;
            a.mean_prob[first + warp] = p;
        }
        dot = fmaf(p, float(c), dot);   // 0 past the last expert
        __syncthreads();
    }
    if (lane == 0) sh_dot[warp] = dot;
    __syncthreads();
    if (warp == 0) {
        dot = warp_sum(sh_dot[lane]);
        if (lane == 0) *cluster.map_shared_rank(sh_all + rank, 0) = dot;
    }
    cluster.sync();
    if (rank == 0 && warp == 0) {
        dot = warp_sum(lane < ranks ? sh_all[lane < ranks ? lane : 0] : 0.0f);
        if (lane == 0) {
            *a.live = n;
            *a.loss = loss_of(a, dot, n);
        }
    }
}

int check(const nest_route_desc *d) {
    if (!d || d->tokens < 0 || d->row_stride < 0 || d->col_stride < 0 || !valid_type(d->dtype) || d->experts < 1 ||
        d->k < 1 || d->k > d->experts || (d->normalize & ~1))
        return NEST_E_INVALID;
    if (d->experts > 1024 || d->k > 32 || d->tokens > INT32_MAX || d->tokens * d->k > INT32_MAX) return NEST_E_LIMITS;
    return NEST_OK;
}

// The forward kernel's blocks and threads; a block alone is no larger than its rows need.
struct Grid {
    int blocks, threads;
    bool apart;   // a second kernel adds the blocks' rows
};
Grid grid_of(const nest_route_desc *d) {
    Grid g;
    with_row(d->experts, d->k, [&](auto lanes, auto values) {
        using S = RouteShape<decltype(values)::v>;
        constexpr int kPerWarp = 32 / decltype(lanes)::v, kRows = S::kWarps * kPerWarp;
        const int64_t b = (d->tokens + kRows - 1) / kRows, most = kSMs * S::kPerSm;
        const int64_t warps = (d->tokens + kPerWarp - 1) / kPerWarp;
        g.blocks = int(b < 1 ? 1 : b < most ? b : most);
        g.threads = 32 * int(warps < 1 ? 1 : warps < S::kWarps ? warps : S::kWarps);
        g.apart = g.blocks > 1 && decltype(values)::v >= kApart;
        return 0;
    });
    return g;
}

RouteArgs args_of(const nest_route_desc *d, const void *logits, const uint8_t *mask) {
    RouteArgs a = {};
    a.logits = logits;
    a.mask = mask;
    a.tokens = d->tokens;
    a.row_stride = d->row_stride;
    a.col_stride = d->col_stride;
    a.experts = d->experts;
    a.k = d->k;
    a.normalize = d->normalize;
    return a;
}

}  // namespace

}  // namespace nest

using namespace nest;

extern "C" {

size_t nest_route_workspace_size(const nest_route_desc *d) {
    if (check(d)) return 0;
    const size_t blocks = size_t(grid_of(d).blocks);
    return 256 + ((blocks > 1 ? blocks * (8 * size_t(row_pitch(d->experts)) + 4) + 255 : 0) & ~size_t(255));
}

int nest_route(const nest_route_desc *d, const void *logits, const uint8_t *mask, int32_t *ids, float *weights,
               int32_t *counts, int32_t *live, float *mean_prob, float *loss, void *workspace, size_t ws_bytes,
               void *stream) {
    if (const int rc = check(d)) return rc;
    if (!counts || !live || !mean_prob || !loss || (d->tokens && (!logits || !ids || !weights))) return NEST_E_INVALID;
    if (d->tokens && !aligned_to(logits, type_bytes(d->dtype))) return NEST_E_INVALID;
    if (!workspace || ws_bytes < nest_route_workspace_size(d) || !aligned_to(workspace, 256)) return NEST_E_WORKSPACE;
    const Grid g = grid_of(d);
    RouteArgs a = args_of(d, logits, mask);
    a.ids = ids;
    a.weights = weights;
    a.ticket = static_cast<uint32_t *>(workspace);
    a.part = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + 256);
    a.part_n = reinterpret_cast<int32_t *>(a.part + int64_t(g.blocks) * 2 * row_pitch(d->experts));
    a.counts = counts;
    a.live = live;
    a.mean_prob = mean_prob;
    a.loss = loss;
    const int rc = d->dtype == NEST_F32    ? launch_route_f32(a, g.blocks, g.threads, stream)
                   : d->dtype == NEST_BF16 ? launch_route_bf16(a, g.blocks, g.threads, stream)
                                           : launch_route_f16(a, g.blocks, g.threads, stream);
    if (rc || !g.apart) return rc;
    const int groups = (d->experts + 31) / 32, cluster = groups < kCluster ? groups : kCluster;
    return launch_kernel(route_add_kernel, dim3(cluster), dim3(32 * kAddWarps), 0, stream, cluster, "route sums launch",
                         a, g.blocks);
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
    RouteArgs a = args_of(d, logits, mask);
    a.ids = const_cast<int32_t *>(ids);
    a.weights = const_cast<float *>(weights);
    a.counts = const_cast<int32_t *>(counts);
    a.live = const_cast<int32_t *>(live);
    a.grad_weights = grad_weights;
    a.grad_loss = grad_loss;
    a.grad = grad_logits;
    a.grad_stride = grad_stride;
    return d->dtype == NEST_F32    ? launch_route_backward_f32(a, stream)
           : d->dtype == NEST_BF16 ? launch_route_backward_bf16(a, stream)
                                   : launch_route_backward_f16(a, stream);
}

}  // extern "C"
