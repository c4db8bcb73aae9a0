// Entry points of the output head's losses (nest_head.h): checks, workspace, tensor maps, and the
// kernels around the products of nest_head.cuh.
#include "nest_head.cuh"

#include <cmath>

namespace nest {
namespace head {
namespace {

constexpr int kRowThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

struct RowArgs {
    const void *hidden;
    int64_t row_stride, col_stride;
    int64_t tokens, hidden_size, packed;   // packed: elements of a compacted row
    int32_t wide;                          // rows can be read 16 bytes at a time
    const void *labels;                    // with labels
    int32_t wide_labels;
    int64_t vocab;
    const uint8_t *flags;                  // with a teacher: which tokens are live
    int32_t chunk;                         // tokens per block
    uint16_t *out;                         // [n][packed]
    int32_t *rows, *count;                 // [n], [1]
    int32_t *column;                       // [T], with labels
    uint32_t *ticket;
    // forward: of tokens that are not live
    float *losses, *lse;
    int32_t *live;
    // backward
    uint16_t *grad;                        // [T][D]
};

__device__ __forceinline__ int label_of(const RowArgs &a, int64_t t) {
    const int64_t l = a.wide_labels ? static_cast<const int64_t *>(a.labels)[t]
                                    : static_cast<const int32_t *>(a.labels)[t];
    return l >= 0 && l < a.vocab ? int(l) : -1;
}
__device__ __forceinline__ bool is_live(const RowArgs &a, int64_t t) {
    return a.flags ? a.flags[t] != 0 : label_of(a, t) >= 0;
}

// Lists the live tokens in order and copies their hidden states next to each other, so that the products
// run over live tokens alone and nothing that another token holds enters a sum.  Every block counts the
// live tokens before its own: a read of all labels, against rows of hidden states of a thousand times
// their size.
__global__ void __launch_bounds__(kRowThreads) rows_kernel(RowArgs a) {
    __shared__ int sh_sum[kRowThreads / 32], sh_before;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t first = int64_t(blockIdx.x) * a.chunk, end = min(first + a.chunk, a.tokens);
    int before = 0;
    for (int64_t t = threadIdx.x; t < first; t += kRowThreads) before += is_live(a, t);
    before = __reduce_add_sync(0xffffffffu, before);
    if (lane == 0) sh_sum[warp] = before;
    __syncthreads();
    if (threadIdx.x == 0) {
        int s = 0;
        for (int w = 0; w < kRowThreads / 32; w++) s += sh_sum[w];
        sh_before = s;
        if (blockIdx.x == 0 && a.ticket) *a.ticket = 0;
    }
    __syncthreads();
    int at = sh_before;
    const uint16_t *hidden = static_cast<const uint16_t *>(a.hidden);
    for (int64_t t0 = first; t0 < end; t0 += 32) {
        // every warp finds the same 32 tokens' places and copies every eighth of them
        const int64_t t = t0 + lane;
        const bool live = t < end && is_live(a, t);
        const uint32_t all = __ballot_sync(0xffffffffu, live);
        if (warp == 0 && t < end) {
            if (live) a.rows[at + __popc(all & ((1u << lane) - 1))] = int(t);
            if (a.column) a.column[t] = label_of(a, t);
            if (!live && a.losses) a.losses[t] = 0.0f, a.lse[t] = 0.0f;
        }
        for (int i = warp; i < 32 && t0 + i < end; i += kRowThreads / 32) {
            const int64_t source = t0 + i;
            if (all >> i & 1) {
                uint16_t *to = a.out + int64_t(at + __popc(all & ((1u << i) - 1))) * a.packed;
                const uint16_t *from = hidden + source * a.row_stride;
                if (a.wide) {
                    const int64_t units = a.hidden_size / 8;
#pragma unroll 4
                    for (int64_t u = lane; u < units; u += 32)
                        reinterpret_cast<uint4 *>(to)[u] = reinterpret_cast<const uint4 *>(from)[u];
                    for (int64_t d = units * 8 + lane; d < a.hidden_size; d += 32) to[d] = from[d];
                } else {
#pragma unroll 8
                    for (int64_t d = lane; d < a.hidden_size; d += 32) to[d] = from[d * a.col_stride];
                }
            } else if (a.grad) {
                uint16_t *to = a.grad + source * a.hidden_size;
#pragma unroll 4
                for (int64_t d = lane; d < a.hidden_size; d += 32) to[d] = 0;
            }
        }
        at += __popc(all);
    }
    if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) {
        *a.count = at;
        if (a.live) *a.live = at;
    }
}

// Rows of weights that TMA cannot read where they are, into rows that it can.
__global__ void __launch_bounds__(kRowThreads) pack_kernel(const uint16_t *from, int64_t row_stride,
                                                          int64_t col_stride, int64_t rows, int64_t cols,
                                                          uint16_t *to, int64_t pitch) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t warps = int64_t(gridDim.x) * (kRowThreads / 32);
    for (int64_t r = int64_t(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5); r < rows; r += warps) {
#pragma unroll 8
        for (int64_t d = lane; d < cols; d += 32) to[r * pitch + d] = from[r * row_stride + d * col_stride];
    }
}

struct TeacherArgs {
    const void *index, *teacher;
    const uint8_t *mask;
    int64_t tokens, vocab;
    int32_t k, wide_index;
    float over;         // 1 / h
    int32_t *ids;       // [T][k] ascending
    float *shares;      // [T][k]
    float *entropy;     // [T] sum of q log q
    uint8_t *flags;     // [T]
};

constexpr int kTeacherMost = 256, kTeacherWarps = 8;

// A warp per token: the softmax over the slots that count, and the slots in the order of their columns
// (each slot's place is the number of slots before it), so that a tile of logits finds its own by bisection.
template <typename T>
__global__ void __launch_bounds__(32 * kTeacherWarps) teacher_kernel(TeacherArgs a) {
    __shared__ int32_t sh_id[kTeacherWarps][kTeacherMost];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kPer = kTeacherMost / 32;
    for (int64_t t = int64_t(blockIdx.x) * kTeacherWarps + warp; t < a.tokens; t += int64_t(gridDim.x) * kTeacherWarps) {
        const bool open = !a.mask || a.mask[t];
        int32_t id[kPer];
        float x[kPer], top = -INFINITY;
        bool any = false;
#pragma unroll
        for (int e = 0; e < kPer; e++) {
            const int j = lane + 32 * e;
            id[e] = kNoColumn;
            x[e] = 0.0f;
            if (open && j < a.k) {
                const int64_t c = a.wide_index ? static_cast<const int64_t *>(a.index)[t * a.k + j]
                                               : static_cast<const int32_t *>(a.index)[t * a.k + j];
                const float v = to_f32(static_cast<const T *>(a.teacher)[t * a.k + j]) * a.over;
                if (c >= 0 && c < a.vocab && v != -INFINITY) {
                    id[e] = int32_t(c);
                    x[e] = v;
                    top = fmaxf(top, v);
                    any = true;
                }
            }
            if (j < a.k) sh_id[warp][j] = id[e];
        }
        __syncwarp();
        any = __any_sync(0xffffffffu, any);
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float sum = 0.0f, p[kPer];
#pragma unroll
        for (int e = 0; e < kPer; e++) {
            p[e] = id[e] != kNoColumn ? expf(x[e] - top) : 0.0f;
            sum += p[e];
        }
        sum = warp_sum(sum);
        const float over = 1.0f / sum, log_sum = logf(sum);
        float entropy = 0.0f;
#pragma unroll
        for (int e = 0; e < kPer; e++) {
            const int j = lane + 32 * e;
            if (j < a.k) {
                const bool in = id[e] != kNoColumn;
                const float q = in ? p[e] * over : 0.0f;
                if (in) entropy += q * (x[e] - top - log_sum);
                int place = 0;
                for (int i = 0; i < a.k; i++) {
                    const int32_t other = sh_id[warp][i];
                    place += other < id[e] || (other == id[e] && i < j);
                }
                a.ids[t * a.k + place] = id[e];
                a.shares[t * a.k + place] = q;
            }
        }
        entropy = warp_sum(entropy);
        if (lane == 0) {
            a.entropy[t] = any ? entropy : 0.0f;
            a.flags[t] = any;
        }
        __syncwarp();
    }
}

struct JoinArgs {
    const int32_t *count, *rows;
    const float *part_max, *part_sum, *part_hit;
    int64_t pitch;
    int32_t tiles;
    float scale;          // log2(e) / h
    float heat;           // h
    const float *entropy; // NULL with labels
    float *losses, *lse, *loss;
    float *sums;          // [blocks]
    uint32_t *ticket;
};

constexpr int kJoinRows = 32, kJoinParts = 16;

// Joins the tiles' maxima and sums: 32 rows a block, 16 threads to a row; the last block adds the rows'
// losses in the blocks' order.
__global__ void __launch_bounds__(kJoinRows *kJoinParts) join_kernel(JoinArgs a) {
    __shared__ float sh_max[kJoinParts][kJoinRows], sh_sum[kJoinParts][kJoinRows], sh_hit[kJoinParts][kJoinRows];
    __shared__ double sh_all[kJoinParts];
    __shared__ bool sh_last;
    pdl_wait();
    pdl_trigger();
    const int n = *a.count, lane = threadIdx.x & 31, part = threadIdx.x >> 5;
    const int64_t r = int64_t(blockIdx.x) * kJoinRows + lane;
    float top = -INFINITY, sum = 0.0f, hit = 0.0f;
    if (r < n) {
#pragma unroll 4
        for (int t = part; t < a.tiles; t += kJoinParts) {
            const int64_t at = int64_t(t) * a.pitch + r;
            const float high = a.part_max[at], s = a.part_sum[at];
            const float both = fmaxf(top, high);
            // a part without a finite value has sum 0 or NaN, which stays
            const float keep = top == both ? 1.0f : exp2_fast((top - both) * a.scale);
            const float take = high == both ? 1.0f : exp2_fast((high - both) * a.scale);
            sum = fmaf(s, take, sum * keep);
            hit += a.part_hit[at];
            top = both;
        }
    }
    sh_max[part][lane] = top;
    sh_sum[part][lane] = sum;
    sh_hit[part][lane] = hit;
    __syncthreads();
    if (part == 0) {
        double loss = 0.0;
        if (r < n) {
            for (int p = 1; p < kJoinParts; p++) {
                const float high = sh_max[p][lane], s = sh_sum[p][lane];
                const float both = fmaxf(top, high);
                const float keep = top == both ? 1.0f : exp2_fast((top - both) * a.scale);
                const float take = high == both ? 1.0f : exp2_fast((high - both) * a.scale);
                sum = fmaf(s, take, sum * keep);
                hit += sh_hit[p][lane];
                top = both;
            }
            const int t = a.rows[r];
            // the difference of near numbers: in 64 bits, of which there is one per row
            const double log_all = double(top) / double(a.heat) + double(logf(sum));
            const double apart = log_all - double(hit) / double(a.heat);
            const float one = float(double(a.heat) * double(a.heat) * (apart + (a.entropy ? a.entropy[t] : 0.0f)));
            a.lse[t] = float(log_all);
            a.losses[t] = one;
            loss = one;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, o);
        if (lane == 0) a.sums[blockIdx.x] = float(loss);
    }
    __syncthreads();
    if (threadIdx.x == 0) sh_last = last_ticket(a.ticket, gridDim.x);
    __syncthreads();
    if (!sh_last) return;
    double all = 0.0;
    for (int b = threadIdx.x; b < int(gridDim.x); b += kJoinRows * kJoinParts) all += __ldcg(a.sums + b);
#pragma unroll
    for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    if (lane == 0) sh_all[part] = all;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int p = 1; p < kJoinParts; p++) all += sh_all[p];
        *a.loss = n ? float(all / n) : 0.0f;
    }
}

struct ScaleArgs {
    const int32_t *count, *rows;
    const float *lse, *grad_loss, *grad_losses;
    float heat;
    float lift;           // 2^15 in half precision
    float *row_lse, *row_scale, *unit;
    uint16_t *hidden;     // the compacted rows, of which those up to a stage's end become zeros
    int64_t packed;
};

constexpr int kScaleThreads = 1024;

// The rows' factors, by block 0; the others clear the rows that the last stage of tokens reads past n.
__global__ void __launch_bounds__(kScaleThreads) scale_kernel(ScaleArgs a) {
    __shared__ float sh_top[kScaleThreads / 32];
    pdl_wait();
    pdl_trigger();
    const int n = *a.count;
    if (blockIdx.x) {
        const int64_t from = int64_t(n) * a.packed, to = int64_t((n + kDepth - 1) / kDepth * kDepth) * a.packed;
        for (int64_t i = from + int64_t(blockIdx.x - 1) * kScaleThreads + threadIdx.x; i < to;
             i += int64_t(gridDim.x - 1) * kScaleThreads)
            a.hidden[i] = 0;
        return;
    }
    const float share = a.grad_loss && n ? *a.grad_loss / float(n) : 0.0f;
    float top = 0.0f;
    if (a.grad_losses) {
        for (int r = threadIdx.x; r < n; r += kScaleThreads) {
            const float g = fabsf((share + a.grad_losses[a.rows[r]]) * a.heat);
            if (g < INFINITY) top = fmaxf(top, g);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if ((threadIdx.x & 31) == 0) sh_top[threadIdx.x >> 5] = top;
        __syncthreads();
        for (int w = 0; w < kScaleThreads / 32; w++) top = fmaxf(top, sh_top[w]);
    } else {
        const float g = fabsf(share * a.heat);
        if (g < INFINITY) top = g;
    }
    // the power of two above it: factors and results are scaled without rounding
    int e = 0;
    if (top > 0.0f) frexpf(top, &e);
    e = max(-100, min(e, 100));
    const float over = ldexpf(a.lift, -e);
    for (int r = threadIdx.x; r < n; r += kScaleThreads) {
        const int t = a.rows[r];
        a.row_scale[r] = (share + (a.grad_losses ? a.grad_losses[t] : 0.0f)) * a.heat * over;
        a.row_lse[r] = a.lse[t] * kLog2e;
    }
    if (threadIdx.x == 0) *a.unit = ldexpf(1.0f / a.lift, e);
}

int check(const nest_head_desc *d) {
    if (!d || d->tokens < 0 || d->vocab < 1 || d->hidden < 1 || d->hidden_row < 0 || d->hidden_col < 0 ||
        d->weight_row < 0 || d->weight_col < 0 || (d->dtype != NEST_BF16 && d->dtype != NEST_F16) ||
        (d->index_type != NEST_I32 && d->index_type != NEST_I64) || d->k < 0 || d->reserved)
        return NEST_E_INVALID;
    if (d->k ? !valid_type(d->teacher_type) || !(d->temperature >= 0.0009765625f && d->temperature <= 1024.0f)
             : d->temperature != 1.0f)
        return NEST_E_INVALID;
    if (d->tokens > 1 << 24 || d->vocab > 1 << 24 || d->hidden > 1 << 16 || d->k > kTeacherMost) return NEST_E_LIMITS;
    return NEST_OK;
}

// Whether TMA reads the weights where they are.
bool in_place(const nest_head_desc *d, const void *weight) {
    return (d->weight_col == 1 || d->hidden == 1) && d->weight_row % 8 == 0 && d->weight_row >= d->hidden &&
           aligned_to(weight, 16);
}

struct Layout {
    int64_t packed;   // elements of a compacted row of hidden states or weights
    int64_t pitch;    // tokens, rounded up
    int64_t piece;    // columns of the vocabulary at a time (backward)
    int32_t tiles;    // column tiles (forward)
    int32_t join;     // blocks of the join
    size_t count, ticket, unit, rows, column, shares, entropy, flags, hidden, weight, part, sums, row, dz, total;
};

// Pieces of the vocabulary: dz of a piece takes up to 256 MiB, or 8192 columns where that is more (the sums
// of the hidden states' gradient are read and written once per piece, 8 bytes for every 2 * 8192 multiply-adds).
int64_t piece_of(int64_t pitch, int64_t vocab) {
    int64_t p = (int64_t(1) << 27) / pitch / kTile * kTile;
    if (p < 8192) p = 8192;
    const int64_t all = align_up(vocab, kTile);
    if (p >= all) return all;
    const int64_t pieces = (all + p - 1) / p;
    return align_up((all + pieces - 1) / pieces, kTile);
}

Layout layout_of(const nest_head_desc *d, const void *weight, bool backward) {
    Layout l = {};
    l.packed = align_up(d->hidden, 8);
    l.pitch = align_up(d->tokens > 0 ? d->tokens : 1, kTile);
    l.piece = piece_of(l.pitch, d->vocab);
    l.tiles = int32_t((d->vocab + kTile - 1) / kTile);
    l.join = d->tokens ? int32_t((d->tokens + kJoinRows - 1) / kJoinRows) : 1;
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t here = at;
        at += size_t(align_up(bytes, 256));
        return here;
    };
    l.count = take(4);
    l.ticket = take(4);
    l.unit = take(4);
    l.rows = take(4 * d->tokens);
    const int64_t slots = d->tokens * (d->k ? d->k : 1);
    l.column = take(4 * slots);
    if (d->k) {
        l.shares = take(4 * slots);
        l.entropy = take(4 * d->tokens);
        l.flags = take(d->tokens);
    }
    l.hidden = take(2 * l.pitch * l.packed);
    if (!in_place(d, weight)) l.weight = take(2 * d->vocab * l.packed);
    if (!backward) {
        l.part = take(3 * 4 * int64_t(l.tiles) * l.pitch);
        l.sums = take(4 * l.join);
    } else {
        l.row = take(2 * 4 * l.pitch);
        l.dz = take(2 * l.pitch * l.piece);
        if (l.piece < d->vocab) l.sums = take(4 * l.pitch * d->hidden);
    }
    l.total = at;
    return l;
}

using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                            const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                            CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

int encoder(Encode *out) {
    static std::atomic<Encode> known{nullptr};
    Encode f = known.load(std::memory_order_acquire);
    if (!f) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (const int rc = cuda_status(
                cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found),
                "tensor map entry point"))
            return rc;
        if (found != cudaDriverEntryPointSuccess || !p) return NEST_E_CUDA;
        f = reinterpret_cast<Encode>(p);
        known.store(f, std::memory_order_release);
    }
    *out = f;
    return NEST_OK;
}

// Rows of 16-bit numbers, read in boxes of 64 of a row by `high` rows; what lies past the ends reads as 0.
int encode(CUtensorMap *map, int32_t dtype, const void *base, int64_t cols, int64_t rows, int64_t pitch, int high) {
    Encode f;
    if (const int rc = encoder(&f)) return rc;
    const cuuint64_t sizes[2] = {cuuint64_t(cols), cuuint64_t(rows)}, strides[1] = {cuuint64_t(pitch) * 2};
    const cuuint32_t box[2] = {64, cuuint32_t(high)}, steps[2] = {1, 1};
    const CUresult r =
        f(map, dtype == NEST_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
          const_cast<void *>(base), sizes, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? NEST_OK : NEST_E_CUDA;
}

// One call: what both directions do before their products.
struct Call {
    const nest_head_desc *d;
    Layout l;
    unsigned char *ws;
    void *stream;
    const void *weight;    // as TMA reads it
    int64_t weight_pitch;

    template <typename T> T *at(size_t offset) const { return reinterpret_cast<T *>(ws + offset); }

    int start(const void *hidden, const void *w, const void *index, const void *teacher, const uint8_t *mask,
              float *losses, float *lse, int32_t *live, void *grad) {
        if (d->k) {
            TeacherArgs t = {};
            t.index = index;
            t.teacher = teacher;
            t.mask = mask;
            t.tokens = d->tokens;
            t.vocab = d->vocab;
            t.k = d->k;
            t.wide_index = d->index_type == NEST_I64;
            t.over = 1.0f / d->temperature;
            t.ids = at<int32_t>(l.column);
            t.shares = at<float>(l.shares);
            t.entropy = at<float>(l.entropy);
            t.flags = at<uint8_t>(l.flags);
            const int64_t blocks = (d->tokens + kTeacherWarps - 1) / kTeacherWarps;
            if (blocks) {
                const int rc = with_type(d->teacher_type, [&](auto type) {
                    return launch_kernel(teacher_kernel<decltype(type)>,
                                         dim3(unsigned(blocks < 8 * kSMs ? blocks : 8 * kSMs)), dim3(32 * kTeacherWarps),
                                         0, stream, 1, "teacher launch", t);
                });
                if (rc) return rc;
            }
        }
        RowArgs r = {};
        r.hidden = hidden;
        r.row_stride = d->hidden_row;
        r.col_stride = d->hidden_col;
        r.tokens = d->tokens;
        r.hidden_size = d->hidden;
        r.packed = l.packed;
        r.wide = (d->hidden_col == 1 || d->hidden == 1) && d->hidden_row % 8 == 0 && aligned_to(hidden, 16);
        r.labels = index;
        r.wide_labels = d->index_type == NEST_I64;
        r.vocab = d->vocab;
        r.flags = d->k ? at<uint8_t>(l.flags) : nullptr;
        r.out = at<uint16_t>(l.hidden);
        r.rows = at<int32_t>(l.rows);
        r.count = at<int32_t>(l.count);
        r.column = d->k ? nullptr : at<int32_t>(l.column);
        r.ticket = live ? at<uint32_t>(l.ticket) : nullptr;
        r.losses = losses;
        r.lse = lse;
        r.live = live;
        r.grad = static_cast<uint16_t *>(grad);
        const int64_t chunk = align_up((d->tokens + 511) / 512, 32);
        r.chunk = int32_t(chunk < 32 ? 32 : chunk);
        const int64_t blocks = (d->tokens + r.chunk - 1) / r.chunk;
        if (const int rc = launch_kernel(rows_kernel, dim3(unsigned(blocks ? blocks : 1)), dim3(kRowThreads), 0, stream,
                                         1, "head rows launch", r))
            return rc;
        weight = w;
        weight_pitch = d->weight_row;
        if (!in_place(d, w)) {
            weight = ws + l.weight;
            weight_pitch = l.packed;
            const int64_t most = (d->vocab + kRowThreads / 32 - 1) / (kRowThreads / 32);
            if (const int rc = launch_kernel(pack_kernel, dim3(unsigned(most < 8 * kSMs ? most : 8 * kSMs)),
                                             dim3(kRowThreads), 0, stream, 1, "head weights launch",
                                             static_cast<const uint16_t *>(w), d->weight_row, d->weight_col, d->vocab,
                                             d->hidden, at<uint16_t>(l.weight), l.packed))
                return rc;
        }
        return NEST_OK;
    }

    GemmArgs products() const {
        GemmArgs g = {};
        g.live = at<int32_t>(l.count);
        g.rows = at<int32_t>(l.rows);
        g.pitch = l.pitch;
        g.ids = at<int32_t>(l.column);
        g.shares = d->k ? at<float>(l.shares) : nullptr;
        g.k = d->k ? d->k : 1;
        g.scale = kLog2e / d->temperature;
        return g;
    }

    // `rows`: at most
    int multiply(Product p, const CUtensorMap &a, const CUtensorMap &b, const GemmArgs &g, int64_t rows) const {
        const int64_t tiles = (rows + kTile - 1) / kTile * ((g.cols + kTile - 1) / kTile);
        const int pairs = int(tiles < kSMs / 2 ? tiles : kSMs / 2);
        return d->dtype == NEST_BF16 ? launch_gemm_bf16(p, a, b, g, pairs, stream)
                                     : launch_gemm_f16(p, a, b, g, pairs, stream);
    }
};

int check_inputs(const nest_head_desc *d, const void *hidden, const void *weight, const void *index,
                 const void *teacher, const uint8_t *mask) {
    if (!weight || !aligned_to(weight, 2)) return NEST_E_INVALID;
    if (!d->k && (teacher || mask)) return NEST_E_INVALID;
    if (!d->tokens) return NEST_OK;
    if (!hidden || !aligned_to(hidden, 2) || !index || !aligned_to(index, d->index_type == NEST_I64 ? 8 : 4))
        return NEST_E_INVALID;
    if (d->k && (!teacher || !aligned_to(teacher, type_bytes(d->teacher_type)))) return NEST_E_INVALID;
    return NEST_OK;
}

}  // namespace
}  // namespace head
}  // namespace nest

using namespace nest;
using namespace nest::head;

extern "C" {

size_t nest_head_loss_workspace_size(const nest_head_desc *d, const void *weight) {
    return check(d) ? 0 : layout_of(d, weight, false).total;
}

size_t nest_head_backward_workspace_size(const nest_head_desc *d, const void *weight) {
    return check(d) ? 0 : layout_of(d, weight, true).total;
}

int nest_head_loss(const nest_head_desc *d, const void *hidden, const void *weight, const void *index,
                   const void *teacher, const uint8_t *mask, float *loss, float *losses, float *lse, int32_t *live,
                   void *workspace, size_t ws_bytes, void *stream) {
    if (const int rc = check(d)) return rc;
    if (const int rc = check_inputs(d, hidden, weight, index, teacher, mask)) return rc;
    if (!loss || !live || (d->tokens && (!losses || !lse))) return NEST_E_INVALID;
    Call c = {d, layout_of(d, weight, false), static_cast<unsigned char *>(workspace), stream};
    if (!workspace || ws_bytes < c.l.total || !aligned_to(workspace, 256)) return NEST_E_WORKSPACE;
    if (const int rc = c.start(hidden, weight, index, teacher, mask, losses, lse, live, nullptr)) return rc;
    GemmArgs g = c.products();
    g.cols = int32_t(d->vocab);
    g.depth = int32_t(d->hidden);
    const int64_t part = int64_t(c.l.tiles) * c.l.pitch;
    g.part_max = c.at<float>(c.l.part);
    g.part_sum = g.part_max + part;
    g.part_hit = g.part_sum + part;
    if (d->tokens) {
        CUtensorMap a, b;
        if (const int rc = encode(&a, d->dtype, c.at<void>(c.l.hidden), d->hidden, c.l.pitch, c.l.packed, kHalf))
            return rc;
        if (const int rc = encode(&b, d->dtype, c.weight, d->hidden, d->vocab, c.weight_pitch, kHalf)) return rc;
        if (const int rc = c.multiply(kLoss, a, b, g, d->tokens)) return rc;
    }
    JoinArgs j = {};
    j.count = g.live;
    j.rows = g.rows;
    j.part_max = g.part_max;
    j.part_sum = g.part_sum;
    j.part_hit = g.part_hit;
    j.pitch = c.l.pitch;
    j.tiles = c.l.tiles;
    j.scale = g.scale;
    j.heat = d->temperature;
    j.entropy = d->k ? c.at<float>(c.l.entropy) : nullptr;
    j.losses = losses;
    j.lse = lse;
    j.loss = loss;
    j.sums = c.at<float>(c.l.sums);
    j.ticket = c.at<uint32_t>(c.l.ticket);
    return launch_kernel(join_kernel, dim3(unsigned(c.l.join)), dim3(kJoinRows * kJoinParts), 0, stream, 1,
                         "head join launch", j);
}

int nest_head_loss_backward(const nest_head_desc *d, const void *hidden, const void *weight, const void *index,
                            const void *teacher, const uint8_t *mask, const float *lse, const float *grad_loss,
                            const float *grad_losses, void *grad_hidden, void *grad_weight, void *workspace,
                            size_t ws_bytes, void *stream) {
    if (const int rc = check(d)) return rc;
    if (const int rc = check_inputs(d, hidden, weight, index, teacher, mask)) return rc;
    if (!grad_weight || !aligned_to(grad_weight, 2) ||
        (d->tokens && (!lse || !grad_hidden || !aligned_to(grad_hidden, 2))))
        return NEST_E_INVALID;
    Call c = {d, layout_of(d, weight, true), static_cast<unsigned char *>(workspace), stream};
    const Layout &l = c.l;
    if (!workspace || ws_bytes < l.total || !aligned_to(workspace, 256)) return NEST_E_WORKSPACE;
    if (const int rc = c.start(hidden, weight, index, teacher, mask, nullptr, nullptr, nullptr, grad_hidden)) return rc;
    ScaleArgs s = {};
    s.count = c.at<int32_t>(l.count);
    s.rows = c.at<int32_t>(l.rows);
    s.lse = lse;
    s.grad_loss = grad_loss;
    s.grad_losses = grad_losses;
    s.heat = d->temperature;
    s.lift = d->dtype == NEST_F16 ? 32768.0f : 1.0f;
    s.row_lse = c.at<float>(l.row);
    s.row_scale = s.row_lse + l.pitch;
    s.unit = c.at<float>(l.unit);
    s.hidden = c.at<uint16_t>(l.hidden);
    s.packed = l.packed;
    if (const int rc = launch_kernel(scale_kernel, dim3(33), dim3(kScaleThreads), 0, stream, 1, "head scale launch", s))
        return rc;

    CUtensorMap hidden_rows, weight_rows, dz_rows, weight_cols, dz_cols, hidden_cols;
    void *h = c.at<void>(l.hidden), *dz = c.at<void>(l.dz);
    int rc = encode(&hidden_rows, d->dtype, h, d->hidden, l.pitch, l.packed, kHalf);
    if (!rc) rc = encode(&weight_rows, d->dtype, c.weight, d->hidden, d->vocab, c.weight_pitch, kHalf);
    if (!rc) rc = encode(&dz_rows, d->dtype, dz, l.piece, l.pitch, l.piece, kHalf);
    if (!rc) rc = encode(&weight_cols, d->dtype, c.weight, d->hidden, d->vocab, c.weight_pitch, kDepth);
    if (!rc) rc = encode(&dz_cols, d->dtype, dz, l.piece, l.pitch, l.piece, kDepth);
    if (!rc) rc = encode(&hidden_cols, d->dtype, h, d->hidden, l.pitch, l.packed, kDepth);
    if (rc) return rc;

    GemmArgs g = c.products();
    g.row_lse = s.row_lse;
    g.row_scale = s.row_scale;
    g.unit = s.unit;
    for (int64_t first = 0; first < d->vocab; first += l.piece) {
        const int64_t cols = d->vocab - first < l.piece ? d->vocab - first : l.piece;
        GemmArgs p = g;
        p.first_col = int32_t(first);
        if (d->tokens) {
            p.cols = int32_t(cols);
            p.depth = int32_t(d->hidden);
            p.out = dz;
            p.out_pitch = l.piece;
            p.wide = 1;
            if (const int e = c.multiply(kDz, hidden_rows, weight_rows, p, d->tokens)) return e;
            p.cols = int32_t(d->hidden);
            p.depth = int32_t(cols);
            p.out = grad_hidden;
            p.out_pitch = d->hidden;
            p.wide = d->hidden % 8 == 0 && aligned_to(grad_hidden, 16);
            p.sums = c.at<float>(l.sums);
            p.first = first == 0;
            p.last = first + l.piece >= d->vocab;
            if (const int e = c.multiply(kGradHidden, dz_rows, weight_cols, p, d->tokens)) return e;
        }
        p.m = int32_t(cols);
        p.cols = int32_t(d->hidden);
        p.out = static_cast<uint16_t *>(grad_weight) + first * d->hidden;
        p.out_pitch = d->hidden;
        p.wide = d->hidden % 8 == 0 && aligned_to(grad_weight, 16);
        if (const int e = c.multiply(kGradWeight, dz_cols, hidden_cols, p, cols)) return e;
    }
    return NEST_OK;
}

}  // extern "C"
