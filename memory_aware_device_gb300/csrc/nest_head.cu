// Entry points of the output head's losses (nest_head.h): checks, workspace, tensor maps, and the
// kernels around the products of nest_head.cuh.
#include "nest_head.cuh"

#include <cmath>

namespace nest {
namespace head {
namespace {

constexpr int kRowThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

// Rows of 16-bit numbers that are copied to 16-byte aligned rows.
struct Rows {
    const uint16_t *from;
    int64_t row_stride, col_stride, width;
    uint16_t *to;
    int64_t pitch;      // elements
};

struct RowArgs {
    Rows hidden;
    int64_t tokens;
    const void *labels;                    // with labels
    int32_t wide_labels;
    int64_t vocab;
    const uint8_t *flags;                  // with a teacher: which tokens are live
    int32_t chunk, blocks;                 // tokens per block; the blocks after these copy weights
    int32_t *rows, *count;                 // [n], [1]
    int32_t *row_labels;                   // [n], with labels
    uint32_t *ticket;
    Rows weight;                           // to copy, or width 0
    // forward: of tokens that are not live
    float *losses, *lse;
    int32_t *live;
    // backward
    int32_t clear;                         // the rows behind the last
    uint16_t *grad;                        // [T][D], or NULL
    int32_t wide_grad;
    const float *lse_in;
    float *row_lse;                        // [n] lse log2(e)
    const float *grad_losses;
    float *row_grad;                       // [n]
    float *parts;                          // [blocks] the largest finite |grad_losses| of live tokens
};

__device__ __forceinline__ int label_of(const RowArgs &a, int64_t t) {
    const int64_t l = a.wide_labels ? static_cast<const int64_t *>(a.labels)[t]
                                    : static_cast<const int32_t *>(a.labels)[t];
    return l >= 0 && l < a.vocab ? int(l) : -1;
}
__device__ __forceinline__ bool is_live(const RowArgs &a, int64_t t) {
    return a.flags ? a.flags[t] != 0 : label_of(a, t) >= 0;
}

constexpr int kSegment = 1024;   // numbers of a row that a warp copies at a time: four loads of 16 bytes per lane

// Numbers [begin, begin + kSegment) of a row by a warp.  Rows off alignment are read from the aligned addresses
// around them and shifted: 16 bytes per lane whatever the offset.  (No 16 bytes are read of which the row has
// none.)
__device__ __forceinline__ void copy_segment(const Rows &x, int64_t source, int64_t target, int begin, int lane) {
    const uint16_t *from = x.from + source * x.row_stride;
    uint16_t *to = x.to + target * x.pitch;
    const int width = int(x.width), end = min(begin + kSegment, width);
    if (x.col_stride != 1 && width != 1) {
#pragma unroll 8
        for (int d = begin + lane; d < end; d += 32) to[d] = from[d * x.col_stride];
        return;
    }
    const uint32_t shift = uint32_t(reinterpret_cast<uintptr_t>(from)) & 15;
    const uint4 *base = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(from) - shift);
    const int last = (int(shift) + 2 * width - 1) >> 4;   // the last aligned address
    uint4 *out = reinterpret_cast<uint4 *>(to);
    const int u0 = begin / 8 + lane, units = (end + 7) / 8;
    constexpr int kPer = kSegment / 8 / 32;
    if (!shift) {
        uint4 v[kPer];
#pragma unroll
        for (int i = 0; i < kPer; i++)
            if (u0 + 32 * i < units) v[i] = base[u0 + 32 * i];
#pragma unroll
        for (int i = 0; i < kPer; i++)
            if (u0 + 32 * i < units) out[u0 + 32 * i] = v[i];
        return;
    }
    const bool two = shift & 8, one = shift & 4, part = shift & 2;
    uint4 p[kPer], q[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const int u = u0 + 32 * i;
        p[i] = u < units ? base[u] : make_uint4(0, 0, 0, 0);
        q[i] = u < units && u < last ? base[u + 1] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        uint32_t w[8] = {p[i].x, p[i].y, p[i].z, p[i].w, q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
        for (int e = 0; e < 6; e++) w[e] = two ? w[e + 2] : w[e];
#pragma unroll
        for (int e = 0; e < 5; e++) w[e] = one ? w[e + 1] : w[e];
#pragma unroll
        for (int e = 0; e < 4; e++) w[e] = part ? __funnelshift_r(w[e], w[e + 1], 16) : w[e];
        if (u0 + 32 * i < units) out[u0 + 32 * i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

__device__ __forceinline__ void clear_row(uint16_t *to, int64_t width, bool wide, int lane) {
    if (wide) {
        for (int64_t u = lane; u < width / 8; u += 32) reinterpret_cast<uint4 *>(to)[u] = make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll 4
        for (int64_t d = lane; d < width; d += 32) to[d] = 0;
    }
}

// Lists the live tokens in order and copies their hidden states next to each other, so that the products
// run over live tokens alone and nothing that another token holds enters a sum; behind them it clears the rows
// that the last stage of tokens reads.  Every block counts the live tokens before its own and in all: a read
// of all labels, against rows of hidden states of a thousand times their size.  Blocks past `blocks` copy
// weights that TMA cannot read where they are.
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const __grid_constant__ RowArgs a) {
    constexpr int kWarps = kRowThreads / 32;
    __shared__ int sh_before[kWarps], sh_all[kWarps];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, block = int(blockIdx.x);
    if (block >= a.blocks) {
        const int64_t warps = int64_t(gridDim.x - a.blocks) * kWarps;
        for (int64_t r = int64_t(block - a.blocks) * kWarps + warp; r < a.vocab; r += warps)
            for (int c = 0; c < a.weight.width; c += kSegment) copy_segment(a.weight, r, r, c, lane);
        return;
    }
    const int64_t first = int64_t(block) * a.chunk, end = min(first + a.chunk, a.tokens);
    int before = 0, all = 0;
    for (int64_t t = threadIdx.x; t < a.tokens; t += kRowThreads) {
        const int live = is_live(a, t);
        all += live;
        before += t < first ? live : 0;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    all = __reduce_add_sync(0xffffffffu, all);
    if (lane == 0) sh_before[warp] = before, sh_all[warp] = all;
    __syncthreads();
    before = all = 0;
    for (int w = 0; w < kWarps; w++) before += sh_before[w], all += sh_all[w];
    if (block == 0 && threadIdx.x == 0) {
        *a.count = all;
        if (a.live) *a.live = all;
        if (a.ticket) *a.ticket = 0;
    }
    // rows from the last token to the end of its stage, which the weights' gradient reads
    for (int64_t r = all + block * kWarps + warp; a.clear && r < (all + kDepth - 1) / kDepth * kDepth; r += a.blocks * kWarps)
        clear_row(a.hidden.to + r * a.hidden.pitch, a.hidden.pitch, true, lane);
    float top = 0.0f;
    int at = before;
    for (int64_t t0 = first; t0 < end; t0 += 32) {
        // every warp finds the same 32 tokens' places; their rows' segments go to the warps in turn
        const int64_t t = t0 + lane;
        const bool live = t < end && is_live(a, t);
        const uint32_t set = __ballot_sync(0xffffffffu, live);
        if (warp == 0 && t < end) {
            const int place = at + __popc(set & ((1u << lane) - 1));
            if (live) a.rows[place] = int(t);
            if (live && a.row_labels) a.row_labels[place] = label_of(a, t);
            if (live && a.row_lse) a.row_lse[place] = a.lse_in[t] * kLog2e;
            if (!live && a.losses) a.losses[t] = 0.0f, a.lse[t] = 0.0f;
            if (live && a.grad_losses) {
                const float g = a.grad_losses[t];
                a.row_grad[place] = g;
                if (fabsf(g) < INFINITY) top = fmaxf(top, fabsf(g));
            }
        }
        const int segments = (int(a.hidden.width) + kSegment - 1) / kSegment, here = int(min(int64_t(32), end - t0));
        for (int i = warp; i < here * segments; i += kWarps) {
            const int row = i / segments, c = (i - row * segments) * kSegment;
            if (set >> row & 1)
                copy_segment(a.hidden, t0 + row, at + __popc(set & ((1u << row) - 1)), c, lane);
            else if (a.grad)
                clear_row(a.grad + (t0 + row) * a.hidden.width + c, min(int64_t(kSegment), a.hidden.width - c), a.wide_grad,
                          lane);
        }
        at += __popc(set);
    }
    if (a.parts && warp == 0) {
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) a.parts[block] = top;
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
// The temperature divides differences from the largest logit: the logits' own quotients may be beyond 32 bits.
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
                const float v = to_f32(static_cast<const T *>(a.teacher)[t * a.k + j]);
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
            x[e] = (x[e] - top) * a.over;
            p[e] = id[e] != kNoColumn ? expf(x[e]) : 0.0f;
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
                if (in && q != 0.0f) entropy += q * (x[e] - log_sum);   // q log q is 0 in the limit
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

constexpr int kJoinParts = 16;

// The join where one block has too many tokens for it: 32 rows a block, 16 threads to a row; the last block adds the
// rows' losses in the blocks' order.
__global__ void __launch_bounds__(kJoinRows *kJoinParts) join_kernel(const __grid_constant__ JoinArgs a) {
    __shared__ JoinShared<kJoinParts> sh;
    __shared__ bool sh_last;
    pdl_wait();
    pdl_trigger();
    const int n = *a.count, lane = threadIdx.x & 31, part = threadIdx.x >> 5;
    const float loss = join_rows<kJoinParts>(a, int64_t(blockIdx.x) * kJoinRows, n, part, lane, sh,
                                             [] { __syncthreads(); });
    if (threadIdx.x == 0) {
        a.sums[blockIdx.x] = loss;
        sh_last = gridDim.x == 1 || last_ticket(a.ticket, gridDim.x);
    }
    __syncthreads();
    if (!sh_last) return;
    // a thread's sum may be of a thousand blocks: what each addition cuts off is added up beside it
    float all = 0.0f, cut = 0.0f;
    for (int b = threadIdx.x; b < int(gridDim.x); b += kJoinRows * kJoinParts) {
        const float v = __ldcg(a.sums + b), next = all + v, back = next - all;
        cut += (all - (next - back)) + (v - back);
        all = next;
    }
    all = fabsf(all) < INFINITY ? all + cut : all;
    all = warp_sum(all);
    if (lane == 0) sh.all[part] = all;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kJoinParts; w++) all += sh.all[w];
        *a.loss = n ? all / float(n) : 0.0f;
    }
}

struct SumArgs {
    const int32_t *live, *rows;
    int32_t piece_rows;         // of grad weight; grad hidden has n
    int32_t cols;               // D
    int32_t splits[2];
    const float *sums[2];       // NULL: nothing to do
    int64_t pitch[2];
    uint16_t *out[2];
    int32_t first_block;        // of grad weight
    Scale by;
};

constexpr int kSumTile = 64, kSumCols = 16;

// Adds the parts of results whose summed index was split, in order, and rounds them: tiles of 64 rows x 16, turned
// from columns to rows in shared memory.  The parts are read before the number of rows is known (the buffers
// have whole tiles of rows).
template <typename T>
__global__ void __launch_bounds__(256) sum_kernel(const __grid_constant__ SumArgs a) {
    __shared__ float tile[kSumTile][kSumCols + 1];
    pdl_wait();
    pdl_trigger();
    const int kind = int(blockIdx.x) >= a.first_block, across = (a.cols + kSumCols - 1) / kSumCols;
    const int at = int(blockIdx.x) - (kind ? a.first_block : 0);
    const int r0 = at / across * kSumTile, c0 = at % across * kSumCols;
    const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
    const float *from = a.sums[kind] + int64_t(c0 + y) * a.pitch[kind] + r0 + x;
    const int64_t part = int64_t(a.cols) * a.pitch[kind];
    constexpr int kPer = kSumCols / 4;
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++) v[i] = 0.0f;
#pragma unroll 4
    for (int s = 0; s < a.splits[kind]; s++) {
#pragma unroll
        for (int i = 0; i < kPer; i++)
            if (c0 + y + 4 * i < a.cols) v[i] += from[s * part + int64_t(4 * i) * a.pitch[kind]];
    }
    const int n = *a.live, rows = kind ? a.piece_rows : n;
    if (r0 >= rows) return;
    const float unit = scaling_of(a.by, n).unit;
#pragma unroll
    for (int i = 0; i < kPer; i++) tile[x][y + 4 * i] = v[i] * unit;
    __syncthreads();
    const int c = threadIdx.x & (kSumCols - 1);
    for (int r = threadIdx.x / kSumCols; r < kSumTile && r0 + r < rows; r += 256 / kSumCols) {
        if (c0 + c < a.cols) {
            const int64_t row = kind ? r0 + r : a.rows[r0 + r];
            const T z = from_f32<T>(tile[r][c]);
            a.out[kind][row * a.cols + c0 + c] = reinterpret_cast<const uint16_t &>(z);
        }
    }
}

int check(const nest_head_desc *d) {
    if (!d || d->tokens < 0 || d->vocab < 1 || d->hidden < 1 || d->hidden_row < 0 || d->hidden_col < 0 ||
        d->weight_row < 0 || d->weight_col < 0 || (d->dtype != NEST_BF16 && d->dtype != NEST_F16) ||
        (d->index_type != NEST_I32 && d->index_type != NEST_I64) || d->k < 0 || d->reserved)
        return NEST_E_INVALID;
    if (d->k ? !valid_type(d->teacher_type) || !(d->temperature >= 0.0009765625f && d->temperature <= 1024.0f)
             : d->temperature != 1.0f)
        return NEST_E_INVALID;
    // the last: tiles of logits are counted in 32 bits
    if (d->tokens > 1 << 24 || d->vocab > 1 << 24 || d->hidden > 1 << 16 || d->k > kTeacherMost ||
        cdiv(d->tokens, kTile) * cdiv(d->vocab, kHalf) > 1 << 30)
        return NEST_E_LIMITS;
    return NEST_OK;
}

// Whether TMA reads the weights where they are.
bool in_place(const nest_head_desc *d, const void *weight) {
    return (d->weight_col == 1 || d->hidden == 1) && d->weight_row % 8 == 0 && d->weight_row >= d->hidden &&
           d->weight_row < int64_t(1) << 38 && aligned_to(weight, 16);
}

constexpr int kPairs = kSMs / 2;

// Stages in whose time a tile of gradients is written: with 4, 5, 7 and 10 those of 64 x 100000 x 1024 take 79, 86, 96
// and 105 us, of 1 x 32000 x 4096 97, 95, 108 and 117 (with 3: 89 and 111).  Rows off alignment take longer: of 64 x 100000 x 1023 161 us with 10 and 144 with 16.
int least_of(int64_t hidden) { return hidden % 8 == 0 ? 4 : 16; }

// Parts of the summed index of the two gradients: one, unless there are fewer tiles than pairs of blocks or one
// product's tiles are longer than an even share of all work.  A part is at least 24 stages: writing and reading
// its 256 KB of sums takes as long (1000 x 5000 x 300: 21.0 us with both kernels, 23.0 with 16).  And at most 2048
// (131072 tokens or columns): what the tensor cores' additions cut off, 0.26 to 0.46 * 2^-24 of the sum per 16 products
// in the mean (over_heat), is then up to 2.3e-4 of it, below the half step of 2^-11 or 2^-8 to which it is rounded.
void split(int64_t tokens, int64_t cols, int64_t hidden, int width, bool pieces, int32_t (&splits)[2]) {
    constexpr int64_t kPart = 24, kLongest = 2048;
    const int64_t across = cdiv(hidden, width), row_tiles[2] = {cdiv(tokens, kTile), cdiv(cols, kTile)};
    const int64_t steps[2] = {cdiv(cols, kDepth), cdiv(tokens, kDepth)}, least = least_of(hidden);
    int64_t share = 0;
    for (int i = 0; i < 2; i++) share += row_tiles[i] * across * (steps[i] > least ? steps[i] : least);
    share = cdiv(share, kPairs);
    if (share < kPart) share = kPart;
    for (int i = 0; i < 2; i++) {
        // with pieces the weights' sums are added up once per piece: no more parts than their length asks for
        const int64_t part = share < kLongest && !(pieces && i == 1) ? share : kLongest, most = cdiv(steps[i], part);
        splits[i] = int32_t(most < 1 ? 1 : most);
    }
}

// Columns of a tile of logits: the multiple of `step` for which the rounds of all pairs take least, counting 900
// columns of one stage for what a tile costs besides (0.7 to 1.5 us).  2048 x 32000 x 4096: 18 rounds of 192
// take 267 us, 14 of 256 273; 300 x 32000 x 4096: 4 of 224 71, 4 of 256 79; 2048 x 32000 x 256: 256 29, 128 38.
int width_of(int64_t tokens, int64_t cols, int64_t hidden, int step) {
    int best = kTile;
    int64_t least = INT64_MAX;
    for (int w = kTile; w >= 128; w -= step) {
        const int64_t time = cdiv(cdiv(tokens, kTile) * cdiv(cols, w), kPairs) * (w * cdiv(hidden, kDepth) + 900);
        if (time < least) least = time, best = w;
    }
    return best;
}

// 1 / h for logits as the tensor cores sum them.  Each step of 16 products cuts a sum in 32 bits off towards zero, which
// takes 0.26 * 2^-24 of a sum like a model's logits (products of either sign, 64 to 16384 terms) per step in the
// mean, in half precision 0.30 (measured), and is given back: the root of the mean square of the error falls from 3.0e-5
// to 5.6e-6 for logits of 7 over 4096 terms in bfloat16, that of the losses of 2048 x 32000 x 4096 from 1.2e-6
// to 1.3e-7 of them (32-bit products: 1.2e-7).  Products of one sign lose more (0.46 over 1024 terms), and a sum that
// loses nothing is off by the factor, 4e-6 of itself over 4096 terms: as far as the others are without it.
float over_heat(const nest_head_desc *d) {
    const double per = d->dtype == NEST_F16 ? 0.30 : 0.26;
    return float((1.0 + per * double(cdiv(d->hidden, 16)) / 16777216.0) / double(d->temperature));
}

struct Layout {
    int64_t packed;   // elements of a compacted row of hidden states or weights
    int64_t pitch;    // tokens, rounded up
    int64_t piece;    // columns of the vocabulary at a time (backward)
    int32_t width;    // of the tiles of logits
    int32_t grad_width;   // of the gradients' tiles
    int32_t tiles;    // column tiles (forward)
    int32_t join;     // blocks of the join
    int32_t chunk, row_blocks;   // of the list of live tokens
    int32_t splits[2];
    int64_t sums_pitch[2];
    size_t count, ticket, rows, column, shares, entropy, flags, hidden, weight, part, sums, parts, dz, row_lse, row_grad,
        grad_sums[2], total;
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
    l.packed = align_up(d->hidden, 16);   // rows of whole 32-byte sectors
    l.pitch = align_up(d->tokens > 0 ? d->tokens : 1, kTile);
    l.piece = piece_of(l.pitch, d->vocab);
    // dz is written in boxes of 64 columns
    l.width = backward ? width_of(d->tokens, l.piece, d->hidden, 64) : width_of(d->tokens, d->vocab, d->hidden, 32);
    // 2048 x 32000 x 128: 48 us in tiles of 128 columns, 53 in 256; x 640: 114 and 106
    l.grad_width = d->hidden > kHalf ? kTile : kHalf;
    l.tiles = int32_t(cdiv(d->vocab, l.width));
    l.join = d->tokens ? int32_t(cdiv(d->tokens, kJoinRows)) : 1;
    l.chunk = d->tokens > kMostRowBlocks ? int32_t(cdiv(d->tokens, kMostRowBlocks)) : 1;
    l.row_blocks = d->tokens ? int32_t(cdiv(d->tokens, l.chunk)) : 1;
    if (backward && l.row_blocks < kDepth) l.row_blocks = kDepth;   // which clear a row each
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t here = at;
        at += size_t(align_up(bytes, 256));
        return here;
    };
    l.count = take(4);
    l.ticket = take(4);
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
        const bool pieces = l.piece < d->vocab;
        split(d->tokens, pieces ? l.piece : d->vocab, d->hidden, l.grad_width, pieces, l.splits);
        l.sums_pitch[0] = l.pitch;
        l.sums_pitch[1] = l.piece;
        l.row_lse = take(4 * d->tokens);
        l.row_grad = take(4 * d->tokens);
        l.parts = take(4 * kMostRowBlocks);
        l.dz = take(2 * l.pitch * l.piece);
        for (int i = 0; i < 2; i++)
            if (l.splits[i] > 1 || (i == 0 && pieces)) l.grad_sums[i] = take(4 * l.splits[i] * d->hidden * l.sums_pitch[i]);
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
    bool copied;

    template <typename T> T *at(size_t offset) const { return reinterpret_cast<T *>(ws + offset); }

    int start(const void *hidden, const void *w, const void *index, const void *teacher, const uint8_t *mask,
              float *losses, float *lse, int32_t *live, void *grad, const float *lse_in, const float *grad_losses) {
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
        r.hidden = Rows{static_cast<const uint16_t *>(hidden), d->hidden_row, d->hidden_col, d->hidden,
                        at<uint16_t>(l.hidden), l.packed};
        r.tokens = d->tokens;
        r.labels = index;
        r.wide_labels = d->index_type == NEST_I64;
        r.vocab = d->vocab;
        r.flags = d->k ? at<uint8_t>(l.flags) : nullptr;
        r.chunk = l.chunk;
        r.blocks = l.row_blocks;
        r.rows = at<int32_t>(l.rows);
        r.count = at<int32_t>(l.count);
        r.row_labels = d->k ? nullptr : at<int32_t>(l.column);
        r.ticket = live ? at<uint32_t>(l.ticket) : nullptr;
        r.losses = losses;
        r.lse = lse;
        r.live = live;
        r.clear = lse_in != nullptr;
        r.grad = static_cast<uint16_t *>(grad);
        r.wide_grad = d->hidden % 8 == 0 && aligned_to(grad, 16);
        r.lse_in = lse_in;
        r.row_lse = lse_in ? at<float>(l.row_lse) : nullptr;
        r.grad_losses = grad_losses;
        r.row_grad = grad_losses ? at<float>(l.row_grad) : nullptr;
        r.parts = grad_losses ? at<float>(l.parts) : nullptr;
        weight = w;
        weight_pitch = d->weight_row;
        int64_t copiers = 0;
        copied = !in_place(d, w);
        if (copied) {
            weight = ws + l.weight;
            weight_pitch = l.packed;
            r.weight = Rows{static_cast<const uint16_t *>(w), d->weight_row, d->weight_col, d->hidden,
                            at<uint16_t>(l.weight), l.packed};
            copiers = cdiv(d->vocab, kRowThreads / 32);
            if (copiers > 8 * kSMs) copiers = 8 * kSMs;
        }
        return launch_kernel(rows_kernel, dim3(unsigned(l.row_blocks + copiers)), dim3(kRowThreads), 0, stream, 1,
                             "head rows launch", r);
    }

    GemmArgs products() const {
        GemmArgs g = {};
        g.live = at<int32_t>(l.count);
        g.rows = at<int32_t>(l.rows);
        g.pitch = l.pitch;
        g.depth = int32_t(d->hidden);
        g.width = l.width;
        g.how[0] = instruction(d->dtype, true, true, l.width);
        // boxes of the tokens that there are: 8 rows, the swizzle's pattern, at least
        g.a_rows = d->tokens < kHalf ? int32_t(align_up(d->tokens, 8)) : kHalf;
        g.a_bytes = g.a_rows * kDepth * 2;
        g.b_bytes = l.width / 2 * kDepth * 2;
        g.stages = kStages * kStage / (g.a_bytes + g.b_bytes);
        if (g.stages > kMostStages) g.stages = kMostStages;
        g.early = d->tokens <= kTile && !copied;
        (d->k ? g.ids : g.labels) = at<int32_t>(l.column);
        g.shares = d->k ? at<float>(l.shares) : nullptr;
        g.k = d->k;
        g.scale = kLog2e * over_heat(d);
        return g;
    }

    int multiply(Product p, const Maps &maps, const GemmArgs &g, int64_t tiles) const {
        const int pairs = int(tiles < kPairs ? tiles : kPairs);
        return d->dtype == NEST_BF16 ? launch_gemm_bf16(p, maps, g, pairs, stream)
                                     : launch_gemm_f16(p, maps, g, pairs, stream);
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

int nest_head_waits_given_up(int64_t *count, void *stream) {
    if (!count) return NEST_E_INVALID;
    int64_t n[2] = {};
    int rc = gave_up_bf16(&n[0], stream);
    if (!rc) rc = gave_up_f16(&n[1], stream);
    if (!rc) *count = n[0] + n[1];
    return rc;
}

int nest_head_loss(const nest_head_desc *d, const void *hidden, const void *weight, const void *index,
                   const void *teacher, const uint8_t *mask, float *loss, float *losses, float *lse, int32_t *live,
                   void *workspace, size_t ws_bytes, void *stream) {
    if (const int rc = check(d)) return rc;
    if (const int rc = check_inputs(d, hidden, weight, index, teacher, mask)) return rc;
    if (!loss || !live || (d->tokens && (!losses || !lse))) return NEST_E_INVALID;
    Call c = {d, layout_of(d, weight, false), static_cast<unsigned char *>(workspace), stream};
    if (!workspace || ws_bytes < c.l.total || !aligned_to(workspace, 256)) return NEST_E_WORKSPACE;
    if (const int rc = c.start(hidden, weight, index, teacher, mask, losses, lse, live, nullptr, nullptr, nullptr))
        return rc;
    GemmArgs g = c.products();
    g.cols = int32_t(d->vocab);
    const int64_t part = int64_t(c.l.tiles) * c.l.pitch;
    g.part_max = c.at<float>(c.l.part);
    g.part_sum = g.part_max + part;
    g.part_hit = g.part_sum + part;
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
    j.over = over_heat(d);
    j.entropy = d->k ? c.at<float>(c.l.entropy) : nullptr;
    j.losses = losses;
    j.lse = lse;
    j.loss = loss;
    j.sums = c.at<float>(c.l.sums);
    j.ticket = c.at<uint32_t>(c.l.ticket);
    g.join = j;
    g.join_here = d->tokens <= kJoinRows;
    if (d->tokens) {
        Maps maps = {};
        int rc = encode(&maps.a, d->dtype, c.at<void>(c.l.hidden), d->hidden, c.l.pitch, c.l.packed, g.a_rows);
        if (!rc) rc = encode(&maps.b, d->dtype, c.weight, d->hidden, d->vocab, c.weight_pitch, c.l.width / 2);
        if (!rc) rc = c.multiply(kLoss, maps, g, cdiv(d->tokens, kTile) * c.l.tiles);
        if (rc || g.join_here) return rc;
    }
    return launch_kernel(join_kernel, dim3(unsigned(c.l.join)), dim3(kJoinRows * kJoinParts), 0, stream, 1,
                         "head join launch", j);
}

int nest_head_loss_backward(const nest_head_desc *d, const void *hidden, const void *weight, const void *index,
                            const void *teacher, const uint8_t *mask, const float *lse, const float *grad_loss,
                            const float *grad_losses, void *grad_hidden, void *grad_weight, void *workspace,
                            size_t ws_bytes, void *stream) {
    if (const int rc = check(d)) return rc;
    if (const int rc = check_inputs(d, hidden, weight, index, teacher, mask)) return rc;
    if ((!grad_weight && (!grad_hidden && d->tokens)) || (d->tokens && !lse) || !aligned_to(grad_weight, 2) ||
        !aligned_to(grad_hidden, 2))
        return NEST_E_INVALID;
    Call c = {d, layout_of(d, weight, true), static_cast<unsigned char *>(workspace), stream};
    const Layout &l = c.l;
    if (!workspace || ws_bytes < l.total || !aligned_to(workspace, 256)) return NEST_E_WORKSPACE;
    if (const int rc =
            c.start(hidden, weight, index, teacher, mask, nullptr, nullptr, nullptr, grad_hidden, lse, grad_losses))
        return rc;

    GemmArgs g = c.products();
    void *h = c.at<void>(l.hidden);
    uint16_t *dz = c.at<uint16_t>(l.dz);
    Maps logits = {}, grads = {};
    int rc = NEST_OK;
    if (d->tokens) rc = encode(&logits.a, d->dtype, h, d->hidden, l.pitch, l.packed, g.a_rows);
    if (!rc) rc = encode(&logits.b, d->dtype, c.weight, d->hidden, d->vocab, c.weight_pitch, l.width / 2);
    if (!rc) rc = encode(&grads.b, d->dtype, c.weight, d->hidden, d->vocab, c.weight_pitch, kDepth);
    if (!rc) rc = encode(&grads.d, d->dtype, h, d->hidden, l.pitch, l.packed, kDepth);
    const bool wide_weight = grad_weight && d->hidden % 8 == 0 && aligned_to(grad_weight, 16);
    if (!rc && wide_weight) rc = encode(&grads.out, d->dtype, grad_weight, d->hidden, d->vocab, d->hidden, 32);
    if (rc) return rc;

    g.row_lse = c.at<float>(l.row_lse);
    g.row_grad = grad_losses ? c.at<float>(l.row_grad) : nullptr;
    g.by = Scale{grad_loss, grad_losses, c.at<float>(l.parts), l.row_blocks, d->temperature,
                 d->dtype == NEST_F16 ? 32768.0f : 1.0f};
    uint16_t *out[2] = {static_cast<uint16_t *>(grad_hidden), static_cast<uint16_t *>(grad_weight)};
    for (int i = 0; i < 2; i++) {
        g.wide[i] = d->hidden % 8 == 0 && aligned_to(out[i], 16);
        g.splits[i] = l.splits[i];
        g.least = least_of(d->hidden);
        g.sums[i] = l.grad_sums[i] ? c.at<float>(l.grad_sums[i]) : nullptr;
        g.sums_pitch[i] = l.sums_pitch[i];
    }
    const bool pieces = l.piece < d->vocab;
    // adds the parts of the wanted results: the hidden states' gradient, and that of `rows` rows of the weights
    auto sums = [&](bool for_hidden, bool for_weight, int64_t rows, uint16_t *to) {
        if (!for_hidden && !for_weight) return int(NEST_OK);
        SumArgs s = {};
        s.live = g.live;
        s.rows = g.rows;
        s.cols = g.depth;
        s.by = g.by;
        const int64_t wide = cdiv(d->hidden, kSumCols);
        const int64_t blocks[2] = {for_hidden ? cdiv(d->tokens, kSumTile) * wide : 0,
                                   for_weight ? cdiv(rows, kSumTile) * wide : 0};
        if (!blocks[0] && !blocks[1]) return int(NEST_OK);
        s.piece_rows = int32_t(rows);
        s.first_block = int32_t(blocks[0]);
        for (int i = 0; i < 2; i++) {
            s.splits[i] = g.splits[i];
            s.sums[i] = g.sums[i];
            s.pitch[i] = g.sums_pitch[i];
            s.out[i] = i ? to : out[0];
        }
        const dim3 grid(unsigned(blocks[0] + blocks[1]));
        return d->dtype == NEST_BF16
                   ? launch_kernel(sum_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream, 1, "head sums launch", s)
                   : launch_kernel(sum_kernel<__half>, grid, dim3(256), 0, stream, 1, "head sums launch", s);
    };
    const int64_t across = cdiv(d->hidden, l.grad_width);
    for (int64_t first = 0; first < d->vocab; first += l.piece) {
        g.cols = int32_t(d->vocab - first < l.piece ? d->vocab - first : l.piece);
        g.first_col = int32_t(first);
        g.add = first > 0;
        if (d->tokens) {
            if ((rc = encode(&logits.out, d->dtype, dz, g.cols, l.pitch, l.piece, 32))) return rc;
            if ((rc = c.multiply(kDz, logits, g, cdiv(d->tokens, kTile) * cdiv(g.cols, l.width)))) return rc;
            rc = encode(&grads.a, d->dtype, dz, g.cols, l.pitch, l.piece, kHalf);
            if (!rc) rc = encode(&grads.c, d->dtype, dz, g.cols, l.pitch, l.piece, kDepth);
            if (rc) return rc;
        }
        GemmArgs p = g;
        p.width = l.grad_width;
        p.a_bytes = p.b_bytes = kOperand;
        p.stages = kStages;
        p.how[0] = instruction(d->dtype, true, false, p.width);
        p.how[1] = instruction(d->dtype, false, false, p.width);
        p.out[0] = out[0];
        p.out[1] = out[1] ? out[1] + first * d->hidden : nullptr;
        const int64_t tiles = (cdiv(d->tokens, kTile) * p.splits[0] + cdiv(p.cols, kTile) * p.splits[1]) * across;
        if ((rc = c.multiply(kGrads, grads, p, tiles))) return rc;
        // before the next piece's take their place
        if ((rc = sums(false, pieces && g.sums[1] && out[1], g.cols, p.out[1]))) return rc;
    }
    return sums(g.sums[0] && out[0], g.sums[1] && out[1] && !pieces, d->vocab, out[1]);
}

}  // extern "C"
