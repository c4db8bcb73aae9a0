// Matrix products of the output head (nest_head.h) on the tensor cores.
//
// One kernel for the products, over tiles of up to 256 x 256 results made by a pair of thread blocks:
// each of the two loads half of both operands' rows by TMA, one thread of the first issues tcgen05.mma
// for both (cta_group::2, so that every operand byte is loaded once for the pair), and the results stay
// in tensor memory until eight warps per block reduce or round them, while the next tile's products run.
//
//   loss    z = hidden weight^T    per row and tile: maximum, sum of exponentials, target logits
//   dz      the same product       p - q, times the row's factor, in 16 bits
//   grads   dz weight and dz^T hidden over a piece of the vocabulary, in one launch: few long tiles of
//           one and many short ones of the other fill each other's last round
#pragma once

#include <cuda.h>

#include <type_traits>

#include "../../include/nest_head.h"
#include "nest_train.cuh"

namespace nest {
namespace head {

constexpr int kTile = 256;        // rows of results of a pair, and columns at most
constexpr int kHalf = 128;        // rows of either operand that one block of the pair loads
constexpr int kDepth = 64;        // of the summed index per stage: 128 bytes, the widest swizzle
constexpr int kOperand = kHalf * kDepth * 2;   // bytes of one operand's half
constexpr int kStage = 2 * kOperand;
constexpr int kStages = 6;                     // of full size; smaller ones are more
constexpr int kMostStages = 12;
constexpr int kEpilogueWarps = 8;    // two for each quarter of the rows
constexpr int kThreads = 64 + 32 * kEpilogueWarps;
constexpr int kStaging = 32 * 128;   // bytes: 32 rows of 64 results in 16 bits, per epilogue warp
constexpr int kGroup = 8;            // row tiles that share a column tile's operand in L2
constexpr int kNoColumn = 0x7fffffff;
constexpr int kMostRowBlocks = 512;  // of the kernel that lists the live tokens

struct Shared {   // after the stages and the staging
    uint64_t full[kMostStages], empty[kMostStages], done[2], free_[2], drain;
    uint32_t tmem;
};
constexpr size_t kSharedBytes = 1024 + size_t(kStages) * kStage + kEpilogueWarps * kStaging + sizeof(Shared);
static_assert(kSharedBytes <= 232448, "shared memory of a block");

enum Product { kLoss, kDz, kGrads };

struct Maps {     // operands: loss and dz: hidden, weight; grads: dz, weight, dz again by columns, hidden
    CUtensorMap a, b, c, d;
    CUtensorMap out;   // dz, or grad weight where it is 16-byte aligned
};

// What the gradients of the losses are scaled by.
struct Scale {
    const float *grad_loss;     // [1], NULL = 0
    const float *grad_losses;   // [T], NULL = 0
    const float *parts;         // with grad_losses: the largest finite size of each of `blocks` parts
    int32_t blocks;
    float heat;                 // h
    float lift;                 // 2^15 in half precision
};

// What the tiles' maxima and sums are joined into.
struct JoinArgs {
    const int32_t *count, *rows;
    const float *part_max, *part_sum, *part_hit;
    int64_t pitch;
    int32_t tiles;
    float scale;          // log2(e) / h
    float heat, over;     // h, 1 / h
    const float *entropy; // NULL with labels
    float *losses, *lse, *loss;
    float *sums;          // [blocks]
    uint32_t *ticket;
};

struct GemmArgs {
    const int32_t *live;      // n
    const int32_t *rows;      // [n] the live tokens
    int64_t pitch;            // tokens rounded up to a tile: rows of the compacted buffers
    int32_t cols, depth;      // loss, dz: columns of the (piece of the) vocabulary, hidden size
    int32_t first_col;        // of the piece: where its columns start in the vocabulary
    int32_t width;            // of a tile
    uint32_t how[2];          // instruction descriptors: loss and dz or grad hidden; grad weight
    int32_t a_bytes, b_bytes; // of a stage: where the second operand starts, and its room
    int32_t a_rows;           // loss, dz: rows in a box of the first operand
    int32_t stages;
    int32_t early;            // loss, dz: one row tile, and weights that the kernel before does not write
    // targets
    const int32_t *labels;    // [n], NULL with a teacher
    const int32_t *ids;       // [T][k] ascending, kNoColumn past the last
    const float *shares;      // [T][k]
    int32_t k;
    float scale;              // log2(e) / h
    float *part_max, *part_sum, *part_hit;   // loss: [column tile][pitch]
    int32_t join_here;        // loss: the last block joins the tiles of up to kJoinRows tokens
    JoinArgs join;
    const float *row_lse;     // dz: [n], lse log2(e)
    const float *row_grad;    // dz: [n], NULL = 0: the gradient of each token's loss
    Scale by;                 // dz, grads
    // grads: hidden, weight (of the piece); NULL: not wanted
    uint16_t *out[2];
    int32_t wide[2];          // rows of out are 16-byte aligned
    int32_t splits[2];        // parts of the summed index
    int32_t least;            // what a tile takes at least, in stages
    float *sums[2];           // [split][column][row], where results are not final; else NULL
    int64_t sums_pitch[2];
    int32_t add;              // a later piece: sums of grad hidden go on
};

__device__ __forceinline__ uint32_t shared_address(const void *p) { return uint32_t(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ uint32_t block_in_pair() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// One lane of the warp, the same every time, as a branch that the compiler knows to be one lane's: what the loops
// around it compute stays in the registers of the whole warp, which the tensor cores' and the copies'
// instructions take (a branch on the lane's number cost twice the time per stage).
__device__ __forceinline__ bool one_lane() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void pair_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of the same variable in the pair's first block.
__device__ __forceinline__ uint32_t in_first(uint32_t address) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(address));
    return r;
}

__device__ __forceinline__ void barrier_init(uint64_t *b, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(shared_address(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void barrier_expect(uint64_t *b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(shared_address(b)), "r"(bytes)
                 : "memory");
}
// What it lets go on are reads of tensor memory, which the fence before it orders: nothing that this thread
// wrote to memory has to be seen by the other block (waiting for that took a seventh of the loss's time).
__device__ __forceinline__ void arrive_at_first(uint64_t *b) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(in_first(shared_address(b)))
                 : "memory");
}
__device__ __forceinline__ bool barrier_try(uint32_t address, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(address), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint64_t nanoseconds() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
constexpr uint64_t kPatience = 2000000000;   // a tile, of 2048 stages at most, takes under a millisecond

// Warps whose wait gave up, since the library was loaded, in the kernels of this type.
template <typename T> __device__ unsigned long long gave_up = 0;

// Waits for the barrier's phase; false when it did not come in `patience` nanoseconds.  A role whose wait gave
// up waits for nothing more, and the results that it did not see are NaN; it is counted in gave_up.
inline __device__ __noinline__ bool barrier_wait_long(uint32_t address, uint32_t parity, uint64_t patience) {
    const uint64_t start = nanoseconds();
    for (;;) {
        for (int i = 0; i < 256; i++)
            if (barrier_try(address, parity)) return true;
        if (nanoseconds() - start > patience) return false;
    }
}
__device__ __forceinline__ bool barrier_wait(uint64_t *b, uint32_t parity) {
    const uint32_t address = shared_address(b);
#pragma unroll 1
    for (int i = 0; i < 32; i++)
        if (barrier_try(address, parity)) return true;
    return barrier_wait_long(address, parity, kPatience);
}

// A box of `map` from (x, y) on into this block's shared memory; its bytes count at the first block's barrier.
__device__ __forceinline__ void load_box(const CUtensorMap *map, uint32_t to, uint32_t barrier, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(to),
        "l"(map), "r"(x), "r"(y), "r"(barrier)
        : "memory");
}

// A box of this block's shared memory to (x, y) of `map`, which cuts off what lies past its ends.
__device__ __forceinline__ void store_box(const CUtensorMap *map, uint32_t from, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x),
                 "r"(y), "r"(from)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Until the boxes of this thread have been read, or written.
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Shared-memory descriptors of operands in 128-byte rows with the 128-byte swizzle, whose pattern repeats
// every 8 rows (1024 bytes).  Summed index along the rows: groups of 8 operand rows follow each other.
// Operand rows along the rows: 64 of them, groups of 8 summed indices follow each other, and the next 64
// operand rows are 64 summed indices further on.
template <bool ALONG>
__device__ __forceinline__ uint64_t descriptor(uint32_t address) {
    const uint64_t leading = ALONG ? 1 : (kDepth * 128) >> 4, stride = 1024 >> 4;
    return uint64_t((address & 0x3ffff) >> 4) | leading << 16 | stride << 32 | uint64_t(1) << 46 | uint64_t(2) << 61;
}
// Descriptor steps of 16 summed indices.
template <bool ALONG> constexpr uint32_t kStep = ALONG ? 32 >> 4 : (16 * 128) >> 4;

// Instruction descriptor: sums in 32 bits, the operands' type and direction, 256 x width results.
inline uint32_t instruction(int32_t dtype, bool a_along, bool b_along, int width) {
    const uint32_t type = dtype == NEST_BF16;
    return 1u << 4 | type << 7 | type << 10 | uint32_t(!a_along) << 15 | uint32_t(!b_along) << 16 |
           uint32_t(width >> 3) << 17 | uint32_t(kTile >> 4) << 24;
}

__device__ __forceinline__ void multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t how, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(how), "r"(add)
        : "memory");
}
// Arrives at the barrier in both blocks once the products issued so far are done.
__device__ __forceinline__ void commit(uint64_t *b) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            shared_address(b)),
        "h"(uint16_t(3))
        : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of this warp's 32 lanes.
__device__ __forceinline__ void read_columns(float (&v)[32], uint32_t at) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
}
__device__ __forceinline__ void reads_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max_of_three(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Two numbers of 32 bits in one operation each.
struct Pair {
    uint64_t v;
    __device__ __forceinline__ Pair() {}
    __device__ __forceinline__ Pair(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ void get(float &a, float &b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ Pair multiply_add(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
    Pair d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Pair times(Pair a, Pair b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
// exp2 of v * by - off, of 32 numbers.
__device__ __forceinline__ void exponentials(float (&v)[32], float by, float off) {
    const Pair two_by(by, by), two_off(-off, -off);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        float x, y;
        multiply_add(Pair(v[e], v[e + 1]), two_by, two_off).get(x, y);
        v[e] = exp2_fast(x);
        v[e + 1] = exp2_fast(y);
    }
}

template <typename T> __device__ __forceinline__ uint32_t pack_two(float low, float high);
template <> __device__ __forceinline__ uint32_t pack_two<__nv_bfloat16>(float low, float high) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(low, high);
    return reinterpret_cast<const uint32_t &>(v);
}
template <> __device__ __forceinline__ uint32_t pack_two<__half>(float low, float high) {
    const __half2 v = __floats2half2_rn(low, high);
    return reinterpret_cast<const uint32_t &>(v);
}

// A tile of results and the stages of its summed index; kind 1: grad weight.
struct Tile {
    int kind, row, col, split, from, steps;
};

// One product's tiles in the order in which they are taken: for each part of the summed index, groups of
// kGroup row tiles, column by column.
struct Tiles {
    int rows, cols, splits, steps;
    int least;   // stages in whose time a tile's results are written
    __device__ __forceinline__ int per() const { return (steps + splits - 1) / splits; }
    __device__ __forceinline__ int cost() const { return max(per(), least); }
    __device__ __forceinline__ int count() const { return rows * cols * splits; }
    __device__ __forceinline__ void at(int i, Tile &t) const {
        t.split = i / (rows * cols);
        i -= t.split * rows * cols;
        const int group = kGroup * cols, g = i / group, left = i - g * group;
        const int high = min(kGroup, rows - g * kGroup);
        t.col = left / high;
        t.row = g * kGroup + left - t.col * high;
        t.from = t.split * per();
        t.steps = max(0, min(per(), steps - t.from));
    }
};

// The tiles of one pair.  Loss, dz: every pairs-th.  Grads: the product with the longer tiles first, every
// pairs-th of its tiles; pairs that get one less then take as many of the other product's tiles as make up for it,
// and the rest goes to all pairs in turn.
struct Work {
    Tiles long_, short_;
    int kind;                 // of the longer
    int pair, pairs, i, extra, idle;

    __device__ __forceinline__ void start(const Tiles &h, const Tiles &w, bool two) {
        pair = int(blockIdx.x >> 1);
        pairs = int(gridDim.x >> 1);
        kind = two && w.per() > h.per();
        long_ = kind ? w : h;
        short_ = kind ? h : w;
        i = pair;
        const int over = long_.count() % pairs;
        idle = over ? pairs - over : 0;      // pairs with one less: the last ones
        extra = two && idle ? (long_.cost() + short_.cost() / 2) / short_.cost() : 0;
        if (!two) short_.rows = 0;
    }
    // phases of i: [0, count) the longer; then, from `count` on, idle rounds and common rounds of the shorter
    int phase = 0, j = 0;
    __device__ __forceinline__ bool next(Tile &t) {
        if (phase == 0) {
            if (i < long_.count()) {
                long_.at(i, t);
                t.kind = kind;
                i += pairs;
                return true;
            }
            phase = 1;
        }
        if (phase == 1) {
            const int mine = pair - (pairs - idle);
            if (mine >= 0 && j < extra) {
                const int at = mine + j++ * idle;
                if (at < short_.count()) {
                    short_.at(at, t);
                    t.kind = !kind;
                    return true;
                }
            }
            phase = 2;
            i = extra * idle + pair;
        }
        if (i >= short_.count()) return false;
        short_.at(i, t);
        t.kind = !kind;
        i += pairs;
        return true;
    }
};

// How dz is scaled: a row's factor is (base + its loss's gradient) * over, and the products are multiplied by unit.
// Without gradients of single losses every row has the same factor, which is left to unit: p - q itself is
// rounded, whose -1 at most labels is exact, and no rounding of the factor is common to all rows.  With them the
// largest finite factor lies below 1 (2^15 where dz is lifted) by a power of two.  By all lanes of a warp.
struct Scaling {
    float base, over, unit;
};
__device__ __forceinline__ Scaling scaling_of(const Scale &s, int n) {
    const float share = s.grad_loss && n ? *s.grad_loss / float(n) : 0.0f;
    if (!s.grad_losses) return Scaling{1.0f, s.lift, share * s.heat / s.lift};
    float top = 0.0f;
    for (int b = threadIdx.x & 31; b < s.blocks; b += 32) top = fmaxf(top, s.parts[b]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (fabsf(share) < INFINITY) top += fabsf(share);
    top = fminf(top * s.heat, 8e37f);
    int e = 0;
    if (top > 0.0f) frexpf(top, &e);
    e = max(-100, e);
    return Scaling{share, ldexpf(s.lift, -e) * s.heat, ldexpf(1.0f / s.lift, e)};
}

// What a row of a tile needs from memory, loaded a tile ahead.
struct Row {
    int token;      // -1: not there
    int label;
    float lse, grad;
};

// A token's targets from a column on, in ascending order.
struct Targets {
    const int32_t *id;
    const float *share;
    int j, k, next;
    __device__ __forceinline__ void start(const GemmArgs &a, const Row &row, int col) {
        k = 0;
        j = 0;
        if (a.labels) {
            next = row.token >= 0 && row.label >= col ? row.label : kNoColumn;
            return;
        }
        next = kNoColumn;
        if (row.token < 0) return;
        k = a.k;
        id = a.ids + int64_t(row.token) * k;
        share = a.shares + int64_t(row.token) * k;
        int low = 0, high = k;   // the first id >= col
        while (low < high) {
            const int mid = (low + high) >> 1;
            if (id[mid] < col) low = mid + 1;
            else high = mid;
        }
        j = low;
        if (j < k) next = id[j];
    }
    __device__ __forceinline__ float weight() const { return k ? share[j] : 1.0f; }
    __device__ __forceinline__ void advance() { next = ++j < k ? id[j] : kNoColumn; }
};

// v[i] by five steps of halving: an index that the compiler does not see would move v to memory.
__device__ __forceinline__ float pick(const float (&v)[32], int i) {
    float t[16];
#pragma unroll
    for (int e = 0; e < 16; e++) t[e] = i & 16 ? v[e + 16] : v[e];
#pragma unroll
    for (int e = 0; e < 8; e++) t[e] = i & 8 ? t[e + 8] : t[e];
#pragma unroll
    for (int e = 0; e < 4; e++) t[e] = i & 4 ? t[e + 4] : t[e];
#pragma unroll
    for (int e = 0; e < 2; e++) t[e] = i & 2 ? t[e + 2] : t[e];
    return i & 1 ? t[1] : t[0];
}

constexpr int kJoinRows = 32;

template <int PARTS>
struct JoinShared {
    float max[PARTS][kJoinRows + 1], sum[PARTS][kJoinRows + 1], hit[PARTS][kJoinRows + 1], all[PARTS];
};

// Joins the tiles' maxima and sums of 32 rows, PARTS warps with a lane to a row, eight tiles at a time so that no
// load waits for another.  Returns the sum of the rows' losses to thread 0 of warp 0.  `sync`: a barrier of
// these warps.
template <int PARTS, typename Sync>
__device__ __forceinline__ float join_rows(const JoinArgs &a, int64_t first, int n, int part, int lane,
                                           JoinShared<PARTS> &sh, Sync sync) {
    constexpr int kAtOnce = 8;
    const int64_t r = first + lane;
    float top = -INFINITY, sum = 0.0f, hit = 0.0f;
    if (r < n) {
        for (int t0 = part; t0 < a.tiles; t0 += PARTS * kAtOnce) {
            float high[kAtOnce], s[kAtOnce], h[kAtOnce], most = top;
#pragma unroll
            for (int i = 0; i < kAtOnce; i++) {
                const int t = t0 + i * PARTS;
                const int64_t at = int64_t(t) * a.pitch + r;
                const bool in = t < a.tiles;
                high[i] = in ? __ldcg(a.part_max + at) : -INFINITY;
                s[i] = in ? __ldcg(a.part_sum + at) : 0.0f;
                h[i] = in ? __ldcg(a.part_hit + at) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; i++) most = fmaxf(most, high[i]);
            sum *= top == most ? 1.0f : exp2_fast((top - most) * a.scale);
            top = most;
            // (a tile of minus infinity alone has a sum of 0, one with NaN a sum of NaN, which stays)
#pragma unroll
            for (int i = 0; i < kAtOnce; i++) {
                sum = fmaf(s[i], high[i] == top ? 1.0f : exp2_fast((high[i] - top) * a.scale), sum);
                hit += h[i];
            }
        }
    }
    sh.max[part][lane] = top;
    sync();
    float high = -INFINITY;
#pragma unroll
    for (int p = 0; p < PARTS; p++) high = fmaxf(high, sh.max[p][lane]);
    sh.sum[part][lane] = sum * (top == high ? 1.0f : exp2_fast((top - high) * a.scale));
    sh.hit[part][lane] = hit;
    sync();
    if (part == 0) sh.max[0][lane] = high;
    sync();
    // a warp adds the parts of 32 / PARTS rows
    const int row = (kJoinRows / PARTS) * part + lane / PARTS, p = lane % PARTS;
    sum = sh.sum[p][row];
    hit = sh.hit[p][row];
#pragma unroll
    for (int o = PARTS / 2; o; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        hit += __shfl_xor_sync(0xffffffffu, hit, o);
    }
    float loss = 0.0f;
    if (p == 0 && first + row < n) {
        const int t = a.rows[first + row];
        // the largest logit's distance from the targets' first: the difference of near numbers is exact
        const float most = sh.max[0][row], log_sum = logf(sum);
        const float apart = fmaf(most - hit, a.over, log_sum) + (a.entropy ? a.entropy[t] : 0.0f);
        loss = a.heat * a.heat * apart;
        a.lse[t] = fmaf(most, a.over, log_sum);
        a.losses[t] = loss;
    }
    loss = warp_sum(loss);
    if (lane == 0) sh.all[part] = loss;
    sync();
    if (part == 0 && lane == 0)
        for (int w = 1; w < PARTS; w++) loss += sh.all[w];
    return loss;
}

// 64 results of each of the warp's 32 rows to shared memory, 128 bytes a row with the 128-byte swizzle.
__device__ __forceinline__ void stage_rows(const uint32_t (&packed)[32], unsigned char *staging, int lane) {
    uint4 *mine = reinterpret_cast<uint4 *>(staging) + lane * 8;
#pragma unroll
    for (int u = 0; u < 8; u++)
        mine[u ^ (lane & 7)] = make_uint4(packed[4 * u], packed[4 * u + 1], packed[4 * u + 2], packed[4 * u + 3]);
}

// And from there to memory where the rows do not follow each other or are off alignment, a row's together.
// `to`: where this lane's row goes, or NULL where nothing is written; `left`: columns that exist from here on.
// Rows off alignment are written in the 16-byte pieces that lie in them, shifted, and the rest one by one.
__device__ __forceinline__ void write_rows(const unsigned char *staging, uint16_t *to, int left, bool wide, int lane) {
    const uint64_t row = reinterpret_cast<uint64_t>(to);
    const int unit = lane & 7;
    if (left > 64) left = 64;
    if (wide) {
        const bool in = left - 8 * unit >= 8;   // of the columns, whose number is a multiple of 8
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
            uint4 v[4];
            uint64_t p[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int r = 4 * (h + i) + (lane >> 3);
                p[i] = __shfl_sync(0xffffffffu, row, r);
                v[i] = (reinterpret_cast<const uint4 *>(staging) + r * 8)[unit ^ (r & 7)];
            }
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (p[i] && in) *(reinterpret_cast<uint4 *>(p[i]) + unit) = v[i];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int r = 4 * i + (lane >> 3);
        uint16_t *p = reinterpret_cast<uint16_t *>(__shfl_sync(0xffffffffu, row, r));
        const uint4 *from = reinterpret_cast<const uint4 *>(staging) + r * 8;
        if (p) {
            // `skip` numbers come before the row's first aligned piece
            const int skip = int((16 - (uint32_t(reinterpret_cast<uintptr_t>(p)) & 15)) & 15) >> 1;
            const uint4 v = from[unit ^ (r & 7)], q = unit < 7 ? from[(unit + 1) ^ (r & 7)] : make_uint4(0, 0, 0, 0);
            if (8 * unit + skip + 8 <= left) {
                uint32_t w[8] = {v.x, v.y, v.z, v.w, q.x, q.y, q.z, q.w};
                const bool two = skip & 4, one = skip & 2, part = skip & 1;
#pragma unroll
                for (int e = 0; e < 6; e++) w[e] = two ? w[e + 2] : w[e];
#pragma unroll
                for (int e = 0; e < 5; e++) w[e] = one ? w[e + 1] : w[e];
#pragma unroll
                for (int e = 0; e < 4; e++) w[e] = part ? __funnelshift_r(w[e], w[e + 1], 16) : w[e];
                *reinterpret_cast<uint4 *>(p + 8 * unit + skip) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            // what no piece holds: the first `skip`, and those behind the last piece
            const int last = left < skip ? skip : skip + (left - skip) / 8 * 8;
            const uint16_t *one = reinterpret_cast<const uint16_t *>(from);
#pragma unroll
            for (int e = unit; e < 16; e += 8) {
                const int at = e < 8 ? e : last + e - 8;
                if (at < (e < 8 ? min(skip, left) : left)) p[at] = one[((at >> 3) ^ (r & 7)) * 8 + (at & 7)];
            }
        }
        __syncwarp();
    }
}

// Warp 0 of each block copies operands, warp 1 of the first issues the products, the others reduce or round them.
// Bound by the tensor cores at large hidden sizes: 2048 x 32000 x 4096 in bf16 takes 267 us for the loss (2.0
// PFLOP/s), 278 for dz and 533 for both gradients, with the tensor pipe 97, 93 and 97 % active.  Tiles of 256 x
// 256 need 64 KB of operands a stage, 16 TB/s over all pairs, which L2 gives; with six stages on their way the
// products do not wait.  At hidden size 64 the epilogue bounds: 4096 x 128000 takes 187 us, 1.8 us a tile.  For few
// tokens memory does: 1 x 32000 x 4096 reads 262 MB in 45 us.
template <Product P, typename T>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ GemmArgs a) {
    extern __shared__ unsigned char raw[];
    unsigned char *base = raw + ((1024 - (shared_address(raw) & 1023)) & 1023);   // the swizzle's alignment
    unsigned char *staging = base + kStages * kStage;
    Shared &sh = *reinterpret_cast<Shared *>(staging + kEpilogueWarps * kStaging);
    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t half = block_in_pair();

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMostStages; i++) {
            barrier_init(&sh.full[i], 1);
            barrier_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; i++) {
            barrier_init(&sh.done[i], 1);
            barrier_init(&sh.free_[i], 2 * kEpilogueWarps);
        }
        barrier_init(&sh.drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         shared_address(&sh.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    pair_sync();
    fence_after();

    const int col_tiles = ((P == kGrads ? a.depth : a.cols) + a.width - 1) / a.width;
    const int stage = a.a_bytes + a.b_bytes, part = a.width / 2;   // bytes; columns that this block loads
    // Few tokens: boxes of no more rows than there are leave room for more stages, and the second block has no
    // rows.  Operand rows that are not loaded make result rows that are not read.
    const bool both = P == kGrads || a.a_rows == kHalf;
    const uint32_t bytes = P == kGrads ? 2 * (kOperand + uint32_t(part) * kDepth * 2)
                                       : kDepth * 2 * ((both ? 2 : 1) * uint32_t(a.a_rows) + 2 * uint32_t(part));
    int ahead = 0;   // stages whose weights are on their way before the kernel before this one has ended
    if (P != kGrads && a.early && warp == 0) {
        // one row tile: the pair's number is its first column tile
        const int x = int(blockIdx.x >> 1) * a.width + int(half) * part, steps = (a.depth + kDepth - 1) / kDepth;
        ahead = min(a.stages, steps);
        if (one_lane()) {
            for (int s = 0; s < ahead; s++) {
                if (half == 0) barrier_expect(&sh.full[s], bytes);
                load_box(&maps.b, shared_address(base + s * stage + a.a_bytes), in_first(shared_address(&sh.full[s])),
                         s * kDepth, a.first_col + x);
            }
        }
        __syncwarp();
    }
    pdl_wait();
    pdl_trigger();

    const uint32_t tmem = sh.tmem;
    const int n = *a.live;
    const int row_tiles = P != kGrads ? max(1, (n + kTile - 1) / kTile) : a.out[0] ? (n + kTile - 1) / kTile : 0;
    Work work;
    work.start(Tiles{row_tiles, col_tiles, P == kGrads ? a.splits[0] : 1,
                     ((P == kGrads ? a.cols : a.depth) + kDepth - 1) / kDepth, a.least},
               Tiles{a.out[1] ? (a.cols + kTile - 1) / kTile : 0, col_tiles, a.splits[1], (n + kDepth - 1) / kDepth, a.least},
               P == kGrads);
    Tile t = {};

    if (warp == 0) {
        int s = 0;
        uint32_t phase = 0;
        bool ok = true;
        const uint32_t stage0 = shared_address(base), full0 = in_first(shared_address(&sh.full[0]));
        const int stages = a.stages;
        // the loop over a tile's stages, of one product each: its loads differ
        auto loads = [&](auto product) {
            constexpr int kKind = decltype(product)::value;   // 0, 1: grad hidden, grad weight; 2: logits
            const int y = t.row * kTile + int(half) * kHalf, x = t.col * a.width + int(half) * part;
            for (int kb = 0; kb < t.steps; kb++) {
                ok = __all_sync(0xffffffffu, barrier_wait(&sh.empty[s], phase ^ 1));
                if (!ok) break;
                const uint32_t to = stage0 + uint32_t(s * stage), bar = full0 + s * 8;
                const int k0 = (t.from + kb) * kDepth;
                const bool begun = ahead > 0;
                if (begun) ahead--;
                if (!one_lane()) {
                } else if constexpr (kKind == 2) {
                    if (half == 0 && !begun) barrier_expect(&sh.full[s], bytes);
                    if (both || half == 0) load_box(&maps.a, to, bar, k0, y);
                    if (!begun) load_box(&maps.b, to + a.a_bytes, bar, k0, a.first_col + x);
                } else {
                    if (half == 0) barrier_expect(&sh.full[s], bytes);
                    const CUtensorMap *map = kKind ? &maps.d : &maps.b;
                    const int r = k0 + (kKind ? 0 : a.first_col);
                    if constexpr (kKind == 0) {
                        load_box(&maps.a, to, bar, k0, y);
                    } else {
                        load_box(&maps.c, to, bar, y, k0);
                        load_box(&maps.c, to + kOperand / 2, bar, y + 64, k0);
                    }
                    load_box(map, to + kOperand, bar, x, r);
                    if (part > 64) load_box(map, to + kOperand + kOperand / 2, bar, x + 64, r);
                }
                __syncwarp();
                if (++s == stages) s = 0, phase ^= 1;
            }
        };
        while (ok && work.next(t)) {
            if constexpr (P != kGrads) loads(std::integral_constant<int, 2>{});
            else if (t.kind == 0) loads(std::integral_constant<int, 0>{});
            else loads(std::integral_constant<int, 1>{});
        }
        if (!ok && lane == 0) atomicAdd(&gave_up<T>, 1ull);
        if (!ok) {   // copies under way end within microseconds: those of the stages that are still open
            for (int i = 0; i < a.stages && half == 0; i++)
                barrier_wait_long(shared_address(&sh.full[i]), i < s ? phase : phase ^ 1, 1000000);
            const uint64_t start = nanoseconds();
            while (nanoseconds() - start < 10000000) __nanosleep(1000);
        }
    } else if (warp == 1 && half == 0) {
        int s = 0, use = 0;
        uint32_t phase = 0;
        bool ok = true;
        const uint32_t stage0 = shared_address(base);
        const int stages = a.stages, step = stage >> 4;   // of descriptors
        // operands whose rows in memory run along the summed index: both; dz; none
        auto products = [&](auto a_along, auto b_along, uint32_t how, uint32_t to) {
            constexpr bool kA = decltype(a_along)::value, kB = decltype(b_along)::value;
            const uint64_t a0 = descriptor<kA>(stage0), b0 = descriptor<kB>(stage0 + a.a_bytes);
            for (int kb = 0, steps = t.steps; kb < steps; kb++) {
                ok = __all_sync(0xffffffffu, barrier_wait(&sh.full[s], phase));
                if (!ok) break;
                fence_after();
                const uint64_t da = a0 + uint32_t(s * step), db = b0 + uint32_t(s * step);
                if (one_lane()) {
#pragma unroll
                    for (int q = 0; q < kDepth / 16; q++) multiply(to, da + q * kStep<kA>, db + q * kStep<kB>, how, kb | q);
                    commit(&sh.empty[s]);
                }
                __syncwarp();
                if (++s == stages) s = 0, phase ^= 1;
            }
        };
        while (ok && work.next(t)) {
            if (!t.steps) continue;
            const int acc = use & 1;
            ok = __all_sync(0xffffffffu, barrier_wait(&sh.free_[acc], ((use >> 1) & 1) ^ 1));
            use++;
            if (!ok) break;
            fence_after();
            const uint32_t to = tmem + acc * kTile;
            if constexpr (P != kGrads) products(std::true_type{}, std::true_type{}, a.how[0], to);
            else if (t.kind == 0) products(std::true_type{}, std::false_type{}, a.how[0], to);
            else products(std::false_type{}, std::false_type{}, a.how[1], to);
            if (ok && one_lane()) commit(&sh.done[acc]);
            __syncwarp();
        }
        if (!ok) {
            if (lane == 0) atomicAdd(&gave_up<T>, 1ull);
            if (one_lane()) commit(&sh.drain);
            __syncwarp();
            barrier_wait(&sh.drain, 0);
        }
    } else if (warp >= 2) {
        const int quarter = warp & 3;   // the lanes of tensor memory that this warp may read
        const int side = (warp - 2) >> 2;   // of the two warps of a quarter: every second chunk of columns each
        unsigned char *mine = staging + (warp - 2) * kStaging;
        const int local = int(half) * kHalf + quarter * 32 + lane;
        const float nan = __int_as_float(0x7fc00000);
        Scaling by = {};
        if constexpr (P != kLoss) by = scaling_of(a.by, n);
        const float unit = by.unit;
        bool ok = true;
        int use = 0;
        auto row_of = [&](const Tile &x) {
            Row row = {-1, kNoColumn, 0.0f, 0.0f};
            const int r = x.row * kTile + local;
            if (x.kind == 0 && r < n) {
                row.token = a.rows[r];
                if (P != kGrads && a.labels) row.label = a.labels[r];
                if constexpr (P == kDz) {
                    row.lse = a.row_lse[r];
                    if (a.row_grad) row.grad = a.row_grad[r];
                }
            }
            return row;
        };
        Tile after = {};
        Row row = {}, row_after = {};
        bool more = work.next(t);
        if (more) row = row_of(t);
        for (; more; t = after, row = row_after) {
            more = work.next(after);
            if (more) row_after = row_of(after);
            const int acc = use & 1, r = t.row * kTile + local, c0 = t.col * a.width;
            const bool there = r < (t.kind ? a.cols : n);
            const uint32_t from = tmem + acc * kTile + (uint32_t(quarter * 32) << 16);
            const int token = row.token;
            Targets hits;
            if constexpr (P != kGrads) hits.start(a, row, a.first_col + c0);
            const float lse = row.lse, factor = (by.base + row.grad) * by.over;
            if (t.steps) ok = ok && barrier_wait(&sh.done[acc], (use >> 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            fence_after();

            if constexpr (P == kLoss) {
                float top = -INFINITY, sum = 0.0f, hit = 0.0f;
                const int chunks = min(a.width, a.cols - c0 + 31) / 32;
                auto reduce = [&](float(&v)[32], int at) {
                    if (__any_sync(0xffffffffu, hits.next < at + 32)) {
                        while (hits.next < at + 32) {
                            // the other warp's chunks lie between; a share of 0 takes nothing of minus infinity
                            if (const float q = hits.weight(); hits.next >= at && q != 0.0f)
                                hit = fmaf(q, pick(v, hits.next - at), hit);
                            hits.advance();
                        }
                        __syncwarp();
                    }
                    if (at + 32 > a.cols) {
#pragma unroll
                        for (int e = 0; e < 32; e++) v[e] = at + e < a.cols ? v[e] : -INFINITY;
                    }
                    float m[4] = {top, top, top, top};
#pragma unroll
                    for (int e = 0; e < 32; e += 2) m[e >> 1 & 3] = max_of_three(m[e >> 1 & 3], v[e], v[e + 1]);
                    // no finite logit yet: 0 is subtracted, so that minus infinity gives exponentials of 0 (and NaN NaN)
                    const float high = max_of_three(fmaxf(m[0], m[1]), m[2], m[3]);
                    const float off = high == -INFINITY ? 0.0f : high * a.scale;
                    // (a product with 0 too: the sum so far may be NaN, of logits that the maximum passes over)
                    const float kept = top == high ? sum : sum * exp2_fast(fmaf(top, a.scale, -off));
                    exponentials(v, a.scale, off);
                    Pair u[4] = {Pair(v[0], v[1]), Pair(v[2], v[3]), Pair(v[4], v[5]), Pair(v[6], v[7])};
#pragma unroll
                    for (int e = 8; e < 32; e += 2) u[e >> 1 & 3] = add(u[e >> 1 & 3], Pair(v[e], v[e + 1]));
                    float x, y;
                    add(add(u[0], u[1]), add(u[2], u[3])).get(x, y);
                    sum = kept + (x + y);
                    top = high;
                };
                // the next chunk is on its way while one is reduced; behind the last it is the last again
                float v[32], w[32];
                const int last = side + ((chunks - 1 - side) & ~1);
                if (side < chunks) {
                    read_columns(v, from + side * 32);
                    reads_wait();
#pragma unroll 1
                    for (int c = side;; c += 4) {
                        read_columns(w, from + min(c + 2, last) * 32);
                        reduce(v, c0 + c * 32);
                        reads_wait();
                        if (c + 2 > last) break;
                        read_columns(v, from + min(c + 4, last) * 32);
                        reduce(w, c0 + (c + 2) * 32);
                        reads_wait();
                        if (c + 4 > last) break;
                    }
                }
                fence_before();
                __syncwarp();
                if (lane == 0) arrive_at_first(&sh.free_[acc]);
                // What the second warp of a quarter found.  It does not wait for the first, which is at most two tiles
                // behind: three places and barriers in turn.  (Nothing else is staged.)
                const int turn = use % 3, place = quarter * 32 + lane, id = 1 + 3 * quarter + turn;
                float(*other)[kHalf] = reinterpret_cast<float(*)[kHalf]>(staging) + 3 * turn;
                if (side) {
                    other[0][place] = top, other[1][place] = sum, other[2][place] = hit;
                    asm volatile("bar.arrive %0, 64;" ::"r"(id) : "memory");
                } else {
                    asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
                }
                if (!side && there) {
                    // without a chunk: minus infinity, 0 and 0
                    const float far = other[0][place], both = fmaxf(top, far);
                    sum = sum * (top == both ? 1.0f : exp2_fast((top - both) * a.scale)) +
                          other[1][place] * (far == both ? 1.0f : exp2_fast((far - both) * a.scale));
                    top = both;
                    hit += other[2][place];
                    const int64_t at = int64_t(t.col) * a.pitch + r;
                    a.part_max[at] = top;
                    a.part_sum[at] = ok ? sum : nan;
                    a.part_hit[at] = hit;
                }
            } else {
                const int columns = P == kDz ? a.cols : a.depth;
                const int chunks = (min(a.width, columns - c0) + 63) / 64;
                float *sums = P == kGrads ? a.sums[t.kind] : nullptr;
                uint16_t *to = nullptr;
                if (P == kGrads && there) to = a.out[t.kind] + int64_t(t.kind ? r : token) * a.depth;
                if (P == kGrads && sums) sums += int64_t(t.split) * a.depth * a.sums_pitch[t.kind] + r;
#pragma unroll 1
                for (int c = side; c < chunks; c += 2) {
                    const int at = c0 + c * 64;
                    uint32_t packed[32];
                    float both[2][32];
                    if (t.steps) {
                        read_columns(both[0], from + c * 64);
                        read_columns(both[1], from + c * 64 + 32);
                        reads_wait();
                    }
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const int here = at + 32 * h;
                        float(&v)[32] = both[h];
                        if (!ok || !t.steps) {
#pragma unroll
                            for (int e = 0; e < 32; e++) v[e] = ok ? 0.0f : nan;
                        }
                        if constexpr (P == kDz) {
                            const int column = a.first_col + here;
                            exponentials(v, a.scale, lse);
                            if (__any_sync(0xffffffffu, hits.next < column + 32)) {
                                while (hits.next < column + 32) {
                                    const float q = hits.weight();
                                    const int d = hits.next - column;   // below 0: the other warp's
#pragma unroll
                                    for (int e = 0; e < 32; e++) v[e] -= e == d ? q : 0.0f;
                                    hits.advance();
                                }
                                __syncwarp();
                            }
#pragma unroll
                            for (int e = 0; e < 32; e += 2)
                                times(Pair(v[e], v[e + 1]), Pair(factor, factor)).get(v[e], v[e + 1]);
                        } else {
                            if (sums) {
                                if (there) {
                                    const int64_t pitch = a.sums_pitch[t.kind];
                                    if (a.add && t.kind == 0) {
#pragma unroll
                                        for (int e = 0; e < 32; e++)
                                            if (here + e < columns) v[e] += sums[int64_t(here + e) * pitch];
                                    }
#pragma unroll
                                    for (int e = 0; e < 32; e++)
                                        if (here + e < columns) sums[int64_t(here + e) * pitch] = v[e];
                                }
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; e++) v[e] *= unit;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 16; e++) packed[16 * h + e] = pack_two<T>(v[2 * e], v[2 * e + 1]);
                    }
                    if (P == kDz && !there) {   // rows past the last enter later sums: zeros
#pragma unroll
                        for (int e = 0; e < 32; e++) packed[e] = 0;
                    }
                    if (P == kDz || !sums) {
                        if (lane == 0) stores_read();   // of the chunk before
                        __syncwarp();
                        stage_rows(packed, mine, lane);
                        if (P == kDz || (t.kind && a.wide[1])) {
                            // rows of dz past n too
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            __syncwarp();
                            if (lane == 0 && (P == kDz || there))
                                store_box(&maps.out, shared_address(mine), at,
                                          (P == kGrads ? a.first_col : 0) + r);
                        } else {
                            __syncwarp();
                            write_rows(mine, to ? to + at : nullptr, columns - at, a.wide[t.kind], lane);
                        }
                    }
                }
                if (t.steps) {
                    fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_at_first(&sh.free_[acc]);
                }
            }
            if (t.steps) use++;
        }
        if (lane == 0) stores_done();
        if (!ok && lane == 0) atomicAdd(&gave_up<T>, 1ull);
        if (P == kLoss && a.join_here) {
            // Few tokens: the last block joins what all blocks left, which saves a launch (32 tokens x 32000
            // columns: 55 KB; for more, one block reads longer than a launch takes).
            auto sync = [] { asm volatile("bar.sync 13, %0;" ::"n"(32 * kEpilogueWarps) : "memory"); };
            auto &last = *reinterpret_cast<int *>(staging);
            auto &room = *reinterpret_cast<JoinShared<kEpilogueWarps> *>(staging + 16);
            sync();
            if (warp == 2 && lane == 0) last = last_ticket(a.join.ticket, gridDim.x);
            sync();
            if (last) {
                const float sum = join_rows<kEpilogueWarps>(a.join, 0, n, warp - 2, lane, room, sync);
                if (warp == 2 && lane == 0) *a.join.loss = n ? sum / float(n) : 0.0f;
            }
        }
    }

    __syncwarp();
    fence_before();
    __syncthreads();
    pair_sync();
    fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// The products' launchers, one translation unit for each type.
int launch_gemm_bf16(Product p, const Maps &maps, const GemmArgs &args, int pairs, void *stream);
int launch_gemm_f16(Product p, const Maps &maps, const GemmArgs &args, int pairs, void *stream);
// gave_up of this type on the current device, behind the work of the stream, which is waited for.
int gave_up_bf16(int64_t *count, void *stream);
int gave_up_f16(int64_t *count, void *stream);

template <typename T> int read_gave_up(int64_t *count, void *stream) {
    unsigned long long n = 0;
    const auto s = static_cast<cudaStream_t>(stream);
    int rc = cuda_status(cudaMemcpyFromSymbolAsync(&n, gave_up<T>, sizeof(n), 0, cudaMemcpyDeviceToHost, s), "waits given up");
    if (!rc) rc = cuda_status(cudaStreamSynchronize(s), "waits given up");
    *count = int64_t(n);
    return rc;
}

template <typename T>
int launch_gemm(Product p, const Maps &maps, const GemmArgs &args, int pairs, void *stream) {
    auto go = [&](auto product, const char *what) {
        constexpr Product P = decltype(product)::value;
        if (const int rc = allow<gemm_kernel<P, T>>(kSharedBytes, what)) return rc;
        return launch_kernel(gemm_kernel<P, T>, dim3(2 * pairs), dim3(kThreads), kSharedBytes, stream, 1, what, maps,
                             args);
    };
    switch (p) {
        case kLoss: return go(std::integral_constant<Product, kLoss>{}, "head loss launch");
        case kDz: return go(std::integral_constant<Product, kDz>{}, "head dz launch");
        default: return go(std::integral_constant<Product, kGrads>{}, "head gradients launch");
    }
}

}  // namespace head
}  // namespace nest
