// Matrix products of the output head (nest_head.h) on the tensor cores.
//
// One kernel for the four products, over tiles of 256 x 256 results made by a pair of thread blocks:
// each of the two loads half of both operands' rows by TMA, one thread of the first issues tcgen05.mma
// for both (cta_group::2, so that every operand byte is loaded once for the pair), and the results stay
// in tensor memory until four warps per block reduce or round them.
//
//   loss         z = hidden weight^T    per row and tile: maximum, sum of exponentials, target logits
//   dz           the same product       p - q, times the row's scale, in 16 bits
//   grad hidden  dz weight              over a piece of the vocabulary
//   grad weight  dz^T hidden            over the live tokens
#pragma once

#include <cuda.h>

#include <type_traits>

#include "../../include/nest_head.h"
#include "nest_train.cuh"

namespace nest {
namespace head {

constexpr int kTile = 256;        // rows and columns of results of a pair
constexpr int kHalf = 128;        // rows of either operand that one block of the pair loads
constexpr int kDepth = 64;        // of the summed index per stage: 128 bytes, the widest swizzle
constexpr int kOperand = kHalf * kDepth * 2;   // bytes of one operand's half
constexpr int kStage = 2 * kOperand;
constexpr int kStages = 6;
constexpr int kEpilogueWarps = 4;
constexpr int kThreads = 64 + 32 * kEpilogueWarps;
constexpr int kStaging = 32 * 128;   // bytes: 32 rows of 64 results in 16 bits, per epilogue warp
constexpr int kGroup = 8;            // row tiles that share a column tile's operand in L2
constexpr int kNoColumn = 0x7fffffff;

struct Shared {   // after the stages and the staging
    uint64_t full[kStages], empty[kStages], done[2], free_[2], drain;
    uint32_t tmem;
};
constexpr size_t kSharedBytes = 1024 + size_t(kStages) * kStage + kEpilogueWarps * kStaging + sizeof(Shared);

enum Product { kLoss, kDz, kGradHidden, kGradWeight };

struct GemmArgs {
    const int32_t *live;      // n
    const int32_t *rows;      // [n] the live tokens
    int64_t pitch;            // tokens rounded up to a tile: rows of the compacted buffers
    int32_t m, cols, depth;   // rows (grad weight), columns and summed length (not grad weight)
    int32_t first_col;        // of the piece: where its columns start in the vocabulary
    // targets, by token
    const int32_t *ids;       // [T][k] ascending, kNoColumn past the last
    const float *shares;      // [T][k], NULL = 1
    int32_t k;
    float scale;              // log2(e) / h
    float *part_max, *part_sum, *part_hit;   // loss: [column tile][pitch]
    const float *row_lse, *row_scale;        // dz: [n], lse log2(e) and the row's factor
    void *out;                // dz, or a gradient
    int64_t out_pitch;        // elements
    int32_t wide;             // rows of out are 16-byte aligned
    float *sums;              // grad hidden: [column][pitch], over the pieces so far
    int32_t first, last;      // piece
    const float *unit;        // gradients: factor of the results
};

__device__ __forceinline__ uint32_t shared_address(const void *p) { return uint32_t(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ uint32_t block_in_pair() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
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
__device__ __forceinline__ void arrive_at_first(uint64_t *b) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_first(shared_address(b)))
                 : "memory");
}
__device__ __forceinline__ bool barrier_try(uint32_t address, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
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
constexpr uint64_t kPatience = 2000000000;   // a tile takes well under a millisecond

// Waits for the barrier's phase; false when it did not come in `patience` nanoseconds.  A role whose wait gave
// up waits for nothing more, and the results that it did not see are NaN.
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

// Sums in 32 bits, the operands' type and direction, 256 x 256 results.
template <typename T, bool A_ALONG, bool B_ALONG>
constexpr uint32_t kInstruction = 1u << 4 | uint32_t(std::is_same<T, __nv_bfloat16>::value) << 7 |
                                  uint32_t(std::is_same<T, __nv_bfloat16>::value) << 10 | uint32_t(!A_ALONG) << 15 |
                                  uint32_t(!B_ALONG) << 16 | uint32_t(kTile >> 3) << 17 | uint32_t(kTile >> 4) << 24;

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

template <typename T> __device__ __forceinline__ uint32_t pack_two(float low, float high);
template <> __device__ __forceinline__ uint32_t pack_two<__nv_bfloat16>(float low, float high) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(low, high);
    return reinterpret_cast<const uint32_t &>(v);
}
template <> __device__ __forceinline__ uint32_t pack_two<__half>(float low, float high) {
    const __half2 v = __floats2half2_rn(low, high);
    return reinterpret_cast<const uint32_t &>(v);
}

// The tiles in the order in which they are taken: groups of kGroup row tiles, column by column.
struct Tiles {
    int rows, cols;
    __device__ __forceinline__ void at(int i, int &row, int &col) const {
        const int per = kGroup * cols, g = i / per, left = i - g * per;
        const int high = min(kGroup, rows - g * kGroup);
        col = left / high;
        row = g * kGroup + left - col * high;
    }
};

// A token's targets from a column on, in ascending order.
struct Targets {
    const int32_t *id;
    const float *share;
    int j, k, next;
    __device__ __forceinline__ void start(const GemmArgs &a, int token, int col) {
        k = token < 0 ? 0 : a.k;
        id = a.ids + int64_t(token < 0 ? 0 : token) * a.k;
        share = a.shares ? a.shares + int64_t(token < 0 ? 0 : token) * a.k : nullptr;
        int low = 0, high = k;   // the first id >= col
        while (low < high) {
            const int mid = (low + high) >> 1;
            if (id[mid] < col) low = mid + 1;
            else high = mid;
        }
        j = low;
        next = j < k ? id[j] : kNoColumn;
    }
    __device__ __forceinline__ float weight() const { return share ? share[j] : 1.0f; }
    __device__ __forceinline__ void advance() { next = ++j < k ? id[j] : kNoColumn; }
};

// 64 results of each of the warp's 32 rows, through shared memory so that a row's are written together.
// `to`: where this lane's row goes, or NULL where nothing is written; `left`: columns that exist from here on.
template <typename T>
__device__ __forceinline__ void write_rows(const uint32_t (&packed)[32], unsigned char *staging, T *to, int left,
                                           bool wide, int lane) {
    uint4 *mine = reinterpret_cast<uint4 *>(staging) + lane * 8;
#pragma unroll
    for (int u = 0; u < 8; u++)
        mine[u ^ (lane & 7)] = make_uint4(packed[4 * u], packed[4 * u + 1], packed[4 * u + 2], packed[4 * u + 3]);
    __syncwarp();
    const uint64_t row = reinterpret_cast<uint64_t>(to);
    const int unit = lane & 7;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int r = 4 * i + (lane >> 3);
        T *p = reinterpret_cast<T *>(__shfl_sync(0xffffffffu, row, r));
        const uint4 v = reinterpret_cast<const uint4 *>(staging)[r * 8 + (unit ^ (r & 7))];
        const int rest = left - 8 * unit;
        if (p && rest > 0) {
            p += 8 * unit;
            if (wide && rest >= 8) {
                *reinterpret_cast<uint4 *>(p) = v;
            } else {
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                uint16_t *h = reinterpret_cast<uint16_t *>(p);
#pragma unroll
                for (int e = 0; e < 8; e++)
                    if (e < rest) h[e] = uint16_t(w[e >> 1] >> (16 * (e & 1)));
            }
        }
    }
    __syncwarp();
}

template <Product P, typename T>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, GemmArgs a) {
    // operands whose rows in memory run along the summed index
    constexpr bool kAAlong = P != kGradWeight, kBAlong = P == kLoss || P == kDz;
    extern __shared__ unsigned char raw[];
    unsigned char *base = raw + ((1024 - (shared_address(raw) & 1023)) & 1023);   // the swizzle's alignment
    unsigned char *staging = base + kStages * kStage;
    Shared &sh = *reinterpret_cast<Shared *>(staging + kEpilogueWarps * kStaging);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t half = block_in_pair();

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; i++) {
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
    pdl_wait();
    pdl_trigger();

    const uint32_t tmem = sh.tmem;
    const int n = *a.live;
    const int m = P == kGradWeight ? a.m : n;
    const int steps = ((P == kGradWeight ? n : a.depth) + kDepth - 1) / kDepth;
    const Tiles tiles = {(m + kTile - 1) / kTile, (a.cols + kTile - 1) / kTile};
    const int count = tiles.rows * tiles.cols, pair = int(blockIdx.x >> 1), pairs = int(gridDim.x >> 1);

    if (warp == 0 && lane == 0) {
        int s = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int i = pair; ok && i < count; i += pairs) {
            int row, col;
            tiles.at(i, row, col);
            const int y = row * kTile + int(half) * kHalf, x = col * kTile + int(half) * kHalf;
            for (int kb = 0; kb < steps; kb++) {
                ok = barrier_wait(&sh.empty[s], phase ^ 1);
                if (!ok) break;
                const uint32_t to = shared_address(base + s * kStage), bar = in_first(shared_address(&sh.full[s]));
                if (half == 0) barrier_expect(&sh.full[s], 2 * kStage);
                if constexpr (kAAlong) {
                    load_box(&map_a, to, bar, kb * kDepth, y);
                } else {
                    load_box(&map_a, to, bar, y, kb * kDepth);
                    load_box(&map_a, to + kOperand / 2, bar, y + 64, kb * kDepth);
                }
                if constexpr (kBAlong) {
                    load_box(&map_b, to + kOperand, bar, kb * kDepth, a.first_col + x);
                } else {   // grad hidden: the piece's rows of the weights; grad weight: tokens
                    const int r = (P == kGradHidden ? a.first_col : 0) + kb * kDepth;
                    load_box(&map_b, to + kOperand, bar, x, r);
                    load_box(&map_b, to + kOperand + kOperand / 2, bar, x + 64, r);
                }
                if (++s == kStages) s = 0, phase ^= 1;
            }
        }
        if (!ok) {   // copies under way end within microseconds: those of the stages that are still open
            for (int i = 0; i < kStages && half == 0; i++)
                barrier_wait_long(shared_address(&sh.full[i]), i < s ? phase : phase ^ 1, 1000000);
            const uint64_t start = nanoseconds();
            while (nanoseconds() - start < 10000000) __nanosleep(1000);
        }
    } else if (warp == 1 && lane == 0 && half == 0) {
        constexpr uint32_t how = kInstruction<T, kAAlong, kBAlong>;
        int s = 0, use = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int i = pair; ok && i < count && steps; i += pairs, use++) {
            const int acc = use & 1;
            ok = barrier_wait(&sh.free_[acc], ((use >> 1) & 1) ^ 1);
            if (!ok) break;
            fence_after();
            for (int kb = 0; kb < steps; kb++) {
                ok = barrier_wait(&sh.full[s], phase);
                if (!ok) break;
                fence_after();
                const uint32_t at = shared_address(base + s * kStage);
                const uint64_t da = descriptor<kAAlong>(at), db = descriptor<kBAlong>(at + kOperand);
#pragma unroll
                for (int q = 0; q < kDepth / 16; q++)
                    multiply(tmem + acc * kTile, da + q * kStep<kAAlong>, db + q * kStep<kBAlong>, how, kb | q);
                commit(&sh.empty[s]);
                if (++s == kStages) s = 0, phase ^= 1;
            }
            if (ok) commit(&sh.done[acc]);
        }
        if (!ok) {
            commit(&sh.drain);
            barrier_wait(&sh.drain, 0);
        }
    } else if (warp >= 2) {
        const int quarter = warp & 3;   // the lanes of tensor memory that this warp may read
        unsigned char *mine = staging + quarter * kStaging;
        const int local = int(half) * kHalf + quarter * 32 + lane;
        const float unit = P == kGradHidden || P == kGradWeight ? *a.unit : 1.0f;
        const float nan = __int_as_float(0x7fc00000);
        bool ok = true;
        int use = 0;
        for (int i = pair; i < count; i += pairs, use++) {
            int row, col;
            tiles.at(i, row, col);
            const int acc = use & 1, r = row * kTile + local, c0 = col * kTile;
            const bool there = r < m;
            const uint32_t from = tmem + acc * kTile + (uint32_t(quarter * 32) << 16);
            int token = -1;
            if constexpr (P != kGradWeight) token = there ? a.rows[r] : -1;
            Targets hits;
            float lse = 0.0f, factor = 0.0f;
            if constexpr (P == kLoss) hits.start(a, token, c0);
            if constexpr (P == kDz) {
                hits.start(a, token, a.first_col + c0);
                if (there) lse = a.row_lse[r], factor = a.row_scale[r];
            }
            if (steps) ok = ok && barrier_wait(&sh.done[acc], (use >> 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            fence_after();

            if constexpr (P == kLoss) {
                float top = -INFINITY, sum = 0.0f, hit = 0.0f;
                const int chunks = min(kTile, a.cols - c0 + 31) / 32;
#pragma unroll 1
                for (int c = 0; c < chunks; c++) {
                    float v[32];
                    read_columns(v, from + c * 32);
                    reads_wait();
                    const int at = c0 + c * 32;
                    while (hits.next < at + 32) {
                        float z = 0.0f;
#pragma unroll
                        for (int e = 0; e < 32; e++) z = e == hits.next - at ? v[e] : z;
                        hit = fmaf(hits.weight(), z, hit);
                        hits.advance();
                    }
                    __syncwarp();
                    if (at + 32 > a.cols) {
#pragma unroll
                        for (int e = 0; e < 32; e++) v[e] = at + e < a.cols ? v[e] : -INFINITY;
                    }
                    float t[4] = {top, top, top, top};
#pragma unroll
                    for (int e = 0; e < 32; e++) t[e & 3] = fmaxf(t[e & 3], v[e]);
                    const float high = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
                    const float off = high * a.scale;
                    float u[4] = {sum * exp2_fast(fmaf(top, a.scale, -off)), 0.0f, 0.0f, 0.0f};
                    if (top == -INFINITY) u[0] = 0.0f;   // nothing yet
#pragma unroll
                    for (int e = 0; e < 32; e++) u[e & 3] += exp2_fast(fmaf(v[e], a.scale, -off));
                    sum = (u[0] + u[1]) + (u[2] + u[3]);
                    top = high;
                }
                fence_before();
                __syncwarp();
                if (lane == 0 && steps) arrive_at_first(&sh.free_[acc]);
                if (there) {
                    const int64_t at = int64_t(col) * a.pitch + r;
                    a.part_max[at] = top;
                    a.part_sum[at] = ok ? sum : nan;
                    a.part_hit[at] = hit;
                }
            } else {
                T *to = nullptr;
                if constexpr (P == kDz) to = static_cast<T *>(a.out) + int64_t(r) * a.out_pitch;
                if constexpr (P == kGradWeight)
                    if (there) to = static_cast<T *>(a.out) + int64_t(r) * a.out_pitch;
                if constexpr (P == kGradHidden)
                    if (there) to = static_cast<T *>(a.out) + int64_t(token) * a.out_pitch;
                const int chunks = P == kDz ? kTile / 64 : min(kTile, a.cols - c0 + 63) / 64;
#pragma unroll 1
                for (int c = 0; c < chunks; c++) {
                    float v[2][32];
                    if (steps) {
                        read_columns(v[0], from + c * 64);
                        read_columns(v[1], from + c * 64 + 32);
                        reads_wait();
                    }
                    const int at = c0 + c * 64;
                    if (!ok || !steps) {
#pragma unroll
                        for (int e = 0; e < 64; e++) v[e >> 5][e & 31] = ok ? 0.0f : nan;
                    }
                    if constexpr (P == kDz) {
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            const int here = at + 32 * h, column = a.first_col + here;
#pragma unroll
                            for (int e = 0; e < 32; e++) v[h][e] = exp2_fast(fmaf(v[h][e], a.scale, -lse));
                            while (hits.next < column + 32) {
                                const float q = hits.weight();
#pragma unroll
                                for (int e = 0; e < 32; e++) v[h][e] -= e == hits.next - column ? q : 0.0f;
                                hits.advance();
                            }
                            __syncwarp();
                            // rows past the last and columns past the vocabulary enter later sums: zeros
                            if (!there || here + 32 > a.cols) {
#pragma unroll
                                for (int e = 0; e < 32; e++)
                                    v[h][e] = there && here + e < a.cols ? v[h][e] * factor : 0.0f;
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; e++) v[h][e] *= factor;
                            }
                        }
                    }
                    if constexpr (P == kGradHidden) {
                        if (!a.first && there) {
#pragma unroll
                            for (int e = 0; e < 64; e++)
                                if (at + e < a.cols) v[e >> 5][e & 31] += a.sums[int64_t(at + e) * a.pitch + r];
                        }
                        if (!a.last) {
                            if (there) {
#pragma unroll
                                for (int e = 0; e < 64; e++)
                                    if (at + e < a.cols) a.sums[int64_t(at + e) * a.pitch + r] = v[e >> 5][e & 31];
                            }
                            __syncwarp();
                            continue;
                        }
                    }
                    uint32_t packed[32];
#pragma unroll
                    for (int e = 0; e < 32; e++) {
                        float low = v[e >> 4][(2 * e) & 31], high = v[e >> 4][(2 * e + 1) & 31];
                        if constexpr (P != kDz) low *= unit, high *= unit;
                        packed[e] = pack_two<T>(low, high);
                    }
                    write_rows<T>(packed, mine, to ? to + at : nullptr, P == kDz ? kTile : a.cols - at, a.wide, lane);
                }
                fence_before();
                __syncwarp();
                if (lane == 0 && steps) arrive_at_first(&sh.free_[acc]);
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
int launch_gemm_bf16(Product p, const CUtensorMap &a, const CUtensorMap &b, const GemmArgs &args, int pairs,
                     void *stream);
int launch_gemm_f16(Product p, const CUtensorMap &a, const CUtensorMap &b, const GemmArgs &args, int pairs,
                    void *stream);

template <typename T>
int launch_gemm(Product p, const CUtensorMap &ma, const CUtensorMap &mb, const GemmArgs &args, int pairs,
                void *stream) {
    auto go = [&](auto product, const char *what) {
        constexpr Product P = decltype(product)::value;
        if (const int rc = allow<gemm_kernel<P, T>>(kSharedBytes, what)) return rc;
        return launch_kernel(gemm_kernel<P, T>, dim3(2 * pairs), dim3(kThreads), kSharedBytes, stream, 1, what, ma, mb,
                             args);
    };
    switch (p) {
        case kLoss: return go(std::integral_constant<Product, kLoss>{}, "head loss launch");
        case kDz: return go(std::integral_constant<Product, kDz>{}, "head dz launch");
        case kGradHidden: return go(std::integral_constant<Product, kGradHidden>{}, "head grad hidden launch");
        default: return go(std::integral_constant<Product, kGradWeight>{}, "head grad weight launch");
    }
}

}  // namespace head
}  // namespace nest
