// The optimizer's operators over lists of tensors: gradient norm and AdamW step, with
// moments in 32 or in 8 bits (definitions in nest_train.h).
//
// The list's blocks of 256 elements are divided evenly between workers, each of them a thread
// block; a worker's blocks are a few segments, each of one tensor, and its warps take every
// kWarps-th of them, a warp a whole block.  The packed table holds the tensors' entries, the
// segments in order and where each worker's begin.
#include <cmath>
#include <cstring>

#include "nest_train.cuh"

namespace nest {

namespace {

constexpr int kBlock = NEST_OPT_BLOCK;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kWorkers = kSMs * 8;   // at most: the norm's thread blocks are all resident at once

struct Entry {            // one tensor
    void *weight;
    const void *grad;
    int64_t numel;
    int64_t first;        // its first block in the list's buffers
    float weight_decay, lr_scale;
    int64_t pad;
};
struct Segment {
    int32_t tensor, block, count;   // blocks [block, block + count) of the tensor
    int32_t before;                 // the worker's blocks in earlier segments
};
static_assert(sizeof(Entry) == 48 && sizeof(Segment) == 16, "table layout");

struct Table {
    const Entry *entries;
    const Segment *segments;
    const int32_t *starts;   // [workers + 1]
};
Table table_of(const void *table, const nest_table_info *info) {
    const Entry *e = static_cast<const Entry *>(table);
    const Segment *s = reinterpret_cast<const Segment *>(e + info->tensors);
    return {e, s, reinterpret_cast<const int32_t *>(s + info->items)};
}
int64_t table_bytes(int64_t tensors, int64_t segments, int64_t workers) {
    return int64_t(sizeof(Entry)) * tensors + int64_t(sizeof(Segment)) * segments + 4 * (workers + 1);
}

// The segments of a thread block's workers, 32 at a time, one per lane.
struct Segments {
    int from, to;
    Segment lane_s;
    __device__ __forceinline__ void fetch(const Table &t) {
        const int at = from + (threadIdx.x & 31);
        lane_s = at < to ? t.segments[at] : Segment{0, 0, 0, 0};
    }
    __device__ __forceinline__ Segments(const Table &t, int worker, int workers) {
        from = worker < workers ? t.starts[worker] : 0;
        to = worker < workers ? t.starts[worker + 1] : 0;
        fetch(t);
    }
    // fn(entry, first, count) for each segment in which the warp has blocks: the first one in the
    // tensor, and how many, `warps` (a power of two) apart; warp: its number among those that
    // share the worker.
    template <typename F>
    __device__ __forceinline__ void each(const Table &t, int warp, int warps, F fn) {
        while (from < to) {
            const Segment all = lane_s;
            from += 32;
            if (from < to) fetch(t);
            const int own = (warp - all.before) & (warps - 1);   // the warp's first block in the segment
            uint32_t with = __ballot_sync(0xffffffffu, own < all.count);
            while (with) {
                const int j = __ffs(with) - 1;
                with &= with - 1;
                const int skip = __shfl_sync(0xffffffffu, own, j), block = __shfl_sync(0xffffffffu, all.block, j);
                const int count = __shfl_sync(0xffffffffu, all.count, j);
                fn(t.entries[__shfl_sync(0xffffffffu, all.tensor, j)], block + skip, (count - skip + warps - 1) / warps);
            }
        }
    }
};

int64_t blocks_in(int64_t numel) { return (numel + kBlock - 1) / kBlock; }

// A lane's share of a block: elements 8 lane .. 8 lane + 7, in one access of 32 bytes (or 16).
// Values stay as they were read until all of a block's loads are under way.
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                 : "l"(p)
                 : "memory");
}
template <typename T>
__device__ __forceinline__ void load8(const T *p, T (&x)[8]) {
    static_assert(sizeof(T) == 2, "16-bit type");
    *reinterpret_cast<uint4 *>(x) = *reinterpret_cast<const uint4 *>(p);
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
    alignas(16) T h[8];
#pragma unroll
    for (int i = 0; i < 8; i++) h[i] = from_f32<T>(x[i]);
    *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(h);
}

template <typename T>
__device__ __forceinline__ bool wide(const T *p) {   // every block of the tensor can be loaded by load8
    return (reinterpret_cast<uintptr_t>(p) & (8 * sizeof(T) - 1)) == 0;
}

// The lane's share of the block that starts at p[0], of which `n` elements (1 to 256) exist; the
// others are 0.  A tensor that does not start at a multiple of 8 elements, and a tensor's last
// block, go through the warp's shared memory: 32 neighbours at a time between it and the tensor.
template <typename T>
__device__ __forceinline__ void load_block(const T *p, int n, bool vector, int lane, float *room, T (&x)[8]) {
    if (vector && n >= kBlock) {
        load8(p + 8 * lane, x);
        return;
    }
    T *own = reinterpret_cast<T *>(room);
    T part[8];
#pragma unroll
    for (int i = 0; i < 8; i++) part[i] = lane + 32 * i < n ? p[lane + 32 * i] : from_f32<T>(0.0f);
#pragma unroll
    for (int i = 0; i < 8; i++) own[lane + 32 * i] = part[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = own[8 * lane + i];
    __syncwarp();
}
template <typename T>
__device__ __forceinline__ void store_block(T *p, int n, bool vector, int lane, float *room, const float (&x)[8]) {
    if (vector && n >= kBlock) {
        store8(p + 8 * lane, x);
        return;
    }
    T *own = reinterpret_cast<T *>(room);
#pragma unroll
    for (int i = 0; i < 8; i++) own[8 * lane + i] = from_f32<T>(x[i]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; i++)
        if (lane + 32 * i < n) p[lane + 32 * i] = own[lane + 32 * i];
    __syncwarp();
}

// ---- gradient norm ----------------------------------------------------------------

// A sum in 32 bits with the rounding error of every addition added up beside it (Knuth's
// exact sum of two numbers).  64-bit additions are many times slower here: with one for every 16
// values of a thread the norm of 201M values takes 64.4 us against 62.6.
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

// The norm.  Every gradient is read once, two blocks of a warp under way at a time; memory bounds it.
// Measured: 201M values in 16 bits 63 us, 6.4 TB/s (a flat loop over one buffer 59 us); the
// smallest lists 3.6 us.  All thread blocks of a long list are resident at once: with six times
// as many 73 us.
constexpr int kNormsPerSm = 8;

template <typename T>
__global__ void __launch_bounds__(kThreads, kNormsPerSm) norm_kernel(Table table, int workers, uint32_t *ticket,
                                                                     float *part, float max_norm, float *out) {
    __shared__ float sh[kWarps];
    __shared__ bool done;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sum sum;
    Segments(table, blockIdx.x, workers).each(table, warp, kWarps, [&](const Entry &e, int block, int count) {
        // a tensor off alignment is read from the aligned address before it on, `off` elements early:
        // its first block lacks them, and its last one has as many more
        const T *g = static_cast<const T *>(e.grad);
        const int off = int(reinterpret_cast<uintptr_t>(g) / sizeof(T) & 7), last = int((e.numel - 1) / kBlock);
        const int64_t end = e.numel + off;
        g -= off;
        while (count > 0) {
            float s = 0.0f;
            const int64_t at = int64_t(block) * kBlock;
            const bool begun = block > 0 || off == 0;
            if (begun && count > 1 && block + kWarps < last) {   // two blocks' loads at once
                alignas(16) T x[8], y[8];
                load8(g + at + 8 * lane, x);
                load8(g + at + kWarps * kBlock + 8 * lane, y);
#pragma unroll
                for (int i = 0; i < 8; i++) s = fmaf(to_f32(x[i]), to_f32(x[i]), s);
#pragma unroll
                for (int i = 0; i < 8; i++) s = fmaf(to_f32(y[i]), to_f32(y[i]), s);
                count--;
                block += kWarps;
            } else if (begun && block < last) {
                alignas(16) T x[8];
                load8(g + at + 8 * lane, x);
#pragma unroll
                for (int i = 0; i < 8; i++) s = fmaf(to_f32(x[i]), to_f32(x[i]), s);
            } else {
                const int64_t stop = block < last ? at + kBlock : end;
                T x[kBlock / 32 + 1];
#pragma unroll
                for (int c = 0; c <= kBlock / 32; c++) {
                    const int64_t i = at + lane + 32 * c;
                    x[c] = i >= off && i < stop ? g[i] : from_f32<T>(0.0f);
                }
#pragma unroll
                for (int c = 0; c <= kBlock / 32; c++) s = fmaf(to_f32(x[c]), to_f32(x[c]), s);
            }
            sum.add(s);
            count--;
            block += kWarps;
        }
    });
    const float own = block_sum(sum.value(), sh);
    if (threadIdx.x == 0) {
        part[blockIdx.x] = own;
        done = last_ticket(ticket, gridDim.x);
    }
    __syncthreads();
    if (!done) return;
    // the last block adds what all have written
    Sum total;
#pragma unroll 8
    for (int b = threadIdx.x; b < int(gridDim.x); b += kThreads) total.add(__ldcg(part + b));
    const float s = block_sum(total.value(), sh);
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

// Codes of a lane's eight pairs of moments; word: the block's noise.  A moment is scaled so that
// the smallest normal code becomes the smallest normal 32-bit number: then exponent field and
// upper three mantissa bits of either kind, normal or not, are the code, and adding 16 bits of
// noise under them and cutting off the rest rounds it.  RARE: the block holds a moment that is
// not finite, or a scale that is clipped or does not fit one factor.
template <bool RARE>
__device__ __forceinline__ void encode(const float (&m)[8], const float (&v)[8], int sm, int sv, uint32_t word,
                                       int lane, uint2 &cm, uint2 &cv) {
    const float fm = power2(RARE ? 8 - sm : -112 - sm), fv = power2(RARE ? -1 - sv : -96 - sv);
    uint32_t a[8], b[8];   // the codes in the upper byte
    word += 8 * lane * 0x9E3779B1u;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        uint32_t x = word + i * 0x9E3779B1u;
        x ^= x >> 15;
        x *= 0x6A09E667u;
        x ^= x >> 16;
        float ym = fabsf(m[i]) * fm, yv = v[i] * fv;
        if (RARE) {
            ym *= 0x1p-120f;
            yv *= 0x1p-95f;
        }
        uint32_t bm = __float_as_uint(ym), bv = __float_as_uint(yv);
        if (RARE) {
            bm = isfinite(m[i]) ? min(bm, 0x7Eu << 20) : 0x7Fu << 20;
            bv = isfinite(v[i]) ? min(bv, 0xFEu << 20) : 0xFFu << 20;
        }
        // added, then moved up: with the product by 16 first, nvcc 13.0.88 drops the scaled bits
        a[i] = (bm + (x >> 12 & 0xFFFF0u)) << 4;
        b[i] = (bv + (x << 4 & 0xFFFF0u)) << 4;
        a[i] = (a[i] & 0x7FFFFFFFu) | (__float_as_uint(m[i]) & 0x80000000u);
    }
    const auto pack = [](const uint32_t *c) {   // the upper bytes of four words
        return __byte_perm(__byte_perm(c[0], c[1], 0x0073), __byte_perm(c[2], c[3], 0x0073), 0x5410);
    };
    cm = make_uint2(pack(a), pack(a + 4));
    cv = make_uint2(pack(b), pack(b + 4));
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
    const float f = power2(min(s + 96, 127));
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = __uint_as_float(((i < 4 ? c.x : c.y) >> (8 * (i & 3)) & 0xFFu) << 20) * f;
    if (s > 31) {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] *= power2(s - 31);
    }
    if (__vcmpeq4(c.x, 0xFFFFFFFFu) | __vcmpeq4(c.y, 0xFFFFFFFFu)) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (((i < 4 ? c.x : c.y) >> (8 * (i & 3)) & 0xFFu) == 0xFFu) v[i] = NAN;
    }
}

// ---- AdamW --------------------------------------------------------------------------

constexpr int kParts = 8, kPartsEight = 4;   // thread blocks to a worker of a long list
constexpr int kStepsPerSm = 3;   // thread blocks: up to 80 registers a thread

struct StepArgs {
    Table table;
    int workers, parts;   // parts: thread blocks that share a worker, a power of two
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
__device__ __forceinline__ float inverse_of(float x) {   // relative error 2^-23; 0 above 2^126
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float larger(float a, float b) {   // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
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

// What a warp needs of a block whose moments are in 8 bits, as it lies in memory.  The codes'
// decoding and encoding leave too few warps on an SM to cover the memory's latency with one
// block each, so blocks are copied ahead.
constexpr int kAhead = 3;
template <typename G>
struct Stage {
    static constexpr int kG = 16 / sizeof(G);
    alignas(16) G grad[kBlock + kG];   // from an aligned address on
    alignas(16) float master[kBlock];
    alignas(16) uint8_t m[kBlock], v[kBlock];

    // g: aligned; with off > 0 the block's gradients start `off` elements later.
    __device__ __forceinline__ void copy(const G *g, int off, const float *p, const uint8_t *cm, const uint8_t *cv,
                                         int lane) {
#pragma unroll
        for (int i = kG * lane; i < kBlock; i += 32 * kG) copy_ahead<16>(grad + i, g + i);   // neighbours by neighbours
        if (off && lane == 0) copy_ahead<16>(grad + kBlock, g + kBlock);
#pragma unroll
        for (int i = 4 * lane; i < kBlock; i += 32 * 4) copy_ahead<16>(master + i, p + i);
        copy_ahead<8>(m + 8 * lane, cm + 8 * lane);
        copy_ahead<8>(v + 8 * lane, cv + 8 * lane);
    }
    __device__ __forceinline__ void read(int off, G (&g)[8], float (&p)[8], uint2 &cm, uint2 &cv, int lane) const {
        if (off == 0) {
#pragma unroll
            for (int i = 0; i < int(sizeof(G) / 2); i++)
                reinterpret_cast<uint4 *>(g)[i] = reinterpret_cast<const uint4 *>(grad + 8 * lane)[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) g[i] = grad[off + 8 * lane + i];
        }
#pragma unroll
        for (int i = 0; i < 2; i++)
            reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(master + 8 * lane)[i];
        cm = *reinterpret_cast<const uint2 *>(m + 8 * lane);
        cv = *reinterpret_cast<const uint2 *>(v + 8 * lane);
    }
};

// Magnitudes of m and v (as bits) from which a block's codes take the checked path: 1.75 * 2^14
// and 1.75 * 2^30, above which the scale is no single factor; infinity; NaN.
constexpr uint32_t kRareM = (uint32_t(14 + 127) << 23) | 0x600000u, kRareV = (uint32_t(30 + 127) << 23) | 0x600000u;

// The step.  Memory bounds it: 28 bytes a weight with 16-bit weights and gradients and moments in
// 32 bits, 16 with moments in 8 bits.  Measured over 201M weights, 32 bits: 820 us, 6.9 TB/s
// (839 with one thread block per worker); 8 bits: 498 us, 6.5 TB/s (537 with one, and 544 with
// 8 instead of 4; 504 with a lane's copies side by side instead of 32 lanes').  Three thread blocks
// to an SM, up to 80 registers: with four the 32-bit step takes 824 us, the 8-bit one the same.
template <typename W, typename G, bool EIGHT>
__global__ void __launch_bounds__(kThreads, kStepsPerSm) adamw_kernel(StepArgs a) {
    constexpr bool kOwnMaster = sizeof(W) == 4;
    __shared__ __align__(16) float room[kWarps][kBlock];
    extern __shared__ __align__(16) unsigned char sh[];
    __shared__ struct {
        float scale, root, eps;
        uint32_t start;
    } shared;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int step = kWarps * a.parts;   // between a warp's blocks
    Segments segments(a.table, blockIdx.x / a.parts, a.workers);   // under way with the step's state
    if (threadIdx.x == 0) {   // what all share, by one thread: 64-bit arithmetic is slow
        const nest_adamw_state st = *a.state;
        shared.scale = a.grad_scale ? *a.grad_scale : 1.0f;
        // m / c1 / (sqrt(v / c2) + eps) = m / (sqrt(v) c1 / sqrt(c2) + c1 eps)
        const float c1 = float(1.0 - st.beta1_t * a.beta1d);
        shared.root = c1 * rsqrtf(float(1.0 - st.beta2_t * a.beta2d));
        shared.eps = c1 * a.eps;
        shared.start = mixed(a.seed ^ mixed(uint32_t(st.step + 1)));
    }
    __syncthreads();
    const float scale = shared.scale, root = shared.root, eps = shared.eps;
    const uint32_t start = shared.start;
    if (!isfinite(scale)) return;
    // says that this block has read the step's state; the last block to say so advances it at
    // its end, when the answer has long arrived
    uint32_t before = 0;
    if (threadIdx.x == 0) {
        __threadfence();
        before = atomicAdd(&a.state->ticket, 1u);
    }
    segments.each(a.table, blockIdx.x % a.parts * kWarps + warp, step, [&](const Entry &e, int b, int count) {
        W *weight = static_cast<W *>(e.weight);
        const G *grad = static_cast<const G *>(e.grad);
        const bool wide_w = wide(weight), wide_g = wide(grad);
        const float lr = a.lr * e.lr_scale, decay = e.weight_decay;
        using S = Stage<G>;
        S *const stages = reinterpret_cast<S *>(sh) + warp * (kAhead + 1);
        // the warp's whole blocks here are copied ahead, gradients off alignment from the aligned
        // address before them: not a tensor's first block then, and only as far as it goes; a single
        // block has nothing to be ahead of
        const int off = int(reinterpret_cast<uintptr_t>(grad) / sizeof(G) % S::kG);
        const int64_t past = (off ? e.numel + off - S::kG : e.numel) / kBlock - b;
        const int whole = EIGHT && count > 1 && (!kOwnMaster || wide_w) && past > 0
                              ? int(past < int64_t(count) * step ? (past + step - 1) / step : count) : 0;
        const int from = off && b == 0;
        auto ahead = [&](int i) {
            if (i >= from && i < whole) {
                const int64_t j = int64_t(b + i * step) * kBlock, own = e.first * kBlock + j;
                const float *p;
                if constexpr (kOwnMaster)
                    p = weight + j;
                else
                    p = a.master + own;
                stages[i % (kAhead + 1)].copy(grad - off + j, off, p, static_cast<const uint8_t *>(a.m) + own,
                                              static_cast<const uint8_t *>(a.v) + own, lane);
            }
            copies_mark();
        };
        if constexpr (EIGHT) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kAhead; i++) ahead(i);
        }
        int lane_sm = 0, lane_sv = 0;   // scales of the warp's next 32 blocks, one per lane
        for (int k = 0; k < count; k++) {
            const int64_t bk = b + k * step, j0 = bk * kBlock, left = e.numel - j0;
            const int n = int(left < kBlock ? left : kBlock);
            const int64_t block = e.first + bk, at = block * kBlock;
            alignas(16) G g[8];
            alignas(16) float p[8];
            float m[8], v[8];
            uint2 cm, cv;
            int sm, sv;
            if constexpr (EIGHT) {
                if (k % 32 == 0 && k + lane < count) {
                    lane_sm = a.m_exp[block + lane * step];
                    lane_sv = a.v_exp[block + lane * step];
                }
                __syncwarp();   // the block before is read, and its place free
                ahead(k + kAhead);
                sm = __shfl_sync(0xffffffffu, lane_sm, k % 32);
                sv = __shfl_sync(0xffffffffu, lane_sv, k % 32);
            }
            if (EIGHT && k >= from && k < whole) {
                copies_wait<kAhead>();
                __syncwarp();
                stages[k % (kAhead + 1)].read(off, g, p, cm, cv, lane);
            } else {
                load_block(grad + j0, n, wide_g, lane, room[warp], g);
                if constexpr (EIGHT) {
                    cm = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.m) + at + 8 * lane);
                    cv = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.v) + at + 8 * lane);
                } else {
                    load8(static_cast<const float *>(a.m) + at + 8 * lane, m);
                    load8(static_cast<const float *>(a.v) + at + 8 * lane, v);
                }
                if constexpr (kOwnMaster)
                    load_block(weight + j0, n, wide_w, lane, room[warp], p);
                else
                    load8(a.master + at + 8 * lane, p);   // the list's own buffers hold whole blocks
            }
            if constexpr (EIGHT) {
                decode_m(cm, sm, m);
                decode_v(cv, sv, v);
            }
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float x = to_f32(g[i]) * scale;
                // each product rounded by itself, so that a moment is the same number wherever
                // these formulas are evaluated, and its 8-bit code with it
                m[i] = __fadd_rn(__fmul_rn(m[i], a.beta1), __fmul_rn(x, a.rest1));
                v[i] = __fadd_rn(__fmul_rn(v[i], a.beta2), __fmul_rn(__fmul_rn(x, x), a.rest2));
                p[i] -= lr * fmaf(decay, p[i], m[i] * inverse_of(fmaf(root_of(v[i]), root, eps)));
            }
            store_block(weight + j0, n, wide_w, lane, room[warp], p);
            if constexpr (!kOwnMaster) store_own(a.master + at, n, lane, p);
            if constexpr (EIGHT) {
                float top_m = 0.0f, top_v = 0.0f;
                if (n < kBlock) {   // what lies past the end has no say in the scale
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        if (8 * lane + i >= n) m[i] = v[i] = 0.0f;
                }
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    top_m = larger(top_m, fabsf(m[i]));
                    top_v = larger(top_v, v[i]);
                }
                uint32_t bits_m = __reduce_max_sync(0xffffffffu, __float_as_uint(top_m));
                uint32_t bits_v = __reduce_max_sync(0xffffffffu, __float_as_uint(top_v));
                const bool rare = bits_m >= kRareM || bits_v >= kRareV;
                if (rare) {   // the largest finite magnitudes
                    bits_m = bits_v = 0;
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        bits_m = max(bits_m, finite_bits(m[i]));
                        bits_v = max(bits_v, finite_bits(v[i]));
                    }
                    bits_m = __reduce_max_sync(0xffffffffu, bits_m);
                    bits_v = __reduce_max_sync(0xffffffffu, bits_v);
                }
                sm = shared_exponent(bits_m);
                sv = shared_exponent(bits_v);
                const uint32_t word = mixed(start + uint32_t(block) * 0x9E3779B1u);
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
    });
    if (threadIdx.x == 0 && before == gridDim.x - 1) {
        a.state->beta1_t *= a.beta1d;
        a.state->beta2_t *= a.beta2d;
        a.state->step++;
        a.state->ticket = 0;
    }
}

// The values of 8-bit moments.  201M weights: 191 us, 6.3 TB/s; memory bounds it.
__global__ void __launch_bounds__(kThreads) values_kernel(int64_t blocks, const uint8_t *m, const uint8_t *v,
                                                          const int8_t *m_exp, const int8_t *v_exp,
                                                          __nv_bfloat16 *m_out, __nv_bfloat16 *v_out) {
    pdl_wait();
    pdl_trigger();
    // a warp takes two blocks at a time, half the grid apart in the list
    const int lane = threadIdx.x & 31;
    const int64_t warps = int64_t(gridDim.x) * kWarps;
    for (int64_t b = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> 5; b < blocks; b += 2 * warps) {
        uint2 cm[2], cv[2];
        int sm[2], sv[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int64_t at = b + h * warps;
            if (at >= blocks) break;
            cm[h] = *reinterpret_cast<const uint2 *>(m + at * kBlock + 8 * lane);
            cv[h] = *reinterpret_cast<const uint2 *>(v + at * kBlock + 8 * lane);
            sm[h] = m_exp[at];
            sv[h] = v_exp[at];
        }
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int64_t at = b + h * warps;
            if (at >= blocks) break;
            float x[8];
            decode_m(cm[h], sm[h], x);
            store8(m_out + at * kBlock + 8 * lane, x);
            decode_v(cv[h], sv[h], x);
            store8(v_out + at * kBlock + 8 * lane, x);
        }
    }
}

// ---- host -----------------------------------------------------------------------------

int64_t workers_for(int64_t blocks) {
    const int64_t w = (blocks + kWarps - 1) / kWarps;
    return w < kWorkers ? w : kWorkers;
}

int check_info(const nest_table_info *info) {
    if (!info || info->tensors < 0 || info->blocks < 0 || info->items < 0 || info->items > info->blocks ||
        info->workers != workers_for(info->blocks) ||
        info->table_bytes < table_bytes(info->tensors, info->items, info->workers))
        return NEST_E_INVALID;
    return info->blocks > INT32_MAX ? NEST_E_LIMITS : NEST_OK;
}

// fn(tensor, block, count, before, worker) for every segment in order: worker w has the list's
// blocks [w blocks / workers, (w + 1) blocks / workers).
template <typename F>
void each_segment(const nest_tensor *t, int32_t n, int64_t blocks, F fn) {
    const int64_t workers = workers_for(blocks);
    int64_t done = 0, worker = 0;
    for (int32_t i = 0; i < n; i++) {
        const int64_t size = blocks_in(t[i].numel);
        for (int64_t b = 0; b < size;) {
            int64_t end = (worker + 1) * blocks / workers;
            while (end <= done) end = (++worker + 1) * blocks / workers;
            const int64_t count = size - b < end - done ? size - b : end - done;
            fn(i, int32_t(b), int32_t(count), int32_t(done - worker * blocks / workers), worker);
            b += count;
            done += count;
        }
    }
}

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
        if (blocks > INT32_MAX) return NEST_E_LIMITS;
    }
    each_segment(t, n, blocks, [&](int32_t, int32_t, int32_t, int32_t, int64_t) { items++; });
    out->blocks = blocks;
    out->items = items;
    out->tensors = n;
    out->workers = int32_t(workers_for(blocks));
    out->table_bytes = table_bytes(n, items, out->workers);
    return NEST_OK;
}

int nest_table_pack(const nest_tensor *t, int32_t n, const nest_table_info *info, void *table) {
    nest_table_info need;
    if (const int rc = nest_table_query(t, n, &need)) return rc;
    if (!info || need.tensors != info->tensors || need.items != info->items || need.blocks != info->blocks ||
        need.workers != info->workers || need.table_bytes != info->table_bytes || !table)
        return NEST_E_INVALID;
    unsigned char *at = static_cast<unsigned char *>(table);   // of any alignment
    int64_t first = 0;
    for (int32_t i = 0; i < n; i++, at += sizeof(Entry)) {
        const Entry e = {t[i].weight, t[i].grad, t[i].numel, first, t[i].weight_decay, t[i].lr_scale, 0};
        std::memcpy(at, &e, sizeof e);
        first += blocks_in(t[i].numel);
    }
    unsigned char *starts = at + sizeof(Segment) * size_t(need.items);
    int32_t segment = 0;
    int64_t known = -1;
    each_segment(t, n, need.blocks, [&](int32_t tensor, int32_t block, int32_t count, int32_t before, int64_t worker) {
        for (; known < worker; known++) std::memcpy(starts + 4 * (known + 1), &segment, 4);
        const Segment s = {tensor, block, count, before};
        std::memcpy(at, &s, sizeof s);
        at += sizeof s;
        segment++;
    });
    std::memcpy(starts + 4 * size_t(need.workers), &segment, 4);
    return NEST_OK;
}

size_t nest_grad_norm_workspace_size(const nest_table_info *info) {
    if (check_info(info)) return 0;
    return NEST_TRAIN_TICKET + ((size_t(info->workers + 1) * 4 + 255) & ~size_t(255));
}

int nest_grad_norm(const nest_table_info *info, const void *table, int32_t grad_type, float max_norm, float *out,
                   void *workspace, size_t ws_bytes, void *stream) {
    if (const int rc = check_info(info)) return rc;
    if (!out || !valid_type(grad_type) || !(max_norm > 0.0f) || (info->items && !table) || !aligned_to(table, 16))
        return NEST_E_INVALID;
    if (!workspace || ws_bytes < nest_grad_norm_workspace_size(info) || !aligned_to(workspace, 256))
        return NEST_E_WORKSPACE;
    const int blocks = info->workers > 1 ? info->workers : 1;
    uint32_t *ticket = static_cast<uint32_t *>(workspace);
    float *part = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + NEST_TRAIN_TICKET);
    return with_type(grad_type, [&](auto t) {
        return launch_kernel(norm_kernel<decltype(t)>, dim3(blocks), dim3(kThreads), 0, stream, 1, "norm launch",
                             table_of(table, info), int(info->workers), ticket, part, max_norm, out);
    });
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
    // several thread blocks to a worker of a long list: SMs finish theirs at different times, and
    // the quicker ones take more
    const int most = p->state_bits == 8 ? kPartsEight : kParts;
    const int parts = info->blocks >= int64_t(kWorkers) * kWarps * most ? most : 1;
    const StepArgs a = {table_of(table, info), info->workers, parts, float(p->lr), float(p->beta1), float(p->beta2),
                        float(1.0 - p->beta1), float(1.0 - p->beta2), float(p->eps), p->beta1, p->beta2, p->seed,
                        p->master, p->m, p->v, p->m_exp, p->v_exp, p->state, p->grad_scale};
    const dim3 grid(info->workers > 1 ? info->workers * parts : 1);
    return with_type(p->weight_type, [&](auto w) {
        using W = decltype(w);
        return with_type(p->grad_type, [&](auto g) {
            using G = decltype(g);
            if (p->state_bits == 32)
                return launch_kernel(adamw_kernel<W, G, false>, grid, dim3(kThreads), 0, stream, 1, "adamw launch", a);
            constexpr int kStages = int(sizeof(Stage<G>)) * kWarps * (kAhead + 1);
            const int rc = allow<adamw_kernel<W, G, true>>(kStages, "adamw attribute");
            return rc ? rc
                      : launch_kernel(adamw_kernel<W, G, true>, grid, dim3(kThreads), kStages, stream, 1,
                                      "adamw launch", a);
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
    const int64_t grid_blocks = (info->blocks + 2 * kWarps - 1) / (2 * kWarps);
    const dim3 grid(unsigned(grid_blocks < kSMs * 8 ? grid_blocks : kSMs * 8));
    return launch_kernel(values_kernel, grid, dim3(kThreads), 0, stream, 1, "adamw values launch", info->blocks,
                         static_cast<const uint8_t *>(m), static_cast<const uint8_t *>(v), m_exp, v_exp,
                         static_cast<__nv_bfloat16 *>(m_out), static_cast<__nv_bfloat16 *>(v_out));
}

}  // extern "C"
