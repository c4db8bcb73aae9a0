// Kernels of the routing operators (definitions in nest_train.h), one instantiation per
// element type in nest_route_f32.cu, nest_route_bf16.cu and nest_route_f16.cu.
//
// A warp takes 32 / LANES rows at a time, each held in the registers of LANES lanes, so that the
// logits are read once and what is done per row (reductions, rounds, results) is shared by
// several rows: forward up to 32 values per lane (262144 x 256 in 32 bits, k = 8: 85 us against 104
// with 16 lanes of 16 values), backward, which has little of that, 8 where the row allows (262144 x 64
// in bfloat16, k = 2: 24 us against 78 with a row to a warp).  Logits are read in pieces per lane where
// alignment allows (VEC: those two 85 us against 106 and 24 against 34).
//
// Choice of the k largest.  A logit becomes a 32-bit word whose order is that of the logits,
// with its lowest bits replaced by the complement of the expert's index: all words of a row
// differ, and among logits that agree in the bits kept the lower index is the larger word.
// Each lane sorts its words once and keeps the largest; then k rounds take the maximum over the
// row's lanes, and the lane that had it moves its list up.  16-bit logits lose nothing to the
// index.  With 32-bit logits up to 10 bits are lost, and the word comes from the exponent
// (x - top) log2(e), at most 0 for every x, which may round two logits to one: one more round
// gives the largest word left, and where two of these neighbours agree in the bits kept their
// logits are compared.  Where more than two agree, or a gate is NaN, the row's choice is made
// again on whole logits.
//
// Sums.  Every lane adds up the gates of its experts in registers, and the block adds its warps
// in order.  A block alone is done with that.  Otherwise each block writes its row of sums to
// the workspace, and the last one to have done so adds the rows; rows of more than 128 experts
// are more than one block should read, and a second kernel adds them (32768 x 1024 in 32 bits: 48 us
// against 57, 262144 x 256 85 against 92; 30011 x 72 in float16: 11.9 us in one launch against 12.3 in
// two).  Either way they are added in an order of their own: no result depends on the order in
// which blocks run.
#pragma once

#include <type_traits>

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
    uint32_t *ticket;   // 0 on entry
    float *part;        // [blocks][2][pitch of the experts]: sums, then counts
    int32_t *part_n;    // [blocks] live rows
    int32_t *counts, *live;
    float *mean_prob, *loss;
    // backward
    const float *grad_weights, *grad_loss;
    void *grad;
    int64_t grad_stride;
    bool vector_grad;
};

// Largest block and blocks per SM that the kernels are compiled for, by the values per lane: the
// registers of the values, of their words and of the sums.  The forward kernel takes any whole
// number of warps up to that.  Blocks of 28 and 20 warps leave it 72 and 96 registers, and up to 96
// bytes of a thread go through memory; with 24 and 16 warps none do, and 262144 x 100 takes 51 us
// against 50, 262144 x 160 71 against 66 (32 bits, k = 4 and 6).
template <int V>
struct RouteShape {
    static constexpr int kWarps = V <= 8 ? 32 : V <= 16 ? 28 : V <= 24 ? 20 : 16;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kPerSm = 1;
};
template <int V>
struct BackwardShape {
    static constexpr int kWarps = V >= 32 ? 8 : 16;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kPerSm = V <= 8 ? 2 : 1;
};

namespace {

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
template <int V, bool VEC, int LANES = 32, int MOST = 8>
struct Place {
    static constexpr int C = VEC ? (V < MOST ? V : MOST) : 1;
    static __device__ __forceinline__ int of(int i, int lane) { return (i / C) * (LANES * C) + lane * C + i % C; }
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

// The forward kernel's rows on their way through shared memory, in pieces of up to 16 bytes: each
// warp has room for two sets of its rows, one being copied while the other is worked on.
template <typename T, int LANES, int V>
struct Rows {
    using L = Place<V, true, LANES, 16 / int(sizeof(T))>;
    T x[32 / LANES][LANES * V];

    __device__ __forceinline__ void copy(const T *row, int experts, int lane) {
        const int g = lane & (LANES - 1);
#pragma unroll
        for (int i = 0; i < V; i += L::C) {
            const int e = L::of(i, g);
            if (e < experts) copy_ahead<L::C * int(sizeof(T))>(&x[lane / LANES][e], row + e);   // E is a multiple of C
        }
    }
    __device__ __forceinline__ void read(int experts, int lane, T (&to)[V]) const {
        const int g = lane & (LANES - 1);
#pragma unroll
        for (int i = 0; i < V; i += L::C) {
            const int e = L::of(i, g);
            if (e < experts) {
                using P = typename Piece<L::C * sizeof(T)>::type;
                *reinterpret_cast<P *>(to + i) = *reinterpret_cast<const P *>(&x[lane / LANES][e]);
            } else {
#pragma unroll
                for (int c = 0; c < L::C; c++) to[i + c] = from_f32<T>(-INFINITY);
            }
        }
    }
};

// A row as the lane holds it; minus infinity past the last expert.
template <typename T, int V, bool VEC, int LANES = 32>
__device__ __forceinline__ void fetch_row(const RouteArgs &a, const T *row, int lane, T (&x)[V]) {
    using L = Place<V, VEC, LANES>;
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

// exp(x - top) as base 2 to the power r, r = (x - top) log2(e) by one multiply-add.  The
// rounding of top log2(e), and the little that `shift` is more so that r is below 0 for every
// x <= top, are the same factor in every gate of the row and leave with the division by their
// sum.  That little grows with top: up to 2^20 it is at most about 1, a bit of the gates' range,
// but from 10^8 on it would take all gates of a row to 0.  Beyond 2^20 (far) the difference is
// taken first: r is then 0 or below, as exact, and in the same order.
struct RowExp {
    float top, shift;
    bool far;
    __device__ __forceinline__ explicit RowExp(float t)
        : top(t), shift(fmaf(t, kLog2e, fmaf(fabsf(t), 0x1p-20f, 0x1p-20f))), far(fabsf(t) > 0x1p20f) {}
    __device__ __forceinline__ float near(float x) const { return fmaf(x, kLog2e, -shift); }
    __device__ __forceinline__ float of(float x) const { return far ? (x - top) * kLog2e : near(x); }
};

// Over the LANES lanes of a row.
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int LANES>
__device__ __forceinline__ float row_max(float v) {   // NaN counts as nothing
    if constexpr (LANES == 32) {
        return warp_max(v);
    } else {
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        return v;
    }
}
template <int LANES, typename U>
__device__ __forceinline__ U row_largest(U v) {
    if constexpr (LANES == 32 && sizeof(U) == 4) {
        return __reduce_max_sync(0xffffffffu, v);
    } else {
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
        return v;
    }
}
// Whether any lane of the row says so.
template <int LANES>
__device__ __forceinline__ bool row_any(bool b) {
    const uint32_t all = __ballot_sync(0xffffffffu, b);
    if constexpr (LANES == 32) return all != 0;
    return (all >> (threadIdx.x & 31 & ~(LANES - 1)) & ((1u << (LANES & 31)) - 1)) != 0;
}

template <int I, int J, int V>
__device__ __forceinline__ void exchange(uint32_t (&w)[V]) {   // the larger to I
    const uint32_t hi = max(w[I], w[J]), lo = min(w[I], w[J]);
    w[I] = hi;
    w[J] = lo;
}
// Batcher's merge of the sorted elements A, A + 2 R, .. and A + R, A + 3 R, .. below A + N.
template <int A, int N, int R, int V>
__device__ __forceinline__ void merge_odd_even(uint32_t (&w)[V]);
template <int I, int END, int R, int V>
__device__ __forceinline__ void exchange_neighbours(uint32_t (&w)[V]) {
    if constexpr (I + R < END) {
        exchange<I, I + R>(w);
        exchange_neighbours<I + 2 * R, END, R>(w);
    }
}
template <int A, int N, int R, int V>
__device__ __forceinline__ void merge_odd_even(uint32_t (&w)[V]) {
    if constexpr (2 * R < N) {
        merge_odd_even<A, N, 2 * R>(w);
        merge_odd_even<A + R, N, 2 * R>(w);
        exchange_neighbours<A + R, A + N, R>(w);
    } else {
        exchange<A, A + R>(w);
    }
}
// Sorts w[A .. A + N) downwards, N a power of two.  (By recursion: a loop that the compiler leaves
// rolled would put w into memory.)
template <int A, int N, int V>
__device__ __forceinline__ void sort_down(uint32_t (&w)[V]) {
    if constexpr (N > 1) {
        sort_down<A, N / 2>(w);
        sort_down<A + N / 2, N / 2>(w);
        merge_odd_even<A, N, 1>(w);
    }
}

// Leaves the N largest of w, downwards, in w[0 .. N): sorted runs of N, merged in pairs.  Of two
// sorted runs the larger of each element and the other's mirror image are the N largest, in an
// order that log2(N) rounds of exchanges sort.
template <int N, int V>
__device__ __forceinline__ void keep_largest(uint32_t (&w)[V]) {
    static_assert(V % N == 0 && V / N <= 8, "whole runs, at most eight");
    sort_down<0, N>(w);
    if constexpr (V / N >= 2) sort_down<N, N>(w);
    if constexpr (V / N >= 3) sort_down<2 * N, N>(w);
    if constexpr (V / N >= 4) sort_down<3 * N, N>(w);
    if constexpr (V / N >= 5) sort_down<4 * N, N>(w);
    if constexpr (V / N >= 6) sort_down<5 * N, N>(w);
    if constexpr (V / N >= 7) sort_down<6 * N, N>(w);
    if constexpr (V / N >= 8) sort_down<7 * N, N>(w);
#pragma unroll
    for (int step = N; step < V; step *= 2)
#pragma unroll
        for (int at = 0; at + step < V; at += 2 * step) {
#pragma unroll
            for (int i = 0; i < N; i++) w[at + i] = max(w[at + i], w[at + step + N - 1 - i]);
#pragma unroll
            for (int q = N / 2; q; q /= 2)
#pragma unroll
                for (int i = 0; i < N; i++)
                    if (!(i & q)) {
                        const uint32_t hi = max(w[at + i], w[at + i + q]), lo = min(w[at + i], w[at + i + q]);
                        w[at + i] = hi;
                        w[at + i + q] = lo;
                    }
        }
}

// Of values held one per chosen expert (number s LANES + g in slot s of lane g), the one of the
// next and of the previous expert.
template <int LANES, int SLOTS>
__device__ __forceinline__ uint32_t following(const uint32_t (&v)[SLOTS], int s) {
    const uint32_t in = __shfl_down_sync(0xffffffffu, v[s], 1, LANES);
    const uint32_t over = __shfl_sync(0xffffffffu, v[s + 1 < SLOTS ? s + 1 : s], 0, LANES);
    return (threadIdx.x & (LANES - 1)) == LANES - 1 ? over : in;
}
template <int LANES, int SLOTS>
__device__ __forceinline__ uint32_t preceding(const uint32_t (&v)[SLOTS], int s) {
    const uint32_t in = __shfl_up_sync(0xffffffffu, v[s], 1, LANES);
    const uint32_t over = __shfl_sync(0xffffffffu, v[s > 0 ? s - 1 : s], LANES - 1, LANES);
    return (threadIdx.x & (LANES - 1)) == 0 ? over : in;
}

// The choice on whole logits, which are read again, for the rows whose lanes have `wanted` set
// (all lanes of the warp take part): lane g of a row's LANES gets in slot s the chosen expert
// number s LANES + g, or -1.
template <typename T, int V, int LANES, int SLOTS>
__device__ __forceinline__ void choose_exactly(const RouteArgs &a, const T *row, bool wanted, int (&id)[SLOTS]) {
    const int g = threadIdx.x & (LANES - 1);
    uint32_t w[V], taken = 0;
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int e = g + LANES * i;
        const float x = wanted && e < a.experts ? to_f32(row[e * a.col_stride]) : -INFINITY;
        w[i] = x > -INFINITY ? order_word(x) : 0u;   // 0 for NaN too
    }
    if (wanted)
#pragma unroll
        for (int s = 0; s < SLOTS; s++) id[s] = -1;
#pragma unroll 1
    for (int j = 0; j < a.k; j++) {
        unsigned long long best = 0;
#pragma unroll
        for (int i = 0; i < V; i++) {
            const unsigned long long c =
                (static_cast<unsigned long long>(w[i]) << 32) | uint32_t(~(g + LANES * i));
            if (w[i] && !(taken >> i & 1) && c > best) best = c;
        }
        best = row_largest<LANES>(best);
        const int e = int(~uint32_t(best));
        if (best && e % LANES == g) taken |= 1u << (e / LANES);
#pragma unroll
        for (int s = 0; s < SLOTS; s++)
            if (wanted && best && s * LANES + g == j) id[s] = e;
    }
}

// The bits of a word that hold the index, for rows of up to n values.
__host__ __device__ constexpr uint32_t index_bits(int n) {
    uint32_t b = 1;
    while (b < uint32_t(n)) b *= 2;
    return b - 1;
}

// Lane g of a row's LANES gets in slot s the row's chosen expert number s LANES + g, or -1.  w:
// the words of the lane's values.  MOST: how many of them are kept, 4, 8 or 16; k is at most that
// for 4 and 8, where one slot is enough, and any for 16.  Rows that draw on one lane more often, or
// as often where a tie has to be looked for, are chosen again.  ex: the row's exponents; again: its
// words cannot be used; idle: nothing is chosen in the row.
template <typename T, int V, int LANES, int MOST, int SLOTS>
__device__ __forceinline__ void choose(const RouteArgs &a, const T *row, const RowExp &ex, uint32_t (&w)[V],
                                       bool again, bool idle, int (&id)[SLOTS]) {
    constexpr uint32_t kIndex = index_bits(LANES * V);
    constexpr bool kWhole = sizeof(T) == 2;      // no bit of a logit is lost
    constexpr int kList = V < MOST ? V : MOST;   // words kept of a lane's
    const int k = a.k, g = threadIdx.x & (LANES - 1);
    uint32_t mine[SLOTS];
#pragma unroll
    for (int s = 0; s < SLOTS; s++) mine[s] = 0;
    keep_largest<kList>(w);
    if constexpr (MOST <= 8) {
#pragma unroll
        for (int j = 0; j < MOST; j++) {
            if (j >= k) break;
            const uint32_t last = row_largest<LANES>(w[0]);
            if (g == j) mine[0] = last;
            if (w[0] == last) {   // of a list only what the rounds left can reach is moved
#pragma unroll
                for (int i = 0; i < kList; i++)
                    if (i < MOST + 1 - j) w[i] = i + 1 < kList ? w[i + 1 < kList ? i + 1 : i] : 0u;
            }
        }
    } else {
#pragma unroll
        for (int s = 0; s < SLOTS; s++)
#pragma unroll 1
            for (int j = 0; j < LANES && s * LANES + j < k; j++) {
                const uint32_t last = row_largest<LANES>(w[0]);
                if (g == j) mine[s] = last;
                if (w[0] == last) {
#pragma unroll
                    for (int i = 0; i + 1 < kList; i++) w[i] = w[i + 1];
                    w[kList - 1] = 0;
                }
            }
    }
    // a lane whose words are used up may have had more (MOST of them and k = MOST: no more was wanted)
    if (kList < V && !(MOST <= 8 && kWhole)) again |= row_any<LANES>(w[0] == 0u);
#pragma unroll
    for (int s = 0; s < SLOTS; s++) id[s] = mine[s] > kClosed ? int(kIndex - (mine[s] & kIndex)) : -1;
    if (!kWhole) {
        const uint32_t next = row_largest<LANES>(w[0]);
        bool tie[SLOTS], any_tie = false, missing = false;   // with the word after it; nothing to choose
#pragma unroll
        for (int s = 0; s < SLOTS; s++) {
            const int j = s * LANES + g;
            uint32_t after = following<LANES, SLOTS>(mine, s);   // by every lane: it exchanges values
            if (j == k - 1) after = next;
            tie[s] = j < k && mine[s] > kClosed && ((mine[s] ^ after) & ~kIndex) == 0;
            any_tie |= tie[s];
            missing |= j < k && mine[s] <= kClosed;
        }
        if (__any_sync(0xffffffffu, any_tie && !idle)) {
            // two words that agree: the logits decide, and the index as it did; more than two: again
            if (w[0] == next) {
#pragma unroll
                for (int i = 0; i + 1 < kList; i++) w[i] = w[i + 1];
                w[kList - 1] = 0;
            }
            const uint32_t second = row_largest<LANES>(w[0]);
            const bool used_up = row_any<LANES>(w[0] == 0u);
            const bool next_tie = ((next ^ second) & ~kIndex) == 0 || (kList < V && used_up);
            const int next_id = int(kIndex - (next & kIndex));
            float x[SLOTS];
            uint32_t bits[SLOTS], flag[SLOTS], ids[SLOTS];
            bool crowd = false;
#pragma unroll
            for (int s = 0; s < SLOTS; s++) {
                x[s] = id[s] >= 0 && !idle ? to_f32(row[id[s] * a.col_stride]) : 0.0f;
                bits[s] = __float_as_uint(x[s]);
                flag[s] = tie[s];
                ids[s] = uint32_t(id[s]);
            }
#pragma unroll
            for (int s = 0; s < SLOTS; s++) {
                const int j = s * LANES + g;
                uint32_t other = following<LANES, SLOTS>(ids, s);
                float y = __uint_as_float(following<LANES, SLOTS>(bits, s));
                bool more = following<LANES, SLOTS>(flag, s);
                const uint32_t before = preceding<LANES, SLOTS>(ids, s);
                const float z = __uint_as_float(preceding<LANES, SLOTS>(bits, s));
                const uint32_t flagged = preceding<LANES, SLOTS>(flag, s);
                const bool behind = j > 0 && j < k && flagged;
                if (j == k - 1) {
                    other = uint32_t(next_id);
                    y = tie[s] && !idle ? to_f32(row[next_id * a.col_stride]) : 0.0f;
                    more = next_tie;
                }
                crowd |= tie[s] && more;
                if (tie[s] && y > x[s])
                    id[s] = int(other);
                else if (behind && x[s] > z)
                    id[s] = int(before);
            }
            again |= row_any<LANES>(crowd);
        }
        if (__any_sync(0xffffffffu, missing && !idle)) {   // closed, or finite with an exponent below the type's range
            bool low = false;
            if (!idle) {
#pragma unroll 1
                for (int e = g; e < a.experts; e += LANES) {
                    const float x = to_f32(row[e * a.col_stride]);
                    low |= x > -INFINITY && ex.of(x) == -INFINITY;
                }
            }
            again |= row_any<LANES>(low);
        }
    }
    if (__any_sync(0xffffffffu, again && !idle))
        choose_exactly<T, V, LANES, SLOTS>(a, row, again && !idle, id);
}

// From the sum over experts of count * mean.
__device__ __forceinline__ float loss_of(const RouteArgs &a, float dot, int n) {
    return n ? dot * float(a.experts) / (float(a.k) * float(n)) : 0.0f;
}

// Values per lane from which a second kernel adds the blocks' rows (over 128 experts).
constexpr int kApart = 24;

// Distance of the workspace's rows: whole pieces of 16 bytes.
__host__ __device__ __forceinline__ int row_pitch(int experts) { return (experts + 3) & ~3; }

// Measured: 262144 x 256 in 32 bits, k = 8: 85 us, 3.4 TB/s of the 285 MB that it must move, whose
// floor is 42 us.  250 instructions a row, for sorting above all, from four warps per scheduler, whose
// waits for their own results they do not cover: issue slots are used 62 % of the time, the integer
// pipe 65 %, memory 42 %.  A row of 16-bit logits costs as many (131072 x 256 in bfloat16 50 us, floor
// 11).  MOST, the words that a lane keeps: with 8 this takes 85 us against 137 with 16; k = 2 with 4
// takes 67 us against 75 with 8 (bfloat16 71 against 80).  With 16, k = 32 of 256 costs 870 instructions
// a row (131072 rows in bfloat16 145 us, floor 15), k = 16 of 512 1160 (65536 rows in 32 bits 105, floor 21).
// Rows whose choice is made again: 262144 x 256 with all logits of a row equal 473 us, with logits
// that are bfloat16 numbers in 32 bits 171.
template <typename T, int LANES, int V, bool VEC, int MOST>
__global__ void __launch_bounds__(RouteShape<V>::kThreads, RouteShape<V>::kPerSm) route_kernel(RouteArgs a) {
    constexpr int kRows = 32 / LANES, kSlots = MOST <= 8 ? 1 : 32 / LANES;
    constexpr uint32_t kIndex = index_bits(LANES * V);
    using R = Rows<T, LANES, V>;
    using L = typename std::conditional<VEC, typename R::L, Place<V, false, LANES>>::type;
    extern __shared__ __align__(16) unsigned char sh[];
    __shared__ float sh_dot[32];
    __shared__ bool sh_last;
    const int threads = blockDim.x, warps = threads >> 5;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane & (LANES - 1);
    R *const rows = reinterpret_cast<R *>(sh) + 2 * warp;                         // [warps][2] (VEC)
    float *sh_sum = reinterpret_cast<float *>(sh + (VEC ? 2 * warps * sizeof(R) : 0));   // [warps][experts]
    int32_t *sh_count = reinterpret_cast<int32_t *>(sh_sum + warps * a.experts);   // [experts], then live rows
    pdl_wait();
    pdl_trigger();
    const int64_t stride = int64_t(gridDim.x) * warps * kRows;
    auto row_of = [&](int64_t t) { return static_cast<const T *>(a.logits) + t * a.row_stride; };
    auto counts = [&](int64_t t) { return t < a.tokens && !(a.mask && !a.mask[t]); };
    const int64_t begin = (int64_t(blockIdx.x) * warps + warp) * kRows + lane / LANES;
    bool next_on = false;
    if constexpr (VEC) {
        next_on = counts(begin);
        if (next_on) rows[0].copy(row_of(begin), a.experts, lane);
        copies_mark();
    }
    for (int e = threadIdx.x; e <= a.experts; e += threads) sh_count[e] = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; i++) acc[i] = 0.0f;
    int live = 0, turn = 0;
    for (int64_t t = begin; t - lane / LANES < a.tokens; t += stride, turn ^= 1) {
        const T *row = row_of(t);
        const bool in = t < a.tokens;
        alignas(16) T raw[V];
        bool on;
        if constexpr (VEC) {
            __syncwarp();   // the other set of rows has been read by all
            on = next_on;
            next_on = counts(t + stride);
            if (next_on) rows[turn ^ 1].copy(row_of(t + stride), a.experts, lane);
            copies_mark();
            copies_wait<1>();
            __syncwarp();
            if (on) rows[turn].read(a.experts, lane, raw);
        } else {
            on = counts(t);
            if (on) fetch_row<T, V, false, LANES>(a, row, g, raw);
        }
        if (!on) {
#pragma unroll
            for (int i = 0; i < V; i++) raw[i] = from_f32<T>(-INFINITY);
        }
        float x[V], top = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; i++) {
            x[i] = to_f32(raw[i]);
            top = fmaxf(top, x[i]);
        }
        top = row_max<LANES>(top);
        bool is_live = top > -INFINITY;
        if (__any_sync(0xffffffffu, on && !is_live)) {   // closed, unless NaN is in it
            bool nan = false;
#pragma unroll
            for (int i = 0; i < V; i++) nan |= isnan(x[i]);
            is_live |= row_any<LANES>(nan);
        }
        if (!(top > -INFINITY)) top = 0.0f;
        const RowExp ex(top);
        uint32_t w[V];
        float sum = 0.0f;
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < V; i++) w[i] = (order_word(x[i]) & ~kIndex) | (kIndex - L::of(i, g));
        }
        if (__any_sync(0xffffffffu, ex.far)) {
#pragma unroll
            for (int i = 0; i < V; i++) x[i] = ex.of(x[i]);
        } else {
#pragma unroll
            for (int i = 0; i < V; i++) x[i] = ex.near(x[i]);
        }
        if constexpr (sizeof(T) == 4) {   // r is below 0, or +0: its bits inverted are in order
#pragma unroll
            for (int i = 0; i < V; i++) w[i] = (~__float_as_uint(x[i]) & ~kIndex) | (kIndex - L::of(i, g));
        }
#pragma unroll
        for (int i = 0; i < V; i++) {
            x[i] = exp2_of(x[i]);
            sum += x[i];
        }
        sum = row_sum<LANES>(sum);
        const float inv = is_live ? __fdividef(1.0f, sum) : 0.0f;
        live += is_live;
#pragma unroll
        for (int i = 0; i < V; i++) acc[i] = fmaf(x[i], inv, acc[i]);

        int id[kSlots];
        choose<T, V, LANES, MOST, kSlots>(a, row, ex, w, isnan(sum), !is_live, id);
        float gate[kSlots], total = 0.0f;
#pragma unroll
        for (int s = 0; s < kSlots; s++) {
            if (!is_live) id[s] = -1;
            gate[s] = 0.0f;
            if (id[s] >= 0) {
                T chosen;
                if constexpr (VEC)
                    chosen = rows[turn].x[lane / LANES][id[s]];
                else
                    chosen = row[id[s] * a.col_stride];
                gate[s] = exp2_of(ex.of(to_f32(chosen)));
                atomicAdd(&sh_count[id[s]], 1);
            }
            total += gate[s];
        }
        // in a row with NaN every gate is NaN, also those that are 0 here
        const float over = a.normalize ? row_sum<LANES>(total) : sum;
        const float by = __fdividef(1.0f, isnan(sum) ? sum : over);
#pragma unroll
        for (int s = 0; s < kSlots; s++) {
            const int j = s * LANES + g;
            if (in && j < a.k) {
                a.ids[t * a.k + j] = id[s];
                a.weights[t * a.k + j] = id[s] >= 0 ? gate[s] * by : 0.0f;
            }
        }
    }
    // the warp's rows of lanes, then its lanes, then the block's warps
#pragma unroll
    for (int i = 0; i < V; i++) {
#pragma unroll
        for (int o = LANES; o < 32; o *= 2) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
        if (lane < LANES && L::of(i, g) < a.experts) sh_sum[warp * a.experts + L::of(i, g)] = acc[i];
    }
    live = __reduce_add_sync(0xffffffffu, g ? 0 : live);
    if (lane == 0 && live) atomicAdd(&sh_count[a.experts], live);
    __syncthreads();
    auto add_warps = [&](int e) {
        float s = 0.0f;
#pragma unroll 4
        for (int w = 0; w < warps; w++) s += sh_sum[w * a.experts + e];
        return s;
    };
    if (gridDim.x > 1) {
        const int pitch = row_pitch(a.experts), blocks = int(gridDim.x);
        float *own = a.part + int64_t(blockIdx.x) * 2 * pitch;
        for (int e = threadIdx.x; e < a.experts; e += threads) {
            own[e] = add_warps(e);
            own[pitch + e] = __int_as_float(sh_count[e]);
        }
        if (threadIdx.x == 0) a.part_n[blockIdx.x] = sh_count[a.experts];
        if constexpr (V >= kApart) return;
        __syncthreads();
        if (threadIdx.x == 0) sh_last = last_ticket(a.ticket, blocks);
        for (int e = threadIdx.x; e <= a.experts; e += threads) sh_count[e] = 0;
        __syncthreads();
        if (!sh_last) return;
        // a warp adds every warps-th row, a lane four experts of each
        if (warp == 0) {
            int n = 0;
            for (int r = lane; r < blocks; r += 32) n += __ldcg(a.part_n + r);
            n = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0) sh_count[a.experts] = n;
        }
        constexpr int kAtOnce = (kSMs + RouteShape<V>::kWarps - 1) / RouteShape<V>::kWarps;   // a warp's rows
        for (int e0 = 4 * lane; e0 < a.experts; e0 += 128) {
            float4 p = {0.0f, 0.0f, 0.0f, 0.0f};
            int4 c = {0, 0, 0, 0};
            for (int r0 = warp; r0 < blocks; r0 += warps * kAtOnce) {
                float4 q[kAtOnce];
                int4 d[kAtOnce];
#pragma unroll
                for (int i = 0; i < kAtOnce; i++) {
                    q[i] = {0.0f, 0.0f, 0.0f, 0.0f};
                    d[i] = {0, 0, 0, 0};
                    if (r0 + i * warps < blocks) {
                        const float *row = a.part + int64_t(r0 + i * warps) * 2 * pitch + e0;
                        q[i] = __ldcg(reinterpret_cast<const float4 *>(row));
                        d[i] = __ldcg(reinterpret_cast<const int4 *>(row + pitch));
                    }
                }
#pragma unroll
                for (int i = 0; i < kAtOnce; i++) {
                    p.x += q[i].x, p.y += q[i].y, p.z += q[i].z, p.w += q[i].w;
                    c.x += d[i].x, c.y += d[i].y, c.z += d[i].z, c.w += d[i].w;
                }
            }
            const float ps[4] = {p.x, p.y, p.z, p.w};
            const int cs[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (e0 + i < a.experts) {
                    sh_sum[warp * a.experts + e0 + i] = ps[i];
                    atomicAdd(&sh_count[e0 + i], cs[i]);
                }
        }
        __syncthreads();
    }
    const int n = sh_count[a.experts];
    const float over = n ? 1.0f / float(n) : 0.0f;
    float dot = 0.0f;
    for (int e = threadIdx.x; e < a.experts; e += threads) {
        const float mean = add_warps(e) * over;
        a.counts[e] = sh_count[e];
        a.mean_prob[e] = mean;
        dot = fmaf(mean, float(sh_count[e]), dot);
    }
    dot = warp_sum(dot);
    if (lane == 0) sh_dot[warp] = dot;
    __syncthreads();
    if (warp == 0) {
        dot = warp_sum(lane < warps ? sh_dot[lane] : 0.0f);
        if (lane == 0) {
            *a.live = n;
            *a.loss = loss_of(a, dot, n);
        }
    }
}

// The gradient.  With the weights w that the forward pass wrote, what reaches a chosen logit
// beyond the softmax's own term is w (grad_weight - dot) for normalised gates and
// w grad_weight for plain ones, dot = sum of w grad_weight over the row's chosen; only plain
// gates leave dot in the row's mean.  The counts enter as c - k n / E: a constant in d
// drops out of the gradient, and without it the subtraction of the mean loses no digits.
// The k terms reach their experts' lanes through the row's share of shared memory.
// Measured: 131071 x 256 in 32 bits, k = 8: 48.7 us, 5.8 TB/s of 281 MB; 262144 rows 92 us, 6.1 TB/s.
// Waits for memory bound it.  Short and 16-bit rows have as much to do for fewer bytes: 262144 x 64
// in bfloat16, k = 2: 24 us, floor 11; 262144 x 16 in 32 bits 19, floor 6; 131072 x 256 in bfloat16,
// k = 8: 39, floor 22: issue slots are used 47 to 63 % of the time, and loads are still what warps
// wait for most.  FEW: one slot per lane holds the k chosen.
template <typename T, int LANES, int V, bool VEC, bool FEW>
__global__ void __launch_bounds__(BackwardShape<V>::kThreads, BackwardShape<V>::kPerSm) route_backward_kernel(RouteArgs a) {
    constexpr int kWarps = BackwardShape<V>::kWarps, kRows = 32 / LANES, kSlots = FEW ? 1 : 32 / LANES;
    using L = Place<V, VEC, LANES>;
    extern __shared__ __align__(16) unsigned char sh[];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane & (LANES - 1);
    float *const extra = reinterpret_cast<float *>(sh) + warp * (32 * V) + lane / LANES * (LANES * V);   // the row's
#pragma unroll
    for (int i = 0; i < V; i++) extra[g + LANES * i] = 0.0f;
    const float n = float(*a.live), even = float(a.k) * n / float(a.experts);
    const float f = a.grad_loss && n > 0.0f ? *a.grad_loss * float(a.experts) / (float(a.k) * n * n) : 0.0f;
    float own[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int e = L::of(i, g);
        own[i] = e < a.experts ? f * (float(a.counts[e]) - even) : 0.0f;
    }
    const int64_t stride = int64_t(gridDim.x) * kWarps * kRows;
    alignas(16) T raw[V];
    int id[kSlots];
    float w[kSlots], u[kSlots];
    // what row t needs, as the lane holds it; whether the row counts
    auto fetch = [&](int64_t t) {
        const bool on = t < a.tokens && !(a.mask && !a.mask[t]);
        if (on) {
            fetch_row<T, V, VEC, LANES>(a, static_cast<const T *>(a.logits) + t * a.row_stride, g, raw);
        } else {
#pragma unroll
            for (int i = 0; i < V; i++) raw[i] = from_f32<T>(-INFINITY);
        }
#pragma unroll
        for (int s = 0; s < kSlots; s++) {
            const int j = s * LANES + g;
            id[s] = -1;
            w[s] = u[s] = 0.0f;
            if (on && a.grad_weights && j < a.k) {
                id[s] = a.ids[t * a.k + j];
                w[s] = a.weights[t * a.k + j];
                u[s] = a.grad_weights[t * a.k + j];
                if (uint32_t(id[s]) >= uint32_t(a.experts)) {
                    id[s] = -1;
                    w[s] = u[s] = 0.0f;
                }
            }
        }
        return on;
    };
    int64_t t = (int64_t(blockIdx.x) * kWarps + warp) * kRows + lane / LANES;
    bool on = fetch(t);
    for (; t - lane / LANES < a.tokens; t += stride) {
        float e[V], top = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; i++) {
            e[i] = to_f32(raw[i]);
            top = fmaxf(top, e[i]);
        }
        top = row_max<LANES>(top);
        bool is_live = top > -INFINITY;
        if (__any_sync(0xffffffffu, on && !is_live)) {   // closed, unless NaN is in it
            bool nan = false;
#pragma unroll
            for (int i = 0; i < V; i++) nan |= isnan(e[i]);
            is_live |= row_any<LANES>(nan);
        }
        const RowExp ex(top > -INFINITY ? top : 0.0f);
        if (__any_sync(0xffffffffu, ex.far)) {
#pragma unroll
            for (int i = 0; i < V; i++) e[i] = exp2_of(ex.of(e[i]));
        } else {
#pragma unroll
            for (int i = 0; i < V; i++) e[i] = exp2_of(ex.near(e[i]));
        }
        float sum = 0.0f, mean = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < V; i++) {
            sum += e[i];
            mean = fmaf(e[i], own[i], mean);
        }
#pragma unroll
        for (int s = 0; s < kSlots; s++) dot = fmaf(w[s], u[s], dot);
        sum = row_sum<LANES>(sum);
        mean = row_sum<LANES>(mean);
        dot = row_sum<LANES>(dot);
        const float inv = __fdividef(1.0f, sum);
        mean *= inv;
        if (!a.normalize) mean += dot;
        int to[kSlots];
        __syncwarp();   // the last rows' terms are gone
#pragma unroll
        for (int s = 0; s < kSlots; s++) {
            to[s] = id[s];
            if (to[s] >= 0) extra[to[s]] = a.normalize ? w[s] * (u[s] - dot) : w[s] * u[s];
        }
        on = fetch(t + stride);
        __syncwarp();
        alignas(16) T out[V];
#pragma unroll
        for (int i = 0; i < V; i++) {
            const float d = fmaf(e[i] * inv, own[i] - mean, extra[L::of(i, g)]);
            out[i] = from_f32<T>(is_live ? d : 0.0f);
        }
        __syncwarp();
#pragma unroll
        for (int s = 0; s < kSlots; s++)
            if (to[s] >= 0) extra[to[s]] = 0.0f;
        if (t >= a.tokens) continue;
        T *row = static_cast<T *>(a.grad) + t * a.grad_stride;
#pragma unroll
        for (int i = 0; i < V; i += L::C) {
            const int e0 = L::of(i, g);
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

template <int N> struct Number { static constexpr int v = N; };

// fn(lanes, values): how a row of `experts` is held.  Eight lanes hold up to 32 values each;
// longer rows take more lanes.  24 values, whole runs of 4 and 8 words but not of 16, are for k up
// to 8 (262144 x 160 in bfloat16, k = 6: 70 us against 87 with 32 values).
template <typename F>
int with_row(int experts, int k, F fn) {
    if (experts <= 32) return fn(Number<8>{}, Number<4>{});
    if (experts <= 64) return fn(Number<8>{}, Number<8>{});
    if (experts <= 128) return fn(Number<8>{}, Number<16>{});
    if (experts <= 192 && k <= 8) return fn(Number<8>{}, Number<24>{});
    if (experts <= 256) return fn(Number<8>{}, Number<32>{});
    if (experts <= 512) return fn(Number<16>{}, Number<32>{});
    return fn(Number<32>{}, Number<32>{});
}

// fn(lanes, values) likewise for the backward kernel: at most 8 values each up to a whole warp.
template <typename F>
int with_backward_row(int experts, F fn) {
    if (experts <= 32) return fn(Number<8>{}, Number<4>{});
    if (experts <= 64) return fn(Number<8>{}, Number<8>{});
    if (experts <= 128) return fn(Number<16>{}, Number<8>{});
    if (experts <= 256) return fn(Number<32>{}, Number<8>{});
    if (experts <= 512) return fn(Number<32>{}, Number<16>{});
    return fn(Number<32>{}, Number<32>{});
}

// Whether every row can be read in pieces of C neighbours.
template <typename T, int V, int C>
bool vector_rows(const RouteArgs &a) {
    return V > 1 && a.col_stride == 1 && a.experts % C == 0 && a.row_stride % C == 0 &&
           aligned_to(a.logits, C * sizeof(T));
}

}  // namespace

// Launches of one element type (each in its own translation unit).
template <typename T, int L, int V, bool VEC, int MOST>
int launch_route_kernel(const RouteArgs &a, int blocks, int threads, void *stream) {
    const auto smem = [](int warps, int experts) {
        return (VEC ? warps * 2 * sizeof(Rows<T, L, V>) : 0) + size_t(4) * (warps * experts + experts + 1);
    };
    const size_t most = smem(RouteShape<V>::kWarps, L * V);
    if (const int rc = allow<route_kernel<T, L, V, VEC, MOST>>(most, "route attribute")) return rc;
    return launch_kernel(route_kernel<T, L, V, VEC, MOST>, dim3(blocks), dim3(threads), smem(threads / 32, a.experts),
                         stream, 1, "route launch", a);
}

template <typename T>
int launch_route_type(const RouteArgs &a, int blocks, int threads, void *stream) {
    return with_row(a.experts, a.k, [&](auto lanes, auto values) {
        constexpr int L = decltype(lanes)::v, V = decltype(values)::v;
        const bool vec = vector_rows<T, V, Rows<T, L, V>::L::C>(a);
        const auto with = [&](auto most) {
            constexpr int M = decltype(most)::v;
            return vec ? launch_route_kernel<T, L, V, true, M>(a, blocks, threads, stream)
                       : launch_route_kernel<T, L, V, false, M>(a, blocks, threads, stream);
        };
        // a list of 4 serves 4 experts where ties need no word more, else 3
        if constexpr (V > 4)
            if (a.k < (sizeof(T) == 2 ? 5 : 4)) return with(Number<4>{});
        if constexpr (V == 24)
            return with(Number<8>{});
        else
            return a.k <= 8 ? with(Number<8>{}) : with(Number<16>{});
    });
}

template <typename T>
int launch_route_backward_type(RouteArgs a, void *stream) {
    return with_backward_row(a.experts, [&](auto lanes, auto values) {
        constexpr int N = decltype(lanes)::v, V = decltype(values)::v;
        using S = BackwardShape<V>;
        using L = Place<V, true, N>;
        a.vector_grad = a.grad_stride % L::C == 0 && aligned_to(a.grad, L::C * sizeof(T));
        const size_t smem = size_t(4) * S::kWarps * 32 * V;
        const int64_t rows = S::kWarps * 32 / N, b = (a.tokens + rows - 1) / rows, most = kSMs * S::kPerSm;
        const bool vec = vector_rows<T, V, L::C>(a), few = a.k <= N;
        auto kernel = vec ? few ? route_backward_kernel<T, N, V, true, true> : route_backward_kernel<T, N, V, true, N == 32>
                          : few ? route_backward_kernel<T, N, V, false, true>
                                : route_backward_kernel<T, N, V, false, N == 32>;
        return launch_kernel(kernel, dim3(unsigned(b < most ? b : most)), dim3(S::kThreads), smem, stream, 1,
                             "route backward launch", a);
    });
}

int launch_route_f32(const RouteArgs &a, int blocks, int threads, void *stream);
int launch_route_bf16(const RouteArgs &a, int blocks, int threads, void *stream);
int launch_route_f16(const RouteArgs &a, int blocks, int threads, void *stream);
int launch_route_backward_f32(const RouteArgs &a, void *stream);
int launch_route_backward_bf16(const RouteArgs &a, void *stream);
int launch_route_backward_f16(const RouteArgs &a, void *stream);

}  // namespace nest
