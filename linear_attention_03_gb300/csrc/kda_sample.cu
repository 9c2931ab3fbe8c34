// kda_sample.cu -- from logits to the distribution that is drawn from, and a token
// (kda_sample): temperature, top-k, top-p, min-p and the draw from a given uniform number.
//
//     w_i = e^{(x_i - max x) / T},   order: by value, then by index
//     top-k: the first k of the order;  top-p: of these the shortest beginning with a p-th of their
//     weight;  min-p: of these the ones with w_i >= m;  the token: the first index at which the
//     weights of the ones that stay, added up in index order, exceed u times their sum
//
// Weights are whole multiples of 2^-42, held in 64 bits, so sums do not depend on their order, nor on how many
// CTAs a row has.  Before it is cut to them a weight is right to some 2^-24 of itself; the cut takes up to 2^-42 off,
// always downward: less than 2^-24 of a weight above 2^-18, all of one below 2^-42, and up to V 2^-42 of a sum.
// Min-p needs no weights: its border is a value, max x + T ln m.
//
// A cluster of up to eight CTAs takes a row, as many as let all rows run at once: more would leave CTAs
// waiting for the next wave (256 rows of 131,072 over clusters of two, 512 CTAs for 304 places, take 39 us in
// place of 31 for the largest logit alone, 96 fp32 rows 88 in place of 61 by top-p; one CTA to an SM takes 43).  The row is read from the
// L2 or the L1 as often as it is needed; held in shared memory, its size left two CTAs to an SM and three
// waves (121 us in place of 80 for 256 rows with settings of their own).  What stays is a
// beginning of the order: a border value, and the last index among the logits equal to it.
//   A small k: k of the largest logits of 2,048 groups bound the k-th largest from below; the few logits above the
// bound, in groups that have one, go to one CTA, which makes the whole choice there, the draw included.
//   top-p alone: a histogram of weights relative to their bin says to within a few bins where the border can
// lie; one exact pass sums up all weights and those above the candidates, and lists the candidates.  Where
// min-p keeps less than that no exact sum of the row is needed, and its logits are listed where they are few.
//   A large k: histograms narrow the values down, first by w (bins of equal width in log2 w, which spread
// the logits well whatever their scale), then by the value's bits.
// Measured: 256 bf16 rows of 131,072 31 us (the largest logit) to 41 (k = 100), 72 (k = 1,000), 117 (top-p alone),
// 250 (k = 5,000 and top-p) and 64 (no filter), where reading them once takes 10; 96 fp32 rows of 131,072 by top-p
// 61 us; one row of 50,257 13-26 us.  For a small k the chain of steps is the bound (20,000 clocks, four meetings of
// the cluster), for a larger one the sort of up to 2,048 in one CTA; for top-p the waits for the L2 and at barriers
// beside the instructions: some 30 an element in the histogram's pass, 40 in the exact one, half of the issue slots.
#include "kda_internal.cuh"
#include "kda_tc.cuh"

#include <cooperative_groups.h>

#include <type_traits>

namespace kda {
namespace {

typedef unsigned long long u64;
constexpr int kThreads = 512, kWarps = kThreads / 32, kMaxRanks = 8;
constexpr int kBins = 512;                      // of a histogram
constexpr float kPerOctave = 12.f;              // bins for a halving of w
constexpr int kGroups = 4;                      // a thread's logits, by which its largest ones are taken
constexpr int kList = 4096;                     // a CTA's candidates for the border
constexpr int kSorted = 4 * kThreads, kListK = 1024;    // logits that one CTA sorts, and the k for which that is tried
constexpr int kListAll = 1024;                  // logits that top-p takes from a list altogether
constexpr int kFew = 128;                       // logits of which every pair is compared instead
constexpr int32_t kAll = 0x7fffffff;
// histograms (two of kBins 64-bit sums in turn, or copies of one of kFine sums) and a list
constexpr int kFine = 4 * kBins, kCopies = 4;   // of the first histogram of top-p
constexpr int kSmem = kCopies * kFine * 4 + kList * 8;
static_assert(2 * kThreads * 8 <= kCopies * kFine * 4, "a list and room to sort it");
static_assert(4 * kFew == kThreads && 2 * kFew <= kList && kSorted <= kList, "threads to the elements of a list");
static_assert(kListK <= kGroups * kThreads / 2, "largest ones enough to bound the k-th");
static_assert(kBins == kThreads, "a thread per bin");

struct Sampling {
    const void *logits;
    int64_t stride;                             // elements from a row to the next
    const float *temperature, *top_p, *min_p, *uniforms;
    const int32_t *top_k;
    int32_t V;
    int32_t *token;
    void *probs;                                // [N, V]
    int32_t probs_bf16;
};

// order-preserving whole numbers of floats (no NaN; both zeros are one)
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b >> 31) != 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float((key >> 31) != 0 ? key & 0x7fffffffu : ~key);
}

// 16 bytes of logits as pairs.  clean: NaN becomes -infinity.
template <typename Tin> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4, GRAIN = 0;      // (low bits in which keys never differ)
    static __device__ __forceinline__ void unpack(uint4 u, float2 (&x)[2]) {
        x[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
        x[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
    }
    static __device__ __forceinline__ uint4 nothing() {
        return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
    }
    static __device__ __forceinline__ float pick(uint4 u, int e) {
        return __uint_as_float(e < 2 ? (e == 0 ? u.x : u.y) : e == 2 ? u.z : u.w);
    }
    static __device__ __forceinline__ uint32_t clean(uint32_t w) {
        return __float_as_uint(fmaxf(__uint_as_float(w), -INFINITY));
    }
    static __device__ __forceinline__ float largest(uint4 u) {
        return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8, GRAIN = 16;
    static __device__ __forceinline__ void unpack(uint4 u, float2 (&x)[4]) {
        x[0] = tc::unpack_bf16x2(u.x);
        x[1] = tc::unpack_bf16x2(u.y);
        x[2] = tc::unpack_bf16x2(u.z);
        x[3] = tc::unpack_bf16x2(u.w);
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));       // (a number beside a NaN)
        return d;
    }
    static __device__ __forceinline__ uint4 nothing() {
        return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
    }
    static __device__ __forceinline__ float pick(uint4 u, int e) {
        const uint32_t w = e < 4 ? (e < 2 ? u.x : u.y) : e < 6 ? u.z : u.w;
        return __uint_as_float((e & 1) != 0 ? w & 0xffff0000u : w << 16);
    }
    static __device__ __forceinline__ uint32_t clean(uint32_t w) { return max2(w, 0xff80ff80u); }
    static __device__ __forceinline__ float largest(uint4 u) {
        const uint32_t m = max2(max2(u.x, u.y), max2(u.z, u.w));
        return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    }
};

// The order as a whole number: by value, then by index, the first of all the largest.
constexpr int kIndexBits = 18;
static_assert(KDA_MAX_VOCABULARY <= 1 << kIndexBits, "an index's bits");
__device__ __forceinline__ u64 ordered(uint32_t key, int i) {
    return (u64)key << kIndexBits | (uint32_t)((1 << kIndexBits) - 1 - i);
}
__device__ __forceinline__ uint32_t ordered_key(u64 c) { return (uint32_t)(c >> kIndexBits); }
__device__ __forceinline__ int ordered_index(u64 c) {
    return (1 << kIndexBits) - 1 - (int)((uint32_t)c & ((1u << kIndexBits) - 1));
}

// log2 w = (x - m)(c + cl); below x = least w counts as zero
struct Scale {
    float m, c, cl, least;
};

// The weights of two logits: the product of x - m with c in one rounding behind the point, 2^f by its series (to
// 2^-27 for |f| <= 1/2) and the exponent put on in whole numbers, in paired arithmetic.  WHOLE: with the rounding
// error of x - m, which bf16 logits have only where one is 2^16 times the other (then 2^-24 of log w).  (No number
// of meaning below s.least.)
template <bool WHOLE> __device__ __forceinline__ float2 weights2(const Scale &s, float2 x) {
    auto both = [](float a) { return make_float2(a, a); };
    const float2 d = tc::f2sub(x, both(s.m));
    const float2 t = tc::f2fma(d, both(s.c), both(12582912.f)), whole = tc::f2sub(both(12582912.f), t);
    float2 f = tc::f2fma(d, both(s.c), whole);
    f = tc::f2fma(d, both(s.cl), f);
    if (WHOLE) {
        const float2 mv = tc::f2sub(x, d), xv = tc::f2add(d, mv);
        f = tc::f2fma(tc::f2add(tc::f2sub(x, xv), tc::f2sub(mv, both(s.m))), both(s.c), f);
    }
    float2 p = both(1.5252733804059841e-5f);    // ln(2)^k / k!, k = 7 .. 0
    p = tc::f2fma(p, f, both(1.5403530393381610e-4f));
    p = tc::f2fma(p, f, both(1.3333558146428443e-3f));
    p = tc::f2fma(p, f, both(9.6181291076284772e-3f));
    p = tc::f2fma(p, f, both(5.5504108664821580e-2f));
    p = tc::f2fma(p, f, both(2.4022650695910071e-1f));
    p = tc::f2fma(p, f, both(6.9314718055994531e-1f));
    p = tc::f2fma(p, f, both(1.f));
    p.x = __int_as_float(__float_as_int(p.x) + (__float_as_int(t.x) << 23));
    p.y = __int_as_float(__float_as_int(p.y) + (__float_as_int(t.y) << 23));
    return p;
}
// A weight as a whole number of 2^-42, cut off, in two digits of 21 bits.  Adding 2^23 with rounding toward
// zero leaves the whole part in the significand's low bits, and what remains is exact.  The digits
// carry 2^23's bits with them.
constexpr uint32_t kBias = 0x4b000000u;
__device__ __forceinline__ float2 fma_cut2(float2 a, float2 b, float2 c) {
    unsigned long long d;
    asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(tc::f2u(a)), "l"(tc::f2u(b)), "l"(tc::f2u(c)));
    return tc::u2f(d);
}
__device__ __forceinline__ void digits42(float2 w, float2 &hi, float2 &lo) {
    const float2 scale = make_float2(2097152.f, 2097152.f), one = make_float2(8388608.f, 8388608.f);
    hi = fma_cut2(w, scale, one);
    lo = fma_cut2(tc::f2fma(w, scale, tc::f2sub(one, hi)), scale, one);
}
__device__ __forceinline__ uint32_t digit(float x) { return __float_as_uint(x) - kBias; }
__device__ __forceinline__ u64 fixed42(float w) {
    float2 hi, lo;
    digits42(make_float2(w, w), hi, lo);
    return ((u64)digit(hi.x) << 21) + digit(lo.x);
}
template <bool WHOLE> __device__ __forceinline__ u64 weight_of(const Scale &s, float x) {
    const float w = weights2<WHOLE>(s, make_float2(x, x)).x;
    return fixed42(x >= s.least ? w : 0.f);
}

// The larger one first (or last).
__device__ __forceinline__ void in_order(u64 &a, u64 &b, bool down) {
    const bool swap = (a < b) == down;
    const u64 x = swap ? b : a, y = swap ? a : b;
    a = x;
    b = y;
}
// The block's elements, thread t's x being 4 t .. 4 t + 3 of `all` (a power of two up to 2,048; the others
// zeros), by size, the largest first.  Bitonic: steps of one and two within a thread, up to 64 within its
// warp, the others through shared memory (2,048 elements: 66 steps, ten of them there).
__device__ __forceinline__ void sort_down(u64 (&x)[4], u64 *room, int all) {
    const int tid = threadIdx.x;
    const bool mine = 4 * (tid & ~31) < all;            // (whole warps)
#pragma unroll 1
    for (int size = 2; size <= all; size *= 2) {
#pragma unroll 1
        for (int step = size / 2; step >= 128; step /= 2) {
            if (mine)
#pragma unroll
                for (int e = 0; e < 4; ++e) room[4 * tid + e] = x[e];
            __syncthreads();
            if (mine)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 4 * tid + e;
                    const u64 y = room[i ^ step];
                    const bool larger = ((i & step) == 0) == ((i & size) == 0);
                    x[e] = (x[e] < y) == larger ? y : x[e];
                }
            __syncthreads();
        }
        if (mine) {
#pragma unroll 1
            for (int step = min(size / 2, 64); step >= 4; step /= 2)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 4 * tid + e;
                    const u64 y = __shfl_xor_sync(0xffffffffu, x[e], step / 4);
                    const bool larger = ((i & step) == 0) == ((i & size) == 0);
                    x[e] = (x[e] < y) == larger ? y : x[e];
                }
            const bool down = (4 * tid & size) == 0;
            if (size >= 4) {
                in_order(x[0], x[2], down);
                in_order(x[1], x[3], down);
                in_order(x[0], x[1], down);
                in_order(x[2], x[3], down);
            } else {
                in_order(x[0], x[1], true);
                in_order(x[2], x[3], false);
            }
        }
    }
}

// A vector at a row's end, from element e0 on; a call, since a dozen places have one.
template <typename Tin> __device__ __noinline__ uint4 row_end(const Tin *row, int e0, int V) {
    uint4 x;
    Tin y[Vec<Tin>::N];
#pragma unroll
    for (int e = 0; e < Vec<Tin>::N; ++e) {
        y[e] = static_cast<Tin>(-INFINITY);
        if (e0 + e >= 0 && e0 + e < V) y[e] = row[e0 + e];
    }
    memcpy(&x, y, 16);
    return x;
}

template <typename Tin>
__global__ void __launch_bounds__(kThreads, 2)
sample_kernel(const Sampling a, const int32_t slice) {
    constexpr int VEC = Vec<Tin>::N;
    constexpr bool WHOLE = sizeof(Tin) == 4;
    extern __shared__ __align__(16) unsigned char smem[];
    // two histograms (low words, then high words) and a list
    uint32_t *const hists = reinterpret_cast<uint32_t *>(smem), *hist = hists;
    u64 *const list = reinterpret_cast<u64 *>(hists + kCopies * kFine);
    __shared__ u64 part[kWarps], part_all, chosen_sum, totals[2][kMaxRanks], more[kWarps], more_totals[2][kMaxRanks];
    __shared__ u64 found[2];                    // what lies above the border's bin, what is in it
    __shared__ float tops[kMaxRanks], warp_top[kWarps];
    __shared__ int32_t found_bin, found_last, reach_least, chosen_index, count, chosen_count;
    __shared__ uint32_t chosen_key;
    __shared__ float2 least_log;                // T ln m, a number and what is left of it
    cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    cluster.barrier_arrive();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t n = blockIdx.x / ranks;
    const int32_t V = a.V;
    const Tin *row = static_cast<const Tin *>(a.logits) + n * a.stride;
    // vectors from the 16-byte boundary at or below the row's start: element i of the row is
    // element i + lead of that grid
    const int lead = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(Tin));
    const int vecs = (V + lead + VEC - 1) / VEC, first = min(vecs, rank * slice), mine = min(vecs - first, slice);
    const int per_warp = (slice + kWarps - 1) / kWarps, w0 = min(mine, warp * per_warp), w1 = min(mine, w0 + per_warp);
    const uint4 *grid = reinterpret_cast<const uint4 *>(row - lead) + first;
    auto index_of = [&](int v) { return (first + v) * VEC - lead; };    // of a vector's first element

    float T = a.temperature != nullptr ? a.temperature[n] : 1.f;
    int32_t k = a.top_k != nullptr ? a.top_k[n] : 0;
    float p = a.top_p != nullptr ? a.top_p[n] : 1.f;
    const float least = a.min_p != nullptr ? a.min_p[n] : 0.f;
    const float u = a.uniforms != nullptr ? a.uniforms[n] : 0.f;
    if (tid == 0) count = 0;
    // min-p's border as a value, max x + T ln m: weights that are compared come in the wrong order where logits are a
    // rounding apart, and their whole multiples know none below 2^-42.  In 64 bits by one thread of the block.
    if (tid == kThreads - 1) {
        const double x = isinf(T) ? -INFINITY : log((double)fminf(least, 1.f)) * (double)(T > 0.f ? T : 1.f);
        least_log.x = least > 0.f && x > -3.402823466e38 ? (float)x : -INFINITY;
        least_log.y = (float)(x - (double)least_log.x);
    }

    // A vector of the row as it is (all -infinity from `end` on), and what it counts as: the row is read as often
    // as it is needed, from the L2 or the L1.
    bool infinite = false;                      // the infinite ones share everything
    const int whole0 = first == 0 && lead > 0 ? 1 : 0, whole1 = min(mine, (V + lead) / VEC - first);
    auto raw = [&](int v, int end) {
        if (v >= whole0 && v < min(end, whole1)) return __ldg(grid + v);
        return v < end ? row_end(row, index_of(v), V) : Vec<Tin>::nothing();
    };
    auto clean = [&](uint4 x) {
        x.x = Vec<Tin>::clean(x.x);
        x.y = Vec<Tin>::clean(x.y);
        x.z = Vec<Tin>::clean(x.z);
        x.w = Vec<Tin>::clean(x.w);
        if (infinite) {
            Tin y[VEC];
            memcpy(y, &x, 16);
#pragma unroll
            for (int e = 0; e < VEC; ++e) y[e] = static_cast<Tin>(static_cast<float>(y[e]) == INFINITY ? 0.f : -INFINITY);
            memcpy(&x, y, 16);
        }
        return x;
    };
    // f(v, y) for the vectors a .. b - 1, a warp's, 32 at a time in order, all lanes together; the next ones
    // are on their way meanwhile.
    auto each_vector = [&](int a_, int b_, auto f) {
        uint4 next = raw(a_ + lane, b_);
#pragma unroll 1
        for (int v0 = a_; v0 < b_; v0 += 32) {
            const uint4 y = next;
            next = raw(v0 + 32 + lane, b_);
            f(v0 + lane, clean(y));
        }
    };
    // The same where few reach `from`: four of a lane's on their way, those that do not are passed by.
    auto each_above = [&](int a_, int b_, float from, auto f) {
#pragma unroll 1
        for (int v0 = a_; v0 < b_; v0 += 128) {
            uint4 y[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) y[g] = raw(v0 + 32 * g + lane, b_);
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {
                const uint4 z = clean(y[0]);
                y[0] = y[1];
                y[1] = y[2];
                y[2] = y[3];
                if (Vec<Tin>::largest(z) >= from) f(v0 + 32 * g + lane, z);
            }
        }
    };

    // ---- the maximum, and the largest of each thread's groups
    float my_top[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) my_top[g] = -INFINITY;
#pragma unroll 1
    for (int v = w0 + lane; v < w1; v += 32 * kGroups) {
        uint4 x[kGroups];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) x[g] = raw(v + 32 * g, w1);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) my_top[g] = fmaxf(my_top[g], Vec<Tin>::largest(clean(x[g])));
    }
    if (!(T > 0.f)) {                           // the first of the order alone
        T = 1.f;
        k = 1;
    }
    if (k == 1) p = 1.f;
    float top = my_top[0];
#pragma unroll
    for (int g = 1; g < kGroups; ++g) top = fmaxf(top, my_top[g]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) warp_top[warp] = top;
    cluster.barrier_wait();                     // every CTA has started
    __syncthreads();
    if (warp == 0) {
        top = lane < kWarps ? warp_top[lane] : -INFINITY;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane < ranks) *cluster.map_shared_rank(&tops[rank], lane) = top;
    }
    cluster.sync();
    top = -INFINITY;
    for (int r = 0; r < ranks; ++r) top = fmaxf(top, tops[r]);
    const bool none = top == -INFINITY;
    if (top == INFINITY) {
        infinite = true;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) my_top[g] = my_top[g] == INFINITY ? 0.f : -INFINITY;
        top = 0.f;
    }
    // log2(e) / T as a number and what is left of it, within a range where nothing overflows
    Scale s;
    s.m = top;
    s.c = fminf(fmaxf(1.44269502f / T, 1e-36f), 5e36f);
    s.cl = s.c < 5e36f && s.c > 1e-36f ? (fmaf(-s.c, T, 1.44269502f) + 1.92596303e-8f) / T : 0.f;
    if (!(fabsf(s.cl) < 1e30f)) s.cl = 0.f;
    s.least = fmaxf(s.m - 44.f / s.c, -3.402823466e38f);
    auto weight = [&](float x) { return weight_of<WHOLE>(s, x); };
    // bins of equal width in log2 w; the last one takes everything below
    const float by = s.c * kPerOctave;
    // (the whole part of the product is in the significand's low bits, as in digits42)
    auto bin_of = [&](float x) {
        return (int)min(__float_as_uint(__fmaf_rz(s.m - x, by, 8388608.f)) - kBias, (uint32_t)(kBins - 1));
    };

    // which of a vector's elements lie in [from, to], few of them
    auto in_range = [&](const uint4 &y, float from, float to) {
        float2 x[VEC / 2];
        Vec<Tin>::unpack(y, x);
        uint32_t bits = 0;
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
            bits |= x[e].x >= from && x[e].x <= to ? 1u << (2 * e) : 0u;
            bits |= x[e].y >= from && x[e].y <= to ? 2u << (2 * e) : 0u;
        }
        return bits;
    };
    // f(i, x) over the warp's elements in [from, to]
    auto each_in = [&](float from, float to, auto f) {
        each_above(w0, w1, from, [&](int v, const uint4 &y) {
            for (uint32_t bits = in_range(y, from, to); bits != 0; bits &= bits - 1) {
                const int e = __ffs(bits) - 1;
                f(index_of(v) + e, Vec<Tin>::pick(y, e));
            }
        });
    };
    // A place in the list for each lane's n_of elements, in any order; `count` counts them all, the list holds
    // the first kList.  One atomic for the warp, none where it has no elements.
    auto places = [&](int n_of) {
        if (!__any_sync(0xffffffffu, n_of != 0)) return 0;
        int at = n_of;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += z;
        }
        int start = 0;
        if (lane == 31) start = atomicAdd(&count, at);
        return at + __shfl_sync(0xffffffffu, start, 31) - n_of;
    };
    auto enlist = [&](int at, float x, int i) {
        if (at < kList) list[at] = ordered(key_of(x), i);
    };
    // The warp's elements in [from, to] of which which(i, x) holds, to the list; four vectors of a lane at a time.
    auto collect = [&](float from, float to, auto which) {
#pragma unroll 1
        for (int v0 = w0; v0 < w1; v0 += 128) {
            uint4 y[4];
            uint32_t bits = 0;                  // VEC of each
#pragma unroll
            for (int g = 0; g < 4; ++g) y[g] = raw(v0 + 32 * g + lane, w1);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                y[g] = clean(y[g]);
                if (Vec<Tin>::largest(y[g]) >= from) bits |= in_range(y[g], from, to) << (VEC * g);
            }
            auto each = [&](auto f) {
                for (uint32_t left = bits; left != 0; left &= left - 1) {
                    const int b = __ffs(left) - 1, g = b / VEC, e = b % VEC;
                    f(b, index_of(v0 + 32 * g + lane) + e, Vec<Tin>::pick(g < 2 ? (g == 0 ? y[0] : y[1]) : g == 2 ? y[2] : y[3], e));
                }
            };
            each([&](int b, int i, float x) {
                if (!which(i, x)) bits &= ~(1u << b);
            });
            int at = places(__popc(bits));
            each([&](int, int i, float x) { enlist(at++, x, i); });
        }
    };
    // The elements from `from` on of the groups that reach it (a thread's vectors v + 32 g of every 128): each lane
    // takes its own groups one after another.
    auto collect_groups = [&](float from) {
        uint32_t groups = 0;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) groups |= my_top[g] >= from ? 1u << g : 0u;
        while (__any_sync(0xffffffffu, groups != 0)) {
            const int until = groups != 0 ? w1 : 0, g = groups != 0 ? __ffs(groups) - 1 : 0;
            groups &= groups - 1;
#pragma unroll 1
            for (int v0 = w0; v0 < w1; v0 += 512) {
                uint4 y[4];
                uint32_t bits = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = raw(v0 + 32 * g + lane + 128 * e, until);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[e] = clean(y[e]);
                    if (Vec<Tin>::largest(y[e]) >= from) bits |= in_range(y[e], from, s.m) << (VEC * e);
                }
                for (int at = places(__popc(bits)); bits != 0; bits &= bits - 1, ++at) {
                    const int b = __ffs(bits) - 1, i = b / VEC, e = b % VEC;
                    enlist(at, Vec<Tin>::pick(i < 2 ? (i == 0 ? y[0] : y[1]) : i == 2 ? y[2] : y[3], e),
                           index_of(v0 + 32 * g + lane + 128 * i) + e);
                }
            }
        }
    };
    // The weights of a vector's elements that are at least `from` and of which which(i, x) holds, added to two digits
    // of 21 bits (no thread has 1,024 elements).  No branches, so that a vector's weights are formed side by side.
    auto add_weights = [&](const uint4 &y, int v, float from, auto which, uint32_t &hi, uint32_t &lo) {
        float2 x[VEC / 2];
        Vec<Tin>::unpack(y, x);
        const int i = index_of(v);
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
            float2 high, low;
            digits42(weights2<WHOLE>(s, x[e]), high, low);
            const uint32_t h0 = digit(high.x), h1 = digit(high.y), l0 = digit(low.x), l1 = digit(low.y);
            const bool on0 = (x[e].x >= from) & which(i + 2 * e, x[e].x);
            const bool on1 = (x[e].y >= from) & which(i + 2 * e + 1, x[e].y);
            hi += (on0 ? h0 : 0) + (on1 ? h1 : 0);
            lo += (on0 ? l0 : 0) + (on1 ? l1 : 0);
        }
    };
    // The thread's part of those of vectors a .. b - 1, a warp's.
    auto weigh = [&](int a_, int b_, float from, auto which) {
        uint32_t hi = 0, lo = 0;
        each_above(a_, b_, from, [&](int v, const uint4 &y) { add_weights(y, v, from, which, hi, lo); });
        return ((u64)hi << 21) + lo;
    };
    // All weights added up, those above `to` as well, and the elements of [from, to] to the list; or, with
    // `above_too` not set, all elements from `from` on.
    auto weigh_and_collect = [&](float from, float to, auto above_too, u64 &all, u64 &above) {
        constexpr bool ABOVE = decltype(above_too)::value;
        uint32_t hi = 0, lo = 0, hi_above = 0, lo_above = 0;
        auto one = [&](const uint4 &y) {        // returns which are for the list
            uint32_t bits = 0;
            float2 x[VEC / 2];
            Vec<Tin>::unpack(y, x);
#pragma unroll
            for (int e = 0; e < VEC / 2; ++e) {
                float2 w = weights2<WHOLE>(s, x[e]), high, low;
                w.x = x[e].x >= s.least ? w.x : 0.f;
                w.y = x[e].y >= s.least ? w.y : 0.f;
                digits42(w, high, low);
                const uint32_t h0 = __float_as_uint(high.x), h1 = __float_as_uint(high.y);
                const uint32_t l0 = __float_as_uint(low.x), l1 = __float_as_uint(low.y);
                hi += h0 + h1;                  // (2^23's bits come off below: of all elements, or of a vector's)
                lo += l0 + l1;
                if (ABOVE) {
                    const bool up0 = x[e].x > to, up1 = x[e].y > to;
                    hi_above += (up0 ? h0 - kBias : 0u) + (up1 ? h1 - kBias : 0u);
                    lo_above += (up0 ? l0 - kBias : 0u) + (up1 ? l1 - kBias : 0u);
                    bits |= (!up0 & (x[e].x >= from) ? 1u << (2 * e) : 0u) | (!up1 & (x[e].y >= from) ? 2u << (2 * e) : 0u);
                } else {
                    bits |= (x[e].x >= from ? 1u << (2 * e) : 0u) | (x[e].y >= from ? 2u << (2 * e) : 0u);
                }
            }
            hi -= VEC * kBias;
            lo -= VEC * kBias;
            return bits;
        };
        // (four vectors of a lane on their way, and to the list, at a time; those for it are read once more)
#pragma unroll 1
        for (int v0 = w0; v0 < w1; v0 += 128) {
            uint4 y[4];
            uint32_t bits = 0;
#pragma unroll
            for (int g = 0; g < 4; ++g) y[g] = raw(v0 + 32 * g + lane, w1);
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {
                bits |= one(clean(y[0])) << (VEC * g);
                y[0] = y[1];
                y[1] = y[2];
                y[2] = y[3];
            }
            for (int at = places(__popc(bits)); bits != 0; bits &= bits - 1, ++at) {
                const int b = __ffs(bits) - 1, i = index_of(v0 + b / VEC * 32 + lane) + b % VEC;
                enlist(at, infinite ? 0.f : static_cast<float>(row[i]), i);
            }
        }
        all = ((u64)hi << 21) + lo;
        above = ((u64)hi_above << 21) + lo_above;
    };

    // Sums over all warps of all CTAs: every thread gets the total, what the warps before its own have,
    // and its warp's.  With its barrier the histograms are complete, too.
    int turn = 0;
    // what the warps before have of the parts that the warps left, and the total
    auto parts_before = [&](u64 &all) {
        __syncthreads();
        if (warp == 0) {
            const u64 x = lane < kWarps ? part[lane] : 0;
            u64 run = x;
#pragma unroll
            for (int o = 1; o < kWarps; o <<= 1) {
                const u64 z = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += z;
            }
            if (lane < kWarps) part[lane] = run - x;
            if (lane == kWarps - 1) part_all = run;
        }
        __syncthreads();
        all = part_all;
        return part[warp];
    };
    auto cluster_sum = [&](u64 x, u64 &before, u64 &here) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        here = x;
        __syncthreads();
        if (lane == 0) part[warp] = x;
        u64 all;
        before = parts_before(all);
        if (tid < ranks) *cluster.map_shared_rank(&totals[turn][rank], tid) = all;
        cluster.sync();
        all = 0;
        for (int r = 0; r < ranks; ++r) {
            before += r < rank ? totals[turn][r] : 0;
            all += totals[turn][r];
        }
        turn ^= 1;
        return all;
    };
    // Two totals over the cluster.
    auto cluster_totals = [&](u64 &x, u64 &y) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            x += __shfl_xor_sync(0xffffffffu, x, o);
            y += __shfl_xor_sync(0xffffffffu, y, o);
        }
        __syncthreads();
        if (lane == 0) {
            part[warp] = x;
            more[warp] = y;
        }
        __syncthreads();
        if (warp == 0) {
            x = lane < kWarps ? part[lane] : 0;
            y = lane < kWarps ? more[lane] : 0;
#pragma unroll
            for (int o = kWarps / 2; o > 0; o >>= 1) {
                x += __shfl_xor_sync(0xffffffffu, x, o);
                y += __shfl_xor_sync(0xffffffffu, y, o);
            }
            if (lane < ranks) {                 // (the lower half's sums: ranks <= kWarps)
                *cluster.map_shared_rank(&totals[turn][rank], lane) = x;
                *cluster.map_shared_rank(&more_totals[turn][rank], lane) = y;
            }
        }
        cluster.sync();
        x = y = 0;
        for (int r = 0; r < ranks; ++r) {
            x += totals[turn][r];
            y += more_totals[turn][r];
        }
        turn ^= 1;
    };
    // Two histograms in turn: when all have come together over one, the last one has been read.
    auto next_histogram = [&]() {
        hist = hist == hists ? hists + 2 * kBins : hists;
        for (int i = tid; i < 2 * kBins; i += kThreads) hist[i] = 0;
        __syncthreads();
    };
    // the thread's bin, added up over the cluster
    auto bin_sum = [&](int word) {
        uint32_t x[kMaxRanks];
#pragma unroll
        for (int r = 0; r < kMaxRanks; ++r) {   // (reads of all ranks on their way together)
            x[r] = 0;
            if (r < ranks) x[r] = cluster.map_shared_rank(hist, r)[word * kBins + tid];
        }
        u64 all = 0;
#pragma unroll
        for (int r = 0; r < kMaxRanks; ++r) all += x[r];
        return all;
    };
    // The first bin at which the bins, added up in order, reach want(total); `above` lies above the first
    // one.  Every CTA does it for itself.  Returns whether they do.
    auto border = [&](u64 x, u64 above, auto want, u64 *up_to = nullptr) {
        u64 run = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 z = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += z;
        }
        __syncthreads();
        if (lane == 31) part[warp] = run;
        u64 total;
        run += parts_before(total) + above;
        total += above;
        const u64 goal = want(total);
        if (up_to != nullptr) *up_to = run;
        if (run >= goal && run - x < goal) {
            found_bin = tid;
            found[0] = run - x;
            found[1] = x;
        }
        __syncthreads();
        return total >= goal;
    };
    auto add_weight = [&](int b, uint32_t hi, uint32_t lo) {        // (two digits of 21 bits)
        const uint32_t low = (hi << 21) + lo, old = atomicAdd(&hist[b], low);
        const uint32_t high = (hi >> 11) + (old + low < old ? 1u : 0u);
        if (high != 0) atomicAdd(&hist[kBins + b], high);
    };

    // What stays: values above the border, and of the equal ones those up to `last`.
    float border_at = -INFINITY;
    int32_t last = kAll;
    auto stays = [&](int i, float x) { return (x > border_at) | ((x == border_at) & (i <= last)); };
    auto lowest_value = [&]() { return fmaxf(border_at, -3.402823466e38f); };
    // the weight that top-p asks of a total (rounded up, at least something)
    auto share = [&](u64 total) {
        const u64 by64 = p > 0.f ? (u64)(p * 0x1p63f) << 1 : 0, whole = __umul64hi(total, by64);
        return max(total * by64 != 0 ? whole + 1 : whole, (u64)1);
    };
    // a value that is below all of the bins before b, give or take the roundings; and one above all from b on
    // (in bins from the maximum; never -infinity, which is what a vector holds beyond the row)
    auto below_bin = [&](float b) {
        const float x = s.m - b / by * (1.f + 1e-6f);
        return fmaxf(x - 4e-7f * (fabsf(s.m) + fabsf(x)) - 1e-37f, -3.402823466e38f);
    };
    auto above_bin = [&](float b) {
        const float x = s.m - b / by * (1.f - 1e-6f);
        return fminf(s.m, x + 4e-7f * (fabsf(s.m) + fabsf(x)) + 1e-37f);
    };

    // min-p lets by the values from least_at on: the least number that is not below the sum (NaN where there is none)
    float least_at;
    {
        const float b = least_log.x, sum = s.m + b, back = sum - s.m;
        least_at = fmaxf(__fadd_ru(sum, (s.m - (sum - back)) + (b - back) + least_log.y), -3.402823466e38f);
    }
    // Where top-p's border is, to a bin or two of log2 w, four times as narrow as the others: a value above all
    // candidates and one below.  A bin's weights lie within 2^(1/48) of each other, so it adds them up relative to
    // its own upper end, in whole multiples of 2^-fine, which 32 bits hold for all elements of a copy (a
    // quarter of the warps).  A sum of bins is off by less than 2^-fine and 2^-17 of it (2^-24 of log w, 30 at
    // most, three times) and 2^18 units of 2^-42, the sum of those above the border as well as of those below: the
    // lesser error counts, and `slack` is more than twice that.  Returns about how many elements of the row reach
    // `from`.  (Its copies lie where the two histograms in turn do: the cluster has come together since either was read.)
    auto candidates = [&](float &from, float &to) {
        const int fine = min(17, __clz(kWarps / kCopies * per_warp * VEC) - 1);
        const float by4 = 4.f * by, unit = __int_as_float((127 + fine) << 23);
        const uint32_t bins_at = tc::smem_u32(hists + warp % kCopies * kFine) - 4 * kBias;
#pragma unroll
        for (int c = 0; c < kCopies; ++c) reinterpret_cast<uint4 *>(hists + c * kFine)[tid] = make_uint4(0u, 0u, 0u, 0u);
        if (tid == 0) chosen_count = reach_least = 0;
        __syncthreads();
        each_vector(w0, w1, [&](int, const uint4 &y) {
            float2 x[VEC / 2];
            Vec<Tin>::unpack(y, x);
            // (nothing for a weight of zero: masked logits would all meet in one bin)
            auto add = [&](uint32_t b, float weight) {
                asm volatile("{\n.reg .pred some;\nsetp.ne.u32 some, %1, 0;\n@some red.shared.add.u32 [%0], %1;\n}\n"
                             ::"r"(bins_at + 4 * b), "r"(digit(weight)) : "memory");
            };
#pragma unroll
            for (int e = 0; e < VEC / 2; ++e) {
                auto both = [](float z) { return make_float2(z, z); };
                const float2 d = tc::f2sub(both(s.m), x[e]), b = fma_cut2(d, both(by4), both(8388608.f));
                const uint32_t b0 = min(__float_as_uint(b.x), kBias + kFine - 1), b1 = min(__float_as_uint(b.y), kBias + kFine - 1);
                // (the bins' upper ends, negated)
                const float2 ends = tc::f2sub(both(8388608.f), make_float2(__uint_as_float(b0), __uint_as_float(b1)));
                const float2 into = tc::f2fma(d, both(by4), ends);
                float2 w = make_float2(tc::ex2(into.x * (-0.25f / kPerOctave)), tc::ex2(into.y * (-0.25f / kPerOctave)));
                w = fma_cut2(w, both(unit), both(8388608.f));
                add(b0, w.x);
                add(b1, w.y);
            }
        });
        __syncthreads();
        // four bins to a thread
        float of_4[4];
        {
            u64 z[4] = {0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < kCopies; ++c) {
                const uint4 y = reinterpret_cast<const uint4 *>(hists + c * kFine)[tid];
                z[0] += y.x;
                z[1] += y.y;
                z[2] += y.z;
                z[3] += y.w;
            }
            reinterpret_cast<float4 *>(hists)[tid] = make_float4((float)z[0], (float)z[1], (float)z[2], (float)z[3]);
        }
        cluster.sync();
        of_4[0] = of_4[1] = of_4[2] = of_4[3] = 0.f;
#pragma unroll
        for (int r = 0; r < kMaxRanks; ++r) {   // (reads of all ranks on their way together)
            const float4 y = reinterpret_cast<const float4 *>(cluster.map_shared_rank(hists, r < ranks ? r : 0))[tid];
            of_4[0] += r < ranks ? y.x : 0.f;
            of_4[1] += r < ranks ? y.y : 0.f;
            of_4[2] += r < ranks ? y.z : 0.f;
            of_4[3] += r < ranks ? y.w : 0.f;
        }
        u64 bins[4], mine_w = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            bins[e] = __float2ull_rz(of_4[e] * exp2f((float)(42 - fine) - (float)(4 * tid + e) * (0.25f / kPerOctave)));
            mine_w += bins[e];
        }
        u64 run = 0, goal = 0, twice = 0;
        border(mine_w, 0, [&](u64 total) {
            goal = share(total);
            twice = 2 * total;
            return goal;
        }, &run);
        auto slack = [&](u64 up_to) { return (min(up_to + goal, twice - up_to - goal) >> (fine - 2)) + (1 << 20); };
        // the first bin with which the sum may reach the goal, and the first with which it must
        if (tid == 0) {
            found_bin = 0;
            found_last = kFine - 1;
        }
        __syncthreads();
        run -= mine_w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const u64 next = run + bins[e];
            if (next + slack(next) >= goal && run + slack(run) < goal) found_bin = 4 * tid + e;
            if (next >= goal + slack(next) && run < goal + slack(run)) found_last = 4 * tid + e;
            run = next;
        }
        __syncthreads();
        const int last_bin = found_last;
        to = above_bin(0.25f * (float)found_bin);
        from = last_bin == kFine - 1 ? -3.402823466e38f : below_bin(0.25f * (float)(last_bin + 1));
        // about how many reach `from`, and how many reach min-p's weight
        const float least_bin = fminf((s.m - least_at) * by4, (float)kFine);
        float about = 0.f, about_least = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            about += 4 * tid + e <= last_bin + 1 ? of_4[e] : 0.f;
            about_least += (float)(4 * tid + e) <= least_bin ? of_4[e] : 0.f;
        }
        const int of_warp = __reduce_add_sync(0xffffffffu, (int)(about * 1.03f / unit) + 1);
        const int least_of_warp = __reduce_add_sync(0xffffffffu, (int)(about_least / unit));
        if (lane == 0) {
            atomicAdd(&chosen_count, of_warp);
            atomicAdd(&reach_least, least_of_warp);
        }
        __syncthreads();
        return chosen_count - kThreads;
    };

    // The block's sums up to each of a thread's four elements; returns all.
    auto scan4 = [&](const u64 (&w)[4], u64 (&cum)[4]) {
        u64 run = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            run += w[e];
            cum[e] = run;
        }
        const u64 own = run;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 z = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += z;
        }
        __syncthreads();
        if (lane == 31) part[warp] = run;
        u64 all;
        const u64 add = parts_before(all) + run - own;
#pragma unroll
        for (int e = 0; e < 4; ++e) cum[e] += add;
        return all;
    };
    // The lengths of all CTAs' lists, one to a lane: `upto` is what the lists up to the lane's have, all is returned.
    auto lengths = [&](int &length, int &upto) {
        length = lane < ranks ? *cluster.map_shared_rank(&count, lane) : 0;
        upto = length;
#pragma unroll
        for (int o = 1; o < kMaxRanks; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += z;
        }
        return __shfl_sync(0xffffffffu, upto, kMaxRanks - 1);
    };
    // The lists one after another, warp r bringing rank r's.
    auto bring = [&](u64 *to, int length, int upto) {
        if (warp < ranks) {
            const int c = __shfl_sync(0xffffffffu, length, warp), at = __shfl_sync(0xffffffffu, upto, warp) - c;
            const u64 *from = cluster.map_shared_rank(list, warp);
            if (to + at != from)
                for (int i = lane; i < c; i += 32) to[at + i] = from[i];
        }
        __syncthreads();
    };

    // Narrows the border down to the first elements of the order that reach a count (k) or a share of
    // the weight: first by bins of log2 w, then by the values' bits.  ahead_w: of top-p's weights, what the
    // thread has above the candidates.
    u64 ahead_w = 0;
    int pooled = 0;
    bool listed = false;                        // the list holds all that stays
    bool summed = true;                         // ahead_w holds what is above the list's
    auto narrow = [&](bool by_weight) {
        u64 want = (u64)k, above = 0, before, here;
        int bin = -1;
        uint32_t most, lowest;
        auto goal = [&](u64 total) {
            if (by_weight) want = share(total);
            return want;
        };
        auto in_bin = [&](int i, float x) { return stays(i, x) && (bin < 0 || bin_of(x) == bin); };
        if (tid == 0) count = 0;
        if (by_weight && border_at == -INFINITY) {
            float from, to;
            const int about = candidates(from, to);
            if (least_at > to) {
                // min-p lets by less than top-p does
                if (reach_least <= kListAll) {
                    collect(least_at, s.m, [](int, float) { return true; });
                    __syncthreads();
                    pooled = count;
                    listed = pooled <= kListAll;
                }
                return;
            }
            u64 total = 0;
            bool again = about > kListAll;
            if (!again) {
                // few enough to be taken from the list, all that stay; one thread adds a mark where there are more (a
                // list's weights are below 2^54, eight marks below 2^64)
                constexpr u64 kTooMany = 1ull << 60;
                weigh_and_collect(from, to, std::false_type{}, total, above);
                __syncthreads();
                const int have = min(count, kList);
                above = tid == 0 && count > kList ? kTooMany : 0;
                for (int i = tid; i < have; i += kThreads) {
                    const float x = value_of(ordered_key(list[i]));
                    above += x > to ? weight(x) : 0;
                }
                cluster_totals(total, above);
                again = above >= kTooMany;
                listed = !again;
                if (again) {
                    if (tid == 0) count = 0;
                    __syncthreads();
                }
            }
            if (again) {
                weigh_and_collect(from, to, std::true_type{}, total, ahead_w);
                above = ahead_w;
                cluster_totals(total, above);
            }
            goal(total);
            most = key_of(to);
            lowest = key_of(from);
            int length, upto;
            const int all = lengths(length, upto);
            if (all <= kThreads) {
                // few candidates in all: sorted in one CTA (in the histograms' place; one row of 131,072 by top-p 52 -> 40
                // us; for up to 2,048 of them the sort takes as long as the histograms, with the other CTAs waiting)
                if (rank == 0) {
                    u64 *const room = reinterpret_cast<u64 *>(hists), *const together = room + kThreads;
                    bring(together, length, upto);
                    u64 c[4], w[4], cum[4];
                    int size = 2;
                    while (size < all) size *= 2;
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[e] = 4 * tid + e < all ? together[4 * tid + e] : 0;
                    sort_down(c, room, size);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t key = ordered_key(c[e]);
                        w[e] = 4 * tid + e < all && key <= most ? weight(value_of(key)) : 0;    // (others are above)
                    }
                    scan4(w, cum);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (above + cum[e] >= want && above + cum[e] - w[e] < want)
                            for (int r = 0; r < ranks; ++r) {
                                *cluster.map_shared_rank(&chosen_key, r) = ordered_key(c[e]);
                                *cluster.map_shared_rank(&chosen_index, r) = ordered_index(c[e]);
                            }
                }
                cluster.sync();
                pooled = count;
                border_at = value_of(chosen_key);
                last = chosen_index;
                return;
            }
        } else {
            next_histogram();
            each_in(lowest_value(), s.m, [&](int i, float x) {
                if (!stays(i, x)) return;
                if (by_weight) {
                    const u64 w = weight(x);
                    if (w != 0) add_weight(bin_of(x), (uint32_t)(w >> 21), (uint32_t)w & 0x1fffffu);
                } else {
                    atomicAdd(&hist[bin_of(x)], 1u);
                }
            });
            cluster.sync();
            if (!border(by_weight ? bin_sum(0) + (bin_sum(1) << 32) : bin_sum(0), 0, goal)) {
                // fewer: all stay.  No CTA leaves while another reads its bins: top-p's first histogram takes the place
                // of both in turn
                cluster.sync();
                return;
            }
            bin = found_bin;
            above = found[0];
            most = key_of(above_bin((float)bin));
            lowest = key_of(bin == kBins - 1 ? -3.402823466e38f : below_bin((float)(bin + 1)));
            collect(value_of(lowest), value_of(most), in_bin);
        }
        __syncthreads();
        pooled = count;
        listed = listed && pooled <= kList;
        for (;;) {
            const int shift = max(Vec<Tin>::GRAIN, 23 - __clz(most - lowest));      // 2^9 bins at most
            next_histogram();
            auto add = [&](uint32_t key) {
                const int b = (int)((most - key) >> shift);
                if (by_weight) {
                    const u64 w = weight(value_of(key));
                    if (w != 0) add_weight(b, (uint32_t)(w >> 21), (uint32_t)w & 0x1fffffu);
                } else {
                    atomicAdd(&hist[b], 1u);
                }
            };
            if (pooled <= kList) {
                for (int i = tid; i < pooled; i += kThreads) {
                    const uint32_t key = ordered_key(list[i]);
                    if (key >= lowest && key <= most) add(key);
                }
            } else {
                each_in(value_of(lowest), value_of(most), [&](int i, float x) { if (in_bin(i, x)) add(key_of(x)); });
            }
            cluster.sync();
            // (the candidates' values lie in that range, so they reach it)
            if (!border(by_weight ? bin_sum(0) + (bin_sum(1) << 32) : bin_sum(0), above, [&](u64) { return want; })) {
                cluster.sync();
                return;
            }
            above = found[0];
            most -= (uint32_t)found_bin << shift;
            if (shift == Vec<Tin>::GRAIN) break;
            lowest = max(lowest, most - ((1u << shift) - 1));
            if (pooled > kList) {
                // what is left may fit
                __syncthreads();
                if (tid == 0) count = 0;
                __syncthreads();
                collect(value_of(lowest), value_of(most), in_bin);
                __syncthreads();
                pooled = count;
                summed = false;
            }
        }
        if (Vec<Tin>::GRAIN > 0) {
            // the one key in (most - 2^GRAIN, most]: negative values' keys end in ones
            const uint32_t ones = (1u << Vec<Tin>::GRAIN) - 1;
            most = (most >> 31) != 0 ? most & ~ones : ((most + 1) & ~ones) - 1;
        }
        // the values equal to the border's: the first of them by their index
        const float it = value_of(most);
        const u64 one = by_weight ? weight(it) : 1, keep = (want - above + one - 1) / one;
        int32_t until = kAll;
        if (found[1] > one) {                   // (where only one is there, it stays)
            u64 equal = 0;
            const bool in_pool = pooled <= kList;
            if (in_pool) {
                for (int i = tid; i < pooled; i += kThreads) equal += ordered_key(list[i]) == most ? 1 : 0;
            } else {
                each_in(it, it, [&](int i, float x) { equal += stays(i, x) ? 1 : 0; });
            }
            const u64 all = cluster_sum(equal, before, here);
            if (keep < all) {
                auto publish = [&](int at) {
                    for (int r = 0; r < ranks; ++r) *cluster.map_shared_rank(&chosen_index, r) = at;
                };
                const u64 ahead = before - part[warp];          // of the CTAs before
                if (in_pool) {
                    // the one by its index in the CTA, the index's upper half first
                    if (keep > ahead && keep <= ahead + part_all) {
                        u64 passed = ahead;
                        int upper = -1;
                        for (int level = 0; level < 2; ++level) {
                            next_histogram();
                            for (int i = tid; i < pooled; i += kThreads) {
                                const int at = ordered_index(list[i]);
                                if (ordered_key(list[i]) == most && (level == 0 || at / kBins == upper))
                                    atomicAdd(&hist[level == 0 ? at / kBins : at % kBins], 1u);
                            }
                            __syncthreads();
                            border(hist[tid], passed, [&](u64) { return keep; });
                            if (level == 0) {
                                upper = found_bin;
                                passed = found[0];
                            }
                        }
                        if (tid == 0) publish(upper * kBins + found_bin);
                    }
                } else if (keep > before && keep <= before + here) {
                    // this warp has the last one
                    u64 seen = before;
                    for (int v0 = w0; v0 < w1; v0 += 32) {
                        const int v = v0 + lane;
                        const uint4 y = clean(raw(v, w1));
                        uint32_t bits = in_range(y, it, it);
                        for (int e = 0; e < VEC; ++e)
                            if (!stays(index_of(v) + e, it)) bits &= ~(1u << e);
                        int run = __popc(bits);
                        const int cnt = run;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const int z = __shfl_up_sync(0xffffffffu, run, o);
                            if (lane >= o) run += z;
                        }
                        if (keep > seen + run - cnt && keep <= seen + run) {
                            for (int c = (int)(keep - (seen + run - cnt)); c > 1; --c) bits &= bits - 1;
                            publish(index_of(v) + __ffs(bits) - 1);
                        }
                        seen += __shfl_sync(0xffffffffu, run, 31);
                    }
                }
                cluster.sync();
                until = chosen_index;
            }
        }
        last = it == border_at ? min(last, until) : until;
        border_at = it;
    };

    u64 sum = 0;                                // of what stays
    // the first token whose running sum exceeds floor(u sum / 2^24) (the sum of all does, since u < 2^24)
    auto drawn = [&]() {
        const uint32_t tick = __float2uint_rz(fminf(fmaxf(u, 0.f) * 16777216.f, 16777215.f));
        return __umul64hi((u64)tick << 40, sum);
    };

    // ---- a small k: the few logits that can be among the first k, sorted in one CTA
    bool done = false;
    if (!none && k > 0 && k < V && k <= kListK) {
        // k of the groups' largest logits lie in the bins up to this one
        next_histogram();
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
            if (my_top[g] != -INFINITY) atomicAdd(&hist[bin_of(my_top[g])], 1u);
        cluster.sync();
        const float from = border(bin_sum(0), 0, [&](u64) { return (u64)k; }) && found_bin < kBins - 1
                               ? below_bin((float)(found_bin + 1)) : -3.402823466e38f;
        collect_groups(from);
        cluster.sync();
        // the lists' lengths, a rank to a lane; warp r brings rank r's to the first CTA
        int length, upto;
        const int all = lengths(length, upto);
        done = all <= kSorted;
        if (done && rank == 0) {
            if (tid == 0) chosen_count = 0;
            bring(list, length, upto);
            auto choose = [&](u64 c, u64 all_of_it) {           // c is the last of the order that stays
                for (int r = 0; r < ranks; ++r) {
                    *cluster.map_shared_rank(&chosen_key, r) = ordered_key(c);
                    *cluster.map_shared_rank(&chosen_index, r) = ordered_index(c);
                    *cluster.map_shared_rank(&chosen_sum, r) = all_of_it;
                }
            };
            if (all <= kFew) {
                // Every pair is compared, four threads to an element: which stand before it in the order, and
                // what they weigh; then what those weigh that stay and have a smaller index.
                u64 *const weights = list + kFew;
                for (int i = tid; i < all; i += kThreads) weights[i] = weight(value_of(ordered_key(list[i])));
                __syncthreads();
                const int i = tid >> 2, h = tid & 3;
                const u64 mine_c = i < all ? list[i] : 0, mine_w = i < all ? weights[i] : 0;
                int place = 0;
                u64 ahead = 0;
                for (int j = h; j < all; j += 4) {
                    const bool it = list[j] > mine_c;
                    place += it ? 1 : 0;
                    ahead += it ? weights[j] : 0;
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    place += __shfl_xor_sync(0xffffffffu, place, o);
                    ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
                }
                // sums over the block, each element once
                auto block_sum = [&](u64 x) {
                    x = h == 0 ? x : 0;
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                    __syncthreads();
                    if (lane == 0) part[warp] = x;
                    __syncthreads();
                    x = 0;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) x += part[w];
                    return x;
                };
                const bool of_k = i < all && place < k;
                const u64 goal = p < 1.f ? share(block_sum(of_k ? mine_w : 0)) : ~(u64)0;
                const bool stay = of_k && ahead < goal && value_of(ordered_key(mine_c)) >= least_at;
                __syncthreads();
                if (i < all && h == 0) weights[i] = stay ? mine_w : 0;
                if (stay && h == 0) atomicAdd(&chosen_count, 1);
                sum = block_sum(stay ? mine_w : 0);
                if (stay && h == 0 && place == chosen_count - 1) choose(mine_c, sum);
                if (a.token != nullptr) {
                    u64 run = 0;
                    for (int j = h; j < all; j += 4) run += ordered_index(list[j]) <= ordered_index(mine_c) ? weights[j] : 0;
#pragma unroll
                    for (int o = 1; o < 4; o <<= 1) run += __shfl_xor_sync(0xffffffffu, run, o);
                    const u64 need = drawn();
                    if (stay && h == 0 && run > need && run - mine_w <= need) a.token[n] = ordered_index(mine_c);
                }
            } else {
                // Sorted, four elements to a thread, and summed up in the order.
                u64 c[4], w[4], cum[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) c[e] = 4 * tid + e < all ? list[4 * tid + e] : 0;
                __syncthreads();
                int size = 2;
                while (size < all) size *= 2;
                sort_down(c, list, size);
                const int first_k = min(k, all);
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = 4 * tid + e < first_k ? weight(value_of(ordered_key(c[e]))) : 0;
                const u64 of_k = scan4(w, cum);
                const u64 goal = p < 1.f ? share(of_k) : ~(u64)0;
                int stay = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    stay += 4 * tid + e < first_k && cum[e] - w[e] < goal && value_of(ordered_key(c[e])) >= least_at ? 1 : 0;
                stay = __reduce_add_sync(0xffffffffu, stay);
                if (lane == 0 && stay != 0) atomicAdd(&chosen_count, stay);
                __syncthreads();
                stay = chosen_count;            // a beginning of the order
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * tid + e == stay - 1) choose(c[e], cum[e]);
                if (a.token != nullptr) {
                    // in index order: by the index's upper half, then by its lower half
                    __syncthreads();
                    sum = chosen_sum;
                    const u64 need = drawn();
                    u64 ahead = 0;
                    int upper = -1;
                    for (int level = 0; level < 2; ++level) {
                        next_histogram();
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int i = ordered_index(c[e]);
                            if (4 * tid + e < stay && (level == 0 || i / kBins == upper))
                                add_weight(level == 0 ? i / kBins : i % kBins, (uint32_t)(w[e] >> 21),
                                           (uint32_t)w[e] & 0x1fffffu);
                        }
                        __syncthreads();
                        border(hist[tid] + ((u64)hist[kBins + tid] << 32), ahead, [&](u64) { return need + 1; });
                        if (level == 0) {
                            upper = found_bin;
                            ahead = found[0];
                        }
                    }
                    if (tid == 0) a.token[n] = upper * kBins + found_bin;
                }
            }
        }
        cluster.sync();
        if (done) {
            border_at = value_of(chosen_key);
            last = chosen_index;
            sum = chosen_sum;
        }
    }
    if (!none && !done) {
        if (k > 0 && k < V) narrow(false);
        if (p < 1.f) narrow(true);
        // ---- the draw, in index order
        u64 before, here;
        u64 mine_w = 0;
        const float from = fmaxf(fmaxf(lowest_value(), s.least), least_at);
        auto in_list = [&](u64 c, u64 &w) {     // does it stay, and its weight
            const float x = value_of(ordered_key(c));
            w = weight(x);
            return stays(ordered_index(c), x) && x >= least_at;
        };
        // (min-p lets all by that top-p does)
        const bool all_pass = border_at > -INFINITY && border_at >= least_at;
        if (listed || (all_pass && summed && pooled <= kList && !(k > 0 && k < V))) {
            // what lies above the candidates was summed up with them, unless they are in the list, too; of those, what
            // stays, to the warps that have it
            if (tid < kWarps) more[tid] = 0;
            __syncthreads();
            for (int i = tid; i < pooled; i += kThreads) {
                u64 w;
                if (in_list(list[i], w)) atomicAdd(&more[((ordered_index(list[i]) + lead) / VEC - first) / per_warp], w);
            }
            __syncthreads();
            mine_w = ahead_w + (lane == 0 ? more[warp] : 0);
        } else if (border_at == -INFINITY) {
            uint32_t hi = 0, lo = 0;
            each_above(w0, w1, from, [&](int, const uint4 &y) {
                float2 x[VEC / 2];
                Vec<Tin>::unpack(y, x);
#pragma unroll
                for (int e = 0; e < VEC / 2; ++e) {
                    float2 w = weights2<WHOLE>(s, x[e]), high, low;
                    w.x = x[e].x >= from ? w.x : 0.f;
                    w.y = x[e].y >= from ? w.y : 0.f;
                    digits42(w, high, low);
                    hi += __float_as_uint(high.x) + __float_as_uint(high.y);
                    lo += __float_as_uint(low.x) + __float_as_uint(low.y);
                }
                hi -= VEC * kBias;
                lo -= VEC * kBias;
            });
            mine_w = ((u64)hi << 21) + lo;
        } else {
            mine_w = weigh(w0, w1, from, stays);
        }
        sum = cluster_sum(mine_w, before, here);
        const u64 need = drawn();
        const bool hit = a.token != nullptr && before <= need && before + here > need;
        const u64 of_before = before - part[warp];      // (of the CTAs before)
        if (__syncthreads_or(hit ? 1 : 0) == 0) {
            // another CTA has it
        } else if (listed) {
            u64 passed = of_before;
            int upper = -1;
            for (int level = 0; level < 2; ++level) {
                next_histogram();
                for (int i = tid; i < pooled; i += kThreads) {
                    const int at = ordered_index(list[i]);
                    u64 w;
                    if (in_list(list[i], w) && (level == 0 || at / kBins == upper))
                        add_weight(level == 0 ? at / kBins : at % kBins, (uint32_t)(w >> 21), (uint32_t)w & 0x1fffffu);
                }
                __syncthreads();
                border(hist[tid] + ((u64)hist[kBins + tid] << 32), passed, [&](u64) { return need + 1; });
                if (level == 0) {
                    upper = found_bin;
                    passed = found[0];
                }
            }
            if (tid == 0) a.token[n] = upper * kBins + found_bin;
        } else {
            // the warp's vectors that hold the token, shared out over the CTA's warps
            if (hit && lane == 0) {
                found_bin = warp;
                found[0] = before;
            }
            __syncthreads();
            const int v0 = min(mine, found_bin * per_warp), v1 = min(mine, v0 + per_warp);
            const int each = (v1 - v0 + kWarps - 1) / kWarps, a0 = min(v1, v0 + warp * each), a1 = min(v1, a0 + each);
            u64 x = weigh(a0, a1, from, stays), run_all;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            if (lane == 0) part[warp] = x;
            u64 at = parts_before(run_all) + found[0];
            if (at <= need && at + x > need) {
                for (int b0 = a0; b0 < a1; b0 += 32) {
                    const int v = b0 + lane;
                    uint32_t hi = 0, lo = 0;
                    const uint4 y = clean(raw(v, a1));
                    add_weights(y, v, from, stays, hi, lo);
                    const u64 own = ((u64)hi << 21) + lo;
                    u64 run = own;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const u64 z = __shfl_up_sync(0xffffffffu, run, o);
                        if (lane >= o) run += z;
                    }
                    const unsigned hits = __ballot_sync(0xffffffffu, at + run > need);
                    if (hits != 0) {
                        if (lane == __ffs(hits) - 1) {
                            at += run - own;
                            int i = index_of(v);
                            for (int e = 0; e < VEC - 1; ++e, ++i) {
                                const float z = Vec<Tin>::pick(y, e);
                                at += z >= from && stays(i, z) ? weight(z) : 0;
                                if (at > need) break;
                            }
                            a.token[n] = i;
                        }
                        break;
                    }
                    at += __shfl_sync(0xffffffffu, run, 31);
                }
            }
        }
    } else if (none && a.token != nullptr && rank == 0 && tid == 0) {
        a.token[n] = -1;
    }
    if (a.probs != nullptr) {
        const float inv = none ? 0.f : (float)(0x1p42 / (double)sum);
        const bool bf16 = a.probs_bf16 != 0;
        Scale deep = s;                         // down to 2^-125
        deep.least = fmaxf(s.m - 125.f / s.c, -3.402823466e38f);
        const float from = none ? INFINITY : fmaxf(fmaxf(lowest_value(), deep.least), least_at);
        unsigned char *out = static_cast<unsigned char *>(a.probs) + n * (int64_t)V * (bf16 ? 2 : 4);
        // whole vectors where the output's rows lie as the input's
        const bool whole = ((reinterpret_cast<uintptr_t>(out) - (size_t)lead * (bf16 ? 2 : 4)) & (bf16 ? VEC * 2 - 1 : 15)) == 0;
        each_vector(w0, w1, [&](int v, const uint4 &raw) {
            if (v >= w1) return;
            const int e0 = index_of(v);
            float y[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) y[e] = 0.f;
            if (Vec<Tin>::largest(raw) >= from) {
                float2 x[VEC / 2];
                Vec<Tin>::unpack(raw, x);
#pragma unroll
                for (int e = 0; e < VEC / 2; ++e) {
                    const float2 w = weights2<true>(deep, x[e]);
                    y[2 * e] = (x[e].x >= from) & stays(e0 + 2 * e, x[e].x) ? w.x * inv : 0.f;
                    y[2 * e + 1] = (x[e].y >= from) & stays(e0 + 2 * e + 1, x[e].y) ? w.y * inv : 0.f;
                }
            }
            if (bf16) {
                __nv_bfloat16 *to = reinterpret_cast<__nv_bfloat16 *>(out) + e0;
                if (whole && e0 >= 0 && e0 + VEC <= V) {
                    uint32_t z[VEC / 2];
#pragma unroll
                    for (int e = 0; e < VEC / 2; ++e) z[e] = tc::pack_bf16x2(y[2 * e], y[2 * e + 1]);
                    if (VEC == 8) *reinterpret_cast<uint4 *>(to) = make_uint4(z[0], z[1], z[2], z[VEC / 2 - 1]);
                    else *reinterpret_cast<uint2 *>(to) = make_uint2(z[0], z[1]);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        if (e0 + e >= 0 && e0 + e < V) to[e] = __float2bfloat16_rn(y[e]);
                }
            } else {
                float *to = reinterpret_cast<float *>(out) + e0;
                if (VEC == 8 && (reinterpret_cast<uintptr_t>(to) & 31) == 0 && e0 >= 0 && e0 + VEC <= V) {
                    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "f"(y[0]), "f"(y[1]),
                                 "f"(y[2]), "f"(y[3]), "f"(y[4 % VEC]), "f"(y[5 % VEC]), "f"(y[6 % VEC]), "f"(y[7 % VEC]) : "memory");
                } else if (whole && e0 >= 0 && e0 + VEC <= V) {
#pragma unroll
                    for (int e = 0; e < VEC; e += 4)
                        *reinterpret_cast<float4 *>(to + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        if (e0 + e >= 0 && e0 + e < V) to[e] = y[e];
                }
            }
        });
    }
    cluster.sync();                             // no CTA leaves while its shared memory is read
}

// How many clusters of so many CTAs the device holds at once; asked once per device.
template <typename Tin> int clusters_at_once(int ranks, cudaLaunchConfig_t &cfg, cudaLaunchAttribute &cluster) {
    static std::atomic<int> known[64][kMaxRanks + 1];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const bool keep = dev >= 0 && dev < 64;
    if (keep && (n = known[dev][ranks].load(std::memory_order_relaxed)) != 0) return n;
    cfg.gridDim = dim3((unsigned)ranks);
    cluster.val.clusterDim.x = ranks;
    if (cudaOccupancyMaxActiveClusters(&n, sample_kernel<Tin>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        n = 0;
    }
    if (keep && n > 0) known[dev][ranks].store(n, std::memory_order_relaxed);
    return n;
}

template <typename Tin> cudaError_t run(const Sampling &a, int32_t N, cudaStream_t stream) {
    constexpr int VEC = Vec<Tin>::N;
    const int vecs = (a.V + VEC - 1) / VEC + 1;
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = allow_dynamic_smem(sample_kernel<Tin>, kSmem, smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.y = 1;
    cluster.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.attrs = &cluster;
    cfg.numAttrs = 1;
    // the largest clusters with which all rows run at once, of CTAs that have something to do
    int ranks = kMaxRanks;
    while (ranks > 1 && (vecs < ranks * 256 || N > clusters_at_once<Tin>(ranks, cfg, cluster))) --ranks;
    const int slice = (vecs + ranks - 1) / ranks;
    cfg.gridDim = dim3((unsigned)N * ranks);
    cluster.val.clusterDim.x = ranks;
    cfg.stream = stream;
    e = cudaLaunchKernelEx(&cfg, sample_kernel<Tin>, a, (int32_t)slice);
    if (e == cudaSuccess) count_launches(1);
    else (void)cudaGetLastError();                     // reported here
    return e;
}

}  // namespace

cudaError_t launch_sample(const void *logits, int64_t stride, int32_t N, int32_t V, kda_dtype dt, const float *temperature,
                          const int32_t *top_k, const float *top_p, const float *min_p, const float *uniforms,
                          int32_t *token, void *probs, kda_dtype probs_dt, cudaStream_t stream) {
    const Sampling a{logits, stride, temperature, top_p, min_p, uniforms, top_k, V, token, probs, probs_dt == KDA_BF16};
    return dt == KDA_BF16 ? run<__nv_bfloat16>(a, N, stream) : run<float>(a, N, stream);
}

}  // namespace kda
