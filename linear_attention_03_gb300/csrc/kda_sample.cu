// kda_sample.cu -- from logits to the distribution that is drawn from, and a token
// (kda_sample): temperature, top-k, top-p, min-p and the draw from a given uniform number.
//
//     w_i = e^{(x_i - max x) / T},   order: by value, then by index
//     top-k: the first k of the order;  top-p: of these the shortest beginning with a p-th of their
//     weight;  min-p: of these the ones with w_i >= m;  the token: the first index at which the
//     weights of the ones that stay, added up in index order, exceed u times their sum
//
// Weights are whole multiples of 2^-42, held in 64 bits, so sums do not depend on their order.
// Each is right to some 2^-24 of itself, with errors of either sign: the draw moves by a token at
// fewer than one in 10^5 rows.
//
// A cluster of up to eight CTAs takes a row and keeps it in shared memory, so that the logits
// are read once.  What stays is a beginning of the order: a border value, and the
// last index among the logits equal to it.
//   A small k: k of the threads' largest logits bound the k-th largest from below; the few logits
// above the bound go to one CTA, which makes the whole choice there, the draw included.
//   Otherwise histograms narrow the values down, first by w (bins of equal width in log2 w,
// which spread the logits well whatever their scale), then by the value's bits: of counts for a
// large k, of weights for top-p.
#include "kda_internal.cuh"
#include "kda_tc.cuh"

#include <cooperative_groups.h>

namespace kda {
namespace {

typedef unsigned long long u64;
constexpr int kThreads = 512, kWarps = kThreads / 32, kMaxRanks = 8;
constexpr int kBins = 512;                      // of a histogram
constexpr float kPerOctave = 12.f;              // bins for a halving of w
constexpr int kList = 2048, kListK = 1024;      // logits that go to one CTA at most, and the k for which that is tried
constexpr int kFew = 128;                       // logits of which every pair is compared instead
constexpr int32_t kAll = 0x7fffffff;
// two histograms and a list; a row of 2^18 logits over eight CTAs beside them
constexpr int kScratch = 4 * kBins * 4 + kList * 8;
constexpr int kMaxSmem = KDA_MAX_VOCABULARY / kMaxRanks * 4 + 32 + kScratch;
static_assert(kList == 4 * kThreads && 4 * kFew == kThreads && 2 * kFew <= kList, "threads to the elements of a list");
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
    static __device__ __forceinline__ uint32_t clean(uint32_t w) {
        return __float_as_uint(fmaxf(__uint_as_float(w), -INFINITY));
    }
    static __device__ __forceinline__ float largest(uint4 u) {
        return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
    }
    static __device__ __forceinline__ float load(const uint4 *p, int e) { return reinterpret_cast<const float *>(p)[e]; }
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
    static __device__ __forceinline__ uint32_t clean(uint32_t w) { return max2(w, 0xff80ff80u); }
    static __device__ __forceinline__ float largest(uint4 u) {
        const uint32_t m = max2(max2(u.x, u.y), max2(u.z, u.w));
        return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    }
    static __device__ __forceinline__ float load(const uint4 *p, int e) {
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[e]);
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

// The weights of two logits, to 2^-24: x - m with its rounding error, the product with c in one
// rounding behind the point, 2^f by its series (to 2^-27 for |f| <= 1/2) and the exponent put on
// in whole numbers.  Paired arithmetic: some 12 instructions a weight.  (No number of meaning below s.least.)
__device__ __forceinline__ float2 weights2(const Scale &s, float2 x) {
    auto both = [](float a) { return make_float2(a, a); };
    const float2 d = tc::f2sub(x, both(s.m)), mv = tc::f2sub(x, d), xv = tc::f2add(d, mv);
    const float2 err = tc::f2add(tc::f2sub(x, xv), tc::f2sub(mv, both(s.m)));
    const float2 t = tc::f2fma(d, both(s.c), both(12582912.f)), whole = tc::f2sub(both(12582912.f), t);
    float2 f = tc::f2fma(d, both(s.c), whole);
    f = tc::f2fma(d, both(s.cl), f);
    f = tc::f2fma(err, both(s.c), f);
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
__device__ __forceinline__ u64 weight(const Scale &s, float x) {
    const float w = weights2(s, make_float2(x, x)).x;
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

template <typename Tin>
__global__ void __launch_bounds__(kThreads, 2)
sample_kernel(const Sampling a, const int32_t slice) {
    constexpr int VEC = Vec<Tin>::N;
    extern __shared__ __align__(16) unsigned char smem[];
    uint4 *const data = reinterpret_cast<uint4 *>(smem);            // the CTA's vectors of the row
    // two histograms (low words, then high words) and a list
    uint32_t *const hists = reinterpret_cast<uint32_t *>(smem + (size_t)slice * 16), *hist = hists;
    u64 *const list = reinterpret_cast<u64 *>(hists + 4 * kBins);
    __shared__ u64 part[kWarps], part_all, chosen_sum, totals[2][kMaxRanks], more[kWarps], more_totals[kMaxRanks];
    __shared__ u64 found[2];                    // what lies above the border's bin, what is in it
    __shared__ float tops[kMaxRanks], warp_top[kWarps];
    __shared__ int32_t found_bin, chosen_index, count, chosen_count;
    __shared__ uint32_t chosen_key;
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

    // ---- the row into shared memory, and its maximum
    float my_top = -INFINITY;
#pragma unroll 4
    for (int v = w0 + lane; v < w1; v += 32) {
        const int e0 = index_of(v);
        uint4 x;
        if (e0 >= 0 && e0 + VEC <= V) {
            x = __ldg(grid + v);
        } else {                                // the row's ends
            Tin y[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                y[e] = static_cast<Tin>(-INFINITY);
                if (e0 + e >= 0 && e0 + e < V) y[e] = row[e0 + e];
            }
            memcpy(&x, y, 16);
        }
        x.x = Vec<Tin>::clean(x.x);
        x.y = Vec<Tin>::clean(x.y);
        x.z = Vec<Tin>::clean(x.z);
        x.w = Vec<Tin>::clean(x.w);
        data[v] = x;
        my_top = fmaxf(my_top, Vec<Tin>::largest(x));
    }
    if (!(T > 0.f)) {                           // the first of the order alone
        T = 1.f;
        k = 1;
    }
    if (k == 1) p = 1.f;
    float top = my_top;
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
    if (top == INFINITY) {                      // the infinite ones share everything
        for (int v = w0 + lane; v < w1; v += 32) {
            Tin y[VEC];
            memcpy(y, &data[v], 16);
#pragma unroll
            for (int e = 0; e < VEC; ++e) y[e] = static_cast<Tin>(static_cast<float>(y[e]) == INFINITY ? 0.f : -INFINITY);
            memcpy(&data[v], y, 16);
        }
        my_top = my_top == INFINITY ? 0.f : -INFINITY;
        top = 0.f;
    }
    // log2(e) / T as a number and what is left of it, within a range where nothing overflows
    Scale s;
    s.m = top;
    s.c = fminf(fmaxf(1.44269502f / T, 1e-36f), 1e37f);
    s.cl = s.c < 1e37f && s.c > 1e-36f ? (fmaf(-s.c, T, 1.44269502f) + 1.92596303e-8f) / T : 0.f;
    if (!(fabsf(s.cl) < 1e30f)) s.cl = 0.f;
    s.least = fmaxf(s.m - 44.f / s.c, -3.402823466e38f);
    // bins of equal width in log2 w; the last one takes everything below
    const float by = s.c * kPerOctave;
    // (the whole part of the product is in the significand's low bits, as in digits42)
    auto bin_of = [&](float x) {
        return (int)min(__float_as_uint(__fmaf_rz(s.m - x, by, 8388608.f)) - kBias, (uint32_t)(kBins - 1));
    };

    // Runs f(i, x) over the elements of the warp that lie in [from, to], few of them (one comparison each lets
    // all others pass by).
    auto each_in = [&](float from, float to, auto f) {
#pragma unroll 1
        for (int v = w0 + lane; v < w1; v += 32) {
            const uint4 y = data[v];
            if (Vec<Tin>::largest(y) < from) continue;
            float2 x[VEC / 2];
            Vec<Tin>::unpack(y, x);
            uint32_t bits = 0;
#pragma unroll
            for (int e = 0; e < VEC / 2; ++e) {
                bits |= x[e].x >= from && x[e].x <= to ? 1u << (2 * e) : 0u;
                bits |= x[e].y >= from && x[e].y <= to ? 2u << (2 * e) : 0u;
            }
            for (; bits != 0; bits &= bits - 1) {
                const int e = __ffs(bits) - 1;
                f(index_of(v) + e, Vec<Tin>::load(data + v, e));
            }
        }
    };
    // The warp's elements of [from, to] that which(i, x) takes go to the list, in any order; `count` counts
    // them all, the list holds the first kList.  One atomic for a warp's 32 vectors.
    auto append = [&](uint32_t bits, int v) {
        if (__any_sync(0xffffffffu, bits != 0) == 0) return;
        const int n_of = __popc(bits);
        int at = n_of;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += z;
        }
        int start = 0;
        if (lane == 31) start = atomicAdd(&count, at);
        at += __shfl_sync(0xffffffffu, start, 31) - n_of;
        for (; bits != 0; bits &= bits - 1, ++at) {
            const int e = __ffs(bits) - 1;
            if (at < kList) list[at] = ordered(key_of(Vec<Tin>::load(data + v, e)), index_of(v) + e);
        }
    };
    auto collect = [&](float from, float to, auto which) {
#pragma unroll 1
        for (int v0 = w0; v0 < w1; v0 += 32) {
            const int v = v0 + lane;
            uint32_t bits = 0;
            if (v < w1) {
                const uint4 y = data[v];
                if (Vec<Tin>::largest(y) >= from) {
                    float2 x[VEC / 2];
                    Vec<Tin>::unpack(y, x);
#pragma unroll
                    for (int e = 0; e < VEC / 2; ++e) {
                        bits |= x[e].x >= from && x[e].x <= to && which(index_of(v) + 2 * e, x[e].x) ? 1u << (2 * e) : 0u;
                        bits |= x[e].y >= from && x[e].y <= to && which(index_of(v) + 2 * e + 1, x[e].y) ? 2u << (2 * e) : 0u;
                    }
                }
            }
            append(bits, v);
        }
    };
    // The weights of the thread's elements that are at least `from` and of which which(i, x, hi, lo) holds (hi, lo:
    // the weight's digits), added up.  No branches, so that a vector's weights are formed side by side.
    auto weigh = [&](float from, auto which) {
        from = fmaxf(from, s.least);
        uint32_t hi = 0, lo = 0;                // (digits of 21 bits: no thread has 2,048 elements)
#pragma unroll 1
        for (int v = w0 + lane; v < w1; v += 32) {
            const uint4 y = data[v];
            if (Vec<Tin>::largest(y) < from) continue;
            float2 x[VEC / 2];
            Vec<Tin>::unpack(y, x);
            const int i = index_of(v);
#pragma unroll
            for (int e = 0; e < VEC / 2; ++e) {
                float2 high, low;
                digits42(weights2(s, x[e]), high, low);
                const uint32_t h0 = digit(high.x), h1 = digit(high.y), l0 = digit(low.x), l1 = digit(low.y);
                const bool on0 = (x[e].x >= from) & which(i + 2 * e, x[e].x, h0, l0);
                const bool on1 = (x[e].y >= from) & which(i + 2 * e + 1, x[e].y, h1, l1);
                hi += (on0 ? h0 : 0) + (on1 ? h1 : 0);
                lo += (on0 ? l0 : 0) + (on1 ? l1 : 0);
            }
        }
        return ((u64)hi << 21) + lo;
    };
    // All weights added up, those above `to` as well, and the elements of [from, to] to the list.
    auto weigh_and_collect = [&](float from, float to, u64 &all, u64 &above) {
        uint32_t hi = 0, lo = 0, hi_above = 0, lo_above = 0;
#pragma unroll 1
        for (int v0 = w0; v0 < w1; v0 += 32) {
            const int v = v0 + lane;
            uint32_t bits = 0;
            uint4 y;
            if (v < w1) y = data[v];
            if (v < w1 && Vec<Tin>::largest(y) >= fminf(from, s.least)) {
                float2 x[VEC / 2];
                Vec<Tin>::unpack(y, x);
#pragma unroll
                for (int e = 0; e < VEC / 2; ++e) {
                    float2 w = weights2(s, x[e]), high, low;
                    w.x = x[e].x >= s.least ? w.x : 0.f;
                    w.y = x[e].y >= s.least ? w.y : 0.f;
                    digits42(w, high, low);
                    const uint32_t h0 = digit(high.x), h1 = digit(high.y), l0 = digit(low.x), l1 = digit(low.y);
                    hi += h0 + h1;
                    lo += l0 + l1;
                    if (x[e].x > to) {
                        hi_above += h0;
                        lo_above += l0;
                    } else if (x[e].x >= from) {
                        bits |= 1u << (2 * e);
                    }
                    if (x[e].y > to) {
                        hi_above += h1;
                        lo_above += l1;
                    } else if (x[e].y >= from) {
                        bits |= 2u << (2 * e);
                    }
                }
            }
            append(bits, v);
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
                *cluster.map_shared_rank(&more_totals[rank], lane) = y;
            }
        }
        cluster.sync();
        x = y = 0;
        for (int r = 0; r < ranks; ++r) {
            x += totals[turn][r];
            y += more_totals[r];
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
        for (int r = 0; r < kMaxRanks; ++r)     // (reads of all ranks on their way together)
            x[r] = cluster.map_shared_rank(hist, r < ranks ? r : 0)[word * kBins + tid];
        u64 all = 0;
#pragma unroll
        for (int r = 0; r < kMaxRanks; ++r) all += r < ranks ? x[r] : 0;
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
    // a value that is below all of the bins up to b, give or take the roundings; and one above all from b on
    auto below_bin = [&](int b) {
        const float d = (float)(b + 1) / by;
        const float x = s.m - d * (1.f + 1e-6f);
        return b >= kBins - 1 || !(x > -3e38f) ? -3.402823466e38f : x - 4e-7f * (fabsf(s.m) + fabsf(x)) - 1e-37f;
    };
    auto above_bin = [&](int b) {
        const float x = s.m - (float)b / by * (1.f - 1e-6f);
        return fminf(s.m, x + 4e-7f * (fabsf(s.m) + fabsf(x)) + 1e-37f);
    };

    // Where top-p's border is, to a bin or two of log2 w: a value above all candidates and one below.  A bin's
    // weights lie within 2^(1/12) of each other, so it adds them up relative to its own upper end, to 2^-16
    // in 32 bits (a CTA has fewer than 2^16 elements).  The estimates are off by less than 2^-14 of the sum and 2^18
    // units of 2^-42, which `slack` covers on either side.
    auto candidates = [&](float &from, float &to) {
        next_histogram();
#pragma unroll 1
        for (int v = w0 + lane; v < w1; v += 32) {
            const uint4 y = data[v];
            if (Vec<Tin>::largest(y) < s.least) continue;
            float2 x[VEC / 2];
            Vec<Tin>::unpack(y, x);
#pragma unroll
            for (int e = 0; e < VEC / 2; ++e) {
                auto both = [](float z) { return make_float2(z, z); };
                const float2 d = tc::f2sub(both(s.m), x[e]), b = fma_cut2(d, both(by), both(8388608.f));
                const uint32_t b0 = min(__float_as_uint(b.x), kBias + kBins - 1), b1 = min(__float_as_uint(b.y), kBias + kBins - 1);
                // (the bins' upper ends, negated)
                const float2 ends = tc::f2sub(both(8388608.f), make_float2(__uint_as_float(b0), __uint_as_float(b1)));
                float2 w = tc::f2fma(tc::f2fma(d, both(by), ends), both(-1.f / kPerOctave), both(16.f));
                w.x = tc::ex2(w.x);
                w.y = tc::ex2(w.y);
                w = fma_cut2(w, both(1.f), both(8388608.f));
                if (digit(w.x) != 0) atomicAdd(&hist[b0 - kBias], digit(w.x));
                if (digit(w.y) != 0) atomicAdd(&hist[b1 - kBias], digit(w.y));
            }
        }
        cluster.sync();
        const u64 mine_w = __float2ull_rz((float)bin_sum(0) * exp2f(26.f - (float)tid / kPerOctave));
        u64 slack = 0, run = 0, goal = 0;
        border(mine_w, 0, [&](u64 total) {
            slack = (total >> 12) + (1 << 20);
            goal = share(total);
            return goal > slack ? goal - slack : (u64)1;
        }, &run);
        const int first_bin = found_bin;
        __syncthreads();
        if (tid == 0) found_bin = kBins - 1;
        __syncthreads();
        if (run >= goal + slack && run - mine_w < goal + slack) found_bin = tid;
        __syncthreads();
        to = above_bin(first_bin);
        from = below_bin(found_bin);
    };

    // Narrows the border down to the first elements of the order that reach a count (k) or a share of
    // the weight: first by bins of log2 w, then by the values' bits.  ahead_w: of top-p's weights, what the
    // thread has above the candidates.
    u64 ahead_w = 0;
    int pooled = 0;
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
            candidates(from, to);
            u64 total;
            weigh_and_collect(from, to, total, ahead_w);
            above = ahead_w;
            cluster_totals(total, above);
            goal(total);
            most = key_of(to);
            lowest = key_of(from);
        } else {
            next_histogram();
            each_in(lowest_value(), s.m, [&](int i, float x) {
                if (!stays(i, x)) return;
                if (by_weight) {
                    const u64 w = weight(s, x);
                    if (w != 0) add_weight(bin_of(x), (uint32_t)(w >> 21), (uint32_t)w & 0x1fffffu);
                } else {
                    atomicAdd(&hist[bin_of(x)], 1u);
                }
            });
            cluster.sync();
            if (!border(by_weight ? bin_sum(0) + (bin_sum(1) << 32) : bin_sum(0), 0, goal)) return;  // fewer: all stay
            bin = found_bin;
            above = found[0];
            most = key_of(above_bin(bin));
            lowest = key_of(below_bin(bin));
            collect(value_of(lowest), value_of(most), in_bin);
        }
        __syncthreads();
        pooled = count;
        for (;;) {
            const int shift = max(Vec<Tin>::GRAIN, 23 - __clz(most - lowest));      // 2^9 bins at most
            next_histogram();
            auto add = [&](uint32_t key) {
                const int b = (int)((most - key) >> shift);
                if (by_weight) {
                    const u64 w = weight(s, value_of(key));
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
            if (!border(by_weight ? bin_sum(0) + (bin_sum(1) << 32) : bin_sum(0), above, [&](u64) { return want; })) return;
            above = found[0];
            most -= (uint32_t)found_bin << shift;
            if (shift == Vec<Tin>::GRAIN) break;
            lowest = max(lowest, most - ((1u << shift) - 1));
        }
        if (Vec<Tin>::GRAIN > 0) {
            // the one key in (most - 2^GRAIN, most]: negative values' keys end in ones
            const uint32_t ones = (1u << Vec<Tin>::GRAIN) - 1;
            most = (most >> 31) != 0 ? most & ~ones : ((most + 1) & ~ones) - 1;
        }
        // the values equal to the border's: the first of them by their index
        const float it = value_of(most);
        const u64 one = by_weight ? weight(s, it) : 1, keep = (want - above + one - 1) / one;
        int32_t until = kAll;
        if (found[1] > one) {                   // (where only one is there, it stays)
            u64 equal = 0;
            const bool in_pool = pooled <= kList;
            if (in_pool) {
                for (int i = tid; i < pooled; i += kThreads) equal += ordered_key(list[i]) == most ? 1 : 0;
            } else {
                each_in(it, it, [&](int i, float x) { equal += stays(i, x) ? 1 : 0; });
            }
            if (tid == 0) chosen_count = 0;
            const u64 all = cluster_sum(equal, before, here);
            if (keep < all) {
                auto publish = [&](int at) {
                    for (int r = 0; r < ranks; ++r) *cluster.map_shared_rank(&chosen_index, r) = at;
                };
                if (in_pool) {
                    // the CTA's equal ones in any order (in the histograms' place, which all have read): the one
                    // with as many smaller indices as are wanted
                    int32_t *const equals = reinterpret_cast<int32_t *>(hists);
                    const u64 ahead = before - part[warp];      // of the CTAs before
                    for (int i = tid; i < pooled; i += kThreads)
                        if (ordered_key(list[i]) == most) equals[atomicAdd(&chosen_count, 1)] = ordered_index(list[i]);
                    __syncthreads();
                    const int of_them = chosen_count;
                    for (int i = tid; i < of_them; i += kThreads) {
                        const int at = equals[i];
                        u64 smaller = ahead;
                        for (int j = 0; j < of_them; ++j) smaller += equals[j] < at ? 1 : 0;
                        if (smaller + 1 == keep) publish(at);
                    }
                } else if (keep > before && keep <= before + here) {
                    // this warp has the last one
                    u64 seen = before;
                    for (int v0 = w0; v0 < w1; v0 += 32) {
                        const int v = v0 + lane;
                        uint32_t bits = 0;
                        if (v < w1)
#pragma unroll
                            for (int e = 0; e < VEC; ++e) {
                                const float x = Vec<Tin>::load(data + v, e);
                                if (x == it && stays(index_of(v) + e, x)) bits |= 1u << e;
                            }
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
    const u64 w_least = least > 0.f ? (u64)(fminf(least, 1.f) * 0x1p42f) : 0;
    // the first token whose running sum exceeds floor(u sum / 2^24) (the sum of all does, since u < 2^24)
    auto drawn = [&]() {
        const uint32_t tick = __float2uint_rz(fminf(fmaxf(u, 0.f) * 16777216.f, 16777215.f));
        return __umul64hi((u64)tick << 40, sum);
    };

    // ---- a small k: the few logits that can be among the first k, sorted in one CTA
    bool done = false;
    if (!none && k > 0 && k < V && k <= kListK && k <= ranks * kThreads / 2) {
        // k of the threads' largest logits lie in the bins up to this one
        next_histogram();
        if (my_top != -INFINITY) atomicAdd(&hist[bin_of(my_top)], 1u);
        cluster.sync();
        const float from = border(bin_sum(0), 0, [&](u64) { return (u64)k; }) ? below_bin(found_bin) : -3.402823466e38f;
        collect(from, s.m, [](int, float) { return true; });
        cluster.sync();
        // the lists' lengths, a rank to a lane; warp r brings rank r's to the first CTA
        const int length = lane < ranks ? *cluster.map_shared_rank(&count, lane) : 0;
        int upto = length;
#pragma unroll
        for (int o = 1; o < kMaxRanks; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += z;
        }
        const int all = __shfl_sync(0xffffffffu, upto, kMaxRanks - 1);
        done = all <= kList;
        if (done && rank == 0) {
            if (warp > 0 && warp < ranks) {
                const int c = __shfl_sync(0xffffffffu, length, warp), at = __shfl_sync(0xffffffffu, upto, warp) - c;
                const u64 *from_it = cluster.map_shared_rank(list, warp);
                for (int i = lane; i < c; i += 32) list[at + i] = from_it[i];
            }
            if (tid == 0) chosen_count = 0;
            __syncthreads();
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
                for (int i = tid; i < all; i += kThreads) weights[i] = weight(s, value_of(ordered_key(list[i])));
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
                const bool stay = of_k && ahead < goal && (place == 0 || mine_w >= w_least);
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
                // sums of f(c) up to each of the thread's elements
                auto scan = [&](auto f) {
                    u64 run = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        w[e] = f(c[e], 4 * tid + e);
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
                    u64 all_of_it;
                    const u64 add = parts_before(all_of_it) + run - own;
#pragma unroll
                    for (int e = 0; e < 4; ++e) cum[e] += add;
                    return all_of_it;
                };
                auto weight_of = [&](u64 x) { return weight(s, value_of(ordered_key(x))); };
#pragma unroll
                for (int e = 0; e < 4; ++e) c[e] = 4 * tid + e < all ? list[4 * tid + e] : 0;
                __syncthreads();
                int size = 2;
                while (size < all) size *= 2;
                sort_down(c, list, size);
                const int first_k = min(k, all);
                const u64 of_k = scan([&](u64 x, int i) { return i < first_k ? weight_of(x) : 0; });
                const u64 goal = p < 1.f ? share(of_k) : ~(u64)0;
                int stay = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    stay += 4 * tid + e < first_k && cum[e] - w[e] < goal && (4 * tid + e == 0 || w[e] >= w_least) ? 1 : 0;
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
        const uint32_t least_hi = (uint32_t)(w_least >> 21), least_lo = (uint32_t)w_least & 0x1fffffu;
        auto counts = [&](int i, float x, uint32_t hi, uint32_t lo) {
            return stays(i, x) & ((hi > least_hi) | ((hi == least_hi) & (lo >= least_lo)));
        };
        u64 mine_w;
        if (border_at > -INFINITY && pooled <= kList && w_least == 0 && !(k > 0 && k < V)) {
            // what lies above the candidates was summed up with them; of these, what stays, to the warps that have it
            if (tid < kWarps) more[tid] = 0;
            __syncthreads();
            for (int i = tid; i < pooled; i += kThreads) {
                const int at = ordered_index(list[i]);
                const float x = value_of(ordered_key(list[i]));
                if (stays(at, x)) atomicAdd(&more[((at + lead) / VEC - first) / per_warp], weight(s, x));
            }
            __syncthreads();
            mine_w = ahead_w + (lane == 0 ? more[warp] : 0);
        } else {
            // (with min-p's weight in mind, as a value with room for roundings)
            const float from = w_least > 0 ? s.m + (log2f(fminf(least, 1.f)) * (1.f + 1e-5f) - 1e-6f) / s.c : -INFINITY;
            mine_w = weigh(fmaxf(lowest_value(), from - 4e-7f * (fabsf(s.m) + fabsf(from)) - 1e-37f), counts);
        }
        sum = cluster_sum(mine_w, before, here);
        const u64 need = drawn();
        if (a.token != nullptr && before <= need && before + here > need) {
            for (int v0 = w0; v0 < w1; v0 += 32) {
                const int v = v0 + lane;
                u64 all = 0;
#pragma unroll 1
                for (int e = 0; e < VEC; ++e) {
                    const float x = v < w1 ? Vec<Tin>::load(data + v, e) : -INFINITY;
                    const u64 w = x > -INFINITY && stays(index_of(v) + e, x) ? weight(s, x) : 0;
                    all += w >= w_least ? w : 0;
                }
                u64 run = all;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const u64 z = __shfl_up_sync(0xffffffffu, run, o);
                    if (lane >= o) run += z;
                }
                const unsigned hit = __ballot_sync(0xffffffffu, before + run > need);
                if (hit != 0) {
                    if (lane == __ffs(hit) - 1) {
                        u64 at = before + run - all;
                        int e = 0;
                        for (; e < VEC - 1; ++e) {
                            const float x = Vec<Tin>::load(data + v, e);
                            const u64 w = x > -INFINITY && stays(index_of(v) + e, x) ? weight(s, x) : 0;
                            at += w >= w_least ? w : 0;
                            if (at > need) break;
                        }
                        a.token[n] = index_of(v) + e;
                    }
                    break;
                }
                before += __shfl_sync(0xffffffffu, run, 31);
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
        const float from = none ? INFINITY : fmaxf(lowest_value(), deep.least);
        unsigned char *out = static_cast<unsigned char *>(a.probs) + n * (int64_t)V * (bf16 ? 2 : 4);
        // whole vectors where the output's rows lie as the input's
        const bool whole = ((reinterpret_cast<uintptr_t>(out) - (size_t)lead * (bf16 ? 2 : 4)) & (bf16 ? VEC * 2 - 1 : 15)) == 0;
#pragma unroll 1
        for (int v = w0 + lane; v < w1; v += 32) {
            const uint4 raw = data[v];
            const int e0 = index_of(v);
            float y[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) y[e] = 0.f;
            if (Vec<Tin>::largest(raw) >= from) {
                float2 x[VEC / 2];
                Vec<Tin>::unpack(raw, x);
#pragma unroll
                for (int e = 0; e < VEC / 2; ++e) {
                    const float2 w = weights2(deep, x[e]);
                    if (x[e].x >= from && stays(e0 + 2 * e, x[e].x) && (w_least == 0 || fixed42(w.x) >= w_least))
                        y[2 * e] = w.x * inv;
                    if (x[e].y >= from && stays(e0 + 2 * e + 1, x[e].y) && (w_least == 0 || fixed42(w.y) >= w_least))
                        y[2 * e + 1] = w.y * inv;
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
                if (whole && e0 >= 0 && e0 + VEC <= V) {
#pragma unroll
                    for (int e = 0; e < VEC; e += 4)
                        *reinterpret_cast<float4 *>(to + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        if (e0 + e >= 0 && e0 + e < V) to[e] = y[e];
                }
            }
        }
    }
    cluster.sync();                             // no CTA leaves while its shared memory is read
}

template <typename Tin> cudaError_t run(const Sampling &a, int32_t N, cudaStream_t stream) {
    int dev = 0, sms = 152;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        sms = 152;
    constexpr int VEC = Vec<Tin>::N;
    const int vecs = (a.V + VEC - 1) / VEC + 1;
    int ranks = kMaxRanks;
    while (ranks > 1 && ((int64_t)ranks * N > 2 * (int64_t)sms || vecs < ranks * 256) &&
           (int64_t)vecs * 16 <= (ranks / 2) * (int64_t)(72 * 1024))
        ranks /= 2;
    const int slice = (vecs + ranks - 1) / ranks;
    const size_t smem = (size_t)slice * 16 + kScratch;
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = allow_dynamic_smem(sample_kernel<Tin>, kMaxSmem, smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = ranks;
    cluster.val.clusterDim.y = 1;
    cluster.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)N * ranks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &cluster;
    cfg.numAttrs = 1;
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
