// kda_sample.cu -- from logits to the distribution that is drawn from, and a token
// (kda_sample): temperature, top-k, top-p, min-p and the draw from a given uniform number.
//
//     w_i = e^{(x_i - max x) / T},   order: by value, then by index
//     top-k: the first k of the order;  top-p: of these the shortest beginning with a p-th of their
//     weight;  min-p: of these the ones with w_i >= m;  the token: the first index at which the
//     weights of the ones that stay, added up in index order, exceed u times their sum
//
// Weights are whole multiples of 2^-42, held in 64 bits, so sums do not depend on their order.
// Each is right to some 2^-25 of itself: the draw moves by a token at one in about 10^6 rows.
//
// A cluster of up to eight CTAs takes a row and keeps it in shared memory, so that the logits
// are read once.  What stays is a beginning of the order: a border value, and the
// last index among the logits equal to it.  It is found by histograms that narrow the values
// down, first by w (bins of equal width in log2 w, which spread the logits well whatever their
// scale), then by the value's bits, each of counts (top-k) or of weights (top-p).
// For the usual small k the histogram is of every thread's largest logit alone: k of these
// bound the k-th largest logit from below, and the few logits above the bound are sorted in
// one CTA, which makes the whole choice there.
#include "kda_internal.cuh"

#include <cooperative_groups.h>

namespace kda {
namespace {

typedef unsigned long long u64;
constexpr int kThreads = 512, kWarps = kThreads / 32, kMaxRanks = 8;
constexpr int kBins = 512;                      // of a histogram; two of 64-bit sums have a list's place
constexpr int kList = 2048, kListK = 1024;      // logits that are sorted at most, and the k for which that is tried
constexpr int kOneBits = 42;                    // w = 1
constexpr float kCut = -43.f;                   // log2 w below which w counts as zero
constexpr int32_t kAll = 0x7fffffff;
// a row of 2^18 logits over eight CTAs, and the histograms
constexpr int kScratch = kList * 8;
static_assert(kList * 8 >= 2 * kBins * 8 && kList <= 4 * kThreads, "histograms in the list's place, four elements a thread");
constexpr int kMaxSmem = KDA_MAX_VOCABULARY / kMaxRanks * 4 + 32 + kScratch;

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

// 16 bytes of logits; NaN becomes -infinity
template <typename Tin> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(uint4 u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint32_t clean(uint32_t w) {
        return __float_as_uint(fmaxf(__uint_as_float(w), -INFINITY));
    }
    static __device__ __forceinline__ uint32_t word(float lo, float) { return __float_as_uint(lo); }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(uint4 u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint32_t clean(uint32_t w) {
        const __nv_bfloat162 low = __halves2bfloat162(__ushort_as_bfloat16(0xff80), __ushort_as_bfloat16(0xff80));
        __nv_bfloat162 x;
        memcpy(&x, &w, 4);
        x = __hmax2(x, low);
        memcpy(&w, &x, 4);
        return w;
    }
};

// log2 w = (x - m)(c + cl)
struct Scale {
    float m, c, cl;
};

// w = 2^n (1 + q), or false where log2 w <= cut.  x - m with its rounding error, the product with c
// in one rounding behind the point, and 2^f - 1 by its series (to 2^-27 for |f| <= 1/2).
__device__ __forceinline__ bool weight_parts(const Scale &s, float x, float cut, float &q, int &n) {
    const float d = x - s.m;
    if (!(d * s.c > cut)) return false;
    const float mv = x - d, xv = d + mv, err = (x - xv) + (mv - s.m);
    const float t = fmaf(d, s.c, 12582912.f), whole = t - 12582912.f;
    float f = fmaf(d, s.c, -whole);
    f = fmaf(d, s.cl, f);
    f = fmaf(err, s.c, f);
    n = __float_as_int(t) - 0x4b400000;
    float p = 1.5252733804059841e-5f;           // ln(2)^k / k!, k = 7 .. 1
    p = fmaf(p, f, 1.5403530393381610e-4f);
    p = fmaf(p, f, 1.3333558146428443e-3f);
    p = fmaf(p, f, 9.6181291076284772e-3f);
    p = fmaf(p, f, 5.5504108664821580e-2f);
    p = fmaf(p, f, 2.4022650695910071e-1f);
    p = fmaf(p, f, 6.9314718055994531e-1f);
    q = p * f;
    return true;
}
__device__ __forceinline__ u64 weight(const Scale &s, float x) {
    float q;
    int n;
    if (!weight_parts(s, x, kCut, q, n)) return 0;
    const uint32_t mant = (1u << 30) + __float2int_rn(q * 0x1p30f);
    return ((u64)mant << 32) >> (62 - kOneBits - n);
}

// list[0 .. n) by size, the largest first; the block's threads.  (Bitonic; what lies behind n up to the
// next power of two is set to zero.)
__device__ __forceinline__ void sort_down(u64 *list, int n, int tid) {
    int all = 2;
    while (all < n) all *= 2;
    for (int i = n + tid; i < all; i += kThreads) list[i] = 0;
    __syncthreads();
    for (int size = 2; size <= all; size *= 2)
        for (int step = size / 2; step > 0; step /= 2) {
            for (int i = tid; i < all / 2; i += kThreads) {
                const int lo = 2 * i - (i & (step - 1)), hi = lo + step;
                const u64 x = list[lo], y = list[hi];
                if ((x < y) == ((lo & size) == 0)) {
                    list[lo] = y;
                    list[hi] = x;
                }
            }
            __syncthreads();
        }
}

template <typename Tin>
__global__ void __launch_bounds__(kThreads, 2)
sample_kernel(const Sampling a, const int32_t slice) {
    constexpr int VEC = Vec<Tin>::N;
    extern __shared__ __align__(16) unsigned char smem[];
    uint4 *data = reinterpret_cast<uint4 *>(smem);                  // the CTA's vectors of the row
    // two histograms: low words, then high words;  in their place: the few that matter, and their sums
    uint32_t *const hists = reinterpret_cast<uint32_t *>(smem + (size_t)slice * 16), *hist = hists;
    u64 *const list = reinterpret_cast<u64 *>(hists);
    __shared__ u64 part[kWarps], found[2];                          // found: what lies above the border, the border bin's
    __shared__ u64 totals[2][kMaxRanks];
    __shared__ float tops[kMaxRanks], warp_top[kWarps];
    __shared__ int32_t found_bin, chosen_index, count, chosen_count;
    __shared__ uint32_t chosen_key;
    __shared__ Scale scale;
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
    const uint4 *grid = reinterpret_cast<const uint4 *>(row - lead);
    auto index_of = [&](int v) { return (first + v) * VEC - lead; };    // of a vector's first element

    float T = a.temperature != nullptr ? a.temperature[n] : 1.f;
    int32_t k = a.top_k != nullptr ? a.top_k[n] : 0;
    const float p = a.top_p != nullptr ? a.top_p[n] : 1.f;
    const float least = a.min_p != nullptr ? a.min_p[n] : 0.f;
    const float u = a.uniforms != nullptr ? a.uniforms[n] : 0.f;
    const bool greedy = !(T > 0.f);             // the first of the order
    if (greedy) {
        T = 1.f;
        k = 1;
    }

    // ---- the row into shared memory, and its maximum
    float top = -INFINITY, my_top;
    for (int v = w0 + lane; v < w1; v += 32) {
        const int e0 = index_of(v);
        uint4 x;
        if (e0 >= 0 && e0 + VEC <= V) {
            x = __ldg(grid + first + v);
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
        float f[VEC];
        Vec<Tin>::unpack(x, f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) top = fmaxf(top, f[e]);
    }
    my_top = top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) warp_top[warp] = top;
    if (tid == 0) count = 0;
    cluster.barrier_wait();                     // every CTA has started
    __syncthreads();
    if (warp == 0) {
        top = lane < kWarps ? warp_top[lane] : -INFINITY;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane < ranks) *cluster.map_shared_rank(&tops[rank], lane) = top;
        if (lane == 0) {
            const double c = 1.4426950408889634 / (double)T;
            scale.c = fminf((float)c, 1e37f);
            scale.cl = scale.c < 1e37f ? (float)(c - (double)scale.c) : 0.f;
        }
    }
    cluster.sync();
    top = -INFINITY;
    for (int r = 0; r < ranks; ++r) top = fmaxf(top, tops[r]);

    // Runs f(index, x) over the warp's elements, VEC to a lane; what lies outside the row is -infinity.
    auto each = [&](auto f) {
        for (int v = w0 + lane; v < w1; v += 32) {
            float x[VEC];
            Vec<Tin>::unpack(data[v], x);
            const int e0 = index_of(v);
#pragma unroll
            for (int e = 0; e < VEC; ++e) f(e0 + e, x[e]);
        }
    };
    bool inf_row = false;
    if (top == INFINITY) {                      // the infinite ones share everything
        inf_row = true;
        top = 0.f;
    }
    Scale s = scale;
    s.m = top;
    auto value = [&](float x) { return !inf_row ? x : x == INFINITY ? 0.f : -INFINITY; };

    // sums over the warps of all CTAs: every thread gets the total, and what the warps before its own hold
    int turn = 0;
    auto cluster_sum = [&](u64 x, u64 &before) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        __syncthreads();
        if (lane == 0) part[warp] = x;
        __syncthreads();
        u64 all = 0;
        before = 0;
        for (int w = 0; w < kWarps; ++w) {
            before += w < warp ? part[w] : 0;
            all += part[w];
        }
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

    // A histogram's bins, added up over the cluster and in order (every CTA for itself): the first bin at
    // which they reach `goal(total)`, at least one; `above` lies above the first bin.  Two histograms in
    // turn: when all have come together here, the last one has been read.
    auto next_histogram = [&]() {
        hist = hist == hists ? hists + 2 * kBins : hists;
        for (int i = tid; i < 2 * kBins; i += kThreads) hist[i] = 0;
        __syncthreads();
    };
    auto border = [&](u64 above, bool wide, auto goal, u64 &total) {
        cluster.sync();                         // the histograms are complete
        u64 x = 0;
        if (tid < kBins)
            for (int r = 0; r < ranks; ++r) {
                const uint32_t *h = cluster.map_shared_rank(hist, r);
                x += wide ? (u64)h[tid] + ((u64)h[kBins + tid] << 32) : (u64)h[tid];
            }
        u64 run = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 z = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += z;
        }
        if (lane == 31) part[warp] = run;
        __syncthreads();
        total = 0;
        for (int w = 0; w < kWarps; ++w) {
            run += w < warp ? part[w] : 0;
            total += part[w];
        }
        const u64 want = goal(total);
        run += above;
        if (tid < kBins && run >= want && run - x < want) {
            found_bin = tid;
            found[0] = run - x;
            found[1] = x;
        }
        __syncthreads();
        return want;
    };
    static_assert(kBins <= kThreads, "a thread per bin");
    auto add_weight = [&](int b, u64 w) {
        const uint32_t lo = (uint32_t)w, old = atomicAdd(&hist[b], lo);
        const uint32_t hi = (uint32_t)(w >> 32) + (old + lo < old ? 1u : 0u);
        if (hi != 0) atomicAdd(&hist[kBins + b], hi);
    };
    // bins of log2 w; the last one takes everything below
    const float by = s.c * ((kBins - 1) / -kCut);
    auto position = [&](float x) { return (s.m - x) * by; };
    auto bin_of = [&](float pos) { return pos < (float)(kBins - 1) ? (int)pos : kBins - 1; };

    // What stays: values above the border's, and of the equal ones those up to `last`.
    uint32_t border_key = 0;                    // (key 0 is no value's)
    int32_t last = kAll;
    auto stays = [&](int i, uint32_t key) { return key > border_key || (key == border_key && i <= last); };

    // Narrows the border down to the first elements of the order that reach a count (k) or a weight.
    auto narrow = [&](bool by_weight, auto goal) {
        u64 total, want = 0;
        next_histogram();
        each([&](int i, float x) {
            x = value(x);
            if (x == -INFINITY || !stays(i, key_of(x))) return;
            const int b = bin_of(position(x));
            if (by_weight) {
                const u64 w = weight(s, x);
                if (w != 0) add_weight(b, w);
            } else {
                atomicAdd(&hist[b], 1u);
            }
        });
        want = border(0, by_weight, goal, total);
        if (total < want || total == 0) return;  // fewer than that: all stay
        const int bin = found_bin;
        // the values of the bin lie between these, give or take the roundings; then by their bits
        const float slack = 4e-7f * fabsf(s.m) + 1e-37f;
        const float width = 1.f / by, below = (float)bin * width, above = (float)(bin + 1) * width;
        uint32_t most = key_of(fminf(s.m, s.m - below * (1.f - 1e-6f) + slack + fabsf(s.m - below) * 4e-7f));
        uint32_t lowest = bin == kBins - 1 || !(above < 3e38f)
                              ? 0x00800000u     // (keys of finite numbers start there)
                              : key_of(s.m - above * (1.f + 1e-6f) - slack - fabsf(s.m - above) * 4e-7f);
        if (lowest > most) lowest = 0;
        for (;;) {
            int shift = 0;
            while (((most - lowest) >> shift) >= (uint32_t)kBins) ++shift;
            next_histogram();
            each([&](int i, float x) {
                x = value(x);
                if (x == -INFINITY) return;
                const uint32_t key = key_of(x);
                if (key < lowest || key > most || !stays(i, key) || bin_of(position(x)) != bin) return;
                const int b = (int)((most - key) >> shift);
                if (by_weight) {
                    const u64 w = weight(s, x);
                    if (w != 0) add_weight(b, w);
                } else {
                    atomicAdd(&hist[b], 1u);
                }
            });
            const u64 above_it = found[0];
            border(above_it, by_weight, [&](u64) { return want; }, total);
            most = most - ((uint32_t)found_bin << shift);
            if (shift == 0) break;
            lowest = max(lowest, most - ((1u << shift) - 1));
        }
        // the values equal to the border's: the first of them by their index
        const uint32_t key = most;
        const u64 one = by_weight ? weight(s, value_of(key)) : 1;
        const u64 rest = want - found[0], keep = (rest + one - 1) / one;
        int32_t until = kAll;
        if (found[1] > rest || found[1] > one) {
            // (where only one is there, it stays)
            u64 equal = 0, before;
            each([&](int i, float x) { equal += value(x) != -INFINITY && key_of(value(x)) == key && stays(i, key) ? 1 : 0; });
            const u64 there = equal;
            const u64 all = cluster_sum(equal, before);
            u64 here = there;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) here += __shfl_xor_sync(0xffffffffu, here, o);
            if (keep < all) {
                if (keep > before && keep <= before + here) {
                    // this warp has the last one
                    u64 seen = before;
                    for (int v0 = w0; v0 < w1; v0 += 32) {
                        const int v = v0 + lane;
                        uint32_t bits = 0;
                        if (v < w1) {
                            float x[VEC];
                            Vec<Tin>::unpack(data[v], x);
#pragma unroll
                            for (int e = 0; e < VEC; ++e)
                                if (value(x[e]) != -INFINITY && key_of(value(x[e])) == key && stays(index_of(v) + e, key))
                                    bits |= 1u << e;
                        }
                        int run = __popc(bits);
                        const int cnt = run;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const int z = __shfl_up_sync(0xffffffffu, run, o);
                            if (lane >= o) run += z;
                        }
                        if (keep > seen + run - cnt && keep <= seen + run) {
                            uint32_t left = bits;
                            for (int c = (int)(keep - (seen + run - cnt)); c > 1; --c) left &= left - 1;
                            const int at = index_of(v) + __ffs(left) - 1;
                            for (int r = 0; r < ranks; ++r) *cluster.map_shared_rank(&chosen_index, r) = at;
                        }
                        seen += __shfl_sync(0xffffffffu, run, 31);
                    }
                }
                cluster.sync();
                until = chosen_index;
            }
        }
        last = key == border_key ? min(last, until) : until;
        border_key = key;
    };

    u64 sum = 0;                                // of what stays
    u64 w_least = 0;
    if (least > 0.f) w_least = (u64)(fminf(least, 1.f) * 0x1p42f);
    const bool none = top == -INFINITY;
    // the weight that top-p asks of a total (rounded up, at least something)
    auto share = [&](u64 total) {
        const u64 by64 = p > 0.f ? (u64)(p * 0x1p63f) << 1 : 0, whole = __umul64hi(total, by64);
        return max(total * by64 != 0 ? whole + 1 : whole, (u64)1);
    };
    // the first token whose running sum exceeds floor(u sum / 2^24) (the sum of all does, since u < 2^24)
    auto drawn = [&]() {
        const uint32_t tick = __float2uint_rz(fminf(fmaxf(u, 0.f) * 16777216.f, 16777215.f));
        return __umul64hi((u64)tick << 40, sum);
    };

    // ---- a small k: the few logits that can be among the first k, sorted in one CTA
    bool done = false;
    if (!none && k > 0 && k < V && k <= kListK && k <= ranks * kThreads / 2) {
        // k of the threads' largest logits are no smaller than this bin's
        next_histogram();
        const float mine_top = value(my_top);
        if (mine_top != -INFINITY) atomicAdd(&hist[bin_of(position(mine_top))], 1u);
        u64 total;
        const u64 want = border(0, false, [&](u64) { return (u64)k; }, total);
        const float until = total < want || found_bin == kBins - 1 ? INFINITY : (float)(found_bin + 1);
        cluster.sync();                         // the histograms are read: the lists take their place
        each([&](int i, float x) {
            x = value(x);
            if (x == -INFINITY || !(position(x) < until)) return;
            const int at = atomicAdd(&count, 1);
            if (at < kList) list[at] = (u64)key_of(x) << 32 | (uint32_t)~i;
        });
        cluster.sync();
        int all = 0, before = 0;
        for (int r = 0; r < ranks; ++r) {
            const int c = *cluster.map_shared_rank(&count, r);
            before += r < rank ? c : 0;
            all += c;
        }
        done = all <= kList;
        if (done && rank == 0) {
            for (int r = 1, at = count; r < ranks; ++r) {
                const int c = *cluster.map_shared_rank(&count, r);
                const u64 *from = cluster.map_shared_rank(list, r);
                for (int i = tid; i < c; i += kThreads) list[at + i] = from[i];
                at += c;
            }
            __syncthreads();
            sort_down(list, all, tid);
            // cum(n, w): the sums of w(i) up to each of the thread's elements 4 tid .. 4 tid + 3 of n
            u64 w[4], cum[4];
            auto scan = [&](int n, auto f) {
                u64 run = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 4 * tid + e;
                    w[e] = i < n ? f(list[i]) : 0;
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
                __syncthreads();
                u64 sum_all = 0, add = run - own;
                for (int x = 0; x < kWarps; ++x) {
                    add += x < warp ? part[x] : 0;
                    sum_all += part[x];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) cum[e] += add;
                return sum_all;
            };
            const int first_k = min(k, all);
            const u64 of_k = scan(first_k, [&](u64 c) { return weight(s, value_of((uint32_t)(c >> 32))); });
            const u64 goal = p < 1.f && !greedy ? share(of_k) : ~(u64)0;
            int stay = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                stay += 4 * tid + e < first_k && cum[e] - w[e] < goal && (4 * tid + e == 0 || w[e] >= w_least) ? 1 : 0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) stay += __shfl_xor_sync(0xffffffffu, stay, o);
            if (tid == 0) chosen_count = 0;
            __syncthreads();
            if (lane == 0) atomicAdd(&chosen_count, stay);
            __syncthreads();
            stay = chosen_count;                // a beginning of the order
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (4 * tid + e == stay - 1) {
                    const u64 c = list[stay - 1];
                    for (int r = 0; r < ranks; ++r) {
                        *cluster.map_shared_rank(&chosen_key, r) = (uint32_t)(c >> 32);
                        *cluster.map_shared_rank(&chosen_index, r) = (int32_t)~(uint32_t)c;
                        *cluster.map_shared_rank(&found[0], r) = cum[e];
                    }
                }
            __syncthreads();
            sum = found[0];
            if (a.token != nullptr) {
                // in index order
                for (int i = tid; i < stay; i += kThreads) list[i] = list[i] << 32 | list[i] >> 32;
                __syncthreads();
                sort_down(list, stay, tid);
                scan(stay, [&](u64 c) { return weight(s, value_of((uint32_t)c)); });
                const u64 need = drawn();
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * tid + e < stay && cum[e] > need && cum[e] - w[e] <= need)
                        a.token[n] = (int32_t)~(uint32_t)(list[4 * tid + e] >> 32);
            }
        }
        cluster.sync();
        if (done) {
            border_key = chosen_key;
            last = chosen_index;
            sum = found[0];
        }
    }
    if (!none && !done) {
        if (k > 0 && k < V) narrow(false, [&](u64) { return (u64)k; });
        if (p < 1.f && !greedy) narrow(true, share);
        // ---- the draw, in index order
        u64 before;
        each([&](int i, float x) {
            x = value(x);
            if (!stays(i, key_of(x))) return;
            const u64 w = weight(s, x);
            sum += w >= w_least ? w : 0;
        });
        u64 here = sum;
        sum = cluster_sum(sum, before);
        if (a.token != nullptr) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) here += __shfl_xor_sync(0xffffffffu, here, o);
            const u64 need = drawn();
            if (before <= need && before + here > need) {
                for (int v0 = w0; v0 < w1; v0 += 32) {
                    const int v = v0 + lane;
                    u64 w[VEC], all = 0;
                    float x[VEC];
                    if (v < w1) Vec<Tin>::unpack(data[v], x);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        w[e] = 0;
                        if (v < w1 && stays(index_of(v) + e, key_of(value(x[e])))) w[e] = weight(s, value(x[e]));
                        if (w[e] < w_least) w[e] = 0;
                        all += w[e];
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
#pragma unroll
                            for (int z = 0; z < VEC; ++z) {
                                at += w[z];
                                if (at <= need) e = z + 1;
                            }
                            a.token[n] = index_of(v) + e;
                        }
                        break;
                    }
                    before += __shfl_sync(0xffffffffu, run, 31);
                }
            }
        }
    } else if (none && a.token != nullptr && rank == 0 && tid == 0) {
        a.token[n] = -1;
    }
    if (a.probs != nullptr) {
        const float inv = none ? 0.f : (float)(0x1p42 / (double)sum);
        const bool bf16 = a.probs_bf16 != 0;
        unsigned char *out = static_cast<unsigned char *>(a.probs) + n * (int64_t)V * (bf16 ? 2 : 4);
        // whole vectors where the output's rows lie as the input's
        const bool whole = ((reinterpret_cast<uintptr_t>(out) - (size_t)lead * (bf16 ? 2 : 4)) & (bf16 ? VEC * 2 - 1 : 15)) == 0;
        for (int v = w0 + lane; v < w1; v += 32) {
            float x[VEC], y[VEC];
            Vec<Tin>::unpack(data[v], x);
            const int e0 = index_of(v);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float z = value(x[e]);
                float q;
                int ex;
                y[e] = 0.f;
                if (!none && z != -INFINITY && stays(e0 + e, key_of(z)) && weight_parts(s, z, -126.f, q, ex) &&
                    (w_least == 0 || weight(s, z) >= w_least))
                    y[e] = (1.f + q) * __int_as_float((ex + 127) << 23) * inv;
            }
            if (bf16) {
                __nv_bfloat16 *to = reinterpret_cast<__nv_bfloat16 *>(out) + e0;
                if (whole && e0 >= 0 && e0 + VEC <= V) {
                    uint32_t z[VEC / 2];
#pragma unroll
                    for (int e = 0; e < VEC / 2; ++e) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * e], y[2 * e + 1]);
                        memcpy(&z[e], &b, 4);
                    }
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
