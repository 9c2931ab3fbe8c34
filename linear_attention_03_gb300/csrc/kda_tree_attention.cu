// kda_tree_attention.cu -- softmax attention of a tree of drafted tokens over
// a paged cache and the tree itself ("From GPT-2 to Kimi K3, from first
// principles", Chapter 1 for softmax attention and its cache, Chapter 14 for
// the drafts; the hybrid's softmax layers sit between its KDA layers).
//
// Row (m, hq) attends to keys 0 .. len-1 of its sequence's cache and to the
// keys of the nodes on m's line.  One pass over the keys per row with a
// running maximum x and sum z:
//     x' = max(x, max_j s_j),  z' = z e^{x - x'} + sum_j e^{s_j - x'},
//     o' = o e^{x - x'} + sum_j e^{s_j - x'} v_j,   out = o / z, lse = x + ln z
//
// This file: the CUDA-core form, for fp32 and for the head and page sizes that
// the tensor-core form does not take.  All rows of a cache head (M nodes x G
// query heads) share its keys; sixteen of them go to a CTA, four to a warp.  A
// long cache is split over CTAs, whose partial sums a second kernel joins.
#include "kda_internal.cuh"
#include "kda_tree.cuh"

#include <math.h>

namespace kda {
namespace {

constexpr int kThreads = 128, kRowsPerWarp = 4, kRows = 16, kKeys = 32;

template <int D> constexpr size_t smem_bytes() {
    return sizeof(float) * (kKeys * (D + 4) + kKeys * D + kRows * D + kRows * kKeys);
}

// Partial results of split s of a row: [unit][s][kRows] x (D sums, maximum, sum).
struct Partials {
    float *o, *x, *z;
};

// A key's address in the cache, or null when the page table's entry is out of
// range (flagged; the key then counts as zeros).
template <typename Tin>
__device__ __forceinline__ const Tin *cached_row(const Tin *cache, const int32_t *table, int pos, int h,
                                                 const TreeAttention &a, int D) {
    const int page = table[pos / a.page_size];
    if (page < 0 || page >= a.num_pages) {
        flag_status(a.status, KDA_DEVICE_BAD_PAGE);
        return nullptr;
    }
    return cache + (((int64_t)page * a.H_kv + h) * a.page_size + pos % a.page_size) * D;
}

template <typename Tin, int D>
__global__ void __launch_bounds__(kThreads)
tree_attention_kernel(const TreeAttention a, int row_tiles, int splits, Partials part) {
    constexpr int LD = D + 4;                     // padded key rows: no bank conflicts down a column
    constexpr int CPL = D < 32 ? 1 : D / 32;      // output columns per lane
    extern __shared__ __align__(16) float smem[];
    float *sk = smem, *sv = sk + kKeys * LD, *sq = sv + kKeys * D, *sp = sq + kRows * D;
    __shared__ int32_t par[kMaxTreeNodes];
    __shared__ uint64_t line[kMaxTreeNodes];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Tin *q = static_cast<const Tin *>(a.q), *k_new = static_cast<const Tin *>(a.k_new),
              *v_new = static_cast<const Tin *>(a.v_new), *k_cache = static_cast<const Tin *>(a.k_cache),
              *v_cache = static_cast<const Tin *>(a.v_cache);
    const int unit = blockIdx.x, split = blockIdx.y;
    const int rt = unit % row_tiles, h = unit / row_tiles % a.H_kv;
    const int64_t n = unit / row_tiles / a.H_kv;
    const int G = a.H / a.H_kv, M = a.M, rows = M * G, row0 = rt * kRows;

    int len = a.cache_lens[n];
    const int64_t room = (int64_t)a.max_pages * a.page_size;
    if (len < 0 || len > room) {
        if (tid == 0) flag_status(a.status, KDA_DEVICE_BAD_LENGTH);
        len = len < 0 ? 0 : (int)room;
    }
    const int32_t *table = a.page_table + n * a.max_pages;
    for (int m = tid; m < M; m += kThreads) par[m] = a.parent[n * M + m];
#pragma unroll
    for (int y = 0; y < (kRows * D / 8 + kThreads - 1) / kThreads; ++y) {
        const int i = tid + y * kThreads, r = row0 + i / (D / 8), c = i % (D / 8) * 8;
        float x[8] = {0.f};
        if (i < kRows * (D / 8)) {
            if (r < rows) Elem<Tin>::load8(q + ((n * M + r / G) * a.H + h * G + r % G) * D + c, x);
            Elem<float>::store8(sq + i * 8, x);
        }
    }
    __syncthreads();
    for (int m = tid; m < M; m += kThreads) line[m] = tree_line(par, m);
    __syncthreads();

    const int cache_tiles = (len + kKeys - 1) / kKeys, tiles = cache_tiles + (M + kKeys - 1) / kKeys;
    const int t0 = (int)((int64_t)tiles * split / splits), t1 = (int)((int64_t)tiles * (split + 1) / splits);
    uint64_t mine[kRowsPerWarp];
    float top[kRowsPerWarp], sum[kRowsPerWarp], acc[kRowsPerWarp][CPL];
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
        const int row = row0 + warp * kRowsPerWarp + r;
        mine[r] = row < rows ? line[row / G] : 0;
        top[r] = -INFINITY;
        sum[r] = 0.f;
#pragma unroll
        for (int e = 0; e < CPL; ++e) acc[r][e] = 0.f;
    }
    // A tile's keys and values pass through registers, so that the next tile is on its
    // way while this one is worked on: PIECES runs of eight channels per thread.
    constexpr int PIECES = kKeys * (D / 8) / kThreads > 0 ? kKeys * (D / 8) / kThreads : 1;
    float nk[PIECES][8], nv[PIECES][8];
    auto base_of = [&](int t) { return t >= cache_tiles ? (t - cache_tiles) * kKeys : t * kKeys; };
    auto count_of = [&](int t) { return min(kKeys, (t >= cache_tiles ? M : len) - base_of(t)); };
    auto fetch = [&](int t) {
        const bool tree = t >= cache_tiles;
        const int base = base_of(t), count = count_of(t);
#pragma unroll
        for (int y = 0; y < PIECES; ++y) {
            const int i = tid + y * kThreads, j = i / (D / 8), c = i % (D / 8) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) nk[y][e] = nv[y][e] = 0.f;
            if (j < count && j < kKeys) {
                const Tin *pk, *pv;
                if (tree) {
                    const int64_t at = ((n * M + base + j) * a.H_kv + h) * D;
                    pk = k_new + at;
                    pv = v_new + at;
                } else {
                    pk = cached_row(k_cache, table, base + j, h, a, D);
                    pv = pk == nullptr ? nullptr : v_cache + (pk - k_cache);
                }
                if (pk != nullptr) {
                    Elem<Tin>::load8(pk + c, nk[y]);
                    Elem<Tin>::load8(pv + c, nv[y]);
                }
            }
        }
    };
    if (t0 < t1) fetch(t0);
    for (int t = t0; t < t1; ++t) {
        const bool tree = t >= cache_tiles;
        const int base = base_of(t), count = count_of(t);
        __syncthreads();
#pragma unroll
        for (int y = 0; y < PIECES; ++y) {
            const int i = tid + y * kThreads, j = i / (D / 8), c = i % (D / 8) * 8;
            if (j >= kKeys) continue;
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                *reinterpret_cast<float4 *>(sk + j * LD + c + e) =
                    make_float4(nk[y][e], nk[y][e + 1], nk[y][e + 2], nk[y][e + 3]);
                *reinterpret_cast<float4 *>(sv + j * D + c + e) =
                    make_float4(nv[y][e], nv[y][e + 1], nv[y][e + 2], nv[y][e + 3]);
            }
        }
        __syncthreads();
        if (t + 1 < t1) fetch(t + 1);
        // lane j holds key j's scores
        float s[kRowsPerWarp];
#pragma unroll
        for (int r = 0; r < kRowsPerWarp; ++r) s[r] = 0.f;
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
            const float4 kv = *reinterpret_cast<const float4 *>(sk + lane * LD + c);
#pragma unroll
            for (int r = 0; r < kRowsPerWarp; ++r) {
                const float4 qv = *reinterpret_cast<const float4 *>(sq + (warp * kRowsPerWarp + r) * D + c);
                s[r] += kv.x * qv.x + kv.y * qv.y + kv.z * qv.z + kv.w * qv.w;
            }
        }
        unsigned seen[kRowsPerWarp];               // which of the 32 keys the row sees
#pragma unroll
        for (int r = 0; r < kRowsPerWarp; ++r) {
            const bool sees = mine[r] != 0 && lane < count && (!tree || (mine[r] >> (base + lane) & 1) != 0);
            seen[r] = __ballot_sync(0xffffffffu, sees);
            s[r] = sees ? s[r] * a.scale : -INFINITY;
            float mx = s[r];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float was = top[r];
            top[r] = fmaxf(was, mx);
            // no key seen yet: every difference below is taken from zero instead
            const float from = top[r] == -INFINITY ? 0.f : top[r];
            const float shrink = __expf(was - from);
            s[r] = sees ? __expf(s[r] - from) : 0.f;
            float add = s[r];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) add += __shfl_xor_sync(0xffffffffu, add, o);
            sum[r] = sum[r] * shrink + add;
#pragma unroll
            for (int e = 0; e < CPL; ++e) acc[r][e] *= shrink;
        }
        if (!tree) {
            // (keys past the count have weight 0 and values 0)
            float *wp = sp + warp * kRowsPerWarp * kKeys;
#pragma unroll
            for (int r = 0; r < kRowsPerWarp; ++r) wp[r * kKeys + lane] = s[r];
            __syncwarp();
#pragma unroll 2
            for (int j = 0; j < kKeys; j += 4) {
                float y[4][CPL];
#pragma unroll
                for (int z = 0; z < 4; ++z)
#pragma unroll
                    for (int e = 0; e < CPL; ++e)
                        y[z][e] = CPL * lane + e < D ? sv[(j + z) * D + CPL * lane + e] : 0.f;
#pragma unroll
                for (int r = 0; r < kRowsPerWarp; ++r) {
                    const float4 w = *reinterpret_cast<const float4 *>(wp + r * kKeys + j);
#pragma unroll
                    for (int e = 0; e < CPL; ++e)
                        acc[r][e] += w.x * y[0][e] + w.y * y[1][e] + w.z * y[2][e] + w.w * y[3][e];
                }
            }
            __syncwarp();
        } else {
            for (int j = 0; j < count; ++j) {
                float y[CPL];
#pragma unroll
                for (int e = 0; e < CPL; ++e) y[e] = CPL * lane + e < D ? sv[j * D + CPL * lane + e] : 0.f;
#pragma unroll
                for (int r = 0; r < kRowsPerWarp; ++r) {
                    const float w = __shfl_sync(0xffffffffu, s[r], j);
                    // a key the row does not see adds nothing, whatever it holds
                    if (seen[r] >> j & 1) {
#pragma unroll
                        for (int e = 0; e < CPL; ++e) acc[r][e] += w * y[e];
                    }
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
        const int lr = warp * kRowsPerWarp + r, row = row0 + lr;
        if (row >= rows) continue;
        if (splits == 1) {
            const int64_t o_row = (n * M + row / G) * a.H + h * G + row % G;
            const float inv = mine[r] == 0 ? 0.f : 1.f / sum[r];
#pragma unroll
            for (int e = 0; e < CPL; ++e)
                if (CPL * lane + e < D)
                    Elem<Tin>::store(static_cast<Tin *>(a.out) + o_row * D + CPL * lane + e,
                                     mine[r] == 0 ? 0.f : acc[r][e] * inv);
            if (lane == 0 && a.lse != nullptr) a.lse[o_row] = mine[r] == 0 ? -INFINITY : top[r] + logf(sum[r]);
        } else {
            const int64_t p = ((int64_t)unit * splits + split) * kRows + lr;
#pragma unroll
            for (int e = 0; e < CPL; ++e)
                if (CPL * lane + e < D) part.o[p * D + CPL * lane + e] = acc[r][e];
            if (lane == 0) {
                part.x[p] = top[r];
                part.z[p] = sum[r];
            }
        }
    }
}

// A warp per row joins the splits' sums.
template <typename Tin, int D>
__global__ void __launch_bounds__(kThreads)
tree_attention_join_kernel(const TreeAttention a, int row_tiles, int splits, Partials part) {
    constexpr int CPL = D < 32 ? 1 : D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int unit = blockIdx.x / (kRows / 4), lr = blockIdx.x % (kRows / 4) * 4 + warp;
    const int rt = unit % row_tiles, h = unit / row_tiles % a.H_kv;
    const int64_t n = unit / row_tiles / a.H_kv;
    const int G = a.H / a.H_kv, row = rt * kRows + lr;
    if (row >= a.M * G) return;
    const int64_t p0 = (int64_t)unit * splits * kRows + lr;
    float top = -INFINITY;
    for (int s = lane; s < splits; s += 32) top = fmaxf(top, part.x[p0 + (int64_t)s * kRows]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float from = top == -INFINITY ? 0.f : top;
    float sum = 0.f, acc[CPL];
#pragma unroll
    for (int e = 0; e < CPL; ++e) acc[e] = 0.f;
    for (int s = 0; s < splits; ++s) {
        const int64_t p = p0 + (int64_t)s * kRows;
        const float w = __expf(part.x[p] - from);
        sum += w * part.z[p];
#pragma unroll
        for (int e = 0; e < CPL; ++e)
            if (CPL * lane + e < D) acc[e] += w * part.o[p * D + CPL * lane + e];
    }
    // a row that sees nothing is no node: every split's sum is zero
    const bool none = sum == 0.f && top == -INFINITY;
    const int64_t o_row = (n * a.M + row / G) * a.H + h * G + row % G;
#pragma unroll
    for (int e = 0; e < CPL; ++e)
        if (CPL * lane + e < D)
            Elem<Tin>::store(static_cast<Tin *>(a.out) + o_row * D + CPL * lane + e, none ? 0.f : acc[e] / sum);
    if (lane == 0 && a.lse != nullptr) a.lse[o_row] = none ? -INFINITY : top + logf(sum);
}

int row_tiles_of(int M, int H, int H_kv) { return (M * (H / H_kv) + kRows - 1) / kRows; }

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
        sms = 152;
    return sms;
}

// Splits of the longest cache the table can hold: about four CTAs per SM in all
// (more even out ragged lengths, 1,262 us instead of 1,390 for sixteen of up to
// 8,192 tokens, but cost 450 us instead of 324 for two long caches), at least
// eight key tiles in each.
int splits_of(int64_t units, int64_t room) {
    const int64_t tiles = room / kKeys + 2;
    int64_t s = (4 * (int64_t)sm_count() + units - 1) / units;
    if (s > tiles / 8) s = tiles / 8;
    return (int)(s < 1 ? 1 : s);
}

template <typename Tin, int D> cudaError_t run(const TreeAttention &a, void *workspace, cudaStream_t stream) {
    const int rt = row_tiles_of(a.M, a.H, a.H_kv);
    const int64_t units = (int64_t)a.N * a.H_kv * rt;
    const int splits = splits_of(units, (int64_t)a.max_pages * a.page_size);
    Partials p{};
    if (splits > 1) {
        p.x = static_cast<float *>(workspace);
        p.z = p.x + units * splits * kRows;
        p.o = p.z + units * splits * kRows;
    }
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = allow_dynamic_smem(tree_attention_kernel<Tin, D>, smem_bytes<D>(), smem_set);
    if (e != cudaSuccess) return e;
    tree_attention_kernel<Tin, D><<<dim3((unsigned)units, (unsigned)splits), kThreads, smem_bytes<D>(), stream>>>(
        a, rt, splits, p);
    count_launches(1);
    if (splits > 1) {
        tree_attention_join_kernel<Tin, D><<<(unsigned)(units * (kRows / 4)), kThreads, 0, stream>>>(a, rt, splits, p);
        count_launches(1);
    }
    return cudaGetLastError();
}

#define KDA_DISPATCH_D(D, CALL)                        \
    switch (D) {                                       \
    case 16: { constexpr int DD = 16; return CALL; }   \
    case 32: { constexpr int DD = 32; return CALL; }   \
    case 64: { constexpr int DD = 64; return CALL; }   \
    case 128: { constexpr int DD = 128; return CALL; } \
    default: return cudaErrorInvalidValue;             \
    }

}  // namespace

size_t tree_attention_partial_bytes(int32_t N, int32_t M, int32_t H, int32_t H_kv, int32_t D, kda_dtype dt,
                                    int32_t page_size, int32_t max_pages) {
    // the number of pages is not known here: room for whichever form the call takes
    const size_t tc = tree_attention_tc_supported(H, H_kv, D, dt, 1, page_size)
                          ? tree_attention_tc_partial_bytes(M, H, H_kv, D) : 0;
    const int64_t units = (int64_t)N * H_kv * row_tiles_of(M, H, H_kv);
    const int splits = splits_of(units, (int64_t)max_pages * page_size);
    const size_t simple = splits > 1 ? (size_t)units * splits * kRows * (D + 2) * 4 : 0;
    return simple > tc ? simple : tc;
}

cudaError_t launch_tree_attention(const TreeAttention &a, int32_t D, kda_dtype dt, void *workspace,
                                  cudaStream_t stream) {
    if (tree_attention_tc_supported(a.H, a.H_kv, D, dt, a.num_pages, a.page_size))
        return launch_tree_attention_tc(a, D, workspace, stream);
    const cudaError_t e = cudaMemsetAsync(a.status, 0, sizeof(int32_t), stream);
    if (e != cudaSuccess) return e;
    if (dt == KDA_BF16) KDA_DISPATCH_D(D, (run<__nv_bfloat16, DD>(a, workspace, stream)))
    KDA_DISPATCH_D(D, (run<float, DD>(a, workspace, stream)))
}

}  // namespace kda
