// kda_tree_attention.cu -- softmax attention of a tree of drafted tokens over
// a paged cache and the tree itself ("From GPT-2 to Kimi K3, from first
// principles", Chapter 1 for softmax attention and its cache, Chapter 14 for
// the drafts; softmax layers with a cache of whole heads between KDA layers).
//
// Row (m, hq) attends to keys 0 .. len-1 of its sequence's cache and to the
// keys of the nodes on m's line.  One pass over the keys per row with a
// running maximum x and sum z:
//     x' = max(x, max_j s_j),  z' = z e^{x - x'} + sum_j e^{s_j - x'},
//     o' = o e^{x - x'} + sum_j e^{s_j - x'} v_j,   out = o / z, lse = x + ln z
//
// This file: the form for fp32 and for the head and page sizes that the tcgen05
// form does not take.  All rows of a cache head (M nodes x G query heads) share
// its keys: a CTA takes up to 64 of them, sixteen to a warp, over tiles of 32
// keys, two of which are in shared memory (cp.async, one on its way).  The keys of
// a tile are dealt to two warps for each sixteen rows, to four where there are two
// times sixteen rows or fewer.  The units' tiles are cut evenly over the CTAs.
//
// Products: mma.sync m16n8k8 on tf32 operands.  An fp32 factor is the nearest tf32
// number and a rest of eleven bits, x = x1 + x2 to 2^-23; x1 y1 + x1 y2 + x2 y1 is
// taken, x2 y2 (up to 2^-22 of x y) is left out.  The tensor cores cut the sums that they add
// to: so sixteen channels' large terms at a time are added up in fp32 registers,
// as are the tiles' output sums, and the scores' small terms have a sum of their
// own.  Against 64 bits the outputs err by 1.2e-7 to 3.6e-7 of their RMS (an fp32
// product and softmax by 5.7e-7; with cut parts and scores summed in the tensor
// cores it was 1.1e-6, 7% faster).  bf16 factors are exact in tf32: one product for
// the scores, two (the weights' parts) for the sums.  An infinity among the keys
// or values that an fp32 row sees gives NaN (inf - inf in the rest), and so does a key or a cached
// value whose nearest tf32 number is infinity.  Neither reaches a row that does not see it.
//
// Measured, fp32, graphs of one call on two inputs in turn: five caches of up to
// 3,001 tokens, 4 heads of 64, 11 nodes x 3 query heads 29 us; sixteen of 512 ..
// 8,192 tokens 103 us; the same with 8 heads of 128 and 16 x 4 rows 428 us, where the
// products alone take 186 (8 clocks each) and the bytes 87; two of about 62,000
// tokens, 4 heads of 128, 7 x 8 rows 369 us (products 168, bytes 76).  The rest is
// what eight to sixteen warps per SM do not hide.  bf16, the sixteen caches with 8
// heads of 128 on pages of 20 tokens: 258 us (bytes 44; 73 us on pages of 64, which
// take the tcgen05 form); with 8 heads of 32: 106 us (bytes 11).  On CUDA cores the four took 47, 309, 1,247 and 1,160
// us with a row and a key per lane, 35, 151, 820 and 572 with two rows x four keys
// per lane, all of it waiting for shared memory.  As many splits for every sequence
// instead of the even cut took 1.4 times as long with ragged lengths.
#include "kda_internal.cuh"
#include "kda_tc.cuh"
#include "kda_tree.cuh"
#include "kda_tree_cut.cuh"
#include "kda_prefix_cut.cuh"

#include <math.h>

#include <algorithm>
#include <type_traits>

namespace kda {
namespace {

constexpr int kKeys = 32, kRowsPerWarp = 16, kMaxRowWarps = 4, kMaxWarps = 8;

// A key's row and a value's row in shared memory, padded: the lanes of a read start in
// different banks.
template <int D> constexpr int kLdk = D + 16;
template <typename Tin, int D> constexpr int kLdv = D + 16 / (int)sizeof(Tin);

// Whether the rests of the queries stand beside them: not where that costs a CTA per SM.
template <typename Tin, int WK> constexpr bool kRests = sizeof(Tin) == 4 && WK > 2;

// Two tiles of keys and values, whose place the warps' sums take at the end; the
// queries, in parts or as they are.
template <typename Tin, int D> constexpr size_t tiles_bytes(int warps) {
    const size_t tiles = 2 * kKeys * (kLdk<D> + kLdv<Tin, D>) * sizeof(Tin),
                 sums = (size_t)warps * kRowsPerWarp * (D + 4) * sizeof(float);
    return tiles > sums ? tiles : sums;
}

template <typename Tin, int D, int WK> constexpr size_t smem_bytes(int row_warps) {
    return tiles_bytes<Tin, D>(row_warps * WK) +
           (size_t)row_warps * kRowsPerWarp * kLdk<D> * (kRests<Tin, WK> ? 2 : 1) * sizeof(float);
}

struct Units {
    // the cache's tiles, then the tree's
    static __device__ __forceinline__ int tiles(int len, int M) {
        return (len + kKeys - 1) / kKeys + (M + kKeys - 1) / kKeys;
    }
};

struct Shape {
    int32_t groups;         // of rows per cache head
    int32_t ctas;
    Place *places;          // one per CTA
    float *part;            // two slots per CTA: rows x D sums, then rows maxima, rows sums of weights
                            // (-1: no node)
};

// W consecutive elements from shared memory.
template <int W> __device__ __forceinline__ void read_run(const float *p, float (&x)[W]) {
    if constexpr (W == 2) {
        const float2 a = *reinterpret_cast<const float2 *>(p);
        x[0] = a.x;
        x[1] = a.y;
    } else {
        const float4 a = *reinterpret_cast<const float4 *>(p);
        x[0] = a.x;
        x[1] = a.y;
        x[2] = a.z;
        x[3] = a.w;
    }
}

template <int W> __device__ __forceinline__ void read_run(const __nv_bfloat16 *p, float (&x)[W]) {
    uint32_t w[W / 2];
    if constexpr (W == 2) {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
        const uint2 a = *reinterpret_cast<const uint2 *>(p);
        w[0] = a.x;
        w[1] = a.y;
    }
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {                       // bf16 -> fp32 is a 16-bit shift
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// x = part + rest: the nearest tf32 number, and what is left, cut to eleven bits.  From
// 2^128 - 2^116 on the nearest one is infinity.  In the tree's tile, where rows that do not see a
// value take it into their products, its part ends at the largest tf32 number, and what the rest
// is cut by has a product of its own, since that rest is longer.  (The limit everywhere took 14%
// more time, the conversion instruction with saturation 21%; in the tree's tile -3 to +2%.)
__device__ __forceinline__ float part_of(float x) {
    return __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xffffe000u);
}
__device__ __forceinline__ float part_below_infinity(float x) {
    const float most = __uint_as_float(0x7f7fe000u);
    return fminf(fmaxf(part_of(x), -most), most);
}
__device__ __forceinline__ float rest_of(float x, float part) {
    return __uint_as_float(__float_as_uint(x - part) & 0xffffe000u);
}

// Four results: o by, or zeros.
__device__ __forceinline__ void store4(float *p, bool none, float4 o, float by) {
    *reinterpret_cast<float4 *>(p) = none ? make_float4(0.f, 0.f, 0.f, 0.f)
                                          : make_float4(o.x * by, o.y * by, o.z * by, o.w * by);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, bool none, float4 o, float by) {
    const uint2 x = make_uint2(tc::pack_bf16x2(o.x * by, o.y * by), tc::pack_bf16x2(o.z * by, o.w * by));
    *reinterpret_cast<uint2 *>(p) = none ? make_uint2(0u, 0u) : x;
}

// Four of a row's sums, for the kernel that joins them with a prefix's.
__device__ __forceinline__ void put_sums(const RowSums &rows, int64_t row, int D, int c, float4 o, float top, float sum) {
    *reinterpret_cast<float4 *>(rows.o + row * D + c) = o;
    if (c == 0) {
        rows.top[row] = top;
        rows.sum[row] = sum;
    }
}

// c += a b; a 16 x 8 (lane 4 g + t: rows g, g + 8 of column t, then of column t + 4),
// b 8 x 8 (rows t, t + 4 of column g), c 16 x 8 (row g, columns 2 t, 2 t + 1; row g + 8)
__device__ __forceinline__ void mma_tf32(float (&c)[4], const float (&a)[4], float b0, float b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])),
          "r"(__float_as_uint(a[3])), "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

// c = a b
__device__ __forceinline__ void mma_tf32_first(float (&c)[4], const float (&a)[4], float b0, float b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])),
          "r"(__float_as_uint(a[3])), "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)), "f"(0.f));
}

// 16 bytes to shared memory, zeros when `from` is not to be read.
__device__ __forceinline__ void copy16(void *to, const void *from, bool read) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
                 "l"(from), "r"(read ? 16 : 0) : "memory");
}

__device__ __forceinline__ const TreeAttention &tree_of(const TreeAttention &a) { return a; }
__device__ __forceinline__ const TreeAttention &tree_of(const PrefixAttention &a) { return a.t; }

// Args: TreeAttention (a sequence's rows, its cache and its tree), or PrefixAttention (the rows of
// all a prefix's sequences and the prefix's keys; no tree).
template <typename Tin, int D, int WK, typename Args>
__global__ void __launch_bounds__(32 * kMaxWarps, 2)
tree_attention_kernel(const Args args, const typename std::conditional<std::is_same<Args, PrefixAttention>::value,
                                                                       PrefixShape, Shape>::type sh) {
    constexpr bool PREFIX = std::is_same<Args, PrefixAttention>::value;
    const TreeAttention &a = tree_of(args);
    constexpr bool SPLIT = sizeof(Tin) == 4;                // operands have a rest
    constexpr bool RESTS = kRests<Tin, WK>;
    constexpr int LK = kLdk<D>, LV = kLdv<Tin, D>, LO = D + 4;
    constexpr int NT = kKeys / 8 / WK;                      // groups of eight keys per warp and tile
    // columns of a value per read; four for d = 128 keep too many registers (20% slower)
    constexpr int W = D == 16 || D == 128 ? 2 : 4, E = D / 8 / W;
    constexpr int kAtOnce = D == 128 ? 1 : 2;               // (likewise, 8%)
    extern __shared__ __align__(16) unsigned char smem[];
    Tin *sk = reinterpret_cast<Tin *>(smem), *sv = sk + 2 * kKeys * LK;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
    const int crows = threads / 32 / WK * kRowsPerWarp, wrow = warp / WK * kRowsPerWarp, wk = warp % WK;
    float *sq = reinterpret_cast<float *>(smem + tiles_bytes<Tin, D>(threads / 32)), *sq_rest = sq + crows * LK;
    __shared__ int32_t par[kMaxTreeNodes];
    __shared__ uint64_t line[kMaxTreeNodes];
    __shared__ float s_top[kMaxWarps * kRowsPerWarp], s_sum[kMaxWarps * kRowsPerWarp];
    const Tin *q = static_cast<const Tin *>(a.q), *k_new = static_cast<const Tin *>(a.k_new),
              *v_new = static_cast<const Tin *>(a.v_new), *k_cache = static_cast<const Tin *>(a.k_cache),
              *v_cache = static_cast<const Tin *>(a.v_cache);
    const int G = a.H / a.H_kv, M = a.M;

    int32_t status;
    auto first_run = [&](int64_t &left) {
        if constexpr (PREFIX) {
            const PrefixPlace first = find_prefix_place<kKeys>(args, sh.units, sh.ctas, blockIdx.x);
            const int64_t stop = piece_start(first.total, sh.ctas, blockIdx.x + 1);
            if (tid == 0) sh.places[blockIdx.x] = first;
            status = first.status;
            left = stop - first.start;
            return left > 0 ? prefix_run<kKeys>(args, first, stop) : PrefixRun<kKeys>{};
        } else {
            __shared__ int64_t buf[34];
            Place first;
            find_place<Units>(a, sh.groups, sh.ctas, blockIdx.x, buf, first);
            const int64_t stop = piece_start(first.total, sh.ctas, blockIdx.x + 1);
            if (tid == 0) sh.places[blockIdx.x] = first;
            status = first.status;
            left = stop - first.start;
            return CutRun<Units>{left, first.n, first.r, first.len, (int32_t)(first.start - first.unit0),
                                 Units::tiles(first.len, M)};
        }
    };
    int64_t todo;
    auto run = first_run(todo);
    if (todo <= 0) {                                        // the whole block
        if (PREFIX) tc::wait_prerequisites();               // (the next kernel counts on the ones before this)
        return;
    }
    auto advance = [&]() {
        if constexpr (PREFIX) run.advance(args, sh.units);
        else run.advance(a, sh.groups);
    };
    __shared__ int32_t s_status;
    if (tid == 0) s_status = status;
    for (; run.left > 0; advance()) {
        // first_node: the unit's rows are those of its nodes there on; groups: units per cache head
        int64_t first_node;
        int groups, rows;
        const int32_t *table;
        if constexpr (PREFIX) {
            first_node = (int64_t)run.seq0 * M;
            groups = run.groups;
            rows = run.rows;
            table = args.table + (int64_t)run.p * args.max_pages;
        } else {
            first_node = (int64_t)run.n * M;
            groups = sh.groups;
            rows = M * G;
            table = a.page_table + (int64_t)run.n * a.max_pages;
        }
        const int h = run.r / groups, row0 = run.r % groups * crows, len = run.len;
        const int cache_tiles = (len + kKeys - 1) / kKeys, t0 = run.t0, t1 = t0 + run.count();
        __syncthreads();                                    // the last unit is done with shared memory
        auto base_of = [&](int t) { return t >= cache_tiles ? (t - cache_tiles) * kKeys : t * kKeys; };

        // Where lane j's key of a tile lies: its page (as the table has it) and its place in
        // the page, asked for a tile before the copy needs them; place -1: no such key.
        int page = 0, place = -1;
        auto ask = [&](int t) {
            const int pos = t * kKeys + lane;
            place = -1;
            if (t < t1 && t < cache_tiles && pos < len) {
                page = table[pos / a.page_size];
                place = pos % a.page_size;
            }
        };
        auto fetch = [&](int t) {
            const bool tree = !PREFIX && t >= cache_tiles;
            int64_t at = -1;                                // the key's row
            if (tree) {
                if (base_of(t) + lane < M) at = (first_node + base_of(t) + lane) * a.H_kv + h;
            } else if (place >= 0) {
                if (page >= 0 && page < a.num_pages)
                    at = ((int64_t)page * a.H_kv + h) * a.page_size + place;
                else
                    atomicOr(&s_status, finding(KDA_DEVICE_BAD_PAGE));      // the key then counts as zeros
            }
            const Tin *pk = tree ? k_new : k_cache, *pv = tree ? v_new : v_cache;
            constexpr int RUN = 16 / (int)sizeof(Tin), CH = D / RUN;
            Tin *dk = sk + (t & 1) * kKeys * LK, *dv = sv + (t & 1) * kKeys * LV;
            // (32 CH pieces: a warp's 32 lanes are all in range or none is)
#pragma unroll 2
            for (int i = tid; i < kKeys * CH; i += threads) {
                const int j = i / CH, c = i % CH * RUN;
                const int64_t row = __shfl_sync(0xffffffffu, (long long)at, j);
                const int64_t off = row < 0 ? 0 : row * D + c;
                copy16(dk + j * LK + c, pk + off, row >= 0);
                copy16(dv + j * LV + c, pv + off, row >= 0);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        ask(t0);
        if (t0 < t1) fetch(t0);
        ask(t0 + 1);

        if (!PREFIX)
            for (int m = tid; m < M; m += threads) par[m] = a.parent[first_node + m];
        for (int i = tid; i < crows * (D / 8); i += threads) {
            const int r = row0 + i / (D / 8), c = i % (D / 8) * 8;
            float x[8] = {0.f};
            if (r < rows) Elem<Tin>::load8(q + ((first_node + r / G) * a.H + h * G + r % G) * D + c, x);
            float x1[8], x2[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x1[e] = RESTS ? part_of(x[e]) : x[e];
                x2[e] = rest_of(x[e], x1[e]);
            }
            Elem<float>::store8(sq + i / (D / 8) * LK + c, x1);
            if (RESTS) Elem<float>::store8(sq_rest + i / (D / 8) * LK + c, x2);
        }
        __syncthreads();
        if (!PREFIX) {
            for (int m = tid; m < M; m += threads) line[m] = tree_line(par, m);
            __syncthreads();
        }

        // A lane's rows of the warp are g, g + 8, its keys of eight 2 t, 2 t + 1.
        const int g = lane >> 2, t4 = lane & 3;
        int node[2];                                            // -1: the row is not of a node
        float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f}, acc[E][W][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = row0 + wrow + g + 8 * r;
            node[r] = row < rows && (PREFIX || line[row / G] != 0) ? row / G : -1;
        }
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int j = 0; j < W; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[e][j][i] = 0.f;
        const int my_q = (wrow + g) * LK + 4 * t4, my_key = wk * 8 * NT;
        for (int t = t0; t < t1; ++t) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();                                    // the tile is there, its predecessor is done with
            if (t + 1 < t1) fetch(t + 1);
            ask(t + 2);
            const bool tree = !PREFIX && t >= cache_tiles;
            const int base = base_of(t), count = min(kKeys, (tree ? M : len) - base);
            const Tin *tk = sk + ((t & 1) * kKeys + my_key + g) * LK + 4 * t4;
            const Tin *tv = sv + ((t & 1) * kKeys + my_key) * LV;
            // Scores: of sixteen channels lane t has 4 t .. 4 t + 3, the first two for one
            // product (as its columns t, t + 4), the others for the next.
            float s1[NT][4], s2[NT][4];
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) s1[i][e] = s2[i][e] = 0.f;
#pragma unroll kAtOnce
            for (int c = 0; c < D; c += 16) {
                float qa[4], qb[4], ra[4], rb[4];
                read_run<4>(sq + my_q + c, qa);
                read_run<4>(sq + my_q + 8 * LK + c, qb);
                if (RESTS) {
                    read_run<4>(sq_rest + my_q + c, ra);
                    read_run<4>(sq_rest + my_q + 8 * LK + c, rb);
                } else if (SPLIT) {
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const float xa = qa[y], xb = qb[y];
                        qa[y] = part_of(xa);
                        qb[y] = part_of(xb);
                        ra[y] = rest_of(xa, qa[y]);
                        rb[y] = rest_of(xb, qb[y]);
                    }
                }
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    float x[4], sum16[4];                   // the large terms of these channels
                    read_run<4>(tk + 8 * i * LK + c, x);
#pragma unroll
                    for (int y = 0; y < 4; y += 2) {
                        const float f[4] = {qa[y], qb[y], qa[y + 1], qb[y + 1]};
                        const float x0 = SPLIT ? part_of(x[y]) : x[y], x1 = SPLIT ? part_of(x[y + 1]) : x[y + 1];
                        if (y == 0)
                            mma_tf32_first(sum16, f, x0, x1);
                        else
                            mma_tf32(sum16, f, x0, x1);
                        if (SPLIT) {
                            const float f2[4] = {ra[y], rb[y], ra[y + 1], rb[y + 1]};
                            mma_tf32(s2[i], f, rest_of(x[y], x0), rest_of(x[y + 1], x1));
                            mma_tf32(s2[i], f2, x0, x1);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) s1[i][e] += sum16[e];
                }
            }
            uint32_t seen[2];                                   // which of the tile's keys the row sees
            float shrink[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                seen[r] = node[r] < 0 ? 0u : (tree ? (uint32_t)(line[node[r]] >> base) : 0xffffffffu) &
                                                  (0xffffffffu >> (kKeys - count));
                const uint32_t bits = seen[r] >> (my_key + 2 * t4);
                float mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float &x = s1[i][2 * r + e];
                        x = (bits >> (8 * i + e) & 1) != 0 ? (x + s2[i][2 * r + e]) * a.scale : -INFINITY;
                        mx = fmaxf(mx, x);
                    }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float was = top[r];
                top[r] = fmaxf(was, mx);
                // no key seen yet: every difference below is taken from zero instead
                const float from = top[r] == -INFINITY ? 0.f : top[r];
                shrink[r] = __expf(was - from);
                sum[r] *= shrink[r];                            // over the lane's own keys; joined at the end
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float &x = s1[i][2 * r + e];
                        x = (bits >> (8 * i + e) & 1) != 0 ? __expf(x - from) : 0.f;
                        sum[r] += x;
                    }
            }
            // Sums: the weights as they lie are the left operand when its columns t, t + 4 are
            // keys 2 t, 2 t + 1.  Column g of product (e, j) is column 8 W e + W g + j.
            float p1[NT][4], p2[NT][4];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const float w[4] = {s1[i][0], s1[i][2], s1[i][1], s1[i][3]};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p1[i][e] = part_of(w[e]);
                    p2[i][e] = rest_of(w[e], p1[i][e]);
                }
            }
            bool odd = false;                                   // a value that is no number
            auto add = [&](auto in_tree) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    float o[W][4];
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        float x[W], z[W];
                        read_run<W>(tv + (8 * i + 2 * t4) * LV + e * 8 * W + W * g, x);
                        read_run<W>(tv + (8 * i + 2 * t4 + 1) * LV + e * 8 * W + W * g, z);
#pragma unroll
                        for (int j = 0; j < W; ++j) {
                            if (decltype(in_tree)::value) {
                                // zero in the products, so that it does not reach rows that do not see it
                                const bool fx = fabsf(x[j]) < INFINITY, fz = fabsf(z[j]) < INFINITY;
                                odd |= !fx || !fz;
                                x[j] = fx ? x[j] : 0.f;
                                z[j] = fz ? z[j] : 0.f;
                            }
                            auto part = [](float f) {
                                return !SPLIT ? f : decltype(in_tree)::value ? part_below_infinity(f) : part_of(f);
                            };
                            const float x1 = part(x[j]), z1 = part(z[j]);
                            if (i == 0)
                                mma_tf32_first(o[j], p2[i], x1, z1);
                            else
                                mma_tf32(o[j], p2[i], x1, z1);
                            if (SPLIT) {
                                const float x2 = rest_of(x[j], x1), z2 = rest_of(z[j], z1);
                                if (decltype(in_tree)::value)
                                    mma_tf32(o[j], p1[i], x[j] - x1 - x2, z[j] - z1 - z2);
                                mma_tf32(o[j], p1[i], x2, z2);
                            }
                            mma_tf32(o[j], p1[i], x1, z1);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < W; ++j)
#pragma unroll
                        for (int y = 0; y < 4; ++y) acc[e][j][y] = fmaf(acc[e][j][y], shrink[y / 2], o[j][y]);
                }
            };
            if (tree)
                add(std::true_type{});
            else
                add(std::false_type{});
            if (tree && __any_sync(0xffffffffu, odd)) {
                // the rows that see it get it, unweighted: no number stays no number
                for (int k = my_key; k < min(my_key + 8 * NT, count); ++k)
#pragma unroll
                    for (int e = 0; e < E; ++e)
#pragma unroll
                        for (int y = 0; y < 2 * W; ++y) {
                            const float x = Elem<Tin>::load(tv + (k - my_key) * LV + e * 8 * W + 2 * W * t4 + y);
#pragma unroll
                            for (int r = 0; r < 2; ++r)
                                if (!(fabsf(x) < INFINITY) && (seen[r] >> k & 1) != 0)
                                    acc[e][y % W][2 * r + y / W] += x;
                        }
            }
        }
        // The warps of the same rows meet in the tiles' place.
        const bool whole = t0 == 0 && t1 == run.tiles;
        float *part = sh.part + (size_t)(2 * blockIdx.x + (t0 > 0 ? 0 : 1)) * crows * (D + 2);
        float *so = reinterpret_cast<float *>(smem);
        if (PREFIX && whole) tc::wait_prerequisites();      // the own keys' sums are there
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int at = warp * kRowsPerWarp + g + 8 * r;
            float z = sum[r];
            z += __shfl_xor_sync(0xffffffffu, z, 1);
            z += __shfl_xor_sync(0xffffffffu, z, 2);
            if (t4 == 0) {
                s_top[at] = top[r];
                s_sum[at] = z;
            }
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
                for (int y = 0; y < 2 * W; y += 2)
                    *reinterpret_cast<float2 *>(so + at * LO + e * 8 * W + 2 * W * t4 + y) =
                        make_float2(acc[e][y % W][2 * r + y / W], acc[e][(y + 1) % W][2 * r + (y + 1) / W]);
        }
        __syncthreads();
        for (int i = tid; i < crows * (D / 4); i += threads) {
            const int lr = i / (D / 4), c = i % (D / 4) * 4, row = row0 + lr;
            if (row >= rows) continue;
            const int at = lr / kRowsPerWarp * WK * kRowsPerWarp + lr % kRowsPerWarp;
            float x = s_top[at], z = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 1; w < WK; ++w) x = fmaxf(x, s_top[at + w * kRowsPerWarp]);
            const float from = x == -INFINITY ? 0.f : x;
#pragma unroll
            for (int w = 0; w < WK; ++w) {
                const float by = WK == 1 ? 1.f : __expf(s_top[at + w * kRowsPerWarp] - from);
                const float4 y = *reinterpret_cast<const float4 *>(so + (at + w * kRowsPerWarp) * LO + c);
                z += by * s_sum[at + w * kRowsPerWarp];
                o.x += by * y.x;
                o.y += by * y.y;
                o.z += by * y.z;
                o.w += by * y.w;
            }
            if constexpr (PREFIX) {
                const int64_t o_row = (first_node + row / G) * a.H + h * G + row % G;
                if (whole) {
                    const RowJoin<false> join(x, z, a.rows.top[o_row], a.rows.sum[o_row]);
                    store_out4(static_cast<Tin *>(a.out) + o_row * D + c,
                               join(o, *reinterpret_cast<const float4 *>(a.rows.o + o_row * D + c)));
                    if (c == 0 && a.lse != nullptr) a.lse[o_row] = join.lse;
                } else {
                    *reinterpret_cast<float4 *>(part + lr * D + c) = o;
                    if (c == 0) {
                        part[crows * D + lr] = x;
                        part[crows * D + crows + lr] = z;
                    }
                }
                continue;
            }
            if (whole) {
                const int64_t o_row = (first_node + row / G) * a.H + h * G + row % G;
                const bool none = line[row / G] == 0;
                if (a.rows.o != nullptr) {
                    put_sums(a.rows, o_row, D, c, o, x, none ? -1.f : z);
                    continue;
                }
                store4(static_cast<Tin *>(a.out) + o_row * D + c, none, o, 1.f / z);
                if (c == 0 && a.lse != nullptr) a.lse[o_row] = none ? -INFINITY : x + logf(z);
            } else {
                *reinterpret_cast<float4 *>(part + lr * D + c) = o;
                if (c == 0) {
                    const bool none = line[row / G] == 0;
                    part[crows * D + lr] = none ? -INFINITY : x;
                    part[crows * D + crows + lr] = none ? -1.f : z;
                }
            }
        }
    }
    __syncthreads();
    if (tid == 0) sh.places[blockIdx.x].status = s_status;
    if (PREFIX) tc::wait_prerequisites();                   // (the next kernel counts on the ones before this)
    tc::launch_dependents();
}

// Joins the units that were cut.  Block (b, y), b > 0: the cut between CTAs
// b - 1 and b, rows 16 y .. 16 y + 15 of its unit; it works when that is the
// unit's first cut.  Block (0, 0) gathers the status.  Its launch overlaps the
// kernel before it, whose results it waits for.
template <typename Tin, int D>
__global__ void __launch_bounds__(256)
tree_attention_join_kernel(const TreeAttention a, const Shape sh) {
    const int b = blockIdx.x, G = a.H / a.H_kv, crows = gridDim.y * kRowsPerWarp;
    if (a.rows.o != nullptr) tc::launch_dependents();       // the prefix's kernel, which waits before it takes the sums
    tc::wait_prerequisites();
    if (b == 0) {
        if (blockIdx.y == 0) gather_status(sh.places, sh.ctas, a.status);
        return;
    }
    const Place p = sh.places[b];
    const int64_t before = sh.places[b - 1].start;
    if (p.start >= p.total || p.unit0 == p.start || before > p.unit0) return;
    const int64_t end = p.unit0 + Units::tiles(p.len, a.M);
    const int parts = first_past(p.total, sh.ctas, end) - (b - 1);
    const int h = p.r / sh.groups;
    // part i is CTA b - 1 + i's: its last unit for the first, its first one after that
    auto piece = [&](int i) { return sh.part + (size_t)(2 * (b - 1 + i) + (i == 0 ? 1 : 0)) * crows * (D + 2); };
    for (int e = threadIdx.x; e < kRowsPerWarp * (D / 4); e += 256) {
        const int lr = blockIdx.y * kRowsPerWarp + e / (D / 4), c = e % (D / 4) * 4, row = p.r % sh.groups * crows + lr;
        if (row >= a.M * G) continue;
        float top = -INFINITY, sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        const bool none = piece(parts - 1)[crows * D + crows + lr] < 0.f;
        for (int i0 = 0; i0 < parts; i0 += 8) {
            // eight parts at a time, so that their reads are under way together
            float x[8], z[8];
            float4 y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float *q = piece(min(i0 + i, parts - 1));
                x[i] = i0 + i < parts ? q[crows * D + lr] : -INFINITY;
                z[i] = q[crows * D + crows + lr];
                y[i] = *reinterpret_cast<const float4 *>(q + lr * D + c);
            }
            float was = top;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, x[i]);
            const float from = top == -INFINITY ? 0.f : top, shrink = __expf(was - from);
            sum *= shrink;
            o.x *= shrink; o.y *= shrink; o.z *= shrink; o.w *= shrink;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // (a part with nothing seen adds zeros; one whose scores are no numbers has a maximum of
                // -infinity too and makes the row one: a weight of zero skips nothing)
                if (i0 + i < parts) {
                    const float w = __expf(x[i] - from);
                    sum += w * z[i];
                    o.x += w * y[i].x; o.y += w * y[i].y; o.z += w * y[i].z; o.w += w * y[i].w;
                }
            }
        }
        const int64_t o_row = ((int64_t)p.n * a.M + row / G) * a.H + h * G + row % G;
        if (a.rows.o != nullptr) {
            put_sums(a.rows, o_row, D, c, o, top, none ? -1.f : sum);
            continue;
        }
        store4(static_cast<Tin *>(a.out) + o_row * D + c, none, o, 1.f / sum);
        if (c == 0 && a.lse != nullptr) a.lse[o_row] = none ? -INFINITY : top + logf(sum);
    }
}

// The rows of a cache head in as few groups as CTAs can hold, the same number of warps in each.
struct Warps {
    int groups, rows, keys;     // groups per head; warps by rows, by keys
};
Warps warps_of(int M, int H, int H_kv) {
    const int all = M * (H / H_kv), most = kMaxRowWarps * kRowsPerWarp, groups = (all + most - 1) / most;
    const int rows = ((all + groups - 1) / groups + kRowsPerWarp - 1) / kRowsPerWarp;
    return {groups, rows, rows <= 2 ? 4 : 2};
}

// CTAs: as many as are resident at once, at the registers that the kernel is held to.
template <typename Tin, int D> int ctas_of(const Warps &w) {
    const size_t smem = (w.keys == 4 ? smem_bytes<Tin, D, 4>(w.rows) : smem_bytes<Tin, D, 2>(w.rows)) + 4096;
    const int by_smem = (int)(228 * 1024 / smem), by_regs = 512 / (32 * w.rows * w.keys);
    return sm_count() * std::max(1, std::min(by_smem, by_regs));
}

template <typename Tin, int D, int WK>
cudaError_t run_main(const TreeAttention &a, const Shape &sh, int row_warps, cudaStream_t stream) {
    static std::atomic<uint64_t> smem_set{0};
    const cudaError_t e = allow_dynamic_smem(tree_attention_kernel<Tin, D, WK, TreeAttention>,
                                             smem_bytes<Tin, D, WK>(kMaxWarps / WK), smem_set);
    if (e != cudaSuccess) return e;
    tree_attention_kernel<Tin, D, WK, TreeAttention>
        <<<sh.ctas, 32 * row_warps * WK, smem_bytes<Tin, D, WK>(row_warps), stream>>>(a, sh);
    count_launches(1);
    return cudaGetLastError();
}

template <typename Tin, int D> cudaError_t run(const TreeAttention &a, void *workspace, cudaStream_t stream) {
    const Warps w = warps_of(a.M, a.H, a.H_kv);
    Shape sh;
    sh.groups = w.groups;
    sh.ctas = ctas_of<Tin, D>(w);
    sh.places = static_cast<Place *>(workspace);
    sh.part = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + place_bytes(sh.ctas));
    cudaError_t e = w.keys == 4 ? run_main<Tin, D, 4>(a, sh, w.rows, stream)
                                : run_main<Tin, D, 2>(a, sh, w.rows, stream);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute overlap;
    overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    overlap.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sh.ctas, w.rows);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = &overlap;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, tree_attention_join_kernel<Tin, D>, a, sh);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();                           // reported here
        return e;
    }
    count_launches(1);
    return cudaSuccess;
}

// The rows of a prefix: sixteen to a warp, four warps (fewer where there are fewer rows), by two of keys.
int prefix_row_warps(int64_t N, int M, int H, int H_kv) {
    const int64_t all = N * M * (H / H_kv);
    return (int)std::min<int64_t>(kMaxRowWarps, (all + kRowsPerWarp - 1) / kRowsPerWarp);
}
template <typename Tin, int D> int prefix_ctas(int row_warps) { return ctas_of<Tin, D>(Warps{0, row_warps, 2}); }

template <typename Tin, int D> cudaError_t run_prefix(const PrefixAttention &a, void *workspace, cudaStream_t stream) {
    const int warps = prefix_row_warps(a.t.N, a.t.M, a.t.H, a.t.H_kv);
    PrefixShape sh;
    sh.units = {1, warps * kRowsPerWarp, warps * kRowsPerWarp};
    sh.ctas = prefix_ctas<Tin, D>(warps);
    sh.places = static_cast<PrefixPlace *>(workspace);
    sh.part = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + prefix_place_bytes(sh.ctas));
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = allow_dynamic_smem(tree_attention_kernel<Tin, D, 2, PrefixAttention>,
                                       smem_bytes<Tin, D, 2>(kMaxRowWarps), smem_set);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute overlap;
    overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    overlap.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sh.ctas);
    cfg.blockDim = dim3(32 * warps * 2);
    cfg.dynamicSmemBytes = smem_bytes<Tin, D, 2>(warps);
    cfg.stream = stream;
    cfg.attrs = &overlap;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, tree_attention_kernel<Tin, D, 2, PrefixAttention>, a, sh);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();                           // reported here
        return e;
    }
    count_launches(1);
    return launch_prefix_join<Tin, D, kKeys, false>(a, sh, stream);
}

template <typename Tin, int D> size_t prefix_bytes(int32_t N, int32_t M, int32_t H, int32_t H_kv) {
    const int warps = prefix_row_warps(N, M, H, H_kv), ctas = prefix_ctas<Tin, D>(warps);
    return prefix_place_bytes(ctas) + prefix_part_bytes(ctas, warps * kRowsPerWarp, D);
}

template <typename Tin, int D> size_t partial_bytes(int M, int H, int H_kv) {
    const Warps w = warps_of(M, H, H_kv);
    const int ctas = ctas_of<Tin, D>(w);
    return place_bytes(ctas) + (size_t)ctas * 2 * w.rows * kRowsPerWarp * (D + 2) * sizeof(float);
}

#define KDA_DISPATCH_D(D, CALL)                        \
    switch (D) {                                       \
    case 16: { constexpr int DD = 16; return CALL; }   \
    case 32: { constexpr int DD = 32; return CALL; }   \
    case 64: { constexpr int DD = 64; return CALL; }   \
    case 128: { constexpr int DD = 128; return CALL; } \
    default: break;                                    \
    }

}  // namespace

size_t tree_attention_partial_bytes(int32_t M, int32_t H, int32_t H_kv, int32_t D, kda_dtype dt, int32_t page_size) {
    // the number of pages is not known here: room for whichever form the call takes
    const size_t tc = tree_attention_tc_supported(H, H_kv, D, dt, 1, page_size)
                          ? tree_attention_tc_partial_bytes(M, H, H_kv, D) : 0;
    const size_t other = [&]() -> size_t {
        if (dt == KDA_BF16) KDA_DISPATCH_D(D, (partial_bytes<__nv_bfloat16, DD>(M, H, H_kv)))
        else KDA_DISPATCH_D(D, (partial_bytes<float, DD>(M, H, H_kv)))
        return 0;
    }();
    return std::max(tc, other);
}

cudaError_t launch_tree_attention(const TreeAttention &a, int32_t D, kda_dtype dt, void *workspace,
                                  cudaStream_t stream) {
    if (tree_attention_tc_supported(a.H, a.H_kv, D, dt, a.num_pages, a.page_size))
        return launch_tree_attention_tc(a, D, workspace, stream);
    if (dt == KDA_BF16) KDA_DISPATCH_D(D, (run<__nv_bfloat16, DD>(a, workspace, stream)))
    else KDA_DISPATCH_D(D, (run<float, DD>(a, workspace, stream)))
    return cudaErrorInvalidValue;
}

size_t prefix_attention_bytes(int32_t N, int32_t M, int32_t P, int32_t H, int32_t H_kv, int32_t D, kda_dtype dt,
                              int32_t page_size) {
    const size_t tc = tree_attention_tc_supported(H, H_kv, D, dt, 1, page_size)
                          ? prefix_attention_tc_bytes(N, M, P, H, H_kv, D) : 0;
    const size_t other = [&]() -> size_t {
        if (dt == KDA_BF16) KDA_DISPATCH_D(D, (prefix_bytes<__nv_bfloat16, DD>(N, M, H, H_kv)))
        else KDA_DISPATCH_D(D, (prefix_bytes<float, DD>(N, M, H, H_kv)))
        return 0;
    }();
    return std::max(tc, other);
}

cudaError_t launch_prefix_attention(const PrefixAttention &a, int32_t D, kda_dtype dt, void *workspace,
                                    cudaStream_t stream) {
    // the form of the own keys' sums, whose units the join shares
    if (tree_attention_tc_supported(a.t.H, a.t.H_kv, D, dt, a.t.num_pages, a.t.page_size))
        return launch_prefix_attention_tc(a, D, workspace, stream);
    if (dt == KDA_BF16) KDA_DISPATCH_D(D, (run_prefix<__nv_bfloat16, DD>(a, workspace, stream)))
    else KDA_DISPATCH_D(D, (run_prefix<float, DD>(a, workspace, stream)))
    return cudaErrorInvalidValue;
}

}  // namespace kda
