// kda_drafts.cu -- acceptance of drafted tokens against the target's
// probabilities (kda_verify_drafts) and the accepted tokens' keys and values
// into a paged cache (kda_cache_append).  "From GPT-2 to Kimi K3, from first
// principles", Chapter 14 (speculative decoding: the target verifies a
// draft's tokens, accepted updates are committed).
//
// Probabilities are compared and summed in fixed point (whole multiples of
// 2^-38, held in 64 bits), so that the drawn token does not depend on the
// order of the sums: any split of the vocabulary gives the same one.  A
// probability below 2^-38 counts as zero; 2^18 tokens of rounding
// shift the distribution by at most 2^-20.
#include "kda_internal.cuh"
#include "kda_tree.cuh"
#include "kda_tree_cut.cuh"

#include <cooperative_groups.h>

namespace kda {
namespace {

// A probability as a whole number of 2^-38, rounded toward zero, in two digits
// of 19 bits.  Adding 2^23 with rounding toward zero leaves the whole part in
// the significand's low bits, and what remains is exact: three fused
// multiply-adds and an add at full rate, where a conversion to 64 bits runs at
// a small part of it (131,072 tokens x 256 chains with draft probabilities: 125
// us converting, 57 us with the digits).  The digits carry 2^23's bits with them.
constexpr uint32_t kBias = 0x4b000000u;
__device__ __forceinline__ void digits38(float p, uint32_t &hi, uint32_t &lo) {
    p = fminf(fmaxf(p, 0.f), 1.f);                     // fmaxf drops a NaN
    const float h = __fmaf_rz(p, 524288.f, 8388608.f);
    const float rest = fmaf(p, 524288.f, -(h - 8388608.f));
    hi = __float_as_uint(h);
    lo = __float_as_uint(__fmaf_rz(rest, 524288.f, 8388608.f));
}
__device__ __forceinline__ uint64_t fixed38(float p) {
    uint32_t hi, lo;
    digits38(p, hi, lo);
    return ((uint64_t)(hi - kBias) << 19) + (lo - kBias);
}
// a uniform number in [0, 1) in steps of 2^-24 (out-of-range and NaN clamped)
__device__ __forceinline__ uint32_t tick24(float u) {
    const float t = fminf(fmaxf(u, 0.f) * 16777216.f, 16777215.f);
    return __float2uint_rz(t);
}

// 16 bytes of probabilities as floats
template <typename Tin> struct Row;
template <> struct Row<float> {
    static constexpr int VEC = 4;
    static __device__ __forceinline__ void load(const float *p, float (&x)[VEC]) {
        const float4 f = __ldg(reinterpret_cast<const float4 *>(p));
        x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
    }
};
template <> struct Row<__nv_bfloat16> {
    static constexpr int VEC = 8;
    static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&x)[VEC]) {
        Elem<__nv_bfloat16>::load8(p, x);
    }
};

constexpr int kVerifyThreads = 256, kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 8;      // CTAs of a sequence
constexpr int kVerifyCtas = 4;      // resident on an SM

// One cluster per sequence.  Every CTA gathers the drafted tokens'
// probabilities and its first warp walks the tree (each step tests one child,
// in index order); the walk is short, so all CTAs make it.  Then each sums its
// share of the last node's row, the totals cross the cluster, and the warp
// whose sums hold the drawn mass finds the token.  The rows' bytes bound it: a
// row is read once, and the one warp's share a second time, from the L2.
// Measured: 256 chains over 131,072 tokens, fp32 with draft probabilities (235
// MB), 52 us, 4.5 TB/s; bf16 43 us; 256 trees without, fp32 44 us (134 MB), bf16 35.
// What is left above the bytes are the prologue's three dependent loads, the
// cluster's meeting and the second pass, and that the CTAs make 1.7 rounds.
template <typename Tin>
__global__ void __launch_bounds__(kVerifyThreads, kVerifyCtas)
verify_kernel(const Tin *__restrict__ target, const Tin *__restrict__ draft,
              const int32_t *__restrict__ tokens, const int32_t *__restrict__ parent,
              const float *__restrict__ uniforms, int32_t M, int32_t V, int32_t *__restrict__ accept,
              int32_t *__restrict__ path, int32_t *__restrict__ next_token) {
    constexpr int VEC = Row<Tin>::VEC, BATCH = 16 / VEC;   // BATCH loads of 16 bytes on their way per lane and row
    typedef unsigned long long u64;
    __shared__ int32_t gone[kMaxTreeNodes];            // the last node's refused children's tokens, each once
    __shared__ int32_t walk_cur, walk_gone, walk_any;
    __shared__ uint32_t walk_draw;
    __shared__ u64 part[kVerifyWarps];
    __shared__ u64 totals[2][kMaxCluster];             // of both attempts
    // a CTA's shared memory may be written once it runs: the walk hides the wait for that
    cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    cluster.barrier_arrive();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t n = blockIdx.x / ranks;

    if (warp == 0) {
        // lane holds nodes lane and lane + 32
        int par[2], tok[2];
        float px[2], qx[2], un[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int m = lane + 32 * y;
            par[y] = m < M ? parent[n * M + m] : -2;
            tok[y] = m < M ? tokens[n * M + m] : -1;
            un[y] = m < M ? uniforms[n * (M + 1) + m] : 0.f;
        }
        const float u_draw = uniforms[n * (M + 1) + M];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const bool good = par[y] >= 0 && par[y] < lane + 32 * y && tok[y] >= 0 && tok[y] < V;
            const int64_t at = (n * M + par[y]) * V + tok[y];
            px[y] = good ? Elem<Tin>::load(target + at) : 0.f;
            qx[y] = good && draft != nullptr ? Elem<Tin>::load(draft + at) : 0.f;
            if (par[y] >= lane + 32 * y) par[y] = -2;
        }
        auto of = [&](const float (&x)[2], int m) {
            const float a = __shfl_sync(0xffffffffu, x[0], m & 31), b = __shfl_sync(0xffffffffu, x[1], m & 31);
            return m < 32 ? a : b;
        };
        int cur = __shfl_sync(0xffffffffu, par[0], 0) == -1 ? 0 : -1, cnt = 0, ng = 0, any = 0;
        while (cur >= 0) {
            if (rank == 0 && lane == 0) path[n * M + cnt] = cur;
            ++cnt;
            const float u = of(un, cur);
            const u64 tick = (u64)tick24(u) << 14;
            u64 kids = __ballot_sync(0xffffffffu, par[0] == cur) | (u64)__ballot_sync(0xffffffffu, par[1] == cur) << 32;
            u64 spent = 0;
            int into = -1;
            ng = any = 0;
            while (kids != 0) {
                const int m = __ffsll((long long)kids) - 1;
                kids &= kids - 1;
                const int t0 = __shfl_sync(0xffffffffu, tok[0], m & 31), t1 = __shfl_sync(0xffffffffu, tok[1], m & 31);
                const int t = m < 32 ? t0 : t1;
                const bool good = t >= 0 && t < V;
                const float p = of(px, m);
                // was this token refused before, as an elder sibling's?
                bool twice = false;
                for (int i = lane; i < ng; i += 32) twice |= gone[i] == t;
                twice = __any_sync(0xffffffffu, twice);
                bool take;
                u64 mass = 0;
                if (draft != nullptr) {
                    // the first child alone was sampled from the whole draft distribution
                    take = good && any == 0 && u * of(qx, m) < p;
                } else {
                    mass = good && !twice ? fixed38(p) : 0;
                    take = tick < spent + mass;
                }
                if (take) {
                    into = m;
                    break;
                }
                spent += mass;
                any = 1;
                if (good && !twice) {
                    if (lane == 0) gone[ng] = t;
                    ++ng;
                    __syncwarp();
                }
            }
            if (into < 0) break;
            cur = into;
        }
        if (rank == 0) {
            for (int m = cnt + lane; m < M; m += 32) path[n * M + m] = -1;
            if (lane == 0) accept[n] = cnt;
        }
        if (lane == 0) {
            walk_cur = cur;
            walk_gone = ng;
            walk_any = any;
            walk_draw = tick24(u_draw);
        }
    }
    __syncthreads();
    const int cur = walk_cur, refused = walk_gone;
    if (cur < 0) {                                     // the whole cluster
        cluster.barrier_wait();
        if (rank == 0 && tid == 0) next_token[n] = -1;
        return;
    }
    const Tin *row = target + (n * M + cur) * V;
    const Tin *qrow = draft != nullptr && walk_any ? draft + (n * M + cur) * V : nullptr;
    bool skip = draft == nullptr && refused > 0;       // leave the refused tokens out
    // vectors from the 16-byte boundary at or below the row's start: element
    // i of the row is element i + lead of that grid
    const int lead = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(Tin));
    const int vecs = (V + lead + VEC - 1) / VEC;
    const int per_warp = (vecs + ranks * kVerifyWarps - 1) / (ranks * kVerifyWarps);
    const int first = min(vecs, (rank * kVerifyWarps + warp) * per_warp), end = min(vecs, first + per_warp);
    // the raw values of vector i of the grid (zero outside the row)
    auto fetch = [&](const Tin *r, int i, float (&x)[VEC]) {
        const int e0 = i * VEC - lead;
        if (e0 >= 0 && e0 + VEC <= V) {
            Row<Tin>::load(r + e0, x);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[e] = e0 + e >= 0 && e0 + e < V ? Elem<Tin>::load(r + e0 + e) : 0.f;
        }
    };
    // What is drawn from, at BATCH vectors of a lane, 32 apart.  Only the batches at the
    // row's and the share's ends look at each vector: a branch per vector kept the
    // loads from being on their way together.
    auto weights = [&](int i0, float (&x)[BATCH][VEC]) {
        if (i0 * VEC >= lead && i0 + 32 * BATCH <= end && (i0 + 32 * BATCH) * VEC - lead <= V) {
            const int e0 = (i0 + lane) * VEC - lead;
#pragma unroll
            for (int y = 0; y < BATCH; ++y) Row<Tin>::load(row + e0 + 32 * VEC * y, x[y]);
            if (qrow != nullptr) {
                float z[BATCH][VEC];
#pragma unroll
                for (int y = 0; y < BATCH; ++y) Row<Tin>::load(qrow + e0 + 32 * VEC * y, z[y]);
#pragma unroll
                for (int y = 0; y < BATCH; ++y)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) x[y][e] = x[y][e] - z[y][e];
            }
            return;
        }
#pragma unroll
        for (int y = 0; y < BATCH; ++y) {
            const int i = i0 + 32 * y + lane;
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[y][e] = 0.f;
            if (i < end) {
                fetch(row, i, x[y]);
                if (qrow != nullptr) {
                    float z[VEC];
                    fetch(qrow, i, z);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) x[y][e] = x[y][e] - z[e];
                }
            }
        }
    };
    u64 all = 0, before = 0;                           // the row's mass, and that of the CTAs before this one
    for (int attempt = 0;; ++attempt) {
        u64 sum = 0;
        for (int i0 = first; i0 < end; i0 += 32 * BATCH) {
            float x[BATCH][VEC];
            uint32_t hi = 0, lo = 0;
            weights(i0, x);
#pragma unroll
            for (int y = 0; y < BATCH; ++y)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    uint32_t h, l;
                    digits38(x[y][e], h, l);
                    hi += h - kBias;
                    lo += l - kBias;
                }
            sum += ((u64)hi << 19) + lo;               // 16 digits of 19 bits fit 32 bits
        }
        if (skip) {
            // the refused tokens come out of the sums that hold them
            for (int i = lane; i < refused; i += 32) {
                const int at = (gone[i] + lead) / VEC;
                if (at >= first && at < end) sum -= fixed38(Elem<Tin>::load(row + gone[i]));
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) part[warp] = sum;
        if (attempt == 0) cluster.barrier_wait();      // every CTA has started
        __syncthreads();
        if (warp == 0) {
            u64 mine = lane < kVerifyWarps ? part[lane] : 0;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
            if (lane < ranks) *cluster.map_shared_rank(&totals[attempt][rank], lane) = mine;
        }
        cluster.sync();
        all = before = 0;
        for (int r = 0; r < ranks; ++r) {
            const u64 x = totals[attempt][r];
            before += r < rank ? x : 0;
            all += x;
        }
        if (all != 0 || attempt > 0 || (qrow == nullptr && !skip)) break;
        // nothing is left beside what was refused: draw from the row itself
        qrow = nullptr;
        skip = false;
    }
    if (all == 0) {
        if (rank == 0 && tid == 0) next_token[n] = -1;
        return;
    }
    // the first token whose running sum exceeds floor(u all / 2^24): the sum
    // of all exceeds it, since u < 2^24
    const u64 need = __umul64hi((u64)walk_draw << 40, all);
    for (int w = 0; w < warp; ++w) before += part[w];
    if (before > need || before + part[warp] <= need) return;
    for (int i0 = first; i0 < end; i0 += 32 * BATCH) {
        float x[BATCH][VEC];
        weights(i0, x);
#pragma unroll
        for (int y = 0; y < BATCH; ++y) {
            const int e0 = (i0 + 32 * y + lane) * VEC - lead;
            u64 w[VEC], sum = 0;
#pragma unroll
            for (int e = 0; e < VEC; ++e) w[e] = fixed38(x[y][e]);
            if (skip) {
                for (int r = 0; r < refused; ++r)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) w[e] = gone[r] == e0 + e ? 0 : w[e];
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum += w[e];
            u64 run = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 z = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += z;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, before + run > need);
            if (hit != 0) {
                if (lane == __ffs(hit) - 1) {
                    u64 at = before + run - sum;
                    int e = 0;
#pragma unroll
                    for (int z = 0; z < VEC; ++z) {
                        at += w[z];
                        if (at <= need) e = z + 1;
                    }
                    next_token[n] = e0 + e;
                }
                return;
            }
            before += __shfl_sync(0xffffffffu, run, 31);
        }
    }
}

template <typename Tin>
cudaError_t run_verify(const void *target, const void *draft, const int32_t *tokens, const int32_t *parent,
                       const float *uniforms, int32_t N, int32_t M, int32_t V, int32_t *accept, int32_t *path,
                       int32_t *next_token, cudaStream_t stream) {
    // CTAs per sequence: up to eight, while all sequences' CTAs make no more than two
    // rounds of the GPU (256 chains: 62 us with two, 52 with four, 53 with eight; 600
    // of 65,536 tokens with draft probabilities: 79 with one, 71 with two) and each
    // still has 4 KB.
    const int64_t two_rounds = 2 * kVerifyCtas * (int64_t)sm_count();
    int ranks = kMaxCluster;
    while (ranks > 1 && (ranks * (int64_t)N > two_rounds || (int64_t)V * (int64_t)sizeof(Tin) < (int64_t)ranks * 4096)) ranks /= 2;
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = ranks;
    cluster.val.clusterDim.y = 1;
    cluster.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)N * ranks);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = stream;
    cfg.attrs = &cluster;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_kernel<Tin>, static_cast<const Tin *>(target),
                                             static_cast<const Tin *>(draft), tokens, parent, uniforms, M, V, accept,
                                             path, next_token);
    if (e == cudaSuccess) count_launches(1);
    else (void)cudaGetLastError();                     // reported here
    return e;
}

constexpr int kAppendTokens = 4;

// A thread moves 16 bytes: token t of the accepted ones, head h, piece x.  One
// read and one write of each byte: eight prompts of 2,048 to 4,096 tokens, 8
// heads of 128 (201 MB moved), 31 us, 6.5 TB/s (35 us with the index arithmetic
// in 64 bits).
__global__ void __launch_bounds__(256)
append_kernel(const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new,
              const int32_t *__restrict__ path, const int32_t *__restrict__ accept,
              const int32_t *__restrict__ page_table, const int32_t *__restrict__ cache_lens, int32_t M,
              int32_t P, int32_t H, int32_t piece_bits, int32_t num_pages, int32_t page_size,
              int32_t max_pages, uint4 *__restrict__ k_cache, uint4 *__restrict__ v_cache,
              int32_t *__restrict__ lens_out) {
    const int64_t n = blockIdx.y;
    int acc = accept != nullptr ? accept[n] : P;
    acc = acc < 0 ? 0 : (acc > P ? P : acc);
    const int len = cache_lens[n];
    if (blockIdx.x == 0 && threadIdx.x == 0 && lens_out != nullptr) {
        // (a length below zero stays one, so that the next attention reports it)
        lens_out[n] = len < 0 ? min(len + acc, -1) : len + acc;
    }
    if (len < 0) return;
    // kAppendTokens tokens per block and pass, so that the index arithmetic stays in 32 bits
    const uint32_t per_token = (uint32_t)H << piece_bits;
    for (int64_t t0 = (int64_t)blockIdx.x * kAppendTokens; t0 < acc; t0 += (int64_t)gridDim.x * kAppendTokens) {
        const uint32_t items = (uint32_t)min((int64_t)kAppendTokens, acc - t0) * per_token;
#pragma unroll 2
        for (uint32_t i = threadIdx.x; i < items; i += 256) {
            const uint32_t dt = i / per_token, r = i - dt * per_token;
            const uint32_t h = r >> piece_bits, x = r & ((1u << piece_bits) - 1);
            const int t = (int)t0 + (int)dt;
            const int src = path != nullptr ? path[n * P + t] : t;
            if (src < 0 || src >= M) continue;
            const uint32_t pos = (uint32_t)len + (uint32_t)t, slot = pos / (uint32_t)page_size;
            if (slot >= (uint32_t)max_pages) continue;
            const int page = page_table[n * max_pages + slot];
            if (page < 0 || page >= num_pages) continue;
            const int64_t from = (((n * M + src) * H + h) << piece_bits) + x;
            const int64_t to = ((((int64_t)page * H + h) * page_size + (pos - slot * page_size)) << piece_bits) + x;
            k_cache[to] = __ldg(k_new + from);
            v_cache[to] = __ldg(v_new + from);
        }
    }
}

}  // namespace

cudaError_t launch_verify_drafts(const void *target, const void *draft, const int32_t *tokens,
                                 const int32_t *parent, const float *uniforms, int32_t N, int32_t M,
                                 int32_t V, kda_dtype dt, int32_t *accept, int32_t *path,
                                 int32_t *next_token, cudaStream_t stream) {
    if (dt == KDA_BF16)
        return run_verify<__nv_bfloat16>(target, draft, tokens, parent, uniforms, N, M, V, accept, path, next_token,
                                         stream);
    return run_verify<float>(target, draft, tokens, parent, uniforms, N, M, V, accept, path, next_token, stream);
}

cudaError_t launch_cache_append(const void *k_new, const void *v_new, const int32_t *path,
                                const int32_t *accept, const int32_t *page_table,
                                const int32_t *cache_lens, int32_t N, int32_t M, int32_t P, int32_t H,
                                int32_t D, int32_t num_pages, int32_t page_size, int32_t max_pages,
                                kda_dtype dt, void *k_cache, void *v_cache, int32_t *lens_out,
                                cudaStream_t stream) {
    int32_t piece_bits = 1;                            // 16-byte pieces of a row: 2 to 32
    while ((16 << piece_bits) < D * (dt == KDA_BF16 ? 2 : 4)) ++piece_bits;
    int64_t blocks = ((int64_t)P + kAppendTokens - 1) / kAppendTokens;
    if (blocks > 4096) blocks = 4096;
    append_kernel<<<dim3((unsigned)blocks, (unsigned)N), 256, 0, stream>>>(
        static_cast<const uint4 *>(k_new), static_cast<const uint4 *>(v_new), path, accept, page_table,
        cache_lens, M, P, H, piece_bits, num_pages, page_size, max_pages, static_cast<uint4 *>(k_cache),
        static_cast<uint4 *>(v_cache), lens_out);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace kda
