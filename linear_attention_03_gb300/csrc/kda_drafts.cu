// kda_drafts.cu -- acceptance of drafted tokens against the target's
// probabilities (kda_verify_drafts) and the accepted tokens' keys and values
// into a paged cache (kda_cache_append).  "From GPT-2 to Kimi K3, from first
// principles", Chapter 14 (speculative decoding: the target verifies a
// draft's tokens, accepted updates are committed).
//
// Probabilities are compared and summed in fixed point (whole multiples of
// 2^-38, held in 64 bits), so that the drawn token does not depend on the
// order of the sums: any split of the vocabulary gives the same one.  A
// probability of 2^-38 and below counts as zero; 2^18 tokens of rounding
// shift the distribution by at most 2^-20.
#include "kda_internal.cuh"
#include "kda_tree.cuh"

namespace kda {
namespace {

__device__ __forceinline__ uint64_t fixed38(float p) {
    // fmaxf drops a NaN; the scaling is exact, the conversion rounds toward zero
    return __float2ull_rz(fminf(fmaxf(p, 0.f), 1.f) * 274877906944.f);
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

struct Walk {
    int32_t cur;        // the last accepted node (-1: the sequence is not in use)
    int32_t refused;    // how many of its children were refused
};

constexpr int kVerifyThreads = 1024;

// One CTA per sequence.  The drafted tokens' probabilities are gathered first,
// then one thread walks the tree (a child's index exceeds its parent's and the
// refused siblings' order is the index order, so one ascending pass visits
// every step), then all warps sum the last node's row and one warp finds the
// token.
template <typename Tin>
__global__ void __launch_bounds__(kVerifyThreads)
verify_kernel(const Tin *__restrict__ target, const Tin *__restrict__ draft,
              const int32_t *__restrict__ tokens, const int32_t *__restrict__ parent,
              const float *__restrict__ uniforms, int32_t M, int32_t V, int32_t *__restrict__ accept,
              int32_t *__restrict__ path, int32_t *__restrict__ next_token) {
    constexpr int VEC = Row<Tin>::VEC, WARPS = kVerifyThreads / 32;
    __shared__ float px[kMaxTreeNodes], qx[kMaxTreeNodes];
    __shared__ int32_t tok[kMaxTreeNodes], par[kMaxTreeNodes], gone[kMaxTreeNodes], step[kMaxTreeNodes];
    __shared__ Walk walk;
    __shared__ int32_t count;
    __shared__ unsigned long long part[WARPS];
    __shared__ unsigned long long whole;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t n = blockIdx.x;

    if (tid < M) {
        const int p = parent[n * M + tid], t = tokens[n * M + tid];
        par[tid] = p;
        tok[tid] = t;
        float a = 0.f, b = 0.f;
        if (p >= 0 && p < tid && t >= 0 && t < V) {
            a = Elem<Tin>::load(target + (n * M + p) * V + t);
            if (draft != nullptr) b = Elem<Tin>::load(draft + (n * M + p) * V + t);
        }
        px[tid] = a;
        qx[tid] = b;
    }
    __syncthreads();
    if (tid == 0) {
        int cur = par[0] == -1 ? 0 : -1, refused = 0, cnt = cur == 0 ? 1 : 0;
        if (cur == 0) step[0] = 0;
        unsigned long long spent = 0;
        for (int m = 1; m < M && cur >= 0; ++m) {
            if (par[m] != cur) continue;
            const int t = tok[m];
            const bool good = t >= 0 && t < V;
            bool take;
            unsigned long long mass = 0;
            if (draft != nullptr) {
                // the first child alone was sampled from the whole draft distribution
                take = good && refused == 0 && uniforms[n * (M + 1) + cur] * qx[m] < px[m];
            } else {
                bool twice = false;
                for (int i = 0; i < refused; ++i) twice |= gone[i] == t;
                mass = good && !twice ? fixed38(px[m]) : 0;
                take = ((unsigned long long)tick24(uniforms[n * (M + 1) + cur]) << 14) < spent + mass;
            }
            if (take) {
                cur = m;
                step[cnt++] = m;
                refused = 0;
                spent = 0;
            } else {
                gone[refused++] = t;
                spent += mass;
            }
        }
        walk.cur = cur;
        walk.refused = refused;
        count = cnt;
        accept[n] = cnt;
    }
    __syncthreads();
    if (tid < M) path[n * M + tid] = tid < count ? step[tid] : -1;
    const int cur = walk.cur, refused = walk.refused;
    if (cur < 0) {
        if (tid == 0) next_token[n] = -1;
        return;
    }
    const Tin *row = target + (n * M + cur) * V;
    const Tin *qrow = draft != nullptr && refused > 0 ? draft + (n * M + cur) * V : nullptr;
    bool skip = draft == nullptr && refused > 0;       // leave the refused tokens out
    // vectors from the 16-byte boundary at or below the row's start: element
    // i of the row is element i + lead of that grid
    const int lead = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(Tin));
    const int vecs = (V + lead + VEC - 1) / VEC;
    const int per_warp = (vecs + WARPS - 1) / WARPS;
    // weights of vector i of the grid (zero outside the row)
    auto weights = [&](int i, unsigned long long (&w)[VEC]) {
        const int e0 = i * VEC - lead;
        float x[VEC];
        if (e0 >= 0 && e0 + VEC <= V) {
            Row<Tin>::load(row + e0, x);
            if (qrow != nullptr) {
                float y[VEC];
                Row<Tin>::load(qrow + e0, y);
#pragma unroll
                for (int e = 0; e < VEC; ++e) x[e] = x[e] - y[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int at = e0 + e;
                x[e] = at >= 0 && at < V ? Elem<Tin>::load(row + at) : 0.f;
                if (qrow != nullptr && at >= 0 && at < V) x[e] = x[e] - Elem<Tin>::load(qrow + at);
            }
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] = fixed38(x[e]);
    };
    for (int attempt = 0;; ++attempt) {
        unsigned long long sum = 0;
        const int end = min(vecs, (warp + 1) * per_warp);
        for (int i = warp * per_warp + lane; i < end; i += 32) {
            unsigned long long w[VEC];
            weights(i, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum += w[e];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) part[warp] = sum;
        __syncthreads();
        if (tid == 0) {
            // the refused tokens (each once) come out of the sums that hold them
            if (skip)
                for (int i = 0; i < refused; ++i) {
                    bool again = gone[i] < 0 || gone[i] >= V;
                    for (int j = 0; j < i; ++j) again |= gone[j] == gone[i];
                    if (!again)
                        part[(gone[i] + lead) / VEC / per_warp] -= fixed38(Elem<Tin>::load(row + gone[i]));
                }
            unsigned long long all = 0;
            for (int w = 0; w < WARPS; ++w) all += part[w];
            whole = all;
        }
        __syncthreads();
        if (whole != 0 || attempt > 0 || (qrow == nullptr && !skip)) break;
        // nothing is left beside what was refused: draw from the row itself
        qrow = nullptr;
        skip = false;
        __syncthreads();
    }
    const unsigned long long all = whole;
    if (all == 0) {
        if (tid == 0) next_token[n] = -1;
        return;
    }
    // the first token whose running sum exceeds floor(u all / 2^24): the sum
    // of all exceeds it, since u < 2^24
    const unsigned long long need =
        __umul64hi((unsigned long long)tick24(uniforms[n * (M + 1) + M]) << 40, all);
    unsigned long long before = 0;
    int mine = 0;
    for (; mine < WARPS - 1; ++mine) {
        if (before + part[mine] > need) break;
        before += part[mine];
    }
    if (warp != mine) return;
    const int end = min(vecs, (warp + 1) * per_warp);
    for (int i0 = warp * per_warp; i0 < end; i0 += 32) {
        unsigned long long w[VEC], sum = 0;
        const int i = i0 + lane;
        if (i < end) {
            weights(i, w);
            if (skip) {
                const int e0 = i * VEC - lead;
                for (int r = 0; r < refused; ++r)
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        if (gone[r] == e0 + e) w[e] = 0;
            }
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) w[e] = 0;
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum += w[e];
        unsigned long long run = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long x = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + run > need);
        if (hit != 0) {
            if (lane == __ffs(hit) - 1) {
                unsigned long long at = before + run - sum;
                int e = 0;
#pragma unroll
                for (int x = 0; x < VEC; ++x) {
                    at += w[x];
                    if (at <= need) e = x + 1;
                }
                next_token[n] = i * VEC - lead + e;
            }
            return;
        }
        before += __shfl_sync(0xffffffffu, run, 31);
    }
}

// A thread moves 16 bytes: token t of the accepted ones, head h, piece x.
__global__ void __launch_bounds__(256)
append_kernel(const uint4 *__restrict__ k_new, const uint4 *__restrict__ v_new,
              const int32_t *__restrict__ path, const int32_t *__restrict__ accept,
              const int32_t *__restrict__ page_table, const int32_t *__restrict__ cache_lens, int32_t M,
              int32_t P, int32_t H, int32_t pieces, int32_t num_pages, int32_t page_size,
              int32_t max_pages, uint4 *__restrict__ k_cache, uint4 *__restrict__ v_cache,
              int32_t *__restrict__ lens_out) {
    const int64_t n = blockIdx.y;
    int acc = accept != nullptr ? accept[n] : P;
    acc = acc < 0 ? 0 : (acc > P ? P : acc);
    const int len = max(cache_lens[n], 0);
    if (blockIdx.x == 0 && threadIdx.x == 0 && lens_out != nullptr) lens_out[n] = len + acc;
    const int per_token = H * pieces;
    const int64_t total = (int64_t)acc * per_token;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int t = (int)(i / per_token), r = (int)(i % per_token);
        const int h = r / pieces, x = r % pieces;
        const int src = path != nullptr ? path[n * P + t] : t;
        if (src < 0 || src >= M) continue;
        const int64_t pos = (int64_t)len + t;
        const int64_t slot = pos / page_size;
        if (slot >= max_pages) continue;
        const int page = page_table[n * max_pages + slot];
        if (page < 0 || page >= num_pages) continue;
        const int64_t from = ((n * M + src) * H + h) * pieces + x;
        const int64_t to = (((int64_t)page * H + h) * page_size + pos % page_size) * pieces + x;
        k_cache[to] = __ldg(k_new + from);
        v_cache[to] = __ldg(v_new + from);
    }
}

}  // namespace

cudaError_t launch_verify_drafts(const void *target, const void *draft, const int32_t *tokens,
                                 const int32_t *parent, const float *uniforms, int32_t N, int32_t M,
                                 int32_t V, kda_dtype dt, int32_t *accept, int32_t *path,
                                 int32_t *next_token, cudaStream_t stream) {
    if (dt == KDA_BF16)
        verify_kernel<__nv_bfloat16><<<N, kVerifyThreads, 0, stream>>>(
            static_cast<const __nv_bfloat16 *>(target), static_cast<const __nv_bfloat16 *>(draft), tokens,
            parent, uniforms, M, V, accept, path, next_token);
    else
        verify_kernel<float><<<N, kVerifyThreads, 0, stream>>>(
            static_cast<const float *>(target), static_cast<const float *>(draft), tokens, parent,
            uniforms, M, V, accept, path, next_token);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_cache_append(const void *k_new, const void *v_new, const int32_t *path,
                                const int32_t *accept, const int32_t *page_table,
                                const int32_t *cache_lens, int32_t N, int32_t M, int32_t P, int32_t H,
                                int32_t D, int32_t num_pages, int32_t page_size, int32_t max_pages,
                                kda_dtype dt, void *k_cache, void *v_cache, int32_t *lens_out,
                                cudaStream_t stream) {
    const int32_t pieces = D * (dt == KDA_BF16 ? 2 : 4) / 16;
    const int64_t work = (int64_t)P * H * pieces;
    int64_t blocks = (work + 255) / 256;
    if (blocks < 1) blocks = 1;
    if (blocks > 4096) blocks = 4096;
    append_kernel<<<dim3((unsigned)blocks, (unsigned)N), 256, 0, stream>>>(
        static_cast<const uint4 *>(k_new), static_cast<const uint4 *>(v_new), path, accept, page_table,
        cache_lens, M, P, H, pieces, num_pages, page_size, max_pages, static_cast<uint4 *>(k_cache),
        static_cast<uint4 *>(v_cache), lens_out);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace kda
