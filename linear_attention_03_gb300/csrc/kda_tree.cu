// kda_tree.cu -- the KDA recurrence over a tree of drafted tokens
// (kda_decode_tree) and the state after its accepted path
// (kda_decode_commit).  "From GPT-2 to Kimi K3, from first principles",
// Chapter 14: drafts run from a read-only state, and the accepted updates are
// replayed.
//
// With the recurrence S_m = (I - beta_m k_m k_m^T) Diag(a_m) S_p + beta_m k_m v_m^T
// (p = parent of m, a = exp(g)), write S_m = Diag(E_m) S_0 + sum_j Diag(D_mj) k_j u_j^T
// over the nodes j on m's line, where D_mj is the product of a over the nodes
// below j down to m and E_m the product over the whole line.  Then
//     u_m = beta_m (v_m - S_0^T (E_m k_m) - sum_{j above m} ((D_mj k_m) . k_j) u_j)
//     o_m = S_0^T (E_m q_m) + sum_{j on m's line} ((D_mj q_m) . k_j) u_j
// so one read of S_0 serves all nodes, and no node's state is ever formed.
// Every product of decays is taken by walking up the line (factors <= 1), so
// deep trees underflow to zero and never overflow.
#include "kda_internal.cuh"
#include "kda_tree.cuh"

namespace kda {
namespace {

constexpr int kNodeBlock = 8;   // nodes whose products share one pass over S_0

template <int D> struct TreeCfg {
    static constexpr int THREADS = D < 32 ? 32 : D;   // a thread per state column
    static size_t smem(int M) {
        const size_t rows = (size_t)((M + kNodeBlock - 1) / kNodeBlock) * kNodeBlock;
        return rows * D * 4 * 5 + (size_t)M * M * 8 + (size_t)M * 16;
    }
};

// One CTA per (sequence, head): fp32 arithmetic throughout.  The line products
// first (a warp per node, lanes over channels), then per block of eight nodes
// one pass over S_0 (thread c reads column c) and the solve, whose columns are
// independent.
template <typename Tin, int D>
__global__ void __launch_bounds__(TreeCfg<D>::THREADS)
decode_tree_kernel(const Tin *__restrict__ q, const Tin *__restrict__ k, const Tin *__restrict__ v,
                   const float *__restrict__ g, const float *__restrict__ beta,
                   const float *__restrict__ state, const int32_t *__restrict__ parent, int32_t M,
                   int32_t H, Tin *__restrict__ out) {
    constexpr int THREADS = TreeCfg<D>::THREADS;
    constexpr int EPL = D < 32 ? 1 : D / 32;          // channels per lane of a warp
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const int rows = (M + kNodeBlock - 1) / kNodeBlock * kNodeBlock;
    float *kE = reinterpret_cast<float *>(smem_raw);  // E_m k_m
    float *qE = kE + rows * D;                        // E_m q_m
    float *kk = qE + rows * D;
    float *al = kk + rows * D;
    float *U = al + rows * D;
    float2 *AB = reinterpret_cast<float2 *>(U + rows * D);   // ((D_mj k_m).k_j, (D_mj q_m).k_j)
    uint64_t *line = reinterpret_cast<uint64_t *>(AB + M * M);
    int32_t *par = reinterpret_cast<int32_t *>(line + M);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t n = blockIdx.x / H;
    const int h = blockIdx.x % H;

    for (int m = tid; m < M; m += THREADS) par[m] = parent[n * M + m];
    for (int i = tid; i < rows * D; i += THREADS) {
        const int m = i / D, c = i % D;
        const int64_t at = ((n * M + m) * H + h) * D + c;
        kk[i] = m < M ? Elem<Tin>::load(k + at) : 0.f;
        al[i] = m < M ? __expf(g[at]) : 0.f;
        kE[i] = qE[i] = 0.f;
    }
    __syncthreads();
    for (int m = tid; m < M; m += THREADS) line[m] = tree_line(par, m);
    __syncthreads();
    for (int m = warp; m < M; m += THREADS / 32) {
        if (line[m] == 0) continue;
        float kd[EPL], qd[EPL];
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            const int c = lane + 32 * e;
            kd[e] = c < D ? kk[m * D + c] : 0.f;
            qd[e] = c < D ? Elem<Tin>::load(q + ((n * M + m) * H + h) * D + c) : 0.f;
        }
        for (int j = m; j >= 0; j = par[j]) {
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int e = 0; e < EPL; ++e) {
                const int c = lane + 32 * e;
                const float kj = c < D ? kk[j * D + c] : 0.f, aj = c < D ? al[j * D + c] : 0.f;
                a += kd[e] * kj;
                b += qd[e] * kj;
                kd[e] *= aj;
                qd[e] *= aj;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                a += __shfl_xor_sync(0xffffffffu, a, o);
                b += __shfl_xor_sync(0xffffffffu, b, o);
            }
            if (lane == 0) AB[m * M + j] = make_float2(a, b);
        }
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            const int c = lane + 32 * e;
            if (c < D) {
                kE[m * D + c] = kd[e];
                qE[m * D + c] = qd[e];
            }
        }
    }
    __syncthreads();
    if (tid >= D) return;
    const int c = tid;
    const float *S = state + (size_t)blockIdx.x * D * D + c;
    for (int m0 = 0; m0 < M; m0 += kNodeBlock) {
        float xk[kNodeBlock], xq[kNodeBlock];
#pragma unroll
        for (int b = 0; b < kNodeBlock; ++b) xk[b] = xq[b] = 0.f;
#pragma unroll 2
        for (int i = 0; i < D; i += 4) {
            float s[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = __ldg(S + (size_t)(i + e) * D);
#pragma unroll
            for (int b = 0; b < kNodeBlock; ++b) {
                const float4 ke = *reinterpret_cast<const float4 *>(kE + (m0 + b) * D + i);
                const float4 qe = *reinterpret_cast<const float4 *>(qE + (m0 + b) * D + i);
                xk[b] += ke.x * s[0] + ke.y * s[1] + ke.z * s[2] + ke.w * s[3];
                xq[b] += qe.x * s[0] + qe.y * s[1] + qe.z * s[2] + qe.w * s[3];
            }
        }
#pragma unroll
        for (int b = 0; b < kNodeBlock; ++b) {
            const int m = m0 + b;
            if (m >= M) break;
            const int64_t row = (n * M + m) * H + h;
            uint64_t up = line[m];
            if (up == 0) {
                Elem<Tin>::store(out + row * D + c, 0.f);
                continue;
            }
            float x = xk[b], o = xq[b];
            up &= ~(uint64_t{1} << m);
            while (up != 0) {
                const int j = __ffsll((long long)up) - 1;
                up &= up - 1;
                const float2 ab = AB[m * M + j];
                const float uj = U[j * D + c];
                x += ab.x * uj;
                o += ab.y * uj;
            }
            const float u = beta[row] * (Elem<Tin>::load(v + row * D + c) - x);
            U[m * D + c] = u;
            Elem<Tin>::store(out + row * D + c, o + AB[m * M + m].y * u);
        }
    }
}

// The state after the first accept[n] nodes of path[n]: a thread keeps one
// state column in registers, and the column's read S^T k, the decay and the
// write stay in that thread, so the state moves once in each direction and a
// token costs no exchange between threads.
template <typename Tin, int D>
__global__ void __launch_bounds__(D < 32 ? 32 : D)
decode_commit_kernel(const Tin *__restrict__ k, const Tin *__restrict__ v, const float *__restrict__ g,
                     const float *__restrict__ beta, const float *state_in,
                     const int32_t *__restrict__ path, const int32_t *__restrict__ accept, int32_t M,
                     int32_t P, int32_t H, float *state_out) {
    constexpr int BATCH = 4;                         // path nodes staged at a time
    __shared__ __align__(16) float2 ak[BATCH][D];   // (decay, k) per channel
    __shared__ int32_t node[BATCH];
    const int tid = threadIdx.x;
    const int64_t n = blockIdx.x / H;
    const int h = blockIdx.x % H;
    const int c = tid < D ? tid : 0;
    const size_t base = (size_t)blockIdx.x * D * D + c;
    float s[D];
#pragma unroll
    for (int i = 0; i < D; ++i) s[i] = __ldcs(state_in + base + (size_t)i * D);
    int acc = accept[n];
    acc = acc < 0 ? 0 : (acc > P ? P : acc);
    bool open = true;                                // no entry outside the tree so far
    for (int t0 = 0; t0 < acc && open; t0 += BATCH) {
        const int cnt = acc - t0 < BATCH ? acc - t0 : BATCH;
        __syncthreads();
        if (tid < cnt) node[tid] = path[n * P + t0 + tid];
        __syncthreads();
        for (int t = 0; t < cnt; ++t) {
            const int m = node[t];
            if (m < 0 || m >= M) break;
            if (tid < D) {
                const int64_t at = ((n * M + m) * H + h) * D + tid;
                ak[t][tid] = make_float2(__expf(g[at]), Elem<Tin>::load(k + at));
            }
        }
        __syncthreads();
        for (int t = 0; t < cnt; ++t) {
            const int m = node[t];
            if (m < 0 || m >= M) {
                open = false;
                break;
            }
            const int64_t row = (n * M + m) * H + h;
            const float vt = Elem<Tin>::load(v + row * D + c), bt = beta[row];
            float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < D; i += 2) {
                const float4 f = *reinterpret_cast<const float4 *>(&ak[t][i]);
                s[i] *= f.x;
                s[i + 1] *= f.z;
                x[i & 3] += f.y * s[i];
                x[(i + 1) & 3] += f.w * s[i + 1];
            }
            const float u = bt * (vt - ((x[0] + x[1]) + (x[2] + x[3])));
#pragma unroll
            for (int i = 0; i < D; i += 2) {
                const float4 f = *reinterpret_cast<const float4 *>(&ak[t][i]);
                s[i] += f.y * u;
                s[i + 1] += f.w * u;
            }
        }
    }
    if (tid < D) {
#pragma unroll
        for (int i = 0; i < D; ++i) __stcs(state_out + base + (size_t)i * D, s[i]);
    }
}

template <typename Tin, int D>
cudaError_t run_tree(const void *q, const void *k, const void *v, const float *g, const float *beta,
                     const float *state, const int32_t *parent, int32_t N, int32_t M, int32_t H,
                     void *out, cudaStream_t stream) {
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = allow_dynamic_smem(decode_tree_kernel<Tin, D>, TreeCfg<D>::smem(kMaxTreeNodes), smem_set);
    if (e != cudaSuccess) return e;
    decode_tree_kernel<Tin, D><<<(unsigned)N * (unsigned)H, TreeCfg<D>::THREADS, TreeCfg<D>::smem(M), stream>>>(
        static_cast<const Tin *>(q), static_cast<const Tin *>(k), static_cast<const Tin *>(v), g, beta,
        state, parent, M, H, static_cast<Tin *>(out));
    count_launches(1);
    return cudaGetLastError();
}

template <typename Tin, int D>
cudaError_t run_commit(const void *k, const void *v, const float *g, const float *beta,
                       const float *state_in, const int32_t *path, const int32_t *accept, int32_t N,
                       int32_t M, int32_t P, int32_t H, float *state_out, cudaStream_t stream) {
    decode_commit_kernel<Tin, D><<<(unsigned)N * (unsigned)H, D < 32 ? 32 : D, 0, stream>>>(
        static_cast<const Tin *>(k), static_cast<const Tin *>(v), g, beta, state_in, path, accept, M, P,
        H, state_out);
    count_launches(1);
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

cudaError_t launch_decode_tree(const void *q, const void *k, const void *v, const float *g,
                               const float *beta, const float *state, const int32_t *parent, int32_t N,
                               int32_t M, int32_t H, int32_t D, kda_dtype dt, void *out,
                               cudaStream_t stream) {
    if (dt == KDA_BF16)
        KDA_DISPATCH_D(D, (run_tree<__nv_bfloat16, DD>(q, k, v, g, beta, state, parent, N, M, H, out, stream)))
    KDA_DISPATCH_D(D, (run_tree<float, DD>(q, k, v, g, beta, state, parent, N, M, H, out, stream)))
}

cudaError_t launch_decode_commit(const void *k, const void *v, const float *g, const float *beta,
                                 const float *state_in, const int32_t *path, const int32_t *accept,
                                 int32_t N, int32_t M, int32_t P, int32_t H, int32_t D, kda_dtype dt,
                                 float *state_out, cudaStream_t stream) {
    if (dt == KDA_BF16)
        KDA_DISPATCH_D(D, (run_commit<__nv_bfloat16, DD>(k, v, g, beta, state_in, path, accept, N, M, P, H,
                                                         state_out, stream)))
    KDA_DISPATCH_D(D, (run_commit<float, DD>(k, v, g, beta, state_in, path, accept, N, M, P, H, state_out,
                                             stream)))
}

}  // namespace kda
