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
#include "kda_tc.cuh"
#include "kda_tree.cuh"

#include <math.h>

namespace kda {
namespace {

constexpr int kNodeBlock = 4;   // nodes of a thread's sums

// The fp32 form: any type and head size.  A unit is a (sequence, head); its threads
// have four state columns each, for four of up to 32 nodes at a time.  Small units
// share a CTA.
struct TreeCut {
    int nodes, threads, units;  // nodes at a time; threads per unit; units per CTA
};
// A unit's shared memory: decays, keys (later v - X_k), and the products' operands E k and
// E q; the line products and W's rows by steps up the line, the nodes reached; lines,
// parents, beta.
__host__ __device__ constexpr size_t tree_unit_bytes(int M, int D) {
    const size_t rows = (M + kNodeBlock - 1) / kNodeBlock * kNodeBlock;
    return (rows * D * 16 + (size_t)M * M * 13 + (size_t)M * 16 + 15) / 16 * 16;
}

inline TreeCut tree_cut(int M, int D) {
    int groups = 1;
    while (groups * kNodeBlock < M && groups < 8) groups *= 2;
    const int threads = D / 4 * groups < 8 ? 8 : D / 4 * groups;
    int units = threads >= 128 ? 1 : 128 / threads;
    while (units > 1 && units * tree_unit_bytes(M, D) > 100 * 1024) units /= 2;
    return {groups * kNodeBlock, threads, units};
}

__device__ __forceinline__ float2 load2(const float *p) { return __ldg(reinterpret_cast<const float2 *>(p)); }
__device__ __forceinline__ float2 load2(const __nv_bfloat16 *p) {
    const uint32_t u = __ldg(reinterpret_cast<const uint32_t *>(p));
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ void store4(float *p, float2 lo, float2 hi) {
    *reinterpret_cast<float4 *>(p) = make_float4(lo.x, lo.y, hi.x, hi.y);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float2 lo, float2 hi) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(tc::pack_bf16x2(lo.x, lo.y), tc::pack_bf16x2(hi.x, hi.y));
}

// Line products and W's rows by eight lanes per node, the sums by threads of four
// nodes x four columns: per four state rows four 16-byte reads of the state and
// eight of the operands feed 64 paired multiply-adds.  Then o = X_q + W (v - X_k)
// along the lines.
// Measured, 16 nodes: 64 x 48 fp32 states of 128 x 128 111 us (bytes 49; 4 nodes 54);
// 128 x 64 of 64 x 64 114 (45); bf16, 128 x 96 of 16 x 16 90 us, where the bytes are
// 7.7: the walks and the solve of so small states outweigh them.  Issue slots are 40%
// busy at the 16 warps per SM that the registers allow (three CTAs of 256: 154 us for
// 112).  With a warp per node, a thread per column and eight nodes it took 218, 288
// and 243.
template <typename Tin, int D>
__global__ void __launch_bounds__(256, 2)
decode_tree_kernel(const Tin *__restrict__ q, const Tin *__restrict__ k, const Tin *__restrict__ v,
                   const float *__restrict__ g, const float *__restrict__ beta,
                   const float *__restrict__ state, const int32_t *__restrict__ parent, int64_t all, int32_t M,
                   int32_t H, int32_t threads, int32_t at_once, Tin *__restrict__ out) {
    constexpr int CQ = D / 4;
    constexpr int PW = D / 8 < 4 ? D / 8 : 4, NP = D / 8 / PW;   // a walking lane's channels: NP runs of PW
    extern __shared__ __align__(16) unsigned char smem_raw[];
    const int tid = threadIdx.x % threads, lane = threadIdx.x & 31, l8 = lane & 7;
    const unsigned group = 0xffu << (lane & 24);
    const int64_t unit = (int64_t)blockIdx.x * (blockDim.x / threads) + threadIdx.x / threads;
    const bool live = unit < all;
    const int rows = (M + kNodeBlock - 1) / kNodeBlock * kNodeBlock, walkers = threads / 8, w8 = tid >> 3;
    float *kE = reinterpret_cast<float *>(smem_raw + tree_unit_bytes(M, D) * (threadIdx.x / threads));
    float *qE = kE + rows * D, *al = qE + rows * D, *kk = al + rows * D, *y = kk;
    uint64_t *line = reinterpret_cast<uint64_t *>(kk + rows * D);
    float2 *AB = reinterpret_cast<float2 *>(line + M);
    float *W = reinterpret_cast<float *>(AB + M * M);
    int32_t *par = reinterpret_cast<int32_t *>(W + M * M);
    float *bet = reinterpret_cast<float *>(par + M);
    uint8_t *up = reinterpret_cast<uint8_t *>(bet + M);
    const int64_t n = live ? unit / H : 0, h = live ? unit % H : 0;
    const int64_t row0 = n * M * H + h;                // row of node m: row0 + m H
    const int m_end = live ? M : 0;

    // a state that several threads read comes to the L2 meanwhile (read once, it is only
    // slower: 61 us for 52 with 64 x 48 states, four nodes), and a thread's first node is
    // asked for before anything is waited for
    if (tid == 0 && live && at_once > kNodeBlock)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(state + unit * D * D), "r"(D * D * 4)
                     : "memory");
    const int32_t par_in = tid < m_end ? parent[n * M + tid] : 0;
    const float bet_in = tid < m_end ? __ldg(beta + row0 + (int64_t)tid * H) : 0.f;
    float2 qd[NP][PW / 2];
    auto load_q = [&](int m) {
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int e = 0; e < PW / 2; ++e)
                qd[p][e] = m < m_end ? load2(q + (row0 + (int64_t)m * H) * D + 8 * PW * p + PW * l8 + 2 * e)
                                     : make_float2(0.f, 0.f);
    };
    load_q(w8);
#pragma unroll 2
    for (int i = tid; i < m_end * (D / 8); i += threads) {
        const int64_t at = (row0 + (int64_t)(i / (D / 8)) * H) * D + i % (D / 8) * 8;
        float x[8], f[8];
        Elem<float>::load8(g + at, x);
        Elem<Tin>::load8(k + at, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __expf(x[e]);
        Elem<float>::store8(al + 8 * i, x);
        Elem<float>::store8(kk + 8 * i, f);
    }
    for (int m = tid; m < m_end; m += threads) {
        par[m] = m == tid ? par_in : parent[n * M + m];
        bet[m] = m == tid ? bet_in : __ldg(beta + row0 + (int64_t)m * H);
    }
    __syncthreads();
    for (int m = w8; m < (live ? rows : 0); m += walkers) {
        float2 kd[NP][PW / 2];
        auto get = [&](const float *from, float2 (&x)[NP][PW / 2]) {
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                if constexpr (PW == 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(from + 32 * p + 4 * l8);
                    x[p][0] = make_float2(f.x, f.y);
                    x[p][1] = make_float2(f.z, f.w);
                } else {
                    x[p][0] = *reinterpret_cast<const float2 *>(from + 2 * l8);
                }
            }
        };
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int e = 0; e < PW / 2; ++e) kd[p][e] = make_float2(0.f, 0.f);
        if (m < M) get(kk + m * D, kd);
        uint64_t on = 0;
        int at = m < M ? m : -1, steps = 0;
        bool whole = false;                            // the walk ended below the prefix
        while (at >= 0) {
            float2 kj[NP][PW / 2], aj[NP][PW / 2], a2 = make_float2(0.f, 0.f), b2 = a2;
            const int next = par[at];
            get(kk + at * D, kj);
            get(al + at * D, aj);
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int e = 0; e < PW / 2; ++e) {
                    a2 = tc::f2fma(kd[p][e], kj[p][e], a2);
                    b2 = tc::f2fma(qd[p][e], kj[p][e], b2);
                    kd[p][e] = tc::f2mul(kd[p][e], aj[p][e]);
                    qd[p][e] = tc::f2mul(qd[p][e], aj[p][e]);
                }
            const float a = a2.x + a2.y, b = b2.x + b2.y;
            // lanes 0-3 of the group sum the k products, lanes 4-7 the q products
            float x = (l8 < 4 ? a : b) + __shfl_xor_sync(group, l8 < 4 ? b : a, 4);
            x += __shfl_xor_sync(group, x, 2);
            x += __shfl_xor_sync(group, x, 1);
            if ((l8 & 3) == 0) reinterpret_cast<float *>(AB + m * M + steps)[l8 >> 2] = x;
            if (l8 == 1) up[m * M + steps] = (uint8_t)at;
            on |= uint64_t{1} << at;
            ++steps;
            whole = next == -1;
            at = next < at ? next : -2;
        }
        if (m < M && l8 == 0) line[m] = whole ? on : 0;
        auto put = [&](float *to, const float2 (&x)[NP][PW / 2]) {
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                if constexpr (PW == 4)
                    store4(to + 32 * p + 4 * l8, x[p][0], x[p][1]);
                else
                    *reinterpret_cast<float2 *>(to + 2 * l8) = x[p][0];
            }
        };
        put(kE + m * D, kd);                           // (of no node: never read into a result)
        put(qE + m * D, qd);
        load_q(m + walkers);
    }
    const int c = tid % CQ * 4, mine = tid / CQ * kNodeBlock;
    const bool sums = live && mine < at_once && mine < M;
    const float *S = state + unit * D * D + c;
    float4 ahead[4];                                   // the next four state rows
    auto fetch = [&](int i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) ahead[e] = __ldg(reinterpret_cast<const float4 *>(S + (i + e) * D));
    };
    if (sums) fetch(0);
    __syncthreads();

    // The rows of W by steps up the line: z starts as the q products; a step's w leaves
    // z's later entries less its k products.  Eight lanes per node, lane l8 the steps
    // l8, l8 + 8, ...
    for (int m = w8; m < m_end; m += walkers) {
        const int steps = __popcll((long long)line[m]);
        float z[kMaxTreeNodes / 8];
#pragma unroll
        for (int r = 0; r < kMaxTreeNodes / 8; ++r) z[r] = 8 * r + l8 < steps ? AB[m * M + 8 * r + l8].y : 0.f;
#pragma unroll
        for (int r = 0; r < kMaxTreeNodes / 8; ++r) {
            for (int s8 = 0; s8 < 8 && 8 * r + s8 < steps; ++s8) {
                const int s = 8 * r + s8, j = up[m * M + s];
                const float w = __shfl_sync(group, z[r], s8, 8) * bet[j];
                const float2 *ab = AB + j * M - s;
#pragma unroll
                for (int i = r; i < kMaxTreeNodes / 8; ++i) {
                    const int t = 8 * i + l8;
                    if (t > s && t < steps) z[i] -= w * ab[t].x;
                }
                if (l8 == 0) W[m * M + s] = w;
            }
        }
    }

    for (int m0 = 0; m0 < M; m0 += at_once) {
        const int m1 = m0 + mine;                      // this thread's nodes: m1 .. m1 + 3
        float2 xk[kNodeBlock][2], xq[kNodeBlock][2];
#pragma unroll
        for (int b = 0; b < kNodeBlock; ++b) xk[b][0] = xk[b][1] = xq[b][0] = xq[b][1] = make_float2(0.f, 0.f);
        if (sums && m1 < M) {
            const float *ke = kE + m1 * D, *qe = qE + m1 * D;
#pragma unroll 2
            for (int i = 0; i < D; i += 4) {
                const float4 s4[4] = {ahead[0], ahead[1], ahead[2], ahead[3]};
                fetch(i + 4 < D ? i + 4 : 0);          // (the first rows again for the next nodes)
#pragma unroll
                for (int b = 0; b < kNodeBlock; ++b) {
                    const float4 x = *reinterpret_cast<const float4 *>(ke + b * D + i),
                                 z = *reinterpret_cast<const float4 *>(qe + b * D + i);
                    const float xs[4] = {x.x, x.y, x.z, x.w}, zs[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 lo = make_float2(s4[e].x, s4[e].y), hi = make_float2(s4[e].z, s4[e].w);
                        xk[b][0] = tc::f2fma(make_float2(xs[e], xs[e]), lo, xk[b][0]);
                        xk[b][1] = tc::f2fma(make_float2(xs[e], xs[e]), hi, xk[b][1]);
                        xq[b][0] = tc::f2fma(make_float2(zs[e], zs[e]), lo, xq[b][0]);
                        xq[b][1] = tc::f2fma(make_float2(zs[e], zs[e]), hi, xq[b][1]);
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < kNodeBlock; ++b) {
                if (m1 + b >= M) break;
                const Tin *from = v + (row0 + (int64_t)(m1 + b) * H) * D + c;
                const float2 lo = load2(from), hi = load2(from + 2);
                *reinterpret_cast<float4 *>(y + (m1 + b) * D + c) =
                    make_float4(lo.x - xk[b][0].x, lo.y - xk[b][0].y, hi.x - xk[b][1].x, hi.y - xk[b][1].y);
            }
        }
        __syncthreads();                               // nodes above are in this pass or an earlier one
        if (sums && m1 < M) {
#pragma unroll
            for (int b = 0; b < kNodeBlock; ++b) {
                const int m = m1 + b;
                if (m >= M) break;
                const int steps = __popcll((long long)line[m]);
                float2 lo = xq[b][0], hi = xq[b][1];
                for (int s = 0; s < steps; ++s) {
                    const float w = W[m * M + s];
                    const float4 yj = *reinterpret_cast<const float4 *>(y + up[m * M + s] * D + c);
                    lo = tc::f2fma(make_float2(w, w), make_float2(yj.x, yj.y), lo);
                    hi = tc::f2fma(make_float2(w, w), make_float2(yj.z, yj.w), hi);
                }
                if (steps == 0) lo = hi = make_float2(0.f, 0.f);
                store4(out + (row0 + (int64_t)m * H) * D + c, lo, hi);
            }
        }
    }
}

// The state after the first accept[n] nodes of path[n].  A warp keeps 16 state
// columns in registers: lane = (row group r of 8, column quad c of 4), rows
// 8i + r, so that a column's read S^T k closes with three shuffles and the
// warps never wait for one another.  The state moves once in each direction.
// A CTA has up to four such warps, so d = 128 takes two CTAs per state.
// Measured: 256 x 96 states of 128 x 128, bf16 inputs: 459 us for one token (7.1
// TB/s), 579 us for 3.5 on average (5.7 TB/s); above one token it is bound by
// what four CTAs' registers (127 a thread) leave of latency to hide: five spill
// (700 us).  Pairs of fp32 in one instruction took 17 us off.
template <int D> struct CommitCfg {
    static constexpr int WARPS = D < 64 ? D / 16 : 4, SPLIT = D / 16 / WARPS;
};
template <typename Tin, int D>
__global__ void __launch_bounds__(32 * CommitCfg<D>::WARPS, D == 128 ? 4 : 1)
decode_commit_kernel(const Tin *__restrict__ k, const Tin *__restrict__ v, const float *__restrict__ g,
                     const float *__restrict__ beta, const float *state_in,
                     const int32_t *__restrict__ path, const int32_t *__restrict__ accept, int32_t M,
                     int32_t P, int32_t H, float *state_out) {
    constexpr int SPLIT = CommitCfg<D>::SPLIT;
    static_assert(32 * CommitCfg<D>::WARPS >= D, "a thread per channel");
    constexpr int BATCH = 4;                         // path nodes staged at a time
    constexpr int ROWS = D / 8;                      // state rows per lane
    constexpr int COLS = 16 * CommitCfg<D>::WARPS;   // state columns of the CTA
    __shared__ __align__(16) float2 ak[BATCH][D];    // (decay, k) per channel
    __shared__ __align__(16) float vs[BATCH][COLS];
    __shared__ float bs[BATCH];
    const int tid = threadIdx.x, lane = tid & 31, r = lane >> 2;
    const int col0 = (blockIdx.x % SPLIT) * COLS, lcol = (tid >> 5) * 16 + (lane & 3) * 4;
    const int unit = blockIdx.x / SPLIT;
    const int64_t n = unit / H;
    const int h = unit % H;
    const size_t base = (size_t)unit * D * D + (size_t)r * D + col0 + lcol;
    float2 s[ROWS][2];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const float4 x = __ldcs(reinterpret_cast<const float4 *>(state_in + base + (size_t)i * 8 * D));
        s[i][0] = make_float2(x.x, x.y);
        s[i][1] = make_float2(x.z, x.w);
    }
    int acc = accept[n];
    acc = acc < 0 ? 0 : (acc > P ? P : acc);
    for (int t0 = 0; t0 < acc; t0 += BATCH) {
        // the batch ends at its first entry outside the tree, and the path with it
        int node[BATCH], cnt = acc - t0 < BATCH ? acc - t0 : BATCH;
#pragma unroll
        for (int t = 0; t < BATCH; ++t) node[t] = t0 + t < P ? path[n * P + t0 + t] : -1;
#pragma unroll
        for (int t = BATCH - 1; t >= 0; --t)
            if (t < cnt && (node[t] < 0 || node[t] >= M)) {
                cnt = t;
                acc = 0;
            }
        // All of the batch's loads go before the first is used: no branch between them
        // (the rows past cnt are the first one again), since a branch per token waited
        // for its loads, 1 us per token.
        const int some = cnt > 0 ? node[0] : 0;
        float gt[BATCH], bt8[BATCH];
        Tin kt[BATCH], vt8[BATCH];
#pragma unroll
        for (int t = 0; t < BATCH; ++t) {
            const int64_t row = (n * M + (t < cnt ? node[t] : some)) * H + h, at = row * D;
            gt[t] = __ldg(g + at + tid % D);
            kt[t] = k[at + tid % D];
            vt8[t] = v[at + col0 + tid % COLS];
            bt8[t] = __ldg(beta + row);
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < BATCH; ++t) {
            if (tid < D) ak[t][tid] = make_float2(__expf(gt[t]), Elem<Tin>::load(&kt[t]));
            if (tid < COLS) vs[t][tid] = Elem<Tin>::load(&vt8[t]);
            if (tid == 0) bs[t] = bt8[t];
        }
        __syncthreads();
#pragma unroll 1
        for (int t = 0; t < cnt; ++t) {
            const float bt = bs[t];
            const float4 vt = *reinterpret_cast<const float4 *>(&vs[t][lcol]);
            float2 x[2];
            x[0] = x[1] = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const float2 f = ak[t][i * 8 + r];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    s[i][y] = tc::f2mul(s[i][y], make_float2(f.x, f.x));
                    x[y] = tc::f2fma(s[i][y], make_float2(f.y, f.y), x[y]);
                }
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                x[0].x += __shfl_xor_sync(0xffffffffu, x[0].x, o);
                x[0].y += __shfl_xor_sync(0xffffffffu, x[0].y, o);
                x[1].x += __shfl_xor_sync(0xffffffffu, x[1].x, o);
                x[1].y += __shfl_xor_sync(0xffffffffu, x[1].y, o);
            }
            const float2 u[2] = {make_float2(bt * (vt.x - x[0].x), bt * (vt.y - x[0].y)),
                                 make_float2(bt * (vt.z - x[1].x), bt * (vt.w - x[1].y))};
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const float ki = ak[t][i * 8 + r].y;
#pragma unroll
                for (int y = 0; y < 2; ++y) s[i][y] = tc::f2fma(u[y], make_float2(ki, ki), s[i][y]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
        __stcs(reinterpret_cast<float4 *>(state_out + base + (size_t)i * 8 * D),
               make_float4(s[i][0].x, s[i][0].y, s[i][1].x, s[i][1].y));
}

// ---- bf16 inputs, d = 32, 64 or 128: the products with S_0 on the tensor cores ----
//
// One CTA per (sequence, head), of four warps at d = 128 and up to 16 nodes.  Nodes 8i .. 8i+7 make row tile
// i: rows 0-7 are E_m k_m, rows 8-15 E_m q_m, so a tile is full whether the
// tree has 8 nodes or 64.  Warp w multiplies all tiles with state columns
// 32w .. 32w+31 (mma.sync m16n8k16): a lane loads 16 bytes of four state rows
// and takes its four columns as column g of four 8-wide tiles (half of all that
// with twice the warps), so the fp32 state goes from HBM to the fragments without
// passing shared memory, in whole 128-byte lines.
//
// The solve does not touch the 128 columns: with y = v - (the k sums) the
// outputs are (the q sums) + W y, where row m of W lives on m's line.  Let s
// count the steps up that line, j_s the node reached, A and B the line
// products.  Then W_m,j_s = z_s beta_{j_s} with, from the bottom up,
//     z_s = B_m,j_s - sum_{s' < s} z_s' beta_{j_s'} A_{j_s',j_s},
// which eight lanes solve for each node in as many steps as its line is long,
// all nodes at once.  W y is one more small product whose accumulators are the
// q sums where they already are; y turns into its operand by 8x8 transposes in
// registers.
//
// All operands are split into a bf16 part and a bf16 rest (16 significant bits
// together), and three of the four partial products are summed in fp32: the
// fourth is below 2^-16 of the product.
//
// Measured: 256 sequences x 96 heads, 16 nodes: 439 us, 5.0 TB/s (8 nodes 336
// us, 5.7 TB/s; 128 x 32 nodes 457 us; 64 x 64 nodes 617 us).  Above eight
// nodes it is bound by the latency that four CTAs' registers leave to hide
// (issue slots 36% busy): the walk, the waits at the three barriers and the
// fragments' loads from the L2.  On the way: fp32 products 1,673 us; the solve
// by a thread per state column 849; its rows on a fifth warp 778; walks of
// eight lanes per node, all nodes at once, 620; W's rows by eight lanes 453.
// 16 nodes, 128 x 64 states of 64 x 64 75 us (floor 35, the fp32 form 116), 128 x
// 96 of 32 x 32 62 us (floor 19, the fp32 form 100).
template <int D, int TILES> struct TcCfg {
    static constexpr int ALD = D + 8;                 // bf16 per operand row: an odd number of 16-byte pieces
    // Warps share the state's columns.  d = 128: four of 32; eight of 16 above 16 nodes and
    // 16 of eight above 32, where shared memory leaves room for two CTAs and one (with four
    // throughout, 128 x 32 nodes took 535 us instead of 457, 64 x 64 nodes 986 instead of
    // 617).  Smaller heads: one column tile more per warp saves operand reads while there
    // are few nodes (d = 64, 6 nodes: 40 us with two warps, 42 with four; d = 32: 26 and
    // 34), and costs registers when there are many (d = 32, 48 nodes: 204 and 113).
    static constexpr int WARPS = D == 128  ? (TILES <= 2 ? 4 : 2 * TILES)
                                 : D == 64 ? (TILES == 1 ? 2 : TILES <= 4 ? 4 : 8)
                                           : (TILES <= 2 ? 2 : 4);
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int NT = D / 8 / WARPS;          // 8-wide column tiles per warp = columns per lane
    static constexpr int CTAS = D == 128  ? (TILES <= 2 ? 4 : TILES == 4 ? 2 : 1)
                                : D == 64 ? (TILES == 1 ? 8 : TILES == 2 ? 6 : TILES == 4 ? 4 : 1)
                                          : (TILES <= 2 ? 12 : 4);
    static constexpr int PAIRS = (TILES + 1) / 2;     // 16-node blocks of W
    static constexpr int WLD = PAIRS * 16 + 8;        // bf16 per row of W: an odd number of 16-byte pieces
    static constexpr size_t A_BYTES = (size_t)TILES * 16 * ALD * 2 * 2;
    static constexpr size_t W_BYTES = (size_t)PAIRS * 16 * WLD * 2 * 2;
    static size_t smem(int M) {
        return A_BYTES + W_BYTES + (size_t)M * (D * (4 + 4) + 16) + (size_t)M * M * (8 + 1);
    }
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&x);
}
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
// two floats as bf16 pairs: the rounded values and the rounded rests
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack2(a, b);
    lo = pack2(a - lo_f(hi), b - hi_f(hi));
}
__device__ __forceinline__ void mma16816(float &d0, float &d1, float &d2, float &d3, const uint32_t (&a)[4],
                                         uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d0), "+f"(d1), "+f"(d2), "+f"(d3)
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// an 8x8 tile of 16-bit values held as (row lane/4, columns 2(lane%4), +1), transposed
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// Whether the nearest bf16 number is finite: |x| < 2^128 - 2^119.
constexpr uint32_t kBf16End = 0x7f7f8000u;
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

template <int D, int TILES>
__global__ void __launch_bounds__(TcCfg<D, TILES>::THREADS, TcCfg<D, TILES>::CTAS)
decode_tree_tc_kernel(const __nv_bfloat16 *__restrict__ q, const __nv_bfloat16 *__restrict__ k,
                      const __nv_bfloat16 *__restrict__ v, const float *__restrict__ g,
                      const float *__restrict__ beta, const float *__restrict__ state,
                      const int32_t *__restrict__ parent, int32_t M, int32_t H,
                      __nv_bfloat16 *__restrict__ out) {
    using C = TcCfg<D, TILES>;
    constexpr int kALd = C::ALD, RUNS = D / 32;       // a walking lane's runs of four channels
    constexpr int KS = D / 16, WARPS = C::WARPS, THREADS = C::THREADS, NT = C::NT;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __nv_bfloat16 *ahi = reinterpret_cast<__nv_bfloat16 *>(smem_raw), *alo = ahi + TILES * 16 * kALd;
    __nv_bfloat16 *whi = reinterpret_cast<__nv_bfloat16 *>(smem_raw + C::A_BYTES),
                  *wlo = whi + C::PAIRS * 16 * C::WLD;
    float *al = reinterpret_cast<float *>(smem_raw + C::A_BYTES + C::W_BYTES);
    float *kk = al + M * D;
    uint64_t *line = reinterpret_cast<uint64_t *>(kk + M * D);
    // by steps up m's line: the products with the node reached, and its index
    float2 *AB = reinterpret_cast<float2 *>(line + M);
    int32_t *par = reinterpret_cast<int32_t *>(AB + M * M);
    float *bet = reinterpret_cast<float *>(par + M);
    uint8_t *up = reinterpret_cast<uint8_t *>(bet + M);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t n = blockIdx.x / H;
    const int h = blockIdx.x % H;
    const int64_t row0 = n * M * H + h;                // row of node m: row0 + m H
    const float *S = state + (size_t)blockIdx.x * D * D;

    // the state comes to the L2 while the line products run
    if (tid == 0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(S), "r"(D * D * 4) : "memory");
    // every load of the inputs is on its way before the first is used
    static_assert(THREADS >= 8 * TILES, "a thread per node");
    const int32_t par_in = tid < M ? parent[n * M + tid] : 0;
    const float bet_in = tid < M ? __ldg(beta + row0 + (int64_t)tid * H) : 0.f;
    // line products: eight lanes per node, channels 32 p + 4 (lane % 8) .. + 3
    const int l8 = lane & 7;
    const unsigned group = 0xffu << (lane & 24);
    int m = warp * 4 + (lane >> 3);
    uint2 qm[RUNS];
    auto load_q = [&]() {
#pragma unroll
        for (int p = 0; p < RUNS; ++p)
            qm[p] = m < M ? __ldg(reinterpret_cast<const uint2 *>(q + (row0 + (int64_t)m * H) * D + 32 * p + 4 * l8))
                          : make_uint2(0u, 0u);
    };
    load_q();
    constexpr int PIECES = 2;                         // of eight channels, per thread and pass
    for (int i0 = tid; i0 < M * (D / 8); i0 += PIECES * THREADS) {
        float x[PIECES][8];
        uint4 y[PIECES];
#pragma unroll
        for (int z = 0; z < PIECES; ++z) {
            const int i = min(i0 + z * THREADS, M * (D / 8) - 1);
            const int64_t at = (row0 + (int64_t)(i / (D / 8)) * H) * D + i % (D / 8) * 8;
            Elem<float>::load8(g + at, x[z]);
            y[z] = __ldg(reinterpret_cast<const uint4 *>(k + at));
        }
#pragma unroll
        for (int z = 0; z < PIECES; ++z) {
            const int i = min(i0 + z * THREADS, M * (D / 8) - 1);   // (the last piece may be written twice)
            const float kf[8] = {lo_f(y[z].x), hi_f(y[z].x), lo_f(y[z].y), hi_f(y[z].y),
                                 lo_f(y[z].z), hi_f(y[z].z), lo_f(y[z].w), hi_f(y[z].w)};
#pragma unroll
            for (int e = 0; e < 8; ++e) x[z][e] = __expf(x[z][e]);
            Elem<float>::store8(al + 8 * i, x[z]);
            Elem<float>::store8(kk + 8 * i, kf);
        }
    }
    if (tid < M) {
        par[tid] = par_in;
        bet[tid] = bet_in;
    }
    for (int i = tid; i < (int)(C::W_BYTES / 16); i += THREADS)
        reinterpret_cast<uint4 *>(whi)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    for (; m < TILES * 8; m += 4 * WARPS) {
        float2 kd[2 * RUNS], qd[2 * RUNS];
#pragma unroll
        for (int p = 0; p < RUNS; ++p) {
            const float4 f = m < M ? *reinterpret_cast<const float4 *>(kk + m * D + 32 * p + 4 * l8)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
            kd[2 * p] = make_float2(f.x, f.y);
            kd[2 * p + 1] = make_float2(f.z, f.w);
            qd[2 * p] = make_float2(lo_f(qm[p].x), hi_f(qm[p].x));
            qd[2 * p + 1] = make_float2(lo_f(qm[p].y), hi_f(qm[p].y));
        }
        uint64_t on = 0;
        int at = m < M ? m : -1, steps = 0;
        bool whole = false;                           // the walk ended below the prefix
        float a = 0.f, b = 0.f;
        // lanes 0-3 of the group sum the k products of a step, lanes 4-7 the q products
        auto close = [&](int step) {
            float x = (l8 < 4 ? a : b) + __shfl_xor_sync(group, l8 < 4 ? b : a, 4);
            x += __shfl_xor_sync(group, x, 2);
            x += __shfl_xor_sync(group, x, 1);
            if ((l8 & 3) == 0) reinterpret_cast<float *>(AB + m * M + step)[l8 >> 2] = x;
        };
        while (at >= 0) {
            const int next = par[at];
            float4 kj[RUNS], aj[RUNS];
#pragma unroll
            for (int p = 0; p < RUNS; ++p) {
                kj[p] = *reinterpret_cast<const float4 *>(kk + at * D + 32 * p + 4 * l8);
                aj[p] = *reinterpret_cast<const float4 *>(al + at * D + 32 * p + 4 * l8);
            }
            if (steps > 0) close(steps - 1);          // the step before, while these load
            if (l8 == 1) up[m * M + steps] = (uint8_t)at;
            on |= uint64_t{1} << at;
            float2 a2[2], b2[2];
            a2[0] = a2[1] = b2[0] = b2[1] = make_float2(0.f, 0.f);
#pragma unroll
            for (int p = 0; p < RUNS; ++p) {
                const float2 k0 = make_float2(kj[p].x, kj[p].y), k1 = make_float2(kj[p].z, kj[p].w);
                const float2 a0 = make_float2(aj[p].x, aj[p].y), a1 = make_float2(aj[p].z, aj[p].w);
                a2[0] = tc::f2fma(kd[2 * p], k0, a2[0]);
                a2[1] = tc::f2fma(kd[2 * p + 1], k1, a2[1]);
                b2[0] = tc::f2fma(qd[2 * p], k0, b2[0]);
                b2[1] = tc::f2fma(qd[2 * p + 1], k1, b2[1]);
                kd[2 * p] = tc::f2mul(kd[2 * p], a0);
                kd[2 * p + 1] = tc::f2mul(kd[2 * p + 1], a1);
                qd[2 * p] = tc::f2mul(qd[2 * p], a0);
                qd[2 * p + 1] = tc::f2mul(qd[2 * p + 1], a1);
            }
            a = (a2[0].x + a2[0].y) + (a2[1].x + a2[1].y);
            b = (b2[0].x + b2[0].y) + (b2[1].x + b2[1].y);
            ++steps;
            whole = next == -1;
            at = next < at ? next : -2;
        }
        if (steps > 0) close(steps - 1);
        if (!whole) {
            on = 0;
#pragma unroll
            for (int x = 0; x < 2 * RUNS; ++x) kd[x] = qd[x] = make_float2(0.f, 0.f);
        }
        if (l8 == 0 && m < M) line[m] = on;
        // row of the k operand, and eight rows on the q operand (zeros where there is no node)
        const int row = (m >> 3) * 16 + (m & 7);
#pragma unroll
        for (int p = 0; p < RUNS; ++p) {
            const int c = 32 * p + 4 * l8;
            uint32_t hi[2], lo[2];
            split2(kd[2 * p].x, kd[2 * p].y, hi[0], lo[0]);
            split2(kd[2 * p + 1].x, kd[2 * p + 1].y, hi[1], lo[1]);
            *reinterpret_cast<uint2 *>(ahi + row * kALd + c) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2 *>(alo + row * kALd + c) = make_uint2(lo[0], lo[1]);
            split2(qd[2 * p].x, qd[2 * p].y, hi[0], lo[0]);
            split2(qd[2 * p + 1].x, qd[2 * p + 1].y, hi[1], lo[1]);
            *reinterpret_cast<uint2 *>(ahi + (row + 8) * kALd + c) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2 *>(alo + (row + 8) * kALd + c) = make_uint2(lo[0], lo[1]);
        }
        m += 4 * WARPS;
        load_q();
        m -= 4 * WARPS;
    }
    // the first state rows and the values set out before the operands are ready
    const int gq = lane & 3, gg = lane >> 2;
    const float *Sw = S + (size_t)(2 * gq) * D + warp * 8 * NT + gg * NT;
    auto fetch = [&](int ks, float (&f)[4][NT]) {
        const float *p = Sw + (size_t)ks * 16 * D;
        const int rows[4] = {0, 1, 8, 9};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            if constexpr (NT == 4) {
                const float4 x = __ldcs(reinterpret_cast<const float4 *>(p + rows[y] * D));
                f[y][0] = x.x; f[y][1] = x.y; f[y][2] = x.z; f[y][3] = x.w;
            } else if constexpr (NT == 2) {
                const float2 x = __ldcs(reinterpret_cast<const float2 *>(p + rows[y] * D));
                f[y][0] = x.x; f[y][1] = x.y;
            } else {
                f[y][0] = __ldcs(p + rows[y] * D);
            }
        }
    };
    constexpr int AHEAD = KS > 3 ? 3 : KS - 1;                          // steps of 16 state rows on their way
    float buf[AHEAD + 1][4][NT];
    const int64_t vcol = warp * 8 * NT + 2 * NT * gq; // values of node 8i + gg, 2 NT state columns from vcol
    uint32_t vv[TILES][NT];
#pragma unroll
    for (int ks = 0; ks < AHEAD; ++ks) fetch(ks, buf[ks]);
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
        const int mm = 8 * i + gg;
#pragma unroll
        for (int x = 0; x < NT; ++x) vv[i][x] = 0u;
        if (mm < M) {
            const __nv_bfloat16 *from = v + (row0 + (int64_t)mm * H) * D + vcol;
            if constexpr (NT == 4) {
                const uint4 x = __ldg(reinterpret_cast<const uint4 *>(from));
                vv[i][0] = x.x; vv[i][1] = x.y; vv[i][2] = x.z; vv[i][3] = x.w;
            } else if constexpr (NT == 2) {
                const uint2 x = __ldg(reinterpret_cast<const uint2 *>(from));
                vv[i][0] = x.x; vv[i][1] = x.y;
            } else {
                vv[i][0] = __ldg(reinterpret_cast<const uint32_t *>(from));
            }
        }
    }
    __syncthreads();

    // the rows of W: eight lanes per node, lane l8 the steps l8, l8 + 8, ...
    for (m = warp * 4 + (lane >> 3); m < M; m += 4 * WARPS) {
        const int steps = __popcll((long long)line[m]);
        float z[TILES];
#pragma unroll
        for (int r = 0; r < TILES; ++r) z[r] = 8 * r + l8 < steps ? AB[m * M + 8 * r + l8].y : 0.f;
#pragma unroll
        for (int r = 0; r < TILES; ++r) {
            for (int s8 = 0; s8 < 8 && 8 * r + s8 < steps; ++s8) {
                const int s = 8 * r + s8, j = up[m * M + s];
                const float w = __shfl_sync(group, z[r], s8, 8) * bet[j];
                const float2 *ab = AB + j * M - s;
#pragma unroll
                for (int i = r; i < TILES; ++i) {
                    const int t = 8 * i + l8;
                    if (t > s && t < steps) z[i] -= w * ab[t].x;
                }
                if (l8 == 0) {
                    const __nv_bfloat16 hi = __float2bfloat16_rn(w);
                    whi[m * C::WLD + j] = hi;
                    wlo[m * C::WLD + j] = __float2bfloat16_rn(w - __bfloat162float(hi));
                }
            }
        }
    }

    __syncwarp();                                     // groups of lanes were on lines of their own
    float acc[TILES][NT][4];
#pragma unroll
    for (int i = 0; i < TILES; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][t][e] = 0.f;
    const uint32_t frag = (uint32_t)(lane & 15), piece = (uint32_t)(lane >> 4) * 16;
    const uint32_t abase = static_cast<uint32_t>(__cvta_generic_to_shared(ahi)) + frag * (kALd * 2) + piece;
    constexpr uint32_t kALo = TILES * 16 * kALd * 2;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        if (ks + AHEAD < KS) fetch(ks + AHEAD, buf[(ks + AHEAD) % (AHEAD + 1)]);
        const float(&f)[4][NT] = buf[ks % (AHEAD + 1)];
        uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int half = 0; half < 2; ++half)
                split2(f[2 * half][t], f[2 * half + 1][t], bh[t][half], bl[t][half]);
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
            uint32_t xh[4], xl[4];
            ldsm4(abase + (i * 16 * kALd + ks * 16) * 2, xh);
            ldsm4(abase + (i * 16 * kALd + ks * 16) * 2 + kALo, xl);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float(&d)[4] = acc[i][t];
                mma16816(d[0], d[1], d[2], d[3], xh, bh[t][0], bh[t][1]);
                mma16816(d[0], d[1], d[2], d[3], xh, bl[t][0], bl[t][1]);
                mma16816(d[0], d[1], d[2], d[3], xl, bh[t][0], bh[t][1]);
            }
        }
    }
    // lane (gg, gq): node 8i + gg's k sums (entries 0, 1; they become y) and q sums
    // (2, 3) of the tile columns 2 gq and 2 gq + 1, i.e. columns vcol + t and vcol + NT + t
    uint32_t most = 0;                                // the largest y (no number is above all)
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint32_t u0 = vv[i][t >> 1], u1 = vv[i][(NT + t) >> 1];
            acc[i][t][0] = ((t & 1) ? hi_f(u0) : lo_f(u0)) - acc[i][t][0];
            acc[i][t][1] = (((NT + t) & 1) ? hi_f(u1) : lo_f(u1)) - acc[i][t][1];
            most = max(most, max(magnitude(acc[i][t][0]), magnitude(acc[i][t][1])));
        }
    }
    const bool dirty = __any_sync(0xffffffffu, most >= kBf16End);
    __syncthreads();                                  // W is there
    // A y that is not finite in bf16 belongs to its own line only: the dense product
    // takes a zero in its place, and it is added where it is seen (a number weighted)
    float seen[TILES][NT][2];
    if (dirty) {
#pragma unroll
        for (int i = 0; i < TILES; ++i)
#pragma unroll
            for (int x = 0; x < 2 * NT; ++x) seen[i][x >> 1][x & 1] = 0.f;
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
#pragma unroll 1
            for (int r = 0; r < 8 && 8 * i + r < M; ++r) {
                float y[NT][2];
#pragma unroll
                for (int x = 0; x < 2 * NT; ++x)
                    y[x >> 1][x & 1] = __shfl_sync(0xffffffffu, acc[i][x >> 1][x & 1], r * 4 + gq);
#pragma unroll
                for (int o = 0; o < TILES; ++o) {
                    const int m = 8 * o + gg;
                    if (m >= M || (line[m] >> (8 * i + r) & 1) == 0) continue;
                    const int at = m * C::WLD + 8 * i + r;
                    const float w = __bfloat162float(whi[at]) + __bfloat162float(wlo[at]);
#pragma unroll
                    for (int x = 0; x < 2 * NT; ++x) {
                        const float f = y[x >> 1][x & 1];
                        if (magnitude(f) >= kBf16End) seen[o][x >> 1][x & 1] += fabsf(f) < INFINITY ? w * f : f;
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < TILES; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (magnitude(acc[i][t][0]) >= kBf16End) acc[i][t][0] = 0.f;
                if (magnitude(acc[i][t][1]) >= kBf16End) acc[i][t][1] = 0.f;
            }
        __syncwarp();
    }
    uint32_t yh[2 * C::PAIRS][NT], yl[2 * C::PAIRS][NT];
#pragma unroll
    for (int i = 0; i < 2 * C::PAIRS; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            yh[i][t] = yl[i][t] = 0u;
            if (i < TILES) {
                uint32_t hi, lo;
                split2(acc[i % TILES][t][0], acc[i % TILES][t][1], hi, lo);
                yh[i][t] = transpose8x8(hi);
                yl[i][t] = transpose8x8(lo);
            }
        }
    const uint32_t wbase = static_cast<uint32_t>(__cvta_generic_to_shared(whi)) + frag * (C::WLD * 2) + piece;
    constexpr uint32_t kWLo = C::PAIRS * 16 * C::WLD * 2;
#pragma unroll
    for (int i = 0; i < C::PAIRS; ++i) {
        float none[NT][2];                             // the upper half of a lone tile
#pragma unroll
        for (int t = 0; t < NT; ++t) none[t][0] = none[t][1] = 0.f;
#pragma unroll
        for (int b = 0; b <= i; ++b) {                // nodes above have lower indices
            uint32_t xh[4], xl[4];
            ldsm4(wbase + (i * 16 * C::WLD + b * 16) * 2, xh);
            ldsm4(wbase + (i * 16 * C::WLD + b * 16) * 2 + kWLo, xl);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float &d0 = acc[2 * i][t][2], &d1 = acc[2 * i][t][3];
                float &d2 = 2 * i + 1 < TILES ? acc[(2 * i + 1) % TILES][t][2] : none[t][0];
                float &d3 = 2 * i + 1 < TILES ? acc[(2 * i + 1) % TILES][t][3] : none[t][1];
                mma16816(d0, d1, d2, d3, xh, yh[2 * b][t], yh[2 * b + 1][t]);
                mma16816(d0, d1, d2, d3, xh, yl[2 * b][t], yl[2 * b + 1][t]);
                mma16816(d0, d1, d2, d3, xl, yh[2 * b][t], yh[2 * b + 1][t]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
        const int m = 8 * i + gg;
        if (m >= M) continue;
        if (dirty) {
            // (dirty too where the state is not finite: such a column's k sums are not, whatever the
            // operands, and a row of no node has taken them against zeros)
            const bool none = line[m] == 0;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                acc[i][t][2] = none ? 0.f : acc[i][t][2] + seen[i][t][0];
                acc[i][t][3] = none ? 0.f : acc[i][t][3] + seen[i][t][1];
            }
        }
        __nv_bfloat16 *to = out + (row0 + (int64_t)m * H) * D + vcol;
        if constexpr (NT == 4)
            *reinterpret_cast<uint4 *>(to) = make_uint4(pack2(acc[i][0][2], acc[i][1][2]), pack2(acc[i][2][2], acc[i][3][2]),
                                                        pack2(acc[i][0][3], acc[i][1][3]), pack2(acc[i][2][3], acc[i][3][3]));
        else if constexpr (NT == 1)
            *reinterpret_cast<uint32_t *>(to) = pack2(acc[i][0][2], acc[i][0][3]);
        else
            *reinterpret_cast<uint2 *>(to) = make_uint2(pack2(acc[i][0][2], acc[i][1][2]), pack2(acc[i][0][3], acc[i][1][3]));
    }
}

template <typename Tin, int D>
cudaError_t run_tree(const void *q, const void *k, const void *v, const float *g, const float *beta,
                     const float *state, const int32_t *parent, int32_t N, int32_t M, int32_t H,
                     void *out, cudaStream_t stream) {
    static std::atomic<uint64_t> smem_set{0};
    const TreeCut c = tree_cut(M, D);
    const int64_t units = (int64_t)N * H;
    cudaError_t e = allow_dynamic_smem(decode_tree_kernel<Tin, D>, 227 * 1024, smem_set);
    if (e != cudaSuccess) return e;
    decode_tree_kernel<Tin, D><<<(unsigned)((units + c.units - 1) / c.units), c.threads * c.units,
                                 tree_unit_bytes(M, D) * c.units, stream>>>(
        static_cast<const Tin *>(q), static_cast<const Tin *>(k), static_cast<const Tin *>(v), g, beta,
        state, parent, units, M, H, c.threads, c.nodes, static_cast<Tin *>(out));
    count_launches(1);
    return cudaGetLastError();
}

template <int D, int TILES>
cudaError_t run_tree_tc(const void *q, const void *k, const void *v, const float *g, const float *beta,
                        const float *state, const int32_t *parent, int32_t N, int32_t M, int32_t H,
                        void *out, cudaStream_t stream) {
    using C = TcCfg<D, TILES>;
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = allow_dynamic_smem(decode_tree_tc_kernel<D, TILES>, C::smem(8 * TILES), smem_set);
    if (e != cudaSuccess) return e;
    decode_tree_tc_kernel<D, TILES><<<(unsigned)N * (unsigned)H, C::THREADS, C::smem(M), stream>>>(
        static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(k),
        static_cast<const __nv_bfloat16 *>(v), g, beta, state, parent, M, H,
        static_cast<__nv_bfloat16 *>(out));
    count_launches(1);
    return cudaGetLastError();
}

// row tiles of eight nodes, as few as hold M
template <int D>
cudaError_t run_tree_tiles(const void *q, const void *k, const void *v, const float *g, const float *beta,
                           const float *state, const int32_t *parent, int32_t N, int32_t M, int32_t H,
                           void *out, cudaStream_t stream) {
    if (M <= 8) return run_tree_tc<D, 1>(q, k, v, g, beta, state, parent, N, M, H, out, stream);
    if (M <= 16) return run_tree_tc<D, 2>(q, k, v, g, beta, state, parent, N, M, H, out, stream);
    if (M <= 32) return run_tree_tc<D, 4>(q, k, v, g, beta, state, parent, N, M, H, out, stream);
    return run_tree_tc<D, 8>(q, k, v, g, beta, state, parent, N, M, H, out, stream);
}

template <typename Tin, int D>
cudaError_t run_commit(const void *k, const void *v, const float *g, const float *beta,
                       const float *state_in, const int32_t *path, const int32_t *accept, int32_t N,
                       int32_t M, int32_t P, int32_t H, float *state_out, cudaStream_t stream) {
    decode_commit_kernel<Tin, D><<<(unsigned)N * (unsigned)H * CommitCfg<D>::SPLIT, 32 * CommitCfg<D>::WARPS, 0,
                                    stream>>>(
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
    if (dt == KDA_BF16 && D == 128) return run_tree_tiles<128>(q, k, v, g, beta, state, parent, N, M, H, out, stream);
    if (dt == KDA_BF16 && D == 64) return run_tree_tiles<64>(q, k, v, g, beta, state, parent, N, M, H, out, stream);
    if (dt == KDA_BF16 && D == 32) return run_tree_tiles<32>(q, k, v, g, beta, state, parent, N, M, H, out, stream);
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
