// kda_norm_rope.cu -- RMS norm of every query and key head and the rotation by
// its position, in one pass (kda_head_norm_rope): what a softmax layer does to
// its projections before its attention.
//
//     y = x / sqrt(mean_c x_c^2 + eps) * w
//     (y_a, y_b) <- (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = position * inv_freq[i]
//
// for the pairs i of the first 2 n_freq channels: (i, i + n_freq), or (2 i, 2 i + 1)
// interleaved.  Every element is read and written once, so HBM bounds it.
//
// A lane holds 16 channels of a row, both members of its pairs, so that the
// rotation needs no exchange and the norm one reduction over D / 16 lanes.  A warp
// takes rows of one token: it forms the token's angles once, two to a lane, and
// keeps the cosines and sines of its channels in registers for all its rows.
//
// Angles: position * inv_freq / (2 pi) modulo 1, as a 64-bit fraction of a turn.
// An fp32 inv_freq is a 24-bit integer times a power of two; its product with
// 2^64 / (2 pi) gives the fraction per position, and the product with the position
// wraps around modulo one turn by itself.  The error is 2^-33 turns at position
// 2^31 for inv_freq <= 1, where an angle in fp32 is off by 0.016 rad at position 262,144.
#include "kda_internal.cuh"

namespace kda {
namespace {

struct NormRope {
    const void *q, *k;
    void *q_out, *k_out;
    int64_t q_stride, k_stride, q_out_stride, k_out_stride;     // elements from a token to the next
    const int32_t *positions;
    const float *inv_freq, *q_weight, *k_weight;
    int64_t T;
    int32_t H, H_kv, n_freq;
    int32_t slices, per_slice;      // warps of a token, rows of each
    float eps;
};

enum { HALVES = 0, PAIRS = 1, ANY = 2 };    // how the pairs lie: whole groups of eight apart, side by side, any halves

// inv_freq / (2 pi) modulo 1 in units of 2^-64
__device__ __forceinline__ uint64_t turns_per_position(float inv_freq) {
    constexpr uint64_t C = 2935890503282001226ull;              // 2^64 / (2 pi)
    const uint32_t bits = __float_as_uint(inv_freq), ex = bits >> 23 & 255u;
    const uint64_t m = ex == 0 ? bits & 0x7fffffu : (bits & 0x7fffffu) | 0x800000u;
    const int shift = 150 - (ex == 0 ? 1 : (int)ex);            // inv_freq = m 2^-shift
    const uint64_t lo = m * C, hi = __umul64hi(m, C);
    uint64_t f;
    if (shift <= 0) f = shift > -64 ? lo << -shift : 0;
    else if (shift < 64) f = lo >> shift | hi << (64 - shift);
    else f = shift < 128 ? hi >> (shift - 64) : 0;
    return (bits >> 31) != 0 ? 0 - f : f;
}

// cos and sin of `turns` (units of 2^-64 of a turn)
__device__ __forceinline__ float2 cos_sin(uint64_t turns) {
    // the nearest quarter and what is left of it, at most 1/4 of pi: its fp32 form is good to 2^-27 turns
    const uint32_t t = (uint32_t)(turns >> 32), quarter = (t + 0x20000000u) >> 30;
    const int64_t rest = (int64_t)(turns - ((uint64_t)quarter << 62));
    float s, c;
    sincospif(2.f * ((float)(int32_t)(rest >> 32) * 0x1p-32f), &s, &c);
    const float a = (quarter & 1) != 0 ? -s : c, b = (quarter & 1) != 0 ? c : s;
    return (quarter & 2) != 0 ? make_float2(-a, -b) : make_float2(a, b);
}

template <typename Tin, int D, int MODE>
__global__ void __launch_bounds__(256)
norm_rope_kernel(const NormRope a) {
    constexpr int LANES = D / 16, ROWS = 32 / LANES;            // lanes of a row, rows of a warp at once
    constexpr int AT_ONCE = sizeof(Tin) == 2 ? 2 : 1;           // rows whose loads are on their way together
    __shared__ float2 angles[8][D / 2];
    __shared__ float rows[MODE == ANY ? 8 : 1][MODE == ANY ? ROWS * D : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = lane % LANES;
    const int64_t unit = (int64_t)blockIdx.x * 8 + warp;
    const int64_t token = unit / a.slices;
    if (token >= a.T) return;
    const int row0 = (int)(unit - token * a.slices) * a.per_slice;
    const int end = min(row0 + a.per_slice, a.H + a.H_kv);
    // the lane's two groups of eight channels
    const int half = a.n_freq / 8;                              // HALVES: groups of a half
    int g0 = 2 * j, g1 = 2 * j + 1;
    bool turned = MODE == PAIRS;
    if (MODE == HALVES && j < half) {
        g0 = j;
        g1 = j + half;
        turned = true;
    }
    auto source = [&](int r) {
        return r < a.H ? static_cast<const Tin *>(a.q) + token * a.q_stride + (int64_t)r * D
                       : static_cast<const Tin *>(a.k) + token * a.k_stride + (int64_t)(r - a.H) * D;
    };
    float x[AT_ONCE][16];
    auto load = [&](int first) {
#pragma unroll
        for (int y = 0; y < AT_ONCE; ++y) {
            const int r = min(first + y * ROWS + lane / LANES, end - 1);
            const Tin *p = source(r);
            float u[8], v[8];
            Elem<Tin>::load8(p + 8 * g0, u);
            Elem<Tin>::load8(p + 8 * g1, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[y][e] = u[e];
                x[y][8 + e] = v[e];
            }
        }
    };
    load(row0);

    const int64_t position = a.positions[token];
    for (int i = lane; i < a.n_freq; i += 32)
        angles[warp][i] = cos_sin(turns_per_position(a.inv_freq[i]) * (uint64_t)position);
    for (int i = a.n_freq + lane; i < D / 2; i += 32) angles[warp][i] = make_float2(1.f, 0.f);
    __syncwarp();
    float co[8], si[8];
    if (MODE != ANY) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 cs = turned ? angles[warp][8 * j + e] : make_float2(1.f, 0.f);
            co[e] = cs.x;
            si[e] = cs.y;
        }
    }

    for (int first = row0; first < end; first += ROWS * AT_ONCE) {
        if (first > row0) load(first);
#pragma unroll
        for (int y = 0; y < AT_ONCE; ++y) {
            const int r = first + y * ROWS + lane / LANES;
            const bool real = r < end, query = r < a.H;
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) sum = fmaf(x[y][e], x[y][e], sum);
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float by = __frsqrt_rn(fmaf(sum, 1.f / D, a.eps));
            const float *w = query ? a.q_weight : a.k_weight;
            float n[16];
            if (w != nullptr) {
                float w0[8], w1[8];
                Elem<float>::load8(w + 8 * g0, w0);
                Elem<float>::load8(w + 8 * g1, w1);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    n[e] = x[y][e] * by * w0[e];
                    n[8 + e] = x[y][8 + e] * by * w1[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) n[e] = x[y][e] * by;
            }
            float u[8], v[8];
            if (MODE == PAIRS) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float z0 = n[2 * e], z1 = n[2 * e + 1];
                    const float r0 = z0 * co[e] - z1 * si[e], r1 = z1 * co[e] + z0 * si[e];
                    if (e < 4) {
                        u[2 * e] = r0;
                        u[2 * e + 1] = r1;
                    } else {
                        v[2 * e - 8] = r0;
                        v[2 * e - 7] = r1;
                    }
                }
            } else if (MODE == HALVES) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    u[e] = n[e] * co[e] - n[8 + e] * si[e];
                    v[e] = n[8 + e] * co[e] + n[e] * si[e];
                }
            } else {
                // partners anywhere in the row: through shared memory
                float *row = rows[warp] + lane / LANES * D;
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 16; ++e) row[16 * j + e] = n[e];
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int c = 16 * j + e;
                    float z = n[e];
                    if (c < 2 * a.n_freq) {
                        const bool low = c < a.n_freq;
                        const float2 cs = angles[warp][low ? c : c - a.n_freq];
                        const float other = row[low ? c + a.n_freq : c - a.n_freq];
                        z = low ? z * cs.x - other * cs.y : z * cs.x + other * cs.y;
                    }
                    if (e < 8) u[e] = z;
                    else v[e - 8] = z;
                }
            }
            if (real) {
                Tin *p = query ? static_cast<Tin *>(a.q_out) + token * a.q_out_stride + (int64_t)r * D
                               : static_cast<Tin *>(a.k_out) + token * a.k_out_stride + (int64_t)(r - a.H) * D;
                Elem<Tin>::store8(p + 8 * g0, u);
                Elem<Tin>::store8(p + 8 * g1, v);
            }
        }
    }
}

template <typename Tin, int D> cudaError_t run(NormRope a, int mode, cudaStream_t stream) {
    constexpr int ROWS = 32 / (D / 16), AT_ONCE = sizeof(Tin) == 2 ? 2 : 1;
    int dev = 0, sms = 152;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        sms = 152;
    // A token's rows in as few warps as still fill the GPU: each forms the token's angles anew.
    const int rows = a.H + a.H_kv, passes = (rows + ROWS - 1) / ROWS;
    int per = passes;
    while (per > AT_ONCE && a.T * ((passes + per - 1) / per) < (int64_t)sms * 32) per = (per + 1) / 2;
    a.per_slice = per * ROWS;
    a.slices = (rows + a.per_slice - 1) / a.per_slice;
    const int64_t blocks = (a.T * a.slices + 7) / 8;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    if (mode == HALVES) norm_rope_kernel<Tin, D, HALVES><<<(unsigned)blocks, 256, 0, stream>>>(a);
    else if (mode == PAIRS) norm_rope_kernel<Tin, D, PAIRS><<<(unsigned)blocks, 256, 0, stream>>>(a);
    else norm_rope_kernel<Tin, D, ANY><<<(unsigned)blocks, 256, 0, stream>>>(a);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_head_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                  const int32_t *positions, const float *inv_freq, int32_t n_freq,
                                  const float *q_weight, const float *k_weight, int64_t T, int32_t H,
                                  int32_t H_kv, int32_t D, kda_dtype dt, bool interleaved, float eps, void *q_out,
                                  int64_t q_out_stride, void *k_out, int64_t k_out_stride, cudaStream_t stream) {
    const NormRope a{q, k, q_out, k_out, q_stride, k_stride, q_out_stride, k_out_stride, positions, inv_freq,
                     q_weight, k_weight, T, H, H_kv, n_freq, 0, 0, eps};
    const int mode = interleaved ? PAIRS : n_freq % 8 == 0 ? HALVES : ANY;
#define KDA_RUN(TIN)                                    \
    switch (D) {                                        \
    case 16: return run<TIN, 16>(a, mode, stream);      \
    case 32: return run<TIN, 32>(a, mode, stream);      \
    case 64: return run<TIN, 64>(a, mode, stream);      \
    case 128: return run<TIN, 128>(a, mode, stream);    \
    default: return cudaErrorInvalidValue;              \
    }
    if (dt == KDA_BF16) { KDA_RUN(__nv_bfloat16) }
    KDA_RUN(float)
#undef KDA_RUN
}

}  // namespace kda
