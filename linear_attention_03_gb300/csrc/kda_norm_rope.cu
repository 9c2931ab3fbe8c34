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
//
// Measured (graphs of the call on two inputs): 32,388 tokens of 96 + 8 heads of 128
// out of a projection, bf16, 1.72 GB: 274 us, 6.3 TB/s, 92% of a copy's rate (269 us
// interleaved); 16,000 tokens in fp32 261 us, 6.5 TB/s; one token 4.2 us.  Half of the pairs
// turned: 300 us in halves, 274 interleaved; 17 halves, whose partners go through shared
// memory with bank conflicts (16 channels from lane to lane): 818 us, fp32 553.  On the way
// (bf16): elements unpacked at their load 333 us, loaded as they lie 288, paired fp32
// arithmetic 276.  Two rows per lane at three CTAs an SM: four CTAs (64 registers,
// spills) take 337, three rows 317, four rows at two CTAs 280, one row at five 374; in
// fp32 two rows at two CTAs 262, one row at three 272.
#include "kda_internal.cuh"
#include "kda_tc.cuh"

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

// 16 channels as pairs of floats
__device__ __forceinline__ void unpack(const uint4 (&raw)[2], float2 (&x)[8]) {
    const uint32_t w[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = tc::unpack_bf16x2(w[i]);
}
__device__ __forceinline__ void unpack(const uint4 (&raw)[4], float2 (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = make_float2(__uint_as_float(raw[i].x), __uint_as_float(raw[i].y));
        x[2 * i + 1] = make_float2(__uint_as_float(raw[i].z), __uint_as_float(raw[i].w));
    }
}
// eight channels
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float2 *x) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(tc::pack_bf16x2(x[0].x, x[0].y), tc::pack_bf16x2(x[1].x, x[1].y),
                                               tc::pack_bf16x2(x[2].x, x[2].y), tc::pack_bf16x2(x[3].x, x[3].y));
}
__device__ __forceinline__ void store8(float *p, const float2 *x) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
}

constexpr int kAtOnce = 2;                                      // rows whose loads are on their way together
template <typename Tin> constexpr int kCtas = sizeof(Tin) == 2 ? 3 : 2;     // resident on an SM

// Which of a lane's 16 channels lie from `from` on and are finite numbers.  (A call: its loads in the loop's own code
// take registers from it, and partly turned bf16 rows 3 to 8% longer.)
template <typename Tin> __device__ __noinline__ uint32_t finite_from(const Tin *x, int g0, int g1, int from) {
    uint32_t bits = 0;
    for (int e = 0; e < 16; ++e) {
        const int c = 8 * (e < 8 ? g0 : g1) + e % 8;
        if (c >= from && fabsf(static_cast<float>(x[c])) < INFINITY) bits |= 1u << e;
    }
    return bits;
}

// PART: some channels are not turned.
template <typename Tin, int D, int MODE, bool PART>
__global__ void __launch_bounds__(256, kCtas<Tin>)
norm_rope_kernel(const NormRope a) {
    constexpr int LANES = D / 16, ROWS = 32 / LANES;            // lanes of a row, rows of a warp at once
    constexpr int AT_ONCE = kAtOnce, WORDS = sizeof(Tin) / 2;      // 16-byte words of eight channels
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
    if (MODE == PAIRS || (MODE == HALVES && j < half)) {
        g0 = j;
        g1 = j + (MODE == PAIRS ? LANES : half);
    } else if (MODE == HALVES) {                                // neighbours over the lanes here, too
        g0 = j + half;
        g1 = j + LANES;
    }
    auto source = [&](int r) {
        return r < a.H ? static_cast<const Tin *>(a.q) + token * a.q_stride + (int64_t)r * D
                       : static_cast<const Tin *>(a.k) + token * a.k_stride + (int64_t)(r - a.H) * D;
    };
    uint4 raw[AT_ONCE][2 * WORDS];                              // as they lie: half the registers in bf16
    // (by plain loads: in place the rows are written here, too, which the read-only path does not allow)
    auto load = [&](int first) {
#pragma unroll
        for (int y = 0; y < AT_ONCE; ++y) {
            const uint4 *p = reinterpret_cast<const uint4 *>(source(min(first + y * ROWS + lane / LANES, end - 1)));
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                raw[y][i] = p[WORDS * g0 + i];
                raw[y][WORDS + i] = p[WORDS * g1 + i];
            }
        }
    };
    load(row0);

    const int64_t position = a.positions[token];
    for (int i = lane; i < a.n_freq; i += 32)
        angles[warp][i] = cos_sin(turns_per_position(a.inv_freq[i]) * (uint64_t)position);
    for (int i = a.n_freq + lane; i < D / 2; i += 32) angles[warp][i] = make_float2(1.f, 0.f);
    __syncwarp();
    // of the lane's eight pairs: HALVES: channel e of both groups; PAIRS: four of each group
    float2 co[4], si[4];
    if (MODE != ANY) {
        float2 cs[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = MODE == PAIRS ? 4 * (e < 4 ? g0 : g1) + e % 4 : 8 * j + e;
            cs[e] = MODE == PAIRS || j < half ? angles[warp][i] : make_float2(1.f, 0.f);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            co[e] = make_float2(cs[2 * e].x, cs[2 * e + 1].x);
            si[e] = make_float2(cs[2 * e].y, cs[2 * e + 1].y);
        }
    }

    for (int first = row0; first < end; first += ROWS * AT_ONCE) {
        if (first > row0) load(first);
#pragma unroll
        for (int y = 0; y < AT_ONCE; ++y) {
            const int r = first + y * ROWS + lane / LANES;
            const bool real = r < end, query = r < a.H;
            float2 n[8];                                        // first group, second group
            unpack(raw[y], n);
            float2 two = tc::f2mul(n[0], n[0]);
#pragma unroll
            for (int e = 1; e < 8; ++e) two = tc::f2fma(n[e], n[e], two);
            float sum = two.x + two.y;
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float by = __frsqrt_rn(fmaf(sum, 1.f / D, a.eps));
#pragma unroll
            for (int e = 0; e < 8; ++e) n[e] = tc::f2mul(n[e], make_float2(by, by));
            const float *w = query ? a.q_weight : a.k_weight;
            if (w != nullptr) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float4 z = __ldg(reinterpret_cast<const float4 *>(w + 8 * (e < 4 ? g0 : g1)) + e % 4 / 2);
                    n[e] = tc::f2mul(n[e], make_float2(z.x, z.y));
                    n[e + 1] = tc::f2mul(n[e + 1], make_float2(z.z, z.w));
                }
            }
            if (MODE == PAIRS) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float c = e & 1 ? co[e / 2].y : co[e / 2].x, z = e & 1 ? si[e / 2].y : si[e / 2].x;
                    n[e] = tc::f2fma(n[e], make_float2(c, c), tc::f2mul(make_float2(n[e].y, n[e].x), make_float2(-z, z)));
                }
            } else if (MODE == HALVES) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 lo = n[e], hi = n[4 + e], minus = make_float2(-si[e].x, -si[e].y);
                    n[e] = tc::f2fma(lo, co[e], tc::f2mul(hi, minus));
                    n[4 + e] = tc::f2fma(hi, co[e], tc::f2mul(lo, si[e]));
                }
            } else {
                // partners anywhere in the row: through shared memory
                float *row = rows[warp] + lane / LANES * D;
                float *mine = reinterpret_cast<float *>(n);
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 16; ++e) row[16 * j + e] = mine[e];
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int c = 16 * j + e;
                    if (c < 2 * a.n_freq) {
                        const bool low = c < a.n_freq;
                        const float2 cs = angles[warp][low ? c : c - a.n_freq];
                        const float other = row[low ? c + a.n_freq : c - a.n_freq];
                        mine[e] = low ? mine[e] * cs.x - other * cs.y : mine[e] * cs.x + other * cs.y;
                    }
                }
            }
            if (PART && MODE != ANY && by == 0.f) {
                // a row with an infinity: its finite channels are zeros, but the rotation by nothing, a factor of zero,
                // carries a NaN over
                const uint32_t finite = finite_from(source(min(r, end - 1)), g0, g1, 2 * a.n_freq);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if ((finite >> e & 1) != 0) (e & 1 ? n[e / 2].y : n[e / 2].x) = 0.f;
            }
            if (real) {
                Tin *p = query ? static_cast<Tin *>(a.q_out) + token * a.q_out_stride + (int64_t)r * D
                               : static_cast<Tin *>(a.k_out) + token * a.k_out_stride + (int64_t)(r - a.H) * D;
                store8(p + 8 * g0, n);
                store8(p + 8 * g1, n + 4);
            }
        }
    }
}

template <typename Tin, int D> cudaError_t run(NormRope a, int mode, cudaStream_t stream) {
    constexpr int ROWS = 32 / (D / 16), AT_ONCE = kAtOnce;
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
    auto launch = [&](auto kernel) { kernel<<<(unsigned)blocks, 256, 0, stream>>>(a); };
    const bool part = 2 * a.n_freq < D;
    if (mode == HALVES) part ? launch(norm_rope_kernel<Tin, D, HALVES, true>) : launch(norm_rope_kernel<Tin, D, HALVES, false>);
    else if (mode == PAIRS) part ? launch(norm_rope_kernel<Tin, D, PAIRS, true>) : launch(norm_rope_kernel<Tin, D, PAIRS, false>);
    else launch(norm_rope_kernel<Tin, D, ANY, true>);
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
