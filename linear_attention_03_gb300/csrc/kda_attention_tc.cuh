// kda_attention_tc.cuh -- what the tcgen05 attention kernels share: the tile's
// sizes, the tensor maps of the paged cache and of the queries, and the way a row
// of outputs is stored.
#pragma once

#include "kda_internal.cuh"
#include "kda_tc.cuh"

#include <cuda.h>

#include <algorithm>

namespace kda {

constexpr int kTile = 128;                 // rows per row tile, keys per key tile
constexpr float kGrow = 8.f;               // log2 growth of the maximum that rescales the sums
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// 64 bytes of a row, in whole 32-byte sectors where the address allows it
__device__ __forceinline__ void store64(void *to, const uint32_t (&u)[16], bool aligned32) {
    if (aligned32) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                             static_cast<unsigned char *>(to) + 32 * e),
                         "r"(u[8 * e]), "r"(u[8 * e + 1]), "r"(u[8 * e + 2]), "r"(u[8 * e + 3]), "r"(u[8 * e + 4]),
                         "r"(u[8 * e + 5]), "r"(u[8 * e + 6]), "r"(u[8 * e + 7])
                         : "memory");
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            reinterpret_cast<uint4 *>(to)[e] = make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
    }
}

// 32 sums of a row, whole 32-byte sectors (the workspace's rows start at multiples of 32 bytes)
__device__ __forceinline__ void store_sums32(float *to, const float (&o)[32]) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + 8 * e),
                     "r"(__float_as_uint(o[8 * e])), "r"(__float_as_uint(o[8 * e + 1])),
                     "r"(__float_as_uint(o[8 * e + 2])), "r"(__float_as_uint(o[8 * e + 3])),
                     "r"(__float_as_uint(o[8 * e + 4])), "r"(__float_as_uint(o[8 * e + 5])),
                     "r"(__float_as_uint(o[8 * e + 6])), "r"(__float_as_uint(o[8 * e + 7]))
                     : "memory");
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess || q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

inline bool make_map(CUtensorMap *map, const void *base, const cuuint64_t (&dims)[4], const cuuint64_t (&strides)[3],
              const cuuint32_t (&box)[4]) {
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, ones,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The cache as groups of eight rows: [groups][D/64 halves][8 rows][64], so that
// a box lands as whole 128-byte-swizzle blocks, the halves of a row next to
// each other.
inline bool cache_map(CUtensorMap *map, const void *base, const TreeAttention &a, int D, int box) {
    const cuuint64_t groups = (cuuint64_t)a.num_pages * a.H_kv * a.page_size / 8;
    return make_map(map, base, {64, 8, (cuuint64_t)(D / 64), groups}, {(cuuint64_t)D * 2, 128, (cuuint64_t)D * 16},
                    {64, 8, (cuuint32_t)(D / 64), (cuuint32_t)(box / 8)});
}
// The queries [N * M][H][D]: a row tile's nodes, the query heads of one cache head, half a row.
inline bool query_map(CUtensorMap *map, const TreeAttention &a, int D, int nodes) {
    return make_map(map, a.q, {64, (cuuint64_t)a.H, (cuuint64_t)(D / 64), (cuuint64_t)a.N * a.M},
                    {(cuuint64_t)D * 2, 128, (cuuint64_t)a.H * D * 2},
                    {64, (cuuint32_t)(a.H / a.H_kv), 1, (cuuint32_t)nodes});
}
// as many whole nodes as 128 rows hold (their query heads are G rows each)
inline int nodes_per_tile(int M, int H, int H_kv) { return std::min(M, kTile / (H / H_kv)); }

}  // namespace kda
