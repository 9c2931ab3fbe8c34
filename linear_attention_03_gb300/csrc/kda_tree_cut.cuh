// kda_tree_cut.cuh -- how the attention kernels share out their work.  A unit is
// the rows of one sequence and cache head that a CTA takes at once (`groups` units
// per head); its key tiles follow one another on a line, unit after unit, and
// every CTA gets the same run of the line, wherever that begins and ends.  What a
// CTA has of a unit that it does not hold whole goes to the workspace, and a
// second kernel joins it.  The cut depends on the lengths alone, so results repeat.
//
// Units::tiles(len, M) is the tiles of a unit.  With fewer tiles than CTAs each has
// one or none: for a single cache of 501 tokens two per CTA took 12.5 us, one 11.7.
#pragma once

#include "kda_internal.cuh"

namespace kda {

__device__ __forceinline__ int clamped_len(const TreeAttention &a, int64_t n) {
    const int len = a.cache_lens[n];
    const int64_t room = (int64_t)a.max_pages * a.page_size;
    return len < 0 ? 0 : (len > room ? (int)room : len);
}

// a / b of non-negative numbers, in 32 bits where they fit (a third of the latency)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}

// where CTA b's piece of `total` tiles starts
__device__ __forceinline__ int64_t piece_start(int64_t total, int ctas, int b) {
    if (total < ctas) return b < total ? b : total;
    return quotient(total * b, ctas);
}

// The first CTA whose piece starts at `end` or later.
__device__ __forceinline__ int first_past(int64_t total, int ctas, int64_t end) {
    return total < ctas ? (int)end : (int)quotient(end * ctas + total - 1, total);
}

// Where a CTA's piece starts: total tiles of the line, its first tile there, and
// the sequence and unit that hold it.  Each CTA leaves its own in the workspace, with the
// status it found, for the kernel that joins the pieces.
struct Place {
    int64_t total, start, unit0;    // unit0: where the unit starts on the line
    int32_t n, r, len;              // sequence, unit within it, its clamped length
    int32_t status;
};

// The whole block calls it; `buf` holds 34 int64 of shared memory.
template <class Units>
__device__ void find_place(const TreeAttention &a, int groups, int ctas, int b, int64_t *buf, Place &out) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int per_seq = a.H_kv * groups;
    auto scan = [&](int64_t run) {                          // sums up to each lane's
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += x;
        }
        return run;
    };
    if (a.N <= 32) {
        // a sequence per lane, in every warp alike: no barriers (1 us less for a small call)
        const bool real = lane < a.N;
        const int raw = real ? a.cache_lens[lane] : 0, len = real ? clamped_len(a, lane) : 0;
        const int tiles = Units::tiles(len, a.M);
        const int64_t mine = real ? (int64_t)tiles * per_seq : 0, run = scan(mine), begin = run - mine;
        out.status = __any_sync(0xffffffffu, raw != len) ? KDA_DEVICE_BAD_LENGTH : KDA_DEVICE_OK;
        out.total = __shfl_sync(0xffffffffu, run, 31);
        out.start = piece_start(out.total, ctas, b);
        const uint32_t here = __ballot_sync(0xffffffffu, mine > 0 && out.start >= begin && out.start < run);
        const int n = here != 0 ? __ffs(here) - 1 : 0;
        const int its = __shfl_sync(0xffffffffu, tiles, n);
        const int64_t from = __shfl_sync(0xffffffffu, begin, n), r = quotient(out.start - from, its);
        out.n = n;
        out.r = (int32_t)r;
        out.unit0 = from + r * its;
        out.len = __shfl_sync(0xffffffffu, len, n);
        return;
    }
    int64_t sum = 0;
    bool bad = false;
    for (int n = tid; n < a.N; n += blockDim.x) {
        const int len = a.cache_lens[n];
        bad = bad || len < 0 || len > (int64_t)a.max_pages * a.page_size;
        sum += (int64_t)Units::tiles(clamped_len(a, n), a.M) * per_seq;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) buf[warp] = sum;
    out.status = __syncthreads_or(bad) != 0 ? KDA_DEVICE_BAD_LENGTH : KDA_DEVICE_OK;
    int64_t total = 0;
    for (int w = 0; w < warps; ++w) total += buf[w];
    __syncthreads();
    out.total = total;
    const int64_t at = piece_start(total, ctas, b);
    out.start = at;
    if (warp == 0) {
        // one warp walks the sequences, 32 at a time
        int64_t base = 0;
        for (int n0 = 0; n0 < a.N; n0 += 32) {
            const int n = n0 + lane;
            const int len = n < a.N ? clamped_len(a, n) : 0;
            const int64_t mine = n < a.N ? (int64_t)Units::tiles(len, a.M) * per_seq : 0;
            const int64_t run = scan(mine);
            const int64_t begin = base + run - mine;
            if (mine > 0 && at >= begin && at < begin + mine) {
                const int64_t r = quotient(at - begin, Units::tiles(len, a.M));
                buf[0] = n;
                buf[1] = r;
                buf[2] = begin + r * Units::tiles(len, a.M);
                buf[3] = len;
            }
            base += __shfl_sync(0xffffffffu, run, 31);
            if (at < base) break;
        }
    }
    __syncthreads();
    out.n = (int32_t)buf[0];
    out.r = (int32_t)buf[1];
    out.unit0 = buf[2];
    out.len = (int32_t)buf[3];
}

// A CTA's run through its piece: segments are the parts of units in it.
template <class Units> struct CutRun {
    int64_t left;           // tiles still to do
    int32_t n, r, len, t0;  // the current unit and its first tile here
    int32_t tiles;          // tiles of the unit
    __device__ __forceinline__ int count() const { return left < tiles - t0 ? (int)left : tiles - t0; }
    __device__ __forceinline__ void advance(const TreeAttention &a, int groups) {
        left -= count();
        t0 = 0;
        if (++r == a.H_kv * groups) {
            r = 0;
            if (++n < a.N && left > 0) {
                len = clamped_len(a, n);
                tiles = Units::tiles(len, a.M);
            }
        }
    }
};

// The block's threads: the status that the CTAs left.
__device__ __forceinline__ void gather_status(const Place *places, int ctas, int32_t *status) {
    int32_t code = 0;
    for (int i = threadIdx.x; i < ctas; i += blockDim.x) code = max(code, places[i].status);
    const bool timeout = __syncthreads_or(code == KDA_DEVICE_TIMEOUT) != 0;
    const bool page = __syncthreads_or(code == KDA_DEVICE_BAD_PAGE) != 0;
    const bool length = __syncthreads_or(code == KDA_DEVICE_BAD_LENGTH) != 0;
    if (threadIdx.x == 0)
        *status = timeout ? KDA_DEVICE_TIMEOUT : page ? KDA_DEVICE_BAD_PAGE
                  : length ? KDA_DEVICE_BAD_LENGTH : KDA_DEVICE_OK;
}

inline int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
        sms = 152;
    return sms;
}

inline size_t place_bytes(int ctas) { return ((size_t)ctas * sizeof(Place) + 255) / 256 * 256; }

}  // namespace kda
