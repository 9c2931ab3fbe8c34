// kda_prefix_cut.cuh -- attention behind shared prefixes: how its work is shared
// out, and how its pieces meet.
//
// A prefix's rows are those of all its sequences' nodes, one after another, so a
// unit is a run of rows of one prefix and cache head that a CTA takes at once.  The
// units' key tiles follow one another on a line that is cut into even pieces, as in
// kda_tree_cut.cuh; what a CTA has of a unit that it does not hold whole goes to the
// workspace.  The sequences' own keys are the tree kernels' work, whose sums wait in
// the workspace row by row (RowSums): whoever has the whole of a prefix's rows joins
// them at once, and prefix_join_kernel does it for the others.
#pragma once

#include "kda_internal.cuh"
#include "kda_tc.cuh"
#include "kda_tree_cut.cuh"

namespace kda {

// Prefix p: sequences seq0 .. seq0 + seqs - 1, keys 0 .. len - 1; what is out of range counts as empty.
struct Prefix {
    int32_t seq0, seqs, len;
    int32_t status;                 // findings
};
__device__ __forceinline__ Prefix prefix_at(const PrefixAttention &a, int p) {
    const int s0 = a.seqs[p], s1 = a.seqs[p + 1], len = a.lens[p];
    const int64_t room = (int64_t)a.max_pages * a.t.page_size;
    Prefix x{0, 0, len, 0};
    if (len < 0 || len > room) {
        x.len = len < 0 ? 0 : (int)room;
        x.status = finding(KDA_DEVICE_BAD_LENGTH);
    }
    if (s0 >= 0 && s1 >= s0 && s1 <= a.t.N) {
        x.seq0 = s0;
        x.seqs = s1 - s0;
    } else {
        x.status |= finding(KDA_DEVICE_BAD_OFFSETS);
    }
    return x;
}

// How rows become units: a unit has `tiles` row tiles of `tile` rows, `used` of which hold rows.
struct RowUnits {
    int32_t tiles, tile, used;
    __device__ __forceinline__ int rows() const { return tiles * used; }
    __device__ __forceinline__ int slots() const { return tiles * tile; }
};

struct PrefixPlace {
    int64_t total, start, unit0;    // tiles of the line, the piece's first one, where its unit starts
    int32_t p, r;                   // the prefix and the unit within it
    int32_t tiles, groups, seq0, rows, len;     // of the unit's prefix, as in PrefixRun: the join needs no table
    int32_t status;                 // findings
};

// A CTA's run through its piece.
template <int KEYS> struct PrefixRun {
    int64_t left;                   // tiles still to do
    int32_t p, r, t0;               // the current unit and its first tile here
    int32_t tiles, groups, units;   // tiles of the unit, units per cache head, units of the prefix
    int32_t seq0, rows, len;        // the prefix's first sequence, its rows of a cache head, its keys
    __device__ __forceinline__ int count() const { return left < tiles - t0 ? (int)left : tiles - t0; }
    __device__ __forceinline__ int32_t load(const PrefixAttention &a, const RowUnits &u) {
        const Prefix x = prefix_at(a, p);
        seq0 = x.seq0;
        len = x.len;
        rows = x.seqs * a.t.M * (a.t.H / a.t.H_kv);
        groups = (rows + u.rows() - 1) / u.rows();
        units = groups * a.t.H_kv;
        tiles = (len + KEYS - 1) / KEYS;
        return x.status;
    }
    __device__ __forceinline__ int64_t line() const { return (int64_t)tiles * units; }
    __device__ __forceinline__ void advance(const PrefixAttention &a, const RowUnits &u) {
        left -= count();
        t0 = 0;
        if (++r < units || left <= 0) return;
        r = 0;
        do {
            ++p;
            load(a, u);
        } while (line() == 0);      // (there is one: tiles are left)
    }
};

// Where CTA b's piece starts.  Each warp walks the prefixes, a lane each, for itself.
template <int KEYS>
__device__ __forceinline__ PrefixPlace find_prefix_place(const PrefixAttention &a, const RowUnits &u, int ctas, int b) {
    const int lane = threadIdx.x & 31;
    PrefixPlace out{0, 0, 0, 0, 0, 1, 1, 0, 0, 0, 0};
    int32_t status = 0;
    PrefixRun<KEYS> it;
    auto one = [&](int p) -> int64_t {
        it.p = p;
        if (p >= a.P) return 0;
        status |= it.load(a, u);
        return it.line();
    };
    int64_t mine = 0;
    for (int p0 = 0; p0 < a.P; p0 += 32) {
        mine = one(p0 + lane);
        int64_t sum = mine;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        out.total += sum;
    }
    out.status = (int32_t)__reduce_or_sync(0xffffffffu, (unsigned)status);
    out.start = out.unit0 = piece_start(out.total, ctas, b);
    int64_t base = 0;
    for (int p0 = 0; p0 < a.P; p0 += 32) {
        if (a.P > 32) mine = one(p0 + lane);
        int64_t run = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += x;
        }
        const int64_t begin = base + run - mine;
        const uint32_t here = __ballot_sync(0xffffffffu, mine > 0 && out.start >= begin && out.start < begin + mine);
        if (here != 0) {
            const int src = __ffs(here) - 1;
            const int64_t from = __shfl_sync(0xffffffffu, begin, src);
            out.p = p0 + src;
            out.tiles = __shfl_sync(0xffffffffu, it.tiles, src);
            out.groups = __shfl_sync(0xffffffffu, it.groups, src);
            out.seq0 = __shfl_sync(0xffffffffu, it.seq0, src);
            out.rows = __shfl_sync(0xffffffffu, it.rows, src);
            out.len = __shfl_sync(0xffffffffu, it.len, src);
            out.r = (int32_t)quotient(out.start - from, out.tiles);
            out.unit0 = from + (int64_t)out.r * out.tiles;
            break;
        }
        base += __shfl_sync(0xffffffffu, run, 31);
    }
    return out;
}

template <int KEYS>
__device__ __forceinline__ PrefixRun<KEYS> prefix_run(const PrefixAttention &a, const PrefixPlace &at, int64_t stop) {
    PrefixRun<KEYS> run;
    run.left = stop - at.start;
    run.p = at.p;
    run.r = at.r;
    run.t0 = (int32_t)(at.start - at.unit0);
    run.tiles = at.tiles;
    run.groups = at.groups;
    run.units = at.groups * a.t.H_kv;
    run.seq0 = at.seq0;
    run.rows = at.rows;
    run.len = at.len;
    return run;
}

// The join of a prefix's sums with those of the sequence's own keys: what each is multiplied by.
// EXP2: maxima are times log2 e.  Rows of no node (own sum below zero) become zeros.
template <bool EXP2> struct RowJoin {
    float prefix, own, lse;
    bool none;
    __device__ __forceinline__ RowJoin(float top, float sum, float own_top, float own_sum) {
        none = own_sum < 0.f;
        const float m = fmaxf(top, own_top), from = m == -INFINITY ? 0.f : m;
        const float x = EXP2 ? exp2f(top - from) : expf(top - from);
        const float y = EXP2 ? exp2f(own_top - from) : expf(own_top - from);
        const float z = x * sum + y * own_sum;
        prefix = none ? 0.f : x / z;
        own = none ? 0.f : y / z;
        lse = none ? -INFINITY : EXP2 ? (m + log2f(z)) * 0.6931471805599453f : m + logf(z);
    }
    __device__ __forceinline__ float4 operator()(float4 o, float4 own_o) const {
        if (none) return make_float4(0.f, 0.f, 0.f, 0.f);
        return make_float4(prefix * o.x + own * own_o.x, prefix * o.y + own * own_o.y, prefix * o.z + own * own_o.z,
                           prefix * o.w + own * own_o.w);
    }
};

__device__ __forceinline__ void store_out4(float *p, float4 o) { *reinterpret_cast<float4 *>(p) = o; }
__device__ __forceinline__ void store_out4(__nv_bfloat16 *p, float4 o) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(tc::pack_bf16x2(o.x, o.y), tc::pack_bf16x2(o.z, o.w));
}

// The kernels' work space: a place per CTA, then two slots per CTA for pieces of units: the rows' D
// sums one row after another, the rows' maxima, their sums of weights.
struct PrefixShape {
    RowUnits units;
    int32_t ctas;
    PrefixPlace *places;
    float *part;
};
inline size_t prefix_place_bytes(int ctas) { return ((size_t)ctas * sizeof(PrefixPlace) + 255) / 256 * 256; }
inline size_t prefix_part_bytes(int ctas, int slots, int D) { return (size_t)ctas * 2 * slots * (D + 2) * 4; }

// Small blocks, four sums of a row to a thread: a unit that is cut into many pieces has to be read
// by many SMs at once, and a block's time is the latency of its few reads (15 us for 64 sequences behind
// 65,001 tokens, whose 152 pieces are 20 MB; 23 us where three prefixes' pieces are).  Two rows to a thread, or more
// rows to a block one after another, take the same to 2% longer for many units and longer for few.
constexpr int kJoinThreads = 128;
template <int D> constexpr int kJoinRows = kJoinThreads * 4 / D;        // rows at a time

// Block (b, y), 0 < b < ctas: the cut between CTAs b - 1 and b, kJoinRows rows of its unit, when
// that is the unit's first cut.  Blocks (0, y): the status.  Block (ctas + n, y): sequence n's rows,
// when no prefix reaches them: their own sums alone.
template <typename Tout, int D, int KEYS, bool EXP2>
__global__ void __launch_bounds__(kJoinThreads)
prefix_join_kernel(const PrefixAttention a, const PrefixShape sh) {
    const int b = blockIdx.x, G = a.t.H / a.t.H_kv, tid = threadIdx.x;
    Tout *out = static_cast<Tout *>(a.t.out);
    tc::wait_prerequisites();
    if (b == 0) {
        if (blockIdx.y != 0) return;
        int32_t mine = 0;
        for (int i = tid; i < sh.ctas; i += kJoinThreads) mine |= sh.places[i].status;
        const int32_t all = all_findings(mine);
        // (the word holds what was found with the sequences' own keys)
        if (tid == 0 && all != 0) *a.t.status = reported(all | finding(*a.t.status));
        return;
    }
    if (b >= sh.ctas) {
        if (blockIdx.y >= 8) return;
        const int n = b - sh.ctas;
        bool covered = false;
        for (int p = tid; p < a.P; p += kJoinThreads) {
            const Prefix x = prefix_at(a, p);
            covered = covered || (x.len > 0 && n >= x.seq0 && n < x.seq0 + x.seqs);
        }
        if (__syncthreads_or(covered) != 0) return;
        const int64_t rows = (int64_t)a.t.M * a.t.H, items = rows * (D / 4);
        for (int64_t i = (int64_t)blockIdx.y * kJoinThreads + tid; i < items; i += (int64_t)min(gridDim.y, 8u) * kJoinThreads) {
            const int64_t row = n * rows + i / (D / 4);
            const int c = (int)(i % (D / 4)) * 4;
            const RowJoin<EXP2> join(-INFINITY, 0.f, a.t.rows.top[row], a.t.rows.sum[row]);
            store_out4(out + row * D + c,
                       join(make_float4(0.f, 0.f, 0.f, 0.f), *reinterpret_cast<const float4 *>(a.t.rows.o + row * D + c)));
            if (c == 0 && a.t.lse != nullptr) a.t.lse[row] = join.lse;
        }
        return;
    }
    const PrefixPlace p = sh.places[b];
    const int64_t before = sh.places[b - 1].start;
    if (p.start >= p.total || p.unit0 == p.start || before > p.unit0) return;
    const int parts = first_past(p.total, sh.ctas, p.unit0 + p.tiles) - (b - 1), slots = sh.units.slots();
    const int h = p.r / p.groups, row0 = p.r % p.groups * sh.units.rows();
    // part i is CTA b - 1 + i's: its last segment for the first, its first one after that
    auto part_of = [&](int i) { return sh.part + (size_t)(2 * (b - 1 + i) + (i == 0 ? 1 : 0)) * slots * (D + 2); };
    const int c = tid % (D / 4) * 4;
    const int lr = blockIdx.y * kJoinRows<D> + tid / (D / 4);
    const int in_tile = lr % sh.units.tile, row = row0 + lr / sh.units.tile * sh.units.used + in_tile;
    if (lr >= slots || in_tile >= sh.units.used || row >= p.rows) return;
    const int64_t o_row = ((int64_t)p.seq0 * a.t.M + row / G) * a.t.H + h * G + row % G;
    const float own_top = a.t.rows.top[o_row], own_sum = a.t.rows.sum[o_row];
    const float4 own = *reinterpret_cast<const float4 *>(a.t.rows.o + o_row * D + c);
    float top = -INFINITY, sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < parts; i0 += 4) {
        // four parts at a time, so that their reads are under way together
        float x[4], z[4];
        float4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float *q = part_of(min(i0 + i, parts - 1));
            x[i] = i0 + i < parts ? q[(size_t)slots * D + lr] : -INFINITY;
            z[i] = q[(size_t)slots * D + slots + lr];
            v[i] = *reinterpret_cast<const float4 *>(q + (size_t)lr * D + c);
        }
        const float was = top;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, x[i]);
        const float from = top == -INFINITY ? 0.f : top, shrink = EXP2 ? exp2f(was - from) : expf(was - from);
        sum *= shrink;
        o.x *= shrink; o.y *= shrink; o.z *= shrink; o.w *= shrink;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i0 + i < parts) {
                const float w = EXP2 ? exp2f(x[i] - from) : expf(x[i] - from);
                sum += w * z[i];
                o.x += w * v[i].x; o.y += w * v[i].y;
                o.z += w * v[i].z; o.w += w * v[i].w;
            }
        }
    }
    const RowJoin<EXP2> join(top, sum, own_top, own_sum);
    store_out4(out + o_row * D + c, join(o, own));
    if (c == 0 && a.t.lse != nullptr) a.t.lse[o_row] = join.lse;
}

// Launched to overlap the kernel before it, whose results it waits for.
template <typename Tout, int D, int KEYS, bool EXP2>
cudaError_t launch_prefix_join(const PrefixAttention &a, const PrefixShape &sh, cudaStream_t stream) {
    cudaLaunchAttribute overlap;
    overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    overlap.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)sh.ctas + a.t.N,
                       (unsigned)((sh.units.tiles * sh.units.tile + kJoinRows<D> - 1) / kJoinRows<D>));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cfg.attrs = &overlap;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, prefix_join_kernel<Tout, D, KEYS, EXP2>, a, sh);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();                           // reported here
        return e;
    }
    count_launches(1);
    return cudaSuccess;
}

}  // namespace kda
