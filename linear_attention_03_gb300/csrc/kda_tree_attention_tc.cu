// kda_tree_attention_tc.cu -- tree attention over a paged cache on the tensor
// cores (tcgen05): bf16, head sizes 64 and 128, page sizes that are multiples
// of 8.  The mathematics is that of kda_tree_attention.cu.
//
// All M x G rows of a cache head read the same keys, so they make the row
// dimension of one product: tiles of 128 rows (as many whole nodes' query heads
// as fit) against tiles of 128 keys,
// S = Q K^T into TMEM, the weights back into TMEM as the operand of O += P V.
// One tile (QT = 1) or two (QT = 2, more than 128 rows) share each key tile in
// shared memory.  The work is bound by the bytes of the cache as long as one
// key tile's two products per row tile (2 x 512 clocks at d = 128) and its
// softmax stay below the tile's 64 KB at the SM's share of HBM (~2,800 clocks).
//
// Split: every (sequence, cache head, row group) is a unit of key tiles, the last
// of which holds the tree, behind the cache's last keys where they leave room.
// The units' tiles in one line are cut into equal pieces, one per CTA, one CTA per
// SM: ragged lengths cost no imbalance, and a long cache needs no separate split.
//
// Roles: warp 0 loads (TMA, one box per page or part of one), warp 1 issues the
// scores' products, warp 2 the sums', and a warpgroup per row tile does the
// softmax with a thread per row (the running maximum needs no exchange).  Keys
// go in steps of 64, half a tile, so that a row's scores fit its thread's
// registers: they are read once, and their columns are free for the next
// step's product while the softmax runs.  The weights have two buffers of their
// own, so neither product waits for the other.  Warp 3 looks at every value tile
// before its product: rows past the last key become zeros, since a weight of zero
// would not cancel a NaN; in the tree tile also the rows of no node and every
// value that is not finite, which the rows that see it get added at the end.
// The sums are rescaled only when the maximum grows by more than 2^8: weights up
// to 2^8 lose nothing in bf16 or in the fp32 sums.  The weights are rounded to
// bf16 for the product (2^-9 relative, the size of the output's own rounding);
// maximum, sum and output sums are fp32.
//
// Measured: four caches of about 256,000 tokens, 4 heads of 128, 7 nodes x 8
// query heads (one row tile): 318 us, 6.6 TB/s, the rate of a copy.  64 caches
// of 512 .. 8,192 tokens, 8 heads, 16 nodes: x 8 query heads (one row tile) 205
// .. 215 us, 5.6 TB/s; x 12 (two row tiles) 263 .. 279, 4.4 TB/s; x 16 265 .. 275.
// With two row tiles a step's four products (8 x 48 + 4 x 64 clocks each row
// tile: 64 key columns use three quarters of the tensor pipe) and the two
// softmaxes share about 1,700 clocks, against the 1,500 that the bytes take; a
// unit's end costs some 3 us.  Together that is some 210 us of the 266 (229 steps and
// 4 to 5 ends per SM); the rest has no account yet.  On the way (x 12): one warp for all products 430
// -> 330 us, value tiles prepared by a warp of their own 286, the joining
// launch overlapped 262 .. 275.  Tried and slower: a part of the exponentials on
// the FMA pipe (274 against 264), weights under the old maximum while the new
// one is taken (290 against 266), 128 keys per step (330).
#include "kda_internal.cuh"
#include "kda_tc.cuh"
#include "kda_tree.cuh"
#include "kda_attention_tc.cuh"
#include "kda_tree_cut.cuh"

#include <math.h>

#include <type_traits>

namespace kda {
namespace {

using namespace tc;

template <int D, int QT> struct Cfg {
    static constexpr int HALVES = D / 64;
    static constexpr int THREADS = 128 + 128 * QT;                // twelve warps leave 168 registers a thread
    static constexpr int SLOT = kTile * D * 2;                    // bytes of a key or value tile
    static constexpr int SLOTS = D == 64 ? 8 : (QT == 1 ? 6 : 5);
    // Barriers of landed tiles, an even number, so that each serves keys alone or values alone
    // (in an odd ring a slot holds them in turn): whoever waits on one waits for all its phases in
    // order and frees the slot itself, so that no phase is passed over.
    static constexpr int FULLS = SLOTS % 2 == 0 ? SLOTS : 2 * SLOTS;
    static constexpr int Q_BYTES = QT * SLOT;
    static constexpr int O_RING = Q_BYTES;
    static constexpr int O_MISC = O_RING + SLOTS * SLOT;
    // TMEM columns per row tile: score buffers of 64, two weight buffers of 32; then the sums
    static constexpr int BUFS = QT == 1 ? 3 : 1, TM_P = 64 * BUFS;
    // Segments (and value tiles) that can be under way at once: a unit's end may still be read
    // while warp 3 prepares the tiles that the ring holds after it.
    static constexpr int RING = D == 64 ? 8 : 4;
    static_assert(RING > (SLOTS + 1) / 2, "ring of lines");
    static constexpr int NBARS = FULLS + SLOTS + (2 * BUFS + 6) * QT + 2 + 2 * RING;
    static constexpr int O_LINES = O_MISC + 8 * NBARS, O_WORDS = O_LINES + RING * 8 * kMaxTreeNodes;
    static constexpr int SMEM = O_MISC + (D == 64 ? 8192 : 3072);
    static_assert(O_WORDS + 20 + 8 * RING <= SMEM, "misc");
    static constexpr int TM_O = 256;
};
static_assert(Cfg<128, 1>::SMEM <= 232448 && Cfg<128, 2>::SMEM <= 232448, "227 KB of shared memory");

// misc: the mbarriers, the trees' lines, then these 32-bit words (two of W_BAD per segment of the ring)
enum { W_TMEM = 0, W_ABORT, W_STATUS, W_PAGE, W_BAD };

struct Maps {
    CUtensorMap q, k, v, k8, v8, kn, vn;   // k8, v8: the cache in boxes of eight rows
};


// The last tile of a unit: the cache's last `keys` keys, and the tree from row `tree` on.
struct Last {
    int keys, tree;
};
__device__ __forceinline__ Last last_tile(int len, int M) {
    const int keys = len % kTile, tree = (keys + 7) & ~7;
    return keys > 0 && tree + M <= kTile ? Last{keys, tree} : Last{0, 0};
}
__device__ __forceinline__ int unit_tiles(int len, int M) {
    return (len + kTile - 1) / kTile + (last_tile(len, M).keys > 0 ? 0 : 1);
}

struct Units {
    static __device__ __forceinline__ int tiles(int len, int M) { return unit_tiles(len, M); }
};
using Run = CutRun<Units>;
struct Shape {
    int32_t box;            // rows per load: the power of two that divides the page size, at most 128
    int32_t nodes;          // nodes per row tile
    int32_t groups;         // row groups (of QT row tiles) per cache head
    int32_t ctas;
    Place *places;          // one per CTA
    float *part;            // two slots per CTA: D/4 x rows float4, then rows maxima, rows sums (-1: no node,
                            // in the part with the unit's last tile)
};

// keys of the unit's tile t
__device__ __forceinline__ int valid_keys(const TreeAttention &a, const Run &run, int t) {
    return t == run.tiles - 1 ? last_tile(run.len, a.M).tree + a.M : min(kTile, run.len - t * kTile);
}

// SUMS: the sums go to a.rows as they are, for the kernel that joins them with a prefix's.
template <int D, int QT, bool SUMS>
__global__ void __launch_bounds__(Cfg<D, QT>::THREADS, 1)
tree_attention_tc_kernel(const __grid_constant__ Maps maps, const TreeAttention a, const Shape sh) {
    using C = Cfg<D, QT>;
    extern __shared__ __align__(1024) unsigned char smem[];
    // warp-uniform by construction (a shuffle from lane 0), so that the compiler keeps
    // them, the role branches and what is derived from them in uniform registers
    const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
    volatile uint32_t *words = reinterpret_cast<uint32_t *>(smem + C::O_WORDS);
    uint64_t *line = reinterpret_cast<uint64_t *>(smem + C::O_LINES);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int G = a.H / a.H_kv;

    const uint32_t bars = base + C::O_MISC;
    auto full = [&](uint32_t f) { return bars + 8u * f; };   // use % FULLS
    auto empty = [&](int s) { return bars + 8u * (C::FULLS + s); };
    constexpr int PER_TILE = 2 * C::BUFS + 6;
    auto tile_bar = [&](int t, uint32_t i) { return bars + 8u * (C::FULLS + C::SLOTS + PER_TILE * t + i); };
    auto s_full = [&](int t, uint32_t b) { return tile_bar(t, b); };
    auto s_free = [&](int t, uint32_t b) { return tile_bar(t, C::BUFS + b); };
    auto p_full = [&](int t, uint32_t i) { return tile_bar(t, 2 * C::BUFS + (i & 1)); };
    auto o_full = [&](int t, uint32_t i) { return tile_bar(t, 2 * C::BUFS + 2 + (i & 3)); };
    const uint32_t q_full = tile_bar(QT, 0), q_free = tile_bar(QT, 1);
    auto v_ready = [&](uint32_t i) { return tile_bar(QT, 2 + i % C::RING); };            // by tile
    auto l_ready = [&](uint32_t i) { return tile_bar(QT, 2 + C::RING + i % C::RING); };  // by segment
    // columns of row tile t: score buffer b, the weights of step i
    auto s_col = [](int t, uint32_t b) { return t * 128 + b * 64; };
    auto p_col = [](int t, uint32_t i) { return t * 128 + C::TM_P + (i & 1) * 32; };

    Place place;
    find_place<Units>(a, sh.groups, sh.ctas, blockIdx.x, reinterpret_cast<int64_t *>(line), place);
    const int64_t start = place.start;
    const int64_t stop = piece_start(place.total, sh.ctas, blockIdx.x + 1);
    Place *left = sh.places + blockIdx.x;
    if (tid == 0) *left = place;
    launch_dependents();
    if (start >= stop) return;                               // the whole block
    Run run;
    run.left = stop - start;
    run.n = place.n;
    run.r = place.r;
    run.len = place.len;
    run.tiles = unit_tiles(place.len, a.M);
    run.t0 = (int32_t)(start - place.unit0);

    if (warp == 0) tmem_alloc(base + C::O_WORDS + 4 * W_TMEM, 512);
    if (tid == 32) {
        for (int f = 0; f < C::FULLS; ++f) mbar_init(full(f), 1);
        for (int s = 0; s < C::SLOTS; ++s) mbar_init(empty(s), 1);
        for (int t = 0; t < QT; ++t) {
            for (int b = 0; b < C::BUFS; ++b) {
                mbar_init(s_full(t, b), 1);
                mbar_init(s_free(t, b), 128);
            }
            for (int b = 0; b < 2; ++b) mbar_init(p_full(t, b), 128);
            for (int b = 0; b < 4; ++b) mbar_init(o_full(t, b), 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_free, 1);
        for (int i = 0; i < C::RING; ++i) {
            mbar_init(v_ready(i), 1);
            mbar_init(l_ready(i), 1);
        }
        fence_mbar_init();
        words[W_ABORT] = words[W_PAGE] = 0;
        words[W_STATUS] = place.status;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, words[W_TMEM], 0);
    bool ok = true;
    // a bounded wait of a whole warp; once one gives up, the warp stops
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (ok && !__all_sync(0xffffffffu, mbar_try(bar, parity))) {
            ok = __all_sync(0xffffffffu, mbar_wait(bar, parity));
            if (!ok) words[W_ABORT] = 1;
        }
        return ok;
    };

    if (warp == 0) {
        // ---------------------------------------------------------------- loads
        const int32_t none = (int32_t)((int64_t)a.num_pages * a.H_kv * a.page_size / 8);   // past the end: zeros
        uint32_t use = 0;                                    // ring uses so far: K of tile j is 2j, V 2j + 1
        for (; run.left > 0 && ok; run.advance(a, sh.groups)) {
            const int h = run.r / sh.groups, cnt = run.count();
            const int32_t *table = a.page_table + (int64_t)run.n * a.max_pages;
            for (int t = run.t0; t < run.t0 + cnt && ok; ++t) {
                // a lane per load: boxes of the cache (of eight rows where the tree follows),
                // then the tree's, eight rows each
                const bool tree = t == run.tiles - 1;
                const Last last = last_tile(run.len, a.M);
                const int keys = tree ? last.keys : valid_keys(a, run, t), box = tree ? 8 : sh.box;
                const int old = (keys + box - 1) / box, loads = old + (tree ? (a.M + 7) / 8 : 0);
                int32_t group = 0;
                if (lane < old) {
                    const int pos = t * kTile + lane * box;
                    const int page = table[pos / a.page_size];
                    if (page < 0 || page >= a.num_pages) {
                        words[W_PAGE] = 1;
                        group = none;
                    } else {
                        group = (int32_t)((((int64_t)page * a.H_kv + h) * a.page_size + pos % a.page_size) / 8);
                    }
                }
                const uint32_t bytes = (uint32_t)loads * box * D * 2;
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv, ++use) {
                    const int s = use % C::SLOTS;
                    if (use >= C::SLOTS && !wait(empty(s), (use / C::SLOTS - 1) & 1)) break;
                    const uint32_t landed = full(use % C::FULLS);
                    if (lane == 0) mbar_expect_tx(landed, bytes);
                    __syncwarp();
                    const uint32_t dst = base + C::O_RING + s * C::SLOT;
                    if (lane < loads) {
                        const uint32_t at = dst + lane * box * D * 2;   // (the tree's rows start at a multiple of 8)
                        if (lane >= old)
                            tma_load_4d(at, kv ? &maps.vn : &maps.kn, 0, run.n * a.M + (lane - old) * 8, 0, h, landed);
                        else if (tree)
                            tma_load_4d(at, kv ? &maps.v8 : &maps.k8, 0, 0, 0, group, landed);
                        else
                            tma_load_4d(at, kv ? &maps.v : &maps.k, 0, 0, 0, group, landed);
                    }
                    __syncwarp();
                }
            }
        }
        if (words[W_ABORT] != 0 || !ok) {
            // loads in flight land before the block leaves
            for (uint32_t f = 0; f < C::FULLS; ++f)
                if (use > f) {
                    const uint32_t last = (use - 1 - f) / C::FULLS;
                    mbar_wait(full(f), last & 1, 100000000ull);
                }
        }
    } else if (warp <= 2) {
        // ---------------------------------------------------------------- products
        // One elected thread of the warp issues.  A ready wait costs the warp some 100
        // clocks and the tensor pipe holds little work ahead: with one warp for all
        // products it stood idle for half of the time.
        const bool sums = warp == 2;
        constexpr uint32_t ID_QK = idesc_bf16(kTile, 64, 0, 0), ID_PV = idesc_bf16(kTile, D, 0, 1);
        constexpr uint64_t HI_Q = sw128_hi(0, 1024), HI_K = sw128_hi(0, C::HALVES * 1024);
        constexpr uint64_t HI_V = sw128_hi(1024, C::HALVES * 1024);
        constexpr uint32_t kHalf = 8 * C::HALVES * 1024;     // bytes of 64 keys
        auto uniform = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
        uint32_t slot = sums ? 1 : 0, fb = 0, par = 0;       // the tile's place in the ring, its keys' barrier
        uint32_t tile = 0, j = 0, seg = 0;                   // before
        for (; run.left > 0 && ok; run.advance(a, sh.groups), ++seg) {
            const int cnt = (int)uniform((uint32_t)run.count());
            if (!sums) {
                // the queries, once the products before are through with the last ones
                if (seg > 0 && !wait(q_free, (seg - 1) & 1)) break;
                if (lane == 0) {
                    mbar_expect_tx(q_full, (uint32_t)(QT * C::HALVES * sh.nodes * G * 128));
                    for (int t = 0; t < QT; ++t)
                        for (int x = 0; x < C::HALVES; ++x)
                            tma_load_4d(base + t * C::SLOT + x * 16384, &maps.q, 0, run.r / sh.groups * G, x,
                                        run.n * a.M + (run.r % sh.groups * QT + t) * sh.nodes, q_full);
                }
                __syncwarp();
                // the next unit's come to the L2 meanwhile
                Run then = run;
                then.advance(a, sh.groups);
                if (then.left > 0 && lane < QT * C::HALVES)
                    tma_prefetch_4d(&maps.q, 0, then.r / sh.groups * G, lane % C::HALVES,
                                    then.n * a.M + (then.r % sh.groups * QT + lane / C::HALVES) * sh.nodes);
                if (!wait(q_full, seg & 1)) {
                    mbar_wait(q_full, seg & 1, 100000000ull);
                    break;
                }
            }
            for (int i = 0; i < cnt && ok; ++i, ++tile) {
                const int valid = (int)uniform((uint32_t)valid_keys(a, run, run.t0 + i));
                if (!(sums ? wait(v_ready(tile), (tile / C::RING) & 1) : wait(full(fb), par))) break;
                for (int x = 0; 64 * x < valid && ok; ++x, ++j) {
                    const uint32_t at = uniform(base + C::O_RING + slot * C::SLOT + x * kHalf);
                    if (!sums) {
                        const uint32_t b = uniform(j % C::BUFS);
#pragma unroll
                        for (int t = 0; t < QT; ++t) {
                            const uint32_t to = tmem + s_col(t, b), qb = base + t * C::SLOT;
                            if (j >= (uint32_t)C::BUFS && !wait(s_free(t, b), (j / C::BUFS - 1) & 1)) break;
                            tc_fence_after();
#pragma unroll
                            for (int ks = 0; ks < D / 16; ++ks)
                                mma_bf16_w(to, HI_Q | sw128_lo(qb + (ks >> 2) * 16384 + (ks & 3) * 32),
                                           HI_K | sw128_lo(at + (ks >> 2) * 1024 + (ks & 3) * 32), ID_QK, ks > 0);
                            mma_commit_w(s_full(t, b));
                        }
                    } else {
                        const uint32_t more = i > 0 || x > 0;        // not the segment's first step
                        const int left = valid - 64 * x;
#pragma unroll
                        for (int t = 0; t < QT; ++t) {
                            const uint32_t p = uniform(tmem + p_col(t, j)), o = tmem + C::TM_O + t * 128;
                            if (!wait(p_full(t, j), (j >> 1) & 1)) break;
                            tc_fence_after();
                            if (left > 48) {
#pragma unroll
                                for (int ks = 0; ks < 4; ++ks)
                                    mma_tmem_a_w(o, p + ks * 8, HI_V | sw128_lo(at + ks * 2 * C::HALVES * 1024), ID_PV,
                                                 ks > 0 ? 1u : more);
                            } else {
#pragma unroll
                                for (int ks = 0; ks < 3; ++ks)
                                    if (16 * ks < left)
                                        mma_tmem_a_w(o, p + ks * 8, HI_V | sw128_lo(at + ks * 2 * C::HALVES * 1024),
                                                     ID_PV, ks > 0 ? 1u : more);
                            }
                            mma_commit_w(o_full(t, j));
                        }
                    }
                }
                mma_commit_w(empty(slot));                   // the tile is read
                slot += 2;
                if (slot >= (uint32_t)C::SLOTS) slot -= C::SLOTS;
                fb += 2;
                if (fb >= (uint32_t)C::FULLS) {
                    fb = 0;
                    par ^= 1;
                }
            }
            if (!sums) mma_commit_w(q_free);
        }
    } else if (warp == 3) {
        // ---------------------------------------------------------------- values
        uint32_t tile = 0, seg = 0;
        for (; run.left > 0 && ok; run.advance(a, sh.groups), ++seg) {
            const int cnt = run.count();
            const bool has_tree = run.t0 + cnt == run.tiles;
            const int32_t *parent = a.parent + (int64_t)run.n * a.M;
            int32_t up[2] = {-2, -2};                        // parents of nodes lane and lane + 32
            if (has_tree) {
                if (lane < a.M) up[0] = parent[lane];
                if (lane + 32 < a.M) up[1] = parent[lane + 32];
            }
            for (int i = 0; i < cnt && ok; ++i, ++tile) {
                const bool tree = run.t0 + i == run.tiles - 1;
                const int valid = valid_keys(a, run, run.t0 + i);
                // (not for the keys: their slot can be free and full again before this warp looks)
                const uint32_t v_use = 2 * tile + 1;
                if (!wait(full(v_use % C::FULLS), (v_use / C::FULLS) & 1)) break;
                uint64_t *ln = line + (seg % C::RING) * kMaxTreeNodes;
                volatile uint32_t *bad = words + W_BAD + 2 * (seg % C::RING);
                if (i == 0) {
                    if (has_tree) {
                        // both nodes' walks at once; the parents come from the lanes that hold them
                        int at[2] = {lane < a.M ? lane : -2, lane + 32 < a.M ? lane + 32 : -2};
                        uint64_t on[2] = {0, 0};
                        while (__any_sync(0xffffffffu, at[0] >= 0 || at[1] >= 0)) {
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const int p0 = __shfl_sync(0xffffffffu, up[0], at[y] & 31);
                                const int p1 = __shfl_sync(0xffffffffu, up[1], at[y] & 31);
                                if (at[y] >= 0) {
                                    const int p = at[y] < 32 ? p0 : p1;
                                    on[y] |= uint64_t{1} << at[y];
                                    if (p != -1 && (p < 0 || p >= at[y])) on[y] = 0;
                                    at[y] = p >= 0 && p < at[y] ? p : -1;
                                }
                            }
                        }
                        ln[lane] = on[0];
                        ln[lane + 32] = on[1];
                        if (lane < 2) bad[lane] = 0;
                        __syncwarp();
                    }
                    if (lane == 0) mbar_arrive(l_ready(seg));
                }
                if (tree || valid < kTile) {
                    unsigned char *vs = smem + C::O_RING + (v_use % C::SLOTS) * C::SLOT;
                    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                    auto piece = [&](int r, int x) {
                        return reinterpret_cast<uint4 *>(vs + (r >> 3) * (C::HALVES * 1024) + (x >> 3) * 1024 +
                                                         sw128_off(r & 7, x & 7));
                    };
                    const Last last = last_tile(run.len, a.M);
                    const int until = (valid + 15) & ~15;
                    for (int e = lane; e < (until - valid) * (D / 8); e += 32)
                        *piece(valid + e / (D / 8), e % (D / 8)) = zero;
                    if (tree) {
                        for (int e = lane; e < (last.tree - last.keys) * (D / 8); e += 32)
                            *piece(last.keys + e / (D / 8), e % (D / 8)) = zero;
#pragma unroll 4
                        for (int e = lane; e < a.M * (D / 8); e += 32) {
                            const int r = e / (D / 8);
                            uint4 *p = piece(last.tree + r, e % (D / 8)), u = *p;
                            uint32_t *w = reinterpret_cast<uint32_t *>(&u);
                            bool odd = false;
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const uint32_t f = w[x] & 0x7f807f80u;
                                if ((f & 0xffffu) == 0x7f80u) { w[x] &= 0xffff0000u; odd = true; }
                                if ((f >> 16) == 0x7f80u) { w[x] &= 0x0000ffffu; odd = true; }
                            }
                            if (ln[r] == 0) *p = zero;
                            else if (odd) {
                                *p = u;
                                atomicOr(const_cast<uint32_t *>(&bad[r >> 5]), 1u << (r & 31));
                            }
                        }
                    }
                    fence_proxy_async();
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(v_ready(tile));
            }
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------------------- softmax
        const int t = (warp - 4) >> 2, wg = tid - 128 - 128 * t;             // row tile, row in it
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;                   // TMEM lane 32 (warp % 4)
        const uint32_t o_col = tmem + lanes + C::TM_O + t * 128;
        const float c = a.scale * kLog2e;
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out);
        const bool out32 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
        uint32_t tile = 0, j = 0, seg = 0;                   // tiles, steps and segments before
        // step i's sums complete phase i / 4 of barrier i % 4
        auto wait_sums = [&](uint32_t i) { return wait(o_full(t, i), (i >> 2) & 1); };
        for (; run.left > 0 && ok; run.advance(a, sh.groups), ++seg) {
            const int h = run.r / sh.groups, cnt = run.count();
            // the thread's node and query head; none past the tile's whole nodes
            const int node = (run.r % sh.groups * QT + t) * sh.nodes + wg / G;
            const bool real = wg < sh.nodes * G && node < a.M;
            const int64_t n = run.n;
            float top = -INFINITY, sum = 0.f;
            uint64_t mine = 0;                       // known from the tree tile on
            int done = 0;                            // steps of this segment
            for (int i = 0; i < cnt && ok; ++i) {
                const int tl = run.t0 + i;
                const bool tree = tl == run.tiles - 1;
                const int valid = valid_keys(a, run, tl);
                if (tree) {
                    if (!wait(l_ready(seg), (seg / C::RING) & 1)) break;
                    mine = real ? line[(seg % C::RING) * kMaxTreeNodes + node] : 0;
                }
                // which of the tile's 128 keys the row sees, where that is not all of them
                const Last last = last_tile(run.len, a.M);
                auto below = [](int x) { return x >= 64 ? ~uint64_t{0} : x <= 0 ? 0 : (uint64_t{1} << x) - 1; };
                uint64_t sees[2];
                if (tree) {
                    sees[0] = below(last.keys) | (last.tree < 64 ? mine << last.tree : 0);
                    sees[1] = below(last.keys - 64) | (last.tree >= 64 ? mine << (last.tree - 64)
                                                       : last.tree > 0 ? mine >> (64 - last.tree) : 0);
                } else {
                    sees[0] = below(valid);
                    sees[1] = below(valid - 64);
                }
                const int halves = (valid + 63) / 64;
                for (int x = 0; x < halves; ++x, ++done, ++j) {
                    const uint32_t b = j % C::BUFS, sc = tmem + lanes + s_col(t, b);
                    if (!wait(s_full(t, b), (j / C::BUFS) & 1)) break;
                    tc_fence_after();
                    float v[64];
                    tmem_ld64(sc, v);
                    tc_fence_before();
                    mbar_arrive(s_free(t, b));
                    if (tree || valid < kTile) {
                        const uint64_t seen = x == 0 ? sees[0] : sees[1];
#pragma unroll
                        for (int e = 0; e < 64; ++e) v[e] = (seen >> e & 1) != 0 ? v[e] : -INFINITY;
                    }
                    float m4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                    for (int e = 4; e < 64; e += 4) {
#pragma unroll
                        for (int y = 0; y < 4; ++y) m4[y] = fmaxf(m4[y], v[e + y]);
                    }
                    const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c;
                    const bool grow = mx > top + kGrow;
                    const float was = top;
                    if (grow) top = mx;
                    const float shrink = grow ? ex2(was - top) : 1.f;
                    sum *= shrink;
                    if (done > 0 && __any_sync(0xffffffffu, grow)) {
                        if (!wait_sums(j - 1)) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int y = 0; y < D; y += 32) {
                            float o[32];
                            tmem_ld32(o_col + y, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= shrink;
                            tmem_st32(o_col + y, o);
                        }
                    }
                    const float from = top == -INFINITY ? 0.f : top;
                    const float2 c2 = make_float2(c, c), f2 = make_float2(-from, -from);
                    float2 add[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    float w[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float2 y = f2fma(make_float2(v[2 * e], v[2 * e + 1]), c2, f2);
                        y.x = ex2(y.x);
                        y.y = ex2(y.y);
                        add[e & 1] = f2add(add[e & 1], y);
                        w[e] = __uint_as_float(pack_bf16x2(y.x, y.y));
                    }
                    // the sums two steps back have read this buffer
                    if (done >= 2 && !wait_sums(j - 2)) break;
                    tmem_st32_nowait(tmem + lanes + p_col(t, j), w);
                    sum += (add[0].x + add[0].y) + (add[1].x + add[1].y);
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(p_full(t, j));
                }
            }
            tile += cnt;
            if (!ok) break;
            if (!wait_sums(j - 1)) break;
            tc_fence_after();
            const bool whole = run.t0 == 0 && cnt == run.tiles;
            const int64_t o_row = (n * a.M + node) * (int64_t)a.H + h * G + wg % G;
            volatile uint32_t *bad = words + W_BAD + 2 * (seg % C::RING);
            const uint64_t add_bad = mine == 0 ? 0 : mine & (bad[0] | (uint64_t)bad[1] << 32);
            constexpr int R = QT * kTile;
            const int slot = 2 * blockIdx.x + (seg == 0 && run.t0 > 0 ? 0 : 1);
            float *part = sh.part + (size_t)slot * R * (D + 2);
            const float inv = mine == 0 ? 0.f : 1.f / sum;
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
                float o[32];
                __syncwarp();                        // (lanes part below)
                tmem_ld32(o_col + x, o);
                if (add_bad != 0) {
                    for (uint64_t left = add_bad; left != 0; left &= left - 1) {
                        const int jn = __ffsll((long long)left) - 1;
                        const __nv_bfloat16 *vn = static_cast<const __nv_bfloat16 *>(a.v_new) +
                                                  ((n * a.M + jn) * a.H_kv + h) * (int64_t)D + x;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float y = __bfloat162float(vn[e]);
                            if (!(fabsf(y) <= 3.402823466e38f)) o[e] += y;
                        }
                    }
                }
                if (!real) continue;
                if (whole && SUMS) {
                    store_sums32(a.rows.o + o_row * D + x, o);
                } else if (whole) {
                    uint32_t u[16];
#pragma unroll
                    for (int y = 0; y < 16; ++y)
                        u[y] = mine == 0 ? 0u : pack_bf16x2(o[2 * y] * inv, o[2 * y + 1] * inv);
                    store64(out + o_row * D + x, u, out32);
                } else if (SUMS) {                   // (one row after another, as the sums are joined)
                    store_sums32(part + (size_t)(t * kTile + wg) * D + x, o);
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(part) + (size_t)(x / 4) * R + t * kTile + wg;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[(size_t)e * R] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
            }
            if (real) {
                if (whole && SUMS) {
                    a.rows.top[o_row] = top;
                    a.rows.sum[o_row] = mine == 0 ? -1.f : sum;
                } else if (whole) {
                    if (a.lse != nullptr) a.lse[o_row] = mine == 0 ? -INFINITY : (top + log2f(sum)) * kLn2;
                } else {
                    float *ml = part + (size_t)R * D + t * kTile + wg;
                    ml[0] = top;
                    ml[R] = run.t0 + cnt == run.tiles && mine == 0 ? -1.f : sum;
                }
            }
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0)
        left->status = (int32_t)words[W_STATUS] | finding(words[W_ABORT] != 0 ? KDA_DEVICE_TIMEOUT : KDA_DEVICE_OK) |
                       finding(words[W_PAGE] != 0 ? KDA_DEVICE_BAD_PAGE : KDA_DEVICE_OK);
}

// Joins the units that were cut.  Block (b, y), b > 0: the cut between CTAs
// b - 1 and b, rows 16 y .. 16 y + 15 of its unit; it works when that is the
// unit's first cut.  Block (0, 0) gathers the status.  Its launch overlaps the
// kernel before it, whose results it waits for.
template <int D, int QT, bool SUMS>
__global__ void __launch_bounds__(256)
tree_attention_tc_join_kernel(const TreeAttention a, const Shape sh) {
    // parts at a time, so that their reads are under way together (SUMS: own keys behind a prefix, units of few
    // tiles and so of few parts: three prefixes 267 us with eight, 264 with four)
    constexpr int R = QT * kTile, ROWS = 16, AT = SUMS ? 4 : 8;
    const int b = blockIdx.x;
    const int G = a.H / a.H_kv;
    if (SUMS) launch_dependents();                   // the prefix's kernel, which waits before it takes the sums
    wait_prerequisites();
    if (b == 0) {
        if (blockIdx.y != 0) return;
        gather_status(sh.places, sh.ctas, a.status);
        return;
    }
    const Place p = sh.places[b];
    const int64_t before = sh.places[b - 1].start;
    if (p.start >= p.total || p.unit0 == p.start || before > p.unit0) return;
    const int64_t end = p.unit0 + unit_tiles(p.len, a.M);
    const int parts = first_past(p.total, sh.ctas, end) - (b - 1);
    const int h = p.r / sh.groups, node0 = p.r % sh.groups * QT * sh.nodes;
    // part i is CTA b - 1 + i's: its last segment for the first, its first one after that
    auto part_of = [&](int i) { return sh.part + (size_t)(2 * (b - 1 + i) + (i == 0 ? 1 : 0)) * R * (D + 2); };
    for (int e = threadIdx.x; e < ROWS * (D / 4); e += 256) {
        const int lr = blockIdx.y * ROWS + (SUMS ? e / (D / 4) : e % ROWS), c4 = SUMS ? e % (D / 4) : e / ROWS;
        const int node = node0 + lr / kTile * sh.nodes + lr % kTile / G;
        if (lr >= R || lr % kTile >= sh.nodes * G || node >= a.M) continue;
        float top = -INFINITY, sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        const bool none = part_of(parts - 1)[(size_t)R * D + R + lr] < 0.f;
        for (int i0 = 0; i0 < parts; i0 += AT) {
            float x[AT], z[AT];
            float4 y[AT];
#pragma unroll
            for (int i = 0; i < AT; ++i) {
                const float *q = part_of(min(i0 + i, parts - 1));
                x[i] = i0 + i < parts ? q[(size_t)R * D + lr] : -INFINITY;
                z[i] = q[(size_t)R * D + R + lr];
                y[i] = reinterpret_cast<const float4 *>(q)[SUMS ? (size_t)lr * (D / 4) + c4 : (size_t)c4 * R + lr];
            }
            float was = top;
#pragma unroll
            for (int i = 0; i < AT; ++i) top = fmaxf(top, x[i]);
            const float from = top == -INFINITY ? 0.f : top, shrink = ex2(was - from);
            sum *= shrink;
            o.x *= shrink; o.y *= shrink; o.z *= shrink; o.w *= shrink;
#pragma unroll
            for (int i = 0; i < AT; ++i) {
                // (a part with nothing seen adds zeros; one whose scores are no numbers has a maximum of
                // -infinity too and makes the row one: a weight of zero skips nothing)
                if (i0 + i < parts) {
                    const float w = ex2(x[i] - from);
                    sum += w * z[i];
                    o.x += w * y[i].x; o.y += w * y[i].y; o.z += w * y[i].z; o.w += w * y[i].w;
                }
            }
        }
        const int64_t o_row = ((int64_t)p.n * a.M + node) * a.H + h * G + lr % kTile % G;
        if (SUMS) {
            *reinterpret_cast<float4 *>(a.rows.o + o_row * D + 4 * c4) = o;
            if (c4 == 0) {
                a.rows.top[o_row] = top;
                a.rows.sum[o_row] = none ? -1.f : sum;
            }
            continue;
        }
        const float inv = 1.f / sum;
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + o_row * D + 4 * c4) =
            none ? make_uint2(0u, 0u)
                 : make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (c4 == 0 && a.lse != nullptr) a.lse[o_row] = none ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
}

// The drafted rows [N * M][H_kv][D], eight rows of one head per box.
bool new_map(CUtensorMap *map, const void *base, const TreeAttention &a, int D) {
    return make_map(map, base, {64, (cuuint64_t)a.N * a.M, (cuuint64_t)(D / 64), (cuuint64_t)a.H_kv},
                    {(cuuint64_t)a.H_kv * D * 2, 128, (cuuint64_t)D * 2}, {64, 8, (cuuint32_t)(D / 64), 1});
}

template <int D, int QT, bool SUMS> cudaError_t run_tc(const TreeAttention &a, void *workspace, cudaStream_t stream) {
    using C = Cfg<D, QT>;
    Maps maps;
    Shape sh;
    sh.box = kTile;
    while (a.page_size % sh.box != 0) sh.box /= 2;
    sh.nodes = nodes_per_tile(a.M, a.H, a.H_kv);
    if (encode_fn() == nullptr || !query_map(&maps.q, a, D, sh.nodes) || !cache_map(&maps.k, a.k_cache, a, D, sh.box) ||
        !cache_map(&maps.v, a.v_cache, a, D, sh.box) || !cache_map(&maps.k8, a.k_cache, a, D, 8) ||
        !cache_map(&maps.v8, a.v_cache, a, D, 8) || !new_map(&maps.kn, a.k_new, a, D) ||
        !new_map(&maps.vn, a.v_new, a, D))
        return cudaErrorInvalidValue;
    sh.groups = (a.M + QT * sh.nodes - 1) / (QT * sh.nodes);
    sh.ctas = sm_count();
    sh.places = static_cast<Place *>(workspace);
    sh.part = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + place_bytes(sh.ctas));
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = allow_dynamic_smem(tree_attention_tc_kernel<D, QT, SUMS>, C::SMEM, smem_set);
    if (e != cudaSuccess) return e;
    tree_attention_tc_kernel<D, QT, SUMS><<<sh.ctas, C::THREADS, C::SMEM, stream>>>(maps, a, sh);
    count_launches(1);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int blocks = QT == 1 ? (sh.nodes * (a.H / a.H_kv) + 15) / 16 : QT * kTile / 16;
    cudaLaunchAttribute overlap;
    overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    overlap.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sh.ctas, blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = &overlap;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, tree_attention_tc_join_kernel<D, QT, SUMS>, a, sh);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();                            // reported here
        return e;
    }
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

bool tree_attention_tc_supported(int32_t H, int32_t H_kv, int32_t D, kda_dtype dt, int64_t num_pages,
                                 int32_t page_size) {
    return dt == KDA_BF16 && H / H_kv <= kTile && (D == 64 || D == 128) && page_size % 8 == 0 &&
           num_pages * H_kv * page_size / 8 < INT32_MAX;
}

size_t tree_attention_tc_partial_bytes(int32_t M, int32_t H, int32_t H_kv, int32_t D) {
    const int tiles = M <= nodes_per_tile(M, H, H_kv) ? 1 : 2;
    const int ctas = sm_count();
    return place_bytes(ctas) + (size_t)ctas * 2 * tiles * kTile * (D + 2) * 4;
}

cudaError_t launch_tree_attention_tc(const TreeAttention &a, int32_t D, void *workspace, cudaStream_t stream) {
    const bool one = a.M <= nodes_per_tile(a.M, a.H, a.H_kv);
    auto pick = [&](auto rows) {
        constexpr bool R = decltype(rows)::value;
        if (D == 64) return one ? run_tc<64, 1, R>(a, workspace, stream) : run_tc<64, 2, R>(a, workspace, stream);
        return one ? run_tc<128, 1, R>(a, workspace, stream) : run_tc<128, 2, R>(a, workspace, stream);
    };
    return a.rows.o != nullptr ? pick(std::true_type{}) : pick(std::false_type{});
}

}  // namespace kda
