// kda_prefix_attention_tc.cu -- attention of many sequences to the prefix that they
// share, on the tensor cores (tcgen05): bf16, head sizes 64 and 128, pages of whole
// groups of eight tokens.  The sequences' own keys are kda_tree_attention_tc.cu's
// work; its sums are joined with the prefix's here.
//
// All nodes of all a prefix's sequences, times the query heads of a cache head, are
// the rows of one product with the prefix's keys: the cache is read once for them, and
// with some 280 rows to a cache head the products and no longer the bytes are the bound.
// A CTA has one row tile of 128 (QT = 1) or two (QT = 2) against key tiles of 128:
//     S = Q K^T,   P = 2^(c S - top),   O += P V.
//
// Roles: warp 0 loads (TMA, one box per page or part of one), warps 1 and 2 issue the
// products of one row tile each, and a warpgroup per row tile does the softmax with a
// thread per row.  A tile's weights lie in the columns of its scores; while one
// tile's softmax runs, the other tile's products do: the two take turns at the tensor
// core.  One thread issues all of a tile's products and the tensor core takes them in
// that order: scores that are there mean sums that are done, and the next scores do not
// overtake the sums that read the weights in their place.
//
// The sums are rescaled only when the maximum grows by more than 2^8; weights are rounded
// to bf16 for their product (2^-9 of each), maximum, sums and output sums are fp32, as
// in the tree kernels.  Keys past the end are masked; the values' rows there are made
// zeros before their product, since a weight of zero would not cancel a NaN.
//
// Measured (d = 128, this kernel alone): 1,024 nodes behind 16,384 keys, 8 cache heads of 8 query heads, so 8,192 rows
// to a cache head, 340 us, 1,617 TFLOP/s in the products (85% of a library product's rate; the whole call 395 us);
// 256 rows to a cache head behind 65,001 keys, 54 us, 4.9 TB/s of keys and values, where reading them takes 39.
// 128 keys of both row tiles take some 3,020 clocks, the products alone 2,048: a tile's softmax (load, maximum,
// exponentials, store) is a chain that the other tile's products do not fill.  By the call of 1,024 nodes: two warps
// to 16 rows in place of one thread to a row took 432 us against 420, the maximum formed beside the exponentials 429
// against 417, the first half of P V outside the turn 459 against 425.
#include "kda_attention_tc.cuh"
#include "kda_prefix_cut.cuh"

#include <math.h>

#include <algorithm>

namespace kda {
namespace {

using namespace tc;

template <int D, int QT> struct Cfg {
    static constexpr int HALVES = D / 64;
    static constexpr int THREADS = 128 + 128 * QT;                // twelve warps leave 168 registers a thread
    static constexpr int SLOT = kTile * D * 2;                    // bytes of a key or value tile
    static constexpr int SLOTS = D == 64 ? 8 : (QT == 1 ? 6 : 5);
    static constexpr int O_RING = QT * SLOT;
    static constexpr int O_MISC = O_RING + SLOTS * SLOT;
    static constexpr int PER_TILE = 4, NBARS = 2 * SLOTS + PER_TILE * QT + 3;
    static constexpr int O_WORDS = O_MISC + 8 * NBARS;
    static constexpr int SMEM = O_MISC + 1024;
    static_assert(O_WORDS + 16 <= SMEM, "misc");
    static constexpr int TM_O = 256;                              // the scores of tile t are in 128 t, its sums in 256 + 128 t
};
static_assert(Cfg<128, 1>::SMEM <= 232448 && Cfg<128, 2>::SMEM <= 232448, "227 KB of shared memory");

constexpr int kLoadRegs = 72, kSoftmaxRegs = 208;                 // of a thread, with two row tiles
enum { W_TMEM = 0, W_ABORT, W_STATUS, W_PAGE };

struct Maps {
    CUtensorMap q, k, v;
};

using Run = PrefixRun<kTile>;

template <int D, int QT>
__global__ void __launch_bounds__(Cfg<D, QT>::THREADS, 1)
prefix_attention_tc_kernel(const __grid_constant__ Maps maps, const PrefixAttention a, const PrefixShape sh,
                           const int32_t box, const int32_t nodes) {
    using C = Cfg<D, QT>;
    extern __shared__ __align__(1024) unsigned char smem[];
    // warp-uniform by construction (a shuffle from lane 0), so that the compiler keeps
    // them, the role branches and what is derived from them in uniform registers
    const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
    volatile uint32_t *words = reinterpret_cast<uint32_t *>(smem + C::O_WORDS);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int G = a.t.H / a.t.H_kv, used = sh.units.used;

    const uint32_t bars = base + C::O_MISC;
    auto full = [&](uint32_t s) { return bars + 8u * s; };
    auto empty = [&](uint32_t s) { return bars + 8u * (C::SLOTS + s); };
    auto tile_bar = [&](int t, uint32_t i) { return bars + 8u * (2 * C::SLOTS + C::PER_TILE * t + i); };
    auto s_full = [&](int t) { return tile_bar(t, 0); };
    auto p_full = [&](int t) { return tile_bar(t, 1); };
    auto o_full = [&](int t) { return tile_bar(t, 2); };
    auto turn = [&](int t) { return tile_bar(t, 3); };
    const uint32_t q_full = tile_bar(QT, 0), q_free = tile_bar(QT, 1), v_ready = tile_bar(QT, 2);

    const PrefixPlace place = find_prefix_place<kTile>(a, sh.units, sh.ctas, blockIdx.x);
    const int64_t start = place.start, stop = piece_start(place.total, sh.ctas, blockIdx.x + 1);
    PrefixPlace *left = sh.places + blockIdx.x;
    if (tid == 0) *left = place;
    launch_dependents();
    if (start >= stop) {                                     // the whole block
        wait_prerequisites();                                // (the next kernel counts on the ones before this)
        return;
    }
    Run run = prefix_run<kTile>(a, place, stop);

    if (warp == 0) tmem_alloc(base + C::O_WORDS + 4 * W_TMEM, 512);
    if (tid == 32) {
        for (int s = 0; s < C::SLOTS; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), QT);
        }
        for (int t = 0; t < QT; ++t) {
            mbar_init(s_full(t), 1);
            mbar_init(p_full(t), 4);
            mbar_init(o_full(t), 1);
            mbar_init(turn(t), 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_free, QT);
        mbar_init(v_ready, 1);
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
    auto valid_keys = [&](const Run &r, int t) { return min(kTile, r.len - t * kTile); };
    auto uniform = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };

    // of the 384 x 168 registers that the block has, most to the softmax (409 -> 392 us for 1,024 nodes
    // behind 16,384 keys)
    if (QT == 2) {
        if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    }
    if (warp == 0) {
        // ---------------------------------------------------------------- loads
        const int32_t none = (int32_t)((int64_t)a.t.num_pages * a.t.H_kv * a.t.page_size / 8);   // past the end: zeros
        uint32_t use = 0, seg = 0;                           // ring uses so far: K of tile j is 2j, V 2j + 1
        auto queries = [&](const Run &r, int t, int x, bool load) {
            const int h = r.r / r.groups, node = (r.r % r.groups * QT + t) * nodes + r.seq0 * a.t.M;
            if (load) tma_load_4d(base + t * C::SLOT + x * 16384, &maps.q, 0, h * G, x, node, q_full);
            else tma_prefetch_4d(&maps.q, 0, h * G, x, node);
        };
        for (; run.left > 0 && ok; run.advance(a, sh.units), ++seg) {
            const int h = run.r / run.groups, cnt = run.count();
            // the queries, once the products before are through with the last ones
            if (seg > 0 && !wait(q_free, (seg - 1) & 1)) break;
            if (lane == 0) {
                mbar_expect_tx(q_full, (uint32_t)(QT * C::HALVES * nodes * G * 128));
                for (int i = 0; i < QT * C::HALVES; ++i) queries(run, i / C::HALVES, i % C::HALVES, true);
            }
            __syncwarp();
            // the next unit's come to the L2 meanwhile
            if (run.left > cnt) {
                Run then = run;
                then.advance(a, sh.units);
                if (lane < QT * C::HALVES) queries(then, lane / C::HALVES, lane % C::HALVES, false);
            }
            __syncwarp();
            const int32_t *table = a.table + (int64_t)run.p * a.max_pages;
            for (int t = run.t0; t < run.t0 + cnt && ok; ++t) {
                const int loads = (valid_keys(run, t) + box - 1) / box;      // a lane each
                int32_t group = 0;
                if (lane < loads) {
                    const int pos = t * kTile + lane * box;
                    const int page = table[pos / a.t.page_size];
                    if (page < 0 || page >= a.t.num_pages) {
                        words[W_PAGE] = 1;
                        group = none;
                    } else {
                        group = (int32_t)((((int64_t)page * a.t.H_kv + h) * a.t.page_size + pos % a.t.page_size) / 8);
                    }
                }
                const uint32_t bytes = (uint32_t)loads * box * D * 2;
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv, ++use) {
                    const uint32_t s = use % C::SLOTS;
                    if (use >= C::SLOTS && !wait(empty(s), (use / C::SLOTS - 1) & 1)) break;
                    if (lane == 0) mbar_expect_tx(full(s), bytes);
                    __syncwarp();
                    if (lane < loads)
                        tma_load_4d(base + C::O_RING + s * C::SLOT + lane * box * D * 2, kv ? &maps.v : &maps.k, 0, 0, 0,
                                    group, full(s));
                    __syncwarp();
                }
            }
        }
        if (words[W_ABORT] != 0 || !ok) {
            // loads in flight land before the block leaves
            for (uint32_t s = 0; s < C::SLOTS; ++s)
                if (use > s) mbar_wait(full(s), ((use - 1 - s) / C::SLOTS) & 1, 100000000ull);
            if (seg > 0 || run.left > 0) mbar_wait(q_full, (run.left > 0 ? seg : seg - 1) & 1, 100000000ull);
        }
    } else if (warp <= QT) {
        // ---------------------------------------------------------------- products
        // One elected thread of the warp issues a tile's products: a step's sums with the next
        // step's scores, in turns with the other tile's.  Side by side the tiles fell into step, so
        // that both softmaxes ran while the tensor core stood still (3,380 clocks for 128 keys).
        const int t = warp - 1;
        constexpr uint32_t ID_QK = idesc_bf16(kTile, kTile, 0, 0), ID_PV = idesc_bf16(kTile, D, 0, 1);
        constexpr uint64_t HI_Q = sw128_hi(0, 1024), HI_K = sw128_hi(0, C::HALVES * 1024);
        constexpr uint64_t HI_V = sw128_hi(1024, C::HALVES * 1024);
        const uint32_t s_col = uniform(tmem + t * 128), o_col = uniform(tmem + C::TM_O + t * 128);
        const uint32_t qb = uniform(base + t * C::SLOT);
        uint32_t j = 0, seg = 0, cuts = 0, turns = 0;        // tiles, segments, tiles cut short, turns before
        // the ring's slot of tile i's keys (kv = 0) or values, and the wait for it
        auto slot_of = [&](uint32_t i, uint32_t kv) { return uniform((2 * i + kv) % C::SLOTS); };
        auto landed = [&](uint32_t i, uint32_t kv) {
            return wait(full(slot_of(i, kv)), ((2 * i + kv) / C::SLOTS) & 1);
        };
        auto my_turn = [&]() {
            const uint32_t n = turns++;
            if (QT == 1 || (t == 0 && n == 0)) return ok;
            return wait(turn(t), (t == 0 ? n - 1 : n) & 1);
        };
        auto your_turn = [&]() {
            if (QT == 2 && lane == 0) mbar_arrive(turn(1 - t));
            __syncwarp();
        };
        auto scores = [&](uint32_t i, bool last) {
            const uint32_t s = slot_of(i, 0), at = uniform(base + C::O_RING + s * C::SLOT);
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                mma_bf16_w(s_col, HI_Q | sw128_lo(qb + (ks >> 2) * 16384 + (ks & 3) * 32),
                           HI_K | sw128_lo(at + (ks >> 2) * 1024 + (ks & 3) * 32), ID_QK, ks > 0);
                if (ks == D / 16 - 3) your_turn();   // the other warp needs some 150 clocks to take it up
            }
            mma_commit_w(s_full(t));
            mma_commit_w(empty(s));                          // the keys are read
            if (last) mma_commit_w(q_free);
        };
        for (; run.left > 0 && ok; run.advance(a, sh.units), ++seg) {
            const int cnt = (int)uniform((uint32_t)run.count());
            if (!wait(q_full, seg & 1) || !landed(j, 0) || !my_turn()) break;
            scores(j, cnt == 1);
            for (int i = 0; i < cnt && ok; ++i, ++j) {
                const int valid = (int)uniform((uint32_t)valid_keys(run, run.t0 + i));
                const uint32_t s = slot_of(j, 1), at = uniform(base + C::O_RING + s * C::SLOT);
                if (!landed(j, 1)) break;
                if (valid < kTile) {
                    if (t == 0) {
                        unsigned char *vs = smem + C::O_RING + s * C::SLOT;
                        const int until = (valid + 15) & ~15;
                        for (int e = lane; e < (until - valid) * (D / 8); e += 32) {
                            const int r = valid + e / (D / 8), x = e % (D / 8);
                            *reinterpret_cast<uint4 *>(vs + (r >> 3) * (C::HALVES * 1024) + (x >> 3) * 1024 +
                                                       sw128_off(r & 7, x & 7)) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(v_ready);
                        __syncwarp();
                    } else if (!wait(v_ready, cuts & 1)) {
                        break;
                    }
                    ++cuts;
                }
                const bool next = i + 1 < cnt;
                if (next && !landed(j + 1, 0)) break;
                if (!my_turn() || !wait(p_full(t), j & 1)) break;
                tc_fence_after();
                const uint32_t more = i > 0;                 // not the segment's first tile
                if (valid == kTile) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        mma_tmem_a_w(o_col, s_col + ks * 8, HI_V | sw128_lo(at + ks * 2 * C::HALVES * 1024), ID_PV,
                                     ks > 0 ? 1u : more);
                } else {
#pragma unroll 1
                    for (int ks = 0; 16 * ks < valid; ++ks)
                        mma_tmem_a_w(o_col, s_col + ks * 8, HI_V | sw128_lo(at + ks * 2 * C::HALVES * 1024), ID_PV,
                                     ks > 0 ? 1u : more);
                }
                mma_commit_w(empty(s));                      // the values are read
                if (next) {
                    scores(j + 1, i + 2 == cnt);
                } else {
                    mma_commit_w(o_full(t));
                    your_turn();
                }
            }
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------------------- softmax
        const int t = (warp - 4) >> 2, wg = tid - 128 - 128 * t;             // row tile, row in it
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;                   // TMEM lane 32 (warp % 4)
        const uint32_t s_col = tmem + lanes + t * 128, o_col = tmem + lanes + C::TM_O + t * 128;
        const float c = a.t.scale * kLog2e;
        const float2 c2 = make_float2(c, c);
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.t.out);
        const bool out32 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
        uint32_t j = 0, seg = 0;                             // tiles, segments before
        for (; run.left > 0 && ok; run.advance(a, sh.units), ++seg) {
            const int h = run.r / run.groups, cnt = run.count();
            const int row = run.r % run.groups * sh.units.rows() + t * used + wg;
            const bool real = wg < used && row < run.rows;
            float top = -INFINITY, sum = 0.f;
            for (int i = 0; i < cnt && ok; ++i, ++j) {
                const int valid = valid_keys(run, run.t0 + i);
                if (!wait(s_full(t), j & 1)) break;
                tc_fence_after();
                uint32_t v[4][32];
#pragma unroll
                for (int x = 0; x < 4; ++x) tmem_ld32_nowait(s_col + 32 * x, v[x]);
#pragma unroll
                for (int x = 0; x < 4; ++x) tmem_wait_ld_regs(v[x]);
                if (valid < kTile) {
#pragma unroll
                    for (int x = 0; x < 4; ++x)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            v[x][e] = 32 * x + e < valid ? v[x][e] : 0xff800000u;    // -infinity
                }
                auto score = [&](int e) { return __uint_as_float(v[e >> 5][e & 31]); };
                float m4[4] = {score(0), score(1), score(2), score(3)};
#pragma unroll
                for (int e = 4; e < 128; e += 4) {
#pragma unroll
                    for (int y = 0; y < 4; ++y) m4[y] = fmaxf(m4[y], score(e + y));
                }
                const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c;
                const bool grow = mx > top + kGrow;
                if (__any_sync(0xffffffffu, grow)) {
                    const float shrink = grow ? ex2(top - mx) : 1.f;
                    if (grow) top = mx;
                    sum *= shrink;
                    if (i > 0) {
#pragma unroll 1
                        for (int y = 0; y < D; y += 16) {
                            float o[16];
                            tmem_ld16w(o_col + y, o);
                            uint32_t u[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * shrink);
                            tmem_st16_nowait(o_col + y, u);
                        }
                    }
                }
                const float from = top == -INFINITY ? 0.f : top;
                const float2 f2 = make_float2(-from, -from);
                float2 add[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float2 y = f2fma(make_float2(score(32 * x + 2 * e), score(32 * x + 2 * e + 1)), c2, f2);
                        y.x = ex2(y.x);
                        y.y = ex2(y.y);
                        add[e & 1] = f2add(add[e & 1], y);
                        w[e] = pack_bf16x2(y.x, y.y);
                    }
                    tmem_st16_nowait(s_col + 16 * x, w);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(t));
                sum += (add[0].x + add[0].y) + (add[1].x + add[1].y);
            }
            if (!ok || !wait(o_full(t), seg & 1)) break;
            tc_fence_after();
            const bool whole = run.t0 == 0 && cnt == run.tiles;
            const int64_t o_row = ((int64_t)run.seq0 * a.t.M + row / G) * a.t.H + h * G + row % G;
            constexpr int R = QT * kTile;
            const int slot = 2 * blockIdx.x + (seg == 0 && run.t0 > 0 ? 0 : 1);
            float *part = sh.part + (size_t)slot * R * (D + 2);
            float own_top = -INFINITY, own_sum = -1.f;
            if (whole) {
                wait_prerequisites();                        // the own keys' sums are there
                if (real) {
                    own_top = a.t.rows.top[o_row];
                    own_sum = a.t.rows.sum[o_row];
                }
            }
            const RowJoin<true> join(top, sum, own_top, own_sum);
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
                float o[32];
                __syncwarp();                                // (lanes part below)
                tmem_ld32(o_col + x, o);
                if (!real) continue;
                if (whole) {
                    const float4 *own = reinterpret_cast<const float4 *>(a.t.rows.o + o_row * D + x);
                    uint32_t u[16];
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const float4 z = join(make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]), own[y]);
                        u[2 * y] = pack_bf16x2(z.x, z.y);
                        u[2 * y + 1] = pack_bf16x2(z.z, z.w);
                    }
                    store64(out + o_row * D + x, u, out32);
                } else {
                    store_sums32(part + (size_t)(t * kTile + wg) * D + x, o);
                }
            }
            if (real) {
                if (whole) {
                    if (a.t.lse != nullptr) a.t.lse[o_row] = join.lse;
                } else {
                    float *ml = part + (size_t)R * D + t * kTile + wg;
                    ml[0] = top;
                    ml[R] = sum;
                }
            }
            __syncwarp();
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
    wait_prerequisites();                                    // (the next kernel counts on the ones before this)
}

// One row tile where a prefix has no more rows on average: the second would hold none, and cost its share of
// the softmax, the ring's slots and the pieces' space.
bool one_tile(int32_t N, int32_t M, int32_t P, int32_t H, int32_t H_kv) {
    return ((int64_t)N * M + P - 1) / P <= kTile / (H / H_kv);
}

template <int D, int QT> cudaError_t run_tc(const PrefixAttention &a, void *workspace, cudaStream_t stream) {
    using C = Cfg<D, QT>;
    Maps maps;
    int32_t box = kTile;
    while (a.t.page_size % box != 0) box /= 2;
    const int64_t all = (int64_t)a.t.N * a.t.M;
    const int G = a.t.H / a.t.H_kv, nodes = (int)std::min<int64_t>(all, kTile / G);
    if (encode_fn() == nullptr || !query_map(&maps.q, a.t, D, nodes) || !cache_map(&maps.k, a.t.k_cache, a.t, D, box) ||
        !cache_map(&maps.v, a.t.v_cache, a.t, D, box))
        return cudaErrorInvalidValue;
    PrefixShape sh;
    sh.units = {QT, kTile, nodes * G};
    sh.ctas = sm_count();
    sh.places = static_cast<PrefixPlace *>(workspace);
    sh.part = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + prefix_place_bytes(sh.ctas));
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = allow_dynamic_smem(prefix_attention_tc_kernel<D, QT>, C::SMEM, smem_set);
    if (e != cudaSuccess) return e;
    if (QT == 2) {
        // the split of the registers draws on what the block was launched with: never on less
        static std::atomic<int> registers{0};
        if (registers.load(std::memory_order_relaxed) == 0) {
            cudaFuncAttributes at;
            e = cudaFuncGetAttributes(&at, prefix_attention_tc_kernel<D, QT>);
            if (e != cudaSuccess) return e;
            registers.store(at.numRegs, std::memory_order_relaxed);
        }
        if (registers.load(std::memory_order_relaxed) * C::THREADS < 128 * kLoadRegs + 256 * kSoftmaxRegs)
            return cudaErrorInvalidConfiguration;
    }
    cudaLaunchAttribute overlap;
    overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    overlap.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(sh.ctas);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cfg.attrs = &overlap;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, prefix_attention_tc_kernel<D, QT>, maps, a, sh, box, (int32_t)nodes);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();                            // reported here
        return e;
    }
    count_launches(1);
    return launch_prefix_join<__nv_bfloat16, D, kTile, true>(a, sh, stream);
}

}  // namespace

size_t prefix_attention_tc_bytes(int32_t N, int32_t M, int32_t P, int32_t H, int32_t H_kv, int32_t D) {
    const int ctas = sm_count();
    return prefix_place_bytes(ctas) + prefix_part_bytes(ctas, (one_tile(N, M, P, H, H_kv) ? 1 : 2) * kTile, D);
}

cudaError_t launch_prefix_attention_tc(const PrefixAttention &a, int32_t D, void *workspace, cudaStream_t stream) {
    const bool one = one_tile(a.t.N, a.t.M, a.P, a.t.H, a.t.H_kv);
    if (D == 64) return one ? run_tc<64, 1>(a, workspace, stream) : run_tc<64, 2>(a, workspace, stream);
    return one ? run_tc<128, 1>(a, workspace, stream) : run_tc<128, 2>(a, workspace, stream);
}

}  // namespace kda
