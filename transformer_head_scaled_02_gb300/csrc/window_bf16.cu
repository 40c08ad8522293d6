// window_bf16.cu -- causal sliding-window attention with sinks over whole sequences, bf16 layers, on
// tcgen05: row i of a sequence sees key j iff j <= i, j < L_b and (i - j < window or j < sinks).
//
// Persistent CTAs, one per SM, which take the items in turn.  A work item is two neighbouring 128-row query tiles of one (batch, head),
// which share every K/V tile the TMA brings in (one tile per 128 rows would ask more of L2 than it
// has).  Key tiles are aligned to the query tiles, so that of a row's window only the oldest and the
// newest tile are cut by a mask; they run from the first row's window to the last row, behind the tiles
// that hold the sinks below.  An item is short (window / 128 + 2 tiles), so nothing is set up per item:
// the K/V ring, the score products and the softmax run on from one item into the next, and an item's
// end (reading the accumulator, the gate, the stores) lies under the next one's loads and products.
//
// Items are numbered from the last rows of all sequences to the first: those, which see less than a
// window, come last and even out the CTAs (numbered the other way, 16 heads of 16384 rows took 219 us for
// 205, with the tensor pipes of the SMs busy for 51 to 70 % of the time).
//
// P is rounded to bf16 for the value product, as the tensor cores take it, by at most 2^-8 of itself; the row sums
// are of the fp32 values.
//
// Measured: 16 heads x 16384 rows, d = 128, window 2048: 192 to 200 us in a captured graph, 66 to 69 % of the measured
// bf16 rate (260 GF: only the visible pairs count), 208 us in a loop of calls; bound by the chain score product, softmax, value product of each query tile with two
// in flight.  4 x 16 heads x 2048 rows, d = 64, window 256: 32 us; most of its tiles are cut by a mask and a
// CTA has three items.  P in columns of its own (d = 64 has room) took 45 us where this took 41, masks kept in
// registers no less than in the scores.
//
// Tensor memory (512 columns): S_t at 128 t (P_t overwrites its first 64 columns), O_t at 256 + HD t, for
// query tile t.  Warp roles (384 threads): warp 0 TMA of K and V; warp 1 TMEM owner and MMA issuer: for
// each key tile J of the items in order and each query tile t that sees it, O_t += P_t V_J and then
// S_t = Q_t K_(J+1) (MMAs of one thread execute in issue order, so S_t may overwrite P_t); warp 2 TMA of Q;
// warp 3 works out the items and hands them to the others through a ring in shared memory; warps 4-7
// softmax and output of query tile 0, warps 8-11 of tile 1 (thread = query row).  The issuer's loop is on
// every tile's critical path and shares the instruction cache with the softmax: it holds the products, the
// waits and little else (with the items' arithmetic in it a tile took six times as long).
//
// Tiles that a warp's 32 rows see whole take a straight path without masks; the few that are cut go in
// 32-column pieces, those that no row of the warp sees neither read nor exponentiated.
#include <math.h>

#include <atomic>

#include "internal.h"
#include "tc_issue.cuh"

namespace mha {
namespace {

constexpr int WN_THREADS = 384;
constexpr int WN_REGS = 168;  // at launch
constexpr int WN_REGS_CTRL = 88;
constexpr int WN_REGS_SOFTMAX = 208;
static_assert(128 * WN_REGS_CTRL + 256 * WN_REGS_SOFTMAX <= WN_THREADS * WN_REGS, "register split");
constexpr int WN_RING = 4;  // items in flight

template <int HD>
struct WnCfg {
    static constexpr int CH = HD / 64;
    static constexpr int CHUNK = 128 * 128;  // 128 rows x 64 bf16
    static constexpr int TILE = CH * CHUNK;
    // a key tile is wanted most of a round before its values: with one K stage more than V stages its
    // load has two rounds to arrive
    static constexpr int SK = HD == 128 ? 3 : 5, SV = HD == 128 ? 2 : 4;
    static constexpr int SMEM = 2 * TILE + (SK + SV) * TILE + 1024 + 1024;
    static constexpr uint32_t O_COL = 256;
};
static_assert(WnCfg<128>::SMEM <= 232448 && WnCfg<64>::SMEM <= 232448, "window smem budget");

// One work item: query tiles at rows q0 and q0 + 128 of (batch b, head).  Key tiles: nst sink tiles over
// [0, s_end), then window tiles from key kA.  Query tile t visits tiles [0, nst) and [first[t], end[t]) of
// them (end[t] == 0: none).
struct WnItem {
    int b, head, q0, L, kA, s_end, nst;
    int first[2], end[2];
    int tiles;  // tiles loaded; -1: no more items
    int bad;
};

// Tile j's keys [key0, key0 + n).
__device__ __forceinline__ void wn_keys(const WnItem& x, int j, int& key0, int& n) {
    const bool sink = j < x.nst;
    key0 = sink ? 128 * j : x.kA + 128 * (j - x.nst);
    n = min(128, (sink ? x.s_end : x.L) - key0);
}

struct WnTail {
    uint64_t kfull[5], vfull[4], kempty[5], vempty[4];
    uint64_t qfull[2], qempty[2], sfull[2], pfull[2], odone[2], ofree[2];
    uint64_t ifull[WN_RING], iempty[WN_RING];
    uint64_t drain;
    uint32_t tmem;
    int abort_flag;
    WnItem items[WN_RING];
};
static_assert(sizeof(WnTail) <= 1024, "window tail");

struct WnMaps {
    CUtensorMap q, k, v;
};

struct WnArgs {
    int B, h, h_kv, T, window, sinks, n_qb;
    int64_t items;
    const int32_t* lengths;
};

__device__ __forceinline__ WnItem wn_item(const WnArgs& a, int64_t k) {
    WnItem x;
    const int heads = a.B * a.h, back_qb = (int)k / heads, bh = (int)k - back_qb * heads;
    const int qb = a.n_qb - 1 - back_qb;
    x.b = bh / a.h;
    x.head = bh - x.b * a.h;
    x.q0 = 256 * qb;
    x.L = a.lengths != nullptr ? a.lengths[x.b] : a.T;
    x.bad = x.L < 1 || x.L > a.T;
    const int back = (a.window + 126) / 128 * 128;  // from a query tile to its oldest key tile
    x.kA = max(0, x.q0 - back);
    x.s_end = min(min(a.sinks, x.kA), x.L);
    x.nst = x.bad ? 0 : (x.s_end + 127) / 128;
    x.tiles = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        // window tiles of this query tile, from its own window's first key on (from the item's, where the
        // sinks reach past that one) to its last row or the length
        const int from = t == 0 || a.sinks > x.kA ? 0 : (max(0, x.q0 + 128 - back) - x.kA) / 128;
        const int to = (min(x.L, x.q0 + 128 * t + 128) - x.kA + 127) / 128;
        const bool none = x.bad || x.q0 + 128 * t >= a.T || (to <= from && x.nst == 0);
        x.first[t] = none ? 0 : x.nst + from;
        x.end[t] = none ? 0 : to > from ? x.nst + to : x.nst;  // x.nst: the sinks only
        x.tiles = max(x.tiles, x.end[t]);
    }
    return x;
}

__device__ __forceinline__ bool wn_visits(int j, int nst, int first, int end) { return j < end && (j < nst || j >= first); }

__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// One row of a score tile from tensor memory (warp-collective).
__device__ __forceinline__ void load_scores(uint32_t taddr, float (&x)[128]) {
    uint32_t sr[4][32];
#pragma unroll
    for (int c = 0; c < 4; ++c) tmem_ld32(taddr + c * 32, sr[c]);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < 128; ++c) x[c] = __uint_as_float(sr[c >> 5][c & 31]);
}

template <int HD, bool GATE>
__global__ void __launch_bounds__(WN_THREADS, 1)
    window_bf16_kernel(const __grid_constant__ WnMaps maps, const __grid_constant__ WnArgs a,
                       const __nv_bfloat16* __restrict__ gate, int64_t ldg, __nv_bfloat16* __restrict__ O,
                       int64_t ldo, float scale_log2, int* status) {
    using C = WnCfg<HD>;
    constexpr int SK = C::SK, SV = C::SV;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t sQ = base, sK = sQ + 2 * C::TILE, sV = sK + SK * C::TILE;
    WnTail* tail = reinterpret_cast<WnTail*>(smem_raw + (base - raw) + C::TILE * (2 + SK + SV));
    volatile int* abort_flag = &tail->abort_flag;
    auto bar = [](uint64_t& b) { return smem_u32(&b); };
    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < SK; ++s) {
            mbar_init(bar(tail->kfull[s]), 1);
            mbar_init(bar(tail->kempty[s]), 1);
        }
        for (int s = 0; s < SV; ++s) {
            mbar_init(bar(tail->vfull[s]), 1);
            mbar_init(bar(tail->vempty[s]), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(tail->qfull[t]), 1);
            mbar_init(bar(tail->qempty[t]), 1);
            mbar_init(bar(tail->sfull[t]), 1);
            mbar_init(bar(tail->pfull[t]), 4);
            mbar_init(bar(tail->odone[t]), 1);
            mbar_init(bar(tail->ofree[t]), 4);
        }
        for (int i = 0; i < WN_RING; ++i) {
            mbar_init(bar(tail->ifull[i]), 1);
            mbar_init(bar(tail->iempty[i]), 11);  // K/V, Q, MMA and the eight softmax warps
        }
        mbar_init(bar(tail->drain), 1);
        tail->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tail->tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tail->tmem;
    grid_dependency_wait();  // Q, K, V and the lengths may come from the previous kernel
    grid_launch_dependents();
    // The i-th item, once it is there; afterwards its slot is released.
    auto item_ready = [&](int i) { return lean_wait(bar(tail->ifull[i % WN_RING]), (uint32_t)(i / WN_RING) & 1u, abort_flag, status); };
    auto item_done = [&](int i) { mbar_arrive(bar(tail->iempty[i % WN_RING])); };

    if (warp < 4) {
      setmaxnreg_dec<WN_REGS_CTRL>();
      if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA: K and V tiles
            tma_prefetch_desc(&maps.k);
            tma_prefetch_desc(&maps.v);
            int nk = 0, nv = 0;
            for (int i = 0; item_ready(i); ++i) {
                const WnItem it = tail->items[i % WN_RING];
                if (it.tiles < 0) break;
                const int col = it.head / (a.h / a.h_kv) * HD;
                bool ok = true;
                for (int j = 0; j < it.tiles; ++j) {
                    const int key0 = j < it.nst ? 128 * j : it.kA + 128 * (j - it.nst);
                    const int sk = nk % SK, sv = nv % SV;
                    ok = lean_wait(bar(tail->kempty[sk]), ((uint32_t)(nk / SK) & 1u) ^ 1u, abort_flag, status);
                    if (!ok) break;
                    mbar_arrive_expect_tx(bar(tail->kfull[sk]), C::TILE);
#pragma unroll
                    for (int c = 0; c < C::CH; ++c)
                        tma_load_3d(sK + sk * C::TILE + c * C::CHUNK, &maps.k, col + c * 64, key0, it.b, bar(tail->kfull[sk]));
                    ++nk;
                    ok = lean_wait(bar(tail->vempty[sv]), ((uint32_t)(nv / SV) & 1u) ^ 1u, abort_flag, status);
                    if (!ok) break;
                    mbar_arrive_expect_tx(bar(tail->vfull[sv]), C::TILE);
#pragma unroll
                    for (int c = 0; c < C::CH; ++c)
                        tma_load_3d(sV + sv * C::TILE + c * C::CHUNK, &maps.v, col + c * 64, key0, it.b, bar(tail->vfull[sv]));
                    ++nv;
                }
                if (!ok) break;
                item_done(i);
            }
            // every load issued lands before the CTA exits
            for (int i = nk > SK ? nk - SK : 0; i < nk; ++i) drain_wait_a(bar(tail->kfull[i % SK]), (uint32_t)(i / SK) & 1u);
            for (int i = nv > SV ? nv - SV : 0; i < nv; ++i) drain_wait_a(bar(tail->vfull[i % SV]), (uint32_t)(i / SV) & 1u);
        }
      } else if (warp == 2) {
        if (lane == 0) {
            // ---------------- TMA: query tiles, each as soon as the last score product of its
            // predecessor is through
            tma_prefetch_desc(&maps.q);
            int nq[2] = {0, 0};
            bool ok = true;
            for (int i = 0; ok && item_ready(i); ++i) {
                const WnItem it = tail->items[i % WN_RING];
                if (it.tiles < 0) break;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (!ok || it.end[t] == 0) continue;
                    if (nq[t] > 0) ok = lean_wait(bar(tail->qempty[t]), (uint32_t)(nq[t] - 1) & 1u, abort_flag, status);
                    if (!ok) continue;
                    mbar_arrive_expect_tx(bar(tail->qfull[t]), C::TILE);
#pragma unroll
                    for (int c = 0; c < C::CH; ++c)
                        tma_load_3d(sQ + t * C::TILE + c * C::CHUNK, &maps.q, it.head * HD + c * 64, it.q0 + 128 * t, it.b,
                                    bar(tail->qfull[t]));
                    ++nq[t];
                }
                item_done(i);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (nq[t] > 0) drain_wait_a(bar(tail->qfull[t]), (uint32_t)(nq[t] - 1) & 1u);
        }
      } else if (warp == 3) {
        if (lane == 0) {
            // ---------------- the items, and an end mark
            int64_t k = blockIdx.x;
            for (int i = 0;; ++i, k += gridDim.x) {
                if (i >= WN_RING &&
                    !lean_wait(bar(tail->iempty[i % WN_RING]), (uint32_t)(i / WN_RING - 1) & 1u, abort_flag, status))
                    break;
                if (k < a.items) {
                    const WnItem x = wn_item(a, k);
                    if (x.bad) record_status(status, kStatusBadLength);
                    tail->items[i % WN_RING] = x;
                } else {
                    tail->items[i % WN_RING].tiles = -1;
                }
                mbar_arrive(bar(tail->ifull[i % WN_RING]));
                if (k >= a.items) break;
            }
        }
      } else {
        {
            // ---------------- MMA issuer (the whole warp, see tc_issue.cuh).  J: tiles of the items before; per query tile t, ns, np, no: query
            // tiles started, P tiles consumed, accumulators begun
            const uint64_t qdesc0 = sdesc_sw128(sQ, 16, 1024);
            const uint64_t kdesc0 = sdesc_sw128(sK, 16, 1024);
            const uint64_t vdesc0 = sdesc_sw128(sV, C::CHUNK, 1024);
            constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false);
            constexpr uint32_t idesc_o = idesc_bf16_f32(128, HD, false, true);
            const uint32_t el = elect_lane();
            int J = 0;
            uint32_t ns[2] = {0, 0}, np[2] = {0, 0}, no[2] = {0, 0};
            auto issue_s = [&](int t, int JJ, bool fresh, bool last) -> bool {
                if (fresh && !warp_wait(bar(tail->qfull[t]), ns[t]++ & 1u, abort_flag, status)) return false;
                const int st = JJ % SK;
                if (!warp_wait(bar(tail->kfull[st]), (uint32_t)(JJ / SK) & 1u, abort_flag, status)) return false;
                tc_fence_after();
                const uint64_t kdesc = kdesc0 + (uint64_t)((st * C::TILE) >> 4);
                const uint64_t qdesc = qdesc0 + (uint64_t)((t * C::TILE) >> 4);
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                    const uint32_t off16 = (uint32_t)(((kk >> 2) * C::CHUNK + (kk & 3) * 32) >> 4);
                    mma_bf16_ss_elect(el, tmem + 128u * t, qdesc + off16, kdesc + off16, idesc_s, kk > 0 ? 1u : 0u);
                }
                tc_commit_elect(el, bar(tail->sfull[t]));
                if (last) tc_commit_elect(el, bar(tail->qempty[t]));
                return true;
            };
            bool ok = __all_sync(0xffffffffu, item_ready(0)), begun = false;  // begun: this item's first scores are under way
            for (int i = 0; ok; ++i) {
                const WnItem& it = tail->items[i % WN_RING];
                const int tiles = it.tiles, nst = it.nst;
                if (tiles < 0) break;
                const int first[2] = {it.first[0], it.first[1]}, end[2] = {it.end[0], it.end[1]};
                int nx_tiles = 0, nx_nst = 0, nx_first[2] = {0, 0}, nx_end[2] = {0, 0};
                bool fresh[2] = {true, true};  // the next value product begins an accumulator
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (!begun && ok && wn_visits(0, nst, first[t], end[t])) ok = issue_s(t, J, true, end[t] == 1);
                if (ok && !begun && tiles > 0) tc_commit_elect(el, bar(tail->kempty[J % SK]));
                // the next item, read while the softmax has this one's scores
                ok = ok && __all_sync(0xffffffffu, item_ready(i + 1));
                if (!ok) break;
                {
                    const WnItem& nx = tail->items[(i + 1) % WN_RING];
                    nx_tiles = nx.tiles;
                    nx_nst = nx.nst;
#pragma unroll
                    for (int t = 0; t < 2; ++t)  // (the end mark has a count of tiles only)
                        if (nx_tiles > 0) nx_first[t] = nx.first[t], nx_end[t] = nx.end[t];
                }
                for (int j = 0; j < tiles && ok; ++j, ++J) {
                    const bool lastj = j + 1 == tiles;
                    const int st = J % SV;
                    ok = warp_wait(bar(tail->vfull[st]), (uint32_t)(J / SV) & 1u, abort_flag, status);
                    const uint64_t vdesc = vdesc0 + (uint64_t)((st * C::TILE) >> 4);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (ok && wn_visits(j, nst, first[t], end[t])) {
                            // the accumulator of the query tile before has been read
                            if (fresh[t] && no[t] > 0) ok = warp_wait(bar(tail->ofree[t]), (no[t] - 1) & 1u, abort_flag, status);
                            ok = ok && warp_wait(bar(tail->pfull[t]), np[t]++ & 1u, abort_flag, status);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                mma_bf16_ts_elect(el, tmem + C::O_COL + HD * t, tmem + 128u * t + kk * 8, vdesc + (uint64_t)((kk * 2048) >> 4),
                                            idesc_o, (!fresh[t] || kk > 0) ? 1u : 0u);
                            if (fresh[t]) ++no[t];
                            fresh[t] = false;
                            if (j + 1 == end[t]) tc_commit_elect(el, bar(tail->odone[t]));
                        }
                        // this query tile's scores of the next tile, the next item's first one included (a new
                        // query tile also if this one passed over the tiles before)
                        const int jn = lastj ? 0 : j + 1, nst_n = lastj ? nx_nst : nst;
                        const int first_n = lastj ? nx_first[t] : first[t], end_n = lastj ? nx_end[t] : end[t];
                        if (wn_visits(jn, nst_n, first_n, end_n))
                            ok = ok && issue_s(t, J + 1, jn == (nst_n > 0 ? 0 : first_n), jn + 1 == end_n);
                    }
                    if (!ok) break;
                    tc_commit_elect(el, bar(tail->vempty[st]));
                    if (!lastj || nx_tiles > 0) tc_commit_elect(el, bar(tail->kempty[(J + 1) % SK]));
                }
                if (tiles > 0) begun = nx_tiles > 0;
                __syncwarp();
                if (ok && lane == 0) item_done(i);
            }
            tc_commit_elect(el, bar(tail->drain));
            drain_wait_a(bar(tail->drain), 0);
        }
      }
    } else {
        setmaxnreg_inc<WN_REGS_SOFTMAX>();
        // ---------------- softmax and output of query tile t
        const int t = (warp - 4) >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t s_col = trow + 128u * t, o_col = trow + C::O_COL + HD * t;
        const bool wide = ((reinterpret_cast<uintptr_t>(O) | (uintptr_t)(ldo * 2)) & 31u) == 0;
        int nj = 0;  // score tiles read
        int no = 0;  // accumulators read
        int J = 0;   // tiles of the items before
        bool ok = true;
        for (int i = 0; ok; ++i) {
            if (!__all_sync(0xffffffffu, item_ready(i))) break;
            const WnItem it = tail->items[i % WN_RING];
            const int first_t = t == 0 ? it.first[0] : it.first[1], end_t = t == 0 ? it.end[0] : it.end[1];
            __syncwarp();
            if (it.tiles < 0) break;
            if (lane == 0) item_done(i);
            const int row0 = it.q0 + 128 * t + quarter * 32, row = row0 + lane;
            const bool store = row < a.T;
            __nv_bfloat16* out = O + ((int64_t)it.b * a.T + row) * ldo + (int64_t)it.head * HD;
            if (end_t == 0) {
                // nothing visible to the whole tile: zeros (padding), NaN for an invalid length
                const uint32_t z = it.bad ? 0x7FC07FC0u : 0u;
                if (store)
#pragma unroll 1
                    for (int e = 0; e < HD; e += 8) *reinterpret_cast<uint4*>(out + e) = make_uint4(z, z, z, z);
                J += it.tiles;
                continue;
            }
            float m = -INFINITY, l = 0.f;
            bool first = true;
            for (int j = 0; j < it.tiles && ok; ++j) {
                if (!wn_visits(j, it.nst, first_t, end_t)) continue;
                if (!__all_sync(0xffffffffu, lean_wait(bar(tail->sfull[t]), (uint32_t)nj & 1u, abort_flag, status))) {
                    ok = false;
                    break;
                }
                ++nj;
                tc_fence_after();
                int key0, n;
                wn_keys(it, j, key0, n);
                // columns [lo, hi) and those below sk are visible; over the warp's rows, lo and hi grow by
                // one from lane to lane
                const int hi0 = row0 + 1 - key0, lo0 = row0 - a.window + 1 - key0, sk = a.sinks - key0;
                const uint64_t c2 = pack2(scale_log2, scale_log2);
                // Any reference m gives the same O / l as long as P stays finite.
                float alpha = 1.f, rowsum = 0.f;
                auto new_reference = [&](float m_new) {
                    alpha = m_new == -INFINITY ? 1.f : ex2_approx(m - m_new);  // 0 when m leaves -inf
                    const bool rescale = m_new != m && !first;
                    // S was issued after the value product of this query tile's last tile: O is complete
                    if (__any_sync(0xffffffffu, rescale)) {
                        const float f = rescale ? alpha : 1.f;
#pragma unroll 1
                        for (int cc = 0; cc < HD; cc += 32) {
                            uint32_t o[32];
                            tmem_ld32(o_col + cc, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st32(o_col + cc, o);
                        }
                    }
                    m = m_new;
                };
                if (min(n, hi0) >= 128 && (lo0 + 31 <= 0 || sk >= 128)) {
                    // the whole tile is visible: keep the reference until a row's sum passes 2^64 (or is
                    // not finite: m = -inf), then take the tile's maximum and redo
                    uint32_t pk[64];
                    bool renew = first;
                    for (;;) {
                        float x[128];
                        load_scores(s_col, x);
                        if (renew) new_reference(fmaxf(m, row_max(x) * scale_log2));
                        rowsum = exp_tile(x, c2, m == -INFINITY && renew ? 0.f : -m, pk);
                        if (renew) break;
                        renew = !__all_sync(0xffffffffu, rowsum <= 18446744073709551616.f);
                        if (!renew) break;
                    }
                    uint32_t (&p0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&pk[0]);
                    uint32_t (&p1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&pk[32]);
                    tmem_st32(s_col, p0);
                    tmem_st32(s_col + 32, p1);
                } else {
                    // a tile that the mask cuts: 32 columns at a time, those that no row of the warp sees
                    // neither read nor exponentiated.  First the maximum (the reference moves when P could
                    // pass 2^32), with the mask left in the scores; then P over the scores just read.
                    const int hi = min(n, hi0 + lane), lo = lo0 + lane;
                    float mt = -INFINITY;
                    unsigned seen = 0u;
#pragma unroll 1
                    for (int c = 0; c < 128; c += 32) {
                        if (c >= min(n, hi0 + 31) || (c + 32 <= lo0 && c >= sk)) continue;
                        seen |= 1u << (c >> 5);
                        uint32_t sr[32];
                        tmem_ld32(s_col + c, sr);
                        tmem_wait_ld();
                        if (c + 32 > min(n, hi0) || (c < lo0 + 31 && c + 32 > sk)) {
#pragma unroll
                            for (int u = 0; u < 32; ++u)
                                if (c + u >= hi || (c + u < lo && c + u >= sk)) sr[u] = 0xFF800000u;
                            tmem_st32(s_col + c, sr);
                        }
#pragma unroll
                        for (int u = 0; u < 32; u += 2) mt = fmax3(mt, __uint_as_float(sr[u]), __uint_as_float(sr[u + 1]));
                    }
                    tmem_wait_st();
                    mt *= scale_log2;
                    new_reference(mt > m + 32.f || first ? fmaxf(m, mt) : m);
                    const float neg = m == -INFINITY ? 0.f : -m;
#pragma unroll 1
                    for (int c = 0; c < 128; c += 32) {
                        uint32_t pk[16];
                        if ((seen >> (c >> 5)) & 1u) {
                            uint32_t sr[32];
                            tmem_ld32(s_col + c, sr);
                            tmem_wait_ld();
                            uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
                            for (int u = 0; u < 16; ++u) {
                                float a0, a1;
                                unpack2(fma2(pack2(__uint_as_float(sr[2 * u]), __uint_as_float(sr[2 * u + 1])), c2, pack2(neg, neg)), a0, a1);
                                const float y0 = ex2_approx(a0), y1 = ex2_approx(a1);
                                acc[u & 1] = add2(acc[u & 1], pack2(y0, y1));
                                pk[u] = pack_bf16x2(y0, y1);
                            }
                            float s0, s1;
                            unpack2(add2(acc[0], acc[1]), s0, s1);
                            rowsum += s0 + s1;
                        } else {
#pragma unroll
                            for (int u = 0; u < 16; ++u) pk[u] = 0u;
                        }
                        tmem_st16(s_col + c / 2, pk);
                    }
                }
                first = false;
                if (it.L < a.T && key0 + 128 > it.L) {
                    // rows past the length may hold anything: zero the V rows the product would multiply by
                    // P = 0 (a NaN there would survive it).  Both query tiles' warps do, each before its own
                    // product.
                    const int st = (J + j) % SV;
                    if (!__all_sync(0xffffffffu, lean_wait(bar(tail->vfull[st]), (uint32_t)((J + j) / SV) & 1u, abort_flag, status))) {
                        ok = false;
                        break;
                    }
                    const int from = it.L - key0;
#pragma unroll 1
                    for (int z = r; z < (128 - from) * C::CH * 8; z += 128) {
                        const int vr = from + z / (C::CH * 8), cu = z % (C::CH * 8);
                        st_shared_v4(sV + st * C::TILE + (uint32_t)((cu >> 3) * C::CHUNK + vr * 128 + ((cu & 7) << 4)), 0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(tail->pfull[t]));
                l = l * alpha + rowsum;
            }
            J += it.tiles;
            if (!ok) break;
            if (!__all_sync(0xffffffffu, lean_wait(bar(tail->odone[t]), (uint32_t)no & 1u, abort_flag, status))) {
                ok = false;
                break;
            }
            ++no;
            tc_fence_after();
            // zeros where the mask leaves nothing (a padding row), which only the mask can tell: a row whose scores
            // are all NaN or -inf has no weights either and is NaN
            const bool sees = row - it.L + 1 < a.window || a.sinks > 0;
            const float inv = sees ? 1.f / l : 0.f;
            const __nv_bfloat16* g = GATE ? gate + ((int64_t)it.b * a.T + row) * ldg + (int64_t)it.head * HD : nullptr;
#pragma unroll 1
            for (int cc = 0; cc < HD; cc += 32) {
                uint32_t o[32];
                tmem_ld32(o_col + cc, o);
                tmem_wait_ld();
                if (cc + 32 == HD) {  // all of O is read: the next query tile's product may start
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(tail->ofree[t]));
                }
                if (store) {
#pragma unroll
                    for (int e = 0; e < 32; e += 16) {
                        float f[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(o[e + i]) * inv;
                        if constexpr (GATE) {
#pragma unroll
                            for (int i = 0; i < 16; i += 8) {
                                const uint4 w = __ldg(reinterpret_cast<const uint4*>(g + cc + e + i));
                                const uint32_t gw[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                                for (int x = 0; x < 4; ++x) {  // sigmoid(x) = 1 / (1 + 2^(-x log2 e))
                                    const float g0 = __uint_as_float(gw[x] << 16), g1 = __uint_as_float(gw[x] & 0xFFFF0000u);
                                    f[i + 2 * x] *= __fdividef(1.f, 1.f + ex2_approx(-1.4426950408889634f * g0));
                                    f[i + 2 * x + 1] *= __fdividef(1.f, 1.f + ex2_approx(-1.4426950408889634f * g1));
                                }
                            }
                        }
                        uint32_t y[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
                        if (wide) {
                            st_global_v8(out + cc + e, y);
                        } else {
                            *reinterpret_cast<uint4*>(out + cc + e) = make_uint4(y[0], y[1], y[2], y[3]);
                            *reinterpret_cast<uint4*>(out + cc + e + 8) = make_uint4(y[4], y[5], y[6], y[7]);
                        }
                    }
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int HD, bool GATE>
cudaError_t launch(const void* Q, int64_t ldq, const void* K, int64_t ldk, const void* V, int64_t ldv, const void* G,
                   int64_t ldg, void* O, int64_t ldo, int B, int h, int h_kv, int T, int window, int sinks,
                   const int32_t* kv_lengths, int num_sms, int* status, cudaStream_t stream) {
    using C = WnCfg<HD>;
    WnMaps maps;
    auto encode = [&](CUtensorMap* m, const void* x, int64_t ld, int heads) {
        const uint64_t dims[3] = {(uint64_t)heads * HD, (uint64_t)T, (uint64_t)B};
        const uint64_t strides[2] = {(uint64_t)ld * 2, (uint64_t)ld * 2 * (uint64_t)T};
        const uint32_t box[3] = {64, 128, 1};
        return encode_tmap_bf16(m, x, 3, dims, strides, box);
    };
    if (!encode(&maps.q, Q, ldq, h) || !encode(&maps.k, K, ldk, h_kv) || !encode(&maps.v, V, ldv, h_kv)) return cudaErrorInvalidValue;
    auto kernel = window_bf16_kernel<HD, GATE>;
    // setmaxnreg.inc waits until the block's register pool can grant the rise: refuse to launch a
    // build whose register count cannot cover the split
    static std::atomic<int> pool_ok{-1};
    int ok = pool_ok.load(std::memory_order_relaxed);
    if (ok < 0) {
        cudaFuncAttributes fa;
        const cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
        if (e != cudaSuccess) return e;
        ok = fa.numRegs * WN_THREADS >= 128 * WN_REGS_CTRL + 256 * WN_REGS_SOFTMAX ? 1 : 0;
        pool_ok.store(ok, std::memory_order_relaxed);
    }
    if (!ok) return cudaErrorInvalidConfiguration;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (err != cudaSuccess) return err;
    WnArgs a;
    a.B = B;
    a.h = h;
    a.h_kv = h_kv;
    a.T = T;
    a.window = window;
    a.sinks = sinks;
    a.n_qb = (T + 255) / 256;
    a.items = (int64_t)B * h * a.n_qb;
    a.lengths = kv_lengths;
    const int64_t grid = a.items < num_sms ? a.items : num_sms;
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(WN_THREADS), C::SMEM, stream, maps, a,
                      reinterpret_cast<const __nv_bfloat16*>(G), ldg, reinterpret_cast<__nv_bfloat16*>(O), ldo,
                      (float)(1.4426950408889634 / sqrt((double)HD)), status);
}

}  // namespace

cudaError_t launch_window_bf16(const void* Q, int64_t ldq, const void* K, int64_t ldk, const void* V, int64_t ldv,
                               const void* G, int64_t ldg, void* O, int64_t ldo, int B, int h, int h_kv, int T, int d,
                               int window, int sinks, const int32_t* kv_lengths, int num_sms, int* status,
                               cudaStream_t stream) {
#define MHA_WN(HD, GATE)                                                                                            \
    if (d == HD && (G != nullptr) == GATE)                                                                          \
        return launch<HD, GATE>(Q, ldq, K, ldk, V, ldv, G, ldg, O, ldo, B, h, h_kv, T, window, sinks, kv_lengths, \
                                num_sms, status, stream);
    MHA_WN(64, false) MHA_WN(64, true) MHA_WN(128, false) MHA_WN(128, true)
#undef MHA_WN
    return cudaErrorInvalidValue;
}

}  // namespace mha
