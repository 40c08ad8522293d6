// span_bf16.cu -- the cache operators of bf16 layers on tcgen05, one launch each: the windowed, shared-
// prefix and weight-accumulating decode steps (span.cuh).
//
// Bound by HBM for the few query rows of a decode step: every visible cached key and value is read once,
// 4 d bytes per token and K/V head.  A persistent CTA per SM takes an even run of 128-key tiles from the
// sequence of all groups (span.cuh); its TMA ring, MMAs and softmax run on across the borders between
// pieces, so neither ragged lengths nor many short windows leave the memory system idle.
//
// The up to 128 query rows of a piece form one tile (rows past them hold whatever lies in shared memory:
// each row's results depend on that row alone).  Alternate key tiles go to two streams, each with its own
// softmax warpgroup, running reference maximum, sum and output accumulator, so that one stream's
// exponentials run under the other's MMAs; a piece's end joins the two.  Tiles that end early (sinks,
// ends of caches) are loaded in boxes of 16 rows and multiplied with as few columns and steps.
//
// When a CTA is through, it waits for the others (a cooperative launch, so all of them run; the wait gives
// up after a second like every other) and then joins its share of the rows that several pieces hold, and
// of the attention weights.  As a kernel of its own that took 12 to 16 us of a step: its blocks find no
// room until these CTAs end, and the next step's CTAs none until they are gone.
//
// Tensor memory (512 columns): S_t at 128 t (P_t overwrites its first 64 columns), O_t at 256 + HD t.
// Warp roles (384 threads): warp 0 TMA; warp 1 TMEM owner and MMA issuer, in the order S(0), S(1), then
// O += P(j) V(j), S(j + 2) for j = 0, 1, ... (MMAs of one thread execute in issue order, so S(j + 2) may
// overwrite the P(j) columns); warps 2-3 gather the next piece's query rows; warps 4-7 softmax of stream 0
// and the pieces' ends, warps 8-11 softmax of stream 1 (thread = query row).
#include <math.h>

#include <atomic>

#include "internal.h"
#include "ptx.cuh"
#include "span_join.cuh"

namespace mha {
namespace {

constexpr int SP_THREADS = 384;
constexpr int SP_TK = 128;   // keys per tile
constexpr int SP_BOX = 16;   // rows of a box of a tile that ends early
// Registers per thread after the split: warps 0-3, and the softmax warps (whose score row, packed
// weights and an output chunk want 200).  The sum fits the 168 per thread of the launch.
constexpr int SP_REGS = 168;  // at launch
constexpr int SP_REGS_CTRL = 88;
constexpr int SP_REGS_SOFTMAX = 208;
static_assert(128 * SP_REGS_CTRL + 256 * SP_REGS_SOFTMAX <= SP_THREADS * SP_REGS, "register split");

template <int HD>
struct SpCfg {
    static constexpr int CH = HD / 64;             // 64-column chunks of a row
    static constexpr int CHUNK = 128 * 128;        // 128 rows x 64 bf16
    static constexpr int TILE = CH * CHUNK;
    static constexpr int STAGES = HD == 128 ? 3 : 6;
    static constexpr int SMEM = TILE + 2 * STAGES * TILE + 1024 + 1024 + 1024;  // + row sums, barriers, alignment
    static constexpr uint32_t O_COL = 256;
};
static_assert(SpCfg<128>::SMEM <= 232448 && SpCfg<64>::SMEM <= 232448, "span smem budget");

// What follows the tiles in shared memory.
struct SpTail {
    float2 ml1[128];  // stream 1's (reference, sum) per row at a piece's end
    uint64_t kfull[6], kempty[6], vfull[6], vempty[6];
    uint64_t qfull[2], qfree[2], sfull[2], pfull[2];
    uint64_t odone, ofree, ml, drain;
    uint32_t tmem;
    int abort_flag, joined;
};
static_assert(sizeof(SpTail) <= 2048, "span tail");

struct SpMaps {
    CUtensorMap k, v, k16, v16, kp, vp, kp16, vp16;
};

// One row of a score tile from TMEM (warp-collective).
__device__ __forceinline__ void load_scores(uint32_t taddr, float (&x)[128]) {
    uint32_t sr[4][32];
#pragma unroll
    for (int c = 0; c < 4; ++c) tmem_ld32(taddr + c * 32, sr[c]);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < 128; ++c) x[c] = __uint_as_float(sr[c >> 5][c & 31]);
}

// 32-byte store, a whole sector.
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// One thread of every CTA of a cooperative grid: waits until all have arrived.  The two words behind the
// status word (arrivals, generation) are as they were when it is over, so nothing has to clear them
// between launches; a CTA arrives whatever happened to it before.
__device__ __forceinline__ bool span_grid_barrier(int* status, int ctas) {
    unsigned* arrived = reinterpret_cast<unsigned*>(status) + 1;
    volatile unsigned* generation = reinterpret_cast<unsigned*>(status) + 2;
    const unsigned g = *generation;
    __threadfence();
    if (atomicAdd(arrived, 1u) == (unsigned)ctas - 1u) {
        *arrived = 0u;
        __threadfence();
        *generation = g + 1u;
        return true;
    }
    const uint64_t t0 = globaltimer_ns();
    while (*generation == g)
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            record_status(status, kStatusTimeout);
            return false;
        }
    __threadfence();
    return true;
}

template <int HD>
__global__ void __launch_bounds__(SP_THREADS, 1)
    span_bf16_kernel(const __grid_constant__ SpMaps maps, const __grid_constant__ SpanShape p, const SpanRecords rec,
                     const __nv_bfloat16* __restrict__ Q, int64_t ldq, __nv_bfloat16* __restrict__ O, int64_t ldo,
                     const int32_t* __restrict__ lengths, float* scores, float* __restrict__ weights, float scale_log2,
                     int* status) {
    using C = SpCfg<HD>;
    constexpr int S = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t sQ = base;
    const uint32_t sK = sQ + C::TILE;
    const uint32_t sV = sK + S * C::TILE;
    SpTail* tail = reinterpret_cast<SpTail*>(smem_raw + (base - raw) + C::TILE * (1 + 2 * S));
    volatile int* abort_flag = &tail->abort_flag;
    auto bar = [](uint64_t& b) { return smem_u32(&b); };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
        for (int s = 0; s < S; ++s) {
            mbar_init(bar(tail->kfull[s]), 1);
            mbar_init(bar(tail->kempty[s]), 1);
            mbar_init(bar(tail->vfull[s]), 1);
            mbar_init(bar(tail->vempty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(tail->qfull[i]), 64);
            mbar_init(bar(tail->qfree[i]), 1);
            mbar_init(bar(tail->sfull[i]), 1);
            mbar_init(bar(tail->pfull[i]), 4);
        }
        mbar_init(bar(tail->odone), 1);
        mbar_init(bar(tail->ofree), 4);
        mbar_init(bar(tail->ml), 4);
        mbar_init(bar(tail->drain), 1);
        tail->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tail->tmem), 512);
        tmem_relinquish();
    }
    grid_launch_dependents();
    const SpanStart start = span_start<SP_TK>(p, lengths);
    if (blockIdx.x == 0)
        for (int b = (int)threadIdx.x; b < p.B; b += SP_THREADS)
            if (lengths[b] < p.T_q || lengths[b] > p.T_max) record_status(status, kStatusBadLength);
    SpanPiece q;
    // query rows of a piece, and where row r of it lies
    auto n_rows = [&](const SpanPiece& x) { return min(128, (x.prefix ? p.B * p.rows : p.rows) - x.rb * 128); };
    auto where = [&](const SpanPiece& x, int r, int& b, int& head, int& t) {
        int rr = x.rb * 128 + r;
        b = x.b;
        if (x.prefix) {
            b = rr / p.rows;
            rr -= b * p.rows;
        }
        const int hg = rr / p.T_q;
        head = x.g * p.per + hg;
        t = rr - hg * p.T_q;
    };
    // The query tile is two buffers of 64 rows: a piece of at most 64 rows takes them in turn, a larger one
    // both.  uses[i]: pieces that have had buffer i.
    struct QueryBuffers {
        int uses[2] = {0, 0}, turn = 0;
        // first and last buffer of the next piece
        __device__ int first(int nr) const { return nr > 64 ? 0 : turn; }
        __device__ int last(int nr) const { return nr > 64 ? 1 : turn; }
        __device__ void take(int nr) {
            if (nr > 64) {
                ++uses[0];
                ++uses[1];
            } else {
                ++uses[turn];
                turn ^= 1;
            }
        }
    };
    // One warp copies query rows [r0, r0 + 32) of a piece of nr rows, 128-byte swizzled like a TMA box: a
    // lane finds one row, a step copies 32 / U rows of U 16-byte units.
    auto gather = [&](const SpanPiece& x, int nr, int buf, int r0) {
        constexpr int U = HD / 8, PER = 32 / U;
        int b, head, t;
        where(x, min(r0 + lane, nr - 1), b, head, t);
        const int64_t off = ((int64_t)b * p.T_q + t) * ldq + (int64_t)head * HD;
        const int u = lane & (U - 1), c = u >> 3;
#pragma unroll 4
        for (int i = 0; i < 32 && r0 + i < nr; i += PER) {
            const int r = r0 + i + lane / U;
            const int64_t o = __shfl_sync(0xffffffffu, off, i + lane / U);
            if (r < nr) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(Q + o + u * 8));
                st_shared_v4(sQ + (uint32_t)(buf * 64 * 128 + c * C::CHUNK + r * 128) + ((uint32_t)((u & 7) ^ (r & 7)) << 4),
                             v.x, v.y, v.z, v.w);
            }
        }
        fence_proxy_async_smem();
    };
    // warp 0, lane 0: tiles through the ring.  nk, nv: K and V tiles issued
    SpanWalk<SP_TK> walk(p, lengths, start);
    SpanPiece qt;
    int i_t = 0, nk = 0, nv = 0;
    bool ok = true;
    qt.i1 = 0;
    auto next_t = [&]() {
        if (!walk.next(qt)) return false;
        i_t = qt.i0;
        return true;
    };
    auto load_tile = [&]() {
        int key0, n;
        span_tile<SP_TK>(qt.v, i_t, key0, n);
        ++i_t;
        const int boxes = n > SP_TK - SP_BOX ? 0 : (n + SP_BOX - 1) / SP_BOX;
        const uint32_t bytes = boxes ? (uint32_t)boxes * SP_BOX * 128 * C::CH : (uint32_t)C::TILE;
        const int st = nk % S;
        const uint32_t ph = ((uint32_t)(nk / S) & 1u) ^ 1u;
        auto load = [&](uint32_t dst, const CUtensorMap* m, const CUtensorMap* m16, uint32_t full) {
            mbar_arrive_expect_tx(full, bytes);
#pragma unroll
            for (int c = 0; c < C::CH; ++c) {
                if (boxes == 0) tma_load_3d(dst + c * C::CHUNK, m, qt.g * HD + c * 64, key0, qt.b, full);
                for (int x = 0; x < boxes; ++x)
                    tma_load_3d(dst + c * C::CHUNK + x * SP_BOX * 128, m16, qt.g * HD + c * 64, key0 + x * SP_BOX, qt.b, full);
            }
        };
        ok = mbar_wait(bar(tail->kempty[st]), ph, abort_flag, status);
        if (!ok) return;
        load(sK + st * C::TILE, qt.prefix ? &maps.kp : &maps.k, qt.prefix ? &maps.kp16 : &maps.k16, bar(tail->kfull[st]));
        ++nk;
        ok = mbar_wait(bar(tail->vempty[st]), ph, abort_flag, status);
        if (!ok) return;
        load(sV + st * C::TILE, qt.prefix ? &maps.vp : &maps.v, qt.prefix ? &maps.vp16 : &maps.v16, bar(tail->vfull[st]));
        ++nv;
    };
    if (warp == 0) {
        // the ring's first fill needs nobody else (this thread set the barriers up): before the block meets
        if (lane == 0)
            while (nk < S && (i_t < qt.i1 || next_t())) load_tile();
    } else if (warp >= 4 && warp < 8) {  // the first piece's rows
        SpanWalk<SP_TK> first = walk;
        if (first.next(q)) {
            const int nr = n_rows(q);
            if ((warp - 4) * 32 < nr) gather(q, nr, 0, (warp - 4) * 32);
        }
    }
    __syncwarp();  // the block's barrier has to see whole warps
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tail->tmem;

    if (warp < 4) {
      setmaxnreg_dec<SP_REGS_CTRL>();
      if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA: K and V tiles
            while (ok && (i_t < qt.i1 || next_t())) load_tile();
            // every load issued lands before the CTA exits
            for (int i = nk > S ? nk - S : 0; i < nk; ++i) drain_wait_a(bar(tail->kfull[i % S]), (uint32_t)(i / S) & 1u);
            for (int i = nv > S ? nv - S : 0; i < nv; ++i) drain_wait_a(bar(tail->vfull[i % S]), (uint32_t)(i / S) & 1u);
        }
      } else if (warp == 1) {
        if (lane == 0) {
            // ---------------- MMA issuer.  js, jp: score and value products issued so far
            const uint64_t qdesc0 = sdesc_sw128(sQ, 16, 1024);
            const uint64_t kdesc0 = sdesc_sw128(sK, 16, 1024);
            const uint64_t vdesc0 = sdesc_sw128(sV, C::CHUNK, 1024);
            SpanWalk<SP_TK> ahead(p, lengths, start);  // walks the score products, two tiles ahead
            SpanPiece qs;
            QueryBuffers qb;
            int js = 0, piece_s = -1, i_s = 0, nr_s = 0, buf_s = 0;
            qs.i1 = 0;
            bool more_s = true;
            auto cols = [&](const SpanPiece& x, int i) {  // keys of a tile in whole boxes
                int key0, n;
                span_tile<SP_TK>(x.v, i, key0, n);
                return n > SP_TK - SP_BOX ? SP_TK : (n + SP_BOX - 1) / SP_BOX * SP_BOX;
            };
            auto issue_s = [&]() -> bool {
                if (i_s == qs.i1) {
                    if (!more_s || !(more_s = ahead.next(qs))) return true;
                    i_s = qs.i0;
                    ++piece_s;
                    nr_s = n_rows(qs);
                    buf_s = qb.first(nr_s);
                    // (for the first piece too, whose rows were there before the roles parted: a warp that
                    // gathers must not be a phase ahead of the other)
                    for (int x = buf_s; x <= qb.last(nr_s); ++x)
                        if (!mbar_wait(bar(tail->qfull[x]), (uint32_t)qb.uses[x] & 1u, abort_flag, status)) return false;
                }
                const int st = js % S;
                if (!mbar_wait(bar(tail->kfull[st]), (uint32_t)(js / S) & 1u, abort_flag, status)) return false;
                tc_fence_after();
                const uint32_t idesc = idesc_bf16_f32(128, cols(qs, i_s), false, false);
                const uint64_t kdesc = kdesc0 + (uint64_t)((st * C::TILE) >> 4);
                const uint64_t qdesc = qdesc0 + (uint64_t)((buf_s * 64 * 128) >> 4);
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                    const uint32_t off16 = (uint32_t)(((kk >> 2) * C::CHUNK + (kk & 3) * 32) >> 4);
                    mma_bf16_ss(tmem + 128u * (js & 1), qdesc + off16, kdesc + off16, idesc, kk > 0 ? 1u : 0u);
                }
                tc_commit(bar(tail->sfull[js & 1]));
                tc_commit(bar(tail->kempty[st]));
                ++js;
                if (++i_s == qs.i1) {
                    for (int x = buf_s; x <= qb.last(nr_s); ++x) tc_commit(bar(tail->qfree[x]));
                    qb.take(nr_s);
                }
                return true;
            };
            bool ok = issue_s() && issue_s();
            int jp = 0;
            for (int piece = 0; ok && walk.next(q); ++piece) {
                // the piece before has been read out of O
                if (piece > 0) ok = mbar_wait(bar(tail->ofree), (uint32_t)(piece - 1) & 1u, abort_flag, status);
                for (int i = q.i0; i < q.i1 && ok; ++i) {
                    const int st = jp % S, t = jp & 1;
                    ok = mbar_wait(bar(tail->vfull[st]), (uint32_t)(jp / S) & 1u, abort_flag, status) &&
                         mbar_wait(bar(tail->pfull[t]), (uint32_t)(jp >> 1) & 1u, abort_flag, status);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t idesc = idesc_bf16_f32(128, HD, false, true);
                    const uint64_t vdesc = vdesc0 + (uint64_t)((st * C::TILE) >> 4);
                    const int steps = cols(q, i) / 16;
                    const bool first = i - q.i0 < 2;  // of its stream
                    for (int kk = 0; kk < steps; ++kk)
                        mma_bf16_ts(tmem + C::O_COL + HD * t, tmem + 128u * t + kk * 8,
                                    vdesc + (uint64_t)((kk * 2048) >> 4), idesc, (!first || kk > 0) ? 1u : 0u);
                    tc_commit(bar(tail->vempty[st]));
                    if (i + 1 == q.i1) tc_commit(bar(tail->odone));
                    ++jp;
                    ok = issue_s();
                }
            }
            tc_commit(bar(tail->drain));
            drain_wait_a(bar(tail->drain), 0);
        }
      } else {
        // ---------------- the next pieces' query rows, into the buffers as they become free
        QueryBuffers qb;
        bool ok = true;
        for (int piece = 0; ok && walk.next(q); ++piece) {
            const int nr = n_rows(q), buf = qb.first(nr), end = qb.last(nr);
            if (piece > 0) {
                for (int x = buf; x <= end && ok; ++x)
                    if (qb.uses[x] > 0) ok = mbar_wait(bar(tail->qfree[x]), (uint32_t)(qb.uses[x] - 1) & 1u, abort_flag, status);
                if (!ok) break;
                for (int r0 = (warp - 2) * 32; r0 < nr; r0 += 64) gather(q, nr, buf, r0);
            }
            for (int x = buf; x <= end; ++x) mbar_arrive(bar(tail->qfull[x]));
            qb.take(nr);
        }
      }
      // the tensor memory goes back once the softmax warps have read it
      __syncwarp();
      named_barrier_sync(1, SP_THREADS);
      if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
      }
    } else {
        setmaxnreg_inc<SP_REGS_SOFTMAX>();
        // ---------------- softmax of stream t; stream 0's warps also end the pieces
        const int t = (warp - 4) >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t s_col = trow + 128u * t, o_col = trow + C::O_COL + HD * t;
        int j = 0;  // tiles before this piece
        bool ok = true;
        for (int piece = 0; ok && walk.next(q); ++piece) {
            const int nr = n_rows(q), nt = q.i1 - q.i0;
            const bool active = quarter * 32 < nr, real = r < nr;
            int rb_, head, tok;
            where(q, real ? r : 0, rb_, head, tok);
            const int pos = q.v.L - p.T_q + tok;
            float m = -INFINITY, l = 0.f;
            for (int k = (j ^ t) & 1; k < nt; k += 2) {
                if (!__all_sync(0xffffffffu, mbar_wait(bar(tail->sfull[t]), (uint32_t)((j + k) >> 1) & 1u, abort_flag, status))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                int key0, n;
                span_tile<SP_TK>(q.v, q.i0 + k, key0, n);
                if (n % SP_BOX != 0) {
                    // rows past the end may hold anything: zero the V rows the product would multiply by
                    // P = 0 (a NaN there would survive it)
                    const int st = (j + k) % S;
                    if (!__all_sync(0xffffffffu, mbar_wait(bar(tail->vfull[st]), (uint32_t)((j + k) / S) & 1u, abort_flag, status))) {
                        ok = false;
                        break;
                    }
                    const int rows = (n + SP_BOX - 1) / SP_BOX * SP_BOX - n;
                    for (int z = quarter * 32 + lane; z < rows * C::CH * 8; z += 128) {
                        const int row = n + z / (C::CH * 8), cu = z % (C::CH * 8);
                        st_shared_v4(sV + st * C::TILE + (uint32_t)((cu >> 3) * C::CHUNK + row * 128 + ((cu & 7) << 4)), 0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                if (active) {
                    if (n < SP_TK || (!q.prefix && (key0 + n > q.v.L - p.T_q ||
                                                    (key0 <= q.v.L - 1 - p.window && key0 + n > p.sinks)))) {
                        // some row does not see all of the tile: mask the scores where they lie, so that
                        // the other tiles' code carries no masks
                        const int hi = q.prefix ? n : min(n, pos + 1 - key0);
                        const int lo = q.prefix ? 0 : pos - p.window + 1 - key0, sk = p.sinks - key0;
#pragma unroll 1
                        for (int c = 0; c < SP_TK; c += 32) {
                            uint32_t sr[32];
                            tmem_ld32(s_col + c, sr);
                            tmem_wait_ld();
#pragma unroll
                            for (int u = 0; u < 32; ++u)
                                if (c + u >= hi || (c + u < lo && c + u >= sk)) sr[u] = 0xFF800000u;
                            tmem_st32(s_col + c, sr);
                        }
                        tmem_wait_st();
                    }
                    if (scores != nullptr && !q.prefix) {
                        // (the loads are warp-wide; a group's padding rows store nothing, keys past the end
                        // are masked and lie in the row's padding)
                        float4* out = reinterpret_cast<float4*>(
                            scores + (((int64_t)q.b * p.h_kv + q.g) * p.rows + q.rb * 128 + (real ? r : 0)) * score_ld(p) + key0);
#pragma unroll 1
                        for (int c = 0; c < n; c += 32) {
                            uint32_t sr[32];
                            tmem_ld32(s_col + c, sr);
                            tmem_wait_ld();
#pragma unroll
                            for (int u = 0; u < 32; u += 4)
                                if (real && c + u < n)
                                    out[(c + u) / 4] = make_float4(__uint_as_float(sr[u]) * scale_log2, __uint_as_float(sr[u + 1]) * scale_log2,
                                                                   __uint_as_float(sr[u + 2]) * scale_log2, __uint_as_float(sr[u + 3]) * scale_log2);
                        }
                    }
                    // any reference m gives the same O / l as long as P stays finite: keep it until a row's
                    // sum passes 2^64 (or is not finite: m = -inf), then take the tile's maximum and redo
                    uint32_t pk[64];
                    float alpha = 1.f, rowsum;
                    bool renew = k < 2;
                    for (;;) {
                        float x[128];
                        load_scores(s_col, x);
                        if (renew) {
                            const float m_new = fmaxf(m, row_max(x) * scale_log2);
                            alpha = m_new == -INFINITY ? 1.f : ex2_approx(m - m_new);  // 0 when m leaves -inf
                            const bool rescale = real && m_new != m && k >= 2;
                            // S(j) was issued after the value product of this stream's last tile: O is complete
                            if (__any_sync(0xffffffffu, rescale)) {
                                const float a = rescale ? alpha : 1.f;
#pragma unroll 1
                                for (int cc = 0; cc < HD; cc += 32) {
                                    uint32_t o[32];
                                    tmem_ld32(o_col + cc, o);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                                    tmem_st32(o_col + cc, o);
                                }
                            }
                            m = m_new;
                        }
                        rowsum = exp_tile(x, pack2(scale_log2, scale_log2), m == -INFINITY && renew ? 0.f : -m, pk);
                        if (renew) break;
                        renew = !__all_sync(0xffffffffu, !real || rowsum <= 18446744073709551616.f);
                        if (!renew) break;
                    }
                    {
                        uint32_t (&p0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&pk[0]);
                        uint32_t (&p1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&pk[32]);
                        tmem_st32(s_col, p0);
                        tmem_st32(s_col + 32, p1);
                    }
                    tmem_wait_st();
                    l = l * alpha + rowsum;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(tail->pfull[t]));
            }
            if (!ok) break;
            // ---------------- the piece's end
            if (t == 1) {
                // the piece before has read ml1
                if (piece > 0 && !__all_sync(0xffffffffu, mbar_wait(bar(tail->ofree), (uint32_t)(piece - 1) & 1u, abort_flag, status))) {
                    ok = false;
                    break;
                }
                tail->ml1[r] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(tail->ml));
            } else {
                if (!__all_sync(0xffffffffu, mbar_wait(bar(tail->odone), (uint32_t)piece & 1u, abort_flag, status) &&
                                                 mbar_wait(bar(tail->ml), (uint32_t)piece & 1u, abort_flag, status))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (active) {
                    const float2 ml1 = tail->ml1[r];
                    const float M = fmaxf(m, ml1.x);
                    // the first tile of the piece went to stream j & 1
                    const bool has0 = nt > 1 || (j & 1) == 0, has1 = nt > 1 || (j & 1) == 1;
                    const float w0 = m == -INFINITY ? 0.f : ex2_approx(m - M);
                    const float w1 = ml1.x == -INFINITY ? 0.f : ex2_approx(ml1.x - M);
                    const float sum = w0 * l + w1 * ml1.y;
                    const bool direct = p.T_p == 0 && q.whole();
                    const int64_t row = rec.row(p, q.prefix, q.block, (int)blockIdx.x / p.gang, (int)blockIdx.x % p.gang) + r;
                    if (real && (!direct || scores != nullptr)) rec.ml[row] = make_float2(M, sum);
                    const float inv = 1.f / sum;
                    __nv_bfloat16* out = O + ((int64_t)rb_ * p.T_q + tok) * ldo + (int64_t)head * HD;
                    float* part = rec.o + row * HD;
                    const bool wide = ((reinterpret_cast<uintptr_t>(O) | (uintptr_t)(ldo * 2)) & 31u) == 0;
#pragma unroll
                    for (int cc = 0; cc < HD / 32; ++cc) {
                        float f[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) f[e] = 0.f;
                        if (has0) {
                            uint32_t a[32];
                            tmem_ld32(trow + C::O_COL + cc * 32, a);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) f[e] = w0 * __uint_as_float(a[e]);
                        }
                        if (has1) {
                            uint32_t a[32];
                            tmem_ld32(trow + C::O_COL + HD + cc * 32, a);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) f[e] = fmaf(w1, __uint_as_float(a[e]), f[e]);
                        }
                        if (real && direct) {
#pragma unroll
                            for (int e = 0; e < 32; e += 16) {
                                uint32_t y[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) y[i] = pack_bf16x2(f[e + 2 * i] * inv, f[e + 2 * i + 1] * inv);
                                if (wide)
                                    st_global_v8(out + cc * 32 + e, y);
                                else {
                                    *reinterpret_cast<uint4*>(out + cc * 32 + e) = make_uint4(y[0], y[1], y[2], y[3]);
                                    *reinterpret_cast<uint4*>(out + cc * 32 + e + 8) = make_uint4(y[4], y[5], y[6], y[7]);
                                }
                            }
                        } else if (real) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8) {
                                uint32_t y[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) y[i] = __float_as_uint(f[e + i]);
                                st_global_v8(part + cc * 32 + e, y);
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(tail->ofree));
            }
            j += nt;
        }
        __syncwarp();
        tc_fence_before();
        __threadfence();  // the records, before this CTA counts as arrived
        named_barrier_sync(1, SP_THREADS);
        // ---------------- all pieces are done: join
        // (by the softmax warps: they have the registers)
        constexpr int JOIN = 256, JOIN_WARPS = JOIN / 32;
        const int jw = warp - 4;
        if (jw == 0 && lane == 0) tail->joined = span_grid_barrier(status, (int)gridDim.x) ? 1 : 0;
        named_barrier_sync(2, JOIN);
        if (!tail->joined) return;
        const int gangs = (int)gridDim.x / p.gang;
        const int heads = p.per * p.h_kv, out_rows = p.B * heads * p.T_q;
        {
            // rows in turn to the CTAs, whose warps share a row's records, where there are few rows; to the
            // warps otherwise
            const bool few = out_rows <= (int)gridDim.x;
            float* sums = reinterpret_cast<float*>(smem_raw + (base - raw));  // [warp][column]
            for (int row = few ? (int)blockIdx.x : (int)blockIdx.x * JOIN_WARPS + jw; row < out_rows;
                 row += few ? (int)gridDim.x : (int)gridDim.x * JOIN_WARPS) {
                const int t = row % p.T_q, bh = row / p.T_q, b = bh / heads, head = bh - b * heads, g = head / p.per;
                const SpanView v = span_view<SP_TK>(p, lengths[b]);
                constexpr int E = HD / 32;  // columns per lane
                __nv_bfloat16* out = O + ((int64_t)b * p.T_q + t) * ldo + (int64_t)head * HD + lane * E;
                float o[E] = {}, l = 1.f;
                bool write = true;
                if (v.nt == 0) {  // invalid length
    #pragma unroll
                    for (int e = 0; e < E; ++e) o[e] = NAN;
                    write = !few || jw == 0;
                } else {
                    int N, off;
                    first_tile<SP_TK>(p, lengths, b, N, off);
                    RowRecords src[2];
                    row_sources<SP_TK>(p, rec, 128, gangs, v, b, g, (head - g * p.per) * p.T_q + t, N, off, src);
                    if (p.T_p == 0 && src[0].n == 1) continue;  // one piece held the whole group and wrote the row
                    const float2 ml = row_sum(rec, src);
                    l = ml.y;
    #pragma unroll 4
                    for (int c = few ? jw : 0; c < src[0].n + src[1].n; c += few ? JOIN_WARPS : 1) {
                        const int64_t k = c < src[0].n ? src[0].first + c * src[0].step : src[1].first + (c - src[0].n) * src[1].step;
                        const float m = __ldcg(rec.ml + k).x;
                        const float w = m == -INFINITY ? 0.f : ex2_approx(m - ml.x);
                        float x[E];
                        if constexpr (E == 4) {
                            const float4 y = __ldcg(reinterpret_cast<const float4*>(rec.o + k * HD) + lane);
                            x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
                        } else {
                            const float2 y = __ldcg(reinterpret_cast<const float2*>(rec.o + k * HD) + lane);
                            x[0] = y.x; x[1] = y.y;
                        }
    #pragma unroll
                        for (int e = 0; e < E; ++e) o[e] = fmaf(w, x[e], o[e]);
                    }
                    if (few) {
    #pragma unroll
                        for (int e = 0; e < E; ++e) sums[jw * HD + lane * E + e] = o[e];
                        named_barrier_sync(2, JOIN);
                        write = jw == 0;
                        if (write)
    #pragma unroll
                            for (int e = 0; e < E; ++e) {
                                float y = 0.f;
                                for (int w = 0; w < JOIN_WARPS; ++w) y += sums[w * HD + lane * E + e];
                                o[e] = y;
                            }
                        named_barrier_sync(2, JOIN);
                    }
                }
                if (write) {
                    const float inv = 1.f / l;
    #pragma unroll
                    for (int e = 0; e < E; e += 2)
                        *reinterpret_cast<uint32_t*>(out + e) = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
                }
            }
        }
        if (weights != nullptr) {
            // a token's weight is the sum over the query rows of 2^(s - M) / l, in row order.  A warp takes 256
            // tokens of one (batch, K/V head) at a time.
            constexpr int PER = 8, KEYS = 32 * PER;
            const int chunks = (p.T_max + KEYS - 1) / KEYS;
            const int64_t tasks = (int64_t)p.B * p.h_kv * chunks;
            for (int64_t task = (int64_t)blockIdx.x * JOIN_WARPS + jw; task < tasks; task += (int64_t)gridDim.x * JOIN_WARPS) {
                const int bg = (int)(task / chunks), k0 = (int)(task - (int64_t)bg * chunks) * KEYS;
                const int b = bg / p.h_kv, g = bg - b * p.h_kv;
                const SpanView v = span_view<SP_TK>(p, lengths[b]);
                if (v.nt == 0 || k0 >= v.L) continue;
                int N, off;
                first_tile<SP_TK>(p, lengths, b, N, off);
                float w[PER] = {}, old[PER];
                float* out = weights + (int64_t)bg * p.T_max + k0 + lane;
                // the new tokens' entries start here, the others grow
    #pragma unroll
                for (int u = 0; u < PER; ++u) old[u] = k0 + lane + 32 * u < v.L - p.T_q ? out[32 * u] : 0.f;
                for (int r0 = 0; r0 < p.rows; r0 += 32) {
                    const int nr = min(32, p.rows - r0);
                    float M = 0.f, il = 0.f;  // of row r0 + lane
                    for (int r = 0; r < nr; ++r) {
                        RowRecords src[2];
                        row_sources<SP_TK>(p, rec, 128, gangs, v, b, g, r0 + r, N, off, src);
                        const float2 ml = row_sum(rec, src);
                        if (lane == r) {
                            M = ml.x;
                            il = 1.f / ml.y;
                        }
                    }
                    const float* s = scores + ((int64_t)bg * p.rows + r0) * score_ld(p) + k0 + lane;
    #pragma unroll 2
                    for (int r = 0; r < nr; ++r) {
                        const float m = __shfl_sync(0xffffffffu, M, r), f = __shfl_sync(0xffffffffu, il, r);
    #pragma unroll
                        for (int u = 0; u < PER; ++u)
                            if (k0 + lane + 32 * u < v.L)
                                w[u] = fmaf(exp2f(__ldcg(s + (int64_t)r * score_ld(p) + 32 * u) - m), f, w[u]);
                    }
                }
    #pragma unroll
                for (int u = 0; u < PER; ++u)
                    if (k0 + lane + 32 * u < v.L) out[32 * u] = old[u] + w[u];
            }
        }
    }
}

template <int HD>
cudaError_t launch(const SpanShape& p, const SpanRecords& rec, const void* Q, int64_t ldq, const void* K, int64_t ldk,
                   const void* V, int64_t ldv, const void* Kp, int64_t ldkp, const void* Vp, int64_t ldvp, void* O,
                   int64_t ldo, const int32_t* lengths, float* scores, float* weights, int gangs, int* status,
                   cudaStream_t stream) {
    using C = SpCfg<HD>;
    SpMaps maps;
    auto encode = [&](CUtensorMap* full, CUtensorMap* part, const void* x, int64_t ld, int T, int B) {
        const uint64_t dims[3] = {(uint64_t)p.h_kv * HD, (uint64_t)T, (uint64_t)B};
        const uint64_t strides[2] = {(uint64_t)ld * 2, (uint64_t)ld * 2 * (uint64_t)T};
        const uint32_t box[3] = {64, SP_TK, 1}, box16[3] = {64, SP_BOX, 1};
        return encode_tmap_bf16(full, x, 3, dims, strides, box) && encode_tmap_bf16(part, x, 3, dims, strides, box16);
    };
    if (!encode(&maps.k, &maps.k16, K, ldk, p.T_max, p.B) || !encode(&maps.v, &maps.v16, V, ldv, p.T_max, p.B))
        return cudaErrorInvalidValue;
    if (p.T_p > 0) {
        if (!encode(&maps.kp, &maps.kp16, Kp, ldkp, p.T_p, 1) || !encode(&maps.vp, &maps.vp16, Vp, ldvp, p.T_p, 1))
            return cudaErrorInvalidValue;
    } else {
        maps.kp = maps.kp16 = maps.k;  // never used
        maps.vp = maps.vp16 = maps.v;
    }
    // setmaxnreg.inc waits until the block's register pool can grant the rise: refuse to launch a
    // build whose register count cannot cover the split
    static std::atomic<int> pool_ok{-1};
    int ok = pool_ok.load(std::memory_order_relaxed);
    if (ok < 0) {
        cudaFuncAttributes fa;
        const cudaError_t e = cudaFuncGetAttributes(&fa, span_bf16_kernel<HD>);
        if (e != cudaSuccess) return e;
        ok = fa.numRegs * SP_THREADS >= 128 * SP_REGS_CTRL + 256 * SP_REGS_SOFTMAX ? 1 : 0;
        pool_ok.store(ok, std::memory_order_relaxed);
    }
    if (!ok) return cudaErrorInvalidConfiguration;
    cudaError_t err = cudaFuncSetAttribute(span_bf16_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (err != cudaSuccess) return err;
    // Cooperative, and not started early behind the previous kernel: its CTAs wait for one another, so
    // they have to be placed together.
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(gangs * p.gang));
    cfg.blockDim = dim3(SP_THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, span_bf16_kernel<HD>, maps, p, rec, reinterpret_cast<const __nv_bfloat16*>(Q), ldq,
                              reinterpret_cast<__nv_bfloat16*>(O), ldo, lengths, scores, weights,
                              (float)(1.4426950408889634 / sqrt((double)HD)), status);
}

}  // namespace

cudaError_t launch_span_bf16(const SpanShape& p, const SpanRecords& rec, const void* Q, int64_t ldq, const void* K,
                             int64_t ldk, const void* V, int64_t ldv, const void* Kp, int64_t ldkp, const void* Vp,
                             int64_t ldvp, void* O, int64_t ldo, int d, const int32_t* lengths, float* scores,
                             float* weights, int gangs, int* status, cudaStream_t stream) {
    if (d == 64)
        return launch<64>(p, rec, Q, ldq, K, ldk, V, ldv, Kp, ldkp, Vp, ldvp, O, ldo, lengths, scores,
                          weights, gangs, status, stream);
    if (d == 128)
        return launch<128>(p, rec, Q, ldq, K, ldk, V, ldv, Kp, ldkp, Vp, ldvp, O, ldo, lengths, scores,
                           weights, gangs, status, stream);
    return cudaErrorInvalidValue;
}

}  // namespace mha
