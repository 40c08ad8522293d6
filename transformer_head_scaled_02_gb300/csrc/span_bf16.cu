// span_bf16.cu -- the cache operators of bf16 layers on tcgen05, one launch each: the windowed, shared-
// prefix and weight-accumulating decode steps (span.cuh).
//
// Bound by HBM for the few query rows of a decode step: every visible cached key and value is read once,
// 4 d bytes per token and K/V head.  Persistent CTAs, one per SM, take units of 128-key tiles (span.cuh) from a
// counter; the TMA ring, the MMAs and the softmax run on across the borders between units.
//
// The up to 128 query rows of a unit form one tile (rows past them hold whatever lies in shared memory:
// each row's results depend on that row alone).  Alternate key tiles go to two streams, each with its own
// softmax warpgroup, running reference maximum, sum and output accumulator, so that one stream's
// exponentials run under the other's MMAs; a unit's end joins the two.  Tiles that end early (sinks,
// ends of caches) are loaded in boxes of 16 rows.
//
// When a CTA is through, it waits for the others (a cooperative launch, so all of them run; the wait gives
// up after a second like every other) and then joins its share of the rows that several units hold, and
// of the attention weights.  As a kernel of its own that took 12 to 16 us of a step: its blocks find no
// room until these CTAs end, and the next step's CTAs none until they are gone.  Code that runs once per
// CTA is kept short throughout: it is fetched from L2 every time.
//
// The softmax weights are rounded to bf16 for the value product, as the tensor cores take them, by at most 2^-8
// of themselves; the row sums are of the fp32 values, and records, joins and accumulated weights stay fp32.
//
// Measured in a captured graph | in a loop of calls: 32 caches of up to 8192 tokens, 16 K/V heads of d = 128,
// window 4096 (1.08 GB) 167 | 169 us, 96 | 95 % of the measured copy rate; 4 K/V heads with weights (409 MB)
// 84 | 89 us, 73 | 69 %; 64 caches of up to 1024 tokens behind a prefix of 32768, 4 query heads each on 4 K/V
// heads, 62 | 65 us; one cache of 1004 visible tokens 12 | 14 us.  Short units
// cost most beside HBM: between two units a stream waits for the last value product and reads the sums, about
// 2 us.  The roles' loops share the instruction cache: with several copies of the score product and of the
// tile loads the same four took 177, 99, 68 and 12 us in a graph.  Slower, too: a unit's end behind the next unit's first
// softmax, few query rows twice in the tile for the two streams to run on two warp schedulers, boxes of 32 rows.
//
// Tensor memory (512 columns): S_t at 128 t (P_t overwrites its first 64 columns), O_t at 256 + HD t.
// Warp roles (384 threads): warp 0 TMA; warp 1 TMEM owner and MMA issuer (from the whole warp, see
// tc_issue.cuh), in the order S(0), S(1), then O += P(j) V(j), S(j + 2) for j = 0, 1, ... (MMAs of one thread
// execute in issue order, so S(j + 2) may overwrite the P(j) columns); warp 2 gathers the next units' query
// rows; warp 3 takes units and hands them to the others through a ring in shared memory; warps 4-7 softmax
// of stream 0, warps 8-11 of stream 1 (thread = query row), and each stream's warps half of a unit's end.
#include <math.h>

#include <atomic>

#include "internal.h"
#include "span_records.cuh"
#include "tc_issue.cuh"

namespace mha {
namespace {

constexpr int SP_THREADS = 384;
constexpr int SP_TK = 128;   // keys per tile
constexpr int SP_BOX = 16;   // rows of a box of a tile that ends early
constexpr int SP_RING = 4;   // units in flight
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
    static constexpr int SMEM = TILE + 2 * STAGES * TILE + 3 * 1024;  // + row sums, barriers, units
    static constexpr uint32_t O_COL = 256;
};
static_assert(SpCfg<128>::SMEM <= 232448 && SpCfg<64>::SMEM <= 232448, "span smem budget");

// What follows the tiles in shared memory.
struct SpTail {
    float2 ml[2][128];  // each stream's (reference, sum) per row at a unit's end
    uint64_t kfull[6], kempty[6], vfull[6], vempty[6];
    uint64_t qfull[2], qfree[2], sfull[2], pfull[2], ufull[SP_RING], uempty[SP_RING];
    uint64_t odone, ofree, mlfull, drain;
    SpanUnit units[SP_RING];
    int nr[SP_RING];  // query rows of the unit
    SpanPlan plan;
    uint32_t tmem;
    int abort_flag, joined;
    unsigned generation;
};
static_assert(sizeof(SpTail) <= 3 * 1024, "span tail");

struct SpMaps {
    CUtensorMap k, k16, v, v16, kp, kp16, vp, vp16;
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

// One thread of every CTA of a cooperative grid: waits until all have arrived; g: the generation word as it
// was when the CTA began.  The words behind the status word (arrivals, generation, units taken) are as they
// were when it is over, so nothing has to clear them between launches; a CTA arrives whatever happened to
// it before.
__device__ __forceinline__ unsigned span_generation(const int* status) {
    unsigned g;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(g) : "l"(status + 2) : "memory");
    return g;
}

__device__ __forceinline__ bool span_grid_barrier(int* status, int ctas, unsigned g) {
    unsigned before, now;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(status + 1) : "memory");
    if (before == (unsigned)ctas - 1u) {
        status[1] = 0;
        status[3] = 0;
        asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(status + 2), "r"(g + 1u) : "memory");
        return true;
    }
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(now) : "l"(status + 2) : "memory");
        if (now != g) return true;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            record_status(status, kStatusTimeout);
            return false;
        }
    }
}

template <int HD>
__global__ void __launch_bounds__(SP_THREADS, 1)
    span_bf16_kernel(const __grid_constant__ SpMaps maps, const __grid_constant__ SpanShape p, const SpanRecords rec,
                     const __nv_bfloat16* __restrict__ Q, int64_t ldq, __nv_bfloat16* __restrict__ O, int64_t ldo,
                     const int32_t* __restrict__ lengths, float* scores, float* __restrict__ weights, float scale_log2,
                     int* status) {
    using C = SpCfg<HD>;
    constexpr int S = C::STAGES;
    // (the tiles' swizzle wants 1024 bytes; there is no room to align by hand)
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t sQ = smem_u32(smem_raw);
    const uint32_t sK = sQ + C::TILE;
    const uint32_t sV = sK + S * C::TILE;
    SpTail* tail = reinterpret_cast<SpTail*>(smem_raw + C::TILE * (1 + 2 * S));
    volatile int* abort_flag = &tail->abort_flag;
    auto bar = [](uint64_t& b) { return smem_u32(&b); };

    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
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
            mbar_init(bar(tail->qfull[i]), 32);
            mbar_init(bar(tail->qfree[i]), 1);
            mbar_init(bar(tail->sfull[i]), 1);
            mbar_init(bar(tail->pfull[i]), 4);
        }
        for (int i = 0; i < SP_RING; ++i) {
            mbar_init(bar(tail->ufull[i]), 1);
            mbar_init(bar(tail->uempty[i]), 11);  // TMA, MMA, gather and the eight softmax warps
        }
        mbar_init(bar(tail->odone), 1);
        mbar_init(bar(tail->ofree), 8);
        mbar_init(bar(tail->mlfull), 8);
        mbar_init(bar(tail->drain), 1);
        tail->abort_flag = 0;
        tail->generation = span_generation(status);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tail->tmem), 512);
        tmem_relinquish();
    }
    grid_launch_dependents();
    // The i-th unit of this CTA, once it is there; its slot is released after the last look at it.
    auto unit_ready = [&](int i) { return lean_wait(bar(tail->ufull[i % SP_RING]), (uint32_t)(i / SP_RING) & 1u, abort_flag, status); };
    auto unit_done = [&](int i) { mbar_arrive(bar(tail->uempty[i % SP_RING])); };
    // where query row r of a unit lies
    auto where = [&](const SpanUnit& x, int r, int& b, int& head, int& t) {
        int rr = x.rb * 128 + r;
        b = x.b;
        if (x.prefix) {
            b = rr / p.rows;
            rr -= b * p.rows;
        }
        const int hg = p.T_q == 1 ? rr : rr / p.T_q;
        head = x.g * p.per + hg;
        t = rr - hg * p.T_q;
    };
    // The query tile is two buffers of 64 rows: a unit of at most 64 rows takes them in turn, a larger one
    // both.  uses[i]: units that have had buffer i.
    struct QueryBuffers {
        int uses[2] = {0, 0}, turn = 0;
        // first and last buffer of the next unit
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
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tail->tmem;

    if (warp < 4) {
      setmaxnreg_dec<SP_REGS_CTRL>();
      if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA: K and V tiles.  nk, nv: issued
            int nk = 0, nv = 0;
            bool ok = true;
#pragma unroll 1
            for (int i = 0; ok && unit_ready(i); ++i) {
                const SpanUnit& q = tail->units[i % SP_RING];
                if (q.unit < 0) break;
                const CUtensorMap* maps_k = q.prefix ? &maps.kp : &maps.k;  // the values' follow: k, k16, v, v16
                const int i1 = q.i1;
#pragma unroll 1
                for (int j2 = 2 * q.i0; j2 < 2 * i1; ++j2) {  // a tile's keys, then its values
                    int key0, n;
                    span_tile<SP_TK>(q.v, j2 >> 1, key0, n);
                    const bool val = j2 & 1;
                    const int st = nv % S;
                    const uint32_t full = bar(val ? tail->vfull[st] : tail->kfull[st]);
                    ok = lean_wait(bar(val ? tail->vempty[st] : tail->kempty[st]), ((uint32_t)(nv / S) & 1u) ^ 1u, abort_flag, status);
                    if (!ok) break;
                    const CUtensorMap* m = maps_k + (val ? 2 : 0);
                    const uint32_t dst = (val ? sV : sK) + st * C::TILE;
                    // the map with boxes of 16 rows follows the whole one
                    const int rows = n > SP_TK - SP_BOX ? SP_TK : SP_BOX, loads = rows == SP_TK ? 1 : (n + SP_BOX - 1) / SP_BOX;
                    mbar_arrive_expect_tx(full, (uint32_t)(loads * rows) * 128 * C::CH);
#pragma unroll 1
                    for (int x = 0; x < loads; ++x)
#pragma unroll
                        for (int c = 0; c < C::CH; ++c)
                            tma_load_3d(dst + c * C::CHUNK + x * SP_BOX * 128, rows == SP_TK ? m : m + 1, q.g * HD + c * 64, key0 + x * SP_BOX,
                                        q.b, full);
                    if (val)
                        ++nv;
                    else
                        ++nk;
                }
                unit_done(i);
            }
            // every load issued lands before the CTA exits
            for (int i = nk > S ? nk - S : 0; i < nk; ++i) drain_wait_a(bar(tail->kfull[i % S]), (uint32_t)(i / S) & 1u);
            for (int i = nv > S ? nv - S : 0; i < nv; ++i) drain_wait_a(bar(tail->vfull[i % S]), (uint32_t)(i / S) & 1u);
        }
      } else if (warp == 1) {
        // ---------------- MMA issuer.  js, jp: score and value products issued so far
        const uint32_t el = elect_lane(), tm = uniform(tmem);
        const uint64_t qdesc0 = sdesc_sw128(sQ, 16, 1024);
        const uint64_t kdesc0 = sdesc_sw128(sK, 16, 1024);
        const uint64_t vdesc0 = sdesc_sw128(sV, C::CHUNK, 1024);
        constexpr uint32_t idesc_s = idesc_bf16_f32(128, SP_TK, false, false);
        constexpr uint32_t idesc_o = idesc_bf16_f32(128, HD, false, true);
        QueryBuffers qb;
        int js = 0, us = -1, left_s = 0, nr_s = 0, buf_s = 0;  // us: the unit of the score products, left_s tiles of it
        bool more_s = true;
        // the next score product, if there is one
        auto issue_s = [&]() -> bool {
            if (left_s == 0) {
                if (!more_s) return true;
                if (!__all_sync(0xffffffffu, unit_ready(us + 1))) return false;
                const SpanUnit& x = tail->units[(us + 1) % SP_RING];
                if (uniform(x.unit) < 0) {
                    more_s = false;
                    return true;
                }
                ++us;
                left_s = uniform(x.i1 - x.i0);
                nr_s = uniform(tail->nr[us % SP_RING]);
                buf_s = qb.first(nr_s);
#pragma unroll 1
                for (int i = buf_s; i <= qb.last(nr_s); ++i)
                    if (!warp_wait(bar(tail->qfull[i]), (uint32_t)qb.uses[i] & 1u, abort_flag, status)) return false;
            }
            const int st = js % S;
            if (!warp_wait(bar(tail->kfull[st]), (uint32_t)(js / S) & 1u, abort_flag, status)) return false;
            tc_fence_after();
            const uint64_t kdesc = kdesc0 + (uint64_t)((st * C::TILE) >> 4);
            const uint64_t qdesc = qdesc0 + (uint64_t)((buf_s * 64 * 128) >> 4);
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
                const uint32_t off16 = (uint32_t)(((kk >> 2) * C::CHUNK + (kk & 3) * 32) >> 4);
                mma_bf16_ss_elect(el, tm + 128u * (js & 1), qdesc + off16, kdesc + off16, idesc_s, kk > 0 ? 1u : 0u);
            }
            tc_commit_elect(el, bar(tail->sfull[js & 1]));
            tc_commit_elect(el, bar(tail->kempty[st]));
            ++js;
            if (--left_s == 0) {
#pragma unroll 1
                for (int i = buf_s; i <= qb.last(nr_s); ++i) tc_commit_elect(el, bar(tail->qfree[i]));
                qb.take(nr_s);
            }
            return true;
        };
        bool ok = true;
        int jp = 0;
#pragma unroll 1
        for (int i = -1; ok; ++i) {
            // (unit -1: the first two score products, by the one copy of their code)
            int i0 = 0, nt = 2;
            SpanView v = {};
            if (i >= 0) {
                ok = __all_sync(0xffffffffu, unit_ready(i));
                const SpanUnit& x = tail->units[i % SP_RING];
                if (!ok || uniform(x.unit) < 0) break;
                i0 = x.i0;
                nt = uniform(x.i1 - i0);
                v = x.v;
            }
            // the unit before has been read out of O
            if (i > 0) ok = warp_wait(bar(tail->ofree), (uint32_t)(i - 1) & 1u, abort_flag, status);
#pragma unroll 1
            for (int k = 0; k < nt && ok; ++k) {
                if (i < 0) {
                    ok = issue_s();
                    continue;
                }
                const int st = jp % S, t = jp & 1;
                ok = warp_wait(bar(tail->vfull[st]), (uint32_t)(jp / S) & 1u, abort_flag, status) &&
                     warp_wait(bar(tail->pfull[t]), (uint32_t)(jp >> 1) & 1u, abort_flag, status);
                if (!ok) break;
                tc_fence_after();
                const uint64_t vdesc = vdesc0 + (uint64_t)((st * C::TILE) >> 4);
                int key0, n;
                span_tile<SP_TK>(v, i0 + k, key0, n);
                n = uniform(n);
                if (n > SP_TK - SP_BOX) {
#pragma unroll
                    for (int kk = 0; kk < SP_TK / 16; ++kk)
                        mma_bf16_ts_elect(el, tm + C::O_COL + HD * t, tm + 128u * t + kk * 8, vdesc + (uint64_t)((kk * 2048) >> 4), idesc_o,
                                          (k >= 2 || kk > 0) ? 1u : 0u);
                } else {  // values past the tile's end were not loaded: no steps over them
#pragma unroll 1
                    for (int kk = 0; 16 * kk < n; ++kk)
                        mma_bf16_ts_elect(el, tm + C::O_COL + HD * t, tm + 128u * t + kk * 8, vdesc + (uint64_t)((kk * 2048) >> 4), idesc_o,
                                          (k >= 2 || kk > 0) ? 1u : 0u);
                }
                tc_commit_elect(el, bar(tail->vempty[st]));
                if (k + 1 == nt) tc_commit_elect(el, bar(tail->odone));
                ++jp;
                ok = issue_s();
            }
            __syncwarp();
            if (ok && lane == 0 && i >= 0) unit_done(i);
        }
        tc_commit_elect(el, bar(tail->drain));
        drain_wait_a(bar(tail->drain), 0);
      } else if (warp == 2) {
        // ---------------- query rows, 128-byte swizzled like a TMA box, into the buffers as they become
        // free.  A lane finds one row of 32, a step copies 32 / U rows of U 16-byte units.
        QueryBuffers qb;
        for (int i = 0; __all_sync(0xffffffffu, unit_ready(i)); ++i) {
            const SpanUnit q = tail->units[i % SP_RING];
            const int nr = tail->nr[i % SP_RING];
            __syncwarp();
            if (q.unit < 0) break;
            if (lane == 0) unit_done(i);
            const int buf = qb.first(nr), end = qb.last(nr);
            bool ok = true;
#pragma unroll 1
            for (int x = buf; x <= end && ok; ++x)
                if (qb.uses[x] > 0) ok = warp_wait(bar(tail->qfree[x]), (uint32_t)(qb.uses[x] - 1) & 1u, abort_flag, status);
            if (!ok) break;
            constexpr int U = HD / 8, PER = 32 / U;
            const int u = lane & (U - 1), c = u >> 3;
#pragma unroll 1
            for (int r0 = 0; r0 < nr; r0 += 32) {
                int b, head, t;
                where(q, min(r0 + lane, nr - 1), b, head, t);
                const int64_t off = ((int64_t)b * p.T_q + t) * ldq + (int64_t)head * HD;
#pragma unroll 1
                for (int s = 0; s < 32 && r0 + s < nr; s += 8 * PER) {  // eight loads under way
                    uint4 v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int from = (s + e * PER + lane / U) & 31;
                        const int64_t o = __shfl_sync(0xffffffffu, off, from);
                        if (s + e * PER < 32) v[e] = __ldg(reinterpret_cast<const uint4*>(Q + o + u * 8));  // (rows past nr: the last one)
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int r = r0 + s + e * PER + lane / U;
                        if (s + e * PER < 32 && r < nr)
                            st_shared_v4(sQ + (uint32_t)(buf * 64 * 128 + c * C::CHUNK + r * 128) + ((uint32_t)((u & 7) ^ (r & 7)) << 4),
                                         v[e].x, v[e].y, v[e].z, v[e].w);
                    }
                }
            }
            fence_proxy_async_smem();
#pragma unroll 1
            for (int x = buf; x <= end; ++x) mbar_arrive(bar(tail->qfull[x]));
            qb.take(nr);
        }
      } else {
        // ---------------- units: the first is this CTA's, the others come from the counter
        if (blockIdx.x == 0)
            for (int b = lane; b < p.B; b += 32)
                if (lengths[b] < p.T_q || lengths[b] > p.T_max) record_status(status, kStatusBadLength);
        SpanSums sums;
        const SpanPlan plan = span_plan<SP_TK>(p, lengths, (int)gridDim.x, sums);
        if (lane == 0) tail->plan = plan;
        int u = (int)blockIdx.x;
        for (int i = 0;; ++i) {
            SpanUnit x;
            x.unit = -1;
            x.prefix = x.rb = 0;
            if ((unsigned)u < (unsigned)plan.N) x = span_unit<SP_TK>(p, lengths, plan, sums, u);  // (whatever the counter held)
            if (i >= SP_RING && !warp_wait(bar(tail->uempty[i % SP_RING]), (uint32_t)(i / SP_RING - 1) & 1u, abort_flag, status)) break;
            if (lane == 0) {
                tail->units[i % SP_RING] = x;
                tail->nr[i % SP_RING] = min(128, (x.prefix ? p.B * p.rows : p.rows) - x.rb * 128);
                mbar_arrive(bar(tail->ufull[i % SP_RING]));
            }
            if (x.unit < 0) break;
            int next = 0;
            if (lane == 0) next = atomicAdd(status + 3, 1);
            u = (int)gridDim.x + __shfl_sync(0xffffffffu, next, 0);
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
        // ---------------- softmax of stream t
        const int t = (warp - 4) >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t s_col = trow + 128u * t, o_col = trow + C::O_COL + HD * t;
        int j = 0;  // tiles before this unit
        bool ok = true;
        for (int iu = 0; ok; ++iu) {
            if (!__all_sync(0xffffffffu, unit_ready(iu))) break;
            const SpanUnit q = tail->units[iu % SP_RING];
            const int nr = tail->nr[iu % SP_RING], nt = q.i1 - q.i0;
            __syncwarp();
            if (q.unit < 0) break;
            if (lane == 0) unit_done(iu);
            const bool active = quarter * 32 < nr, real = r < nr;
            int rb_, head, tok;
            where(q, real ? r : 0, rb_, head, tok);
            const int pos = q.v.L - p.T_q + tok;
            float m = -INFINITY, l = 0.f;
            for (int k = (j ^ t) & 1; k < nt; k += 2) {
                if (!__all_sync(0xffffffffu, lean_wait(bar(tail->sfull[t]), (uint32_t)((j + k) >> 1) & 1u, abort_flag, status))) {
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
                    if (!__all_sync(0xffffffffu, lean_wait(bar(tail->vfull[st]), (uint32_t)((j + k) / S) & 1u, abort_flag, status))) {
                        ok = false;
                        break;
                    }
                    const int rows = (n + SP_BOX - 1) / SP_BOX * SP_BOX - n;
#pragma unroll 1
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
                    // any reference m gives the same O / l as long as P stays finite: keep it until a row's
                    // sum passes 2^64 (or is not finite: m = -inf), then take the tile's maximum and redo
                    uint32_t pk[64];
                    float alpha = 1.f, rowsum;
                    bool renew = k < 2;
                    for (;;) {
                        float x[128];
                        load_scores(s_col, x);
                        if (scores != nullptr && real && !q.prefix) {
                            // (keys past the end are masked and lie in the row's padding)
                            float4* out = reinterpret_cast<float4*>(
                                scores + (((int64_t)q.b * p.h_kv + q.g) * p.rows + q.rb * 128 + r) * score_ld(p) + key0);
#pragma unroll
                            for (int c = 0; c < SP_TK; c += 4)
                                if (c < n) out[c / 4] = make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]);
                        }
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
            // ---------------- the unit's end
            // each stream's warps join half of the columns
            {
                // (the sums of the unit before have been read)
                if (iu > 0 && !__all_sync(0xffffffffu, lean_wait(bar(tail->ofree), (uint32_t)(iu - 1) & 1u, abort_flag, status))) {
                    ok = false;
                    break;
                }
                tail->ml[t][r] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(tail->mlfull));
                if (!__all_sync(0xffffffffu, lean_wait(bar(tail->odone), (uint32_t)iu & 1u, abort_flag, status) &&
                                                 lean_wait(bar(tail->mlfull), (uint32_t)iu & 1u, abort_flag, status))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (active) {
                    // in the order of the unit's tiles, the first of which went to stream j & 1: which one that
                    // is depends on what this CTA took before, and must not show in the sums
                    const int s0 = j & 1;
                    const float2 ml0 = tail->ml[s0][r], ml1 = tail->ml[s0 ^ 1][r];
                    const float M = fmaxf(ml0.x, ml1.x);
                    const uint32_t o0 = trow + C::O_COL + HD * s0, o1 = trow + C::O_COL + HD * (s0 ^ 1);
                    const float w0 = ml0.x == -INFINITY ? 0.f : ex2_approx(ml0.x - M);
                    const float w1 = ml1.x == -INFINITY ? 0.f : ex2_approx(ml1.x - M);
                    const float sum = w0 * ml0.y + w1 * ml1.y;
                    const bool direct = p.T_p == 0 && q.whole();
                    const int64_t row = rec.row(p, q.unit, tail->plan.np) + r;
                    if (t == 0 && real && (!direct || scores != nullptr)) rec.ml[row] = make_float2(M, sum);
                    const float inv = 1.f / sum;
                    __nv_bfloat16* out = O + ((int64_t)rb_ * p.T_q + tok) * ldo + (int64_t)head * HD;
                    float* part = rec.o + row * HD;
#pragma unroll 1
                    for (int c2 = 0; c2 < HD / 64; ++c2) {
                        const int cc = t * (HD / 64) + c2;
                        float f[32];
                        {
                            uint32_t a[32];
                            tmem_ld32(o0 + cc * 32, a);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) f[e] = w0 * __uint_as_float(a[e]);
                        }
                        if (nt > 1) {
                            uint32_t a[32];
                            tmem_ld32(o1 + cc * 32, a);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) f[e] = fmaf(w1, __uint_as_float(a[e]), f[e]);
                        }
                        if (real && direct) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
                                *reinterpret_cast<uint4*>(out + cc * 32 + e) =
                                    make_uint4(pack_bf16x2(f[e] * inv, f[e + 1] * inv), pack_bf16x2(f[e + 2] * inv, f[e + 3] * inv),
                                               pack_bf16x2(f[e + 4] * inv, f[e + 5] * inv), pack_bf16x2(f[e + 6] * inv, f[e + 7] * inv));
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
        named_barrier_sync(1, SP_THREADS);
        // ---------------- all units are done: join (the softmax warps: they have the registers).  What does
        // not need the records is worked out before the others have arrived.
        constexpr int JOIN = 256, JOIN_WARPS = JOIN / 32, E = HD / 32;  // E columns per lane
        const int jw = warp - 4;
        SpanSums sums;
        const SpanPlan plan = span_plan<SP_TK>(p, lengths, (int)gridDim.x, sums);
        const int heads = p.per * p.h_kv, out_rows = p.B * heads * p.T_q;
        // rows in turn to the CTAs, whose warps share a row's records, where there are few rows; to the
        // warps otherwise
        const bool few = out_rows <= (int)gridDim.x;
        int row = few ? (int)blockIdx.x : (int)blockIdx.x * JOIN_WARPS + jw;
        float* part = reinterpret_cast<float*>(smem_raw);  // [warp][column]
#pragma unroll 1
        for (bool waited = false;; row += few ? (int)gridDim.x : (int)gridDim.x * JOIN_WARPS) {
            __nv_bfloat16* out = nullptr;
            RowRecords src;
            if (row < out_rows) {
                const int bh = p.T_q == 1 ? row : row / p.T_q, t = row - bh * p.T_q, b = bh / heads, head = bh - b * heads;
                int L;
                const int unit0 = span_first_unit<SP_TK>(p, lengths, plan, sums, b, L);
                const SpanView v = span_view<SP_TK>(p, L);
                const int g = head / p.per;
                out = O + ((int64_t)b * p.T_q + t) * ldo + (int64_t)head * HD + lane * E;
                src = row_records<SP_TK>(p, rec, plan, unit0, v.nt, b, g, (head - g * p.per) * p.T_q + t);
                if (v.nt == 0) src.n[0] = src.n[1] = 0;  // invalid length
            }
            if (!waited) {
                waited = true;
                // (the records of all this CTA's warps are behind the block barrier above)
                if (jw == 0 && lane == 0) tail->joined = span_grid_barrier(status, (int)gridDim.x, tail->generation) ? 1 : 0;
                named_barrier_sync(2, JOIN);
                if (!tail->joined) return;
            }
            if (row >= out_rows) break;
            const int n = src.count();
            if (n == 1) continue;  // one unit held the whole group and wrote the row
            float o[E], l = 1.f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = n == 0 ? NAN : 0.f;
            if (n > 0) {
                // one pass, the sums following the running maximum
                float M = -INFINITY;
                l = 0.f;
#pragma unroll 4
                for (int c = few ? jw : 0; c < n; c += few ? JOIN_WARPS : 1) {
                    const int64_t k = src.at(c);
                    const float2 ml = __ldcg(rec.ml + k);
                    float x[E];
                    if constexpr (E == 4) {
                        const float4 y = __ldcg(reinterpret_cast<const float4*>(rec.o + k * HD) + lane);
                        x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
                    } else {
                        const float2 y = __ldcg(reinterpret_cast<const float2*>(rec.o + k * HD) + lane);
                        x[0] = y.x; x[1] = y.y;
                    }
                    const float m = fmaxf(M, ml.x);
                    const float f = M == -INFINITY ? 0.f : ex2_approx(M - m), w = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m);
                    l = fmaf(w, ml.y, l * f);
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] = fmaf(w, x[e], o[e] * f);
                    M = m;
                }
                if (few) {
                    float* mine = part + jw * (HD + 4);
#pragma unroll
                    for (int e = 0; e < E; ++e) mine[lane * E + e] = o[e];
                    if (lane == 0) mine[HD] = l, mine[HD + 1] = M;
                    named_barrier_sync(2, JOIN);
                    l = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll
                    for (int w = 0; w < JOIN_WARPS; ++w) M = fmaxf(M, part[w * (HD + 4) + HD + 1]);
#pragma unroll
                    for (int w = 0; w < JOIN_WARPS; ++w) {
                        const float* his = part + w * (HD + 4);
                        const float f = his[HD + 1] == -INFINITY ? 0.f : ex2_approx(his[HD + 1] - M);
                        l = fmaf(f, his[HD], l);
#pragma unroll
                        for (int e = 0; e < E; ++e) o[e] = fmaf(f, his[lane * E + e], o[e]);
                    }
                    named_barrier_sync(2, JOIN);
                }
            }
            if (!few || jw == 0) {
                const float inv = 1.f / l;
#pragma unroll
                for (int e = 0; e < E; e += 2)
                    *reinterpret_cast<uint32_t*>(out + e) = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
            }
        }
        if (weights != nullptr) {
            // a token's weight is the sum over the query rows of 2^(c s - M) / l, in row order.  A warp takes 512
            // tokens of one (batch, K/V head) at a time, from the last CTA on (the first have rows to join).
            constexpr int PER = 16, KEYS = 32 * PER;
            const int chunks = (p.T_max + KEYS - 1) / KEYS;
            const int64_t tasks = (int64_t)p.B * p.h_kv * chunks;
            const int64_t ld = score_ld(p);
            for (int64_t task = (int64_t)jw * gridDim.x + (gridDim.x - 1 - blockIdx.x); task < tasks; task += (int64_t)gridDim.x * JOIN_WARPS) {
                const int bg = (int)(task / chunks), k0 = (int)(task - (int64_t)bg * chunks) * KEYS;
                const int b = bg / p.h_kv, g = bg - b * p.h_kv;
                int L;
                const int unit0 = span_first_unit<SP_TK>(p, lengths, plan, sums, b, L);
                const SpanView v = span_view<SP_TK>(p, L);
                if (v.nt == 0 || k0 >= v.L) continue;
                // this lane's keys; those past the length read the last one's scores and are dropped
                int key[PER];
#pragma unroll
                for (int u = 0; u < PER; ++u) key[u] = min(k0 + lane + 32 * u, v.L - 1);
                float w[PER] = {};
                for (int r0 = 0; r0 < p.rows; r0 += 32) {
                    const int nr = min(32, p.rows - r0);
                    // the sums of row r0 + (lane mod span), its records shared by 32 / span lanes
                    const int span = nr == 1 ? 1 : 1 << (32 - __clz(nr - 1));
                    const RowRecords x = row_records<SP_TK>(p, rec, plan, unit0, v.nt, b, g, r0 + min(lane & (span - 1), nr - 1));
                    float M = -INFINITY, l = 0.f;
                    auto add = [&](float m2, float l2) {
                        const float m = fmaxf(M, m2);
                        const float f = M == -INFINITY ? 0.f : ex2_approx(M - m), f2 = m2 == -INFINITY ? 0.f : ex2_approx(m2 - m);
                        l = fmaf(f2, l2, l * f);
                        M = m;
                    };
#pragma unroll 8
                    for (int c = lane / span; c < x.count(); c += 32 / span) {
                        const float2 ml = __ldcg(rec.ml + x.at(c));
                        add(ml.x, ml.y);
                    }
                    for (int o = span; o < 32; o <<= 1) {
                        const float m2 = __shfl_xor_sync(0xffffffffu, M, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
                        add(m2, l2);
                    }
                    const float il = 1.f / l;
                    const float* s = scores + ((int64_t)bg * p.rows + r0) * ld;
#pragma unroll 1
                    for (int r = 0; r < nr; r += 2, s += 2 * ld) {
                        float sv[2][PER];
#pragma unroll
                        for (int u = 0; u < PER; ++u) sv[0][u] = __ldcg(s + key[u]);
                        const bool two = r + 1 < nr;
#pragma unroll
                        for (int u = 0; u < PER; ++u) sv[1][u] = two ? __ldcg(s + ld + key[u]) : -INFINITY;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float m = __shfl_sync(0xffffffffu, M, min(r + i, nr - 1)), f = __shfl_sync(0xffffffffu, il, min(r + i, nr - 1));
#pragma unroll
                            for (int u = 0; u < PER; ++u) w[u] = fmaf(ex2_approx(fmaf(sv[i][u], scale_log2, -m)), f, w[u]);
                        }
                    }
                }
                float* to = weights + (int64_t)bg * p.T_max + k0 + lane;
                float old[PER];
                // the new tokens' entries start here, the others grow
#pragma unroll
                for (int u = 0; u < PER; ++u) old[u] = k0 + lane + 32 * u < v.L - p.T_q ? to[32 * u] : 0.f;
#pragma unroll
                for (int u = 0; u < PER; ++u)
                    if (k0 + lane + 32 * u < v.L) to[32 * u] = old[u] + w[u];
            }
        }
    }
}

template <int HD>
cudaError_t launch(const SpanShape& p, const SpanRecords& rec, const void* Q, int64_t ldq, const void* K, int64_t ldk,
                   const void* V, int64_t ldv, const void* Kp, int64_t ldkp, const void* Vp, int64_t ldvp, void* O,
                   int64_t ldo, const int32_t* lengths, float* scores, float* weights, int ctas, int* status,
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
    cfg.gridDim = dim3((unsigned)ctas);
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
                             float* weights, int ctas, int* status, cudaStream_t stream) {
    if (d == 64)
        return launch<64>(p, rec, Q, ldq, K, ldk, V, ldv, Kp, ldkp, Vp, ldvp, O, ldo, lengths, scores,
                          weights, ctas, status, stream);
    if (d == 128)
        return launch<128>(p, rec, Q, ldq, K, ldk, V, ldv, Kp, ldkp, Vp, ldvp, O, ldo, lengths, scores,
                           weights, ctas, status, stream);
    return cudaErrorInvalidValue;
}

}  // namespace mha
