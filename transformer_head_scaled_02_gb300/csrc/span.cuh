// span.cuh -- how the cache operators (windowed, shared-prefix and weight-accumulating decode steps) cut
// their work, shared by the kernels that compute the units and those that join them.
//
// The query rows that share cached keys form groups: one per (batch, lane) over the batch's own cache,
// and, with a shared prefix, one per lane over the prefix, whose rows are those of the whole batch; a lane is
// a (K/V head, block of query rows).  A group's visible keys are at most two ranges, the sinks
// [0, s) and the window [lo, L), each cut into tiles.  A unit is U consecutive tiles of one group (Up of a
// prefix group): the CTAs take units one after another, so ragged lengths, group counts that do not
// divide the SMs and SMs that are slower than others leave none idle (an even cut made beforehand left the
// first CTA idle for a fifth of a step).  Units are numbered prefix first, then by batch, chunk and lane,
// lanes fastest: a cached token's rows of all heads lie side by side, and units taken at about the same
// time read whole pieces of DRAM pages.  U is chosen so that every CTA gets 6 to 16 units, but no
// unit's record of its rows costs more than a few percent of the unit; Up so that every CTA gets at most about one
// of the prefix.  A unit that holds a whole
// group writes its output itself; the others leave a record per row (maximum, sum, weighted values), and
// the join adds them in order:
//   O = sum_u 2^(m_u - M) o_u / sum_u 2^(m_u - M) l_u,  M = max_u m_u   (scores in base 2).
// Everything follows from the lengths alone, not from which CTA took what.
#pragma once

#include <stdint.h>

namespace mha {

// Largest grid of the unit kernels (bounds the records; the host knows no SM count when it computes
// workspace sizes), and most units per CTA to aim for.
constexpr int kSpanMaxCtas = 320;
constexpr int kSpanUnits = 16;

struct SpanShape {
    int B, h_kv;
    int per;     // query heads per K/V head
    int T_q, T_max;
    int rows;    // per * T_q: query rows of one (batch, K/V head)
    int nrb;     // row blocks of such a group
    int T_p;     // shared prefix tokens (0: none)
    int nrbp;    // row blocks of the B * rows rows over the prefix
    int bm_c, bm_p;  // rows of a row block of a cache and of the prefix
    int aim;     // units per CTA to aim for, at most kSpanUnits; 0: by the number of tiles
    int step;    // tiles that a CTA of the caches' kernel works on at a time: larger units are multiples of it
    int window;  // <= T_max; T_max: no window
    int sinks;

    __host__ __device__ int lanes_c() const { return h_kv * nrb; }
    __host__ __device__ int lanes_p() const { return h_kv * nrbp; }
    // rows of a record; fewest tiles of a unit whose records stay cheap beside its tiles
    __host__ __device__ int rps_c() const { return rows < bm_c ? rows : bm_c; }
    __host__ __device__ int rps_p() const { return (int64_t)B * rows < bm_p ? B * rows : bm_p; }
    __host__ __device__ int least_c() const { return (rps_c() + 15) / 16; }
    __host__ __device__ int least_p() const { return (rps_p() + 15) / 16; }
};

// The visible keys of a batch with L cached tokens: [0, s_keys) and [lo, L); nst sink tiles, nt tiles in all
// (0 for an invalid length).
struct SpanView {
    int L, s_keys, lo, nst, nt;
};

template <int TILE>
__host__ __device__ inline SpanView span_view(const SpanShape& p, int L) {
    SpanView v;
    v.L = L;
    v.s_keys = 0;
    v.nst = 0;
    v.nt = 0;
    v.lo = 0;
    if (L < p.T_q || L > p.T_max) return v;
    const int lo = L - p.T_q - p.window + 1;  // first key in the window of new token 0
    if (lo > p.sinks) {
        v.s_keys = p.sinks;
        v.lo = lo;
    }  // else the two ranges meet: one range from 0
    v.nst = (v.s_keys + TILE - 1) / TILE;
    v.nt = v.nst + (L - v.lo + TILE - 1) / TILE;
    return v;
}

// Keys [key0, key0 + n) of tile i of a view.
template <int TILE>
__device__ __forceinline__ void span_tile(const SpanView& v, int i, int& key0, int& n) {
    const bool sink = i < v.nst;
    key0 = sink ? i * TILE : v.lo + (i - v.nst) * TILE;
    const int end = sink ? v.s_keys : v.L;
    n = end - key0 < TILE ? end - key0 : TILE;
}

// Does the new token at cache position pos see the key?
__device__ __forceinline__ bool span_visible(const SpanShape& p, int pos, int key) {
    return key <= pos && (pos - key < p.window || key < p.sinks);
}

template <int TILE>
__host__ __device__ inline int span_prefix_tiles(const SpanShape& p) {
    return (p.T_p + TILE - 1) / TILE;
}

// Most tiles of all groups together (the host checks that they fit 32 bits and launches no more CTAs).
template <int TILE>
inline int64_t span_most_tiles(const SpanShape& p) {
    const int64_t all = ((int64_t)p.T_max + TILE - 1) / TILE;
    const int64_t win = ((int64_t)p.sinks + TILE - 1) / TILE + ((int64_t)p.window + p.T_q - 1 + TILE - 1) / TILE;
    return (int64_t)span_prefix_tiles<TILE>(p) * p.lanes_p() + (int64_t)p.B * p.lanes_c() * (all < win ? all : win);
}

// Most records (units) of the prefix and of the caches, for any lengths and any grid up to kSpanMaxCtas:
// U tiles a unit, U at least total / (kSpanUnits * CTAs), leave at most that many units and a rest per group.
template <int TILE>
inline void span_most_units(const SpanShape& p, int64_t& units_p, int64_t& units_c) {
    const int64_t cap = (int64_t)kSpanUnits * kSpanMaxCtas;
    const int64_t np = span_prefix_tiles<TILE>(p), nt = ((int64_t)p.T_max + TILE - 1) / TILE + 1;
    const int64_t lp = p.lanes_p(), lc = (int64_t)p.B * p.lanes_c();
    const int64_t ap = (np + p.least_p() - 1) / p.least_p() * lp, ac = (nt + p.least_c() - 1) / p.least_c() * lc;
    units_p = ap < cap + lp ? ap : cap + lp;
    units_c = ac < cap + lc ? ac : cap + lc;
}

// The cut, from the lengths; and one lane's part of its prefix sums over the batches.
struct SpanPlan {
    int U, Up;   // tiles of a unit
    int np;      // units of the prefix
    int N;       // units in all
};

struct SpanSums {
    int i0, i1;       // this lane's batches
    int L0;           // length of batch i0: up to 32 batches, lengths are read once
    int before, sum;  // first unit of batch i0, units of the lane's batches
    __device__ __forceinline__ int length(const int32_t* lengths, int i) const { return i == i0 ? L0 : __ldcg(lengths + i); }
};

template <int TILE>
__device__ __forceinline__ int span_units(const SpanShape& p, const SpanPlan& q, int L) {
    return (span_view<TILE>(p, L).nt + q.U - 1) / q.U * p.lanes_c();
}

// All lanes of a warp call it; ctas: the grid of the unit kernel.
template <int TILE>
__device__ inline SpanPlan span_plan(const SpanShape& p, const int32_t* lengths, int ctas, SpanSums& s) {
    const int lane = (int)threadIdx.x & 31;
    const int run = (p.B + 31) / 32;
    s.i0 = min(p.B, lane * run);
    s.i1 = min(p.B, s.i0 + run);
    s.L0 = s.i0 < s.i1 ? __ldcg(lengths + s.i0) : 0;
    int tiles = 0;
#pragma unroll 1
    for (int i = s.i0; i < s.i1; ++i) tiles += span_view<TILE>(p, s.length(lengths, i)).nt;
    const int np = span_prefix_tiles<TILE>(p);
    const unsigned total = __reduce_add_sync(0xffffffffu, (unsigned)tiles) * (unsigned)p.lanes_c() + (unsigned)(np * p.lanes_p());
    // With many tiles short units at the end even out the CTAs; with few, a unit's own cost counts.  Units per
    // CTA 6 | 10 | 14 | 20, us: 20 tiles a CTA 39 | 43 | 43 | 60, 40 tiles 72 | 73 | 76 | 81, 160 tiles 238 | 233 |
    // 232 | 232.
    const unsigned aim = p.aim > 0 ? (unsigned)p.aim : min((unsigned)kSpanUnits, max(6u, total / (6u * (unsigned)ctas)));
    const unsigned target = aim * (unsigned)ctas;
    SpanPlan q;
    q.U = max(p.least_c(), (int)((total + target - 1) / target));
    q.U = max(q.U, 1);
    if (q.U > p.step / 2) q.U = (q.U + p.step - 1) / p.step * p.step;
    q.Up = max(max(q.U, p.least_p()), (np * p.lanes_p() + ctas - 1) / ctas);
    q.np = p.T_p > 0 ? (np + q.Up - 1) / q.Up * p.lanes_p() : 0;
    s.sum = 0;
#pragma unroll 1
    for (int i = s.i0; i < s.i1; ++i) s.sum += span_units<TILE>(p, q, s.length(lengths, i));
    int inc = s.sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    s.before = q.np + inc - s.sum;
    q.N = q.np + __shfl_sync(0xffffffffu, inc, 31);
    return q;
}

// First unit and length of batch b (all lanes of a warp; b the same in all).
template <int TILE>
__device__ __forceinline__ int span_first_unit(const SpanShape& p, const int32_t* lengths, const SpanPlan& q, const SpanSums& s,
                                               int b, int& L) {
    int at = 0, len = 0;
    const bool mine = s.i0 <= b && b < s.i1;
    if (mine) {
        at = s.before;
#pragma unroll 1
        for (int i = s.i0; i < b; ++i) at += span_units<TILE>(p, q, s.length(lengths, i));
        len = s.length(lengths, b);
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
    L = __shfl_sync(0xffffffffu, len, src);
    return __shfl_sync(0xffffffffu, at, src);
}

struct SpanUnit {
    int unit;        // -1: no more
    int prefix;
    int b, g, rb;
    int i0, i1;      // tiles [i0, i1) of the group
    SpanView v;      // the batch's view (prefix: L = T_p, one range)
    __device__ bool whole() const { return i0 == 0 && i1 == v.nt; }
};

// Unit u < N (all lanes of a warp; every lane gets it).
template <int TILE>
__device__ inline SpanUnit span_unit(const SpanShape& p, const int32_t* lengths, const SpanPlan& q, const SpanSums& s, int u) {
    SpanUnit x;
    x.unit = u;
    int k, lane_i, U, nrb;
    if (u < q.np) {
        x.prefix = 1;
        x.b = 0;
        x.v.L = p.T_p;
        x.v.s_keys = x.v.lo = x.v.nst = 0;
        x.v.nt = span_prefix_tiles<TILE>(p);
        k = u / p.lanes_p();
        lane_i = u - k * p.lanes_p();
        U = q.Up;
        nrb = p.nrbp;
    } else {
        x.prefix = 0;
        int b = 0, at = 0, len = 0;
        const bool mine = s.before <= u && u < s.before + s.sum;
        if (mine) {
            at = s.before;
#pragma unroll 1
            for (b = s.i0;; ++b) {
                len = s.length(lengths, b);
                const int n = span_units<TILE>(p, q, len);
                if (u < at + n) break;
                at += n;
            }
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
        x.b = __shfl_sync(0xffffffffu, b, src);
        at = __shfl_sync(0xffffffffu, at, src);
        x.v = span_view<TILE>(p, __shfl_sync(0xffffffffu, len, src));
        k = (u - at) / p.lanes_c();
        lane_i = u - at - k * p.lanes_c();
        U = q.U;
        nrb = p.nrb;
    }
    x.g = lane_i / nrb;
    x.rb = lane_i - x.g * nrb;
    x.i0 = k * U;
    x.i1 = min(x.v.nt, x.i0 + U);
    return x;
}

}  // namespace mha
