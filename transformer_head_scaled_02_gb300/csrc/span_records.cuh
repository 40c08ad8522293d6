// span_records.cuh -- where the units of span.cuh leave their partial results, and how a row's are found.
#pragma once

#include <math.h>
#include <stddef.h>

#include "span.cuh"

namespace mha {

// Records of the units: per query row (m, l) -- the base-2 reference maximum and the sum of 2^(s - m) -- and
// the dv weighted values.  Prefix and cache units have their own row counts, so the two sets lie one after
// the other.
struct SpanRecords {
    float2* ml;
    float* o;
    int64_t base_c;  // first record row of the cache units
    int dv;

    // Record row of a unit's first query row; np: units of the prefix.
    __host__ __device__ int64_t row(const SpanShape& p, int unit, int np) const {
        return unit < np ? (int64_t)unit * p.rps_p() : base_c + (int64_t)(unit - np) * p.rps_c();
    }
};

// Row stride of the scores: 16-byte rows.
__host__ __device__ inline int64_t score_ld(const SpanShape& p) { return ((int64_t)p.T_max + 3) & ~(int64_t)3; }

struct SpanLayout {
    size_t ml_off, o_off, s_off, total;  // bytes from the workspace area's start
    int64_t base_c;
};

template <int TILE>
inline SpanLayout span_layout(const SpanShape& p, int dv, bool scores) {
    SpanLayout w;
    int64_t units_p, units_c;
    span_most_units<TILE>(p, units_p, units_c);
    w.base_c = p.T_p > 0 ? units_p * p.rps_p() : 0;
    const size_t rec = (size_t)(w.base_c + units_c * p.rps_c());
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    w.ml_off = 0;
    w.o_off = up(rec * sizeof(float2));
    w.s_off = w.o_off + up(rec * (size_t)dv * sizeof(float));
    w.total = w.s_off + (scores ? up((size_t)p.B * p.h_kv * p.rows * (size_t)score_ld(p) * sizeof(float)) : 0);
    return w;
}

// The records of query row rr of (batch b, K/V head g): record c of its n[0] own ones is at first[0] +
// c * step[0]; the prefix's n[1] likewise.  Everything is read from L2: the records were written by other
// SMs, possibly in the same kernel.
struct RowRecords {
    int64_t first[2], step[2];
    int n[2];

    __device__ int count() const { return n[0] + n[1]; }
    __device__ int64_t at(int c) const { return c < n[0] ? first[0] + c * step[0] : first[1] + (c - n[0]) * step[1]; }
};

// unit0: first unit of batch b; nt: its tiles (a valid length).
template <int TILE>
__device__ __forceinline__ RowRecords row_records(const SpanShape& p, const SpanRecords& rec, const SpanPlan& q, int unit0, int nt,
                                                  int b, int g, int rr) {
    RowRecords x;
    const int rb = p.nrb == 1 ? 0 : rr / p.bm_c;
    x.n[0] = (nt + q.U - 1) / q.U;
    x.first[0] = rec.row(p, unit0 + g * p.nrb + rb, q.np) + (rr - rb * p.bm_c);
    x.step[0] = (int64_t)p.lanes_c() * p.rps_c();
    x.n[1] = 0;
    x.first[1] = x.step[1] = 0;
    if (p.T_p > 0) {
        const int rp = b * p.rows + rr, rbp = rp / p.bm_p;
        x.n[1] = q.np / p.lanes_p();
        x.first[1] = rec.row(p, g * p.nrbp + rbp, q.np) + (rp - rbp * p.bm_p);
        x.step[1] = (int64_t)p.lanes_p() * p.rps_p();
    }
    return x;
}

// M and l of a row over all its records (warp-collective, a lane per record).
__device__ __forceinline__ float2 row_sum(const SpanRecords& rec, const RowRecords& x) {
    const int lane = (int)threadIdx.x & 31;
    float M = -INFINITY, l = 0.f;
    for (int c = lane; c < x.count(); c += 32) {
        const float2 ml = __ldcg(rec.ml + x.at(c));
        if (ml.x == -INFINITY) continue;  // a unit without a visible key
        const float m = fmaxf(M, ml.x);
        l = l * exp2f(M - m) + ml.y * exp2f(ml.x - m);
        M = m;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float Mo = __shfl_xor_sync(0xffffffffu, M, o), lo = __shfl_xor_sync(0xffffffffu, l, o);
        const float m = fmaxf(M, Mo);
        if (m != -INFINITY) l = l * exp2f(M - m) + lo * exp2f(Mo - m);
        M = m;
    }
    return make_float2(M, l);
}

}  // namespace mha
