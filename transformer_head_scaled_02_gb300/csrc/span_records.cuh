// span_records.cuh -- where the pieces of span.cuh leave their partial results.
#pragma once

#include <stddef.h>

#include "span.cuh"

namespace mha {

// Records of the pieces: per query row of a slot (m, l) -- the base-2 reference maximum and the sum of
// 2^(s - m) -- and the dv weighted values.  Prefix groups (row blocks of the whole batch's rows) and
// cache groups have their own row counts per slot, so the two sets lie one after the other.
struct SpanRecords {
    float2* ml;
    float* o;
    int rps_p, rps_c;  // rows per slot
    int64_t base_c;    // first record row of the cache groups
    int dv;

    __host__ __device__ int64_t row(bool prefix, int64_t groups_p, int64_t group, int cta) const {
        return prefix ? (cta + group) * rps_p : base_c + (cta + group - groups_p) * rps_c;
    }
};

struct SpanLayout {
    size_t ml_off, o_off, s_off, total;  // bytes from the workspace area's start
    int rps_p, rps_c;
    int64_t base_c;
};

// bm: query rows of a row block (shape.nrb and nrbp were computed with it).
inline SpanLayout span_layout(const SpanShape& p, int dv, int bm, bool scores) {
    SpanLayout w;
    const int64_t rows_p = (int64_t)p.B * p.rows;
    w.rps_p = p.T_p > 0 ? (int)(rows_p < bm ? rows_p : bm) : 0;
    w.rps_c = p.rows < bm ? p.rows : bm;
    const int64_t gp = p.T_p > 0 ? (int64_t)p.h_kv * p.nrbp : 0, gc = (int64_t)p.B * p.h_kv * p.nrb;
    w.base_c = p.T_p > 0 ? (kSpanMaxCtas + gp) * w.rps_p : 0;
    const size_t rec = (size_t)(w.base_c + (kSpanMaxCtas + gc) * w.rps_c);
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    w.ml_off = 0;
    w.o_off = up(rec * sizeof(float2));
    w.s_off = w.o_off + up(rec * (size_t)dv * sizeof(float));
    w.total = w.s_off + (scores ? up((size_t)p.B * p.h_kv * p.rows * p.T_max * sizeof(float)) : 0);
    return w;
}

}  // namespace mha
