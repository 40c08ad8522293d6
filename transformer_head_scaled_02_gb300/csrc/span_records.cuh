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

    // Record row of the first query row of a piece: lane block `block` (see SpanPiece), a gang's member.
    __host__ __device__ int64_t row(const SpanShape& p, bool prefix, int block, int gang, int member) const {
        const int64_t slot = (int64_t)(gang + block - (prefix ? 0 : p.blocks_p())) * p.gang + member;
        return prefix ? slot * rps_p : base_c + slot * rps_c;
    }
};

// Row stride of the scores: 16-byte rows.
__host__ __device__ inline int64_t score_ld(const SpanShape& p) { return ((int64_t)p.T_max + 3) & ~(int64_t)3; }

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
    w.total = w.s_off + (scores ? up((size_t)p.B * p.h_kv * p.rows * (size_t)score_ld(p) * sizeof(float)) : 0);
    return w;
}

}  // namespace mha
