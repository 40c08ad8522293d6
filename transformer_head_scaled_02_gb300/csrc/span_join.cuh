// span_join.cuh -- finding the records of a query row, for the code that joins the pieces of span.cuh.
// Everything is read from L2: the records were written by other SMs, possibly in the same kernel.
#pragma once

#include <math.h>

#include "span_records.cuh"

namespace mha {

// The record rows of query row r of a lane's group: the pieces of gangs c0 .. c1, one slot row apart.
struct RowRecords {
    int64_t first, step;
    int n;
};

// lane: (K/V head, row block) of the prefix or of a batch whose lane blocks start at place `off` and index
// `block0`; nt tiles a group.
__device__ __forceinline__ RowRecords row_records(const SpanShape& p, const SpanRecords& rec, bool prefix, int lane,
                                                  int off, int block0, int nt, int N, int gangs, int r) {
    const int bl = lane / p.gang, member = lane - bl * p.gang;
    const int t0 = off + bl * (nt + kSpanPieceCost);
    int c0, c1;
    span_gangs(N, gangs, t0, t0 + nt, c0, c1);
    RowRecords x;
    x.first = rec.row(p, prefix, block0 + bl, c0, member) + r;
    x.step = (int64_t)p.gang * (prefix ? rec.rps_p : rec.rps_c);
    x.n = c1 - c0 + 1;
    return x;
}

// The number of places N and the first one of batch b's lane blocks (b has a valid length).
template <int TILE>
__device__ __forceinline__ void first_tile(const SpanShape& p, const int32_t* lengths, int b, int& N, int& off) {
    const int lane = (int)threadIdx.x & 31;
    const int npt = span_prefix_places<TILE>(p);
    int below = 0, all = 0;
    for (int i = lane; i < p.B; i += 32) {
        const int n = span_view<TILE>(p, __ldcg(lengths + i)).places() * p.blocks_c();
        all += n;
        if (i < b) below += n;
    }
    N = npt + __reduce_add_sync(0xffffffffu, all);
    off = npt + __reduce_add_sync(0xffffffffu, below);
}

// M and l of a row over all its records (warp-collective, a lane per record).
__device__ __forceinline__ float2 row_sum(const SpanRecords& rec, const RowRecords (&src)[2]) {
    const int lane = (int)threadIdx.x & 31;
    float M = -INFINITY;
#pragma unroll
    for (int s = 0; s < 2; ++s)
        for (int c = lane; c < src[s].n; c += 32) M = fmaxf(M, __ldcg(rec.ml + src[s].first + c * src[s].step).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float l = 0.f;
#pragma unroll
    for (int s = 0; s < 2; ++s)
        for (int c = lane; c < src[s].n; c += 32) {
            const float2 ml = __ldcg(rec.ml + src[s].first + c * src[s].step);
            if (ml.x != -INFINITY) l = fmaf(exp2f(ml.x - M), ml.y, l);  // else a piece without a visible key
        }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    return make_float2(M, l);
}

// The records of query row rr of (batch b, K/V head g): its own cache's, and the prefix's.  v: the batch's
// view, with a valid length; N, off: from first_tile.
template <int TILE>
__device__ __forceinline__ void row_sources(const SpanShape& p, const SpanRecords& rec, int bm, int gangs, const SpanView& v,
                                            int b, int g, int rr, int N, int off, RowRecords (&src)[2]) {
    src[0] = row_records(p, rec, false, g * p.nrb + rr / bm, off, p.blocks_p() + b * p.blocks_c(), v.nt, N, gangs, rr % bm);
    src[1].n = 0;
    if (p.T_p > 0) {
        const int rp = b * p.rows + rr;
        src[1] = row_records(p, rec, true, g * p.nrbp + rp / bm, 0, 0, span_prefix_tiles<TILE>(p), N, gangs, rp % bm);
    }
}

}  // namespace mha
