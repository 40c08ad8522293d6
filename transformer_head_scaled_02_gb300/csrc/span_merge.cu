// span_merge.cu -- joins the units of the fp32 cache steps (span_simt.cu): the output rows of groups of
// several units (or of a prefix and a cache), and the attention weights per cached token.
#include <math.h>

#include "internal.h"
#include "ptx.cuh"
#include "span_records.cuh"

namespace mha {
namespace {

constexpr int SM_THREADS = 128;
constexpr int SM_WARPS = SM_THREADS / 32;
constexpr int SM_TILE = 64;    // keys per tile of the pieces
constexpr int SM_KEYS = 1024;  // cached tokens per block of the weight sums

// Blocks [0, B * heads * T_q): one output row each; a warp adds every SM_WARPS-th record, a lane every
// 32nd column, and the warps' sums meet in shared memory.  The blocks after them (WEIGHTS): SM_KEYS cached
// tokens of one (batch, K/V head) each; with M and l of every query row known, a token's weight is the
// sum over the rows of 2^(s - M) / l, added in row order.  The new tokens' entries start here (they have
// no earlier weight), those past the length stay as they are.  Latency is what counts: the rows of a
// decode step are few, so everything that does not need the records is done before the wait for them.
template <bool WEIGHTS>
__global__ void __launch_bounds__(SM_THREADS)
    span_merge_kernel(const SpanShape p, const SpanRecords rec, int ctas, float* __restrict__ O, int64_t ldo,
                      const int32_t* __restrict__ lengths, const float* __restrict__ scores,
                      float* __restrict__ weights) {
    // The unit kernel lets this one start once its own wait for earlier work is over, so the lengths can
    // be read at once (from L2: nothing older may be served); the records it is still writing cannot.
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int heads = p.per * p.h_kv, out_rows = p.B * heads * p.T_q;
    SpanSums sums;
    const SpanPlan plan = span_plan<SM_TILE>(p, lengths, ctas, sums);
    if (!WEIGHTS || (int)blockIdx.x < out_rows) {
        const int row = (int)blockIdx.x;  // (b * heads + head) * T_q + t
        const int t = row % p.T_q, bh = row / p.T_q, b = bh / heads, head = bh - b * heads;
        float* out = O + ((int64_t)b * p.T_q + t) * ldo + (int64_t)head * rec.dv;
        const int g = head / p.per, rr = (head - g * p.per) * p.T_q + t;
        int L;
        const int unit0 = span_first_unit<SM_TILE>(p, lengths, plan, sums, b, L);
        const SpanView v = span_view<SM_TILE>(p, L);
        const RowRecords src = row_records<SM_TILE>(p, rec, plan, unit0, v.nt, b, g, rr);
        grid_dependency_wait();
        grid_launch_dependents();
        if (v.nt == 0) {  // invalid length
            for (int e = tid; e < rec.dv; e += SM_THREADS) out[e] = NAN;
            return;
        }
        if (src.count() == 1) return;  // one unit held the whole group and wrote the row
        __shared__ float part[SM_WARPS][256];
        const float2 ml = row_sum(rec, src);
        float o[8] = {};  // d_v <= 256
        for (int c = warp; c < src.count(); c += SM_WARPS) {
            const int64_t k = src.at(c);
            const float m = rec.ml[k].x;
            const float w = m == -INFINITY ? 0.f : exp2f(m - ml.x);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (lane + 32 * u < rec.dv) o[u] = fmaf(w, rec.o[k * rec.dv + lane + 32 * u], o[u]);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (lane + 32 * u < rec.dv) part[warp][lane + 32 * u] = o[u];
        __syncthreads();
        for (int e = tid; e < rec.dv; e += SM_THREADS) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < SM_WARPS; ++w) sum += part[w][e];
            out[e] = sum / ml.y;
        }
        return;
    }
    if constexpr (WEIGHTS) {
        __shared__ float2 row_ml[SM_THREADS];  // (M, 1 / l)
        const int chunks = (p.T_max + SM_KEYS - 1) / SM_KEYS;
        const int i = (int)blockIdx.x - out_rows;
        const int bg = i / chunks, k0 = (i - bg * chunks) * SM_KEYS;
        const int b = bg / p.h_kv, g = bg - b * p.h_kv;
        int L;
        const int unit0 = span_first_unit<SM_TILE>(p, lengths, plan, sums, b, L);
        const SpanView v = span_view<SM_TILE>(p, L);
        grid_dependency_wait();
        grid_launch_dependents();
        if (v.nt == 0 || k0 >= v.L) return;
        float w[SM_KEYS / SM_THREADS] = {};
        for (int r0 = 0; r0 < p.rows; r0 += SM_THREADS) {
            const int nr = min(SM_THREADS, p.rows - r0);
            __syncthreads();
            for (int r = warp; r < nr; r += SM_WARPS) {
                const int rr = r0 + r;
                const float2 ml = row_sum(rec, row_records<SM_TILE>(p, rec, plan, unit0, v.nt, b, g, rr));
                if (lane == 0) row_ml[r] = make_float2(ml.x, 1.f / ml.y);
            }
            __syncthreads();
            const float* s = scores + ((int64_t)bg * p.rows + r0) * score_ld(p) + k0;
#pragma unroll 2
            for (int r = 0; r < nr; ++r) {
                const float2 ml = row_ml[r];
#pragma unroll
                for (int u = 0; u < SM_KEYS / SM_THREADS; ++u) {
                    const int j = tid + u * SM_THREADS;
                    if (k0 + j < v.L) w[u] = fmaf(exp2f(s[(int64_t)r * score_ld(p) + j] - ml.x), ml.y, w[u]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < SM_KEYS / SM_THREADS; ++u) {
            const int j = k0 + tid + u * SM_THREADS;
            if (j >= v.L) continue;
            float* out = weights + (int64_t)bg * p.T_max + j;
            *out = j < v.L - p.T_q ? *out + w[u] : w[u];
        }
    }
}

}  // namespace

int64_t span_merge_blocks(const SpanShape& p, bool weights) {
    const int64_t out_rows = (int64_t)p.B * p.per * p.h_kv * p.T_q;
    return out_rows + (weights ? (int64_t)p.B * p.h_kv * ((p.T_max + SM_KEYS - 1) / SM_KEYS) : 0);
}

cudaError_t launch_span_merge(const SpanShape& p, const SpanRecords& rec, int ctas, float* O, int64_t ldo,
                              const int32_t* lengths, const float* scores, float* weights, cudaStream_t stream) {
    const int64_t blocks = span_merge_blocks(p, weights != nullptr);  // (the caller has checked that they are a grid)
    auto kernel = weights != nullptr ? span_merge_kernel<true> : span_merge_kernel<false>;
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(SM_THREADS), 0, stream, p, rec, ctas, O, ldo, lengths,
                      scores, weights);
}

}  // namespace mha
