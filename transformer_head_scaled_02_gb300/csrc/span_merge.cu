// span_merge.cu -- joins the pieces of span.cuh: the output rows of groups that several CTAs (or a
// prefix and a cache) share, and the attention weights per cached token.
#include <math.h>

#include "internal.h"
#include "ptx.cuh"
#include "span_records.cuh"

namespace mha {
namespace {

constexpr int SM_THREADS = 128;
constexpr int SM_KEYS = 512;  // cached tokens per block of the weight sums

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The record rows of query row r of a lane's group: the pieces of gangs c0 .. c1, one slot row apart.
struct RowRecords {
    int64_t first, step;
    int n;
};

// lane: (K/V head, row block) of the prefix or of a batch whose lane blocks start at tile `off` and index
// `block0`; nt tiles a group.
__device__ __forceinline__ RowRecords row_records(const SpanShape& p, const SpanRecords& rec, bool prefix, int lane,
                                                  int off, int block0, int nt, int N, int gangs, int r) {
    const int bl = lane / p.gang, member = lane - bl * p.gang;
    const int t0 = off + bl * nt;
    int c0, c1;
    span_gangs(N, gangs, t0, t0 + nt, c0, c1);
    RowRecords x;
    x.first = rec.row(p, prefix, block0 + bl, c0, member) + r;
    x.step = (int64_t)p.gang * (prefix ? rec.rps_p : rec.rps_c);
    x.n = c1 - c0 + 1;
    return x;
}

// The number of tiles N and the first tile of batch b's lane blocks (b has a valid length).
template <int TILE>
__device__ __forceinline__ void first_tile(const SpanShape& p, const int32_t* lengths, int b, int& N, int& off) {
    const int lane = (int)threadIdx.x & 31;
    const int npt = span_prefix_tiles<TILE>(p) * p.blocks_p();
    int below = 0, all = 0;
    for (int i = lane; i < p.B; i += 32) {
        const int n = span_view<TILE>(p, __ldcg(lengths + i)).nt * p.blocks_c();
        all += n;
        if (i < b) below += n;
    }
    N = npt + __reduce_add_sync(0xffffffffu, all);
    off = npt + __reduce_add_sync(0xffffffffu, below);
}

// Blocks [0, B * heads * T_q): one output row each, thread = output column.  The blocks after them
// (WEIGHTS): SM_KEYS cached tokens of one (batch, K/V head) each; with M and l of every query row
// known, a token's weight is the sum over the rows of 2^(s - M) / l, added in row order.  The new
// tokens' entries start here (they have no earlier weight), those past the length stay as they are.
template <typename T, int TILE, bool WEIGHTS>
__global__ void __launch_bounds__(SM_THREADS)
    span_merge_kernel(const SpanShape p, const SpanRecords rec, int bm, int gangs, T* __restrict__ O, int64_t ldo,
                      const int32_t* __restrict__ lengths, const float* __restrict__ scores,
                      float* __restrict__ weights) {
    // The piece kernel lets this one start once its own wait for earlier work is over, so the lengths can
    // be read at once (from L2: nothing older may be served); the records it is still writing cannot.
    const int tid = (int)threadIdx.x;
    const int heads = p.per * p.h_kv, out_rows = p.B * heads * p.T_q;
        if (!WEIGHTS || (int)blockIdx.x < out_rows) {
        const int row = (int)blockIdx.x;  // (b * heads + head) * T_q + t
        const int t = row % p.T_q, bh = row / p.T_q, b = bh / heads, head = bh - b * heads;
        T* out = O + ((int64_t)b * p.T_q + t) * ldo + (int64_t)head * rec.dv;
        const int g = head / p.per, rr = (head - g * p.per) * p.T_q + t;
        const SpanView v = span_view<TILE>(p, __ldcg(lengths + b));
        if (v.nt == 0) {  // invalid length
            grid_dependency_wait();
            grid_launch_dependents();
            for (int e = tid; e < rec.dv; e += SM_THREADS) out[e] = from_f32<T>(NAN);
            return;
        }
        int N, off;
        first_tile<TILE>(p, lengths, b, N, off);
        const int block0 = p.blocks_p() + b * p.blocks_c();
        RowRecords src[2];
        src[0] = row_records(p, rec, false, g * p.nrb + rr / bm, off, block0, v.nt, N, gangs, rr % bm);
        src[1].n = 0;
        if (p.T_p > 0) {
            const int rp = b * p.rows + rr, np = span_prefix_tiles<TILE>(p);
            src[1] = row_records(p, rec, true, g * p.nrbp + rp / bm, 0, 0, np, N, gangs, rp % bm);
        }
        grid_dependency_wait();
        grid_launch_dependents();
        if (p.T_p == 0 && src[0].n == 1) return;  // one piece held the whole group and wrote the row
        float M = -INFINITY;
        for (int s = 0; s < 2; ++s)
            for (int c = 0; c < src[s].n; ++c) M = fmaxf(M, rec.ml[src[s].first + c * src[s].step].x);
        float l = 0.f, o[2] = {0.f, 0.f};  // d_v <= 256: two columns a thread
        for (int s = 0; s < 2; ++s)
            for (int c = 0; c < src[s].n; ++c) {
                const int64_t k = src[s].first + c * src[s].step;
                const float2 ml = rec.ml[k];
                const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);  // a piece without a visible key
                l = fmaf(w, ml.y, l);
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    if (tid + u * SM_THREADS < rec.dv) o[u] = fmaf(w, rec.o[k * rec.dv + tid + u * SM_THREADS], o[u]);
            }
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (tid + u * SM_THREADS < rec.dv) out[tid + u * SM_THREADS] = from_f32<T>(o[u] / l);
        return;
    }
    if constexpr (WEIGHTS) {
        __shared__ float2 row_ml[SM_THREADS];  // (M, 1 / l)
        const int chunks = (p.T_max + SM_KEYS - 1) / SM_KEYS;
        const int i = (int)blockIdx.x - out_rows;
        const int bg = i / chunks, k0 = (i - bg * chunks) * SM_KEYS;
        const int b = bg / p.h_kv, g = bg - b * p.h_kv;
        const SpanView v = span_view<TILE>(p, __ldcg(lengths + b));
        int N, off;
        first_tile<TILE>(p, lengths, b, N, off);
        grid_dependency_wait();
        grid_launch_dependents();
        if (v.nt == 0 || k0 >= v.L) return;
        float w[SM_KEYS / SM_THREADS] = {};
        for (int r0 = 0; r0 < p.rows; r0 += SM_THREADS) {
            __syncthreads();
            const int rr = r0 + tid;
            if (rr < p.rows) {
                const RowRecords x = row_records(p, rec, false, g * p.nrb + rr / bm, off,
                                                 p.blocks_p() + b * p.blocks_c(), v.nt, N, gangs, rr % bm);
                float M = -INFINITY, l = 0.f;
                for (int c = 0; c < x.n; ++c) M = fmaxf(M, rec.ml[x.first + c * x.step].x);
                for (int c = 0; c < x.n; ++c) {
                    const float2 ml = rec.ml[x.first + c * x.step];
                    if (ml.x != -INFINITY) l = fmaf(exp2f(ml.x - M), ml.y, l);
                }
                row_ml[tid] = make_float2(M, 1.f / l);
            }
            __syncthreads();
            const int nr = min(SM_THREADS, p.rows - r0);
            const float* s = scores + ((int64_t)bg * p.rows + r0) * score_ld(p) + k0;
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

template <typename T, int TILE>
cudaError_t merge(const SpanShape& p, const SpanRecords& rec, int bm, int gangs, void* O, int64_t ldo,
                  const int32_t* lengths, const float* scores, float* weights, cudaStream_t stream) {
    const int64_t out_rows = (int64_t)p.B * p.per * p.h_kv * p.T_q;
    const int64_t blocks =
        out_rows + (weights != nullptr ? (int64_t)p.B * p.h_kv * ((p.T_max + SM_KEYS - 1) / SM_KEYS) : 0);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    auto kernel = weights != nullptr ? span_merge_kernel<T, TILE, true> : span_merge_kernel<T, TILE, false>;
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(SM_THREADS), 0, stream, p, rec, bm, gangs,
                      static_cast<T*>(O), ldo, lengths, scores, weights);
}

}  // namespace

cudaError_t launch_span_merge(mha_dtype dtype, const SpanShape& p, const SpanRecords& rec, int bm, int gangs, void* O,
                              int64_t ldo, const int32_t* lengths, const float* scores, float* weights,
                              cudaStream_t stream) {
    if (dtype == MHA_F32) return merge<float, 64>(p, rec, bm, gangs, O, ldo, lengths, scores, weights, stream);
    return merge<__nv_bfloat16, 128>(p, rec, bm, gangs, O, ldo, lengths, scores, weights, stream);
}

}  // namespace mha
