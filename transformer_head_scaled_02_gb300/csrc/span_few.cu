// span_few.cu -- the units of the fp32 cache steps (span.cuh) with few query rows: bound by HBM, so keys and
// values go straight from global memory to registers, once, in pieces of 16 bytes.
//
// A block takes a unit at a time; its 8 warps take 32 keys at a time in turn, each with its own running maximum, sum and
// values, joined at the unit's end.  16 lanes hold a key (4 of its elements per lane and chunk of 64), so a warp
// reads two keys with one load.  A row's 16 partial products per lane meet by halving: in each of four steps a
// lane hands over the half of its keys that the other half of the lanes ends up with, 15 shuffles for
// 32 keys, after which every lane holds one key's score.  R rows share each key: R * CH <= 8 keeps the
// queries, the accumulators and 16 keys' loads in registers (blocks of one row were no faster than of two).
// Units are multiples of 4 tiles where there are enough keys, so that no warp idles: with 2 tiles a unit the
// same work took twice as long.
//
// Bound by HBM latency: 179 to 255 registers leave one block an SM, whose warps have 8 KB in flight each and wait
// for K before V.  16 caches of 4096 tokens, 4 K/V
// heads, one row: d = 64 40 us (134 MB, 50 % of the measured copy rate; in tiles, span_simt.cu, 106), d = 128
// 63 us (64 %; 170), d = 256 242 us (33 %; 356).
#include <math.h>

#include "internal.h"
#include "ptx.cuh"
#include "span_records.cuh"

namespace mha {
namespace {

constexpr int SF_THREADS = 256;
constexpr int SF_WARPS = SF_THREADS / 32;
constexpr int SF_TILE = 64;

// 4 consecutive elements of a row, zeros past n.
template <bool VEC>
__device__ __forceinline__ float4 few_load(const float* p, int n) {
    if constexpr (VEC) return n > 0 ? __ldg(reinterpret_cast<const float4*>(p)) : make_float4(0.f, 0.f, 0.f, 0.f);
    return make_float4(n > 0 ? __ldg(p) : 0.f, n > 1 ? __ldg(p + 1) : 0.f, n > 2 ? __ldg(p + 2) : 0.f, n > 3 ? __ldg(p + 3) : 0.f);
}

__device__ __forceinline__ float dot4(const float4 a, const float4 b, float s) {
    return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, s))));
}

template <int R, int CH, bool VEC>
__global__ void __launch_bounds__(SF_THREADS)
    span_few_kernel(const SpanShape p, const SpanRecords rec, const float* __restrict__ Q, int64_t ldq,
                    const float* __restrict__ K, int64_t ldk, const float* __restrict__ V, int64_t ldv,
                    const float* __restrict__ Kp, int64_t ldkp, const float* __restrict__ Vp, int64_t ldvp,
                    float* __restrict__ O, int64_t ldo, int dk, int dv, const int32_t* __restrict__ lengths,
                    float* __restrict__ scores, float scale_log2, int prefix_units, int cache_units, int* status) {
    constexpr int KB = 16 / CH;  // key pairs loaded at a time
    __shared__ float part[SF_WARPS][R][64 * CH + 2];
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5, half = lane >> 4, l16 = lane & 15;
    grid_dependency_wait();  // lengths, queries and caches may come from the previous kernel
    grid_launch_dependents();
    SpanSums sums;
    const SpanPlan plan = span_plan<SF_TILE>(p, lengths, (int)gridDim.x, sums);
    if (blockIdx.x == 0)
        for (int b = tid; b < p.B; b += SF_THREADS)
            if (lengths[b] < p.T_q || lengths[b] > p.T_max) record_status(status, kStatusBadLength);
    const int end = cache_units ? plan.N : plan.np;
    for (int unit = (prefix_units ? 0 : plan.np) + (int)blockIdx.x; unit < end; unit += (int)gridDim.x) {
        const SpanUnit q = span_unit<SF_TILE>(p, lengths, plan, sums, unit);
        const int bm = q.prefix ? p.bm_p : p.bm_c;
        const int r0 = q.rb * bm;
        const int nr = min(bm, (q.prefix ? p.B * p.rows : p.rows) - r0);  // <= R
        auto where = [&](int r, int& b, int& head, int& t) {
            int rr = r0 + r;
            b = q.b;
            if (q.prefix) {
                b = rr / p.rows;
                rr -= b * p.rows;
            }
            const int hg = rr / p.T_q;
            head = q.g * p.per + hg;
            t = rr - hg * p.T_q;
        };
        float4 qv[R][CH], o[R][CH];
        float m[R], l[R];
        int pos[R];  // cache position of the row's token
#pragma unroll
        for (int r = 0; r < R; ++r) {
            int b, head, t;
            where(min(r, nr - 1), b, head, t);
            pos[r] = q.v.L - p.T_q + t;
            m[r] = -INFINITY;
            l[r] = 0.f;
            const float* src = Q + ((int64_t)b * p.T_q + t) * ldq + (int64_t)head * dk;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int e = 64 * c + 4 * l16;
                qv[r][c] = few_load<VEC>(src + e, dk - e);
                qv[r][c].x *= scale_log2; qv[r][c].y *= scale_log2; qv[r][c].z *= scale_log2; qv[r][c].w *= scale_log2;
                o[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        const float* Kb = (q.prefix ? Kp : K + (int64_t)q.b * p.T_max * ldk) + (int64_t)q.g * dk + 4 * l16;
        const float* Vb = (q.prefix ? Vp : V + (int64_t)q.b * p.T_max * ldv) + (int64_t)q.g * dv + 4 * l16;
        const int64_t lk = q.prefix ? ldkp : ldk, lv = q.prefix ? ldvp : ldv;
        for (int step = 2 * q.i0 + warp; step < 2 * q.i1; step += SF_WARPS) {
            int key0, n;
            span_tile<SF_TILE>(q.v, step >> 1, key0, n);
            key0 += 32 * (step & 1);
            n -= 32 * (step & 1);
            if (n <= 0) continue;
            n = min(n, 32);
            // scores: this lane's key of the 32 is 2 l16 + half
            float s[R];
            if constexpr (KB == 16) {
                float4 k[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    k[i] = 2 * i + half < n ? few_load<VEC>(Kb + (int64_t)(key0 + 2 * i + half) * lk, dk - 4 * l16) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float x[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = dot4(qv[r][0], k[i], 0.f);
#pragma unroll
                    for (int w = 8; w >= 1; w >>= 1)
#pragma unroll
                        for (int i = 0; i < w; ++i) {
                            const float give = (l16 & w) ? x[i] : x[i + w], keep = (l16 & w) ? x[i + w] : x[i];
                            x[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
                        }
                    s[r] = x[0];
                }
            } else {
                float x[R][16];
#pragma unroll
                for (int i0 = 0; i0 < 16; i0 += KB) {
                    float4 k[KB][CH];
#pragma unroll
                    for (int i = 0; i < KB; ++i)
#pragma unroll
                        for (int c = 0; c < CH; ++c)
                            k[i][c] = 2 * (i0 + i) + half < n
                                          ? few_load<VEC>(Kb + (int64_t)(key0 + 2 * (i0 + i) + half) * lk + 64 * c, dk - 64 * c - 4 * l16)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int i = 0; i < KB; ++i) {
                            float y = 0.f;
#pragma unroll
                            for (int c = 0; c < CH; ++c) y = dot4(qv[r][c], k[i][c], y);
                            x[r][i0 + i] = y;
                        }
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
#pragma unroll
                    for (int w = 8; w >= 1; w >>= 1)
#pragma unroll
                        for (int i = 0; i < w; ++i) {
                            const float give = (l16 & w) ? x[r][i] : x[r][i + w], keep = (l16 & w) ? x[r][i + w] : x[r][i];
                            x[r][i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
                        }
                    s[r] = x[r][0];
                }
            }
            const int j = 2 * l16 + half, key = key0 + j;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (j >= n || !(q.prefix || span_visible(p, pos[r], key))) s[r] = -INFINITY;
                if (scores != nullptr && j < n && r < nr)
                    scores[(((int64_t)q.b * p.h_kv + q.g) * p.rows + r0 + r) * score_ld(p) + key] = s[r];
                float top = s[r];
#pragma unroll
                for (int w = 16; w >= 1; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                if (top > m[r]) {  // the same in all lanes
                    const float f = exp2f(m[r] - top);  // 0 when m leaves -inf
                    l[r] *= f;
#pragma unroll
                    for (int c = 0; c < CH; ++c) o[r][c].x *= f, o[r][c].y *= f, o[r][c].z *= f, o[r][c].w *= f;
                    m[r] = top;
                }
                s[r] = m[r] == -INFINITY ? 0.f : exp2f(s[r] - m[r]);  // masked: 2^-inf = 0
                l[r] += s[r];  // per lane: added up at the end
            }
#pragma unroll
            for (int i0 = 0; i0 < 16; i0 += KB) {
                float4 v[KB][CH];
#pragma unroll
                for (int i = 0; i < KB; ++i)
#pragma unroll
                    for (int c = 0; c < CH; ++c)
                        v[i][c] = 2 * (i0 + i) + half < n
                                      ? few_load<VEC>(Vb + (int64_t)(key0 + 2 * (i0 + i) + half) * lv + 64 * c, dv - 64 * c - 4 * l16)
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < KB; ++i)
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float w = __shfl_sync(0xffffffffu, s[r], i0 + i, 16);  // of this half's key
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            o[r][c].x = fmaf(w, v[i][c].x, o[r][c].x);
                            o[r][c].y = fmaf(w, v[i][c].y, o[r][c].y);
                            o[r][c].z = fmaf(w, v[i][c].z, o[r][c].z);
                            o[r][c].w = fmaf(w, v[i][c].w, o[r][c].w);
                        }
                    }
            }
        }
        // the warps' results meet
        __syncthreads();  // the previous unit's are no longer read
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int w = 16; w >= 1; w >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], w);
            if (lane == 0) part[warp][r][64 * CH] = m[r], part[warp][r][64 * CH + 1] = l[r];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                o[r][c].x += __shfl_xor_sync(0xffffffffu, o[r][c].x, 16);
                o[r][c].y += __shfl_xor_sync(0xffffffffu, o[r][c].y, 16);
                o[r][c].z += __shfl_xor_sync(0xffffffffu, o[r][c].z, 16);
                o[r][c].w += __shfl_xor_sync(0xffffffffu, o[r][c].w, 16);
                if (half == 0) {
                    float* to = &part[warp][r][64 * c + 4 * l16];
                    to[0] = o[r][c].x; to[1] = o[r][c].y; to[2] = o[r][c].z; to[3] = o[r][c].w;
                }
            }
        }
        __syncthreads();
        const bool direct = p.T_p == 0 && q.whole();
        const int64_t slot = rec.row(p, q.unit, plan.np);
        for (int i = tid; i < nr * 64 * CH; i += SF_THREADS) {
            const int r = i / (64 * CH), e = i - r * (64 * CH);
            if (e >= dv) continue;
            float M = -INFINITY, sum = 0.f, x = 0.f;
#pragma unroll
            for (int w = 0; w < SF_WARPS; ++w) M = fmaxf(M, part[w][r][64 * CH]);
#pragma unroll
            for (int w = 0; w < SF_WARPS; ++w) {
                const float mw = part[w][r][64 * CH], f = mw == -INFINITY ? 0.f : exp2f(mw - M);
                sum = fmaf(f, part[w][r][64 * CH + 1], sum);
                x = fmaf(f, part[w][r][e], x);
            }
            if (e == 0 && (!direct || scores != nullptr)) rec.ml[slot + r] = make_float2(M, sum);
            if (direct) {
                int b, head, t;
                where(r, b, head, t);
                O[((int64_t)b * p.T_q + t) * ldo + (int64_t)head * dv + e] = x / sum;
            } else {
                rec.o[(slot + r) * dv + e] = x;
            }
        }
    }
}

}  // namespace

// Rows a block of the kernel holds for this width of a head: R * CH <= 8.
int span_few_rows(int d_k, int d_v) {
    const int d = d_k > d_v ? d_k : d_v;
    return d <= 64 ? 8 : d <= 128 ? 4 : 2;
}

cudaError_t launch_span_few(const SpanShape& p, const SpanRecords& rec, const float* Q, int64_t ldq, const float* K,
                            int64_t ldk, const float* V, int64_t ldv, const float* Kp, int64_t ldkp, const float* Vp,
                            int64_t ldvp, float* O, int64_t ldo, int d_k, int d_v, const int32_t* lengths, float* scores,
                            bool prefix_units, bool cache_units, int ctas, int* status, cudaStream_t stream) {
    auto al = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
    const bool vec = al(Q) && al(K) && al(V) && ldq % 4 == 0 && ldk % 4 == 0 && ldv % 4 == 0 && d_k % 4 == 0 &&
                     d_v % 4 == 0 && (p.T_p == 0 || (al(Kp) && al(Vp) && ldkp % 4 == 0 && ldvp % 4 == 0));
    const float scale = (float)(1.4426950408889634 / sqrt((double)d_k));
    const int d = d_k > d_v ? d_k : d_v, ch = d <= 64 ? 1 : d <= 128 ? 2 : 4;
    int rows = 1;  // of the blocks that this launch has
    if (prefix_units && p.T_p > 0) rows = p.rps_p();
    if (cache_units && p.rps_c() > rows) rows = p.rps_c();
    auto launch = [&](auto kernel) {
        return launch_pdl(kernel, dim3((unsigned)ctas), dim3(SF_THREADS), 0, stream, p, rec, Q, ldq, K, ldk, V, ldv, Kp,
                          ldkp, Vp, ldvp, O, ldo, d_k, d_v, lengths, scores, scale, prefix_units ? 1 : 0,
                          cache_units ? 1 : 0, status);
    };
#define MHA_SF(R, CH) \
    if (rows <= R && ch == CH) return vec ? launch(span_few_kernel<R, CH, true>) : launch(span_few_kernel<R, CH, false>);
    MHA_SF(2, 1) MHA_SF(4, 1) MHA_SF(8, 1) MHA_SF(2, 2) MHA_SF(4, 2) MHA_SF(2, 4)
#undef MHA_SF
    return cudaErrorInvalidValue;
}

}  // namespace mha
