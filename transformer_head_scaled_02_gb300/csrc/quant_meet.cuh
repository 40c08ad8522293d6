// quant_meet.cuh -- how a CTA's warps join their results of a piece (quant.cuh), and the rows of invalid lengths.
#pragma once

#include <math.h>

#include "ptx.cuh"
#include "quant.cuh"

namespace mha {

__device__ __forceinline__ void quant_put(float* p, float x) { *p = x; }
__device__ __forceinline__ void quant_put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Where row r of the block that begins at row r0 of a head's rows goes.
template <typename T>
__device__ __forceinline__ T* quant_out(const QuantStep& s, T* O, int64_t ldo, int b, int g, int rr) {
    const int hg = rr / s.T_q;
    return O + ((int64_t)b * s.T_q + (rr - hg * s.T_q)) * ldo + (int64_t)(g * s.per + hg) * s.dv;
}

// Batches with an invalid length: NaN rows and a status, by the CTA of the batch's number modulo the grid.
template <int THREADS, typename T>
__device__ __forceinline__ void quant_invalid(const QuantStep& s, const int32_t* lengths, T* O, int64_t ldo, int* status) {
    for (int b = (int)blockIdx.x; b < s.B; b += (int)gridDim.x) {
        const int L = __ldcg(lengths + b);
        if (L >= s.T_q && L <= s.T_max) continue;
        if (threadIdx.x == 0) record_status(status, kStatusBadLength);
        const int width = s.h_kv * s.per * s.dv;
        for (int t = 0; t < s.T_q; ++t)
            for (int e = (int)threadIdx.x; e < width; e += THREADS) quant_put(O + ((int64_t)b * s.T_q + t) * ldo + e, NAN);
    }
}

// Value c of row r over the warps' results: warp w's at value[w * stride], its m and l at ml[w * stride].  A group that
// the CTA has alone is finished, another leaves a record.
template <int WARPS, typename T>
__device__ __forceinline__ void quant_meet(const QuantStep& s, const QuantPiece& z, const float* value, const float* ml,
                                           int stride, int g, int r0, int r, int c, T* O, int64_t ldo, float* part) {
    float M = -INFINITY, sum = 0.f, x = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, ml[w * stride]);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        const float m = ml[w * stride], f = m == -INFINITY ? 0.f : exp2f(m - M);
        sum = fmaf(f, ml[w * stride + 1], sum);
        x = fmaf(f, value[w * stride], x);
    }
    if (z.whole()) {
        quant_put(quant_out(s, O, ldo, z.b, g, r0 + r) + c, x / sum);
        return;
    }
    float* rec = part + s.slot((int)blockIdx.x, z.q0 == 0 ? 1 : 0, r);
    rec[2 + c] = x;
    if (c == 0) rec[0] = M, rec[1] = sum;
}

}  // namespace mha
