// quant_meet.cuh -- how a CTA's warps join their results of a piece (quant.cuh), and the rows of invalid lengths.
#pragma once

#include <math.h>

#include "ptx.cuh"
#include "quant.cuh"

namespace mha {

__device__ __forceinline__ void quant_put(float* p, float x) { *p = x; }
__device__ __forceinline__ void quant_put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float quant_power2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 .. 127
__device__ __forceinline__ int quant_exponent(float x) { return (int)(__float_as_uint(x) >> 23 & 255u) - 127; }

// A row's weights times steps, p s, are rounded to fp16 as p s vs, vs a power of two.  They fit while a step times vs is at
// most this, as a weight is at most 2^8 (a larger one moves the row's reference); what does not, or moves it, asks for
// the new vs where the largest p s of the tokens at hand is `need` and the row's sums so far are about to be multiplied
// by f <= 1: to [4, 8) downwards if it is above 16, and upwards, as far as f makes room for it, if it is below 1/4.
// (Steps differ by tokens: with [32, 64) a third of quant_rows.cu's tiles had to ask.)
constexpr float kQuantStepMost = 255.f;
__device__ __forceinline__ float quant_move_scale(float vs, float need, float f) {
    const float x = need * vs;
    if (x > 16.f || (x < 0.25f && f < 1.f)) {
        const int now = quant_exponent(vs), most = x > 16.f ? now : max(now, min(100, now - 1 - quant_exponent(f)));
        vs = quant_power2(max(-126, min(most, 2 - quant_exponent(need))));
    }
    return vs;
}
// to / from for two of them, times f <= 1 (which is zero where the quotient may not be finite).
__device__ __forceinline__ float quant_rescale(float to, float from, float f) { return f * to * quant_power2(-quant_exponent(from)); }

// Where row r of the block that begins at row r0 of a head's rows goes.
template <typename T>
__device__ __forceinline__ T* quant_out(const QuantStep& s, T* O, int64_t ldo, int b, int g, int rr) {
    const int hg = s.by_T_q((uint32_t)rr);
    return O + ((int64_t)b * s.T_q + (rr - hg * s.T_q)) * ldo + (int64_t)(g * s.per + hg) * s.dv;
}

// Batches b, b + step, .. with an invalid length: NaN rows and a status.
template <int THREADS, typename T>
__device__ __noinline__ void quant_invalid(const QuantStep& s, int b, int step, const int32_t* lengths, T* O, int64_t ldo, int* status) {
    for (; b < s.B; b += step) {
        const int L = __ldcg(lengths + b);
        if (L >= s.T_q && L <= s.T_max) continue;
        if (threadIdx.x == 0) record_status(status, kStatusBadLength);
        const int width = s.h_kv * s.per * s.dv;
        for (int t = 0; t < s.T_q; ++t)
            for (int e = (int)threadIdx.x; e < width; e += THREADS) quant_put(O + ((int64_t)b * s.T_q + t) * ldo + e, NAN);
    }
}

// A piece's ENTRIES results for each of `rows` rows (the warps', or several of a warp), [entry][row] of `stride` floats:
// dv values, then at ml m and l.  Either they are finished (whole), or they become records at rec.  All threads, behind a
// barrier; an entry's m becomes its factor.  DV: dv if it is known.
template <int ENTRIES, int THREADS, int DV, typename T>
__device__ __forceinline__ void quant_meet(const QuantStep& s, bool whole, float* rec, float* res, int rows, int stride, int ml,
                                           int b, int g, int r0, int nr, T* O, int64_t ldo) {
    const int tid = (int)threadIdx.x, dv = DV > 0 ? DV : s.dv, record = dv + 2;
    // ENTRIES lanes a row: maximum and sum
    for (int r = tid / ENTRIES; r < nr; r += THREADS / ENTRIES) {
        float* a = res + ((tid % ENTRIES) * rows + r) * stride + ml;
        const unsigned lanes = ((1u << ENTRIES) - 1) << (tid & 31 & ~(ENTRIES - 1));
        const float m = a[0];
        float M = m;
#pragma unroll
        for (int w = ENTRIES / 2; w >= 1; w >>= 1) M = fmaxf(M, __shfl_xor_sync(lanes, M, w));
        const float f = m == -INFINITY ? 0.f : exp2f(m - M);
        float l = f * a[1];
#pragma unroll
        for (int w = ENTRIES / 2; w >= 1; w >>= 1) l += __shfl_xor_sync(lanes, l, w);
        if (whole) {
            a[0] = f / l;  // (l is NaN, or above zero: a whole group has a visible token for every row)
        } else {
            a[0] = f;
            if (tid % ENTRIES == 0) {
                rec[r * record] = M;
                rec[r * record + 1] = l;
            }
        }
    }
    __syncthreads();
    for (int e = tid; e < nr * dv; e += THREADS) {
        const int r = e / dv, c = e - r * dv;
        const float* a = res + r * stride;
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < ENTRIES; ++w) x = fmaf(a[w * rows * stride + ml], a[w * rows * stride + c], x);
        if (whole) quant_put(quant_out(s, O, ldo, b, g, r0 + r) + c, x);
        else rec[r * record + 2 + c] = x;
    }
}

}  // namespace mha
