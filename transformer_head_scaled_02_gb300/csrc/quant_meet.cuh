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
// by f <= 1: to [4, 8) downwards if it is above 16, and upwards, by `room` powers of two at most, if it is below 1/4.
// (Steps differ by tokens: with [32, 64) a third of quant_rows.cu's tiles had to ask.)
constexpr float kQuantStepMost = 255.f;
constexpr int kQuantScaleMost = 118;  // log2 of the largest vs: weights of 2^8 times it stay below 2^127
__device__ __forceinline__ bool quant_scale_rises(float vs, float need, float f) { return need * vs < 0.25f && f < 1.f; }
__device__ __forceinline__ float quant_move_scale(float vs, float need, float f, int room) {
    const float x = need * vs;
    if (x > 16.f || quant_scale_rises(vs, need, f)) {
        const int now = quant_exponent(vs), most = x > 16.f ? now : max(now, min(kQuantScaleMost, now + room));
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

__device__ __forceinline__ void quant_put4(float* p, float4 x) {  // (fp32 rows may begin anywhere)
    p[0] = x.x, p[1] = x.y, p[2] = x.z, p[3] = x.w;
}
__device__ __forceinline__ void quant_put4(__nv_bfloat16* p, float4 x) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
}

// Where a cluster's CTAs put their records of a group: each CTA finishes dv / 2^shift columns of all rows, and has the
// others' values of those, [CTA][row][column], and after them every CTA's (m, l), [CTA][row].  DV: dv.
template <int ROWS, int DV>
struct QuantShare {
    static constexpr int BYTES = ROWS * DV * 4 + kQuantCluster * ROWS * 8;
    uint32_t base;  // shared memory, the same in every CTA
    int cluster, rank;
    __device__ __forceinline__ int cols() const { return DV / cluster; }
    __device__ __forceinline__ uint32_t value(int cta, int row, int col) const { return base + (uint32_t)(((cta * ROWS + row) * cols() + col) * 4); }
    __device__ __forceinline__ uint32_t sums(int cta, int row) const { return base + (uint32_t)(ROWS * DV * 4 + (cta * ROWS + row) * 8); }
};

// A piece's ENTRIES results for each of ROWS rows (the warps', or several of a warp), [entry][row] of DV + 4 floats: DV
// values, m, l and two unused.  Either they are finished (whole), or they become records at rec, or (rec null) go to the
// cluster's CTAs.  All threads, behind a barrier; an entry's m becomes its factor.
template <int ENTRIES, int THREADS, int DV, int ROWS, typename T>
__device__ __forceinline__ void quant_meet(const QuantStep& s, bool whole, float* rec, const QuantShare<ROWS, DV>& share, float* res,
                                           int b, int g, int r0, int nr, T* O, int64_t ldo) {
    constexpr int STRIDE = DV + 4, RECORD = DV + 2;
    const int tid = (int)threadIdx.x;
    // ENTRIES lanes a row: maximum and sum
    for (int r = tid / ENTRIES; r < nr; r += THREADS / ENTRIES) {
        float* a = res + ((tid % ENTRIES) * ROWS + r) * STRIDE + DV;
        const unsigned lanes = ((1u << ENTRIES) - 1) << (tid & 31 & ~(ENTRIES - 1));
        const float m = a[0];
        float M = m;
#pragma unroll
        for (int w = ENTRIES / 2; w >= 1; w >>= 1) M = fmaxf(M, __shfl_xor_sync(lanes, M, w));
        const float f = exp2f(m - M);
        float l = f * a[1];
#pragma unroll
        for (int w = ENTRIES / 2; w >= 1; w >>= 1) l += __shfl_xor_sync(lanes, l, w);
        a[0] = whole ? f / l : f;  // (l is NaN, or above zero: a whole group has a visible token for every row)
        if (!whole) {
            const int i = tid % ENTRIES;
            if (rec != nullptr) {
                if (i == 0) *reinterpret_cast<float2*>(rec + r * RECORD) = make_float2(M, l);
            } else if (i < share.cluster) {
                st_shared_cluster_v2(mapa_shared(share.sums(share.rank, r), (uint32_t)i), M, l);
            }
        }
    }
    __syncthreads();
    for (int e = tid; e < nr * (DV / 4); e += THREADS) {
        const int r = e / (DV / 4), c = 4 * (e % (DV / 4));
        const float* a = res + r * STRIDE;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < ENTRIES; ++w) {
            const float f = a[w * ROWS * STRIDE + DV];
            const float4 v = *reinterpret_cast<const float4*>(a + w * ROWS * STRIDE + c);
            x = make_float4(fmaf(f, v.x, x.x), fmaf(f, v.y, x.y), fmaf(f, v.z, x.z), fmaf(f, v.w, x.w));
        }
        if (whole) {
            T* to = quant_out(s, O, ldo, b, g, r0 + r) + c;
            if (sizeof(T) == 2 || c + 4 <= s.dv) {
                quant_put4(to, x);
            } else {  // fp32 layers' heads may have fewer channels than are computed with
                const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + i < s.dv) quant_put(to + i, v[i]);
            }
        } else if (rec != nullptr) {
            *reinterpret_cast<float2*>(rec + r * RECORD + 2 + c) = make_float2(x.x, x.y);
            *reinterpret_cast<float2*>(rec + r * RECORD + 4 + c) = make_float2(x.z, x.w);
        } else {
            const int to = c / share.cols();
            st_shared_cluster_v4(mapa_shared(share.value(share.rank, r, c - to * share.cols()), (uint32_t)to), x);
        }
    }
}

}  // namespace mha
