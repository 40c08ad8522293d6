// quant_decode.cu -- a decode step over a quantised cache (quant.cuh) on CUDA cores, for any head size.
//
// With codes c, steps s and lowest values m per group G of channels, and the query row q (log2(e)/sqrt(d) folded in):
//   score_j = sum_G s_jG (sum_c q_c code_jc) + m_jG (sum_c q_c)          the codes are never turned into values
//   o       = sum_j p_j (s_jG code_jc + m_jG),  p_j = 2^(score_j - M)
// in fp32 throughout.  A CTA takes a part of one head's cached tokens for up to R query rows; its warps take 32
// tokens at a time in turn, a lane per token for the scores and a lane per eight channels for the values, each with
// its own running maximum, sum and values, joined at the end.  Parts leave records (maximum, sum, values), which the
// join adds in order.
#include <math.h>

#include "internal.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace mha {
namespace {

constexpr int QD_THREADS = 256;
constexpr int QD_WARPS = QD_THREADS / 32;
constexpr int QD_ROWS = 4;

__device__ __forceinline__ float elem(const float* p) { return *p; }
__device__ __forceinline__ float elem(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Eight codes of a row as fp32.
template <int BITS>
__device__ __forceinline__ void codes8(const uint8_t* p, float (&x)[8]) {
    if constexpr (BITS == 4) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)(w >> (4 * i) & 15u);
    } else {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)((i < 4 ? w.x : w.y) >> (8 * (i & 3)) & 255u);
    }
}

// dynamic shared memory: q[R][dpk], its sums qs[R][groups], and per warp p[R][32] or at the end m, l, o[dpv] per row
template <typename T, int BITS>
__global__ void __launch_bounds__(QD_THREADS)
    quant_decode_kernel(const QuantStep s, const QuantPlane pk, const QuantPlane pv, const T* __restrict__ Q, int64_t ldq,
                        T* __restrict__ O, int64_t ldo, const int32_t* __restrict__ lengths, float scale_log2,
                        float* __restrict__ part, int* status) {
    constexpr int R = QD_ROWS;
    extern __shared__ float sm[];
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int dpk = (pk.d + 31) & ~31, dpv = (pv.d + 31) & ~31;
    float* q = sm;
    float* qs = q + R * dpk;
    float* own = qs + R * pk.groups + warp * R * (dpv + 32);
    grid_dependency_wait();
    grid_launch_dependents();
    int i = (int)blockIdx.x;
    const int rb = i % s.nrb;
    i /= s.nrb;
    const int split = i % s.splits;
    i /= s.splits;
    const int g = i % s.h_kv, b = i / s.h_kv;
    const int L = lengths[b], r0 = rb * R, nr = min(R, s.rows - r0);
    auto out_row = [&](int r, int& head, int& t) {
        head = g * s.per + (r0 + r) / s.T_q;
        t = (r0 + r) % s.T_q;
        return O + ((int64_t)b * s.T_q + t) * ldo + (int64_t)head * pv.d;
    };
    if (L < s.T_q || L > s.T_max) {
        if (split == 0) {
            if (tid == 0) record_status(status, kStatusBadLength);
            int head, t;
            for (int r = 0; r < nr; ++r)
                for (int e = tid; e < pv.d; e += QD_THREADS) put(out_row(r, head, t) + e, NAN);
        }
        return;
    }
    const int span = s.part(L), k0 = split * span, k1 = min(L, k0 + span);
    if (k0 >= k1) return;
    for (int e = tid; e < R * dpk; e += QD_THREADS) {
        const int r = e / dpk, c = e - r * dpk, rr = r0 + min(r, nr - 1);
        q[e] = c < pk.d ? scale_log2 * elem(Q + ((int64_t)b * s.T_q + rr % s.T_q) * ldq + (int64_t)(g * s.per + rr / s.T_q) * pk.d + c) : 0.f;
    }
    __syncthreads();
    for (int e = tid; e < R * pk.groups; e += QD_THREADS) {
        const int r = e / pk.groups, c0 = (e - r * pk.groups) * kQuantGroup;
        float x = 0.f;
        for (int c = c0; c < min(dpk, c0 + kQuantGroup); ++c) x += q[r * dpk + c];
        qs[e] = x;
    }
    __syncthreads();
    const int64_t head_row = ((int64_t)b * s.h_kv + g) * s.T_max;
    const uint8_t* kc = pk.codes + head_row * pk.row;
    const uint32_t* kp = pk.params + head_row * pk.groups;
    const uint8_t* vc = pv.codes + head_row * pv.row;
    const uint32_t* vp = pv.params + head_row * pv.groups;
    // values: `width` lanes hold a token's channels, 32 / width tokens at a time
    const int width = dpv <= 32 ? 4 : dpv <= 64 ? 8 : dpv <= 128 ? 16 : 32, c0 = 8 * (lane % width), sub = lane / width;
    const bool has = c0 < dpv;
    float m[R], l[R], o[R][8];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[r][e] = 0.f;
    }
    for (int key0 = k0 + 32 * warp; key0 < k1; key0 += 32 * QD_WARPS) {
        const int key = key0 + lane;
        float x[R];
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = 0.f;
        if (key < k1)
            for (int G = 0; G < pk.groups; ++G) {
                float dot[R];
#pragma unroll
                for (int r = 0; r < R; ++r) dot[r] = 0.f;
                for (int c = G * kQuantGroup; c < min(dpk, (G + 1) * kQuantGroup); c += 8) {
                    float v[8];
                    codes8<BITS>(kc + (int64_t)key * pk.row + c * BITS / 8, v);
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int e = 0; e < 8; ++e) dot[r] = fmaf(q[r * dpk + c + e], v[e], dot[r]);
                }
                const uint32_t par = __ldg(kp + (int64_t)key * pk.groups + G);
#pragma unroll
                for (int r = 0; r < R; ++r)
                    x[r] = fmaf(quant_step(par), dot[r], fmaf(quant_lowest(par), qs[r * pk.groups + G], x[r]));
            }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int pos = L - s.T_q + (r0 + min(r, nr - 1)) % s.T_q;
            if (key >= k1 || key > pos) x[r] = -INFINITY;
            float top = x[r];
#pragma unroll
            for (int w = 16; w >= 1; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
            if (top > m[r]) {
                const float f = exp2f(m[r] - top);
                l[r] *= f;
#pragma unroll
                for (int e = 0; e < 8; ++e) o[r][e] *= f;
                m[r] = top;
            }
            const float p = x[r] == -INFINITY ? 0.f : exp2f(x[r] - m[r]);  // (NaN stays NaN)
            l[r] += p;
            own[r * 32 + lane] = p;
        }
        __syncwarp();
        for (int j = sub; j < min(32, k1 - key0); j += 32 / width) {
            if (!has) continue;
            float v[8];
            codes8<BITS>(vc + (int64_t)(key0 + j) * pv.row + c0 * BITS / 8, v);
            const uint32_t par = __ldg(vp + (int64_t)(key0 + j) * pv.groups + c0 / kQuantGroup);
            const float vs = quant_step(par), vm = quant_lowest(par);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = fmaf(v[e], vs, vm);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float p = own[r * 32 + j];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[r][e] = fmaf(p, v[e], o[r][e]);
            }
        }
        __syncwarp();
    }
    // the warps' results meet
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int w = 16; w >= 1; w >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], w);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            for (int w = width; w < 32; w <<= 1) o[r][e] += __shfl_xor_sync(0xffffffffu, o[r][e], w);
        float* to = own + r * (dpv + 32);
        if (lane == 0) to[dpv] = m[r], to[dpv + 1] = l[r];
        if (has && sub == 0)
#pragma unroll
            for (int e = 0; e < 8; ++e) to[c0 + e] = o[r][e];
    }
    __syncthreads();
    const bool whole = span >= L;
    const float* all = qs + R * pk.groups;
    for (int e = tid; e < nr * pv.d; e += QD_THREADS) {
        const int r = e / pv.d, c = e - r * pv.d;
        float M = -INFINITY, sum = 0.f, x = 0.f;
#pragma unroll
        for (int w = 0; w < QD_WARPS; ++w) M = fmaxf(M, all[(w * R + r) * (dpv + 32) + dpv]);
#pragma unroll
        for (int w = 0; w < QD_WARPS; ++w) {
            const float* a = all + (w * R + r) * (dpv + 32);
            const float f = a[dpv] == -INFINITY ? 0.f : exp2f(a[dpv] - M);
            sum = a[dpv + 1] == 0.f ? sum : fmaf(f, a[dpv + 1], sum);
            x = fmaf(f, a[c], x);
        }
        int head, t;
        T* out = out_row(r, head, t);
        if (whole) {
            put(out + c, x / sum);
        } else {
            float* rec = part + ((((int64_t)b * s.h_kv * s.per + head) * s.T_q + t) * s.splits + split) * (pv.d + 2);
            rec[2 + c] = x;
            if (c == 0) rec[0] = M, rec[1] = sum;
        }
    }
}

// The join: one output row per block.
template <typename T>
__global__ void __launch_bounds__(128)
    quant_join_kernel(const QuantStep s, const float* __restrict__ part, T* __restrict__ O, int64_t ldo, int dv,
                      const int32_t* __restrict__ lengths) {
    const int heads = s.h_kv * s.per, row = (int)blockIdx.x;
    const int t = row % s.T_q, bh = row / s.T_q, b = bh / heads, head = bh - b * heads;
    grid_dependency_wait();
    grid_launch_dependents();
    const int L = lengths[b];
    if (L < s.T_q || L > s.T_max) return;  // written as NaN already
    const int span = s.part(L), n = (L + span - 1) / span;
    if (n == 1) return;
    const float* rec = part + (int64_t)row * s.splits * (dv + 2);
    float M = -INFINITY;
    for (int c = 0; c < n; ++c) M = fmaxf(M, rec[(int64_t)c * (dv + 2)]);
    for (int e = (int)threadIdx.x; e < dv; e += 128) {
        float sum = 0.f, x = 0.f;
        for (int c = 0; c < n; ++c) {
            const float* a = rec + (int64_t)c * (dv + 2);
            const float f = a[0] == -INFINITY ? 0.f : exp2f(a[0] - M);
            sum = fmaf(f, a[1], sum);
            x = fmaf(f, a[2 + e], x);
        }
        put(O + ((int64_t)b * s.T_q + t) * ldo + (int64_t)head * dv + e, x / sum);
    }
}

size_t qd_smem(const QuantPlane& pk, const QuantPlane& pv) {
    const int dpk = (pk.d + 31) & ~31, dpv = (pv.d + 31) & ~31;
    return sizeof(float) * (size_t)QD_ROWS * (dpk + pk.groups + QD_WARPS * (dpv + 32));
}

}  // namespace

// Rows of a block, and parts of a cache: enough of them to fill the GPU a few times over, none shorter than 256
// tokens.  Independent of the GPU, so that the workspace's size is.
QuantStep quant_step_shape(int B, int h, int h_kv, int T_q, int T_max) {
    QuantStep s;
    s.B = B;
    s.h_kv = h_kv;
    s.per = h / h_kv;
    s.T_q = T_q;
    s.T_max = T_max;
    s.rows = s.per * T_q;
    s.rb = QD_ROWS;
    s.nrb = (s.rows + s.rb - 1) / s.rb;
    const int64_t groups = (int64_t)B * h_kv * s.nrb;
    int64_t splits = (1024 + groups - 1) / groups;
    const int64_t most = ((int64_t)T_max + 255) / 256;
    if (splits > most) splits = most;
    s.splits = splits < 1 ? 1 : (int)splits;
    return s;
}

size_t quant_step_bytes(const QuantStep& s, int dv) {
    return s.splits == 1 ? 0 : sizeof(float) * (size_t)s.B * s.h_kv * s.rows * s.splits * (size_t)(dv + 2);
}

bool quant_step_fits(const QuantStep& s) {
    return (int64_t)s.B * s.h_kv * s.nrb * s.splits <= INT32_MAX && (int64_t)s.B * s.h_kv * s.rows <= INT32_MAX;
}

cudaError_t launch_quant_decode(const QuantStep& s, bool f32, int bits, const QuantPlane& pk, const QuantPlane& pv,
                                const void* Q, int64_t ldq, void* O, int64_t ldo, const int32_t* lengths, float* part,
                                int* status, cudaStream_t stream) {
    const float scale = (float)(1.4426950408889634 / sqrt((double)pk.d));
    const dim3 grid((unsigned)((int64_t)s.B * s.h_kv * s.nrb * s.splits));
    const size_t smem = qd_smem(pk, pv);
    auto go = [&](auto* x, auto kernel, auto join) {
        using T = std::remove_pointer_t<decltype(x)>;
        cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 << 10);
        if (err != cudaSuccess) return err;
        err = launch_pdl(kernel, grid, dim3(QD_THREADS), smem, stream, s, pk, pv, static_cast<const T*>(Q), ldq,
                         static_cast<T*>(O), ldo, lengths, scale, part, status);
        if (err != cudaSuccess || s.splits == 1) return err;
        return launch_pdl(join, dim3((unsigned)((int64_t)s.B * s.h_kv * s.rows)), dim3(128), 0, stream, s,
                          static_cast<const float*>(part), static_cast<T*>(O), ldo, pv.d, lengths);
    };
    if (f32) {
        float* x = nullptr;
        return bits == 4 ? go(x, quant_decode_kernel<float, 4>, quant_join_kernel<float>)
                         : go(x, quant_decode_kernel<float, 8>, quant_join_kernel<float>);
    }
    __nv_bfloat16* x = nullptr;
    return bits == 4 ? go(x, quant_decode_kernel<__nv_bfloat16, 4>, quant_join_kernel<__nv_bfloat16>)
                     : go(x, quant_decode_kernel<__nv_bfloat16, 8>, quant_join_kernel<__nv_bfloat16>);
}

}  // namespace mha
