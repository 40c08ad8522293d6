// quant_cache.cu -- writing keys and values into a quantised cache (quant.cuh) and reading them back.
//
// For a group of 64 channels x, n = 2^bits - 1:
//   m    = the largest bf16 not above min x
//   s    = the smallest bf16 with n s >= max x - m, at least 2^-126
//   code = (x - m) / s rounded to the nearest whole number, ties to even
// so every code fits and s code + m is within s / 2 of x.  bf16 inputs have their minimum as m exactly.  These are
// definitions over the real numbers: codes next to a border between two are settled exactly, so a cache does not
// depend on how a machine rounds on the way.  A group with a value that is not finite in bf16 gets NaN for s and m
// and reads back as NaN.
//
// Eight lanes hold a group, eight channels each (16 bytes of bf16); a warp takes 16 groups of one token's keys or
// values, all loads first.  Both directions are bound by HBM.
#include <math.h>

#include "internal.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace mha {
namespace {

constexpr int QC_THREADS = 256;
constexpr int QC_WARPS = QC_THREADS / 32;
constexpr int QC_RUN = 4;                // groups per eight lanes
constexpr int QC_GROUPS = 4 * QC_RUN;    // groups per warp
constexpr float kBf16Max = 3.3895313892515355e38f;

// Which of a call's rows a warp has: token of the cache, batch; false: none.
__device__ __forceinline__ bool quant_warp_row(int B, int T, int T_max, const int32_t* lengths, const int32_t* counts,
                                               int* status, int64_t& row, int& b, int& token) {
    row = (int64_t)blockIdx.x * QC_WARPS + (threadIdx.x >> 5);
    if (row >= (int64_t)B * T) return false;
    b = (int)row / T;
    const int i = (int)row - b * T;
    const QuantRows r = quant_rows(lengths[b], counts != nullptr ? counts[b] : T, T, T_max);
    if (!r.valid) {
        if (i == 0 && blockIdx.y == 0 && (threadIdx.x & 31) == 0) record_status(status, kStatusBadLength);
        return false;
    }
    token = r.first + i;
    return i < r.n;
}

// x to bf16 (as fp32), towards minus infinity.
__device__ __forceinline__ float bf16_down(float x) {
    const uint32_t u = __float_as_uint(x), cut = u & 0xffff0000u;
    return __uint_as_float((u >> 31) && cut != u ? cut + 0x10000u : cut);
}

// a - b = s + e exactly (no overflow).
__device__ __forceinline__ void two_diff(float a, float b, float& s, float& e) {
    s = __fsub_rn(a, b);
    const float bb = __fsub_rn(s, a);  // -b as it went into s
    e = __fsub_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fadd_rn(b, bb));
}

// The smallest bf16 s >= 2^-126 with n s >= hi - m.  n s is exact in fp32.
__device__ __forceinline__ float group_step(float hi, float m, float n) {
    float a, e;
    two_diff(hi, m, a, e);
    // from below: a / n less up to 2 units in the last place of bf16, cut; at most 4 units above lies the step
    float s = __uint_as_float(__float_as_uint(__fmul_rn(__fdiv_rn(a, n), 0.9921875f)) & 0xffff0000u);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (__fsub_rn(__fmul_rn(n, s), a) < e) s = __uint_as_float(__float_as_uint(s) + 0x10000u);
    return fmaxf(s, 1.17549435e-38f);
}

// The code of x: q is (x - m) / s to within 2^-14.
__device__ __noinline__ int code_at_border(float x, float m, float s, float q) {
    const float k = floorf(q);
    float a, e;
    two_diff(x, m, a, e);
    // both terms are exact: (k + 1/2) s has at most 17 bits, and a is near it
    const float over = __fadd_rn(__fsub_rn(a, __fmul_rn(k + 0.5f, s)), e);
    const int c = (int)k;
    return over > 0.f ? c + 1 : over < 0.f ? c : c + (c & 1);
}

__device__ __forceinline__ int code_of(float x, float m, float s, float inv) {
    const float q = __fmul_rn(__fsub_rn(x, m), inv);  // off by at most 255 * 3 * 2^-24
    const float r = rintf(q);
    if (fabsf(q - r) > 0.5f - 6.1e-5f) return code_at_border(x, m, s, q);
    return (int)r;
}

template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int n, float (&x)[8]) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (n > 0) v = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

template <bool VEC>
__device__ __forceinline__ void load8(const float* p, int n, float (&x)[8]) {
    if constexpr (VEC) {  // n is 0, 4 or 8
        const float4 a = n > 0 ? __ldg(reinterpret_cast<const float4*>(p)) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 b = n > 4 ? __ldg(reinterpret_cast<const float4*>(p) + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < n ? __ldg(p + i) : 0.f;
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16* p, int n, const float (&x)[8]) {
    if (n > 0)
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                                  pack_bf16x2(x[6], x[7]));
}

template <bool VEC>
__device__ __forceinline__ void store8(float* p, int n, const float (&x)[8]) {
    if constexpr (VEC) {
        if (n > 0) *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
        if (n > 4) *(reinterpret_cast<float4*>(p) + 1) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = x[i];
    }
}

// This thread's channels of its u-th group: head, channel in the head, how many of the eight exist.
struct QuantEight {
    int head, sub, c0, n;
    __device__ __forceinline__ QuantEight(const QuantPlane& p, int h_kv, int chunk, int u) {
        const int lane = (int)threadIdx.x & 31, gi = chunk * QC_GROUPS + 4 * u + (lane >> 3);
        head = p.groups == 1 ? gi : gi / p.groups;
        sub = gi - head * p.groups;
        c0 = sub * kQuantGroup + 8 * (lane & 7);
        n = head < h_kv ? max(0, min(8, p.d - c0)) : 0;
    }
};

template <typename T, int BITS, bool VEC>
__global__ void __launch_bounds__(QC_THREADS)
    quant_write_kernel(const QuantPlane pk, const QuantPlane pv, const T* __restrict__ K, int64_t ldk,
                       const T* __restrict__ V, int64_t ldv, int B, int T_new, int T_max, int h_kv, int k_chunks,
                       const int32_t* __restrict__ lengths, const int32_t* __restrict__ counts, int* status) {
    constexpr int N = (1 << BITS) - 1;
    grid_dependency_wait();
    grid_launch_dependents();
    int64_t row;
    int b, token;
    if (!quant_warp_row(B, T_new, T_max, lengths, counts, status, row, b, token)) return;
    const bool values = (int)blockIdx.y >= k_chunks;
    const QuantPlane p = values ? pv : pk;
    const int chunk = (int)blockIdx.y - (values ? k_chunks : 0);
    const T* src = values ? V + row * ldv : K + row * ldk;
    float x[QC_RUN][8];
#pragma unroll
    for (int u = 0; u < QC_RUN; ++u) {
        const QuantEight a(p, h_kv, chunk, u);
        load8<VEC>(src + (int64_t)a.head * p.d + a.c0, a.n, x[u]);
    }
    const int lane = (int)threadIdx.x & 31;
#pragma unroll
    for (int u = 0; u < QC_RUN; ++u) {
        const QuantEight a(p, h_kv, chunk, u);
        float lo = INFINITY, hi = -INFINITY;
        bool fine = true;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < a.n) {
                lo = fminf(lo, x[u][i]);
                hi = fmaxf(hi, x[u][i]);
                fine = fine && fabsf(x[u][i]) <= kBf16Max;
            }
#pragma unroll
        for (int w = 1; w < 8; w <<= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, w));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, w));
        }
        const uint32_t good = __ballot_sync(0xffffffffu, fine) >> (lane & 24) & 0xffu;
        if (a.head >= h_kv) continue;
        uint32_t par = 0x7fff7fffu;  // NaN
        uint32_t c[BITS == 4 ? 1 : 2] = {};
        if (good == 0xffu) {
            float m = bf16_down(lo), f = 1.f;
            if (hi - m > 3.4e38f) {  // differences would overflow: in halves, which changes no code
                f = 0.5f;
                m *= f;
                hi *= f;
#pragma unroll
                for (int i = 0; i < 8; ++i) x[u][i] *= f;
            }
            const float s = group_step(hi, m, (float)N), inv = __fdiv_rn(1.f, s);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < a.n) c[i * BITS / 32] |= (uint32_t)min(code_of(x[u][i], m, s, inv), N) << (i * BITS % 32);
            par = __float_as_uint(s / f) >> 16 | (__float_as_uint(m / f) & 0xffff0000u);
        }
        const int64_t at = ((int64_t)b * h_kv + a.head) * T_max + token;
        if (a.c0 * BITS / 8 < p.row) {
            uint8_t* out = p.codes + at * p.row + a.c0 * BITS / 8;
            if constexpr (BITS == 4) *reinterpret_cast<uint32_t*>(out) = c[0];
            else *reinterpret_cast<uint2*>(out) = make_uint2(c[0], c[1]);
        }
        if ((lane & 7) == 0) p.params[at * p.groups + a.sub] = par;
    }
}

template <typename T, int BITS, bool VEC>
__global__ void __launch_bounds__(QC_THREADS)
    quant_read_kernel(const QuantPlane pk, const QuantPlane pv, T* __restrict__ K, int64_t ldk, T* __restrict__ V,
                      int64_t ldv, int B, int T_out, int T_max, int h_kv, int k_chunks,
                      const int32_t* __restrict__ lengths, const int32_t* __restrict__ counts, int* status) {
    grid_dependency_wait();
    grid_launch_dependents();
    int64_t row;
    int b, token;
    if (!quant_warp_row(B, T_out, T_max, lengths, counts, status, row, b, token)) return;
    const bool values = (int)blockIdx.y >= k_chunks;
    const QuantPlane p = values ? pv : pk;
    const int chunk = (int)blockIdx.y - (values ? k_chunks : 0);
    T* dst = values ? V + row * ldv : K + row * ldk;
    uint2 c[QC_RUN];
    uint32_t par[QC_RUN];
#pragma unroll
    for (int u = 0; u < QC_RUN; ++u) {
        const QuantEight a(p, h_kv, chunk, u);
        const int64_t at = ((int64_t)b * h_kv + a.head) * T_max + token;
        c[u] = make_uint2(0u, 0u);
        par[u] = 0;
        if (a.n > 0) {
            const uint8_t* in = p.codes + at * p.row + a.c0 * BITS / 8;
            if constexpr (BITS == 4) c[u].x = __ldg(reinterpret_cast<const uint32_t*>(in));
            else c[u] = __ldg(reinterpret_cast<const uint2*>(in));
            par[u] = __ldg(p.params + at * p.groups + a.sub);
        }
    }
#pragma unroll
    for (int u = 0; u < QC_RUN; ++u) {
        const QuantEight a(p, h_kv, chunk, u);
        const float s = quant_step(par[u]), m = quant_lowest(par[u]);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t w = i * BITS < 32 ? c[u].x : c[u].y;
            x[i] = fmaf((float)(w >> (i * BITS % 32) & ((1 << BITS) - 1)), s, m);  // s code is exact
        }
        store8<VEC>(dst + (int64_t)a.head * p.d + a.c0, a.n, x);
    }
}

int chunks(const QuantPlane& p, int h_kv) {
    return (int)(((int64_t)h_kv * p.groups + QC_GROUPS - 1) / QC_GROUPS);
}

bool vec_ok(const QuantPlane& p, const void* x, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(x) & 15) == 0 && ld % 4 == 0 && p.d % 4 == 0;
}

}  // namespace

bool quant_copy_fits(const QuantPlane& pk, const QuantPlane& pv, int h_kv) {
    return (int64_t)h_kv * pk.groups <= (int64_t)32767 * QC_GROUPS && (int64_t)h_kv * pv.groups <= (int64_t)32767 * QC_GROUPS;
}

cudaError_t launch_quant_copy(bool write, bool f32, int bits, const QuantPlane& pk, const QuantPlane& pv, void* K,
                              int64_t ldk, void* V, int64_t ldv, int B, int T, int T_max, int h_kv,
                              const int32_t* lengths, const int32_t* counts, int* status, cudaStream_t stream) {
    const int kc = chunks(pk, h_kv), vc = chunks(pv, h_kv);
    const dim3 grid((unsigned)(((int64_t)B * T + QC_WARPS - 1) / QC_WARPS), (unsigned)(kc + vc));
    const bool vec = !f32 || (vec_ok(pk, K, ldk) && vec_ok(pv, V, ldv));
    auto go = [&](auto* x, auto kw, auto kr) {
        using T_ = std::remove_pointer_t<decltype(x)>;
        if (write)
            return launch_pdl(kw, grid, dim3(QC_THREADS), 0, stream, pk, pv, static_cast<const T_*>(K), ldk,
                              static_cast<const T_*>(V), ldv, B, T, T_max, h_kv, kc, lengths, counts, status);
        return launch_pdl(kr, grid, dim3(QC_THREADS), 0, stream, pk, pv, static_cast<T_*>(K), ldk, static_cast<T_*>(V), ldv,
                          B, T, T_max, h_kv, kc, lengths, counts, status);
    };
#define MHA_QC(T, BITS, VEC) return go(static_cast<T*>(nullptr), quant_write_kernel<T, BITS, VEC>, quant_read_kernel<T, BITS, VEC>)
    if (!f32) {
        if (bits == 4) MHA_QC(__nv_bfloat16, 4, true);
        MHA_QC(__nv_bfloat16, 8, true);
    }
    if (vec) {
        if (bits == 4) MHA_QC(float, 4, true);
        MHA_QC(float, 8, true);
    }
    if (bits == 4) MHA_QC(float, 4, false);
    MHA_QC(float, 8, false);
#undef MHA_QC
}

}  // namespace mha
