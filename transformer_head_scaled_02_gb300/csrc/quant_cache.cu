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
// A warp takes a run of tokens of one head's keys or values: 8 lanes a group, 8 channels a lane (16 bytes of bf16, 4
// or 8 of codes), so codes move in whole pieces and keys in rows of a head; all loads first.  Neighbouring warps have
// neighbouring heads.
//
// Measured, 4 bits, heads of 128, bf16.  Reading back 32 x 8192 tokens of 4 heads: 78.3 us, 99 % of the rate of a plain
// copy.  Writing 8 x 8192 of 16 heads: 154 us, 671 MB at 4.4 TB/s: nothing is at its limit, HBM at 66 %, the ALU at 65 %,
// issue at 70 % (126 instructions for eight channels, most of them the exact quotients and the packing), as a warp's loads
// and its arithmetic take turns; reading those back takes 104 us.  fp32, 8 x 8192 of 16 heads of 64: written in 110 us, 612 MB
// at 5.6 TB/s, read back in 123.
#include <cuda_bf16.h>
#include <math.h>

#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace mha {
namespace {

constexpr int QC_THREADS = 256;
constexpr int QC_WARPS = QC_THREADS / 32;
// Items (8 channels) of a lane: many where there is work for every SM, few for calls whose warps would be too few.  Few |
// many, us: 3 x 1001 tokens of 8 heads of 64 in fp32 and 8 bits, written 4.8 | 5.8, read 5.3 | 7.8; 4 x 2048 of 16 heads
// in bf16 and 4 bits, written 13.2 | 10.1, read 8.2 | 6.1.
constexpr int kFewItems = 2;
template <typename T>
constexpr int kWriteItems = sizeof(T) == 2 ? 8 : 4;
constexpr int kReadItems = 8;
constexpr unsigned kFewUnits = 4096;  // warps below which a call is short
constexpr float kBf16Max = 3.3895313892515355e38f;

// A call's rows, and how the warps take them: a unit is (batch, `run` x tokens-of-a-warp tokens, head of K or V).
struct QuantCopy {
    QuantPlane pk, pv;
    int64_t ldk, ldv;
    int B, T, T_max, h_kv;
    int lanes;        // of a token: 8, 16 or 32
    Divide tiles;     // units of a head and sequence
    Divide heads;     // of keys and values together
    unsigned units;
    const int32_t *lengths, *counts;
    int* status;
};

// This lane's part of a unit.
struct QuantUnit {
    QuantPlane p;
    bool values;
    int b, head;
    int row, rows;     // first of its rows of the call, and how many the batch has
    int token;         // of the first row
    int step;          // rows from one item to the next
    int sub, c0, n;    // group, first channel, how many of the eight exist
    __device__ __forceinline__ bool has(int i) const { return row + i * step < rows; }
};

template <int RUN>
__device__ __forceinline__ bool quant_unit(const QuantCopy& c, QuantUnit& u) {
    const unsigned id = blockIdx.x * QC_WARPS + (threadIdx.x >> 5);
    if (id >= c.units) return false;
    const unsigned v = c.heads(id), hv = id - v * c.heads.by, b = c.tiles(v), tile = v - b * c.tiles.by;
    u.b = (int)b;
    u.values = hv >= (unsigned)c.h_kv;
    u.head = (int)hv - (u.values ? c.h_kv : 0);
    u.p = u.values ? c.pv : c.pk;
    const int L = __ldg(c.lengths + b), n = c.counts != nullptr ? __ldg(c.counts + b) : c.T;
    if (n < 0 || n > c.T || n > L || L > c.T_max) {
        if (tile == 0 && hv == 0 && (threadIdx.x & 31) == 0) record_status(c.status, kStatusBadLength);
        return false;
    }
    const int lane = (int)threadIdx.x & 31, in = lane & (c.lanes - 1);
    u.step = 32 / c.lanes;
    u.row = (int)tile * RUN * u.step + lane / c.lanes;
    u.rows = n;
    u.token = L - n + u.row;
    u.sub = in >> 3;
    u.c0 = 8 * in;
    u.n = max(0, min(8, u.p.d - u.c0));
    return (int)tile * RUN * u.step < n;
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

// The smallest bf16 s >= 2^-126 with N s >= hi - m.  t is below (hi - m) / N by 2^-21 of it, give or take 2^-22, so the
// step is the first or the second bf16 above t; N s is exact in fp32, and so is its difference from a number near it.
template <int N>
__device__ __forceinline__ float group_step(float hi, float m) {
    float a, e;
    two_diff(hi, m, a, e);
    const float t = __fmul_rn(a, (float)((1.0 - 1.0 / 2097152) / N));
    float s = __uint_as_float((__float_as_uint(t) & 0xffff0000u) + 0x10000u);
    if (__fsub_rn(__fmul_rn((float)N, s), a) < e) s = __uint_as_float(__float_as_uint(s) + 0x10000u);
    return a > 0.f ? fmaxf(s, 1.17549435e-38f) : 1.17549435e-38f;
}

// The code of an x whose (x - m) / s is next to k + 1/2.
__device__ __forceinline__ int code_at_border(float x, float m, float s, float k) {
    float a, e;
    two_diff(x, m, a, e);
    // both terms are exact: (k + 1/2) s has at most 17 bits, and a is near it
    const float over = __fadd_rn(__fsub_rn(a, __fmul_rn(k + 0.5f, s)), e);
    const int c = (int)k;
    return over > 0.f ? c + 1 : over < 0.f ? c : c + (c & 1);
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ float min_nan(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

__device__ __forceinline__ uint32_t bmin2(uint32_t a, uint32_t b) {  // bf16 pairs, NaN wins
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t bmax2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Eight channels of a lane as they come from memory, their minimum and maximum (NaN if any is; maxima are minima of the
// negated), and how these meet with other lanes'.
template <typename T, bool VEC>
struct Eight;

template <bool VEC>
struct Eight<__nv_bfloat16, VEC> {  // groups are whole
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p, bool any, int) {
        v = any ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
    }
    using Range = uint32_t;  // (minimum, -maximum) side by side
    __device__ __forceinline__ Range range(int) const {
        const uint32_t a = bmin2(bmin2(v.x, v.y), bmin2(v.z, v.w));
        const uint32_t b = bmax2(bmax2(v.x, v.y), bmax2(v.z, v.w)) ^ 0x80008000u;
        return bmin2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
    }
    __device__ __forceinline__ static Range meet(Range a, Range b) { return bmin2(a, b); }
    __device__ __forceinline__ static Range other(Range a, int w) { return __shfl_xor_sync(0xffffffffu, a, w); }
    __device__ __forceinline__ static float lo(Range a) { return __uint_as_float(a << 16); }
    __device__ __forceinline__ static float hi(Range a) { return -__uint_as_float(a & 0xffff0000u); }
    static constexpr bool kWhole = true;
    // the least magnitude of m and the lane's values
    __device__ __forceinline__ float least(float m) const {
        constexpr uint32_t mag = 0x7fff7fffu;
        const uint32_t a = bmin2(bmin2(v.x & mag, v.y & mag), bmin2(v.z & mag, v.w & mag));
        return fminf(fabsf(m), fminf(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u)));
    }
    __device__ __forceinline__ void values(float (&x)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

template <bool VEC>
struct Eight<float, VEC> {
    float x[8];
    __device__ __forceinline__ void load(const float* p, bool any, int n) {
        if constexpr (VEC) {  // n is 0, 4 or 8
            const float4 a = any && n > 0 ? __ldg(reinterpret_cast<const float4*>(p)) : make_float4(0.f, 0.f, 0.f, 0.f);
            const float4 b = any && n > 4 ? __ldg(reinterpret_cast<const float4*>(p) + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = any && i < n ? __ldg(p + i) : 0.f;
        }
    }
    using Range = float2;  // minimum, -maximum
    __device__ __forceinline__ Range range(int n) const {
        Range a = make_float2(INFINITY, INFINITY);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) a = make_float2(min_nan(a.x, x[i]), min_nan(a.y, -x[i]));
        return a;
    }
    __device__ __forceinline__ static Range meet(Range a, Range b) { return make_float2(min_nan(a.x, b.x), min_nan(a.y, b.y)); }
    __device__ __forceinline__ static Range other(Range a, int w) {
        return make_float2(__shfl_xor_sync(0xffffffffu, a.x, w), __shfl_xor_sync(0xffffffffu, a.y, w));
    }
    __device__ __forceinline__ static float lo(Range a) { return a.x; }
    __device__ __forceinline__ static float hi(Range a) { return -a.y; }
    static constexpr bool kWhole = false;
    __device__ __forceinline__ float least(float) const { return 0.f; }
    __device__ __forceinline__ void values(float (&y)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i];
    }
};

// What a group's codes are computed with.  inv is 1 / s to a unit in its last place; NaN: no codes (a value that is not
// finite); below zero: in halves, as differences would overflow.
struct QuantScale {
    float m, s, inv;
    uint32_t params;
};

template <int N>
__device__ __forceinline__ QuantScale group_scale(float lo, float hi) {
    QuantScale g;
    if (!(lo >= -kBf16Max && hi <= kBf16Max)) {
        g.m = 0.f;
        g.s = g.inv = NAN;
        g.params = 0x7fff7fffu;
        return g;
    }
    g.m = bf16_down(lo);
    const bool halves = hi - g.m > 3.4e38f;
    if (halves) {
        g.m *= 0.5f;
        hi *= 0.5f;
    }
    g.s = group_step<N>(hi, g.m);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(g.inv) : "f"(g.s));
    const float back = halves ? 2.f : 1.f;
    g.params = __float_as_uint(g.s * back) >> 16 | (__float_as_uint(g.m * back) & 0xffff0000u);
    if (halves) g.inv = -g.inv;
    return g;
}

// Codes of eight channels (n of them exist).
//
// q = (x - m) / s in fp32, to about half a unit in its last place: a product with 1 / s, and its remainder's.  Exact
// quotients, k + 1/2 among them, come out exact, and adding 1.5 * 2^23 rounds to the nearest whole number, ties to even.
// What is left are quotients so near to k + 1/2 that q may be on its wrong side.  Those of bf16 values need an x - m of
// more than 20 bits, for which some value (`least`) or m has to be far smaller than the range; with fp32 values any
// near one is looked at.  They are settled by exact differences.
template <int BITS, typename E>
__device__ __forceinline__ void eight_codes(const E& in, int n, float m, float s, float inv, uint32_t (&c)[BITS / 4]) {
    constexpr int N = (1 << BITS) - 1;
    constexpr float magic = 12582912.f;  // 1.5 * 2^23
    constexpr float near = BITS == 4 ? 0.5f - 1.f / 262144 : 0.5f - 1.f / 16384;  // q is off by 2^-20, 2^-16
    float x[8];
    in.values(x);
    if (!(inv > 0.f)) {  // NaN, or in halves, which changes no code
        inv = -inv;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * 0.5f != 0.f ? x[i] * 0.5f : x[i];  // (the smallest number keeps its side of 0)
    }
    if constexpr (!E::kWhole)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < n ? x[i] : m;  // code 0
    const uint64_t m2 = pack2(-m, -m), inv2 = pack2(inv, inv), step2 = pack2(-s, -s), magic2 = pack2(magic, magic);
    const uint64_t minus2 = pack2(-1.f, -1.f);
    float far = 0.f;
    uint64_t r2[4];  // the codes, negated, of channels i and i + 4
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t a = add2(pack2(x[i], x[i + 4]), m2), q0 = mul2(a, inv2);
        const uint64_t q = fma2(fma2(q0, step2, a), inv2, q0);
        r2[i] = fma2(add2(q, magic2), minus2, magic2);
        float d0, d1;
        unpack2(add2(q, r2[i]), d0, d1);
        far = fmax3(far, fabsf(d0), fabsf(d1));
    }
    if (far > near && in.least(m) < (float)N / 2048.f * s) {  // (N s is not below the range, or its half)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float r[2];
            unpack2(r2[i], r[0], r[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float v = x[i + 4 * h], q = (v - m) * inv, down = q < -r[h] ? -r[h] - 1.f : -r[h];
                if (fabsf(q - down - 0.5f) < 1.f / 4096) r[h] = -(float)code_at_border(v, m, s, down);
            }
            r2[i] = pack2(r[0], r[1]);
        }
    }
    // side by side: sums below 2^16 with 1.5 * 2^23, whose low bits they are
    auto put2 = [](uint64_t r, float at, uint64_t y) { return fma2(r, pack2(-at, -at), y); };
    float y0, y1;
    if constexpr (BITS == 4) {
        unpack2(put2(r2[3], 4096.f, put2(r2[2], 256.f, put2(r2[1], 16.f, put2(r2[0], 1.f, magic2)))), y0, y1);
        c[0] = __byte_perm(__float_as_uint(y0), __float_as_uint(y1), 0x5410);
    } else {
        float y2, y3;
        unpack2(put2(r2[1], 256.f, put2(r2[0], 1.f, magic2)), y0, y1);
        unpack2(put2(r2[3], 256.f, put2(r2[2], 1.f, magic2)), y2, y3);
        c[0] = __byte_perm(__float_as_uint(y0), __float_as_uint(y2), 0x5410);
        c[1] = __byte_perm(__float_as_uint(y1), __float_as_uint(y3), 0x5410);
    }
    if (inv != inv)
#pragma unroll
        for (int i = 0; i < BITS / 4; ++i) c[i] = 0;
}

// The group's eight lanes share the work on its scale: the ranges of their RUN items meet by halving, after which a
// lane has one item's range of the group, computes that item's scale and hands it out.  (With every lane computing
// every scale an item took 171 instructions instead of 126, and a long write 242 us instead of 153.)
template <typename T, int BITS, bool VEC, int RUN>
__global__ void __launch_bounds__(QC_THREADS, 4)  // (24 warps an SM instead of 32: 164 us of the long write, not 153)
    quant_write_kernel(const QuantCopy a, const T* __restrict__ K, const T* __restrict__ V) {
    using E = Eight<T, VEC>;
    grid_dependency_wait();
    grid_launch_dependents();
    QuantUnit u;
    if (!quant_unit<RUN>(a, u)) return;
    const int64_t ld = u.values ? a.ldv : a.ldk;
    const T* src = (u.values ? V : K) + ((int64_t)u.b * a.T + u.row) * ld + (int64_t)u.head * u.p.d + u.c0;
    E in[RUN];
#pragma unroll
    for (int i = 0; i < RUN; ++i, src += u.step * ld) in[i].load(src, u.has(i) && u.n > 0, u.n);
    const int64_t head = ((int64_t)u.b * a.h_kv + u.head) * a.T_max;
    uint8_t* codes = u.p.codes + (head + u.token) * u.p.row + u.c0 * BITS / 8;
    uint32_t* params = u.p.params + (head + u.token) * u.p.groups + u.sub;
    const bool store = u.c0 * BITS / 8 < u.p.row, param = u.sub < u.p.groups;
    const int lane = (int)threadIdx.x & 31;
    typename E::Range range[RUN];
#pragma unroll
    for (int i = 0; i < RUN; ++i) range[i] = in[i].range(u.n);
    int mine = 0;  // item whose range this lane ends up with
#pragma unroll
    for (int w = 1, left = RUN; w < 8; w <<= 1) {
        if (left > 1) {
            left /= 2;
            const bool upper = (lane & w) != 0;
            mine += upper ? left : 0;
#pragma unroll
            for (int i = 0; i < left; ++i) {
                const typename E::Range keep = upper ? range[i + left] : range[i], give = upper ? range[i] : range[i + left];
                range[i] = E::meet(keep, E::other(give, w));
            }
        } else {
            range[0] = E::meet(range[0], E::other(range[0], w));
        }
    }
    const QuantScale g = group_scale<(1 << BITS) - 1>(E::lo(range[0]), E::hi(range[0]));
    if (param && (lane & 7) < RUN && u.has(mine)) params[mine * u.step * u.p.groups] = g.params;
#pragma unroll
    for (int i = 0; i < RUN; ++i, codes += u.step * u.p.row) {
        // the lane of the eight that has item i: its bits from the highest on
        const int from = (lane & 24) | (RUN == 8 ? (i >> 2 & 1) | (i & 2) | (i << 2 & 4) : RUN == 4 ? (i >> 1 & 1) | (i << 1 & 2) : i);
        const float m = __shfl_sync(0xffffffffu, g.m, from), s = __shfl_sync(0xffffffffu, g.s, from),
                    inv = __shfl_sync(0xffffffffu, g.inv, from);
        if (!u.has(i) || !store) continue;
        uint32_t c[BITS / 4];
        eight_codes<BITS>(in[i], u.n, m, s, inv, c);
        if constexpr (BITS == 4) *reinterpret_cast<uint32_t*>(codes) = c[0];
        else *reinterpret_cast<uint2*>(codes) = make_uint2(c[0], c[1]);
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16* p, int, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                              pack_bf16x2(x[6], x[7]));
}

template <bool VEC>
__device__ __forceinline__ void store8(float* p, int n, const float (&x)[8]) {
    if constexpr (VEC) {
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
        if (n > 4) *(reinterpret_cast<float4*>(p) + 1) = make_float4(x[4], x[5], x[6], x[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = x[i];
    }
}

template <typename T, int BITS, bool VEC, int RUN>
__global__ void __launch_bounds__(QC_THREADS)
    quant_read_kernel(const QuantCopy a, T* __restrict__ K, T* __restrict__ V) {
    grid_dependency_wait();
    grid_launch_dependents();
    QuantUnit u;
    if (!quant_unit<RUN>(a, u) || u.n <= 0) return;
    const int64_t ld = u.values ? a.ldv : a.ldk;
    T* dst = (u.values ? V : K) + ((int64_t)u.b * a.T + u.row) * ld + (int64_t)u.head * u.p.d + u.c0;
    const int64_t head = ((int64_t)u.b * a.h_kv + u.head) * a.T_max;
    const uint8_t* codes = u.p.codes + (head + u.token) * u.p.row + u.c0 * BITS / 8;
    const uint32_t* params = u.p.params + (head + u.token) * u.p.groups + u.sub;
    uint32_t c[RUN][BITS / 4], par[RUN];
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
        if (!u.has(i)) continue;
        const uint8_t* from = codes + i * u.step * u.p.row;
        if constexpr (BITS == 4) {
            c[i][0] = __ldg(reinterpret_cast<const uint32_t*>(from));
        } else {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(from));
            c[i][0] = w.x;
            c[i][1] = w.y;
        }
        par[i] = __ldg(params + i * u.step * u.p.groups);
    }
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
        if (!u.has(i)) continue;
        const float s = quant_step(par[i]), m = quant_lowest(par[i]);
        const uint64_t s2 = pack2(s, s), m2 = pack2(m, m), base2 = pack2(-8388608.f, -8388608.f);
        // bytes as fp32 numbers of 2^23 and more
        uint32_t by[2];
        if constexpr (BITS == 4) by[0] = c[i][0] & 0x0f0f0f0fu, by[1] = c[i][0] >> 4 & 0x0f0f0f0fu;
        else by[0] = c[i][0], by[1] = c[i][1];
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            uint32_t f0, f1;
            if constexpr (BITS == 4) {
                f0 = __byte_perm(by[0], 0x4b000000u, 0x7440 | (j / 2));
                f1 = __byte_perm(by[1], 0x4b000000u, 0x7440 | (j / 2));
            } else {
                f0 = __byte_perm(by[j / 4], 0x4b000000u, 0x7440 | (j & 3));
                f1 = __byte_perm(by[j / 4], 0x4b000000u, 0x7440 | ((j + 1) & 3));
            }
            const uint64_t code = add2(pack2(__uint_as_float(f0), __uint_as_float(f1)), base2);
            unpack2(fma2(code, s2, m2), x[j], x[j + 1]);  // s code is exact
        }
        store8<VEC>(dst + i * u.step * ld, u.n, x);
    }
}

bool vec_ok(const QuantPlane& p, const void* x, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(x) & 15) == 0 && ld % 4 == 0 && p.d % 4 == 0;
}

}  // namespace

// Units of a call with `items` items a lane; 0: more than a grid takes.
unsigned quant_copy_units(int items, const QuantPlane& pk, const QuantPlane& pv, int B, int T, int h_kv, int* lanes,
                          unsigned* tiles) {
    const int groups = pk.groups > pv.groups ? pk.groups : pv.groups;
    *lanes = groups == 1 ? 8 : groups == 2 ? 16 : 32;
    const int tokens = 32 / *lanes * items;
    *tiles = (unsigned)(((int64_t)T + tokens - 1) / tokens);
    const double units = (double)B * *tiles * 2.0 * h_kv;
    return units > (double)INT32_MAX ? 0u : (unsigned)units;
}

int most_items(bool write, bool f32) { return !write ? kReadItems : f32 ? kWriteItems<float> : kWriteItems<__nv_bfloat16>; }

bool quant_copy_fits(bool write, bool f32, const QuantPlane& pk, const QuantPlane& pv, int B, int T, int h_kv) {
    int lanes;
    unsigned tiles;
    return quant_copy_units(most_items(write, f32), pk, pv, B, T, h_kv, &lanes, &tiles) > 0;
}

cudaError_t launch_quant_copy(bool write, bool f32, int bits, const QuantPlane& pk, const QuantPlane& pv, void* K,
                              int64_t ldk, void* V, int64_t ldv, int B, int T, int T_max, int h_kv,
                              const int32_t* lengths, const int32_t* counts, int* status, cudaStream_t stream) {
    QuantCopy a;
    a.pk = pk;
    a.pv = pv;
    a.ldk = ldk;
    a.ldv = ldv;
    a.B = B;
    a.T = T;
    a.T_max = T_max;
    a.h_kv = h_kv;
    unsigned tiles;
    int items = most_items(write, f32);
    a.units = quant_copy_units(items, pk, pv, B, T, h_kv, &a.lanes, &tiles);
    const bool few = a.units < kFewUnits;
    if (few) a.units = quant_copy_units(kFewItems, pk, pv, B, T, h_kv, &a.lanes, &tiles);
    if (a.units == 0) return cudaErrorInvalidValue;
    a.tiles = Divide(tiles);
    a.heads = Divide(2u * (unsigned)h_kv);
    a.lengths = lengths;
    a.counts = counts;
    a.status = status;
    const dim3 grid((a.units + QC_WARPS - 1) / QC_WARPS);
    const bool vec = !f32 || (vec_ok(pk, K, ldk) && vec_ok(pv, V, ldv));
    auto go = [&](auto* x, auto kw, auto kr) {
        using T_ = std::remove_pointer_t<decltype(x)>;
        if (write)
            return launch_pdl(kw, grid, dim3(QC_THREADS), 0, stream, a, static_cast<const T_*>(K), static_cast<const T_*>(V));
        return launch_pdl(kr, grid, dim3(QC_THREADS), 0, stream, a, static_cast<T_*>(K), static_cast<T_*>(V));
    };
#define MHA_QC(T, BITS, VEC)                                                                                        \
    if (f32 == std::is_same_v<T, float> && bits == BITS && vec == VEC) {                                              \
        T* x = nullptr;                                                                                              \
        return few ? go(x, quant_write_kernel<T, BITS, VEC, kFewItems>, quant_read_kernel<T, BITS, VEC, kFewItems>)    \
                   : go(x, quant_write_kernel<T, BITS, VEC, kWriteItems<T>>, quant_read_kernel<T, BITS, VEC, kReadItems>); \
    }
    MHA_QC(__nv_bfloat16, 4, true)
    MHA_QC(__nv_bfloat16, 8, true)
    MHA_QC(float, 4, true)
    MHA_QC(float, 8, true)
    MHA_QC(float, 4, false)
    MHA_QC(float, 8, false)
#undef MHA_QC
    return cudaErrorInvalidValue;
}

}  // namespace mha
