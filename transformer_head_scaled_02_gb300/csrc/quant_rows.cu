// quant_rows.cu -- a step of many query rows over a quantised cache (quant.cuh), bf16 layers with heads of 64 and 128
// channels, on tcgen05: speculative tokens behind grouped heads, a prompt's next piece.
//
// The arithmetic is quant_mma.cu's: with codes as (subnormal) fp16 numbers, steps s, lowest values m and 64-channel
// groups G
//   score_j = sum_G s_jG (q_G . code_jG) + m_jG (sum of q_G)
//   o       = sum_j (p_j s_jG) code_j + sum_j p_j m_jG
// Here up to 128 query rows are the M side, so that a tile's codes are unpacked once for all of them (quant_mma.cu
// unpacks them once for every 8 or 16 rows).  Every group has its own score accumulator and its own operand p s:
//   S_G (128 x 128) = Q_G K_G^T          O_G (128 x 64) += P_G V_G
// with S, P and O in tensor memory (2 x 128 + 2 x 64 + 128 columns for 128 channels: all of it).
//
// Warps 0-3 unpack: codes from global memory, a tile ahead in registers, as fp16 into swizzled tiles of shared memory
// (two of keys and two of values), with the tokens' steps and lowest values beside them.  Warps 4-11: softmax, two threads
// a row, which halve its tokens and agree on its maximum through shared memory (with one thread a row its 128 scores did
// not fit the registers).  Warp 12: products.  Tiles are quanta of 128 tokens; pieces follow one another with a barrier
// between.
//
// Measured, 4 bits: 512 new tokens of one sequence of 8192, 16 query heads over 4 of 128: 145 us, 21 of them the join,
// 237 TFLOP/s (quant_mma.cu 218); 128 new tokens of each of 4 ragged sequences of up to 4096, 16 heads over 4 of 64: 50 us
// (64).  Nothing is at its limit: a tile of 128 channels takes 8700 cycles, of which its instructions need 3800 to be issued
// and the tensor core is busy for 1000.  The rest is the chain of a tile: scores, maximum, the two warps' meeting, the wait
// for the tile before's product, exponentials, P, product.
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "quant.cuh"
#include "quant_meet.cuh"

namespace mha {
namespace {

constexpr int QR_THREADS = 416;
constexpr int QR_MMA_WARP = 12;
constexpr int QR_SOFTMAX = 256;  // threads
constexpr int QR_ROWS = 128;
constexpr int QR_SUMS = 16;    // tiles after which long pieces' sums are moved
constexpr int QR_PARAMS = 4;  // tiles whose parameters are kept: a tile's are read until its values are asked for
constexpr float kRowsNone = -3e38f;

template <int BITS, int D>
struct QrCfg {
    static constexpr int G = D / kQuantGroup;
    static constexpr int CHUNK = 128 * 128;             // 128 rows of 64 fp16
    static constexpr int TILE = G * CHUNK;
    static constexpr int ROW = D * BITS / 8;
    static constexpr int LOADS = 128 * ROW / 16 / 128;  // 16-byte pieces of a tile per unpacking thread
    static constexpr int Q = 0, K = TILE, V = 3 * TILE;
    static constexpr int KP = 5 * TILE, VP = KP + QR_PARAMS * 128 * 16;
    static constexpr int TOP = VP + QR_PARAMS * 128 * 16;    // largest value step of a tile, per unpacking warp
    static constexpr int QS = TOP + QR_PARAMS * 16;          // per row: sums of q per group, score factor
    static constexpr int XM = QS + QR_ROWS * (G + 1) * 4;    // a row's maxima, by tile parity and half; at the end its sums
    static constexpr int MS = XM + 2 * 2 * QR_ROWS * 4 * 2;  // a softmax thread's reference that its moved sums go by
    static constexpr int BARS = MS + QR_SOFTMAX * 4;
    static constexpr int SMEM = BARS + 17 * 8 + 16 + 1024;
    static constexpr int OUT = D + 3;                        // floats of a row of results (odd: rows in other banks)
    static_assert(QR_ROWS * OUT * 4 <= 4 * TILE, "the results fit the key and value tiles");
    static constexpr uint32_t COLS = D == 64 ? 256 : 512;
    static constexpr uint32_t S_COL = 0, O_COL = 128 * G, P_COL = O_COL + D;  // P_G at P_COL + 64 G
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(P_COL + 64 * G <= COLS, "tensor memory");
};

// Eight channels of a word (4 bits) or two (8 bits) as fp16, in the order channel_of() names; odd positions of 4 bits
// count 16 times as much.
template <int BITS>
__device__ __forceinline__ uint4 eight_halves(uint32_t w0, uint32_t w1) {
    if constexpr (BITS == 4) return make_uint4(w0 & 0x000f000fu, w0 & 0x00f000f0u, w0 >> 8 & 0x000f000fu, w0 >> 8 & 0x00f000f0u);
    return make_uint4(w0 & 0x00ff00ffu, w0 >> 8 & 0x00ff00ffu, w1 & 0x00ff00ffu, w1 >> 8 & 0x00ff00ffu);
}
template <int BITS>
__host__ __device__ constexpr int channel_of(int p) {  // of eight positions
    return BITS == 4 ? (p >> 1) + 4 * (p & 1) : (p & 4) + (p >> 1 & 1) + 2 * (p & 1);
}
template <int BITS>
__host__ __device__ constexpr float unit_of(int p) {
    return BITS == 4 && (p >> 1 & 1) ? 16.f * 5.9604644775390625e-8f : 5.9604644775390625e-8f;
}

// 16 columns of tensor memory.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Where a softmax thread's sums are: [channel][row] for each CTA, behind the records.
template <int D>
__device__ __forceinline__ float* moved_sums(const QuantStep& s, float* part, int half, int r) {
    return part + s.slot((int)gridDim.x, 0, 0) + ((int64_t)blockIdx.x * D + half * (D / 2)) * QR_ROWS + r;
}

// A row's sums of QR_SUMS tiles, half of its channels, go from tensor memory there: as values, added to f times what
// is there, or the first ones.  inv: 1 / vs.
template <int BITS, int D>
__device__ __forceinline__ void move_sums(uint32_t taddr, float* sums, bool first, float f, float inv) {
#pragma unroll 1
    for (int c = 0; c < D / 2; c += 32, sums += 32 * QR_ROWS) {
        uint32_t o[32];
        tmem_ld32(taddr + c, o);
        tmem_wait_ld();
        reg_fence(o);
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
            float old[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) old[k] = first ? 0.f : sums[(e + k) * QR_ROWS];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                sums[(e + k) * QR_ROWS] = fmaf(__uint_as_float(o[e + k]) * (1.f / unit_of<BITS>(k)), inv, f * old[k]);
        }
    }
}

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// LONG: the sums go to memory every QR_SUMS tiles, where they are added in fp32, as the tensor core cuts off what its sums
// cannot hold, always towards zero (2.8e-8 of a sum of codes with each of a tile's eight products).  For pieces of more than
// kQuantRowsLong tokens: 8 rows of a head over 20 x 32768 tokens of values around zero were off by 2.6 % at 4 bits and 3.7 %
// at 8, of which bf16's rounding is 0.17 %, and are by 0.19 and 0.29 %; it takes 5 % longer (1182 us | 1238).
template <int BITS, int D, bool LONG>
__global__ void __launch_bounds__(QR_THREADS, 1)
    quant_rows_kernel(const QuantStep s, const QuantPlane pk, const QuantPlane pv, const __nv_bfloat16* __restrict__ Q, int64_t ldq,
                      __nv_bfloat16* __restrict__ O, int64_t ldo, const int32_t* __restrict__ lengths, float scale_log2,
                      float* __restrict__ part, int* status) {
    using C = QrCfg<BITS, D>;
    constexpr int G = C::G;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t* sm = smem_raw + (base - raw);
    const uint32_t bars = base + C::BARS;
    const uint32_t k_full = bars, k_empty = bars + 16, v_full = bars + 32, v_empty = bars + 48;  // two each
    const uint32_t s_full = bars + 64, s_free = bars + 72, p_full = bars + 80, pv_done = bars + 88, drain = bars + 96, pair = bars + 104;  // four
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::BARS + 136);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(k_full + 8u * i, 128);
            mbar_init(k_empty + 8u * i, 1);
            mbar_init(v_full + 8u * i, 128);
            mbar_init(v_empty + 8u * i, 1);
        }
        mbar_init(s_full, 2);
        mbar_init(s_free, QR_SOFTMAX);
        mbar_init(p_full, QR_SOFTMAX);
        mbar_init(pv_done, 1);
        mbar_init(drain, 1);
        for (int i = 0; i < 4; ++i) mbar_init(pair + 8u * i, 64);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == QR_MMA_WARP) {
        tmem_alloc(smem_u32(tmem_slot), C::COLS);
        tmem_relinquish();
    }
    grid_dependency_wait();
    grid_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const QuantPlan plan = quant_plan(s, lengths);
    if (plan.bad) quant_invalid<QR_THREADS>(s, (int)blockIdx.x, (int)gridDim.x, lengths, O, ldo, status);
    const int end = plan.first(s, (int)blockIdx.x + 1);
    int n0 = 0;  // tiles before this piece
    uint32_t meets = 0;  // of a softmax warp with the other one of its rows
#pragma unroll 1
    for (int q_at = plan.first(s, (int)blockIdx.x); q_at < end;) {
        const QuantPiece z = quant_piece(s, lengths, plan, q_at, end);
        q_at = z.next;
        const int b = z.b, g = s.by_nrb((uint32_t)z.lane), L = z.L, k0 = z.k0(), k1 = z.k1();
        const int r0 = (z.lane - g * s.nrb) * QR_ROWS, nr = min(QR_ROWS, s.rows - r0);
        const int n_tiles = (k1 - k0 + 127) / 128;
        // ---------------- the first tile's codes are asked for before anything else
        const int64_t head = ((int64_t)b * s.h_kv + g) * s.T_max;
        uint4 kc[C::LOADS], vc[C::LOADS];
        uint32_t kp[G], vp[G];
        auto load = [&](const QuantPlane& p, int key0, uint4 (&c)[C::LOADS], uint32_t (&par)[G]) {
#pragma unroll
            for (int i = 0; i < C::LOADS; ++i) {
                const int at = tid + 128 * i, token = min(key0 + at / (C::ROW / 16), s.T_max - 1);
                c[i] = __ldg(reinterpret_cast<const uint4*>(p.codes + (head + token) * C::ROW) + at % (C::ROW / 16));
            }
            const int token = min(key0 + tid, s.T_max - 1);
#pragma unroll
            for (int u = 0; u < G; ++u) par[u] = __ldg(p.params + (head + token) * G + u);
        };
        if (warp < 4) {
            load(pk, k0, kc, kp);
            load(pv, k0, vc, vp);
        }
        // ---------------- queries: eight lanes a row, 16 bytes (8 channels) at a time; rows past nr keep what they had (rows
        // do not meet, and theirs go nowhere).  Rolled: code that runs once is paid for in instruction fetches, and a warp
        // per row with eleven rows unrolled took 10000 cycles.
        if (warp < 12) {
            const int in = lane & 7;
#pragma unroll 1
            for (int r = 4 * warp + (lane >> 3); r < ((nr + 3) & ~3); r += 48) {
                const int rr = r0 + min(r, nr - 1), hg = s.by_T_q((uint32_t)rr), t = rr - hg * s.T_q;
                const uint4* src = reinterpret_cast<const uint4*>(Q + ((int64_t)b * s.T_q + t) * ldq + (int64_t)(g * s.per + hg) * D) + in;
                uint4 v[G];
                float top = 0.f;
#pragma unroll
                for (int u = 0; u < G; ++u) v[u] = src[8 * u];
#pragma unroll
                for (int u = 0; u < G; ++u) {
                    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        top = fmax3(top, fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u)));
                }
                const unsigned lanes = 0xffu << (lane & 24);
#pragma unroll
                for (int o = 4; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(lanes, top, o));
                // the largest element to [2^13, 2^14); zero, infinite, tiny and huge (2^118) rows as far as powers of two go
                const int e2 = top > 0.f && top < INFINITY ? max(-104, min(126, 13 - quant_exponent(top))) : 0;
                const float f = quant_power2(e2);
                float sum[G];
#pragma unroll
                for (int u = 0; u < G; ++u) {
                    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
                    float x[8];
                    sum[u] = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[2 * e] = f * __uint_as_float(w[e] << 16);
                        x[2 * e + 1] = f * __uint_as_float(w[e] & 0xffff0000u);
                        sum[u] += x[2 * e] + x[2 * e + 1];
                    }
                    uint32_t h[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        constexpr float u0 = unit_of<BITS>(0);
                        h[e] = half2_of(x[channel_of<BITS>(2 * e)] * (u0 / unit_of<BITS>(2 * e)),
                                        x[channel_of<BITS>(2 * e + 1)] * (u0 / unit_of<BITS>(2 * e + 1)));
                    }
                    if (r < nr) st_shared_v4(base + C::Q + (uint32_t)(u * C::CHUNK + r * 128 + ((in ^ (r & 7)) << 4)), h[0], h[1], h[2], h[3]);
#pragma unroll
                    for (int o = 4; o >= 1; o >>= 1) sum[u] += __shfl_xor_sync(lanes, sum[u], o);
                }
                if (in == 0 && r < nr) {
                    float* qv = reinterpret_cast<float*>(sm + C::QS) + r * (G + 1);
#pragma unroll
                    for (int u = 0; u < G; ++u) qv[u] = sum[u] * unit_of<BITS>(0);
                    qv[G] = scale_log2 / unit_of<BITS>(0) * quant_power2(-e2);
                }
            }
            fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp < 4) {
            // ---------------- unpacking
            // a tile's codes into its swizzled place; tokens at or past the length get steps and lowest values of zero
            auto store = [&](uint32_t tile, const uint4 (&c)[C::LOADS]) {
#pragma unroll
                for (int i = 0; i < C::LOADS; ++i) {
                    const int at = tid + 128 * i, row = at / (C::ROW / 16), ch = at % (C::ROW / 16) * (128 / BITS);
                    const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
                    for (int j = 0; j < 16 / BITS; ++j) {
                        const uint4 h = BITS == 4 ? eight_halves<BITS>(w[j], 0) : eight_halves<BITS>(w[2 * j & 3], w[2 * j + 1 & 3]);
                        const int cc = ch + 8 * j;
                        st_shared_v4(tile + (uint32_t)((cc >> 6) * C::CHUNK + row * 128 + (((cc >> 3 & 7) ^ (row & 7)) << 4)), h.x, h.y, h.z, h.w);
                    }
                }
            };
            auto floats = [&](const uint32_t (&par)[G], bool live) {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (live) {
                    x.x = quant_step(par[0]);
                    x.y = quant_lowest(par[0]);
                    if constexpr (G > 1) x.z = quant_step(par[G - 1]), x.w = quant_lowest(par[G - 1]);
                }
                return x;
            };
#pragma unroll 1
            for (int i = 0; i < n_tiles; ++i) {
                const int n = n0 + i, key0 = k0 + 128 * i;
                const uint32_t st = (uint32_t)n & 1u, ph = ((uint32_t)(n >> 1) & 1u) ^ 1u;
                const bool live = key0 + tid < L;
                if (!__all_sync(0xffffffffu, mbar_wait(k_empty + 8u * st, ph, abort_flag, status))) break;
                store(base + C::K + st * C::TILE, kc);
                reinterpret_cast<float4*>(sm + C::KP)[(n % QR_PARAMS) * 128 + tid] = floats(kp, live);
                fence_proxy_async_smem();
                mbar_arrive(k_full + 8u * st);
                if (i + 1 < n_tiles) load(pk, key0 + 128, kc, kp);
                if (!__all_sync(0xffffffffu, mbar_wait(v_empty + 8u * st, ph, abort_flag, status))) break;
                store(base + C::V + st * C::TILE, vc);
                const float4 par = floats(vp, live);
                reinterpret_cast<float4*>(sm + C::VP)[(n % QR_PARAMS) * 128 + tid] = par;
                float top = fmaxf(par.x, par.z);
#pragma unroll
                for (int w = 16; w >= 1; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                if (lane == 0) reinterpret_cast<float*>(sm + C::TOP)[(n % QR_PARAMS) * 4 + warp] = top;
                fence_proxy_async_smem();
                mbar_arrive(v_full + 8u * st);
                if (i + 1 < n_tiles) load(pv, key0 + 128, vc, vp);
            }
        } else if (warp == QR_MMA_WARP) {
            if (lane == 0) {
                // ---------------- products
                const uint32_t idesc_s = idesc_f16_f32(128, 128, false, false), idesc_o = idesc_f16_f32(128, 64, false, true);
                const uint64_t qd = sdesc_sw128(base + C::Q, 16, 1024), kd0 = sdesc_sw128(base + C::K, 16, 1024),
                               vd0 = sdesc_sw128(base + C::V, C::CHUNK, 1024);
                auto scores = [&](int i) -> bool {
                    const int n = n0 + i;
                    const uint32_t st = (uint32_t)n & 1u;
                    if (!mbar_wait(k_full + 8u * st, (uint32_t)(n >> 1) & 1u, abort_flag, status)) return false;
                    if (n > 0 && !mbar_wait(s_free, (uint32_t)(n - 1) & 1u, abort_flag, status)) return false;
                    mbar_arrive(s_full);  // the keys' parameters are there (its other arrival: the products)
                    tc_fence_after();
                    const uint64_t kd = kd0 + (uint64_t)((st * C::TILE) >> 4);
#pragma unroll
                    for (int u = 0; u < G; ++u)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint32_t off = (uint32_t)((u * C::CHUNK + kk * 32) >> 4);
                            mma_bf16_ss(tmem + C::S_COL + 128 * u, qd + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
                        }
                    tc_commit(s_full);
                    tc_commit(k_empty + 8u * st);
                    return true;
                };
                bool ok = scores(0);
#pragma unroll 1
                for (int i = 0; i < n_tiles && ok; ++i) {
                    if (i + 1 < n_tiles) ok = scores(i + 1);
                    if (!ok) break;
                    const int n = n0 + i;
                    const uint32_t st = (uint32_t)n & 1u;
                    ok = mbar_wait(v_full + 8u * st, (uint32_t)(n >> 1) & 1u, abort_flag, status) &&
                         mbar_wait(p_full, (uint32_t)n & 1u, abort_flag, status);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t vd = vd0 + (uint64_t)((st * C::TILE) >> 4);
#pragma unroll
                    for (int u = 0; u < G; ++u)
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            mma_bf16_ts(tmem + C::O_COL + 64 * u, tmem + C::P_COL + 64 * u + kk * 8,
                                        vd + (uint64_t)((u * C::CHUNK + kk * 2048) >> 4), idesc_o,
                                        ((LONG ? i % QR_SUMS : i) > 0 || kk > 0) ? 1u : 0u);
                    tc_commit(pv_done);
                    tc_commit(v_empty + 8u * st);
                }
            }
        } else {
            // ---------------- softmax: two threads a query row, 64 of a tile's tokens each
            const int half = (warp - 4) >> 2, r = (warp & 3) * 32 + lane, c0 = 64 * half;
            const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
            const bool idle = 32 * (warp & 3) >= nr;  // no real row in the warp: it only keeps the others going
            const int rr = r0 + min(r, nr - 1);
            const int lim = L - s.T_q + rr - s.by_T_q((uint32_t)rr) * s.T_q + 1;  // tokens before it are visible
            const float* qv = reinterpret_cast<const float*>(sm + C::QS) + r * (G + 1);
            float* xm = reinterpret_cast<float*>(sm + C::XM);
            // the row's two warps (bounded like every wait: they may not both have got here)
            auto meet = [&]() -> bool {
                const uint32_t bar = pair + 8u * (uint32_t)(warp & 3);
                __syncwarp();
                mbar_arrive(bar);
                const bool fine = __all_sync(0xffffffffu, mbar_wait(bar, meets & 1u, abort_flag, status));
                ++meets;
                return fine;
            };
            float qs[G], om[G], m = kRowsNone, l = 0.f, vs = quant_power2(kQuantScaleMost);
#pragma unroll
            for (int u = 0; u < G; ++u) qs[u] = qv[u], om[u] = 0.f;
            const float rs = qv[G];
            bool ok = true;
#pragma unroll 1
            for (int i = 0; i < n_tiles && ok; ++i) {
                const int n = n0 + i, key0 = k0 + 128 * i + c0;
                if (LONG && i > 0 && i % QR_SUMS == 0) {
                    ok = __all_sync(0xffffffffu, mbar_wait(pv_done, (uint32_t)(n - 1) & 1u, abort_flag, status));
                    if (!ok) break;
                    tc_fence_after();
                    if (!idle) {
                        volatile float* m_sums = reinterpret_cast<float*>(sm + C::MS) + half * QR_ROWS + r;
                        const bool first = i == QR_SUMS;
                        move_sums<BITS, D>(trow + C::O_COL + half * (D / 2), moved_sums<D>(s, part, half, r), first,
                                           first ? 0.f : ex2_approx(*m_sums - m), 1.f / vs);
                        *m_sums = m;
                    }
                }
                const uint32_t st = (uint32_t)n & 1u, ph = (uint32_t)(n >> 1) & 1u;
                // (Not k_full: the tile after the next may be there before a late warp asks, and the barrier's parity be this
                // one's again.  Every other barrier's next phase but one waits for those who wait for this one.)
                ok = __all_sync(0xffffffffu, mbar_wait(s_full, (uint32_t)n & 1u, abort_flag, status));
                if (!ok) break;
                tc_fence_after();
                float y[64], top = -INFINITY;
                if (!idle) {
                    const float4* par = reinterpret_cast<const float4*>(sm + C::KP) + (n % QR_PARAMS) * 128 + c0;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t a[G][32];
#pragma unroll
                        for (int u = 0; u < G; ++u) tmem_ld32(trow + C::S_COL + 128 * u + c0 + 32 * c, a[u]);
                        tmem_wait_ld();
#pragma unroll
                        for (int u = 0; u < G; ++u) reg_fence(a[u]);
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float4 p = par[32 * c + e];
                            float x = fmaf(p.x, __uint_as_float(a[0][e]), p.y * qs[0]);
                            if constexpr (G > 1) x = fmaf(p.z, __uint_as_float(a[G - 1][e]), fmaf(p.w, qs[G - 1], x));
                            y[32 * c + e] = x * rs;
                        }
                    }
                    if (key0 + 64 > lim)
#pragma unroll
                        for (int c = 0; c < 64; ++c) y[c] = key0 + c < lim ? y[c] : -INFINITY;
#pragma unroll
                    for (int c = 0; c < 64; c += 2) top = fmax3(top, y[c], y[c + 1]);
                }
                tc_fence_before();
                mbar_arrive(s_free);
                ok = __all_sync(0xffffffffu, mbar_wait(v_full + 8u * st, ph, abort_flag, status));  // steps of the values
                // The reference moves when a score exceeds it by 2^8; p s is held as p s vs (quant_meet.cuh).
                float alpha = 1.f, back = 1.f;
                bool moved = false;
                if (!idle) {  // (both warps of a row are, or neither)
                    float* mine = xm + (n & 1) * 2 * QR_ROWS;
                    mine[half * QR_ROWS + r] = top;
                    if (!meet()) break;
                    top = fmaxf(top, mine[(1 - half) * QR_ROWS + r]);
                    if (top - m > 8.f) {  // (m + 8, rounded, could be 2^16 in a weight)
                        alpha = ex2_approx(m - top);
                        m = top;
                        moved = true;
                    }
                    const float4 w = *reinterpret_cast<const float4*>(sm + C::TOP + (n % QR_PARAMS) * 16);
                    // (rows past nr have queries of some earlier block, and no say in when the others' scales follow)
                    moved = (moved || fmaxf(fmaxf(w.x, w.y), fmaxf(w.z, w.w)) * vs > kQuantStepMost) && r < nr;
                    if (__any_sync(0xffffffffu, moved)) {  // (so says the row's other warp)
                        const uint32_t par = base + C::VP + (uint32_t)(((n % QR_PARAMS) * 128 + c0) * 16);
                        float need = 0.f;
#pragma unroll
                        for (int c = 0; c < 64; ++c) {
                            float s0, s1 = 0.f;  // (in order: 64 loads ahead would take the registers of y)
                            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s0) : "r"(par + 16u * c) : "memory");
                            if constexpr (G > 1) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s1) : "r"(par + 16u * c + 8u) : "memory");
                            need = fmaxf(need, ex2_approx(y[c] - m) * fmaxf(s0, s1));
                        }
                        mine += 4 * QR_ROWS;
                        mine[half * QR_ROWS + r] = need;
                        if (!meet()) break;
                        need = fmaxf(need, mine[(1 - half) * QR_ROWS + r]);
                        const float to = quant_move_scale(vs, need, alpha, -quant_exponent(alpha));  // (what alpha <= 2^-8 takes away, and less than one more)
                        back = quant_rescale(to, vs, alpha);
                        vs = to;
                    }
                }
                if (!ok) break;
                if (n > 0) {
                    ok = __all_sync(0xffffffffu, mbar_wait(pv_done, (uint32_t)(n - 1) & 1u, abort_flag, status));
                    if (!ok) break;
                }
                tc_fence_after();
                if (!idle) {
                    if ((LONG ? i % QR_SUMS : i) > 0 && __any_sync(0xffffffffu, moved)) {  // each of the two warps half of the columns
                        #pragma unroll
                        for (int c = 0; c < D / 64; ++c) {
                            uint32_t o[32];
                            tmem_ld32(trow + C::O_COL + half * (D / 2) + 32 * c, o);
                            tmem_wait_ld();
                            reg_fence(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * back);
                            tmem_st32(trow + C::O_COL + half * (D / 2) + 32 * c, o);
                        }
                    }
                    l *= alpha;
#pragma unroll
                    for (int u = 0; u < G; ++u) om[u] *= alpha;
                    const float4* par = reinterpret_cast<const float4*>(sm + C::VP) + (n % QR_PARAMS) * 128 + c0;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t w[G][16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float x[G][2];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const float4 q = par[32 * c + 2 * e + h];
                                const float p = ex2_approx(y[32 * c + 2 * e + h] - m), pw = p * vs;
                                l += p;
                                om[0] = fmaf(p, q.y, om[0]);
                                x[0][h] = pw * q.x;
                                if constexpr (G > 1) {
                                    om[G - 1] = fmaf(p, q.w, om[G - 1]);
                                    x[G - 1][h] = pw * q.z;
                                }
                            }
#pragma unroll
                            for (int u = 0; u < G; ++u) w[u][e] = half2_of(x[u][0], x[u][1]);
                        }
#pragma unroll
                        for (int u = 0; u < G; ++u) tmem_st16(trow + C::P_COL + 64 * u + 32 * half + 16 * c, w[u]);
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                mbar_arrive(p_full);
            }
            if (ok && __all_sync(0xffffffffu, mbar_wait(pv_done, (uint32_t)(n0 + n_tiles - 1) & 1u, abort_flag, status)) && !idle) {
                tc_fence_after();
                // the halves' sums meet; each warp then has half of the channels
                ok = meet();  // (the last maxima are read)
                float* mine = xm + (half * QR_ROWS + r) * 4;
                mine[0] = l;
#pragma unroll
                for (int u = 0; u < G; ++u) mine[1 + u] = om[u];
                ok = meet() && ok;
                const float* other = xm + ((1 - half) * QR_ROWS + r) * 4;
                l += other[0];
#pragma unroll
                for (int u = 0; u < G; ++u) om[u] += other[1 + u];
                // every key and value tile is used: the rows meet there, to be written as rows
                float* row = reinterpret_cast<float*>(sm + C::K) + r * C::OUT;
                const float inv = z.whole() ? 1.f / l : 1.f, back = 1.f / vs;  // (vs goes down to 2^-126: 2^24 / vs may be infinite)
                const bool moved = LONG && n_tiles > QR_SUMS;
                const float f_sums = moved ? ex2_approx(reinterpret_cast<const float*>(sm + C::MS)[half * QR_ROWS + r] - m) : 0.f;
                const float* sums = moved_sums<D>(s, part, half, r);
                if (half == 0) row[0] = m, row[1] = l;
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const int col = half * (D / 2) + 32 * c;
                    const float z0 = G == 1 || half == 0 ? om[0] : om[G - 1];  // 64 channels: both halves in one group
                    uint32_t o[32];
                    tmem_ld32(trow + C::O_COL + col, o);
                    tmem_wait_ld();
                    reg_fence(o);
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
#pragma unroll
                        for (int p = 0; p < 8; ++p) {
                            const float before = moved ? fmaf(f_sums, sums[(32 * c + e + p) * QR_ROWS], z0) : z0;
                            row[2 + col + e + channel_of<BITS>(p)] =
                                inv * fmaf(__uint_as_float(o[e + p]) * (1.f / unit_of<BITS>(p)), back, before);
                        }
                }
            }
        }
        __syncwarp();
        __syncthreads();
        {
            const float* rows = reinterpret_cast<const float*>(sm + C::K);
            float* rec = part + s.slot((int)blockIdx.x, z.q0 == 0 ? 1 : 0, 0);
            if (z.whole()) {
                for (int e = tid; e < nr * (D / 2); e += QR_THREADS) {
                    const int r = e / (D / 2), c = 2 * (e % (D / 2));
                    *reinterpret_cast<uint32_t*>(quant_out(s, O, ldo, b, g, r0 + r) + c) = pack_bf16x2(rows[r * C::OUT + 2 + c], rows[r * C::OUT + 3 + c]);
                }
            } else {
                for (int e = tid; e < nr * (D / 2 + 1); e += QR_THREADS) {
                    const int r = e / (D / 2 + 1), c = 2 * (e % (D / 2 + 1));
                    *reinterpret_cast<float2*>(rec + r * (D + 2) + c) = make_float2(rows[r * C::OUT + c], rows[r * C::OUT + c + 1]);
                }
            }
        }
        n0 += n_tiles;
        __syncwarp();
        tc_fence_before();
        __syncthreads();  // the piece is through: its queries, O and S may be written again
        tc_fence_after();
        if (*abort_flag) break;
    }
    if (warp == QR_MMA_WARP) {
        if (lane == 0) {  // every product has ended before tensor memory is given back
            tc_commit(drain);
            drain_wait_a(drain, 0);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == QR_MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, C::COLS);
    }
}

template <int BITS, int D>
cudaError_t launch(const QuantStep& s, const QuantPlane& pk, const QuantPlane& pv, const void* Q, int64_t ldq, void* O, int64_t ldo,
                   const int32_t* lengths, float* part, int* status, cudaStream_t stream) {
    using C = QrCfg<BITS, D>;
    const float scale = (float)(1.4426950408889634 / sqrt((double)D));
    auto go = [&](auto is_long) {
        auto kernel = quant_rows_kernel<BITS, D, is_long.value>;
        static std::atomic<uint64_t> done{0};
        return launch_with_smem(kernel, C::SMEM, done, [&] {
            return launch_pdl(kernel, dim3((unsigned)s.ctas), dim3(QR_THREADS), C::SMEM, stream, s, pk, pv,
                              static_cast<const __nv_bfloat16*>(Q), ldq, static_cast<__nv_bfloat16*>(O), ldo, lengths, scale, part, status);
        });
    };
    return quant_most_tokens(s) > kQuantRowsLong ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace

cudaError_t launch_quant_rows(const QuantStep& s, int bits, const QuantPlane& pk, const QuantPlane& pv, const void* Q, int64_t ldq,
                              void* O, int64_t ldo, const int32_t* lengths, float* part, int* status, cudaStream_t stream) {
    if (bits == 4)
        return pk.d == 64 ? launch<4, 64>(s, pk, pv, Q, ldq, O, ldo, lengths, part, status, stream)
                          : launch<4, 128>(s, pk, pv, Q, ldq, O, ldo, lengths, part, status, stream);
    return pk.d == 64 ? launch<8, 64>(s, pk, pv, Q, ldq, O, ldo, lengths, part, status, stream)
                      : launch<8, 128>(s, pk, pv, Q, ldq, O, ldo, lengths, part, status, stream);
}

}  // namespace mha
