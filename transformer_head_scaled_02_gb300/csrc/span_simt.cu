// span_simt.cu -- the windowed attention and the cache operators on CUDA cores (fp32 layers):
//   window_simt_kernel  causal sliding-window attention with sinks over whole sequences
//   span_simt_kernel    the units of span.cuh: windowed, shared-prefix and weight-accumulating
//                       decode steps
// Both form score tiles of BQ = 16 RQ query rows x 64 keys as small matrix products in full fp32
// (256 threads: thread (tx, ty) owns rows RQ ty.. and keys tx + 16 c), keep the online softmax in
// base 2 (log2(e) / sqrt(d_k) folded into one multiply per score; row maximum and sum over the 16
// threads sharing the rows, by shuffles), stage P in shared memory and add P V to RQ x 4 CV outputs
// per thread.  Q, K and V tiles are row-major in shared memory with rows padded by 4 floats: global
// loads are coalesced 16-byte pieces and the 16-byte reads of a product step (8 keys a quarter
// warp apart by d_k + 4 floats) touch every bank once.  One K and one V tile: the next K comes in behind
// the score product, the next V behind the value product, each under the other half of the work.
//
// Bound by the issue of FMAs and the waits between the halves (two blocks an SM, one where shared memory holds no
// more: 64 rows of d = 128).  Measured with asynchronous
// copies and packed score products | with plain loads of both tiles before a step: window of 256 over 2 x 8
// heads x 2048 rows, d = 64 98 | 112 us (36 % of the FMA rate), d = 128 218 (200 in 32-row blocks) | 306, d = 256
// 360 | 548; weights of 16 caches of 4096 tokens, 4 K/V heads, 20 rows of d = 64 180 | 227, 64 rows of d = 128
// 611 | 759; but one or two tiles a block (64 rows of d = 64 over a prefix of 4096) 59 | 51.  Packed value products
// as well, with P twice in shared memory, took 102 | 98 at d = 64, 204 | 200 at d = 128 and 343 | 360 at d = 256.
// The windows' blocks go from the last rows to the first: under a window of 2048 the same heads of d = 64 take 276
// us, from the first to the last 367 (256: 95 | 98).
#include <math.h>

#include "internal.h"
#include "ptx.cuh"
#include "span_records.cuh"

namespace mha {
namespace {

constexpr int SS_BK = 64;
constexpr int SS_THREADS = 256;
constexpr int SS_DK = 256;  // widest d_k
constexpr int SS_PS = SS_BK + 4;  // row stride of P

// 16 bytes, or 16 zero bytes, to shared memory.
__device__ __forceinline__ void cp_async16(float* dst, const float* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int RQ, int CV>
struct SimtTile {
    static constexpr int BQ = 16 * RQ;
    static constexpr int VS = 64 * CV;
    float *Qs, *Ks, *Vs, *Ps;
    int ks;  // row stride of Qs and Ks
    int dk, dk4, dv;
    float m[RQ], l[RQ], o[RQ][4 * CV];

    static constexpr size_t smem_bytes(int dk) {
        const size_t ks = (size_t)((dk + 3) & ~3) + 4;
        return sizeof(float) * (BQ * ks + SS_BK * ks + (size_t)SS_BK * VS + (size_t)BQ * SS_PS);
    }

    __device__ SimtTile(float* smem, int dk_, int dv_) : dk(dk_), dk4((dk_ + 3) & ~3), dv(dv_) {
        ks = dk4 + 4;
        Qs = smem;
        Ks = Qs + BQ * ks;
        Vs = Ks + SS_BK * ks;
        Ps = Vs + SS_BK * VS;
    }

    __device__ void reset() {
#pragma unroll
        for (int r = 0; r < RQ; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int u = 0; u < 4 * CV; ++u) o[r][u] = 0.f;
        }
    }

    // 4 consecutive elements of a row, zeros past n
    static __device__ float4 load4(const float* p, int n, bool vec) {
        if (vec && n >= 4) return __ldg(reinterpret_cast<const float4*>(p));
        return make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, n > 3 ? p[3] : 0.f);
    }

    // Row r of the query tile is at row(r), nullptr for rows that do not exist (zeros).
    template <class F>
    __device__ void load_q(F row, bool vec) {
        const int n4 = dk4 / 4;
        for (int i = (int)threadIdx.x; i < BQ * n4; i += SS_THREADS) {
            const int r = i / n4, e = (i - r * n4) * 4;
            const float* p = row(r);
            *reinterpret_cast<float4*>(&Qs[r * ks + e]) =
                p != nullptr ? load4(p + e, dk - e, vec) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }

    // n rows of a key or value tile, zeros past them and past `width` (whatever lies there never reaches a
    // product): asynchronous copies where 16-byte pieces are aligned.
    static __device__ void load_rows(float* dst, int stride, int cols, const float* src, int64_t ld, int n, int width, bool vec) {
        const int tx = (int)threadIdx.x & 15, ty = (int)threadIdx.x >> 4;
        for (int e = 4 * tx; e < cols; e += 64)
#pragma unroll
            for (int i = 0; i < SS_BK / 16; ++i) {
                const int j = ty + 16 * i;
                const bool in = j < n && e < width;
                float* to = dst + j * stride + e;
                if (vec)
                    cp_async16(to, in ? src + j * ld + e : src, in ? 16 : 0);
                else
                    *reinterpret_cast<float4*>(to) = in ? load4(src + j * ld + e, width - e, false) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
    }

    __device__ void load_k(const float* K, int64_t ld, int n, bool vec) { load_rows(Ks, ks, dk4, K, ld, n, dk, vec); }
    __device__ void load_v(const float* V, int64_t ld, int n, bool vec) { load_rows(Vs, VS, VS, V, ld, n, dv, vec); }

    // All key tiles of a range: tile(i, k0, n) gives their keys [k0, k0 + n); visible(row in block, key) and
    // score(row in block, key, s), which sees every masked base-2 score.  The next keys are on their way
    // during the softmax and the value product, the next values during the score product.
    template <class T, class F, class G>
    __device__ void run(int i0, int i1, T tile, const float* K, int64_t ldk, const float* V, int64_t ldv, bool vec,
                        float scale_log2, F visible, G score) {
        int k0, n;
        tile(i0, k0, n);
        __syncthreads();  // the tiles of the last range are no longer read
        load_k(K + k0 * ldk, ldk, n, vec);
        cp_async_commit();
        load_v(V + k0 * ldv, ldv, n, vec);
        cp_async_commit();
        for (int i = i0; i < i1; ++i) {
            int next_k0 = 0, next_n = 0;
            if (i + 1 < i1) tile(i + 1, next_k0, next_n);
            cp_async_wait<1>();
            __syncthreads();
            uint64_t sc2[RQ][4];
            products(sc2);
            __syncthreads();
            if (next_n > 0) load_k(K + next_k0 * ldk, ldk, next_n, vec);
            cp_async_commit();
            softmax(sc2, n, scale_log2, [&](int r, int j) { return visible(r, k0 + j); }, [&](int r, int j, float v) { score(r, k0 + j, v); });
            cp_async_wait<1>();
            __syncthreads();
            values(n);
            if (next_n > 0) {
                __syncthreads();
                load_v(V + next_k0 * ldv, ldv, next_n, vec);
            }
            cp_async_commit();
            k0 = next_k0;
            n = next_n;
        }
    }

    // Scores of a tile before their scale, as sums over the even and the odd elements (packed products: half
    // the instructions).
    __device__ void products(uint64_t (&sc)[RQ][4]) {
        const int tx = (int)threadIdx.x & 15, ty = (int)threadIdx.x >> 4;
#pragma unroll
        for (int r = 0; r < RQ; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) sc[r][c] = 0ull;
#pragma unroll 2
        for (int e = 0; e < dk4; e += 4) {
            ulonglong2 q[RQ], k[4];
#pragma unroll
            for (int r = 0; r < RQ; ++r) q[r] = *reinterpret_cast<const ulonglong2*>(&Qs[(ty * RQ + r) * ks + e]);
#pragma unroll
            for (int c = 0; c < 4; ++c) k[c] = *reinterpret_cast<const ulonglong2*>(&Ks[(tx + 16 * c) * ks + e]);
#pragma unroll
            for (int r = 0; r < RQ; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    sc[r][c] = fma2(q[r].x, k[c].x, sc[r][c]);
                    sc[r][c] = fma2(q[r].y, k[c].y, sc[r][c]);
                }
        }
    }

    template <class F, class G>
    __device__ void softmax(const uint64_t (&sc2)[RQ][4], int n, float scale_log2, F visible, G score) {
        const int tx = (int)threadIdx.x & 15, ty = (int)threadIdx.x >> 4;
        float sc[RQ][4];
#pragma unroll
        for (int r = 0; r < RQ; ++r) {
            float tmax = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int j = tx + 16 * c;
                float even, odd;
                unpack2(sc2[r][c], even, odd);
                sc[r][c] = j < n && visible(ty * RQ + r, j) ? (even + odd) * scale_log2 : -INFINITY;
                if (j < n) score(ty * RQ + r, j, sc[r][c]);
                tmax = fmaxf(tmax, sc[r][c]);
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, off));
            const float m_new = fmaxf(m[r], tmax);
            float psum = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                sc[r][c] = m_new == -INFINITY ? 0.f : exp2f(sc[r][c] - m_new);  // masked: 2^-inf = 0
                psum += sc[r][c];
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) psum += __shfl_xor_sync(0xffffffffu, psum, off);
            const float alpha = m_new == -INFINITY ? 1.f : exp2f(m[r] - m_new);  // 0 when m = -inf
            l[r] = l[r] * alpha + psum;
            m[r] = m_new;
#pragma unroll
            for (int u = 0; u < 4 * CV; ++u) o[r][u] *= alpha;
#pragma unroll
            for (int c = 0; c < 4; ++c) Ps[(ty * RQ + r) * SS_PS + tx + 16 * c] = sc[r][c];
        }
        __syncwarp();  // a row's P is written and read by the same half warp
    }

    __device__ void values(int n) {
        const int tx = (int)threadIdx.x & 15, ty = (int)threadIdx.x >> 4;
        const int n4 = (n + 3) & ~3;  // rows past n are zero on both sides
        for (int j = 0; j < n4; j += 4) {
            float p[RQ][4];
#pragma unroll
            for (int r = 0; r < RQ; ++r) {
                const float4 p4 = *reinterpret_cast<const float4*>(&Ps[(ty * RQ + r) * SS_PS + j]);
                p[r][0] = p4.x; p[r][1] = p4.y; p[r][2] = p4.z; p[r][3] = p4.w;
            }
#pragma unroll
            for (int jj = 0; jj < 4; ++jj)
#pragma unroll
                for (int c = 0; c < CV; ++c) {
                    const float4 v = *reinterpret_cast<const float4*>(&Vs[(j + jj) * VS + c * 64 + tx * 4]);
#pragma unroll
                    for (int r = 0; r < RQ; ++r) {
                        o[r][4 * c + 0] = fmaf(p[r][jj], v.x, o[r][4 * c + 0]);
                        o[r][4 * c + 1] = fmaf(p[r][jj], v.y, o[r][4 * c + 1]);
                        o[r][4 * c + 2] = fmaf(p[r][jj], v.z, o[r][4 * c + 2]);
                        o[r][4 * c + 3] = fmaf(p[r][jj], v.w, o[r][4 * c + 3]);
                    }
                }
        }
    }
};

static_assert(SimtTile<4, 4>::smem_bytes(SS_DK) <= 232448, "tiles fit shared memory");

// One block = BQ query rows of one (batch, head): the sinks below the rows' windows, then the keys
// from the first row's window to the last row.
template <int RQ, int CV>
__global__ void __launch_bounds__(SS_THREADS, RQ <= 2 ? (CV == 1 ? 4 : CV == 2 ? 3 : 2) : CV <= 2 ? 2 : 1)
    window_simt_kernel(const float* __restrict__ Q, int64_t ldq, const float* __restrict__ K, int64_t ldk,
                       const float* __restrict__ V, int64_t ldv, const float* __restrict__ G, int64_t ldg,
                       float* __restrict__ O, int64_t ldo, int h, int h_kv, int T, int dk, int dv,
                       int window, int sinks, const int32_t* __restrict__ kv_lengths, float scale_log2,
                       bool vec, int* status) {
    using X = SimtTile<RQ, CV>;
    extern __shared__ __align__(16) float fsm[];
    X x(fsm, dk, dv);
    const int tid = (int)threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int b = (int)blockIdx.x / h, head = (int)blockIdx.x - b * h;
    const int kvh = head / (h / h_kv);
    const int q0 = (int)(gridDim.y - 1 - blockIdx.y) * X::BQ;  // the last rows, which see the most keys, first
    const int L = kv_lengths != nullptr ? kv_lengths[b] : T;
    const int64_t row0 = (int64_t)b * T + q0;
    if (L < 1 || L > T) {
        if (tid == 0) record_status(status, kStatusBadLength);
        for (int i = tid; i < X::BQ * dv; i += SS_THREADS) {
            const int r = i / dv;
            if (q0 + r < T) O[(row0 + r) * ldo + (int64_t)head * dv + (i - r * dv)] = NAN;
        }
        return;
    }
    x.load_q([&](int r) { return q0 + r < T ? Q + (row0 + r) * ldq + (int64_t)head * dk : nullptr; }, vec);
    x.reset();
    const float* Kb = K + (int64_t)b * T * ldk + (int64_t)kvh * dk;
    const float* Vb = V + (int64_t)b * T * ldv + (int64_t)kvh * dv;
    const int end = min(L, q0 + X::BQ);
    int lo = max(0, q0 - window + 1);
    int s_end = min(sinks, L);  // sinks below the windows
    if (s_end >= lo) s_end = lo = 0;
    const int nst = (s_end + SS_BK - 1) / SS_BK, nt = nst + (max(0, end - lo) + SS_BK - 1) / SS_BK;
    if (nt > 0)
        x.run(0, nt,
              [&](int i, int& k0, int& n) {
                  k0 = i < nst ? i * SS_BK : lo + (i - nst) * SS_BK;
                  n = min(SS_BK, (i < nst ? s_end : end) - k0);
              },
              Kb, ldk, Vb, ldv, vec, scale_log2,
              [&](int r, int key) {
                  const int i = q0 + r;
                  return key <= i && (i - key < window || key < sinks);
              },
              [](int, int, float) {});
#pragma unroll
    for (int r = 0; r < RQ; ++r) {
        const int t = ty * RQ + r;
        if (q0 + t >= T) continue;
        // zeros where the mask leaves nothing, which only the mask can tell: a row whose scores are all NaN or
        // -inf has no weights either and is NaN
        const bool sees = q0 + t - L + 1 < window || sinks > 0;
        const float inv = sees ? 1.f / x.l[r] : 0.f;
#pragma unroll
        for (int u = 0; u < 4 * CV; ++u) {
            const int e = (u >> 2) * 64 + tx * 4 + (u & 3);
            if (e >= dv) continue;
            float y = x.o[r][u] * inv;
            if (G != nullptr) y *= 1.f / (1.f + expf(-G[(row0 + t) * ldg + (int64_t)head * dv + e]));
            O[(row0 + t) * ldo + (int64_t)head * dv + e] = y;
        }
    }
}

template <int RQ, int CV>
__global__ void __launch_bounds__(SS_THREADS, CV <= 2 ? 2 : 1)
    span_simt_kernel(const SpanShape p, const SpanRecords rec, const float* __restrict__ Q, int64_t ldq,
                     const float* __restrict__ K, int64_t ldk, const float* __restrict__ V, int64_t ldv,
                     const float* __restrict__ Kp, int64_t ldkp, const float* __restrict__ Vp, int64_t ldvp,
                     float* __restrict__ O, int64_t ldo, int dk, int dv,
                     const int32_t* __restrict__ lengths, float* __restrict__ scores, float scale_log2,
                     bool vec, int prefix_units, int cache_units, int* status) {
    using X = SimtTile<RQ, CV>;
    extern __shared__ __align__(16) float fsm[];
    X x(fsm, dk, dv);
    const int tid = (int)threadIdx.x, tx = tid & 15, ty = tid >> 4;
    grid_dependency_wait();  // lengths, queries and caches may come from the previous kernel
    grid_launch_dependents();
    SpanSums sums;
    const SpanPlan plan = span_plan<SS_BK>(p, lengths, (int)gridDim.x, sums);
    if (blockIdx.x == 0)
        for (int b = tid; b < p.B; b += SS_THREADS)
            if (lengths[b] < p.T_q || lengths[b] > p.T_max) record_status(status, kStatusBadLength);
    const int end = cache_units ? plan.N : plan.np;
    for (int u = (prefix_units ? 0 : plan.np) + (int)blockIdx.x; u < end; u += (int)gridDim.x) {
        const SpanUnit q = span_unit<SS_BK>(p, lengths, plan, sums, u);
        const int r0 = q.rb * X::BQ;
        const int nr = min(X::BQ, (q.prefix ? p.B * p.rows : p.rows) - r0);
        // batch, head and new token of row r of the block
        auto where = [&](int r, int& b, int& head, int& t) {
            int rr = r0 + r;
            b = q.b;
            if (q.prefix) {
                b = rr / p.rows;
                rr -= b * p.rows;
            }
            head = q.g * p.per + rr / p.T_q;
            t = rr % p.T_q;
        };
        __syncthreads();  // the previous unit's tiles are no longer read
        x.load_q([&](int r) -> const float* {
            if (r >= nr) return nullptr;
            int b, head, t;
            where(r, b, head, t);
            return Q + ((int64_t)b * p.T_q + t) * ldq + (int64_t)head * dk;
        }, vec);
        x.reset();
        const float* Kb = q.prefix ? Kp + (int64_t)q.g * dk : K + (int64_t)q.b * p.T_max * ldk + (int64_t)q.g * dk;
        const float* Vb = q.prefix ? Vp + (int64_t)q.g * dv : V + (int64_t)q.b * p.T_max * ldv + (int64_t)q.g * dv;
        const int64_t lk = q.prefix ? ldkp : ldk, lv = q.prefix ? ldvp : ldv;
        x.run(q.i0, q.i1, [&](int i, int& k0, int& n) { span_tile<SS_BK>(q.v, i, k0, n); }, Kb, lk, Vb, lv, vec, scale_log2,
              [&](int r, int key) { return q.prefix || span_visible(p, q.v.L - p.T_q + (r0 + r) % p.T_q, key); },
              [&](int r, int key, float s) {
                  if (scores != nullptr && r < nr) scores[(((int64_t)q.b * p.h_kv + q.g) * p.rows + r0 + r) * score_ld(p) + key] = s;
              });
        const bool direct = p.T_p == 0 && q.whole();
        const int64_t slot = rec.row(p, q.unit, plan.np);
#pragma unroll
        for (int r = 0; r < RQ; ++r) {
            const int rr = ty * RQ + r;
            if (rr >= nr) continue;
            if (tx == 0 && (!direct || scores != nullptr)) rec.ml[slot + rr] = make_float2(x.m[r], x.l[r]);
            float* out = rec.o + (slot + rr) * dv;
            float inv = 1.f;
            if (direct) {
                int b, head, t;
                where(rr, b, head, t);
                out = O + ((int64_t)b * p.T_q + t) * ldo + (int64_t)head * dv;
                inv = 1.f / x.l[r];
            }
#pragma unroll
            for (int u = 0; u < 4 * CV; ++u) {
                const int e = (u >> 2) * 64 + tx * 4 + (u & 3);
                if (e < dv) out[e] = x.o[r][u] * inv;
            }
        }
    }
}

}  // namespace

cudaError_t launch_window_f32(const float* Q, int64_t ldq, const float* K, int64_t ldk, const float* V,
                              int64_t ldv, const float* G, int64_t ldg, float* O, int64_t ldo, int B, int h,
                              int h_kv, int T, int d_k, int d_v, int window, int sinks,
                              const int32_t* kv_lengths, int* status, cudaStream_t stream) {
    auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    const bool vec = al(Q) && al(K) && al(V) && ldq % 4 == 0 && ldk % 4 == 0 && ldv % 4 == 0 && d_k % 4 == 0 && d_v % 4 == 0;
    const float scale = (float)(1.4426950408889634 / sqrt((double)d_k));
    const int cv = (d_v + 63) / 64;
    // 32-row blocks where 64-row ones leave SMs idle, and where an SM holds one block of 64 rows but two of 32:
    // 2 x 8 heads x 2048 rows of d = 128, window 64 | 256 | 1024: 90 | 200 | 542 us, in 64-row blocks 109 | 218 | 541
    // (d = 64 44 | 105 | 291 for 45 | 98 | 256, d = 80 156 for 141 under 256; d = 256 198 | 436 | 1155 for
    // 181 | 360 | 888)
    const bool one = cv <= 2 && SimtTile<4, 2>::smem_bytes(d_k) > 113 * 1024;
    const bool small = (int64_t)B * h * ((T + 63) / 64) < 256 || one;
    // most: what the kernel may ever need.  The limit belongs to the process, so every launch sets the same
    auto launch = [&](auto kernel, size_t smem, size_t most, int bq) {
        cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (err != cudaSuccess) return err;
        kernel<<<dim3((unsigned)(B * h), (unsigned)((T + bq - 1) / bq)), SS_THREADS, smem, stream>>>(
            Q, ldq, K, ldk, V, ldv, G, ldg, O, ldo, h, h_kv, T, d_k, d_v, window, sinks, kv_lengths, scale, vec,
            status);
        return cudaGetLastError();
    };
#define MHA_WS(RQ, CV) \
    if ((small ? 2 : 4) == RQ && cv == CV) \
        return launch(window_simt_kernel<RQ, CV>, SimtTile<RQ, CV>::smem_bytes(d_k), SimtTile<RQ, CV>::smem_bytes(SS_DK), \
                      16 * RQ);
    MHA_WS(2, 1) MHA_WS(2, 2) MHA_WS(2, 3) MHA_WS(2, 4) MHA_WS(4, 1) MHA_WS(4, 2) MHA_WS(4, 3) MHA_WS(4, 4)
#undef MHA_WS
    return cudaErrorInvalidValue;
}

cudaError_t launch_span_f32(const SpanShape& p, const SpanRecords& rec, const float* Q, int64_t ldq, const float* K,
                            int64_t ldk, const float* V, int64_t ldv, const float* Kp, int64_t ldkp, const float* Vp,
                            int64_t ldvp, float* O, int64_t ldo, int d_k, int d_v, const int32_t* lengths, float* scores,
                            bool prefix_units, bool cache_units, int ctas, int* status, cudaStream_t stream) {
    auto al = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
    const bool vec = al(Q) && al(K) && al(V) && ldq % 4 == 0 && ldk % 4 == 0 && ldv % 4 == 0 && d_k % 4 == 0 &&
                     d_v % 4 == 0 && (p.T_p == 0 || (al(Kp) && al(Vp) && ldkp % 4 == 0 && ldvp % 4 == 0));
    const float scale = (float)(1.4426950408889634 / sqrt((double)d_k));
    const int cv = (d_v + 63) / 64;
    auto launch = [&](auto kernel, size_t smem, size_t most) {  // most: as for the windows
        cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (err != cudaSuccess) return err;
        return launch_pdl(kernel, dim3((unsigned)ctas), dim3(SS_THREADS), smem, stream, p, rec, Q, ldq, K,
                          ldk, V, ldv, Kp, ldkp, Vp, ldvp, O, ldo, d_k, d_v, lengths, scores, scale, vec,
                          prefix_units ? 1 : 0, cache_units ? 1 : 0, status);
    };
    const int bm = cache_units ? p.bm_c : p.bm_p;
#define MHA_SS(RQ, CV) \
    if (bm == 16 * RQ && cv == CV) \
        return launch(span_simt_kernel<RQ, CV>, SimtTile<RQ, CV>::smem_bytes(d_k), SimtTile<RQ, CV>::smem_bytes(SS_DK));
    MHA_SS(1, 1) MHA_SS(1, 2) MHA_SS(1, 3) MHA_SS(1, 4) MHA_SS(2, 1) MHA_SS(2, 2) MHA_SS(2, 3) MHA_SS(2, 4)
    MHA_SS(4, 1) MHA_SS(4, 2) MHA_SS(4, 3) MHA_SS(4, 4)
#undef MHA_SS
    return cudaErrorInvalidValue;
}

}  // namespace mha
