// quant_decode.cu -- a decode step over a quantised cache (quant.cuh): which kernel takes it and how it is cut, the join
// of what several CTAs leave of a group, and the kernel for the head sizes that the tensor-core ones do not have.
//
// Heads of up to 128 channels go to quant_mma.cu, bf16 steps of hundreds of query rows to quant_rows.cu; what is left
// are fp32 layers whose heads are larger, or not of one size for keys and values, on CUDA cores.  With codes c, steps s and lowest values m per group G of channels,
// and the query row q (log2(e)/sqrt(d) folded in):
//   score_j = sum_G s_jG (sum_c q_c code_jc) + m_jG (sum_c q_c)          the codes are never turned into values
//   o       = sum_j p_j (s_jG code_jc + m_jG),  p_j = 2^(score_j - M)
// in fp32 throughout.  A CTA takes a part of one head's cached tokens for up to R query rows; its warps take 32
// tokens at a time in turn, a lane per token for the scores and a lane per eight channels for the values, each with
// its own running maximum, sum and values, joined at the end.  It is bound by its two multiply-adds and one conversion
// per code and row, and by latency before that: 5 ragged sequences of up to 1500 tokens, 16 heads of 80, 4 bits, which
// quant_mma.cu now has: 27 us (14.7 there).  16 of 4096, 8 heads of 64 for keys and 128 for values, 8 bits: 109 us, where 16
// would move the bytes; a third of the cycles issue, most of the others wait for codes and parameters out of memory.
#include <math.h>

#include "internal.h"
#include "ptx.cuh"
#include "quant.cuh"
#include "quant_meet.cuh"

namespace mha {
namespace {

constexpr int QD_THREADS = 256;
constexpr int QD_WARPS = QD_THREADS / 32;
constexpr int QD_ROWS = 4;

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

// The warps' results of a piece meet, as quant_meet() of quant_meet.cuh has it for known sizes: [warp][row] of `stride`
// floats, dv values, at ml m and l.
__device__ __forceinline__ void meet_any(const QuantStep& s, bool whole, float* rec, float* res, int stride, int ml, int b, int g,
                                         int r0, int nr, float* O, int64_t ldo) {
    constexpr int ENTRIES = QD_WARPS, THREADS = QD_THREADS, rows = QD_ROWS;
    const int tid = (int)threadIdx.x, dv = s.dv, record = s.record();
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

// dynamic shared memory: q[R][dpk], its sums qs[R][groups], and per warp p[R][32] or at the end m, l, o[dpv] per row
template <int BITS>
__global__ void __launch_bounds__(QD_THREADS)
    quant_decode_kernel(const QuantStep s, const QuantPlane pk, const QuantPlane pv, const float* __restrict__ Q, int64_t ldq,
                        float* __restrict__ O, int64_t ldo, const int32_t* __restrict__ lengths, float scale_log2,
                        float* __restrict__ part, int* status) {
    constexpr int R = QD_ROWS;
    extern __shared__ float sm[];
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int dpk = (pk.d + 31) & ~31, dpv = (pv.d + 31) & ~31;
    float* q = sm;
    float* qs = q + R * dpk;
    float* all = qs + R * pk.groups;
    float* own = all + warp * R * (dpv + 32);
    grid_dependency_wait();
    grid_launch_dependents();
    const QuantPlan plan = quant_plan(s, lengths);
    if (plan.bad) quant_invalid<QD_THREADS>(s, (int)blockIdx.x, (int)gridDim.x, lengths, O, ldo, status);
    const int end = plan.first(s, (int)blockIdx.x + 1);
    for (int at = plan.first(s, (int)blockIdx.x); at < end;) {
        const QuantPiece z = quant_piece(s, lengths, plan, at, end);
        at = z.next;
        const int b = z.b, g = s.by_nrb((uint32_t)z.lane), L = z.L, k0 = z.k0(), k1 = z.k1();
        const int r0 = (z.lane - g * s.nrb) * R, nr = min(R, s.rows - r0);
        __syncthreads();  // the piece before is written
        for (int e = tid; e < R * dpk; e += QD_THREADS) {
            const int r = e / dpk, c = e - r * dpk, rr = r0 + min(r, nr - 1);
            q[e] = c < pk.d ? scale_log2 * Q[((int64_t)b * s.T_q + rr % s.T_q) * ldq + (int64_t)(g * s.per + rr / s.T_q) * pk.d + c] : 0.f;
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
        meet_any(s, z.whole(), part + s.slot((int)blockIdx.x, z.q0 == 0 ? 1 : 0, 0), all, dpv + 32, dpv, b, g, r0, nr, O, ldo);
    }
}

// The join, 2 to 4 us behind the kernel before it, mostly the two round trips.  A block has `run` rows of a group; its threads take (row, slice of the records, column), `width` columns and
// `slices` slices.  A slice's maxima, sums and values are loaded together, so that a row costs about one round trip to L2
// and one more for every eight records of a slice; slices meet in shared memory.
template <typename T>
__global__ void __launch_bounds__(1024)
    quant_join_kernel(const QuantStep s, const float* __restrict__ part, T* __restrict__ O, int64_t ldo,
                      const int32_t* __restrict__ lengths, int width, int slices, int run, int chunks) {
    __shared__ float ys[1024], ms[1024], ls[1024];
    const int tid = (int)threadIdx.x;
    const int group = (int)blockIdx.x / chunks, chunk = (int)blockIdx.x - group * chunks;
    const int b = s.by_lanes((uint32_t)group), lane_i = group - b * s.lanes(), g = s.by_nrb((uint32_t)lane_i);
    const int r0 = (lane_i - g * s.nrb) * s.rb, nr = min(s.rb, s.rows - r0);
    // The kernel before lets this one start once its own wait for earlier work is over: the lengths can be read (from
    // L2), its records not yet.
    const float *first, *others;  // row 0 of the group's first record, and of record i >= 1 at others + i * stride
    int64_t stride;
    int n;
    if (s.cluster) {  // one record a cluster
        n = quant_quanta(s, __ldcg(lengths + b)) > 0 ? s.parts : 0;
        stride = (int64_t)s.rb * s.record();
        first = others = part + (int64_t)group * s.parts * stride;
    } else {
        const QuantPlan p = quant_plan(s, lengths);
        int at = 0, len = 0;
        const bool mine = p.i0 <= b && b < p.i1;
        if (mine) {
            at = p.before;
#pragma unroll 1
            for (int i = p.i0; i < b; ++i) at += quant_quanta(s, p.length(lengths, i)) * s.lanes();
            len = p.length(lengths, b);
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
        const int nq = quant_quanta(s, __shfl_sync(0xffffffffu, len, src));
        const int q0 = __shfl_sync(0xffffffffu, at, src) + lane_i * nq;
        const int c0 = nq > 0 ? p.owner(s, q0) : 0;
        n = nq > 0 ? p.owner(s, q0 + nq - 1) - c0 + 1 : 0;
        // of the first CTA its last group, of the others their first
        first = part + s.slot(c0, 1, 0);
        others = part + s.slot(c0, 0, 0);
        stride = s.slot(1, 0, 0);
    }
    const int e = tid % width, slice = tid / width % slices, at_once = (int)blockDim.x / (width * slices);
    grid_dependency_wait();
    grid_launch_dependents();
    if (n <= 1 && !s.cluster) return;  // an invalid length (written as NaN already), or a group that one CTA had alone
    if (n == 0) return;
#pragma unroll 1
    for (int k0 = 0; k0 < run; k0 += at_once) {
        const int r = chunk * run + k0 + tid / (width * slices);
        const bool live = r < nr && k0 + tid / (width * slices) < run;
        float M = -INFINITY, l = 0.f, x = 0.f;
        for (int i0 = slice; live && i0 < n; i0 += 8 * slices) {
            float m[8], sum[8], v[8], top = M;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int i = min(i0 + k * slices, n - 1);
                const float* a = (i == 0 ? first : others + i * stride) + r * s.record();
                m[k] = i0 + k * slices < n ? __ldcg(a) : -INFINITY;
                sum[k] = __ldcg(a + 1);
                v[k] = e < s.dv ? __ldcg(a + 2 + e) : 0.f;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) top = fmaxf(top, m[k]);
            const float f = M == -INFINITY ? 0.f : exp2f(M - top);
            l *= f;
            x *= f;
            M = top;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (m[k] != -INFINITY || sum[k] != sum[k]) {  // (a record of NaN alone has no maximum, but a sum of NaN)
                    const float fk = m[k] == -INFINITY ? 0.f : exp2f(m[k] - M);
                    l = fmaf(fk, sum[k], l);
                    x = fmaf(fk, v[k], x);
                }
        }
        if (slices > 1) {
            __syncthreads();  // the rows before are read
            ys[tid] = x;
            ms[tid] = M;
            ls[tid] = l;
            __syncthreads();
            if (slice > 0) continue;
            for (int k = 1; k < slices; ++k) M = fmaxf(M, ms[tid + k * width]);
            l = x = 0.f;
            for (int k = 0; k < slices; ++k) {
                const float m = ms[tid + k * width], f = m == -INFINITY ? 0.f : exp2f(m - M);
                l = fmaf(f, ls[tid + k * width], l);
                x = fmaf(f, ys[tid + k * width], x);
            }
        }
        if (live && e < s.dv) quant_put(quant_out(s, O, ldo, b, g, r0 + r) + e, x / l);
    }
}

size_t qd_smem(const QuantPlane& pk, const QuantPlane& pv) {
    const int dpk = (pk.d + 31) & ~31, dpv = (pv.d + 31) & ~31;
    return sizeof(float) * (size_t)QD_ROWS * (dpk + pk.groups + QD_WARPS * (dpv + 32));  // at most 41 KB
}

}  // namespace

// When a step's groups each get a cluster (us, cluster | even cut and join): 16 sequences of 1500 tokens, 16 K/V heads of
// 64, 12 quanta a CTA 10.1 | 16.7; 8 of 2048, 16 of 128, 8 quanta 14.4 | 19.5; 32 ragged of up to 8192, 4 of 128, 32 quanta
// 35.2 | 34.1 (all of 8192: 36.3 | 39.7).
// All clusters have to run at a time: a second wave costs 5 to 6 us, a CTA's latency from its lengths to its outputs.  One
// sequence is cut into more clusters a group from 6 quanta a CTA on: 16384 tokens, 4 heads, 16 quanta in one cluster
// 14.2, several 9.3, even cut 13.0; 131072 tokens, 2 heads, 8 bits: even cut 26.3, clusters on all SMs 37 (they do not all
// fit), on 85 % of them 22.7.
constexpr int kClusterQuanta = 16;
constexpr int kClusterQuantaOne = 6;
constexpr int kClusterQuantaWide = 6;  // of CTAs that an SM holds one of: 8 of 8192, one head of 128, 32 rows, 8 quanta 26.4 | 20.1

// With more groups than CTAs: the quanta that a CTA may have more than others, where groups are not cut at all, for the
// join and the shared groups' ends that this saves (32 sequences of 300 tokens, 16 heads of 128, 8 bits: 18.7 | 22.2 us).
constexpr int kJoinQuanta = 6;

// bf16 steps of at least this many rows of a cached head go to quant_rows.cu, in blocks of 128 (us, there | quant_mma.cu, 4
// bits, of 192, 256, 384 and 512 rows.  One sequence of 8192 tokens, 4 heads of 128: 40 | 31, 40 | 37, 50 | 50, 60 | 63; 4
// ragged of up to 4096, 4 of 64: 34 | 32, 34 | 39, 42 | 52, 50 | 64; 8 ragged of up to 8192, one of 128: 51 | 42, 55 | 54, 63 |
// 75, 75 | 95.  Its records are large).
constexpr int kManyRows = 256;
constexpr int kManyRowsBlock = 128;
constexpr int kManyRowsCtas = 320;  // most of its CTAs: one an SM

static int64_t most_ctas(const QuantStep& s) { return s.rb == kManyRowsBlock ? kManyRowsCtas : kQuantMaxCtas; }

// Rows of a block by the kernel that serves the head size; CTAs: as many as the GPU holds at a time, but no more than
// there may be quanta.
QuantStep quant_step_shape(bool f32, int bits, int d_k, int d_v, int B, int h, int h_kv, int T_q, int T_max, int sms) {
    QuantStep s;
    s.B = B;
    s.h_kv = h_kv;
    s.per = h / h_kv;
    s.T_q = T_q;
    s.T_max = T_max;
    s.rows = s.per * T_q;
    s.dv = d_v;
    s.rec = quant_mma_serves(d_k, d_v) ? quant_mma_width(d_k) : d_v;
    const bool many = !f32 && s.rows >= kManyRows, mma = !many && quant_mma_serves(d_k, d_v);
    s.rb = many ? kManyRowsBlock : mma ? quant_mma_rows(f32, bits, d_k, s.rows) : QD_ROWS;
    s.nrb = (s.rows + s.rb - 1) / s.rb;
    int64_t ctas = (int64_t)sms * (many ? 1 : mma ? quant_mma_ctas(f32, d_k, s.rb) : 2);
    const int64_t most = quant_most_quanta(s), groups = (int64_t)B * s.lanes();
    const int nq = (T_max + kQuantum - 1) / kQuantum;
    if (ctas > most_ctas(s)) ctas = most_ctas(s);
    s.quantum = kQuantum;
    if (groups > ctas && (groups + ctas - 1) / ctas * nq <= groups * nq / ctas + kJoinQuanta) s.quantum = nq * kQuantum;
    s.cluster = 0;
    s.parts = 1;
    if (mma) {
        int c = kQuantCluster;  // as large as lets all groups run at a time, and no larger than there are quanta
        while (c > 1 && (groups * c > ctas || nq < c)) c /= 2;
        const int64_t parts = ctas * 85 / 100 / (groups * kQuantCluster);
        if (B == 1 && parts > 1 && nq > kQuantCluster * kClusterQuantaOne) {
            s.cluster = kQuantCluster;
            s.parts = (int)parts;
        } else if (groups * c <= ctas && nq <= c * (quant_mma_ctas(f32, d_k, s.rb) == 1 ? kClusterQuantaWide : kClusterQuanta)) {
            s.cluster = c;
        }
    }
    if (ctas > most) ctas = most;
    if (s.cluster) ctas = groups * s.cluster * s.parts;
    s.ctas = ctas < 1 ? 1 : (int)ctas;
    s.by_T_q = Divide((uint32_t)(T_q < 1 ? 1 : T_q));
    s.by_nrb = Divide((uint32_t)(s.nrb < 1 ? 1 : s.nrb));
    s.by_lanes = Divide((uint32_t)(s.lanes() < 1 ? 1 : s.lanes()));
    s.by_quantum = Divide((uint32_t)s.quantum);
    s.by_ctas = Divide((uint32_t)s.ctas);
    s.by_group = Divide((uint32_t)(s.cluster * s.parts < 1 ? 1 : s.cluster * s.parts));
    return s;
}

int64_t quant_most_quanta(const QuantStep& s) { return (int64_t)s.B * s.h_kv * s.nrb * ((s.T_max + kQuantum - 1) / kQuantum); }

int64_t quant_most_tokens(const QuantStep& s) {
    const int64_t nq = (s.T_max + kQuantum - 1) / kQuantum, ctas = s.cluster * s.parts;
    const int64_t each = s.cluster ? (nq + ctas - 1) / ctas : s.quantum > kQuantum ? nq : quant_most_quanta(s) / s.ctas + 1;
    return kQuantum * (each < nq ? each : nq);
}

// For any number of SMs: two records a CTA, and behind them one place for sums of blocks of many rows whose pieces may
// be long.
size_t quant_step_bytes(const QuantStep& s) {
    const int64_t most = quant_most_quanta(s);
    const int64_t ctas = most < most_ctas(s) ? most : most_ctas(s);
    const int sums = s.rb == kManyRowsBlock && s.T_max > kQuantRowsLong ? s.dv : 0;
    return sizeof(float) * (size_t)ctas * s.rb * (2 * s.record() + sums);
}

bool quant_step_fits(const QuantStep& s) {
    return quant_most_quanta(s) <= INT32_MAX && (int64_t)s.B * s.h_kv * s.nrb * s.rb <= INT32_MAX;
}

cudaError_t launch_quant_decode(const QuantStep& s, bool f32, int bits, const QuantPlane& pk, const QuantPlane& pv,
                                const void* Q, int64_t ldq, void* O, int64_t ldo, const int32_t* lengths, float* part,
                                int* status, cudaStream_t stream) {
    cudaError_t err;
    if (s.rb == kManyRowsBlock) {
        err = launch_quant_rows(s, bits, pk, pv, Q, ldq, O, ldo, lengths, part, status, stream);
    } else if (quant_mma_serves(pk.d, pv.d)) {
        err = launch_quant_mma(s, f32, bits, pk, pv, Q, ldq, O, ldo, lengths, part, status, stream);
    } else if (f32) {
        const float scale = (float)(1.4426950408889634 / sqrt((double)pk.d));
        err = launch_pdl(bits == 4 ? quant_decode_kernel<4> : quant_decode_kernel<8>, dim3((unsigned)s.ctas), dim3(QD_THREADS),
                         qd_smem(pk, pv), stream, s, pk, pv, static_cast<const float*>(Q), ldq, static_cast<float*>(O), ldo, lengths,
                         scale, part, status);
    } else {
        err = cudaErrorInvalidValue;  // bf16 layers have no other heads
    }
    if (err != cudaSuccess || (s.cluster ? s.parts == 1 : s.T_max <= s.quantum)) return err;  // (groups of one quantum are never shared)
    // slices: as many as leave each about eight records of an evenly cut step; rows of a block: one, more if there
    // are more rows than some blocks an SM
    const int64_t groups = (int64_t)s.B * s.lanes(), n = s.cluster ? s.parts : s.ctas / groups + 2;
    const int width = s.dv <= 64 ? 64 : s.dv <= 128 ? 128 : 256;
    int slices = 1;
    while (slices * width < 1024 && n > 8 * slices) slices *= 2;
    const int threads = slices * width > 256 ? slices * width : 256, most = s.rows < s.rb ? s.rows : s.rb;
    int run = threads / (width * slices);
    while (run < most && groups * ((most + run - 1) / run) > 1024) run *= 2;
    const int chunks = (most + run - 1) / run;
    auto join = [&](auto* out) {
        using T = std::remove_pointer_t<decltype(out)>;
        return launch_pdl(quant_join_kernel<T>, dim3((unsigned)(groups * chunks)), dim3((unsigned)threads), 0, stream, s,
                          static_cast<const float*>(part), out, ldo, lengths, width, slices, run, chunks);
    };
    return f32 ? join(static_cast<float*>(O)) : join(static_cast<__nv_bfloat16*>(O));
}

}  // namespace mha
