// quant_mma.cu -- a decode step over a quantised cache (quant.cuh) for heads of up to 128 channels, on the tensor
// cores: the codes themselves are the matrix operands.
//
// A code in a 16-bit half whose other bits are zero is an fp16 number as it stands, a subnormal one: code 2^-24 exactly
// in the low bits, up to code 2^-18 further up the fraction.  So with steps s, lowest values m and 64-channel groups G
//   score_j = sum_G s_jG (q_G . code_jG) + m_jG (sum of q_G)
//   o       = sum_j (p_j s_jG) code_j + sum_j p_j m_jG
// need no more unpacking than masks, and the two products are exact but for the 16-bit forms of q and of p s; sums,
// softmax and the m terms are fp32.  q is scaled by a power of two so that fp16 holds it: exactly for bf16 layers, as
// high and low part for fp32 layers (22 bits); likewise p s, against a running power of two: 11 bits for bf16 layers,
// high and low part for fp32 ones.
//
// The cached tokens are the M side of both products (16 at a time) and the query rows the N side (8 or 16 columns), so
// a few rows waste no tensor work and the exponentials spread over all lanes.  Up to 4 rows leave half of the columns:
// every other block of 16 tokens takes those, as rows of their own until the end, and two blocks share one softmax.
// Which channel or token is which k of a product is free as long as both operands agree: it is chosen so that one mask
// takes two elements out of a word.
//   scores:  A = keys [token][channel], lane (gid, tig) holds 16 channels of a group of tokens gid and gid + 8
//   values:  A = values transposed [channel][token], the words of two tokens interleaved by a byte permutation;
//            B = p s, which the scores' layout becomes by transposing 8 x 8 pieces (movmatrix)
// mma.sync feeds operands from registers, where the unpacked codes are; tcgen05 would take them through shared memory:
// 64 KB of fp16 keys and values for 128 tokens of 128 channels, written and read once more, about 1000 cycles at 128
// bytes a cycle, where an SM's share of HBM's rate brings their 4-bit codes in 870.
//
// Stages of tokens come by bulk copies (a head's codes lie in one piece) into a ring; each warp takes a run of a
// stage's 16-token blocks with its own maximum, sum and values, and the last warp to finish a stage asks for the next
// one in its place.  (A ring per warp cost 200 instructions per stage and warp instead of some 30; with stages of half
// the size the first step below took 123 us instead of 99.)  Warps meet at the end of a piece.  The reference maximum
// moves only when a score exceeds it by 2^8, which one vote per block finds.
//
// Measured, bf16 layers, 4 bits, heads of 128, 32 ragged sequences of up to 8192 tokens: 16 heads with one query row each
// 93 us, 453 MB at 4.9 TB/s.  Copies alone take 72 us; with all of them out of L2 it is the same 93: what bounds it is in
// the SMs, where half of all cycles issue an instruction, with 16 warps, which is all that the registers hold (a tenth
// fewer instructions, products interleaved, loads ahead or a third stage changed nothing).  4 heads with 4 rows each
// 34.2 us, of which the join 4 and starts and ends of pieces 11.  One sequence of 4096 tokens, 4 heads of 64: 5.4 us,
// latency; of 131072 tokens, 2 heads of 128, 8 bits: 22.6 us, HBM's rate but for its start and end.
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "quant.cuh"
#include "quant_meet.cuh"

namespace mha {
namespace {

constexpr int QM_WARPS = 8;
constexpr float kNone = -3e38f;  // the reference of a row that has seen nothing: below every score, finite
constexpr int QM_THREADS = 32 * QM_WARPS;

// D: channels that are computed with, DP: those that a row of the cache has.  (What lies behind a short row is the next
// one's codes: finite numbers, which meet queries of zero and make values that nobody stores.)
// SPLIT: the columns are shared out to the groups as well.  ROUND: sums over blocks are added outside the tensor core, which
// cuts off what its sums cannot hold, always towards zero, 3.6e-8 of a sum of codes with every product.
template <int BITS, int D, int DP, int TERMS, int NT, int SUB, bool SPLIT>
struct QmCfg {
    static constexpr int G = D / kQuantGroup;
    static constexpr int GL = SPLIT ? 1 : G;                  // groups of a column
    static constexpr int ROW = DP * BITS / 8;
    static constexpr int TOK = 131072 / (D * BITS);           // tokens of a stage: 32 KB of codes
    static constexpr int STAGE = 2 * TOK * (ROW + 4 * G);     // key codes, value codes, key and value parameters
    static constexpr int CTAS = NT * TERMS * G > 2 ? 1 : 2;   // of an SM (registers)
    static constexpr int STAGES = CTAS == 1 ? 4 : 2;
    static constexpr int COLS = 8 * NT;                       // columns of the products
    static constexpr int COPIES = SPLIT ? SUB * G : SUB;      // of a query row among the columns
    static constexpr int ROWS = COLS / COPIES;                // query rows of a block
    static constexpr int RESULTS = SUB * ROWS;                // of a warp
    static constexpr int REC = D + 4;                         // floats of a result: values, m, l
    static constexpr int RES = STAGES * STAGE;                // the warps' results
    static constexpr int QF = RES + QM_WARPS * RESULTS * REC * 4;  // queries as operands, their sums and scales
    static constexpr int QS = QF + TERMS * NT * G * 32 * 32;
    static constexpr int QEND = QS + COLS * (G + 1) * 4;
    using Share = QuantShare<ROWS, D>;                        // of a cluster: a place of its own, or if that does not fit the
    static constexpr int TAIL = 16 * STAGES + 48;             // one of the queries
    static constexpr bool ROOM = CTAS * (QEND + Share::BYTES + TAIL + 1024) <= 228 * 1024;
    static constexpr int SHARE = ROOM ? QEND : QF;
    static constexpr int BARS = SHARE + Share::BYTES > QEND ? SHARE + Share::BYTES : QEND;
    static constexpr int SMEM = BARS + TAIL;                  // barriers, counts of the warps done, QmNext, abort flag
    static_assert(SUB == 1 || NT == 1, "only a few rows leave columns for a second block");
    static_assert(!SPLIT || (SUB == 2 && G == 2), "four sets of two columns");
    static_assert(BARS % 16 == 0 && SHARE % 16 == 0 && SMEM <= 232448, "");
    static_assert(TOK % kQuantum == 0, "a stage's tokens are dealt out evenly");
    static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory of an SM");
};

// Where the next stage to be copied begins.
struct QmNext {
    int64_t row;       // the piece's head in the cache
    int at, from, to;  // quantum behind the piece; what is left of it
    int issued;        // stages so far
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 half2_floats(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

// Codes of a word as fp16 pairs, two at a time.  The two are 16 bits apart:
// nibbles i and i + 4, or bytes i and i + 2, in x[i].  bf16 layers take them where they are, which is cheapest;
// fp32 layers move them to the top of the fraction, as the tensor core adds products by their exponents, which
// subnormal numbers' leading zeros do not lower: 7 bits lost show in fp32 (1.4e-5 of an output) but not in bf16.
template <int BITS, int TERMS>
__device__ __forceinline__ void codes_of(uint32_t w, uint32_t (&x)[BITS == 4 ? 4 : 2]) {
    if constexpr (BITS == 4 && TERMS == 1) {
        x[0] = w & 0x000f000fu;
        x[1] = w & 0x00f000f0u;
        x[2] = w >> 8 & 0x000f000fu;
        x[3] = w >> 8 & 0x00f000f0u;
    } else if constexpr (BITS == 4) {
        x[0] = w << 6 & 0x03c003c0u;
        x[1] = w << 2 & 0x03c003c0u;
        x[2] = w >> 2 & 0x03c003c0u;
        x[3] = w >> 6 & 0x03c003c0u;
    } else if constexpr (TERMS == 1) {
        x[0] = w & 0x00ff00ffu;
        x[1] = w >> 8 & 0x00ff00ffu;
    } else {
        x[0] = w << 2 & 0x03fc03fcu;
        x[1] = w >> 6 & 0x03fc03fcu;
    }
}

// What a code counts in even (h = 0) and odd (h = 1) places.
template <int BITS, int TERMS>
__device__ __forceinline__ constexpr float unit(int h) {
    constexpr float u = 5.9604644775390625e-8f;  // 2^-24
    return TERMS == 1 ? (BITS == 4 && h == 1 ? 16.f * u : u) : BITS == 4 ? 64.f * u : 4.f * u;
}

// 16 of a row's channels in a group (keys), as the A operands of the group's four products for one token: x[c][0] its
// k = 2 tig, 2 tig + 1, x[c][1] its k = 2 tig + 8, 2 tig + 9.  Which channels these are: q_place().
template <int BITS, int TERMS>
__device__ __forceinline__ void key_operands(uint32_t addr, uint32_t (&x)[4][2]) {
    uint32_t w[BITS / 2];
    if constexpr (BITS == 4) asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    else asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
#pragma unroll
    for (int i = 0; i < BITS / 2; ++i) {
        uint32_t y[BITS == 4 ? 4 : 2];
        codes_of<BITS, TERMS>(w[i], y);
#pragma unroll
        for (int c = 0; c < 8 / BITS; ++c) {
            x[i * 8 / BITS + c][0] = y[2 * c];
            x[i * 8 / BITS + c][1] = y[2 * c + 1];
        }
    }
}

// Product c, half h (k = 2 tig, .. or 2 tig + 8, ..) and element of the pair behind channel j of a lane's 16.
template <int BITS>
__device__ __forceinline__ void q_place(int j, int& c, int& h, int& e) {
    h = j & 1;
    c = BITS == 4 ? (j >> 3) * 2 + (j >> 1 & 1) : j >> 2;
    e = BITS == 4 ? j >> 2 & 1 : j >> 1 & 1;
}

// Codes as TERMS = 2 has them, in both halves, less 8 or 128.  Exact.
__device__ __forceinline__ uint32_t sub_centre(uint32_t x) {
    const uint32_t c = 0x02000200u;
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&c));
    return *reinterpret_cast<const uint32_t*>(&y);
}

// Eight of a row's channels in a group (values) of two tokens a, b, as the A operands of the group's four products:
// x[t][0] channel 2 t of both tokens, x[t][1] channel 2 t + 1.  fp32 layers take half the range off the codes (and add it to
// the lowest values): over thousands of tokens the sums of codes are far larger than what is left of them in the output
// (5400 tokens of small scores: 2e-5 of the outputs with neither this nor ROUND, 1.3e-6 with this alone, 1e-7 with both).
template <int BITS, int TERMS>
__device__ __forceinline__ void value_operands(uint32_t addr_a, uint32_t addr_b, uint32_t (&x)[4][2]) {
    uint32_t a[BITS / 4], b[BITS / 4];
    if constexpr (BITS == 4) {
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(a[0]) : "r"(addr_a));
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(b[0]) : "r"(addr_b));
    } else {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(a[0]), "=r"(a[1]) : "r"(addr_a));
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(b[0]), "=r"(b[1]) : "r"(addr_b));
    }
#pragma unroll
    for (int i = 0; i < BITS / 2; ++i) {
        const uint32_t w = __byte_perm(a[i / 2], b[i / 2], (i & 1) ? 0x7632 : 0x5410);  // half of a, half of b
        uint32_t y[BITS == 4 ? 4 : 2];
        codes_of<BITS, TERMS>(w, y);
#pragma unroll
        for (int c = 0; c < 8 / BITS; ++c) {
            x[i * 8 / BITS + c][0] = TERMS == 1 ? y[2 * c] : sub_centre(y[2 * c]);
            x[i * 8 / BITS + c][1] = TERMS == 1 ? y[2 * c + 1] : sub_centre(y[2 * c + 1]);
        }
    }
}

// Parameters of a token's G groups.
template <int G>
__device__ __forceinline__ void token_params(uint32_t addr, uint32_t (&p)[G]) {
    if constexpr (G == 1) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(p[0]) : "r"(addr));
    else asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(p[0]), "=r"(p[1]) : "r"(addr));
}

__device__ __forceinline__ float elem(const float* p) { return __ldg(p); }
__device__ __forceinline__ float elem(const __nv_bfloat16* p) { return __bfloat162float(*p); }

template <int BITS, int D, int DP, int TERMS, int NT, int SUB, bool SPLIT, bool ROUND, typename T>
__global__ void __launch_bounds__(QM_THREADS, QmCfg<BITS, D, DP, TERMS, NT, SUB, SPLIT>::CTAS)
    quant_mma_kernel(const QuantStep s, const QuantPlane pk, const QuantPlane pv, const T* __restrict__ Q, int64_t ldq,
                     T* __restrict__ O, int64_t ldo, const int32_t* __restrict__ lengths, float scale_log2,
                     float* __restrict__ part, int* status) {
    using C = QmCfg<BITS, D, DP, TERMS, NT, SUB, SPLIT>;
    constexpr int G = C::G, GL = C::GL;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5, gid = lane >> 2, tig = lane & 3;
    const uint32_t ring = smem_u32(smem), bars = ring + C::BARS;
    uint32_t* done = reinterpret_cast<uint32_t*>(smem + C::BARS + 8 * C::STAGES);
    QmNext* next = reinterpret_cast<QmNext*>(smem + C::BARS + 16 * C::STAGES);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(next + 1);
    if (tid == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(bars + 8u * i, 1);
            done[i] = 0;
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();

    QuantPlan plan;
    QuantPiece own;  // of a cluster's CTA
    int begin, end;
    if (s.cluster) {
        own = quant_cluster_piece(s, lengths);
        begin = own.q0;
        end = own.q1;
        if (C::ROOM && s.cluster > 1) cluster_arrive_relaxed();  // this CTA's shared memory may be written
        if (own.nq == 0) {
            if (blockIdx.x % (unsigned)(s.cluster * s.parts * s.lanes()) == 0) quant_invalid<QM_THREADS>(s, own.b, s.B, lengths, O, ldo, status);
            if (C::ROOM && s.cluster > 1) cluster_wait();
            return;
        }
    } else {
        plan = quant_plan(s, lengths);
        begin = plan.first(s, (int)blockIdx.x);
        end = plan.first(s, (int)blockIdx.x + 1);
        if (plan.bad) quant_invalid<QM_THREADS>(s, (int)blockIdx.x, (int)gridDim.x, lengths, O, ldo, status);
    }
    auto piece = [&](int q) { return s.cluster ? own : quant_piece(s, lengths, plan, q, end); };
    // One warp at a time asks for the next stage (all its lanes call this): at first the last warp, then whichever is the last
    // to have used the stage whose place it takes.
    auto fetch = [&](QmNext& x) {
        while (x.from >= x.to) {
            if (x.at >= end) return;
            const QuantPiece z = piece(x.at);
            x.at = z.next;
            x.row = ((int64_t)z.b * s.h_kv + s.by_nrb((uint32_t)z.lane)) * s.T_max;
            x.from = z.k0();
            x.to = z.k1();
        }
        // whole sixteens: caches hold multiples of them.  Codes and parameters of keys and values: a lane each.
        const uint32_t tok = (uint32_t)min(C::TOK, (x.to - x.from + 15) & ~15);
        const uint32_t at = ring + (uint32_t)(x.issued % C::STAGES * C::STAGE), bar = bars + 8u * (uint32_t)(x.issued % C::STAGES);
        if (lane == 0) mbar_arrive_expect_tx(bar, 2u * tok * (C::ROW + 4 * G));
        __syncwarp();
        if (lane < 4) {
            const bool values = lane & 1, params = lane & 2;
            const int64_t r = x.row + x.from;
            const uint8_t* codes = (values ? pv.codes : pk.codes) + r * C::ROW;
            const uint32_t* pars = (values ? pv.params : pk.params) + r * G;
            const uint32_t to = params ? at + 2 * C::TOK * C::ROW + (values ? C::TOK * 4 * G : 0) : at + (values ? C::TOK * C::ROW : 0);
            bulk_load(to, params ? static_cast<const void*>(pars) : codes, params ? tok * 4 * G : tok * C::ROW, bar);
        }
        x.from += C::TOK;
        ++x.issued;
    };
    auto share = [&] { return typename C::Share{ring + C::SHARE, s.cluster, s.cluster > 1 ? (int)cluster_ctarank() : 0}; };
    if (warp == QM_WARPS - 1) {  // (the first warps have queries to see to)
        QmNext x{0, begin, 0, 0, 0};
#pragma unroll 1
        for (int n = 0; n < C::STAGES; ++n) fetch(x);
        if (lane == 0) *next = x;
    }

    bool ok = true;
    uint32_t used = 0;  // stages
#pragma unroll 1
    for (int q_at = begin; q_at < end;) {
    const QuantPiece z = piece(q_at);
    q_at = z.next;
    const int b = z.b, g = s.by_nrb((uint32_t)z.lane), L = z.L;
    const int r0 = (z.lane - g * s.nrb) * C::ROWS, nr = min(C::ROWS, s.rows - r0);

    // queries: a warp makes a row's B operands, as the lanes will want them, its sum per group and the factor that turns
    // a product with it into a score
    {
        constexpr int CPL = D / 32;  // channels of a lane
        __half* qh = reinterpret_cast<__half*>(smem + C::QF);
        float* qv = reinterpret_cast<float*>(smem + C::QS);
#pragma unroll
        for (int r = warp; r < C::ROWS; r += QM_WARPS) {
            const int rr = r0 + min(r, nr - 1), hg = s.by_T_q((uint32_t)rr), t = rr - hg * s.T_q;
            const T* src = Q + ((int64_t)b * s.T_q + t) * ldq + (int64_t)(g * s.per + hg) * (TERMS == 1 ? D : s.dv) + lane * CPL;
            float x[CPL], top = 0.f;
#pragma unroll
            for (int e = 0; e < CPL; ++e) x[e] = TERMS == 1 || lane * CPL + e < s.dv ? elem(src + e) : 0.f;
#pragma unroll
            for (int e = 0; e < CPL; ++e) top = fmaxf(top, fabsf(x[e]));
#pragma unroll
            for (int w = 16; w >= 1; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
            // the largest element to [2^13, 2^14); zero, infinite, tiny and huge (2^118) rows as far as powers of two go
            const int e2 = top > 0.f && top < INFINITY ? max(-104, min(126, 13 - quant_exponent(top))) : 0;
            const float f = quant_power2(e2);
            const int u = G == 1 ? 0 : lane / 16;
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < CPL; ++e) {
                const int j = lane * CPL + e & 15, to = lane * CPL + e >> 4 & 3;  // channel of lane `to` of four
                int c, h, half;
                q_place<BITS>(j, c, h, half);
                const float v = f * x[e] * (h == 0 ? 1.f : unit<BITS, TERMS>(0) / unit<BITS, TERMS>(1));
                sum = fmaf(h == 0 ? unit<BITS, TERMS>(0) : unit<BITS, TERMS>(1), v, sum);
                const __half hi = __float2half_rn(v), lo = __float2half_rn(v - __half2float(hi));
#pragma unroll
                for (int k = 0; k < C::COPIES; ++k) {
                    const int n = r % 8 + k * C::ROWS;  // column
                    const int at = (((r / 8 * G + u) * 32 + 4 * n + to) * 8 + 2 * c + h) * 2 + half;
                    qh[at] = hi;
                    if constexpr (TERMS == 2) qh[NT * G * 512 + at] = lo;
                }
            }
#pragma unroll
            for (int w = 8; w >= 1; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            if constexpr (G == 1) sum += __shfl_xor_sync(0xffffffffu, sum, 16);
#pragma unroll
            for (int k = 0; k < C::COPIES; ++k) {
                if (lane % 16 == 0 && lane / 16 < G) qv[(r + k * C::ROWS) * (G + 1) + u] = sum;
                if (lane == 0) qv[(r + k * C::ROWS) * (G + 1) + G] = scale_log2 / unit<BITS, TERMS>(0) * quant_power2(-e2);
            }
        }
    }
    __syncthreads();
    uint32_t qf[TERMS][NT][G][4][2];
    const int set = SPLIT ? tig : 0, first = set % 2;  // of a lane's columns: block * 2 + group, and that group
    float qs[NT][GL][2], rs[NT][2];  // y rs is a score
    const int lim_min = L - s.T_q + 1;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int w = 0; w < TERMS; ++w)
#pragma unroll
            for (int u = 0; u < G; ++u) {
                const uint4* from = reinterpret_cast<const uint4*>(smem + C::QF) + (((w * NT + nt) * G + u) * 32 + lane) * 2;
                const uint4 v0 = from[0], v1 = from[1];
                qf[w][nt][u][0][0] = v0.x; qf[w][nt][u][0][1] = v0.y; qf[w][nt][u][1][0] = v0.z; qf[w][nt][u][1][1] = v0.w;
                qf[w][nt][u][2][0] = v1.x; qf[w][nt][u][2][1] = v1.y; qf[w][nt][u][3][0] = v1.z; qf[w][nt][u][3][1] = v1.w;
            }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float* from = reinterpret_cast<const float*>(smem + C::QS) + (8 * nt + 2 * tig + e) * (G + 1);
#pragma unroll
            for (int u = 0; u < GL; ++u) qs[nt][u][e] = from[first + u];
            rs[nt][e] = from[G];
        }
    }

    if (!C::ROOM && s.cluster > 1) cluster_arrive();  // the queries' place may be written

    float o[NT][GL][4][4], om[NT][GL][2], m[NT][2], l[NT][2];
    float vs[NT][2];   // p s is held as p s vs: of each column, as a token may matter to one row and not to another
    float far[NT][2];  // the y that moves the reference m, which is a y too (a rounded score could be far from a large one)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            m[nt][e] = far[nt][e] = kNone;
            vs[nt][e] = quant_power2(kQuantScaleMost);
            l[nt][e] = 0.f;
#pragma unroll
            for (int u = 0; u < GL; ++u) {
                om[nt][u][e] = 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) o[nt][u][c][2 * e] = o[nt][u][c][2 * e + 1] = 0.f;
            }
        }
    const int block = SUB == 1 ? 0 : SPLIT ? tig / 2 : 2 * tig / C::ROWS;  // whose columns the lane has
    const int pa = gid ^ (gid >> 1 & 1);                          // this lane's key token, and its second at + 8: the
    const int va = 2 * tig ^ (tig & 1), vb = (2 * tig + 1) ^ (tig & 1);  // order in which neither load meets itself in a bank
#pragma unroll 1
    for (int t_stage = z.k0(); t_stage < z.k1() && ok; t_stage += C::TOK) {
        const uint32_t slot = used % C::STAGES;
        if (!__all_sync(0xffffffffu, mbar_wait(bars + 8u * slot, used / C::STAGES & 1u, abort_flag, status))) {
            ok = false;
            break;
        }
        const uint32_t at = ring + slot * C::STAGE;
        // the stage's 16-token blocks, a run of them for each warp
        const uint32_t blocks = min((uint32_t)C::TOK / 16u, (uint32_t)(z.k1() - t_stage + 15) / 16u);
        const int w_end = min(z.k1(), t_stage + (int)((uint32_t)(warp + 1) * blocks / QM_WARPS * 16u));  // the run's end
#pragma unroll 1
        for (int sub = (int)((uint32_t)warp * blocks / QM_WARPS * 16u); t_stage + sub < w_end; sub += 16 * SUB) {
            const int t0 = t_stage + sub;
            const bool edge = t0 + 16 * SUB > min(lim_min, w_end);  // some column does not see all of its 16
            const uint32_t kc = at + (uint32_t)(sub * C::ROW), vc = kc + C::TOK * C::ROW;
            const uint32_t kp = at + 2 * C::TOK * C::ROW + (uint32_t)((sub + 16 * block) * 4 * G + 4 * first), vp = kp + C::TOK * 4 * G;
            // scores; with two blocks, columns 0 .. 3 are the first one's and columns 4 .. 7 the second one's
            float y[NT][4];
            {
                float acc[NT][GL][4];
#pragma unroll
                for (int k = 0; k < SUB; ++k)
#pragma unroll
                    for (int u = 0; u < G; ++u) {
                        uint32_t ka[4][2], kb[4][2];
                        const uint32_t col = (uint32_t)((u * kQuantGroup + 16 * tig) * BITS / 8);
                        key_operands<BITS, TERMS>(kc + (uint32_t)((pa + 16 * k) * C::ROW) + col, ka);
                        key_operands<BITS, TERMS>(kc + (uint32_t)((pa + 16 * k + 8) * C::ROW) + col, kb);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const uint32_t a[4] = {ka[c][0], kb[c][0], ka[c][1], kb[c][1]};
#pragma unroll
                                for (int w = 0; w < TERMS; ++w) mma_f16(d, a, qf[w][nt][u][c][0], qf[w][nt][u][c][1]);
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if constexpr (SPLIT) acc[nt][0][e] = k + u == 0 || set == 2 * k + u ? d[e] : acc[nt][0][e];
                                else acc[nt][u][e] = k == 0 ? d[e] : block == 0 ? acc[nt][u][e] : d[e];
                            }
                        }
                    }
                uint32_t p0[GL], p1[GL];
                token_params<GL>(kp + (uint32_t)(pa * 4 * G), p0);
                token_params<GL>(kp + (uint32_t)((pa + 8) * 4 * G), p1);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[nt][e] = quant_lowest(e < 2 ? p0[0] : p1[0]) * qs[nt][0][e & 1];
#pragma unroll
                        for (int u = 0; u < GL; ++u) {
                            const uint32_t par = e < 2 ? p0[u] : p1[u];
                            if (u > 0) y[nt][e] = fmaf(quant_lowest(par), qs[nt][u][e & 1], y[nt][e]);
                            y[nt][e] = fmaf(quant_step(par), acc[nt][u][e], y[nt][e]);
                        }
                        if constexpr (SPLIT) y[nt][e] += __shfl_xor_sync(0xffffffffu, y[nt][e], 1);  // the other group's part
                    }
            }
            uint32_t v0[GL], v1[GL];
            token_params<GL>(vp + (uint32_t)(pa * 4 * G), v0);
            token_params<GL>(vp + (uint32_t)((pa + 8) * 4 * G), v1);
            if (edge) {  // tokens at or past the length hold anything
                const int ta = t0 + 16 * block + pa, tb = ta + 8;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = (8 * nt + 2 * tig + e) % C::ROWS;
                        const int rr = r0 + min(r, nr - 1), lim = min(w_end, lim_min + rr - s.by_T_q((uint32_t)rr) * s.T_q);
                        if (ta >= lim) y[nt][e] = -INFINITY;
                        if (tb >= lim) y[nt][e + 2] = -INFINITY;
                    }
#pragma unroll
                for (int u = 0; u < GL; ++u) {
                    if (ta >= w_end) v0[u] = 0;
                    if (tb >= w_end) v1[u] = 0;
                }
            }
            // references
            float steps = 0.f;
#pragma unroll
            for (int u = 0; u < GL; ++u) steps = fmax3(steps, quant_step(v0[u]), quant_step(v1[u]));
            bool move = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    move = move || fmaxf(y[nt][e], y[nt][e + 2]) > far[nt][e] || steps * vs[nt][e] > kQuantStepMost;
            if (__any_sync(0xffffffffu, move)) {
                float step0 = 0.f, step1 = 0.f, f[NT][2], fr[NT][2], need[NT][2], seen = 0.f;
                bool rises = false;
#pragma unroll
                for (int u = 0; u < GL; ++u) {
                    step0 = fmaxf(step0, quant_step(v0[u]));
                    step1 = fmaxf(step1, quant_step(v1[u]));
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(y[nt][e], y[nt][e + 2]);
#pragma unroll
                        for (int w = 16; w >= 4; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                        f[nt][e] = 1.f;
                        if (top > m[nt][e]) {
                            f[nt][e] = ex2_approx((m[nt][e] - top) * rs[nt][e]);
                            m[nt][e] = top;
                            far[nt][e] = __fadd_rd(top, __fdividef(8.f, rs[nt][e]));  // (rounded up, weights could be 2^16)
                        }
                        // the column's largest p s
                        need[nt][e] = fmaxf(step0 * ex2_approx((y[nt][e] - m[nt][e]) * rs[nt][e]),
                                            step1 * ex2_approx((y[nt][e + 2] - m[nt][e]) * rs[nt][e]));
#pragma unroll
                        for (int w = 16; w >= 4; w >>= 1) need[nt][e] = fmaxf(need[nt][e], __shfl_xor_sync(0xffffffffu, need[nt][e], w));
                        rises = rises || quant_scale_rises(vs[nt][e], need[nt][e], f[nt][e]);
                        seen += l[nt][e];
                    }
                // A scale rises as far as the column's sums leave fp32 room.  (The room that f makes is not enough: one column's
                // reference moves whenever another's does, and rounded down to powers of two many small f make none.)
                int room[NT][2] = {};
                if (__any_sync(0xffffffffu, rises)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float most = 0.f;
#pragma unroll
                            for (int u = 0; u < GL; ++u)
#pragma unroll
                                for (int c = 0; c < 4; ++c) most = fmax3(most, fabsf(o[nt][u][c][e]), fabsf(o[nt][u][c][e + 2]));
#pragma unroll
                            for (int w = 16; w >= 4; w >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, w));
                            room[nt][e] = min(100, 38 - quant_exponent(most));
                        }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float to = quant_move_scale(vs[nt][e], need[nt][e], f[nt][e], room[nt][e]);
                        fr[nt][e] = quant_rescale(to, vs[nt][e], f[nt][e]);
                        vs[nt][e] = to;
                    }
                if (__any_sync(0xffffffffu, seen != 0.f)) {  // not at a warp's first tokens
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            l[nt][e] *= f[nt][e];
#pragma unroll
                            for (int u = 0; u < GL; ++u) {
                                om[nt][u][e] *= f[nt][e];
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    o[nt][u][c][e] *= fr[nt][e];
                                    o[nt][u][c][e + 2] *= fr[nt][e];
                                }
                            }
                        }
                }
            }
            // weights, and their products with the steps as B operands
            uint32_t bf[TERMS][NT][GL][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = ex2_approx((y[nt][e] - m[nt][e & 1]) * rs[nt][e & 1]);
                l[nt][0] += p[0] + p[2];
                l[nt][1] += p[1] + p[3];
                float pw[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) pw[e] = p[e] * vs[nt][e & 1];
#pragma unroll
                for (int u = 0; u < GL; ++u) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t par = h == 0 ? v0[u] : v1[u];
                        const float w = quant_step(par);
                        const float z = TERMS == 1 ? quant_lowest(par) : fmaf(w, BITS == 4 ? 8.f : 128.f, quant_lowest(par));
                        om[nt][u][0] = fmaf(p[2 * h], z, om[nt][u][0]);
                        om[nt][u][1] = fmaf(p[2 * h + 1], z, om[nt][u][1]);
                        const float w0 = pw[2 * h] * w, w1 = pw[2 * h + 1] * w;
                        const uint32_t hi = half2_bits(w0, w1);
                        bf[0][nt][u][h] = transpose8(hi);
                        if constexpr (TERMS == 2) {
                            const float2 back = half2_floats(hi);
                            bf[TERMS - 1][nt][u][h] = transpose8(half2_bits(w0 - back.x, w1 - back.y));
                        }
                    }
                }
            }
            // values: each block's tokens with its own columns
#pragma unroll
            for (int k = 0; k < SUB; ++k)
#pragma unroll
                for (int u = 0; u < G; ++u) {
                    uint32_t xa[4][2], xb[4][2], w2[TERMS][NT][2];
                    const uint32_t col = (uint32_t)((u * kQuantGroup + 8 * gid) * BITS / 8), from = vc + (uint32_t)(16 * k * C::ROW) + col;
                    value_operands<BITS, TERMS>(from + (uint32_t)(va * C::ROW), from + (uint32_t)(vb * C::ROW), xa);
                    value_operands<BITS, TERMS>(from + (uint32_t)((va + 8) * C::ROW), from + (uint32_t)((vb + 8) * C::ROW), xb);
#pragma unroll
                    for (int w = 0; w < TERMS; ++w)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                w2[w][nt][h] = SUB == 1 || gid / C::ROWS == (SPLIT ? 2 * k + u : k) ? bf[w][nt][SPLIT ? 0 : u][h] : 0u;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t a[4] = {xa[c][0], xa[c][1], xb[c][0], xb[c][1]};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float(&to)[4] = o[nt][SPLIT ? 0 : u][c];
                            if constexpr (!ROUND) {
                                mma_f16(to, a, w2[0][nt][0], w2[0][nt][1]);
                            } else {
                                float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                                for (int w = 0; w < TERMS; ++w) mma_f16(d, a, w2[w][nt][0], w2[w][nt][1]);
#pragma unroll
                                for (int e = 0; e < 4; ++e) to[e] += d[e];
                            }
                        }
                    }
                }
        }
        ++used;
        uint32_t last = 0;
        __syncwarp();  // the stage is read
        if (lane == 0) {
            asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;" : "=r"(last) : "r"(bars + 8u * C::STAGES + 4u * slot) : "memory");
            last = last % QM_WARPS == QM_WARPS - 1;
        }
        if (__shfl_sync(0xffffffffu, last, 0)) {
            QmNext x = *next;
            fetch(x);
            __syncwarp();
            if (lane == 0) *next = x;
        }
    }

    // this warp's result: rows of D values, m, l.  2^24 / vs takes the sums back; where it would be past fp32's range (steps
    // of 2^104 and more), the sums are multiplied by its two factors one after the other.
    float up = 1.f / unit<BITS, TERMS>(0);
    {
        bool tiny = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) tiny = tiny || fminf(vs[nt][0], vs[nt][1]) < 7.8886090522101181e-31f;  // 2^-100
        if (__any_sync(0xffffffffu, tiny)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int u = 0; u < GL; ++u)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[nt][u][c][e] *= up;
            up = 1.f;
        }
    }
    float* own = reinterpret_cast<float*>(smem + C::RES) + warp * C::RESULTS * C::REC;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float inv = up / vs[nt][e];
#pragma unroll
            for (int w = 4; w <= 16; w <<= 1) {
                l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], w);
#pragma unroll
                for (int u = 0; u < GL; ++u) om[nt][u][e] += __shfl_xor_sync(0xffffffffu, om[nt][u][e], w);
            }
            float* row = own + (SPLIT ? block * C::ROWS + e : 8 * nt + 2 * tig + e) * C::REC + first * kQuantGroup;
#pragma unroll
            for (int u = 0; u < GL; ++u)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *reinterpret_cast<float2*>(row + u * kQuantGroup + 8 * gid + 2 * c) =
                        make_float2(fmaf(o[nt][u][c][e], inv, om[nt][u][e]),
                                    fmaf(o[nt][u][c][e + 2], inv * (unit<BITS, TERMS>(0) / unit<BITS, TERMS>(1)), om[nt][u][e]));
            if (gid == 0 && first == 0) *reinterpret_cast<float2*>(row + D) = make_float2(m[nt][e] == kNone ? kNone : m[nt][e] * rs[nt][e], l[nt][e]);
        }
    if (s.cluster > 1) cluster_wait();
    __syncthreads();
    const bool whole = s.cluster ? s.cluster * s.parts == 1 : z.whole();
    float* rec = s.cluster > 1 ? nullptr : part + s.slot((int)blockIdx.x, z.q0 == 0 ? 1 : 0, 0);
    quant_meet<QM_WARPS * SUB, QM_THREADS, D, C::ROWS>(s, whole, rec, share(), reinterpret_cast<float*>(smem + C::RES), b, g, r0, nr, O, ldo);
    __syncthreads();
    }
    if (s.cluster > 1) {  // the CTAs' records have met, a share of the columns in each
        const int g = s.by_nrb((uint32_t)own.lane), r0 = (own.lane - g * s.nrb) * C::ROWS, nr = min(C::ROWS, s.rows - r0);
        const typename C::Share to = share();
        if (begin == end) {  // had nothing
            if (!C::ROOM) cluster_arrive();
            cluster_wait();
            for (int i = tid; i < nr * s.cluster; i += QM_THREADS) {
                const int r = i / s.cluster;
                st_shared_cluster_v2(mapa_shared(to.sums(to.rank, r), (uint32_t)(i - r * s.cluster)), kNone, 0.f);
            }
        }
        cluster_sync_all();
        const int cols = to.cols();
        const uint8_t* mine = smem + C::SHARE;
        for (int e = tid; e < nr * cols; e += QM_THREADS) {
            const int r = e / cols, c = e - r * cols;
            float m[kQuantCluster], l[kQuantCluster], v[kQuantCluster], M = kNone, sum = 0.f, x = 0.f;
#pragma unroll
            for (int k = 0; k < kQuantCluster; ++k) {
                const int from = min(k, s.cluster - 1);
                const float2 ml = *reinterpret_cast<const float2*>(mine + (to.sums(from, r) - to.base));
                m[k] = k < s.cluster ? ml.x : kNone;
                l[k] = ml.y;
                v[k] = *reinterpret_cast<const float*>(mine + (to.value(from, r, c) - to.base));
                M = fmaxf(M, m[k]);
            }
#pragma unroll
            for (int k = 0; k < kQuantCluster; ++k)
                if (m[k] != kNone || l[k] != l[k]) {  // (a piece of NaN alone has no maximum, but a sum of NaN)
                    const float f = exp2f(m[k] - M);
                    sum = fmaf(f, l[k], sum);
                    x = fmaf(f, v[k], x);
                }
            if (s.parts == 1) {
                if (TERMS == 1 || to.rank * cols + c < s.dv) quant_put(quant_out(s, O, ldo, own.b, g, r0 + r) + to.rank * cols + c, x / sum);
            } else {
                float* rec = part + ((int64_t)((int)blockIdx.x / s.cluster) * C::ROWS + r) * s.record();
                rec[2 + to.rank * cols + c] = x;
                if (to.rank == 0 && c == 0) rec[0] = M, rec[1] = sum;
            }
        }
    }
    if (*abort_flag && tid == 0)  // a copy did not arrive: wait for those in flight, and leave
        for (int k = max(0, next->issued - C::STAGES); k < next->issued; ++k)
            drain_wait_a(bars + 8u * (uint32_t)(k % C::STAGES), (uint32_t)(k / C::STAGES) & 1u);
}

// Products that a warp's sums take, from when on bf16 layers add them outside the tensor core (fp32 layers always do).  With
// 32 the cut is 1.2e-6 of the codes' part of an output, which is below bf16's rounding where the outputs are 1/2000 of it;
// values around zero under even weights come to that at 65536 tokens: 512 products were off by 1.2 % there, 0.17 % so, of
// which the outputs' own rounding is all.  It takes 1 to 3 % longer (us, within | outside, 16 heads as in the file's
// comment 92.8 | 94.7, 4 heads of 4 rows 34.1 | 35.1).
constexpr int kRoundProducts = 32;

template <int BITS, int D, int DP, int TERMS, int NT, int SUB, bool SPLIT, typename T>
cudaError_t launch(const QuantStep& s, const QuantPlane& pk, const QuantPlane& pv, const void* Q, int64_t ldq, void* O,
                   int64_t ldo, const int32_t* lengths, float* part, int* status, cudaStream_t stream) {
    using C = QmCfg<BITS, D, DP, TERMS, NT, SUB, SPLIT>;
    const float scale = (float)(1.4426950408889634 / sqrt((double)pk.d));
    auto go = [&](auto round) {
        auto kernel = quant_mma_kernel<BITS, D, DP, TERMS, NT, SUB, SPLIT, round.value, T>;
        static std::atomic<uint64_t> done{0};
        return launch_with_smem(kernel, C::SMEM, done, [&] {
            return launch_pdl_cluster(kernel, s.cluster > 1 ? s.cluster : 1, dim3((unsigned)s.ctas), dim3(QM_THREADS), C::SMEM, stream, s,
                                      pk, pv, static_cast<const T*>(Q), ldq, static_cast<T*>(O), ldo, lengths, scale, part, status);
        });
    };
    if constexpr (TERMS == 1)
        if (quant_most_tokens(s) <= kRoundProducts * 16 * QM_WARPS * SUB) return go(std::false_type{});
    return go(std::true_type{});
}

// (fp32 layers of 128 channels have no room in the registers for 16 rows)
constexpr bool most_rows_16(int terms, int d) { return !(terms == 2 && d == 128); }

template <int BITS, int D, int DP, typename T, typename... A>
cudaError_t launch_rows(int rb, A... a) {
    constexpr int TERMS = std::is_same_v<T, float> ? 2 : 1;
    if constexpr (BITS * D == 512 && D == 128)
        if (rb == 2) return launch<BITS, D, DP, TERMS, 1, 2, true, T>(a...);
    if constexpr (BITS * D <= 512)
        if (rb == 4) return launch<BITS, D, DP, TERMS, 1, 2, false, T>(a...);
    if (rb == 8) return launch<BITS, D, DP, TERMS, 1, 1, false, T>(a...);
    if constexpr (most_rows_16(TERMS, D)) return launch<BITS, D, DP, TERMS, 2, 1, false, T>(a...);
    return cudaErrorInvalidValue;
}

// bf16 layers have heads of 64 and 128 channels.  fp32 ones compute short rows with 64 or 128 (16 ragged sequences of up
// to 4096 tokens, 8 heads of 80, 8 bits: 33 us, 95 on CUDA cores).
template <int BITS, typename T, typename... A>
cudaError_t launch_width(int d, int rb, A... a) {
    if constexpr (std::is_same_v<T, float>) {
        if (d <= 32) return launch_rows<BITS, 64, 32, T>(rb, a...);
        if (d > 64 && d <= 96) return launch_rows<BITS, 128, 96, T>(rb, a...);
    }
    return d <= 64 ? launch_rows<BITS, 64, 64, T>(rb, a...) : launch_rows<BITS, 128, 128, T>(rb, a...);
}

}  // namespace

bool quant_mma_serves(int d_k, int d_v) { return d_k == d_v && d_k <= 128; }

// Channels that are computed with.
int quant_mma_width(int d) { return d <= 64 ? 64 : 128; }

// Query rows of a block: 2, whose columns two blocks of tokens and two groups share; 4, whose columns two blocks of tokens share (a warp's part of a stage of 8 bits and 128 channels
// is one block), 8, or 16 (two sets of operands and sums beside each unpacked code).
int quant_mma_rows(bool f32, int bits, int d_k, int rows) {
    const int d = quant_mma_width(d_k);
    if (rows <= 2 && bits * d == 512 && d == 128) return 2;
    if (rows <= 4 && bits * d <= 512) return 4;
    return rows <= 8 || !most_rows_16(f32 ? 2 : 1, d) ? 8 : 16;
}

int quant_mma_ctas(bool f32, int d_k, int rb) { return (f32 ? 2 : 1) * (quant_mma_width(d_k) / 64) * (rb == 16 ? 2 : 1) > 2 ? 1 : 2; }

cudaError_t launch_quant_mma(const QuantStep& s, bool f32, int bits, const QuantPlane& pk, const QuantPlane& pv, const void* Q,
                             int64_t ldq, void* O, int64_t ldo, const int32_t* lengths, float* part, int* status,
                             cudaStream_t stream) {
    auto go = [&](auto* x) {
        using T = std::remove_pointer_t<decltype(x)>;
        return bits == 4 ? launch_width<4, T>(pk.d, s.rb, s, pk, pv, Q, ldq, O, ldo, lengths, part, status, stream)
                         : launch_width<8, T>(pk.d, s.rb, s, pk, pv, Q, ldq, O, ldo, lengths, part, status, stream);
    };
    return f32 ? go(static_cast<float*>(nullptr)) : go(static_cast<__nv_bfloat16*>(nullptr));
}

}  // namespace mha
