// quant.cuh -- the quantised key/value cache: layout, and where a call's rows lie in it.
//
// Per (sequence, K/V head, token): the codes of the head's d channels, padded to 32 of them (4 bits: channel 2i in
// the low half of byte i), and per group of 64 channels a step s and a lowest value m, both bf16.  A code c stands
// for s c + m.  Tokens of a head lie side by side, so a decode step streams a head's keys in whole pieces; rows are
// multiples of 16 bytes and caches hold multiples of 16 tokens, so any 16 tokens can be fetched by one bulk copy.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace mha {

constexpr int kQuantGroup = 64;   // channels that share a step and a lowest value
constexpr int kQuantTokens = 16;  // caches hold multiples of this many tokens

// Keys or values of a cache: rows [B * h_kv][T_max].
struct QuantPlane {
    uint8_t* codes;
    uint32_t* params;  // [row][groups]: s in the low half, m in the high half
    int d, row, groups;  // channels; bytes of a row's codes; groups of a row
};

__host__ __device__ inline int quant_row_bytes(int d, int bits) { return (d + 31) / 32 * 4 * bits; }
__host__ __device__ inline int quant_groups(int d) { return (d + kQuantGroup - 1) / kQuantGroup; }

__device__ __forceinline__ float quant_step(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float quant_lowest(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

// Division of numbers below 2^31 by a number known on the host.
struct Divide {
    uint32_t mul, shift, by;
    __host__ explicit Divide(uint32_t d = 1) : shift(0), by(d) {
        while ((1ull << shift) < d) ++shift;
        mul = (uint32_t)(((((uint64_t)1 << shift) - d) << 32) / d + 1);  // 2^(32 + shift) / d, upwards, less 2^32
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int operator()(uint32_t n) const { return (int)((__umulhi(n, mul) + n) >> shift); }
#endif
};

// ------------------------------------------------------------------ how a decode step is cut
//
// The query rows that share a cached head are taken `rb` at a time: a group is (batch, K/V head, block of rows), and
// its visible tokens are cut into quanta of 128, or where that would only cost a join, into one.  All quanta of all
// groups, numbered by batch, head, block and token, are dealt out evenly: CTA c of C <= N takes those from c N / C to
// (c + 1) N / C, whatever the lengths are.  A CTA therefore has pieces of at most two groups that others share, its first
// and its last, and leaves records of those (per row: m, l and the values, scores in base 2); groups that it has alone it
// finishes.  The join adds a group's records in the order of its tokens.  Which CTA has what follows from the lengths and
// C alone.
//
// Steps whose groups' tokens are few for a CTA give each group a cluster of 1, 2, 4 or 8 CTAs instead, which cut its quanta
// evenly among themselves and join their results through distributed shared memory: one launch, no records.  So do steps
// of one sequence, whose groups are equally long: `parts` clusters a group, each of which leaves one record.

constexpr int kQuantum = 128;      // tokens
constexpr int kQuantMaxCtas = 640; // largest grid, for the size of the workspace
constexpr int kQuantCluster = 8;   // largest cluster
constexpr int kQuantRowsLong = 4096;  // tokens of a piece that quant_rows.cu's tensor-core sums may take

struct QuantStep {
    int B, h_kv, per, T_q, T_max;
    int rows;     // per * T_q: query rows of a cached head
    int rb, nrb;  // rows of a row block; row blocks
    int ctas;     // grid: C is this, or the number of quanta if that is less
    int dv;
    int rec;      // values of a row's record: dv, or as many as the kernel computes
    int quantum;  // tokens of a quantum: a multiple of kQuantum
    int cluster;  // CTAs of a cluster, each with one piece; 0: the even cut.  ctas is then cluster * parts * groups
    int parts;    // clusters of a group
    // divisions by T_q, nrb, lanes(), quantum, ctas and the CTAs of a group (a runtime division is some 150 cycles of
    // a chain that a step has to wait for)
    Divide by_T_q, by_nrb, by_lanes, by_quantum, by_ctas, by_group;
    __host__ __device__ int lanes() const { return h_kv * nrb; }   // groups of a batch
    __host__ __device__ int record() const { return rec + 2; }     // floats
    // Record of a row of a CTA's first (which = 0: it began in another CTA) or last group.
    __host__ __device__ int64_t slot(int cta, int which, int row) const { return ((int64_t)(2 * cta + which) * rb + row) * record(); }
};

#ifdef __CUDACC__

__device__ __forceinline__ int quant_quanta(const QuantStep& s, int L) {
    return L < s.T_q || L > s.T_max ? 0 : s.by_quantum((uint32_t)(L - 1)) + 1;  // (T_q is at least 1)
}

// A lane's part of the prefix sums over the batches; N quanta in all, of which a CTA has `each` or one more.
struct QuantPlan {
    int i0, i1, L0, before, sum, N, C, each, rest;
    bool bad;  // some length is invalid
    __device__ __forceinline__ int length(const int32_t* lengths, int i) const { return i == i0 ? L0 : __ldcg(lengths + i); }
    // First quantum of a CTA: floor(cta N / C); C is the grid, or N with a quantum for each.
    __device__ __forceinline__ int first(const QuantStep& s, int cta) const {
        return cta < C ? cta * each + s.by_ctas((uint32_t)(cta * rest)) : N;
    }
    // The CTA that has a quantum.
    __device__ __forceinline__ int owner(const QuantStep& s, int q) const {
        int c = min(C - 1, (int)((float)q * __fdividef((float)C, (float)N)));  // off by one at most
        if (first(s, c) > q) --c;
        if (first(s, c + 1) <= q) ++c;
        return c;
    }
};

// a / b of a below 2^31 whose quotient is small.
__device__ __forceinline__ int quant_quotient(int a, int b) {
    int q = (int)__fdividef((float)a, (float)b), r = a - q * b;
    while (r < 0) --q, r += b;
    while (r >= b) ++q, r -= b;
    return q;
}

// All lanes of a warp call it, and the next two.
__device__ __forceinline__ QuantPlan quant_plan(const QuantStep& s, const int32_t* lengths) {
    const int lane = (int)threadIdx.x & 31, run = (s.B + 31) / 32;
    QuantPlan p;
    p.i0 = min(s.B, lane * run);
    p.i1 = min(s.B, p.i0 + run);
    p.L0 = p.i0 < p.i1 ? __ldcg(lengths + p.i0) : 0;
    p.sum = 0;
    p.bad = false;
#pragma unroll 1
    for (int i = p.i0; i < p.i1; ++i) {
        const int n = quant_quanta(s, p.length(lengths, i));
        p.sum += n;
        p.bad = p.bad || n == 0;
    }
    p.bad = __any_sync(0xffffffffu, p.bad);
    p.sum *= s.lanes();
    int inc = p.sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    p.before = inc - p.sum;
    p.N = __shfl_sync(0xffffffffu, inc, 31);
    p.C = min(s.ctas, p.N);
    p.each = p.N < s.ctas ? 1 : s.by_ctas((uint32_t)p.N);
    p.rest = p.N < s.ctas ? 0 : p.N - p.each * s.ctas;
    return p;
}

// The piece of a group that begins at quantum q of a CTA whose quanta end at `end`.
struct QuantPiece {
    int b, lane;   // batch; head * nrb + block
    int L;
    int q0, q1;    // quanta [q0, q1) of the group
    int next;      // quantum behind the piece
    int nq;        // quanta of the group
    int quantum;
    __device__ __forceinline__ int k0() const { return q0 * quantum; }
    __device__ __forceinline__ int k1() const { return q1 == nq ? L : q1 * quantum; }
    __device__ __forceinline__ bool whole() const { return q0 == 0 && q1 == nq; }
};

__device__ __forceinline__ QuantPiece quant_piece(const QuantStep& s, const int32_t* lengths, const QuantPlan& p, int q, int end) {
    int b = 0, at = 0, len = 0;
    const bool mine = p.before <= q && q < p.before + p.sum;
    if (mine) {
        at = p.before;
#pragma unroll 1
        for (b = p.i0;; ++b) {
            len = p.length(lengths, b);
            const int n = quant_quanta(s, len) * s.lanes();
            if (q < at + n) break;
            at += n;
        }
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
    QuantPiece x;
    x.b = __shfl_sync(0xffffffffu, b, src);
    at = __shfl_sync(0xffffffffu, at, src);
    x.L = __shfl_sync(0xffffffffu, len, src);
    x.nq = quant_quanta(s, x.L);
    x.quantum = s.quantum;
    x.lane = quant_quotient(q - at, x.nq);
    const int start = at + x.lane * x.nq;
    x.q0 = q - start;
    x.q1 = min(x.nq, end - start);
    x.next = start + x.q1;
    return x;
}

// A cluster's CTA's piece of its group.  q0 == q1: none (an invalid length: nq is 0).
__device__ __forceinline__ QuantPiece quant_cluster_piece(const QuantStep& s, const int32_t* lengths) {
    const int n = s.cluster * s.parts, group = s.by_group(blockIdx.x), i = (int)blockIdx.x - group * n;
    QuantPiece x;
    x.b = s.by_lanes((uint32_t)group);
    x.lane = group - x.b * s.lanes();
    x.L = __ldcg(lengths + x.b);
    x.nq = quant_quanta(s, x.L);
    x.quantum = s.quantum;
    const int each = s.by_group((uint32_t)x.nq), rest = x.nq - each * n;  // q0 = floor(i nq / n) in 32 bits
    x.q0 = each * i + s.by_group((uint32_t)(rest * i));
    x.q1 = each * (i + 1) + s.by_group((uint32_t)(rest * (i + 1)));
    x.next = x.q1;
    return x;
}

#endif

}  // namespace mha
