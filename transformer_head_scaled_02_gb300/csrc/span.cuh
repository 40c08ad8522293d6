// span.cuh -- how the cache operators (windowed, shared-prefix and weight-accumulating decode
// steps) cut their work, shared by the kernels that compute the pieces and those that join them.
//
// The query rows that share cached keys form groups: one per (batch, K/V head, row block) over the
// batch's own cache, and, with a shared prefix, one per (K/V head, row block) over the prefix, whose
// rows are those of the whole batch.  A group's visible keys are at most two ranges, the sinks
// [0, s) and the window [lo, L), each cut into tiles.  All groups' tiles in order form one
// sequence, which D = min(G, N) of the G CTAs divide evenly: CTA c takes tiles [N c / D, N (c + 1) / D),
// so ragged lengths and group counts that do not divide the SMs leave no CTA idle.  A CTA's run
// crosses group borders; each crossing starts a piece.  A piece that holds a whole group writes its
// output itself; the others leave (maximum, sum, weighted values) records that the merge joins:
//   O = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p,  M = max_p m_p   (scores in base 2).
// Record slot of a piece: CTA index + group index.  Both only grow along the sequence and one of
// them does at every piece, so slots are distinct.
#pragma once

#include <stdint.h>

namespace mha {

// Largest grid of a piece kernel (bounds the record slots; the host knows no SM count when it
// computes workspace sizes).
constexpr int kSpanMaxCtas = 320;

struct SpanShape {
    int B, h_kv;
    int per;     // query heads per K/V head
    int T_q, T_max;
    int rows;    // per * T_q: query rows of one (batch, K/V head)
    int nrb;     // row blocks of such a group
    int T_p;     // shared prefix tokens (0: none)
    int nrbp;    // row blocks of the B * rows rows over the prefix
    int window;  // <= T_max; T_max: no window
    int sinks;
};

// The visible keys of a batch with L cached tokens: [0, s_keys) and [lo, L); nt tiles in all (0 for
// an invalid length).
struct SpanView {
    int L, s_keys, lo, nst, nt;
};

template <int TILE>
__host__ __device__ inline SpanView span_view(const SpanShape& p, int L) {
    SpanView v;
    v.L = L;
    v.s_keys = 0;
    v.nst = 0;
    v.nt = 0;
    v.lo = 0;
    if (L < p.T_q || L > p.T_max) return v;
    const int lo = L - p.T_q - p.window + 1;  // first key in the window of new token 0
    if (lo > p.sinks) {
        v.s_keys = p.sinks;
        v.lo = lo;
    }  // else the two ranges meet: one range from 0
    v.nst = (v.s_keys + TILE - 1) / TILE;
    v.nt = v.nst + (L - v.lo + TILE - 1) / TILE;
    return v;
}

// Keys [key0, key0 + n) of tile i of a view.
template <int TILE>
__device__ __forceinline__ void span_tile(const SpanView& v, int i, int& key0, int& n) {
    const bool sink = i < v.nst;
    key0 = sink ? i * TILE : v.lo + (i - v.nst) * TILE;
    const int end = sink ? v.s_keys : v.L;
    n = end - key0 < TILE ? end - key0 : TILE;
}

// Does the new token at cache position pos see the key?
__device__ __forceinline__ bool span_visible(const SpanShape& p, int pos, int key) {
    return key <= pos && (pos - key < p.window || key < p.sinks);
}

template <int TILE>
__host__ __device__ inline int span_prefix_tiles(const SpanShape& p) {
    return (p.T_p + TILE - 1) / TILE;
}

// CTAs that share N tiles when G are launched: each of them holds at least one.
__host__ __device__ inline int64_t span_parts(int64_t N, int G) { return N < G ? N : G; }

// CTAs [c0, c1] that hold tiles [t0, t1) of N when a grid of G divides them.
__device__ __forceinline__ void span_ctas(int64_t N, int G, int64_t t0, int64_t t1, int& c0, int& c1) {
    const int64_t D = span_parts(N, G);
    c0 = (int)(((t0 + 1) * D - 1) / N);
    c1 = (int)((t1 * D - 1) / N);
}

// Where a CTA starts in the tile sequence.
struct SpanStart {
    int64_t N;       // tiles in all
    int64_t t0, t1;  // this CTA's tiles
    int b;           // batch that holds the CTA's first tile past the prefix
    int64_t off;     // first tile of that batch's groups
};

// One contiguous run of tiles within one group.
struct SpanPiece {
    bool prefix;
    int b, g, rb;
    int64_t group;  // index among all groups
    int i0, i1;     // tiles [i0, i1) of the group
    SpanView v;     // the batch's view (prefix: L = T_p, one range)
    __device__ bool whole() const { return i0 == 0 && i1 == v.nt; }
};

// Walks a CTA's pieces in order.
template <int TILE>
struct SpanWalk {
    const SpanShape& p;
    const int32_t* lengths;
    int64_t t, t1, off;
    int b;

    __device__ SpanWalk(const SpanShape& p_, const int32_t* lengths_, const SpanStart& s)
        : p(p_), lengths(lengths_), t(s.t0), t1(s.t1), off(s.off), b(s.b) {}

    __device__ bool next(SpanPiece& q) {
        if (t >= t1) return false;
        const int np = span_prefix_tiles<TILE>(p);
        const int64_t npt = (int64_t)np * p.h_kv * p.nrbp;
        int64_t in;  // tile within the group
        if (t < npt) {
            q.prefix = true;
            q.group = t / np;
            in = t - q.group * np;
            q.b = 0;
            q.g = (int)(q.group / p.nrbp);
            q.rb = (int)(q.group - (int64_t)q.g * p.nrbp);
            q.v.L = p.T_p;
            q.v.s_keys = q.v.lo = q.v.nst = 0;
            q.v.nt = np;
        } else {
            q.prefix = false;
            q.v = span_view<TILE>(p, lengths[b]);
            while (t >= off + (int64_t)q.v.nt * p.h_kv * p.nrb) {  // the next batch (some hold no tile)
                off += (int64_t)q.v.nt * p.h_kv * p.nrb;
                ++b;
                q.v = span_view<TILE>(p, lengths[b]);
            }
            const int gr = (int)((t - off) / q.v.nt);
            in = t - off - (int64_t)gr * q.v.nt;
            q.b = b;
            q.g = gr / p.nrb;
            q.rb = gr - q.g * p.nrb;
            q.group = (int64_t)p.h_kv * p.nrbp + (int64_t)b * p.h_kv * p.nrb + gr;
        }
        q.i0 = (int)in;
        const int64_t left = t1 - t;
        q.i1 = left < q.v.nt - in ? (int)(in + left) : q.v.nt;
        t += q.i1 - q.i0;
        return true;
    }
};

// First tile of batch b's groups and the number of tiles in all; every thread of the block (of
// THREADS) calls it and gets the answer.
template <int TILE, int THREADS>
__device__ inline void span_offset(const SpanShape& p, const int32_t* lengths, int b, int64_t& off,
                                   int64_t& total) {
    const int64_t npt = (int64_t)span_prefix_tiles<TILE>(p) * p.h_kv * p.nrbp;
    int64_t below = 0, all = 0;
    for (int i = (int)threadIdx.x; i < p.B; i += THREADS) {
        const int64_t n = (int64_t)span_view<TILE>(p, lengths[i]).nt * p.h_kv * p.nrb;
        all += n;
        if (i < b) below += n;
    }
    __shared__ int64_t part[2][THREADS / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        below += __shfl_xor_sync(0xffffffffu, below, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    if ((threadIdx.x & 31) == 0) {
        part[0][threadIdx.x >> 5] = below;
        part[1][threadIdx.x >> 5] = all;
    }
    __syncthreads();
    off = total = npt;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        off += part[0][w];
        total += part[1][w];
    }
    __syncthreads();
}

// This CTA's share of the sequence; every thread of the block calls it.
template <int TILE, int THREADS>
__device__ inline SpanStart span_start(const SpanShape& p, const int32_t* lengths) {
    __shared__ int64_t part[THREADS / 32];
    __shared__ int64_t base_s;
    __shared__ int found_b;
    __shared__ int64_t found_off;
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t npt = (int64_t)span_prefix_tiles<TILE>(p) * p.h_kv * p.nrbp;
    SpanStart s;
    int64_t unused;
    span_offset<TILE, THREADS>(p, lengths, 0, unused, s.N);
    const int64_t D = span_parts(s.N, (int)gridDim.x), c = min((int64_t)blockIdx.x, D);
    s.t0 = D > 0 ? s.N * c / D : 0;
    s.t1 = c < D ? s.N * (c + 1) / D : s.t0;
    const int64_t want = s.t0 > npt ? s.t0 : npt;  // the batch in which the own-cache tiles start
    if (tid == 0) {
        found_b = 0;
        found_off = npt;
        base_s = npt;
    }
    __syncthreads();
    for (int i0 = 0; i0 < p.B; i0 += THREADS) {
        const int i = i0 + tid;
        const int64_t n = i < p.B ? (int64_t)span_view<TILE>(p, lengths[i]).nt * p.h_kv * p.nrb : 0;
        int64_t inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
        }
        if (lane == 31) part[warp] = inc;
        __syncthreads();
        int64_t before = base_s + inc - n;
        int64_t sum = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) before += part[w];
            sum += part[w];
        }
        if (n > 0 && before <= want && want < before + n) {
            found_b = i;
            found_off = before;
        }
        __syncthreads();
        if (tid == 0) base_s += sum;
        __syncthreads();
    }
    s.b = found_b;
    s.off = found_off;
    return s;
}


}  // namespace mha
