// span.cuh -- how the cache operators (windowed, shared-prefix and weight-accumulating decode
// steps) cut their work, shared by the kernels that compute the pieces and those that join them.
//
// The query rows that share cached keys form groups: one per (batch, K/V head, row block) over the
// batch's own cache, and, with a shared prefix, one per (K/V head, row block) over the prefix, whose
// rows are those of the whole batch.  A group's visible keys are at most two ranges, the sinks
// [0, s) and the window [lo, L), each cut into tiles.
//
// The CTAs work in gangs of H: the member CTAs of a gang walk the same tiles of H neighbouring lanes
// (K/V head, row block) side by side.  A cached token's rows of all heads lie side by side, so what a
// gang reads at a time is whole pieces of DRAM pages: 32 sequences of 16 heads with d = 128 ran at 54% of
// the copy bandwidth without gangs (each CTA somewhere else, 256 bytes at a time).  The tiles of
// all batches and lane blocks in order form one sequence of N, which D = min(gangs, N) gangs divide
// evenly: gang c takes tiles [N c / D, N (c + 1) / D), so ragged lengths and group counts that do not
// divide the SMs leave no CTA idle.  A gang's run crosses group borders; each crossing starts a piece.
// A piece that holds a whole group writes its output itself; the others leave (maximum, sum, weighted
// values) records that the merge joins:
//   O = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p,  M = max_p m_p   (scores in base 2).
// Record slot of a piece: (gang + block index in the sequence) H + member.  Gang and block only grow
// along the sequence and one of them does at every piece, so slots are distinct.
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
    int gang;    // H: divides h_kv * nrb and h_kv * nrbp

    __host__ __device__ int blocks_c() const { return h_kv * nrb / gang; }   // lane blocks of a batch
    __host__ __device__ int blocks_p() const { return h_kv * nrbp / gang; }  // of the prefix
};

// The largest gang that leaves at most 3% of the CTAs without one.
inline int span_gang(const SpanShape& p, int ctas) {
    for (int H = p.h_kv * p.nrb; H > 1; --H)
        if (p.h_kv * p.nrb % H == 0 && p.h_kv * p.nrbp % H == 0 && ctas / H * H * 100 >= ctas * 97) return H;
    return 1;
}

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

// Gangs that share N tiles when G are launched: each of them holds at least one.
__host__ __device__ inline int span_parts(int N, int G) { return N < G ? N : G; }

// Gangs [c0, c1] that hold tiles [t0, t1) of N when G divide them.
__device__ __forceinline__ void span_gangs(int N, int G, int t0, int t1, int& c0, int& c1) {
    const int64_t D = span_parts(N, G);
    c0 = (int)(((t0 + 1) * D - 1) / N);
    c1 = (int)((t1 * D - 1) / N);
}

// Tiles of one lane's sequence if every batch had the longest cache (the host checks that they fit 32
// bits and launches no more gangs).
template <int TILE>
inline int64_t span_most_tiles(const SpanShape& p) {
    const int64_t all = ((int64_t)p.T_max + TILE - 1) / TILE;
    const int64_t win = ((int64_t)p.sinks + TILE - 1) / TILE + ((int64_t)p.window + p.T_q - 1 + TILE - 1) / TILE;
    return (int64_t)span_prefix_tiles<TILE>(p) * p.blocks_p() + (int64_t)p.B * p.blocks_c() * (all < win ? all : win);
}

// Where a gang starts in the tile sequence.
struct SpanStart {
    int N;       // tiles in all
    int t0, t1;  // this gang's tiles
    int b;       // batch that holds the gang's first tile past the prefix
    int off;     // first tile of that batch's lane blocks
};

// The sequence as seen from its prefix sums over the batches: all lanes of a warp call it and get N, the
// batch that holds tile want(N) (of the batches' own tiles) and that batch's first tile.  A lane sums a
// run of consecutive batches; loads only, no block-wide step.
template <int TILE, typename F>
__device__ __forceinline__ void span_find(const SpanShape& p, const int32_t* lengths, F want, int& N, int& b, int& off) {
    const int lane = (int)threadIdx.x & 31;
    const int run = (p.B + 31) / 32, i0 = lane * run, i1 = min(p.B, i0 + run);
    const int npt = span_prefix_tiles<TILE>(p) * p.blocks_p();
    int sum = 0;
    for (int i = i0; i < i1; ++i) sum += span_view<TILE>(p, lengths[i]).nt * p.blocks_c();
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    N = npt + __shfl_sync(0xffffffffu, inc, 31);
    const int t = want(N);
    int before = npt + inc - sum, found = 0;
    const bool mine = before <= t && t < before + sum;
    if (mine)
        for (int i = i0; i < i1; ++i) {
            const int n = span_view<TILE>(p, lengths[i]).nt * p.blocks_c();
            if (t < before + n) {
                found = i;
                break;
            }
            before += n;
        }
    const unsigned who = __ballot_sync(0xffffffffu, mine);
    const int src = who ? __ffs(who) - 1 : 0;
    b = __shfl_sync(0xffffffffu, found, src);
    off = __shfl_sync(0xffffffffu, before, src);
}

// This gang's share of the sequence; all lanes of a warp call it.
template <int TILE>
__device__ __forceinline__ SpanStart span_start(const SpanShape& p, const int32_t* lengths) {
    const int gangs = (int)gridDim.x / p.gang, c = (int)blockIdx.x / p.gang;
    const int npt = span_prefix_tiles<TILE>(p) * p.blocks_p();
    SpanStart s;
    span_find<TILE>(p, lengths, [&](int N) {
        const int D = span_parts(N, gangs);
        s.t0 = c < D ? (int)((int64_t)N * c / D) : N;
        s.t1 = c < D ? (int)((int64_t)N * (c + 1) / D) : N;
        return max(s.t0, npt);
    }, s.N, s.b, s.off);
    return s;
}

// One contiguous run of tiles within one group.
struct SpanPiece {
    bool prefix;
    int b, g, rb;
    int block;   // lane block's index in the sequence
    int i0, i1;  // tiles [i0, i1) of the group
    SpanView v;  // the batch's view (prefix: L = T_p, one range)
    __device__ bool whole() const { return i0 == 0 && i1 == v.nt; }
};

// Walks a gang's pieces in order.
template <int TILE>
struct SpanWalk {
    const SpanShape& p;
    const int32_t* lengths;
    int t, t1, off, b;

    __device__ SpanWalk(const SpanShape& p_, const int32_t* lengths_, const SpanStart& s)
        : p(p_), lengths(lengths_), t(s.t0), t1(s.t1), off(s.off), b(s.b) {}

    __device__ bool next(SpanPiece& q) {
        if (t >= t1) return false;
        const int np = span_prefix_tiles<TILE>(p);
        const int member = (int)blockIdx.x % p.gang;
        int in;  // tile within the group
        int lane;
        if (t < np * p.blocks_p()) {
            q.prefix = true;
            q.block = t / np;
            in = t - q.block * np;
            q.b = 0;
            lane = q.block * p.gang + member;
            q.g = lane / p.nrbp;
            q.rb = lane - q.g * p.nrbp;
            q.v.L = p.T_p;
            q.v.s_keys = q.v.lo = q.v.nst = 0;
            q.v.nt = np;
        } else {
            q.prefix = false;
            q.v = span_view<TILE>(p, lengths[b]);
            while (t - off >= q.v.nt * p.blocks_c()) {  // the next batch (some hold no tile)
                off += q.v.nt * p.blocks_c();
                ++b;
                q.v = span_view<TILE>(p, lengths[b]);
            }
            const int bl = (t - off) / q.v.nt;
            in = t - off - bl * q.v.nt;
            q.b = b;
            lane = bl * p.gang + member;
            q.g = lane / p.nrb;
            q.rb = lane - q.g * p.nrb;
            q.block = p.blocks_p() + b * p.blocks_c() + bl;
        }
        q.i0 = in;
        q.i1 = t1 - t < q.v.nt - in ? in + t1 - t : q.v.nt;
        t += q.i1 - q.i0;
        return true;
    }
};

}  // namespace mha
