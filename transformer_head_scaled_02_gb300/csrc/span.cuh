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

// Ending a piece (joining its streams, writing its rows, starting the next) takes about as long as a tile:
// every group occupies that many places more in the sequence than it has tiles, so that a gang with many
// short groups gets fewer tiles.  Nothing is read for those places.
constexpr int kSpanPieceCost = 1;

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
    __host__ __device__ int places() const { return nt > 0 ? nt + kSpanPieceCost : 0; }  // in the sequence
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

// Places of the sequence that the prefix's groups take.
template <int TILE>
__host__ __device__ inline int span_prefix_places(const SpanShape& p) {
    return p.T_p > 0 ? (span_prefix_tiles<TILE>(p) + kSpanPieceCost) * p.blocks_p() : 0;
}

// Gangs that share N tiles when G are launched: each of them holds at least one.
__host__ __device__ inline int span_parts(int N, int G) { return N < G ? N : G; }

// a * b / c, in 32 bits where the product fits (a 64-bit division costs several hundred cycles)
__device__ __forceinline__ int span_muldiv(int a, int b, int add, int c) {
    if (a < (1 << 21) && b <= 1024) return (int)(((unsigned)a * (unsigned)b + (unsigned)add) / (unsigned)c);
    return (int)(((int64_t)a * b + add) / c);
}

// Gangs [c0, c1] that hold places [t0, t1) of N when G divide them.
__device__ __forceinline__ void span_gangs(int N, int G, int t0, int t1, int& c0, int& c1) {
    const int D = span_parts(N, G);
    c0 = span_muldiv(t0, D, D - 1, N);  // ((t0 + 1) D - 1) / N
    c1 = span_muldiv(t1, D, -1, N);
}

// Places of the sequence if every batch had the longest cache (the host checks that they fit 32 bits and
// launches no more gangs).
template <int TILE>
inline int64_t span_most_places(const SpanShape& p) {
    const int64_t all = ((int64_t)p.T_max + TILE - 1) / TILE;
    const int64_t win = ((int64_t)p.sinks + TILE - 1) / TILE + ((int64_t)p.window + p.T_q - 1 + TILE - 1) / TILE;
    const int64_t pre = p.T_p > 0 ? ((int64_t)span_prefix_tiles<TILE>(p) + kSpanPieceCost) * p.blocks_p() : 0;
    return pre + (int64_t)p.B * p.blocks_c() * ((all < win ? all : win) + kSpanPieceCost);
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
    const int npt = span_prefix_places<TILE>(p);
    int sum = 0;
    for (int i = i0; i < i1; ++i) sum += span_view<TILE>(p, lengths[i]).places() * p.blocks_c();
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
            const int n = span_view<TILE>(p, lengths[i]).places() * p.blocks_c();
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
    const int npt = span_prefix_places<TILE>(p);
    SpanStart s;
    span_find<TILE>(p, lengths, [&](int N) {
        const int D = span_parts(N, gangs);
        s.t0 = c < D ? span_muldiv(N, c, 0, D) : N;
        s.t1 = c < D ? span_muldiv(N, c + 1, 0, D) : N;
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

// Walks a gang's pieces in order.  Divisions only at the start: afterwards the walk steps from group to
// group.
template <int TILE>
struct SpanWalk {
    const SpanShape& p;
    const int32_t* lengths;
    int left;   // places left
    int in;     // next place within the current group
    int bl;     // current lane block within its batch (or within the prefix)
    int b;      // current batch; -1: the prefix
    int first;  // first batch after the prefix
    SpanView v;

    __device__ SpanWalk(const SpanShape& p_, const int32_t* lengths_, const SpanStart& s)
        : p(p_), lengths(lengths_), left(s.t1 - s.t0), in(0), bl(0), b(s.b), first(s.b) {
        if (left <= 0) return;
        const int npt = span_prefix_places<TILE>(p);
        int at = s.t0 - s.off;  // within the batch's groups
        if (s.t0 < npt) {
            at = s.t0;
            b = -1;
            prefix_view();
        } else {
            v = span_view<TILE>(p, lengths[b]);
        }
        bl = at / v.places();
        in = at - bl * v.places();
    }

    __device__ void prefix_view() {
        v.L = p.T_p;
        v.s_keys = v.lo = v.nst = 0;
        v.nt = span_prefix_tiles<TILE>(p);
    }

    __device__ void next_batch() {
        bl = 0;
        b = b < 0 ? first : b + 1;
        v = span_view<TILE>(p, lengths[b]);
    }

    // The next piece, or false (and q as it was) at the end.
    __device__ bool next(SpanPiece& q) {
        while (left > 0) {
            if (in == v.places()) {  // the next group; batches without a tile are passed over
                in = 0;
                ++bl;
                if (bl == (b < 0 ? p.blocks_p() : p.blocks_c())) next_batch();
                while (v.nt == 0) next_batch();
            }
            const int i0 = in, end = min(v.places(), in + left);
            left -= end - in;
            in = end;
            if (i0 >= v.nt) continue;
            q.prefix = b < 0;
            q.v = v;
            q.i0 = i0;
            q.i1 = min(v.nt, end);
            q.b = b < 0 ? 0 : b;
            const int lane = bl * p.gang + (int)blockIdx.x % p.gang, nrb = b < 0 ? p.nrbp : p.nrb;
            q.g = nrb == 1 ? lane : lane / nrb;
            q.rb = nrb == 1 ? 0 : lane - q.g * nrb;
            q.block = b < 0 ? bl : p.blocks_p() + b * p.blocks_c() + bl;
            return true;
        }
        return false;
    }
};

}  // namespace mha
