// evict.cu -- eviction from a KV cache by accumulated attention weight: per (batch, K/V head) keep the
// last `recent` tokens and, of the earlier ones, the keep - recent of largest weight (ties: the lowest
// index), then move their K, V and weight rows together in their order.
//
//   evict_select_kernel   one block per (batch, K/V head).  The weights as order-preserving 32-bit
//                         keys; the keep - recent largest are found by radix selection (8 bits at a
//                         time: a histogram of the keys that agree with the digits fixed so far, one
//                         private histogram per warp because most weights share their first digits),
//                         which gives the smallest kept key and how many tokens equal to it are kept;
//                         a pass in index order then numbers the kept tokens (ballots and warp
//                         totals).  Reads the weights six times, from L2 after the first.
//   evict_move_kernel     row copies, bound by HBM: kept rows are read and written once.
#include <math.h>

#include "internal.h"
#include "ptx.cuh"

namespace mha {
namespace {

constexpr int EV_THREADS = 1024;
constexpr int EV_WARPS = EV_THREADS / 32;

// Ascending keys for ascending weights; NaN below everything, -0 equal to +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (isnan(w)) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(EV_THREADS)
    evict_select_kernel(int T_max, int h_kv, int keep, int recent, const int32_t* __restrict__ lengths,
                        const float* weights, int32_t* __restrict__ kept, float* weights_out, int T_out,
                        int* status) {
    __shared__ uint32_t hist[EV_WARPS][256];
    __shared__ uint32_t total[256];
    __shared__ uint32_t digit_s, need_s;
    __shared__ int warp_eq[EV_WARPS], warp_keep[EV_WARPS];
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bg = (int)blockIdx.x, b = bg / h_kv;
    const int L = lengths[b];
    int32_t* out = kept + (int64_t)bg * keep;
    const float* w = weights + (int64_t)bg * T_max;
    float* w_out = weights_out + (int64_t)bg * T_out;
    if (L < 0 || L > T_max) {
        if (tid == 0) record_status(status, kStatusBadLength);
        for (int i = tid; i < keep; i += EV_THREADS) out[i] = -1;
        return;
    }
    if (L <= keep) {
        for (int i = tid; i < keep; i += EV_THREADS) {
            out[i] = i < L ? i : -1;
            if (i < L) w_out[i] = w[i];  // the same entry when in place
        }
        return;
    }
    const int n_early = L - recent;  // > keep - recent >= 0
    uint32_t need = (uint32_t)(keep - recent), prefix = 0u;
    // radix selection: prefix holds the digits fixed so far, need the rank left within them
    for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
        for (int i = tid; i < EV_WARPS * 256; i += EV_THREADS) (&hist[0][0])[i] = 0u;
        __syncthreads();
        const uint32_t fixed = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
        for (int j = tid; j < n_early; j += EV_THREADS) {
            const uint32_t k = weight_key(w[j]);
            if ((k & fixed) == prefix) atomicAdd(&hist[warp][(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (tid < 256) {
            uint32_t s = 0;
#pragma unroll
            for (int q = 0; q < EV_WARPS; ++q) s += hist[q][tid];
            total[tid] = s;
        }
        __syncthreads();
        if (warp == 0) {
            // lane l: digits 255 - 8 l down to 248 - 8 l; the digit where the running count reaches need
            uint32_t c[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = total[255 - 8 * lane - i];
                sum += c[i];
            }
            uint32_t inc = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += u;
            }
            uint32_t before = inc - sum;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (before < need && need <= before + c[i]) {
                    digit_s = (uint32_t)(255 - 8 * lane - i);
                    need_s = need - before;
                }
                before += c[i];
            }
        }
        __syncthreads();
        prefix |= digit_s << shift;
        need = need_s;
    }
    // tokens above `prefix` are kept, and the first `need` of those equal to it (none if keep == recent)
    const bool any = keep > recent;
    int eq_base = 0, keep_base = 0;
    for (int j0 = 0; j0 < L; j0 += EV_THREADS) {
        const int j = j0 + tid;
        const float wj = j < L ? w[j] : 0.f;
        const uint32_t k = j < n_early ? weight_key(wj) : 0u;
        const bool eq = any && j < n_early && k == prefix;
        const uint32_t eq_mask = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) warp_eq[warp] = __popc(eq_mask);
        __syncthreads();
        int eq_rank = eq_base + __popc(eq_mask & ((1u << lane) - 1u)), eq_sum = 0;
#pragma unroll
        for (int q = 0; q < EV_WARPS; ++q) {
            if (q < warp) eq_rank += warp_eq[q];
            eq_sum += warp_eq[q];
        }
        const bool take = j < L && (j >= n_early || (any && (k > prefix || (eq && eq_rank < (int)need))));
        const uint32_t mask = __ballot_sync(0xffffffffu, take);
        if (lane == 0) warp_keep[warp] = __popc(mask);
        __syncthreads();
        int at = keep_base + __popc(mask & ((1u << lane) - 1u)), sum = 0;
#pragma unroll
        for (int q = 0; q < EV_WARPS; ++q) {
            if (q < warp) at += warp_keep[q];
            sum += warp_keep[q];
        }
        // in place: at <= j, and every entry up to this block of tokens has been read
        if (take) {
            out[at] = j;
            w_out[at] = wj;
        }
        eq_base += eq_sum;
        keep_base += sum;
        __syncthreads();
    }
}

// Rows [i0, i0 + n) of one column slice: U units per row, one unit per thread and round.
struct MoveSide {
    const uint8_t* src;
    uint8_t* dst;
    int64_t ld_src, ld_dst;  // bytes
    int head_bytes;
};

constexpr int MV_THREADS = 256;
constexpr int MV_ROUNDS = 8;  // rows in flight per thread

// Out of place: block = (row block, batch, side); a thread copies unit (row, head, column).
template <typename UNIT>
__global__ void __launch_bounds__(MV_THREADS)
    evict_move_kernel(MoveSide k, MoveSide v, int T_max, int T_out, int h_kv, int keep,
                      const int32_t* __restrict__ kept, int32_t* __restrict__ new_lengths, int rows_per_block) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int b = (int)blockIdx.y;
    const MoveSide s = blockIdx.z == 0 ? k : v;
    const int32_t* at = kept + (int64_t)b * h_kv * keep;
    if (blockIdx.x == 0 && blockIdx.z == 0)
        for (int i = (int)threadIdx.x; i <= keep; i += MV_THREADS)  // the valid entries come first
            if ((i == 0 || at[i - 1] >= 0) && (i == keep || at[i] < 0)) new_lengths[b] = i;
    const int upr = s.head_bytes / (int)sizeof(UNIT) * h_kv;  // units per row
    const int uph = s.head_bytes / (int)sizeof(UNIT);
    const int i0 = (int)blockIdx.x * rows_per_block;
    const int total = min(rows_per_block, keep - i0) * upr;
    for (int u0 = (int)threadIdx.x; u0 < total; u0 += MV_THREADS * MV_ROUNDS) {
        UNIT x[MV_ROUNDS];
        int64_t to[MV_ROUNDS];
#pragma unroll
        for (int r = 0; r < MV_ROUNDS; ++r) {
            const int u = u0 + r * MV_THREADS;
            to[r] = -1;
            if (u < total) {
                const int row = u / upr, c = u - row * upr, g = c / uph;
                const int from = at[g * keep + i0 + row];
                if (from >= 0) {
                    to[r] = ((int64_t)b * T_out + i0 + row) * s.ld_dst + (int64_t)c * sizeof(UNIT);
                    x[r] = *reinterpret_cast<const UNIT*>(s.src + ((int64_t)b * T_max + from) * s.ld_src + (int64_t)c * sizeof(UNIT));
                }
            }
        }
#pragma unroll
        for (int r = 0; r < MV_ROUNDS; ++r)
            if (to[r] >= 0) *reinterpret_cast<UNIT*>(s.dst + to[r]) = x[r];
    }
}

// In place: block = (column slice of one head, batch, side), rows in order: a round's rows are all
// read before any of them is written, and no row is written past the one it came from, so a later
// round's rows are still there.
constexpr int MV_SLICE = 4;  // units per row of a slice

template <typename UNIT>
__global__ void __launch_bounds__(MV_THREADS)
    evict_move_inplace_kernel(MoveSide k, MoveSide v, int T_max, int h_kv, int keep,
                              const int32_t* __restrict__ kept, int32_t* __restrict__ new_lengths) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int b = (int)blockIdx.y;
    const MoveSide s = blockIdx.z == 0 ? k : v;
    const int uph = s.head_bytes / (int)sizeof(UNIT);
    const int slices = (uph + MV_SLICE - 1) / MV_SLICE;  // of this side
    const int32_t* at0 = kept + (int64_t)b * h_kv * keep;
    if (blockIdx.x == 0 && blockIdx.z == 0)
        for (int i = (int)threadIdx.x; i <= keep; i += MV_THREADS)
            if ((i == 0 || at0[i - 1] >= 0) && (i == keep || at0[i] < 0)) new_lengths[b] = i;
    const int g = (int)blockIdx.x / slices, sl = (int)blockIdx.x - g * slices;
    if (g >= h_kv) return;  // the other side has more slices
    const int32_t* at = at0 + (int64_t)g * keep;
    const int c = sl * MV_SLICE + (int)threadIdx.x % MV_SLICE;
    const bool col = c < uph;
    const int64_t cb = (int64_t)(g * uph + c) * sizeof(UNIT);
    constexpr int ROWS = MV_THREADS / MV_SLICE;
    for (int i0 = (int)threadIdx.x / MV_SLICE; ; i0 += ROWS * MV_ROUNDS) {
        UNIT x[MV_ROUNDS];
        bool has[MV_ROUNDS];
#pragma unroll
        for (int r = 0; r < MV_ROUNDS; ++r) {
            const int i = i0 + r * ROWS;
            const int from = col && i < keep ? at[i] : -1;
            has[r] = from > i;  // the others stay where they are
            if (has[r]) x[r] = *reinterpret_cast<const UNIT*>(s.src + ((int64_t)b * T_max + from) * s.ld_src + cb);
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < MV_ROUNDS; ++r)
            if (has[r]) *reinterpret_cast<UNIT*>(s.dst + ((int64_t)b * T_max + i0 + r * ROWS) * s.ld_dst + cb) = x[r];
        if (i0 - (int)threadIdx.x / MV_SLICE + ROWS * MV_ROUNDS >= keep) break;  // block-uniform
    }
}

template <typename UNIT>
cudaError_t move(const MoveSide& k, const MoveSide& v, int B, int T_max, int T_out, int h_kv, int keep, bool in_place,
                 const int32_t* kept, int32_t* new_lengths, cudaStream_t stream) {
    if (in_place) {
        const int widest = (k.head_bytes > v.head_bytes ? k.head_bytes : v.head_bytes) / (int)sizeof(UNIT);
        return launch_pdl(evict_move_inplace_kernel<UNIT>,
                          dim3((unsigned)(h_kv * ((widest + MV_SLICE - 1) / MV_SLICE)), (unsigned)B, 2),
                          dim3(MV_THREADS), 0, stream, k, v, T_max, h_kv, keep, kept, new_lengths);
    }
    // about 64 KB of a side's rows per block
    const int64_t row_bytes = (int64_t)k.head_bytes * h_kv;
    int rpb = (int)(65536 / (row_bytes > 65536 ? 65536 : row_bytes));
    if (rpb > keep) rpb = keep;
    return launch_pdl(evict_move_kernel<UNIT>, dim3((unsigned)((keep + rpb - 1) / rpb), (unsigned)B, 2),
                      dim3(MV_THREADS), 0, stream, k, v, T_max, T_out, h_kv, keep, kept, new_lengths, rpb);
}

}  // namespace

cudaError_t launch_evict(const void* K, int64_t ldk, const void* V, int64_t ldv, void* Ko, int64_t ldko, void* Vo,
                         int64_t ldvo, int elem, int B, int h_kv, int T_max, int T_out, int d_k, int d_v, int keep,
                         int recent, const int32_t* lengths, const float* weights, float* weights_out,
                         int32_t* kept, int32_t* new_lengths, int* status, cudaStream_t stream) {
    cudaError_t err = launch_pdl(evict_select_kernel, dim3((unsigned)(B * h_kv)), dim3(EV_THREADS), 0, stream, T_max,
                                 h_kv, keep, recent, lengths, weights, kept, weights_out, T_out, status);
    if (err != cudaSuccess) return err;
    const MoveSide k{static_cast<const uint8_t*>(K), static_cast<uint8_t*>(Ko), ldk * elem, ldko * elem, d_k * elem};
    const MoveSide v{static_cast<const uint8_t*>(V), static_cast<uint8_t*>(Vo), ldv * elem, ldvo * elem, d_v * elem};
    auto mult16 = [](const MoveSide& s) {
        return ((reinterpret_cast<uintptr_t>(s.src) | reinterpret_cast<uintptr_t>(s.dst) | (uintptr_t)s.ld_src |
                 (uintptr_t)s.ld_dst | (uintptr_t)s.head_bytes) & 15u) == 0;
    };
    const bool in_place = K == Ko;
    if (mult16(k) && mult16(v))
        return move<uint4>(k, v, B, T_max, T_out, h_kv, keep, in_place, kept, new_lengths, stream);
    return move<uint32_t>(k, v, B, T_max, T_out, h_kv, keep, in_place, kept, new_lengths, stream);  // fp32
}

}  // namespace mha
