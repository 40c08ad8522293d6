// evict.cu -- eviction from a KV cache by accumulated attention weight: per (batch, K/V head) keep the
// last `recent` tokens and, of the earlier ones, the keep - recent of largest weight (ties: the lowest
// index), then move their K, V and weight rows together in their order.
//
//   evict_select_kernel   one block per (batch, K/V head).  The weights as order-preserving 32-bit
//                         keys, in shared memory where they fit, so that they are read once; the
//                         keep - recent largest are found by radix selection (digits of 11, 11 and 10
//                         bits: a histogram of the keys that agree with the digits fixed so far), which
//                         gives the smallest kept key and how many tokens equal to it are kept; two
//                         counts in index order (ballots, one block-wide scan each) then number the
//                         kept tokens.  Bound by latency: a few block-wide steps per block.
//   evict_move_kernel     row copies, bound by HBM: kept rows are read and written once.
//
// 32 caches of up to 8192 tokens cut to 2048, 16 K/V heads of d = 128: 212 us, 163 at the measured copy rate;
// the moves run at it, the selections add 30 us and HBM drains the last moves' writes under them.  Both in one
// kernel, tasks taken in order from a counter and the moves waiting for their batch's selections, took 295 us
// (and two caches of 1000 tokens 15 us instead of 8): a task's chain of ticket, wait, marks, rows and stores
// left less in flight than many short blocks do.
// In place (evict_move_inplace_kernel) the same caches take 248 us where new buffers take 217, each call by itself.
#include <math.h>

#include "internal.h"
#include "ptx.cuh"

namespace mha {
namespace {

constexpr int EV_THREADS = 512;
constexpr int EV_WARPS = EV_THREADS / 32;
constexpr int EV_BINS = 2048;
// Tokens per scan: every warp counts 32 at a time, EV_STEPS times.
constexpr int EV_STEPS = 32;
constexpr int EV_SCAN = EV_THREADS * EV_STEPS;
// Tokens whose keys fit shared memory beside the histogram and the counts.
constexpr int EV_SMEM_TOKENS = 48 * 1024;

// Ascending keys for ascending weights; NaN below everything, -0 equal to +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (isnan(w)) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Exclusive sum over the block of one value per thread; total: the whole sum.  Two barriers.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
    const int lane = (int)threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    const int s = lane < EV_WARPS ? warp_sums[lane] : 0;
    int ws = s;
#pragma unroll
    for (int o = 1; o < EV_WARPS; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, ws, o);
        if (lane >= o) ws += u;
    }
    total = __shfl_sync(0xffffffffu, ws, EV_WARPS - 1);
    const int before = __shfl_sync(0xffffffffu, ws - s, warp);
    __syncthreads();
    return before + inc - v;
}

// KEYS: the keys fit shared memory (T_max <= EV_SMEM_TOKENS); otherwise every pass reads the weights.
template <bool KEYS>
__global__ void __launch_bounds__(EV_THREADS)
    evict_select_kernel(int T_max, int h_kv, int keep, int recent, const int32_t* __restrict__ lengths,
                        const float* weights, int32_t* __restrict__ kept, float* weights_out, int T_out,
                        int* status) {
    extern __shared__ uint32_t keys_s[];
    __shared__ int hist[EV_BINS];
    __shared__ int warp_sums[EV_WARPS];
    __shared__ int digit_s, need_s, count_s;
    __shared__ int16_t counts[EV_STEPS * EV_WARPS];  // of 32 tokens each
    __shared__ int base[EV_STEPS * EV_WARPS];
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
    auto key = [&](int j) { return KEYS ? keys_s[j] : weight_key(w[j]); };
    // radix selection: `prefix` holds the digits fixed so far, `need` how many of the keys that agree
    // with them are kept, `equal` how many there are
    int need = keep - recent, equal = 0;
    uint32_t prefix = 0u, fixed = 0u;
#pragma unroll 1
    for (int shift = 21; shift >= 0 && need > 0; shift = shift == 21 ? 10 : shift == 10 ? 0 : -1) {
        const uint32_t mask = shift == 0 ? 1023u : 2047u;
        for (int i = tid; i < EV_BINS; i += EV_THREADS) hist[i] = 0;
        __syncthreads();
        if (!KEYS || shift == 21) {  // from the weights
#pragma unroll 4
            for (int j = tid; j < n_early; j += EV_THREADS) {
                const uint32_t k = weight_key(w[j]);
                if constexpr (KEYS) keys_s[j] = k;
                if ((k & fixed) == prefix) atomicAdd(&hist[(k >> shift) & mask], 1);
            }
        } else {
#pragma unroll 4
            for (int j = tid; j < n_early; j += EV_THREADS) {
                const uint32_t k = keys_s[j];
                if ((k & fixed) == prefix) atomicAdd(&hist[(k >> shift) & mask], 1);
            }
        }
        __syncthreads();
        // thread i: digits from the top down; the digit where the running count reaches need
        constexpr int PER = EV_BINS / EV_THREADS;
        int c[PER], sum = 0, total;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            c[i] = hist[EV_BINS - 1 - PER * tid - i];
            sum += c[i];
        }
        int before = block_scan(sum, warp_sums, total);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (before < need && need <= before + c[i]) {
                digit_s = EV_BINS - 1 - PER * tid - i;
                need_s = need - before;
                count_s = c[i];
            }
            before += c[i];
        }
        __syncthreads();
        prefix |= (uint32_t)digit_s << shift;
        fixed |= mask << shift;
        need = need_s;
        equal = count_s;
    }
    // Tokens above `prefix` are kept and the first `need` of those equal to it (keep == recent: none).
    // Numbering in index order, EV_SCAN tokens at a time: the ballots of 32 tokens each are counted, the
    // counts scanned over the block, the places read back.
    const bool any = keep > recent;
    int eq_base = 0, keep_base = 0;
    for (int j0 = 0; j0 < L; j0 += EV_SCAN) {
        const int steps = min(EV_STEPS, (L - j0 + EV_THREADS - 1) / EV_THREADS);
        // places of the first token of each 32, counting those that f says; bit i of the result: what f says of
        // this thread's token of step i
        auto number = [&](auto f, int& sum) {
            uint32_t mine = 0u;
#pragma unroll 4
            for (int i = 0; i < steps; ++i) {
                const bool is = f(i, j0 + i * EV_THREADS + tid);
                const unsigned m = __ballot_sync(0xffffffffu, is);
                mine |= is ? 1u << i : 0u;
                if (lane == 0) counts[i * EV_WARPS + warp] = (int16_t)__popc(m);
            }
            __syncthreads();
            int at = tid < steps * EV_WARPS ? counts[tid] : 0;  // EV_STEPS * EV_WARPS == EV_THREADS
            at = block_scan(at, warp_sums, sum);
            base[tid] = at;
            __syncthreads();
            return mine;
        };
        static_assert(EV_STEPS * EV_WARPS == EV_THREADS, "one count per thread");
        uint32_t eq_taken = 0u;  // bit i: this thread's token of step i is equal and among the first `need`
        if (any && need < equal) {
            int sum;
            const uint32_t eq = number([&](int, int j) { return j < n_early && key(j) == prefix; }, sum);
            for (int i = 0; i < steps; ++i) {
                const bool e = (eq >> i) & 1u;
                const unsigned m = __ballot_sync(0xffffffffu, e);
                if (e && eq_base + base[i * EV_WARPS + warp] + __popc(m & ((1u << lane) - 1u)) < need) eq_taken |= 1u << i;
            }
            eq_base += sum;
            __syncthreads();  // base is about to be overwritten
        } else if (any) {
            eq_taken = 0xFFFFFFFFu;
        }
        auto taken = [&](int i, int j) {
            if (j >= L) return false;
            if (j >= n_early) return true;
            const uint32_t k = key(j);
            return any && (k > prefix || (k == prefix && ((eq_taken >> i) & 1u)));
        };
        int sum;
        const uint32_t mine = number(taken, sum);
        // in place: a token's place is at most its index, every weight up to j0 has been read, and
        // those of some steps are read by all before any of theirs is written
        constexpr int AT_ONCE = 8;
        for (int i0 = 0; i0 < steps; i0 += AT_ONCE) {
            float wj[AT_ONCE];
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i)
                if ((mine >> (i0 + i)) & 1u) wj[i] = w[j0 + (i0 + i) * EV_THREADS + tid];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                const bool t = (mine >> (i0 + i)) & 1u;
                const unsigned m = __ballot_sync(0xffffffffu, t);
                if (t) {
                    const int at = keep_base + base[(i0 + i) * EV_WARPS + warp] + __popc(m & ((1u << lane) - 1u));
                    out[at] = j0 + (i0 + i) * EV_THREADS + tid;
                    w_out[at] = wj[i];
                }
            }
        }
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
                // (unsigned: h_kv * keep may pass 2^31, but not 2^32, which the host checks; a 64-bit product takes
                // the kernel from 64 to 67 registers, from four blocks an SM to three, and 211 us to 233)
                const int from = at[(uint32_t)g * (uint32_t)keep + (uint32_t)(i0 + row)];
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
    // up to 32 KB of a side's rows per block (every thread keeps MV_ROUNDS pieces in flight), less where
    // that would leave SMs without a block
    const int64_t row_bytes = (int64_t)(k.head_bytes > v.head_bytes ? k.head_bytes : v.head_bytes) * h_kv;
    int64_t rpb = 32768 / (row_bytes > 32768 ? 32768 : row_bytes);
    const int64_t spread = ((int64_t)keep * B * 2 + 1023) / 1024;
    if (rpb > spread) rpb = spread < 1 ? 1 : spread;
    return launch_pdl(evict_move_kernel<UNIT>, dim3((unsigned)((keep + rpb - 1) / rpb), (unsigned)B, 2),
                      dim3(MV_THREADS), 0, stream, k, v, T_max, T_out, h_kv, keep, kept, new_lengths, (int)rpb);
}

}  // namespace

cudaError_t launch_evict(const void* K, int64_t ldk, const void* V, int64_t ldv, void* Ko, int64_t ldko, void* Vo,
                         int64_t ldvo, int elem, int B, int h_kv, int T_max, int T_out, int d_k, int d_v, int keep,
                         int recent, const int32_t* lengths, const float* weights, float* weights_out,
                         int32_t* kept, int32_t* new_lengths, int* status, cudaStream_t stream) {
    const bool keys = T_max <= EV_SMEM_TOKENS;
    auto select = keys ? evict_select_kernel<true> : evict_select_kernel<false>;
    const size_t smem = keys ? (size_t)T_max * sizeof(uint32_t) : 0;
    cudaError_t err = cudaSuccess;
    // past what a launch gets unasked (with the static 11 KB).  The limit belongs to the process, where another
    // thread may be launching a larger selection: always the largest
    if (smem > 32 * 1024)
        err = cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize, EV_SMEM_TOKENS * (int)sizeof(uint32_t));
    if (err != cudaSuccess) return err;
    err = launch_pdl(select, dim3((unsigned)(B * h_kv)), dim3(EV_THREADS), smem, stream, T_max, h_kv, keep, recent, lengths,
                     weights, kept, weights_out, T_out, status);
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
