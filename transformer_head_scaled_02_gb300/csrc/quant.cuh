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

// The cache tokens [first, first + n) that rows 0 .. n - 1 of batch b stand for.
struct QuantRows {
    int first, n;
    bool valid;
};
__device__ __forceinline__ QuantRows quant_rows(int L, int n, int most, int T_max) {
    QuantRows r;
    r.valid = n >= 0 && n <= most && n <= L && L <= T_max;
    r.n = n;
    r.first = L - n;
    return r;
}

__device__ __forceinline__ float quant_step(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float quant_lowest(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

// How a decode step is cut (host and device compute the same).  The query rows that share a cached head are taken
// `rb` at a time; each batch's tokens are cut into at most `splits` equal parts of whole 64s.
struct QuantStep {
    int B, h_kv, per, T_q, T_max;
    int rows;    // per * T_q: query rows of a cached head
    int rb, nrb; // rows of a row block; row blocks
    int splits;
    __host__ __device__ int part(int L) const { return ((L + splits - 1) / splits + 63) / 64 * 64; }
};

}  // namespace mha
