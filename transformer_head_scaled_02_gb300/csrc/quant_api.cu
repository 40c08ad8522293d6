// quant_api.cu -- the C ABI of the quantised key/value cache (include/mha.h): its size and layout, writing, reading
// back, and the decode step over it.  Host checks and launches; nothing is allocated or synchronised here.
#include <stdint.h>

#include "../../include/mha.h"
#include "api_util.h"
#include "internal.h"
#include "quant.cuh"

using namespace mha;

namespace {

struct Cache {
    QuantPlane k, v;
    size_t off[4], bytes;
};

bool cache_sizes_ok(const mha_s* m, int bits, int B, int T_max) {
    return (bits == 4 || bits == 8) && B >= 0 && T_max >= 0 && T_max % kQuantTokens == 0 &&
           (int64_t)B * T_max <= kMostRows && (int64_t)B * m->h_kv <= INT32_MAX;
}

Cache cache_layout(const mha_s* m, int bits, int B, int T_max, void* base) {
    Cache c;
    const size_t rows = (size_t)B * m->h_kv * (size_t)T_max;
    uint8_t* p = static_cast<uint8_t*>(base);
    size_t at = 0;
    auto plane = [&](int d, int i) {
        QuantPlane x;
        x.d = d;
        x.row = quant_row_bytes(d, bits);
        x.groups = quant_groups(d);
        c.off[i] = at;
        at += align256(rows * (size_t)x.row);
        c.off[i + 1] = at;
        at += align256(rows * (size_t)x.groups * 4);
        x.codes = p + c.off[i];
        x.params = reinterpret_cast<uint32_t*>(p + c.off[i + 1]);
        return x;
    };
    c.k = plane(m->dk, 0);
    c.v = plane(m->dv, 2);
    c.bytes = at;
    return c;
}

mha_status shape_supported(const mha_s* m) {
    if (m->dtype == MHA_BF16) return bf16_shape_supported(m) ? MHA_OK : MHA_ERR_UNSUPPORTED;
    return m->dk <= 256 && m->dv <= 256 ? MHA_OK : MHA_ERR_UNSUPPORTED;
}

size_t extent(int64_t rows, int64_t ld, int64_t width, size_t elem) {
    return rows > 0 ? ((size_t)(rows - 1) * (size_t)ld + (size_t)width) * elem : 0;
}

bool rows_ok(const mha_s* m, const void* p, int64_t ld, int64_t width) {
    if (p == nullptr || ld < width) return false;
    return m->dtype != MHA_BF16 || (ld % 8 == 0 && aligned16(p));
}

bool cache_ptr_ok(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

mha_status copy(mha_s* m, bool write, int bits, int B, int T_max, const void* cache, int T, const void* K, int64_t ldk,
                const void* V, int64_t ldv, const int32_t* lengths, const int32_t* counts, void* stream) {
    if (m == nullptr || !cache_sizes_ok(m, bits, B, T_max) || T < 0 || (int64_t)B * T > kMostRows) return MHA_ERR_INVALID_ARG;
    const mha_status sup = shape_supported(m);
    if (sup != MHA_OK) return sup;
    if (B == 0 || T == 0) return MHA_OK;
    const Widths wd = widths(m);
    if (T_max == 0 || !cache_ptr_ok(cache) || lengths == nullptr || !rows_ok(m, K, ldk, wd.k) || !rows_ok(m, V, ldv, wd.v))
        return MHA_ERR_INVALID_ARG;
    const Cache c = cache_layout(m, bits, B, T_max, const_cast<void*>(cache));
    const size_t s = elem_bytes(m->dtype);
    const int64_t n = (int64_t)B * T;
    const size_t kb = extent(n, ldk, wd.k, s), vb = extent(n, ldv, wd.v, s), ib = (size_t)B * sizeof(int32_t);
    if (overlaps(cache, c.bytes, K, kb) || overlaps(cache, c.bytes, V, vb)) return MHA_ERR_INVALID_ARG;
    if (write) {
        if (overlaps(cache, c.bytes, lengths, ib) || overlaps(cache, c.bytes, counts, ib)) return MHA_ERR_INVALID_ARG;
    } else {
        if (overlaps(lengths, ib, K, kb) || overlaps(lengths, ib, V, vb) || overlaps(counts, ib, K, kb) || overlaps(counts, ib, V, vb))
            return MHA_ERR_INVALID_ARG;
        // K and V may be column views of one buffer: their rows interleave
        if (overlaps(K, kb, V, vb)) {
            const int64_t ld = ldk * (int64_t)s, d = static_cast<const uint8_t*>(V) - static_cast<const uint8_t*>(K);
            const int64_t col = ((d % ld) + ld) % ld;  // V's first column, K's at 0
            if (ldk != ldv || col < wd.k * (int64_t)s || col + wd.v * (int64_t)s > ld) return MHA_ERR_INVALID_ARG;
        }
    }
    if (!quant_copy_fits(write, m->dtype == MHA_F32, c.k, c.v, B, T, m->h_kv)) return MHA_ERR_UNSUPPORTED;
    const cudaError_t err = launch_quant_copy(write, m->dtype == MHA_F32, bits, c.k, c.v, const_cast<void*>(K), ldk,
                                              const_cast<void*>(V), ldv, B, T, T_max, m->h_kv, lengths, counts,
                                              status_ptr(m), static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

bool step_sizes_ok(const mha_s* m, int B, int T_q, int T_max) {
    return T_q >= 0 && (int64_t)B * m->h * T_q <= kMostRows;
}

QuantStep step_shape(const mha_s* m, int bits, int B, int T_q, int T_max, int sms) {
    return quant_step_shape(m->dtype == MHA_F32, bits, m->dk, m->dv, B, m->h, m->h_kv, T_q, T_max, sms);
}

}  // namespace

extern "C" {

size_t mha_quant_cache_size(mha_t handle, int bits, int B, int T_max, size_t* offsets) {
    if (handle == nullptr || !cache_sizes_ok(handle, bits, B, T_max)) return 0;
    const Cache c = cache_layout(handle, bits, B, T_max, nullptr);
    if (offsets != nullptr)
        for (int i = 0; i < 4; ++i) offsets[i] = c.off[i];
    return c.bytes;
}

mha_status mha_quant_write(mha_t handle, int bits, int B, int T_max, void* cache, int T_new, const void* K, int64_t ldk,
                           const void* V, int64_t ldv, const int32_t* cache_lengths, const int32_t* counts, void* stream) {
    return copy(handle, true, bits, B, T_max, cache, T_new, K, ldk, V, ldv, cache_lengths, counts, stream);
}

mha_status mha_quant_read(mha_t handle, int bits, int B, int T_max, const void* cache, int T_out, void* K, int64_t ldk,
                          void* V, int64_t ldv, const int32_t* cache_lengths, const int32_t* counts, void* stream) {
    return copy(handle, false, bits, B, T_max, cache, T_out, K, ldk, V, ldv, cache_lengths, counts, stream);
}

size_t mha_decode_quant_workspace_size(mha_t handle, int B, int T_q, int T_max) {
    if (handle == nullptr || !cache_sizes_ok(handle, 4, B, T_max) || !step_sizes_ok(handle, B, T_q, T_max)) return 0;
    if (B == 0 || T_q == 0 || T_max == 0) return kStatusBytes;
    const size_t four = quant_step_bytes(step_shape(handle, 4, B, T_q, T_max, 1)),
                 eight = quant_step_bytes(step_shape(handle, 8, B, T_q, T_max, 1));
    return kStatusBytes + align256(four > eight ? four : eight);
}

mha_status mha_decode_quant(mha_t handle, int bits, int B, int T_q, int T_max, const void* Q, int64_t ldq,
                            const void* cache, const int32_t* cache_lengths, void* O, int64_t ldo, void* stream) {
    const mha_s* m = handle;
    if (m == nullptr || !cache_sizes_ok(m, bits, B, T_max) || !step_sizes_ok(m, B, T_q, T_max)) return MHA_ERR_INVALID_ARG;
    const mha_status sup = shape_supported(m);
    if (sup != MHA_OK) return sup;
    if (B == 0 || T_q == 0) return MHA_OK;
    const Widths wd = widths(m);
    const int64_t hv = (int64_t)m->h * m->dv, n = (int64_t)B * T_q;
    if (T_q > T_max || !cache_ptr_ok(cache) || cache_lengths == nullptr || !rows_ok(m, Q, ldq, wd.q) || !rows_ok(m, O, ldo, hv))
        return MHA_ERR_INVALID_ARG;
    const Cache c = cache_layout(m, bits, B, T_max, const_cast<void*>(cache));
    const size_t s = elem_bytes(m->dtype), ob = extent(n, ldo, hv, s);
    if (overlaps(O, ob, Q, extent(n, ldq, wd.q, s)) || overlaps(O, ob, cache, c.bytes) ||
        overlaps(O, ob, cache_lengths, (size_t)B * sizeof(int32_t)))
        return MHA_ERR_INVALID_ARG;
    QuantStep q = step_shape(m, bits, B, T_q, T_max, 1);
    if (!quant_step_fits(q)) return MHA_ERR_UNSUPPORTED;
    if (m->ws == nullptr || m->ws_bytes < kStatusBytes + quant_step_bytes(q)) return MHA_ERR_WORKSPACE;
    int sms = 0;
    const mha_status st = query_sms(&sms);
    if (st != MHA_OK) return st;
    q = step_shape(m, bits, B, T_q, T_max, sms);
    float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(m->ws) + kStatusBytes);
    const cudaError_t err = launch_quant_decode(q, m->dtype == MHA_F32, bits, c.k, c.v, Q, ldq, O, ldo, cache_lengths, part,
                                                status_ptr(m), static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

}  // extern "C"
