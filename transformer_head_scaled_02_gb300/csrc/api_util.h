// api_util.h -- what the C-ABI translation units share on the host: workspace layout, argument
// helpers, the SM count.  Not part of the public interface.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "../../include/mha.h"
#include "internal.h"

namespace mha {

constexpr size_t kStatusBytes = 256;

// Most rows (tokens of all batches, query rows) of a long-context call: its kernels count them in 32 bits
// and step past the last one by up to a scan or a grid.
constexpr int64_t kMostRows = INT32_MAX - 65535;

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline size_t elem_bytes(mha_dtype t) { return t == MHA_F32 ? 4 : 2; }

// Bytes of [p, p + n) overlap [q, q + m)?
inline bool overlaps(const void* p, size_t n, const void* q, size_t m) {
    if (!p || !q || n == 0 || m == 0) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + m && b < a + n;
}

// Column widths of the fused projection [Q | K | V | G].
struct Widths {
    int64_t q, k, v, g;  // h*dk, h_kv*dk, h_kv*dv, gated ? h*dv : 0
    int64_t all() const { return q + k + v + g; }
};

inline Widths widths(const mha_s* m) {
    Widths w;
    w.q = (int64_t)m->h * m->dk;
    w.k = (int64_t)m->h_kv * m->dk;
    w.v = (int64_t)m->h_kv * m->dv;
    w.g = m->gated ? (int64_t)m->h * m->dv : 0;
    return w;
}

struct WsLayout {
    size_t q_off, kv_off, o_off, total;
};

// status | Q and G (B,T_q,h*dk [+ h*dv]) | KV (B,T_kv,h_kv*(dk+dv)) | Ocat (B,T_q,h*dv).  For
// self-attention the Q and KV regions are used as one fused (B,T,[Q|K|V|G]) buffer starting
// at q_off, which needs no more bytes than the two regions together.
inline WsLayout ws_layout(const mha_s* m, int B, int T_q, int T_kv) {
    const size_t s = elem_bytes(m->dtype);
    const Widths wd = widths(m);
    const size_t hv = (size_t)m->h * m->dv;
    WsLayout w;
    w.q_off = kStatusBytes;
    w.kv_off = w.q_off + align256((size_t)B * T_q * (size_t)(wd.q + wd.g) * s);
    w.o_off = w.kv_off + align256((size_t)B * T_kv * (size_t)(wd.k + wd.v) * s);
    w.total = w.o_off + align256((size_t)B * T_q * hv * s);
    return w;
}

inline mha_status query_sms(int* out) {
    static std::atomic<int> g_num_sms[64];  // SM count per device, 0 until asked
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MHA_ERR_CUDA;
    int n = dev >= 0 && dev < 64 ? g_num_sms[dev].load(std::memory_order_relaxed) : 0;
    if (n <= 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            return MHA_ERR_CUDA;
        if (dev >= 0 && dev < 64) g_num_sms[dev].store(n, std::memory_order_relaxed);
    }
    *out = n;
    return MHA_OK;
}

// Does this build have tensor-core kernels for the handle's shape?
inline bool bf16_shape_supported(const mha_s* m) {
    return m->dk == m->dv && (m->dk == 64 || m->dk == 128) && (m->D % 8) == 0;
}

inline int* status_ptr(const mha_s* m) { return m->ws ? reinterpret_cast<int*>(m->ws) : nullptr; }

}  // namespace mha
