// span_api.cu -- the C ABI of the long-context operators (include/mha.h): windowed attention with
// sinks, the windowed, shared-prefix and weight-accumulating decode steps, and the eviction.  Host
// checks, workspace layout and launch sequences; nothing is allocated or synchronised here.
#include <math.h>
#include <stdint.h>

#include "../../include/mha.h"
#include "api_util.h"
#include "internal.h"
#include "span_records.cuh"

using namespace mha;

namespace {


// Query rows of a row block: a tensor-core tile for bf16; for fp32 what a block of the few-row kernel holds
// if it holds them all, else the smallest of 16, 32 and 64 that does (a thread of span_simt.cu's kernel owns
// 1, 2 or 4 of them).  Measured both ways, 16 caches of 4096 tokens, 4 K/V heads, few rows | tiles: d = 64, 1
// row 40 | 106 us, 8 rows 75 | 107; d = 128, 4 rows 67 | 172; d = 256, 2 rows 243 | 356.  Two caches of 1000:
// 10 | 12, 17 | 12, 14 | 16, 21 | 22.  With 10 rows of d = 64 in two blocks of 8 instead of one of 16, 3 caches
// of 300 visible tokens took 17 us instead of 12.
int row_block(const mha_s* m, int64_t rows) {
    if (m->dtype == MHA_BF16) return 128;
    if (rows <= span_few_rows(m->dk, m->dv)) return span_few_rows(m->dk, m->dv);
    return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

SpanShape span_shape(const mha_s* m, int B, int T_q, int T_max, int T_p, int window, int sinks) {
    SpanShape p;
    p.B = B;
    p.h_kv = m->h_kv;
    p.per = m->h / m->h_kv;
    p.T_q = T_q;
    p.T_max = T_max;
    p.rows = p.per * T_q;
    p.T_p = T_p;
    // a prefix's rows are those of the whole batch
    const int64_t rows_p = (int64_t)B * p.rows;
    p.bm_c = row_block(m, p.rows);
    p.bm_p = row_block(m, rows_p);
    p.nrb = (p.rows + p.bm_c - 1) / p.bm_c;
    p.nrbp = T_p > 0 ? (int)((rows_p + p.bm_p - 1) / p.bm_p) : 0;
    const bool few = p.bm_c < 16;
    p.aim = few ? 1 : 0;  // few rows: its units are long (1, 2 and 4 of them: 41, 46 and 50 us of the
                                   // first case above)
    p.step = few ? 4 : 1;
    p.window = window < T_max ? window : T_max;
    p.sinks = sinks < T_max ? sinks : T_max;
    return p;
}

SpanLayout layout(const mha_s* m, const SpanShape& p, bool scores) {
    return m->dtype == MHA_F32 ? span_layout<64>(p, m->dv, scores) : span_layout<128>(p, m->dv, scores);
}

// Bytes from the first to the last element of `rows` rows of `width` elements.
size_t extent(int64_t rows, int64_t ld, int64_t width, size_t elem) {
    return rows > 0 ? ((size_t)(rows - 1) * (size_t)ld + (size_t)width) * elem : 0;
}

bool rows_ok(const mha_s* m, const void* p, int64_t ld, int64_t width) {
    if (p == nullptr || ld < width) return false;
    return m->dtype != MHA_BF16 || (ld % 8 == 0 && aligned16(p));
}

mha_status shape_supported(const mha_s* m) {
    if (m->dtype == MHA_BF16) return bf16_shape_supported(m) ? MHA_OK : MHA_ERR_UNSUPPORTED;
    return m->dk <= 256 && m->dv <= 256 ? MHA_OK : MHA_ERR_UNSUPPORTED;
}

// What a window's sizes are refused for, before the layer's projections as well as before the attention.
mha_status window_supported(const mha_s* m, int B, int T, int window, int sinks) {
    if (B < 0 || T < 0 || window < 1 || sinks < 0) return MHA_ERR_INVALID_ARG;
    if ((int64_t)B * T > kMostRows || (int64_t)B * m->h > INT32_MAX) return MHA_ERR_INVALID_ARG;
    const mha_status sup = shape_supported(m);
    if (sup != MHA_OK) return sup;
    const bool fits = m->dtype == MHA_F32 ? ((int64_t)T + 31) / 32 <= 65535
                                          : (int64_t)B * m->h * (((int64_t)T + 127) / 128) <= INT32_MAX;
    return fits ? MHA_OK : MHA_ERR_UNSUPPORTED;
}

struct CacheStep {
    int B, T_q, T_max, T_p, window, sinks;
    const void *Q, *K, *V, *Kp, *Vp;
    int64_t ldq, ldk, ldv, ldkp, ldvp;
    const int32_t* lengths;
    float* weights;
    void* O;
    int64_t ldo;
};

// Sizes that every cache step shares (the int32 row arithmetic of the kernels).
bool step_sizes_ok(const mha_s* m, int B, int T_q, int T_p, int T_max) {
    return B >= 0 && T_q >= 0 && T_p >= 0 && T_max >= 0 && T_p <= kMostRows && (int64_t)B * T_max <= kMostRows &&
           (int64_t)B * m->h * T_q <= kMostRows;
}

mha_status run_cache_step(mha_s* m, const CacheStep& a, cudaStream_t stream) {
    if (m == nullptr) return MHA_ERR_INVALID_ARG;
    if (!step_sizes_ok(m, a.B, a.T_q, a.T_p, a.T_max) || a.window < 1 || a.sinks < 0) return MHA_ERR_INVALID_ARG;
    if (a.B == 0 || a.T_q == 0) return MHA_OK;
    if (a.T_q > a.T_max || a.lengths == nullptr) return MHA_ERR_INVALID_ARG;
    const Widths wd = widths(m);
    const int64_t hv = (int64_t)m->h * m->dv;
    const size_t s = elem_bytes(m->dtype);
    const mha_status sup = shape_supported(m);
    if (sup != MHA_OK) return sup;
    if (!rows_ok(m, a.Q, a.ldq, wd.q) || !rows_ok(m, a.K, a.ldk, wd.k) || !rows_ok(m, a.V, a.ldv, wd.v) ||
        !rows_ok(m, a.O, a.ldo, hv))
        return MHA_ERR_INVALID_ARG;
    if (a.T_p > 0 && (!rows_ok(m, a.Kp, a.ldkp, wd.k) || !rows_ok(m, a.Vp, a.ldvp, wd.v))) return MHA_ERR_INVALID_ARG;
    const int64_t nq = (int64_t)a.B * a.T_q, nc = (int64_t)a.B * a.T_max;
    const size_t wbytes = a.weights != nullptr ? (size_t)nc * m->h_kv * sizeof(float) : 0;
    struct Span {
        const void* p;
        size_t n;
    };
    const Span in[5] = {{a.Q, extent(nq, a.ldq, wd.q, s)},
                        {a.K, extent(nc, a.ldk, wd.k, s)},
                        {a.V, extent(nc, a.ldv, wd.v, s)},
                        {a.T_p > 0 ? a.Kp : nullptr, extent(a.T_p, a.ldkp, wd.k, s)},
                        {a.T_p > 0 ? a.Vp : nullptr, extent(a.T_p, a.ldvp, wd.v, s)}};
    const size_t obytes = extent(nq, a.ldo, hv, s);
    for (const Span& x : in)
        if (overlaps(a.O, obytes, x.p, x.n) || overlaps(a.weights, wbytes, x.p, x.n)) return MHA_ERR_INVALID_ARG;
    if (overlaps(a.O, obytes, a.weights, wbytes)) return MHA_ERR_INVALID_ARG;

    const SpanShape p = span_shape(m, a.B, a.T_q, a.T_max, a.T_p, a.window, a.sinks);
    const int64_t most = m->dtype == MHA_F32 ? span_most_tiles<64>(p) : span_most_tiles<128>(p);
    if (most > INT32_MAX || (m->dtype == MHA_F32 && span_merge_blocks(p, a.weights != nullptr) > INT32_MAX))
        return MHA_ERR_UNSUPPORTED;
    const SpanLayout w = layout(m, p, a.weights != nullptr);
    if (m->ws == nullptr || m->ws_bytes < kStatusBytes + w.total) return MHA_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(m->ws) + kStatusBytes;
    SpanRecords rec;
    rec.ml = reinterpret_cast<float2*>(ws + w.ml_off);
    rec.o = reinterpret_cast<float*>(ws + w.o_off);
    rec.base_c = w.base_c;
    rec.dv = m->dv;
    float* scores = a.weights != nullptr ? reinterpret_cast<float*>(ws + w.s_off) : nullptr;
    int sms = 0;
    const mha_status st = query_sms(&sms);
    if (st != MHA_OK) return st;
    // one CTA per SM holds the tensor-core kernel's tiles, two mostly the CUDA-core tiles (span_simt.cu); of the
    // few-row kernel and of 64-row tiles at d = 128 an SM holds one, and the second takes its turn
    int ctas = m->dtype == MHA_F32 ? 2 * sms : sms;
    if (ctas > kSpanMaxCtas) ctas = kSpanMaxCtas;
    if (most < ctas) ctas = (int)most;
    cudaError_t err;
    if (m->dtype == MHA_F32) {
        auto f = [](const void* x) { return static_cast<const float*>(x); };
        float* O = static_cast<float*>(a.O);
        // each kind of unit in the row blocks made for its rows: one launch if they are the same
        auto units = [&](bool prefix, bool cache) {
            const int bm = cache ? p.bm_c : p.bm_p;
            auto launch = bm < 16 ? launch_span_few : launch_span_f32;
            return launch(p, rec, f(a.Q), a.ldq, f(a.K), a.ldk, f(a.V), a.ldv, f(a.Kp), a.ldkp, f(a.Vp), a.ldvp, O, a.ldo,
                          m->dk, m->dv, a.lengths, scores, prefix, cache, ctas, status_ptr(m), stream);
        };
        if (p.T_p == 0 || p.bm_p == p.bm_c) {
            err = units(true, true);
        } else {
            err = units(true, false);
            if (err == cudaSuccess) err = units(false, true);
        }
        if (err == cudaSuccess)
            err = launch_span_merge(p, rec, ctas, O, a.ldo, a.lengths, scores, a.weights, stream);
    } else {
        err = launch_span_bf16(p, rec, a.Q, a.ldq, a.K, a.ldk, a.V, a.ldv, a.Kp, a.ldkp, a.Vp, a.ldvp, a.O, a.ldo,
                               m->dk, a.lengths, scores, a.weights, ctas, status_ptr(m), stream);
    }
    return err == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

}  // namespace

extern "C" {

mha_status mha_attention_window(mha_t handle, int B, int T, const void* Q, int64_t ldq, const void* K, int64_t ldk,
                                const void* V, int64_t ldv, const void* G, int64_t ldg, int window, int sinks,
                                const int32_t* kv_lengths, void* O, int64_t ldo, void* stream) {
    const mha_s* m = handle;
    if (m == nullptr) return MHA_ERR_INVALID_ARG;
    const mha_status sup = window_supported(m, B, T, window, sinks);
    if (sup != MHA_OK) return sup;
    if (B == 0 || T == 0) return MHA_OK;
    const Widths wd = widths(m);
    const int64_t hv = (int64_t)m->h * m->dv, n = (int64_t)B * T;
    const size_t s = elem_bytes(m->dtype);
    if (!rows_ok(m, Q, ldq, wd.q) || !rows_ok(m, K, ldk, wd.k) || !rows_ok(m, V, ldv, wd.v) || !rows_ok(m, O, ldo, hv) ||
        (G != nullptr && !rows_ok(m, G, ldg, hv)))
        return MHA_ERR_INVALID_ARG;
    const size_t ob = extent(n, ldo, hv, s);
    if (overlaps(O, ob, Q, extent(n, ldq, wd.q, s)) || overlaps(O, ob, K, extent(n, ldk, wd.k, s)) ||
        overlaps(O, ob, V, extent(n, ldv, wd.v, s)) || overlaps(O, ob, G, extent(n, ldg, hv, s)))
        return MHA_ERR_INVALID_ARG;
    window = window < T ? window : T;
    sinks = sinks < T ? sinks : T;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    cudaError_t err;
    if (m->dtype == MHA_F32) {
        auto f = [](const void* x) { return static_cast<const float*>(x); };
        err = launch_window_f32(f(Q), ldq, f(K), ldk, f(V), ldv, f(G), ldg, static_cast<float*>(O), ldo, B, m->h,
                                m->h_kv, T, m->dk, m->dv, window, sinks, kv_lengths, status_ptr(m), cs);
    } else {
        int sms = 0;
        const mha_status st = query_sms(&sms);
        if (st != MHA_OK) return st;
        err = launch_window_bf16(Q, ldq, K, ldk, V, ldv, G, ldg, O, ldo, B, m->h, m->h_kv, T, m->dk, window, sinks,
                                 kv_lengths, sms, status_ptr(m), cs);
    }
    return err == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

mha_status mha_forward_window(mha_t handle, const void* X, int B, int T, const void* W_qkv, const void* b_qkv,
                              const void* W_o, const void* b_o, int window, int sinks, const int32_t* kv_lengths,
                              const void* residual, void* out, void* stream) {
    const mha_s* m = handle;
    if (m == nullptr) return MHA_ERR_INVALID_ARG;
    mha_status st = window_supported(m, B, T, window, sinks);
    if (st != MHA_OK) return st;
    st = check_forward(m, X, nullptr, B, T, T, W_qkv, b_qkv, W_o, b_o, 1, residual, out);
    if (st != MHA_OK) return st;
    if (B == 0 || T == 0) return MHA_OK;
    const WsLayout w = ws_layout(m, B, T, T);
    if (m->ws == nullptr || m->ws_bytes < w.total) return MHA_ERR_WORKSPACE;
    const Widths wd = widths(m);
    const int64_t n = wd.all(), hv = (int64_t)m->h * m->dv;
    const size_t s = elem_bytes(m->dtype);
    uint8_t* qkv = static_cast<uint8_t*>(m->ws) + w.q_off;
    void* ocat = static_cast<uint8_t*>(m->ws) + w.o_off;
    st = mha_linear_ex(handle, X, m->D, B * T, m->D, W_qkv, n, (int)n, b_qkv, nullptr, 0, qkv, n, stream);
    if (st != MHA_OK) return st;
    st = mha_attention_window(handle, B, T, qkv, n, qkv + wd.q * s, n, qkv + (wd.q + wd.k) * s, n,
                              m->gated ? qkv + (wd.q + wd.k + wd.v) * s : nullptr, n, window, sinks, kv_lengths, ocat,
                              hv, stream);
    if (st != MHA_OK) return st;
    return mha_linear_ex(handle, ocat, hv, B * T, (int)hv, W_o, m->D, m->D, b_o, residual, m->D, out, m->D, stream);
}

size_t mha_cache_step_workspace_size(mha_t handle, int B, int T_q, int T_prefix, int T_max, int weights) {
    if (handle == nullptr || !step_sizes_ok(handle, B, T_q, T_prefix, T_max)) return 0;
    if (B == 0 || T_q == 0 || T_max == 0) return kStatusBytes;
    return kStatusBytes + layout(handle, span_shape(handle, B, T_q, T_max, T_prefix, T_max, 0), weights != 0).total;
}

mha_status mha_decode_window(mha_t handle, int B, int T_q, int T_max, const void* Q, int64_t ldq, const void* K_cache,
                             int64_t ldk, const void* V_cache, int64_t ldv, int window, int sinks,
                             const int32_t* cache_lengths, void* O, int64_t ldo, void* stream) {
    const CacheStep a{B, T_q, T_max, 0, window, sinks, Q, K_cache, V_cache, nullptr, nullptr, ldq, ldk, ldv, 0, 0,
                      cache_lengths, nullptr, O, ldo};
    return run_cache_step(handle, a, static_cast<cudaStream_t>(stream));
}

mha_status mha_decode_shared(mha_t handle, int B, int T_q, int T_prefix, const void* K_prefix, int64_t ldkp,
                             const void* V_prefix, int64_t ldvp, int T_max, const void* Q, int64_t ldq,
                             const void* K_cache, int64_t ldk, const void* V_cache, int64_t ldv,
                             const int32_t* cache_lengths, void* O, int64_t ldo, void* stream) {
    const CacheStep a{B, T_q, T_max, T_prefix, T_max > 0 ? T_max : 1, 0, Q, K_cache, V_cache, K_prefix, V_prefix, ldq,
                      ldk, ldv, ldkp, ldvp, cache_lengths, nullptr, O, ldo};
    return run_cache_step(handle, a, static_cast<cudaStream_t>(stream));
}

mha_status mha_decode_weights(mha_t handle, int B, int T_q, int T_max, const void* Q, int64_t ldq,
                              const void* K_cache, int64_t ldk, const void* V_cache, int64_t ldv,
                              const int32_t* cache_lengths, float* weights, void* O, int64_t ldo, void* stream) {
    if (handle != nullptr && B > 0 && T_q > 0 && weights == nullptr) return MHA_ERR_INVALID_ARG;
    const CacheStep a{B, T_q, T_max, 0, T_max > 0 ? T_max : 1, 0, Q, K_cache, V_cache, nullptr, nullptr, ldq, ldk, ldv,
                      0, 0, cache_lengths, weights, O, ldo};
    return run_cache_step(handle, a, static_cast<cudaStream_t>(stream));
}

mha_status mha_cache_evict(mha_t handle, int B, int T_max, int keep, int recent, const void* K_cache, int64_t ldk,
                           const void* V_cache, int64_t ldv, const int32_t* cache_lengths, const float* weights,
                           int T_out, void* K_out, int64_t ldko, void* V_out, int64_t ldvo, float* weights_out,
                           int32_t* kept, int32_t* new_lengths, void* stream) {
    const mha_s* m = handle;
    if (m == nullptr) return MHA_ERR_INVALID_ARG;
    if (B < 0 || T_max < 0 || keep < 1 || recent < 0 || recent > keep || T_out < keep) return MHA_ERR_INVALID_ARG;
    if ((int64_t)B * T_max > kMostRows || (int64_t)B * T_out > kMostRows || (int64_t)B * m->h_kv > INT32_MAX)
        return MHA_ERR_INVALID_ARG;
    const mha_status sup = shape_supported(m);
    if (sup != MHA_OK) return sup;
    if (B > 65535) return MHA_ERR_UNSUPPORTED;
    if (B == 0) return MHA_OK;
    if (T_max == 0) return MHA_ERR_INVALID_ARG;
    const Widths wd = widths(m);
    if (cache_lengths == nullptr || weights == nullptr || weights_out == nullptr || kept == nullptr ||
        new_lengths == nullptr)
        return MHA_ERR_INVALID_ARG;
    if (!rows_ok(m, K_cache, ldk, wd.k) || !rows_ok(m, V_cache, ldv, wd.v) || !rows_ok(m, K_out, ldko, wd.k) ||
        !rows_ok(m, V_out, ldvo, wd.v))
        return MHA_ERR_INVALID_ARG;
    // in place: all three at once, with the same layout; else no output may touch an input
    const size_t s = elem_bytes(m->dtype);
    const bool in_place = K_out == K_cache;
    if (in_place) {
        if (V_out != V_cache || weights_out != weights || T_out != T_max || ldko != ldk || ldvo != ldv)
            return MHA_ERR_INVALID_ARG;
    }
    if (!in_place && (int64_t)m->h_kv * keep > UINT32_MAX) return MHA_ERR_UNSUPPORTED;
    const int64_t ni = (int64_t)B * T_max, no = (int64_t)B * T_out;
    struct Span {
        const void* p;
        size_t n;
    };
    const Span in[4] = {{K_cache, extent(ni, ldk, wd.k, s)},
                        {V_cache, extent(ni, ldv, wd.v, s)},
                        {weights, (size_t)ni * m->h_kv * sizeof(float)},
                        {cache_lengths, (size_t)B * sizeof(int32_t)}};
    const Span out[5] = {{K_out, extent(no, ldko, wd.k, s)},
                         {V_out, extent(no, ldvo, wd.v, s)},
                         {weights_out, (size_t)no * m->h_kv * sizeof(float)},
                         {new_lengths, (size_t)B * sizeof(int32_t)},
                         {kept, (size_t)B * m->h_kv * keep * sizeof(int32_t)}};
    // K and V may be column views of one buffer: rows interleave, so two views of the same rows
    // overlap only if their columns do
    auto touch = [&](const Span& x, int64_t ldx, int64_t wx, const Span& y, int64_t ldy, int64_t wy) {
        if (!overlaps(x.p, x.n, y.p, y.n)) return false;
        if (ldx != ldy || ldx <= 0) return true;
        const int64_t d = static_cast<const uint8_t*>(y.p) - static_cast<const uint8_t*>(x.p);
        const int64_t ld = ldx * (int64_t)s, c = ((d % ld) + ld) % ld;  // y's first column, x's at 0
        return c < wx * (int64_t)s || c + wy * (int64_t)s > ld;
    };
    const int64_t ldi[2] = {ldk, ldv}, ldo[2] = {ldko, ldvo}, wk[2] = {wd.k, wd.v};
    for (int o = 0; o < 5; ++o) {
        for (int i = 0; i < 4; ++i) {
            if ((o == i && o < 3 && in_place) || (o == 3 && i == 3 && new_lengths == cache_lengths)) continue;
            const bool hit = o < 2 && i < 2 ? touch(in[i], ldi[i], wk[i], out[o], ldo[o], wk[o])
                                            : overlaps(out[o].p, out[o].n, in[i].p, in[i].n);
            if (hit) return MHA_ERR_INVALID_ARG;
        }
        for (int q = o + 1; q < 5; ++q) {
            const bool hit = o < 2 && q < 2 ? touch(out[o], ldo[o], wk[o], out[q], ldo[q], wk[q])
                                            : overlaps(out[o].p, out[o].n, out[q].p, out[q].n);
            if (hit) return MHA_ERR_INVALID_ARG;
        }
    }
    const cudaError_t err = launch_evict(K_cache, ldk, V_cache, ldv, K_out, ldko, V_out, ldvo, (int)s, B, m->h_kv, T_max,
                                         T_out, m->dk, m->dv, keep, recent, cache_lengths, weights, weights_out, kept,
                                         new_lengths, status_ptr(m), static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

}  // extern "C"
