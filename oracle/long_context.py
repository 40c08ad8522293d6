"""The long-context operators in 64 bits, from their definitions: one query row at a time, the scores
materialised, numpy only.  Test infrastructure; shares no code with the kernels.

Rows and heads as in include/mha.h: Q (B, T, h*d_k), K (B, T, h_kv*d_k), V (B, T, h_kv*d_v); query head i
reads K/V head i // (h // h_kv).
"""
import numpy as np


def _f64(a):
    return np.asarray(a, dtype=np.float64)


def _row(q, K, V, keys):
    """One softmax row over the listed keys: (output, weights, sum of weight * |v|)."""
    if len(keys) == 0:
        z = np.zeros(V.shape[1])
        return z, np.zeros(0), z
    s = K[keys] @ q / np.sqrt(q.shape[0])
    e = np.exp(s - s.max())
    w = e / e.sum()
    return w @ V[keys], w, w @ np.abs(V[keys])


def _heads(x, n, i):
    d = x.shape[-1] // n
    return x[..., i * d:(i + 1) * d]


def attention_window(Q, K, V, h, window, sinks=0, h_kv=None, kv_lengths=None, G=None):
    """Row i sees j iff j <= i, j < L_b and (i - j < window or j < sinks); a row without keys is zero, a
    batch with an invalid length NaN.  Returns (O, A): A bounds O's rounding, sum of weight * |v|."""
    Q, K, V = _f64(Q), _f64(K), _f64(V)
    h_kv = h if h_kv is None else h_kv
    B, T, _ = Q.shape
    dv = V.shape[2] // h_kv
    O, A = np.zeros((B, T, h * dv)), np.zeros((B, T, h * dv))
    for b in range(B):
        L = T if kv_lengths is None else int(kv_lengths[b])
        if not 1 <= L <= T:
            O[b] = np.nan
            continue
        for i in range(h):
            k, v = _heads(K[b], h_kv, i // (h // h_kv)), _heads(V[b], h_kv, i // (h // h_kv))
            q = _heads(Q[b], h, i)
            for t in range(T):
                lo = max(0, t - window + 1)
                end = min(t + 1, L)
                keys = np.r_[0:min(sinks, lo, end), lo:max(lo, end)]
                o, _, a = _row(q[t], k, v, keys)
                if G is not None:
                    gate = 1.0 / (1.0 + np.exp(-_heads(_f64(G)[b], h, i)[t]))
                    o, a = o * gate, a * gate
                O[b, t, i * dv:(i + 1) * dv], A[b, t, i * dv:(i + 1) * dv] = o, a
    return O, A


def decode(Q, K, V, h, lengths, h_kv=None, window=None, sinks=0, K_prefix=None, V_prefix=None, weights=None):
    """One decode step: new token t at position p = L_b - T_q + t sees cache keys j <= p (under a window:
    and (p - j < window or j < sinks)) and the whole prefix.  Returns (O, A, W): W the accumulated
    weights (B, h_kv, T_max) if `weights` is given (new tokens' entries start at zero)."""
    Q, K, V = _f64(Q), _f64(K), _f64(V)
    h_kv = h if h_kv is None else h_kv
    per = h // h_kv
    B, Tq, _ = Q.shape
    Tmax = K.shape[1]
    dv = V.shape[2] // h_kv
    O, A = np.zeros((B, Tq, h * dv)), np.zeros((B, Tq, h * dv))
    W = None if weights is None else _f64(weights).copy()
    for b in range(B):
        L = int(lengths[b])
        if not Tq <= L <= Tmax:
            O[b] = np.nan
            continue
        if W is not None:
            W[b, :, L - Tq:L] = 0.0
        for i in range(h):
            g = i // per
            k, v = _heads(K[b, :L], h_kv, g), _heads(V[b, :L], h_kv, g)
            n_p = 0
            if K_prefix is not None:
                n_p = K_prefix.shape[0]
                k = np.concatenate((_heads(_f64(K_prefix), h_kv, g), k))
                v = np.concatenate((_heads(_f64(V_prefix), h_kv, g), v))
            q = _heads(Q[b], h, i)
            for t in range(Tq):
                p = L - Tq + t
                j = np.arange(p + 1)
                if window is not None:
                    j = j[(p - j < window) | (j < sinks)]
                o, w, a = _row(q[t], k, v, np.concatenate((np.arange(n_p), n_p + j)))
                O[b, t, i * dv:(i + 1) * dv], A[b, t, i * dv:(i + 1) * dv] = o, a
                if W is not None:
                    W[b, g, j] += w[n_p:]
    return O, A, W


def evict(weights, lengths, keep, recent):
    """Kept token indices per (b, g): a list of lists of ascending lists; None for an invalid length."""
    weights = np.asarray(weights)
    B, h_kv, T = weights.shape
    out = []
    for b in range(B):
        L = int(lengths[b])
        if not 0 <= L <= T:
            out.append([None] * h_kv)
            continue
        rows = []
        for g in range(h_kv):
            if L <= keep:
                rows.append(list(range(L)))
                continue
            w = [(-np.inf if np.isnan(x) else float(x)) for x in weights[b, g, :L - recent]]
            # NaN lies below every number, -inf included
            nan = [bool(np.isnan(x)) for x in weights[b, g, :L - recent]]
            order = sorted(range(L - recent), key=lambda j: (nan[j], -w[j], j))
            rows.append(sorted(order[:keep - recent]) + list(range(L - recent, L)))
        out.append(rows)
    return out
