"""The quantised key/value cache from its definition (include/mha.h), numpy and exact fractions only.  Test
infrastructure; shares no code with the kernels.

quantise() works in 64 bits, which settles every code of inputs whose exponents lie within 2^29 of each other;
quantise_exact() one group in fractions, for any finite input.  Rows and heads as in include/mha.h.
"""
import math
from fractions import Fraction

import numpy as np

GROUP = 64
BF16_MAX = 3.3895313892515355e38
LEAST_STEP = 2.0 ** -126


def _grid(x, up):
    """x to bf16's 8 significant bits, upwards or downwards, in 64 bits (x normal in bf16, or zero)."""
    mant, exp = np.frexp(x)
    return np.ldexp((np.ceil if up else np.floor)(mant * 256.0), exp - 8)


def quantise(x, bits):
    """x (..., d): codes (..., d) and [step, lowest] (..., groups, 2), all in 64 bits."""
    x = np.asarray(x, np.float64)
    n = 2 ** bits - 1
    codes, params = np.zeros(x.shape), []
    for c in range(0, x.shape[-1], GROUP):
        y = x[..., c:c + GROUP]
        bad = ~(np.abs(y) <= BF16_MAX).all(-1)
        y = np.where(bad[..., None], 0.0, y)
        low = _grid(y.min(-1), False)
        step = np.maximum(_grid((y.max(-1) - low) / n, True), LEAST_STEP)
        codes[..., c:c + GROUP] = np.rint((y - low[..., None]) / step[..., None])
        params.append(np.where(bad[..., None], np.nan, np.stack((step, low), -1)))
    return codes, np.stack(params, -2)


def _bf16_neighbours(f):
    """The bf16 values around the fraction f: the largest not above, the smallest not below."""
    if f == 0:
        return Fraction(0), Fraction(0)
    e = max(math.floor(math.log2(abs(f))) - 1, -126)
    while abs(f) >= Fraction(2) ** (e + 1):
        e += 1
    unit = Fraction(2) ** (e - 7)
    return math.floor(f / unit) * unit, math.ceil(f / unit) * unit


def quantise_exact(x, bits):
    """One group of finite numbers: (codes, step, lowest), without any rounding."""
    x = [Fraction(float(v)) for v in x]
    n = 2 ** bits - 1
    low = _bf16_neighbours(min(x))[0]
    step = max(_bf16_neighbours((max(x) - low) / n)[1], Fraction(2) ** -126)
    codes = [round((v - low) / step) for v in x]  # (of a fraction: ties to even)
    return codes, float(step), float(low)


def pack(codes, bits):
    """Codes (..., d) as cache rows (..., bytes)."""
    codes = np.asarray(codes).astype(np.uint8)
    d = codes.shape[-1]
    row = np.zeros(codes.shape[:-1] + ((d + 31) // 32 * 32,), np.uint8)
    row[..., :d] = codes
    return row if bits == 8 else row[..., 0::2] | (row[..., 1::2] << 4)


def unpack(row, bits, d):
    row = np.asarray(row, np.uint8)
    if bits == 4:
        row = np.stack((row & 15, row >> 4), -1).reshape(row.shape[:-1] + (-1,))
    return row[..., :d].astype(np.float64)


def values(codes, params):
    """What codes (..., d) under params (..., groups, 2) stand for, in 64 bits."""
    p = np.repeat(params, GROUP, axis=-2)[..., :codes.shape[-1], :]
    return codes * p[..., 0] + p[..., 1]


def spread(codes, params):
    """s code: the part of a value that meets a rounded weight in a kernel (the other, m, is added in fp32)."""
    return codes * np.repeat(params, GROUP, axis=-2)[..., :codes.shape[-1], 0]


def heads(x, n):
    """(B, T, n d) -> (B, n, T, d)."""
    x = np.asarray(x)
    return np.moveaxis(x.reshape(x.shape[0], x.shape[1], n, -1), 2, 1)


def decode(Q, codes_k, params_k, codes_v, params_v, h, lengths):
    """One decode step over a cache (codes (B, h_kv, T, d), params (B, h_kv, T, groups, 2)): (O, A, S) with
    A = sum of weight * |v| and S = sum of weight * spread, which bound O's rounding."""
    Q = np.asarray(Q, np.float64)
    B, Tq, _ = Q.shape
    h_kv, T = codes_k.shape[1], codes_k.shape[2]
    K, V, W = values(codes_k, params_k), values(codes_v, params_v), spread(codes_v, params_v)
    dk, dv = K.shape[-1], V.shape[-1]
    O, A, S = (np.zeros((B, Tq, h * dv)) for _ in range(3))
    for b in range(B):
        L = int(lengths[b])
        if not Tq <= L <= T:
            O[b] = np.nan
            continue
        for i in range(h):
            g = i // (h // h_kv)
            for t in range(Tq):
                n = L - Tq + t + 1
                s = K[b, g, :n] @ Q[b, t, i * dk:(i + 1) * dk] / np.sqrt(dk)
                w = np.exp(s - s.max())
                w /= w.sum()
                c = slice(i * dv, (i + 1) * dv)
                O[b, t, c], A[b, t, c], S[b, t, c] = w @ V[b, g, :n], w @ np.abs(V[b, g, :n]), w @ W[b, g, :n]
    return O, A, S
