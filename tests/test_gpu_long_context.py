"""Windowed attention with sinks, the windowed / shared-prefix / weight-accumulating decode steps and the
cache eviction against their 64-bit definitions (oracle/long_context.py).

Tolerances.  fp32: the normwise 1e-5 every fp32 parity test uses.  bf16 outputs, element by element: the
softmax weights are rounded to bf16 (each by at most 2^-8 of itself) before the value product, which is
off by at most 2^-8 sum_j w_j |v_j| = 2^-8 A; the output is rounded once, by at most 2^-8 |o|; everything
else is fp32 and bounded by 1e-4 A (scores of a few units, off by at most (d + 8) 2^-23 sum |q||k| / sqrt(d)
each, about 1e-5 .. 1e-4 absolute).  Accumulated weights stay fp32 throughout: each is off by at most
twice the largest score error of its row, relative; the tests allow 2e-4 of the weight (the same bound)
and 1e-5 normwise.
"""
import itertools

import numpy as np
import pytest

from gpu_util import F32_NORMWISE, errors, to_device, to_host, torch_dtype

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
from oracle import long_context as lc  # noqa: E402
from transformer_head_scaled_02_gb300 import Mha, _lib  # noqa: E402
from transformer_head_scaled_02_gb300 import workloads as wl  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build_library()
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)


def _check(got, ref, A, dtype, what):
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    if dtype == "f32":
        assert errors(got, ref)["normwise"] <= F32_NORMWISE, f"{what}: {errors(got, ref)}"
    else:
        over = np.abs(got - ref) - (2.0 ** -8 * (A + np.abs(ref)) + 1e-4 * A)
        assert over.max() <= 0, f"{what}: {over.max()} over the bound; {errors(got, ref)}"


def _check_weights(got, ref, what):
    d = np.abs(got - ref)
    assert (d <= 2e-4 * np.abs(ref) + 1e-7).all(), f"{what}: {(d / np.maximum(np.abs(ref), 1e-9)).max()}"
    assert errors(got, ref)["normwise"] <= F32_NORMWISE, f"{what}: {errors(got, ref)}"


def _layer(dtype, h, d, h_kv, d_v=None, gated=False):
    return Mha(h * d, h, d, d if d_v is None else d_v, dtype=torch_dtype(dtype), h_kv=h_kv, gated=gated)


def _rand(shape, seed, dtype):
    return wl.random_tensor(shape, seed, dtype)


def _lens(lengths):
    return torch.tensor(lengths, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ whole sequences

WINDOW_SHAPES = [
    # dtype, d, d_v, h, h_kv
    ("bf16", 64, 64, 4, 4), ("bf16", 64, 64, 4, 1), ("bf16", 128, 128, 2, 2), ("bf16", 128, 128, 4, 2),
    ("f32", 32, 32, 4, 2), ("f32", 20, 37, 3, 1), ("f32", 7, 130, 2, 2), ("f32", 256, 256, 1, 1)]


def _window_case(seed, dtype, d, dv, h, h_kv, B, T, window, sinks, lengths=None, gated=False):
    Q, K, V = _rand((B, T, h * d), seed, dtype), _rand((B, T, h_kv * d), seed + 1, dtype), _rand((B, T, h_kv * dv), seed + 2, dtype)
    G = _rand((B, T, h * dv), seed + 3, dtype) if gated else None
    layer = _layer(dtype, h, d, h_kv, dv, gated)
    out = layer.attention_window(to_device(Q, dtype), to_device(K, dtype), to_device(V, dtype), window, sinks,
                                 kv_lengths=None if lengths is None else _lens(lengths), G=to_device(G, dtype))
    torch.cuda.synchronize()
    ref, A = lc.attention_window(Q, K, V, h, window, sinks, h_kv, lengths, G)
    return layer, to_host(out), ref, A


@pytest.mark.parametrize("dtype,d,dv,h,h_kv", WINDOW_SHAPES)
@pytest.mark.parametrize("T,window,sinks", [
    (1, 1, 0), (5, 2, 1), (127, 40, 3), (128, 128, 0), (129, 64, 4), (300, 1, 0), (300, 1, 1), (300, 128, 17),
    (300, 129, 0), (300, 500, 0), (300, 60, 200), (389, 127, 130), (515, 256, 1), (700, 97, 5)])
def test_window(dtype, d, dv, h, h_kv, T, window, sinks):
    layer, got, ref, A = _window_case(T + window, dtype, d, dv, h, h_kv, 2, T, window, sinks)
    _check(got, ref, A, dtype, "window")


@pytest.mark.parametrize("dtype,d,dv,h,h_kv", [WINDOW_SHAPES[1], WINDOW_SHAPES[3], WINDOW_SHAPES[5]])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("window,sinks", [(30, 0), (130, 4), (200, 140), (1000, 0)])
def test_window_ragged(dtype, d, dv, h, h_kv, gated, window, sinks):
    """Ragged padded batch: the padding rows past L_b + window see the sinks only, or nothing (zeros)."""
    lengths = [420, 1, 128, 250, 129]
    layer, got, ref, A = _window_case(17 + window, dtype, d, dv, h, h_kv, 5, 420, window, sinks, lengths, gated)
    _check(got, ref, A, dtype, "window ragged")
    if sinks == 0 and window == 30:
        assert (got[1, 31:] == 0).all() and (ref[1, 31:] == 0).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 16)])
def test_window_of_the_whole_sequence_is_causal_attention(dtype, d):
    h, B, T = 4, 2, 333
    x = [to_device(_rand((B, T, h * d), s, dtype), dtype) for s in (1, 2, 3)]
    layer = _layer(dtype, h, d, h)
    lens = _lens([333, 200])
    a = to_host(layer.attention_window(*x, T, 0, kv_lengths=lens))
    b = to_host(layer.attention_window(*x, 2 ** 31 - 1, 2 ** 31 - 1, kv_lengths=lens))
    c = to_host(layer.attention(*x, causal=True, kv_lengths=lens))
    ref = oracle.attention(*[to_host(t) for t in x], h, causal=True, kv_lengths=[333, 200])
    for got in (a, b, c):
        e = errors(got, ref)
        assert e["normwise"] <= F32_NORMWISE if dtype == "f32" else e["max_abs"] <= 2e-2 and e["rel_fro"] <= 5e-3


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 16)])
def test_window_invalid_lengths_and_padding_garbage(dtype, d):
    """Invalid lengths give NaN rows and a status; keys past L_b may be NaN or infinite."""
    h, B, T = 2, 4, 260
    lengths = [260, 0, 100, 261]
    Q, K, V = (_rand((B, T, h * d), s, dtype) for s in (4, 5, 6))
    Kn, Vn = K.copy(), V.copy()
    Kn[2, 100:], Vn[2, 100:] = np.nan, np.inf
    layer = _layer(dtype, h, d, h)
    layer.ensure_workspace(1, 1, 1)
    out = layer.attention_window(to_device(Q, dtype), to_device(Kn, dtype), to_device(Vn, dtype), 70, 5,
                                 kv_lengths=_lens(lengths))
    got = to_host(out)
    ref, A = lc.attention_window(Q, K, V, h, 70, 5, kv_lengths=lengths)
    assert np.isnan(got[1]).all() and np.isnan(got[3]).all()
    _check(got[[0, 2]], ref[[0, 2]], A[[0, 2]], dtype, "window beside invalid batches")
    assert layer.status() == _lib.MHA_ERR_BAD_LENGTH and layer.status() == 0


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 12)])
def test_window_views_and_guard_bands(dtype, d):
    """Column views of one fused buffer, an output with gaps: nothing outside the rows is written."""
    h, h_kv, B, T = 4, 2, 2, 200
    width = (h + 2 * h_kv) * d
    x = _rand((B, T, width), 8, dtype)
    t = to_device(x, dtype)
    big = torch.full((B, T, h * d + 16), 7.0, dtype=torch_dtype(dtype), device="cuda")
    layer = _layer(dtype, h, d, h_kv)
    layer.attention_window(t[..., :h * d], t[..., h * d:(h + h_kv) * d], t[..., (h + h_kv) * d:], 50, 3,
                           out=big[..., 8:8 + h * d])
    ref, A = lc.attention_window(x[..., :h * d], x[..., h * d:(h + h_kv) * d], x[..., (h + h_kv) * d:], h, 50, 3, h_kv)
    got = to_host(big)
    _check(got[..., 8:8 + h * d], ref, A, dtype, "window views")
    assert (got[..., :8] == 7).all() and (got[..., 8 + h * d:] == 7).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 16)])
def test_window_large_scores(dtype, d):
    """Scores of hundreds, rising and falling along the keys: the softmax reference has to follow."""
    h, B, T = 2, 1, 600
    Q, K, V = (_rand((B, T, h * d), s, dtype) for s in (31, 32, 33))
    ramp = np.linspace(0.1, 12.0, T)[None, :, None]
    for scale in (ramp, ramp[:, ::-1]):
        Ks = wl.bf16_to_f32(wl.bf16_bits((K * scale).astype(np.float32))) if dtype == "bf16" else (K * scale).astype(np.float32)
        Qs = Q * 4  # exact in both types
        layer = _layer(dtype, h, d, h)
        got = to_host(layer.attention_window(to_device(Qs, dtype), to_device(Ks, dtype), to_device(V, dtype), 200, 4))
        ref, A = lc.attention_window(Qs, Ks, V, h, 200, 4)
        if dtype == "bf16":
            _check(got, ref, A, dtype, "large scores")
        else:
            # scores reach 4 * 12 * |q||k| / sqrt(d): an fp32 score is off by up to 2^-24 (d + 2) of
            # that sum of products, and the weights by twice as much, relative
            s = 4 * 12 * (np.abs(Q).max() * np.abs(K).max() * d) / np.sqrt(d)
            assert (np.abs(got - ref) <= 2 * s * (d + 2) * 2.0 ** -24 * A + 1e-5 * A).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 16)])
@pytest.mark.parametrize("gated", [False, True])
def test_forward_window(dtype, d, gated):
    """The whole layer: projection, windowed attention, output projection with residual."""
    h, h_kv, B, T, window, sinks = 4, 2, 2, 300, 64, 4
    D = h * d
    layer = _layer(dtype, h, d, h_kv, gated=gated)
    width = layer.proj_width
    X, W, b = _rand((B, T, D), 41, dtype), _rand((D, width), 42, dtype) * 0.0625, _rand((width,), 43, dtype) * 0.0625
    Wo, bo = _rand((h * d, D), 44, dtype) * 0.0625, _rand((D,), 45, dtype)
    t = [to_device(a.astype(np.float32), dtype) for a in (X, W, b, Wo, bo)]
    lens = [300, 77]
    got = to_host(layer.forward(t[0], t[1], t[2], t[3], t[4], causal=True, kv_lengths=_lens(lens), residual=t[0],
                                window=window, sinks=sinks))
    assert layer.status() == 0
    rnd = (lambda a: wl.bf16_to_f32(wl.bf16_bits(np.asarray(a, np.float32))).astype(np.float64)) if dtype == "bf16" else (lambda a: a)
    p = rnd(X.astype(np.float64) @ W + b)
    cut = np.cumsum([h * d, h_kv * d, h_kv * d])
    q, k, v = p[..., :cut[0]], p[..., cut[0]:cut[1]], p[..., cut[1]:cut[2]]
    o, _ = lc.attention_window(q, k, v, h, window, sinks, h_kv, lens, p[..., cut[2]:] if gated else None)
    ref = X + rnd(o) @ Wo + bo
    e = errors(got, ref)
    # bf16: the output's own rounding (2^-8 of values up to about 5) dominates
    assert e["normwise"] <= 1e-5 if dtype == "f32" else e["rel_fro"] <= 5e-3 and e["max_abs"] <= 4e-2


# ------------------------------------------------------------------ decode steps

STEP_SHAPES = [
    # dtype, d, d_v, h, h_kv
    ("bf16", 64, 64, 4, 4), ("bf16", 64, 64, 8, 1), ("bf16", 128, 128, 4, 4), ("bf16", 128, 128, 8, 2),
    ("f32", 32, 32, 4, 4), ("f32", 20, 37, 6, 2), ("f32", 9, 200, 8, 1)]


def _cache(seed, dtype, B, Tq, Tmax, h, h_kv, d, dv):
    return (_rand((B, Tq, h * d), seed, dtype), _rand((B, Tmax, h_kv * d), seed + 1, dtype),
            _rand((B, Tmax, h_kv * dv), seed + 2, dtype))


def _garbage(K, V, lengths):
    """The caches with everything past the lengths NaN or infinite."""
    Kn, Vn = K.copy(), V.copy()
    for b, L in enumerate(lengths):
        if 0 <= L < K.shape[1]:
            Kn[b, L:], Vn[b, L:] = np.nan, (np.nan if b % 2 else np.inf)
    return Kn, Vn


@pytest.mark.parametrize("dtype,d,dv,h,h_kv", STEP_SHAPES)
@pytest.mark.parametrize("Tq", [1, 3])
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 0), (100, 5), (128, 130), (400, 16), (5000, 0)])
def test_decode_window(dtype, d, dv, h, h_kv, Tq, window, sinks):
    B, Tmax = 5, 900
    lengths = [900, Tq, 128, 517, 300]
    Q, K, V = _cache(window + Tq, dtype, B, Tq, Tmax, h, h_kv, d, dv)
    Kn, Vn = _garbage(K, V, lengths)
    layer = _layer(dtype, h, d, h_kv, dv)
    got = to_host(layer.decode_window(to_device(Q, dtype), to_device(Kn, dtype), to_device(Vn, dtype), _lens(lengths),
                                      window, sinks))
    assert layer.status() == 0
    ref, A, _ = lc.decode(Q, K, V, h, lengths, h_kv, window, sinks)
    _check(got, ref, A, dtype, "decode window")


@pytest.mark.parametrize("dtype,d,dv,h,h_kv", STEP_SHAPES)
@pytest.mark.parametrize("B,Tq,Tp", [(1, 1, 1), (3, 1, 300), (5, 2, 129), (40, 1, 700), (7, 20, 260)])
def test_decode_shared(dtype, d, dv, h, h_kv, B, Tq, Tp):
    Tmax = 150
    lengths = [(Tmax, Tq, 128, 77)[b % 4] if (Tmax, Tq, 128, 77)[b % 4] >= Tq else Tq for b in range(B)]
    Q, K, V = _cache(B + Tp, dtype, B, Tq, Tmax, h, h_kv, d, dv)
    Kp, Vp = _rand((Tp, h_kv * d), 71, dtype), _rand((Tp, h_kv * dv), 72, dtype)
    Kn, Vn = _garbage(K, V, lengths)
    layer = _layer(dtype, h, d, h_kv, dv)
    got = to_host(layer.decode_shared(to_device(Q, dtype), to_device(Kp, dtype), to_device(Vp, dtype),
                                      to_device(Kn, dtype), to_device(Vn, dtype), _lens(lengths)))
    assert layer.status() == 0
    ref, A, _ = lc.decode(Q, K, V, h, lengths, h_kv, K_prefix=Kp, V_prefix=Vp)
    _check(got, ref, A, dtype, "decode shared")


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 24)])
def test_decode_shared_without_prefix_is_decode(dtype, d):
    h, h_kv, B, Tq, Tmax = 4, 2, 3, 2, 333
    lengths = [333, 2, 200]
    Q, K, V = _cache(3, dtype, B, Tq, Tmax, h, h_kv, d, d)
    layer = _layer(dtype, h, d, h_kv)
    t = [to_device(x, dtype) for x in (Q, K, V)]
    none = t[1][0, :0]
    got = to_host(layer.decode_shared(t[0], none, none, t[1], t[2], _lens(lengths)))
    ref, A, _ = lc.decode(Q, K, V, h, lengths, h_kv)
    _check(got, ref, A, dtype, "shared without prefix")
    _check(to_host(layer.decode(*t, _lens(lengths))), ref, A, dtype, "decode")


@pytest.mark.parametrize("dtype,d,dv,h,h_kv", STEP_SHAPES)
@pytest.mark.parametrize("Tq", [1, 3])
def test_decode_weights(dtype, d, dv, h, h_kv, Tq):
    B, Tmax = 5, 700
    lengths = [700, Tq, 128, 517, 300]
    Q, K, V = _cache(90 + Tq, dtype, B, Tq, Tmax, h, h_kv, d, dv)
    Kn, Vn = _garbage(K, V, lengths)
    w0 = np.abs(_rand((B, h_kv, Tmax), 93, "f32"))
    for b, L in enumerate(lengths):
        w0[b, :, L - Tq:L] = np.nan       # new tokens' entries start here
    layer = _layer(dtype, h, d, h_kv, dv)
    w = to_device(w0, "f32")
    t = [to_device(x, dtype) for x in (Q, Kn, Vn)]
    got = to_host(layer.decode_weights(*t, _lens(lengths), w))
    ref, A, W = lc.decode(Q, K, V, h, lengths, h_kv, weights=w0)
    _check(got, ref, A, dtype, "decode weights output")
    gw = to_host(w)
    for b, L in enumerate(lengths):
        _check_weights(gw[b, :, :L], W[b, :, :L], "weights")
        assert (gw[b, :, L:] == w0[b, :, L:]).all()          # rows behind the sequence stay
    # the same inputs again: the same bits
    w2 = to_device(w0, "f32")
    layer.decode_weights(*t, _lens(lengths), w2)
    torch.cuda.synchronize()
    assert torch.equal(w.view(torch.int32), w2.view(torch.int32))
    assert layer.status() == 0


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 16)])
@pytest.mark.parametrize("step", ["window", "shared", "weights"])
def test_steps_invalid_lengths(dtype, d, step):
    h, h_kv, B, Tq, Tmax = 4, 2, 5, 2, 300
    lengths = [-7, 300, 1, 301, 150]
    Q, K, V = _cache(95, dtype, B, Tq, Tmax, h, h_kv, d, d)
    t = [to_device(x, dtype) for x in (Q, K, V)]
    layer = _layer(dtype, h, d, h_kv)
    w0 = np.ones((B, h_kv, Tmax))
    w = to_device(w0, "f32")
    kw = {}
    if step == "window":
        got = layer.decode_window(*t, _lens(lengths), 40, 3)
        kw = dict(window=40, sinks=3)
    elif step == "shared":
        got = layer.decode_shared(t[0], t[1][0, :130], t[2][0, :130], t[1], t[2], _lens(lengths))
        kw = dict(K_prefix=K[0, :130], V_prefix=V[0, :130])
    else:
        got = layer.decode_weights(*t, _lens(lengths), w)
    got = to_host(got)
    ref, A, _ = lc.decode(Q, K, V, h, lengths, h_kv, **kw)
    for b in (0, 2, 3):
        assert np.isnan(got[b]).all()
        assert (to_host(w)[b] == 1).all()
    _check(got[[1, 4]], ref[[1, 4]], A[[1, 4]], dtype, step)
    assert layer.status() == _lib.MHA_ERR_BAD_LENGTH and layer.status() == 0
    # no valid length at all
    bad = _lens([0, -1, 1, 301, 999])
    got = to_host(layer.decode_window(*t, bad, 40, 3) if step == "window" else
                  layer.decode_shared(t[0], t[1][0, :130], t[2][0, :130], t[1], t[2], bad) if step == "shared"
                  else layer.decode_weights(*t, bad, w))
    assert np.isnan(got).all() and layer.status() == _lib.MHA_ERR_BAD_LENGTH


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 16)])
def test_decode_large_scores(dtype, d):
    """Scores that jump by hundreds from tile to tile, in every step's form."""
    h, h_kv, B, Tq, Tmax = 4, 2, 2, 2, 1000
    Q, K, V = _cache(97, dtype, B, Tq, Tmax, h, h_kv, d, d)
    Q = Q * 4
    K = K * np.where((np.arange(Tmax) // 100) % 3 == 1, 16.0, 0.25)[None, :, None].astype(np.float32)
    lengths = [1000, 640]
    t = [to_device(np.ascontiguousarray(x, dtype=np.float32), dtype) for x in (Q, K, V)]
    layer = _layer(dtype, h, d, h_kv)
    for kw, got in ((dict(window=333, sinks=7), layer.decode_window(*t, _lens(lengths), 333, 7)),
                    (dict(K_prefix=K[1], V_prefix=V[1]), layer.decode_shared(t[0], t[1][1], t[2][1], t[1], t[2], _lens(lengths)))):
        ref, A, _ = lc.decode(Q, K, V, h, lengths, h_kv, **kw)
        # an fp32 score is off by up to 2^-23 (d + 8) times its sum of products, its weight by twice that
        s = np.abs(Q).max() * np.abs(K).max() * d / np.sqrt(d)
        tol = 2 * s * (d + 8) * 2.0 ** -23 * A + (2.0 ** -8 * (A + np.abs(ref)) if dtype == "bf16" else 0) + 1e-5 * A
        assert (np.abs(to_host(got) - ref) <= tol).all()


def test_many_new_tokens_and_heads():
    """More than 128 query rows per K/V head (several row blocks), bf16 and fp32."""
    for dtype, d in (("bf16", 64), ("f32", 16)):
        h, h_kv, B, Tq, Tmax = 8, 1, 2, 33, 400
        lengths = [400, 70]
        Q, K, V = _cache(99, dtype, B, Tq, Tmax, h, h_kv, d, d)
        t = [to_device(x, dtype) for x in (Q, K, V)]
        layer = _layer(dtype, h, d, h_kv)
        ref, A, _ = lc.decode(Q, K, V, h, lengths, h_kv, 50, 3)
        _check(to_host(layer.decode_window(*t, _lens(lengths), 50, 3)), ref, A, dtype, "window, 264 rows")
        w0 = np.zeros((B, h_kv, Tmax), dtype=np.float32)
        w = to_device(w0, "f32")
        ref, A, W = lc.decode(Q, K, V, h, lengths, h_kv, weights=w0)
        _check(to_host(layer.decode_weights(*t, _lens(lengths), w)), ref, A, dtype, "weights, 264 rows")
        _check_weights(to_host(w)[0], W[0], "weights, 264 rows")


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 16)])
def test_long_cache_few_groups(dtype, d):
    """One sequence, one K/V head, a long cache: every CTA holds a piece of the same group."""
    h, h_kv, B, Tq, Tmax = 4, 1, 1, 1, 50001
    Q, K, V = _cache(101, dtype, B, Tq, Tmax, h, h_kv, d, d)
    t = [to_device(x, dtype) for x in (Q, K, V)]
    layer = _layer(dtype, h, d, h_kv)
    w0 = np.zeros((B, h_kv, Tmax), dtype=np.float32)
    w = to_device(w0, "f32")
    ref, A, W = lc.decode(Q, K, V, h, [Tmax], h_kv, weights=w0)
    _check(to_host(layer.decode_weights(*t, _lens([Tmax]), w)), ref, A, dtype, "long cache")
    _check_weights(to_host(w), W, "long cache weights")
    ref, A, _ = lc.decode(Q, K, V, h, [Tmax], h_kv, 30001, 100)
    _check(to_host(layer.decode_window(*t, _lens([Tmax]), 30001, 100)), ref, A, dtype, "long window")


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 16)])
def test_many_short_sequences(dtype, d):
    """More groups than CTAs, and more sequences than a block has threads."""
    h, h_kv, B, Tq, Tmax = 2, 2, 333, 1, 40
    lengths = [1 + (7 * b) % Tmax for b in range(B)]
    lengths[5] = 0
    Q, K, V = _cache(103, dtype, B, Tq, Tmax, h, h_kv, d, d)
    t = [to_device(x, dtype) for x in (Q, K, V)]
    layer = _layer(dtype, h, d, h_kv)
    ref, A, _ = lc.decode(Q, K, V, h, lengths, h_kv, 20, 2)
    got = to_host(layer.decode_window(*t, _lens(lengths), 20, 2))
    ok = [b for b in range(B) if b != 5]
    assert np.isnan(got[5]).all()
    _check(got[ok], ref[ok], A[ok], dtype, "many sequences")
    ref, A, _ = lc.decode(Q, K, V, h, lengths, h_kv, K_prefix=K[0], V_prefix=V[0])
    got = to_host(layer.decode_shared(t[0], t[1][0], t[2][0], t[1], t[2], _lens(lengths)))
    _check(got[ok], ref[ok], A[ok], dtype, "many sequences, shared")


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 16)])
def test_views_of_one_cache_buffer(dtype, d):
    """K and V as column views of one [K | V] buffer, Q the last token of a longer tensor."""
    h, h_kv, B, Tmax = 4, 2, 3, 400
    kv = _rand((B, Tmax, 2 * h_kv * d), 105, dtype)
    x = _rand((B, 9, h * d), 106, dtype)
    t, tx = to_device(kv, dtype), to_device(x, dtype)
    K, V = kv[..., :h_kv * d], kv[..., h_kv * d:]
    layer = _layer(dtype, h, d, h_kv)
    lengths = [400, 123, 64]
    out = torch.full((B, 5, h * d), 3.0, dtype=torch_dtype(dtype), device="cuda")
    layer.decode_window(tx[:, -1:], t[..., :h_kv * d], t[..., h_kv * d:], _lens(lengths), 99, 4, out=out[:, 2:3])
    ref, A, _ = lc.decode(x[:, -1:], K, V, h, lengths, h_kv, 99, 4)
    got = to_host(out)
    _check(got[:, 2:3], ref, A, dtype, "views")
    assert (got[:, :2] == 3).all() and (got[:, 3:] == 3).all()


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements: the last sequence's rows lie past every 32-bit offset."""
    h = h_kv = 16
    d, B, Tmax = 128, 5, 450_000
    K = torch.empty((B, Tmax, h_kv * d), dtype=torch.bfloat16, device="cuda")
    V = torch.empty_like(K)
    assert K.numel() > 2 ** 32
    n = 600
    lengths = [n, n, n, n, Tmax]
    Q = _rand((B, 1, h * d), 107, "bf16")
    kb, vb = _rand((n, h_kv * d), 108, "bf16"), _rand((n, h_kv * d), 109, "bf16")
    for b in range(4):
        K[b, :n], V[b, :n] = to_device(kb, "bf16"), to_device(vb, "bf16")
    K[4, Tmax - n:], V[4, Tmax - n:] = to_device(kb, "bf16"), to_device(vb, "bf16")
    layer = _layer("bf16", h, d, h_kv)
    got = to_host(layer.decode_window(to_device(Q, "bf16"), K, V, _lens(lengths), n, 0))
    ref, A, _ = lc.decode(Q, np.broadcast_to(kb, (B, n, h * d)), np.broadcast_to(vb, (B, n, h * d)), h, [n] * B, h_kv)
    _check(got, ref, A, "bf16", "past 32 bits")
    w = torch.zeros((B, h_kv, Tmax), device="cuda")
    w[4, :, Tmax - n:] = 1.0
    Ko, Vo, lo, wo, kept = layer.evict(K, V, _lens(lengths), w, n, 10)
    assert torch.equal(Ko[4], K[4, Tmax - n:]) and torch.equal(Vo[4], V[4, Tmax - n:])
    assert lo.tolist() == [n] * 5


# ------------------------------------------------------------------ eviction

def _evict_case(layer, dtype, B, T, h_kv, d, dv, lengths, w, keep, recent, seed, T_out=None, in_place=False, fused=False):
    if fused:
        buf = to_device(_rand((B, T, h_kv * (d + dv)), seed, dtype), dtype)
        K, V = buf[..., :h_kv * d], buf[..., h_kv * d:]
    else:
        K, V = to_device(_rand((B, T, h_kv * d), seed, dtype), dtype), to_device(_rand((B, T, h_kv * dv), seed + 1, dtype), dtype)
    K0, V0 = to_host(K), to_host(V)
    w = np.ascontiguousarray(w)
    tw = torch.tensor(w, dtype=torch.float32, device="cuda")
    T_out = keep if T_out is None else T_out
    lens = _lens(lengths)
    if in_place:
        Ko, Vo, lo, wo, kept = layer.evict(K, V, lens, tw, keep, recent, K_out=K, V_out=V, weights_out=tw, lengths_out=lens)
        assert lo is lens
        rows = T
    else:
        Ko = torch.full((B, T_out, h_kv * d), 5.0, dtype=K.dtype, device="cuda")
        Vo = torch.full((B, T_out, h_kv * dv), 5.0, dtype=K.dtype, device="cuda")
        wo = torch.full((B, h_kv, T_out), 5.0, device="cuda")
        Ko, Vo, lo, wo, kept = layer.evict(K, V, lens, tw, keep, recent, K_out=Ko, V_out=Vo, weights_out=wo)
        rows = T_out
    ref = lc.evict(np.asarray(w, np.float32), lengths, keep, recent)
    Ko, Vo, wo, kept = to_host(Ko), to_host(Vo), wo.cpu().numpy(), kept.cpu().numpy()
    w32 = np.asarray(w, np.float32)
    for b, g in itertools.product(range(B), range(h_kv)):
        want = ref[b][g]
        n = 0 if want is None else len(want)
        assert kept[b, g, :n].tolist() == (want or []) and (kept[b, g, n:] == -1).all()
        assert lo[b].item() == n
        for got, src, width in ((Ko, K0, d), (Vo, V0, dv)):
            c = slice(g * width, (g + 1) * width)
            assert (got[b, :n, c] == src[b, want or [], c]).all()
            rest = src[b, n:rows, c] if in_place else 5.0
            assert (got[b, n:, c] == rest).all()          # rows behind the kept ones stay
        assert np.array_equal(wo[b, g, :n], w32[b, g, want or []], equal_nan=True)
        rest = w32[b, g, n:rows] if in_place else np.full(rows - n, 5.0, np.float32)
        assert np.array_equal(wo[b, g, n:], rest, equal_nan=True)


EVICT_SHAPES = [("bf16", 64, 64, 2), ("bf16", 128, 128, 3), ("f32", 16, 20, 2), ("f32", 7, 3, 2)]


@pytest.mark.parametrize("dtype,d,dv,h_kv", EVICT_SHAPES)
@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (40, 40), (40, 0), (257, 30), (1500, 700), (3100, 5)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(dtype, d, dv, h_kv, keep, recent, in_place):
    B, T = 4, 3300
    lengths = [3300, 0, min(keep, 3300), 1025]
    rng = np.random.default_rng(keep + recent)
    w = np.exp(2 * rng.standard_normal((B, h_kv, T)))
    layer = _layer(dtype, h_kv, d, h_kv, dv)
    _evict_case(layer, dtype, B, T, h_kv, d, dv, lengths, w, keep, recent, 5, T_out=keep + 3, in_place=in_place)
    assert layer.status() == 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["ties", "zeros", "special", "close", "sorted", "reversed"])
def test_evict_orders(kind, in_place):
    """Ties go to the lower index; NaN lies lowest; signed zeros are equal; infinities and subnormals
    take their places; keys that differ in their last bit only."""
    B, h_kv, T, keep, recent = 2, 2, 2100, 700, 100
    rng = np.random.default_rng(7)
    w = rng.integers(0, 4, (B, h_kv, T)).astype(np.float64)
    if kind == "zeros":
        w = np.where(rng.random(w.shape) < 0.5, 0.0, -0.0)
    if kind == "special":
        w = rng.choice([np.nan, np.inf, -np.inf, -1.0, -0.0, 0.0, 1e-42, 3.0], w.shape)
    if kind == "close":
        w = 1.0 + rng.integers(0, 40, w.shape) * 2.0 ** -23
    if kind == "sorted":
        w = np.broadcast_to(np.arange(T, dtype=float), w.shape)
    if kind == "reversed":
        w = np.broadcast_to(np.arange(T, dtype=float)[::-1], w.shape)
    layer = _layer("bf16", h_kv, 64, h_kv)
    _evict_case(layer, "bf16", B, T, h_kv, 64, 64, [T, 1500], w, keep, recent, 9, in_place=in_place)


@pytest.mark.parametrize("T", [16384, 17000, 50000, 70001])
@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_long(T, ties, in_place):
    """Caches longer than one scan of the selection, and longer than shared memory holds."""
    rng = np.random.default_rng(T)
    w = rng.integers(0, 3, (2, 1, T)).astype(float) if ties else rng.random((2, 1, T))
    layer = _layer("f32", 1, 4, 1)
    _evict_case(layer, "f32", 2, T, 1, 4, 4, [T, T - 333], w, T - 1000 if ties else T // 3, 77, 13, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_views_of_one_buffer_and_invalid_lengths(in_place):
    layer = _layer("bf16", 4, 64, 4)
    w = np.random.default_rng(1).random((4, 4, 900))
    _evict_case(layer, "bf16", 4, 900, 4, 64, 64, [900, -1, 901, 300], w, 256, 32, 11, in_place=in_place, fused=True)
    assert layer.status() == _lib.MHA_ERR_BAD_LENGTH


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 6)])
@pytest.mark.parametrize("shared", ["outputs", "all"])
def test_evict_into_column_views(dtype, d, shared):
    """K_out and V_out as columns of one buffer, or of the buffer that the caches are columns of."""
    h_kv, B, T, keep, recent = 2, 3, 500, 120, 20
    w_, lengths = h_kv * d, [500, 119, 301]
    buf = to_device(_rand((B, T, 4 * w_), 31, dtype), dtype)
    K, V = buf[..., :w_], buf[..., w_:2 * w_]
    out = buf if shared == "all" else torch.full((B, keep + 9, 4 * w_), 5.0, dtype=torch_dtype(dtype), device="cuda")
    Ko, Vo = out[..., 2 * w_:3 * w_], out[..., 3 * w_:]
    before, src = to_host(out), to_host(buf)
    w = np.random.default_rng(3).random((B, h_kv, T)).astype(np.float32)
    layer = _layer(dtype, h_kv, d, h_kv)
    wo = torch.zeros((B, h_kv, out.shape[1]), device="cuda")
    layer.evict(K, V, _lens(lengths), torch.tensor(w, device="cuda"), keep, recent, K_out=Ko, V_out=Vo, weights_out=wo)
    ref, got = lc.evict(w, lengths, keep, recent), to_host(out)
    for b, g in itertools.product(range(B), range(h_kv)):
        n, at = len(ref[b][g]), ref[b][g]
        for i in range(2):
            c = slice((2 + i) * w_ + g * d, (2 + i) * w_ + (g + 1) * d)
            f = slice(i * w_ + g * d, i * w_ + (g + 1) * d)
            assert (got[b, :n, c] == src[b, at, f]).all() and (got[b, n:, c] == before[b, n:, c]).all()
    assert (got[..., :2 * w_] == before[..., :2 * w_]).all()
    assert layer.status() == 0


def test_evict_budget_whose_indices_pass_32_bits():
    """h_kv * keep beyond 2^31: the kept tokens' indices of the last head lie past every 32-bit offset."""
    h_kv, T, L = 17, 100, 60
    keep = 2 ** 27 + 5
    layer = _layer("f32", h_kv, 1, h_kv, 1)
    K, V = (to_device(_rand((1, T, h_kv), s, "f32"), "f32") for s in (21, 22))
    w = to_device(_rand((1, h_kv, T), 23, "f32"), "f32")
    Ko, Vo = (torch.full((1, keep, h_kv), 5.0, device="cuda") for _ in range(2))
    wo = torch.full((1, h_kv, keep), 5.0, device="cuda")
    _, _, lo, _, kept = layer.evict(K, V, _lens([L]), w, keep, 7, K_out=Ko, V_out=Vo, weights_out=wo)
    assert h_kv * keep > 2 ** 31 and kept.shape == (1, h_kv, keep) and lo.tolist() == [L]
    assert (kept[0, :, :L] == torch.arange(L, device="cuda")).all() and (kept[0, :, L:] == -1).all()
    for got, src in ((Ko, K), (Vo, V)):
        assert torch.equal(got[:, :L], src[:, :L]) and (got[:, L:] == 5).all()
    assert torch.equal(wo[..., :L], w[..., :L]) and (wo[..., L:] == 5).all()
    assert layer.status() == 0


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 32)])
def test_generation_with_eviction(dtype, d):
    """As they would be used: a few prompts, decode steps that accumulate weights, an eviction in place when
    the caches reach their budget, more steps on what is left; every step against the 64-bit model of
    the same cache."""
    h, h_kv, B, Tmax, keep, recent = 4, 2, 2, 200, 96, 16
    rng = np.random.default_rng(d)
    lens = [150, 140]
    K, V = _rand((B, Tmax, h_kv * d), 1, dtype), _rand((B, Tmax, h_kv * d), 2, dtype)
    W = np.zeros((B, h_kv, Tmax), dtype=np.float64)
    layer = _layer(dtype, h, d, h_kv)
    tK, tV, tw, tl = to_device(K, dtype), to_device(V, dtype), to_device(W, "f32"), _lens(lens)
    K, V = K.astype(np.float64), V.astype(np.float64)
    for step in range(60):
        new = [_rand((B, 1, n * d), 1000 + 3 * step + i, dtype) for i, n in enumerate((h, h_kv, h_kv))]
        for b in range(B):
            K[b, lens[b]], V[b, lens[b]] = new[1][b, 0], new[2][b, 0]
            lens[b] += 1
        at = tl.long()[:, None, None].expand(B, 1, h_kv * d)
        tK.scatter_(1, at, to_device(new[1], dtype))
        tV.scatter_(1, at, to_device(new[2], dtype))
        tl += 1
        got = to_host(layer.decode_weights(to_device(new[0], dtype), tK, tV, tl, tw))
        ref, A, W = lc.decode(new[0], K, V, h, lens, h_kv, weights=W)
        _check(got, ref, A, dtype, f"step {step}")
        gw = to_host(tw)
        for b in range(B):
            _check_weights(gw[b, :, :lens[b]], W[b, :, :lens[b]], f"step {step}")
        if max(lens) >= Tmax - 20:
            # the GPU goes by its own fp32 weights: the model follows them
            _, _, _, _, kept = layer.evict(tK, tV, tl, tw, keep, recent, K_out=tK, V_out=tV, weights_out=tw,
                                           lengths_out=tl)
            want = lc.evict(gw.astype(np.float32), lens, keep, recent)
            assert kept.tolist() == want
            for b, g in itertools.product(range(B), range(h_kv)):
                c = slice(g * d, (g + 1) * d)
                K[b, :keep, c], V[b, :keep, c] = K[b, want[b][g], c], V[b, want[b][g], c]
                W[b, g, :keep] = W[b, g, want[b][g]]
            lens = [keep, keep]
            assert tl.tolist() == lens
    assert layer.status() == 0


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 16)])
def test_captured_and_replayed(dtype, d):
    """All steps captured in one graph and replayed with new contents and lengths in the same buffers; a
    larger eager call of the same layer in between must not disturb the graph."""
    h, h_kv, B, Tq, Tmax, Tp = 4, 2, 3, 1, 500, 200
    layer = _layer(dtype, h, d, h_kv)
    Q, K, V = (torch.zeros(s, dtype=torch_dtype(dtype), device="cuda")
               for s in ((B, Tq, h * d), (B, Tmax, h_kv * d), (B, Tmax, h_kv * d)))
    Kp, Vp = torch.zeros_like(K[0, :Tp]), torch.zeros_like(V[0, :Tp])
    lens, w = _lens([5, 5, 5]), torch.zeros((B, h_kv, Tmax), device="cuda")
    outs = [torch.zeros((B, Tq, h * d), dtype=torch_dtype(dtype), device="cuda") for _ in range(3)]
    ev = [torch.zeros((B, 64, h_kv * d), dtype=torch_dtype(dtype), device="cuda") for _ in range(2)]
    wo, lo = torch.zeros((B, h_kv, 64), device="cuda"), torch.zeros_like(lens)

    def steps():
        layer.decode_window(Q, K, V, lens, 77, 3, out=outs[0])
        layer.decode_shared(Q, Kp, Vp, K, V, lens, out=outs[1])
        layer.decode_weights(Q, K, V, lens, w, out=outs[2])
        return layer.evict(K, V, lens, w, 64, 8, K_out=ev[0], V_out=ev[1], weights_out=wo, lengths_out=lo)[4]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        steps()
        steps()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = steps()
    big = torch.randn((9, 3000, h_kv * d), device="cuda").to(torch_dtype(dtype))
    layer.decode_weights(big[:, :4, :1].expand(9, 4, h * d).contiguous(), big, big, _lens([3000] * 9),
                         torch.zeros((9, h_kv, 3000), device="cuda"))
    filler = torch.full((1 << 24,), 3, dtype=torch.uint8, device="cuda")  # would take a freed workspace's place
    for seed, lengths in ((1, [500, 1, 90]), (2, [64, 333, 500])):
        q, k, v = _cache(200 + seed, dtype, B, Tq, Tmax, h, h_kv, d, d)
        kp, vp = _rand((Tp, h_kv * d), 210 + seed, dtype), _rand((Tp, h_kv * d), 220 + seed, dtype)
        for dst, src in ((Q, q), (K, k), (V, v), (Kp, kp), (Vp, vp)):
            dst.copy_(to_device(src, dtype))
        lens.copy_(_lens(lengths))
        w.zero_()
        g.replay()
        torch.cuda.synchronize()
        for out, kw in zip(outs, (dict(window=77, sinks=3), dict(K_prefix=kp, V_prefix=vp), {})):
            ref, A, W = lc.decode(q, k, v, h, lengths, h_kv, weights=np.zeros(w.shape), **kw)
            _check(to_host(out), ref, A, dtype, "replayed")
        assert (filler == 3).all()
        want = lc.evict(w.cpu().numpy(), lengths, 64, 8)
        for b, gg in itertools.product(range(B), range(h_kv)):
            n = len(want[b][gg])
            assert kept[b, gg, :n].tolist() == want[b][gg]
        assert lo.tolist() == [min(x, 64) for x in lengths]


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 16)])
def test_on_another_stream(dtype, d):
    """Two layers on two streams at once, each with its own workspace."""
    h, h_kv, B, Tmax = 4, 2, 2, 2000
    Q, K, V = _cache(301, dtype, B, 1, Tmax, h, h_kv, d, d)
    t = [to_device(x, dtype) for x in (Q, K, V)]
    lengths = [2000, 1111]
    ref, A, _ = lc.decode(Q, K, V, h, lengths, h_kv, 600, 5)
    lens = _lens(lengths)
    layers = [_layer(dtype, h, d, h_kv) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                outs[i].append(layers[i].decode_window(*t, lens, 600, 5))
    torch.cuda.synchronize()
    for o in outs[0] + outs[1]:
        _check(to_host(o), ref, A, dtype, "streams")


# Few query rows per K/V head in fp32 (they take a kernel of their own): every number of rows and width
# that it holds, and one more row.
FEW_SHAPES = [
    # d, d_v, h, h_kv, T_q
    (64, 64, 4, 4, 1), (64, 60, 8, 4, 2), (61, 64, 4, 4, 1), (32, 64, 8, 1, 1), (64, 64, 9, 1, 1),
    (128, 128, 4, 4, 1), (128, 96, 4, 2, 2), (66, 65, 4, 4, 2), (100, 100, 5, 1, 1),
    (256, 256, 2, 2, 1), (200, 256, 4, 2, 1), (130, 255, 2, 2, 2), (256, 192, 3, 1, 1)]


@pytest.mark.parametrize("d,dv,h,h_kv,Tq", FEW_SHAPES)
def test_few_rows_f32(d, dv, h, h_kv, Tq):
    B, Tmax, Tp = 3, 700, 150
    lengths = [700, Tq, 261]
    Q, K, V = _cache(400 + d + dv, "f32", B, Tq, Tmax, h, h_kv, d, dv)
    Kp, Vp = _rand((Tp, h_kv * d), 401, "f32"), _rand((Tp, h_kv * dv), 402, "f32")
    Kn, Vn = _garbage(K, V, lengths)
    t = [to_device(x, "f32") for x in (Q, Kn, Vn)]
    layer = _layer("f32", h, d, h_kv, dv)
    for window, sinks in ((200, 5), (64, 0), (1, 0)):
        ref, A, _ = lc.decode(Q, K, V, h, lengths, h_kv, window, sinks)
        _check(to_host(layer.decode_window(*t, _lens(lengths), window, sinks)), ref, A, "f32", "few rows, window")
    # the prefix's rows are the batch's: another kernel than the caches' where those are many
    ref, A, _ = lc.decode(Q, K, V, h, lengths, h_kv, K_prefix=Kp, V_prefix=Vp)
    _check(to_host(layer.decode_shared(t[0], to_device(Kp, "f32"), to_device(Vp, "f32"), *t[1:], _lens(lengths))),
           ref, A, "f32", "few rows, shared")
    w0 = np.abs(_rand((B, h_kv, Tmax), 403, "f32"))
    w = to_device(w0, "f32")
    ref, A, W = lc.decode(Q, K, V, h, lengths, h_kv, weights=w0)
    _check(to_host(layer.decode_weights(*t, _lens(lengths), w)), ref, A, "f32", "few rows, weights")
    for b, L in enumerate(lengths):
        _check_weights(to_host(w)[b, :, :L], W[b, :, :L], "few rows, weights")
    assert layer.status() == 0


@pytest.mark.parametrize("Tq", [1, 9])
def test_offsets_past_32_bits_f32(Tq):
    h = h_kv = 16
    d, B, Tmax = 64, 5, 850_000
    K = torch.empty((B, Tmax, h_kv * d), device="cuda")
    V = torch.empty_like(K)
    assert K.numel() > 2 ** 32
    n = 300
    lengths = [n, n, n, n, Tmax]
    Q = _rand((B, Tq, h * d), 110, "f32")
    kb, vb = _rand((n, h_kv * d), 111, "f32"), _rand((n, h_kv * d), 112, "f32")
    for b in range(4):
        K[b, :n], V[b, :n] = to_device(kb, "f32"), to_device(vb, "f32")
    K[4, Tmax - n:], V[4, Tmax - n:] = to_device(kb, "f32"), to_device(vb, "f32")
    layer = _layer("f32", h, d, h_kv)
    W = n - Tq + 1  # the first new token's window begins with the filled rows
    got = to_host(layer.decode_window(to_device(Q, "f32"), K, V, _lens(lengths), W, 0))
    ref, A, _ = lc.decode(Q, np.broadcast_to(kb, (B, n, h * d)), np.broadcast_to(vb, (B, n, h * d)), h, [n] * B, h_kv, W, 0)
    _check(got, ref, A, "f32", "past 32 bits")


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 64)])
def test_two_graphs_share_a_workspace(dtype, d):
    """Graphs of different sizes captured from one layer, replayed in turn with eager calls between them."""
    h, h_kv = 8, 2
    layer = _layer(dtype, h, d, h_kv)
    cases = []
    for i, (B, Tmax, lengths) in enumerate(((1, 1500, [1500]), (7, 400, [400, 3, 77, 128, 399, 1, 200]))):
        Q, K, V = _cache(500 + 10 * i, dtype, B, 1, Tmax, h, h_kv, d, d)
        t = [to_device(x, dtype) for x in (Q, K, V)]
        w0 = np.zeros((B, h_kv, Tmax), dtype=np.float32)
        ref, A, W = lc.decode(Q, K, V, h, lengths, h_kv, weights=w0)
        out = torch.zeros((B, 1, h * d), dtype=torch_dtype(dtype), device="cuda")
        cases.append((t, _lens(lengths), lengths, to_device(w0, "f32"), out, ref, A, W))
    for t, lens, _, w, out, *_ in cases[::-1]:
        layer.decode_weights(*t, lens, w, out=out)
    torch.cuda.synchronize()
    graphs = []
    for t, lens, _, w, out, *_ in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.decode_weights(*t, lens, w, out=out)
        graphs.append(g)
    for turn in range(3):
        for i in (0, 1, 1, 0):
            t, lens, lengths, w, out, ref, A, W = cases[i]
            w.zero_()
            out.zero_()
            graphs[i].replay()
            _check(to_host(out), ref, A, dtype, "graph")
            for b, L in enumerate(lengths):
                _check_weights(to_host(w)[b, :, :L], W[b, :, :L], "graph")
            t, lens, _, w, out, ref, A, _ = cases[1 - i]
            _check(to_host(layer.decode_weights(*t, lens, w)), ref, A, dtype, "eager between graphs")
    assert layer.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_status_word_outlives_a_larger_workspace(dtype):
    """attention_window and evict need the workspace for its status word only: one that a graph of them was
    captured with stays theirs when a larger call replaces it."""
    h, h_kv, d, B, T = 4, 2, 64, 2, 100
    for op in ("window", "evict"):
        layer = _layer(dtype, h, d, h_kv)
        Q, K, V = (to_device(x, dtype) for x in _cache(600, dtype, B, T, T, h, h_kv, d, d))
        lens, w = _lens([T, T + 1]), torch.ones((B, h_kv, T), device="cuda")  # the second is invalid

        def call():
            if op == "window":
                return layer.attention_window(Q, K, V, 10, kv_lengths=lens)
            return layer.evict(K, V, lens, w, 10, 2)
        layer.ensure_workspace(0, 0, 0, need=256)
        call()
        assert layer.status() == 6
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        old = layer._ws
        layer.ensure_workspace(0, 0, 0, need=1 << 20)
        assert layer._ws is not old and any(x is old for x in layer._kept_ws)
        g.replay()
        torch.cuda.synchronize()
        assert int(old[:4].view(torch.int32).item()) == 6 and layer.status() == 0


# ------------------------------------------------------------------ workspaces

def _busy(ms=30.0):
    """About that many milliseconds of ordinary work on the current stream (a product of 8192^3 takes more
    than half a millisecond)."""
    a = torch.zeros((8192, 8192), dtype=torch.bfloat16, device="cuda")
    for _ in range(int(ms / 0.55)):
        a = a @ a


def _step_cases(dtype, d, seed, h=8, h_kv=2):
    """A small and a larger batch for decode_weights: tensors, lengths, and the 64-bit results."""
    cases = []
    for i, (B, Tmax, lengths) in enumerate(((2, 700, [700, 391]), (6, 2000, [2000, 1, 1333, 640, 129, 1999]))):
        Q, K, V = _cache(seed + 10 * i, dtype, B, 1, Tmax, h, h_kv, d, d)
        t = [to_device(x, dtype) for x in (Q, K, V)]
        w0 = np.zeros((B, h_kv, Tmax), dtype=np.float32)
        ref, A, W = lc.decode(Q, K, V, h, lengths, h_kv, weights=w0)
        cases.append((t, _lens(lengths), lengths, to_device(w0, "f32"), ref, A, W))
    return cases


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 32)])
def test_workspace_of_a_side_stream_under_a_busy_default_stream(dtype, d):
    """The first and a larger step on a side stream, in memory that still has writes pending there, while the
    default stream is busy: each starts from a zeroed status block."""
    h, h_kv = 8, 2
    cases = _step_cases(dtype, d, 700)
    layer = _layer(dtype, h, d, h_kv)
    sizes = [_lib.mha_cache_step_workspace_size(layer.handle, len(c[2]), 1, 0, c[0][1].shape[1], 1) for c in cases]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _busy(1.0)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    _busy()
    with torch.cuda.stream(side):
        dirty = []
        for c, n in zip(cases, sizes):
            out = torch.empty((len(c[2]), 1, h * d), dtype=torch_dtype(dtype), device="cuda")
            _busy(2.0)
            x = torch.full((n,), 1, dtype=torch.uint8, device="cuda")  # counters of 0x01010101
            dirty.append(x.data_ptr())
            del x
            layer.decode_weights(*c[0], c[1], c[3], out=out)
            assert layer._ws.data_ptr() == dirty[-1]                   # or this tests nothing
            c[0].append(out)
        status = layer.status()
    assert status == 0
    torch.cuda.synchronize()
    for t, _, lengths, w, ref, A, W in cases:
        _check(to_host(t[3]), ref, A, dtype, "side stream")
        for b, n in enumerate(lengths):
            _check_weights(to_host(w)[b, :, :n], W[b, :, :n], "side stream")


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 32)])
def test_workspace_attached_under_capture(dtype, d):
    """A layer whose first steps are captured: eager steps before the first replay, then replays, then eager
    steps again, all from the same workspace."""
    h, h_kv = 8, 2
    cases = _step_cases(dtype, d, 750)
    warm = _layer(dtype, h, d, h_kv)
    for t, lens, _, w, *_ in cases:
        warm.decode_weights(*t, lens, w)
    torch.cuda.synchronize()
    layer = _layer(dtype, h, d, h_kv)
    outs = [torch.zeros((len(c[2]), 1, h * d), dtype=torch_dtype(dtype), device="cuda") for c in cases]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        # a temporary of the graph where its pool may hand out memory again
        torch.full((1 << 22,), 1, dtype=torch.uint8, device="cuda")
        for (t, lens, _, w, *_), out in zip(cases, outs):
            layer.decode_weights(*t, lens, w, out=out)
    ws = layer._ws
    for turn in range(3):
        for (t, lens, lengths, w, ref, A, W), out in zip(cases, outs):
            w.zero_()
            _check(to_host(layer.decode_weights(*t, lens, w)), ref, A, dtype, "eager")
            assert layer._ws is ws
            out.zero_()
            w.zero_()
        g.replay()
        for (t, lens, lengths, w, ref, A, W), out in zip(cases, outs):
            _check(to_host(out), ref, A, dtype, "replayed")
            for b, n in enumerate(lengths):
                _check_weights(to_host(w)[b, :, :n], W[b, :, :n], "replayed")
    assert layer.status() == 0


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 32)])
def test_replaced_workspace_stays_until_its_steps_are_through(dtype, d):
    """A step on a side stream with a workspace of the default stream, then a larger one there: the memory of the
    first must not be given to a tensor of the default stream before the step has run."""
    h, h_kv = 8, 2
    cases = _step_cases(dtype, d, 800)
    layer = _layer(dtype, h, d, h_kv)
    (t, lens, _, w, *_), (t2, lens2, _, w2, *_) = cases
    layer.decode_weights(*t, lens, w)
    w.zero_()
    torch.cuda.synchronize()
    old, n = layer._ws.data_ptr(), layer._ws.numel()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        outs = [torch.empty((len(c[2]), 1, h * d), dtype=torch_dtype(dtype), device="cuda") for c in cases]
        _busy()
        layer.decode_weights(*t, lens, w, out=outs[0])
        layer.decode_weights(*t2, lens2, w2, out=outs[1])
    assert layer._ws.data_ptr() != old
    taken = [torch.full((n,), 1, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert not any(x.data_ptr() <= old < x.data_ptr() + n for x in taken)
    torch.cuda.synchronize()
    for (_, _, lengths, w, ref, A, W), out in zip(cases, outs):
        _check(to_host(out), ref, A, dtype, "replaced workspace")
        for b, m in enumerate(lengths):
            _check_weights(to_host(w)[b, :, :m], W[b, :, :m], "replaced workspace")
    assert layer.status() == 0


# ------------------------------------------------------------------ schedules, host threads, non-finite queries

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("step", ["window", "shared", "weights"])
def test_results_do_not_depend_on_the_schedule(d, step):
    """Several units of odd tile counts per CTA, taken from a counter: 50 runs give the same bits while another
    stream's work varies which CTA takes which."""
    h, h_kv, B, Tmax = 16, 16, 40, 3000
    gen = torch.Generator(device="cuda").manual_seed(d)
    Q, K, V, Kp, Vp = (torch.randn(s, generator=gen, device="cuda").bfloat16() for s in (
        (B, 2, h * d), (B, Tmax, h_kv * d), (B, Tmax, h_kv * d), (5000, h_kv * d), (5000, h_kv * d)))
    lens = torch.randint(2, Tmax + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    w0 = torch.rand((B, h_kv, Tmax), generator=gen, device="cuda")
    layer = _layer("bf16", h, d, h_kv)
    side = torch.cuda.Stream()
    noise = torch.zeros((1 << 24,), device="cuda")

    def run():
        w = w0.clone()
        if step == "window":
            return layer.decode_window(Q, K, V, lens, 1777, 5), w
        if step == "shared":
            return layer.decode_shared(Q, Kp, Vp, K, V, lens), w
        return layer.decode_weights(Q, K, V, lens, w), w
    first = run()
    torch.cuda.synchronize()
    differ = 0
    for i in range(50):
        with torch.cuda.stream(side):
            for _ in range(i % 4):
                noise[: 1 << (14 + i % 11)].add_(1.0)
        again = run()
        differ += not all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(first, again))
        side.synchronize()
    assert differ == 0
    assert layer.status() == 0


# Two layers of one kernel instantiation that need different amounts of shared memory.
THREAD_CASES = {
    # operator: (d_k, d_v, tokens) of the smaller and of the larger layer
    "evict": ((4, 4, 9000), (4, 4, 45000)), "attention_window": ((16, 48, 40), (256, 48, 40)),
    "decode_window": ((16, 48, 40), (256, 48, 40)), "attention": ((16, 48, 40), (256, 48, 40)),
    "decode": ((16, 48, 40), (256, 256, 40))}


@pytest.mark.parametrize("op", THREAD_CASES)
def test_layers_of_different_sizes_in_two_threads(op, monkeypatch):
    """Each host thread has a layer and a stream of its own: what one launches must not change the shared-memory
    limit that the other's launch of the same kernel needs."""
    import threading
    entry = {"evict": "mha_cache_evict", "attention": "mha_attention_ex"}.get(op, f"mha_{op}")
    real, taken = getattr(_lib, entry), []
    monkeypatch.setattr(_lib, entry, lambda *a: taken.append(a) or real(*a))
    jobs, keep = [], []
    for d, dv, T in THREAD_CASES[op]:
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            layer = _layer("f32", 1, d, 1, dv)
            Q, K, V = (torch.zeros((1, T, n), device="cuda") for n in (d, d, dv))
            q = torch.zeros((1, 20, d), device="cuda")
            if op == "evict":
                lens, w = _lens([50]), torch.zeros((1, 1, T), device="cuda")
                out = layer.evict(K, V, lens, w, 100, 10)
            elif op == "attention_window":
                lens, w, out = None, None, layer.attention_window(Q, K, V, 8)
            elif op == "attention":
                lens, w, out = None, None, layer.attention(Q, K, V, causal=True)
            else:
                lens, w = _lens([T]), torch.zeros((1, 20, dv), device="cuda")
                out = layer.decode_window(q, K, V, lens, 8, out=w) if op == "decode_window" else \
                    layer.decode(q, K, V, lens, out=w)
        keep.append((layer, Q, q, K, V, lens, w, out))
        jobs.append((taken[-1], stream))
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(2)

    def work(args, stream):
        start.wait()
        try:
            for i in range(10000):   # the C entry by itself: no interpreter lock is held in it
                real(*args)
                if i % 500 == 0:
                    stream.synchronize()
        except Exception as e:  # noqa: BLE001 (reported below)
            failed.append(e)
    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed


def _non_finite_queries(Q, d):
    """Rows of head 0 that hold a NaN, an infinity of either sign, or one that makes every score -inf (the keys'
    first element is positive); the row numbers."""
    rows = {3: (1, np.nan), 40: (1, np.inf), 41: (1, -np.inf), 100: (0, -np.inf), 150: (0, np.inf), 0: (0, -np.inf),
            199: (0, -np.inf)}
    for i, (e, x) in rows.items():
        Q[:, i, e] = x
    return sorted(rows)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 16), ("f32", 200)])
@pytest.mark.parametrize("window,sinks", [(1000, 0), (30, 0), (30, 3), (1, 0), (130, 140)])
@pytest.mark.parametrize("gated", [False, True])
def test_window_non_finite_queries(dtype, d, window, sinks, gated):
    """A query row that is not finite gives NaN in its head, as in attention(); zeros are for padding rows that
    see no key, whatever their queries hold.  The other rows and heads are as without it."""
    h, h_kv, B, T = 2, 1, 2, 230
    lengths = [230, 120]
    Q, K, V = (_rand((B, T, n * d), s, dtype) for s, n in ((11, h), (12, h_kv), (13, h_kv)))
    G = _rand((B, T, h * d), 14, dtype) if gated else None
    K[..., 0] = np.abs(K[..., 0]) + 0.25                     # (exact enough: rounded again below)
    if dtype == "bf16":
        K = wl.bf16_to_f32(wl.bf16_bits(np.ascontiguousarray(K, dtype=np.float32)))
    ref, A = lc.attention_window(Q, K, V, h, window, sinks, h_kv, lengths, G)
    Qn = Q.copy()
    rows = _non_finite_queries(Qn, d)
    layer = _layer(dtype, h, d, h_kv, gated=gated)
    t = [to_device(x, dtype) for x in (Qn, K, V)]
    tg = to_device(G, dtype)
    got = to_host(layer.attention_window(*t, window, sinks, kv_lengths=_lens(lengths), G=tg))
    i, j = np.arange(T)[:, None], np.arange(T)
    for b, L in enumerate(lengths):
        sees = ((j <= i) & (j < L) & ((i - j < window) | (j < sinks))).any(1)
        want_nan = np.zeros((T, h), bool)
        want_nan[rows, 0] = sees[rows]
        nan = np.isnan(got[b]).reshape(T, h, d)
        assert (nan.all(-1) == want_nan).all() and (nan.any(-1) == want_nan).all()
        assert (got[b][~sees] == 0).all()
        keep = ~np.repeat(want_nan, d, -1)
        _check(np.where(keep, got[b], 0), np.where(keep, ref[b], 0), np.where(keep, A[b], 0), dtype, "beside NaN rows")
    if window >= T:
        # the batch without padding rows: attention() the same
        full = to_host(layer.attention(*t, causal=True, kv_lengths=_lens(lengths), G=tg))
        assert (np.isnan(full[0]) == np.isnan(got[0])).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 16), ("f32", 200)])
@pytest.mark.parametrize("step", ["window", "shared", "weights"])
@pytest.mark.parametrize("Tq", [1, 9])
def test_steps_non_finite_queries(dtype, d, step, Tq):
    """The same for the cache steps, which have no rows that see nothing."""
    h, h_kv, B, Tmax = 4, 2, 5, 700
    lengths = [700, Tq, 300, 129, 512]
    Q, K, V = _cache(900, dtype, B, Tq, Tmax, h, h_kv, d, d)
    K[..., ::d] = np.abs(K[..., ::d]) + 0.25
    if dtype == "bf16":
        K = wl.bf16_to_f32(wl.bf16_bits(np.ascontiguousarray(K, dtype=np.float32)))
    kw = dict(window=333, sinks=4) if step == "window" else dict(K_prefix=K[0], V_prefix=V[0]) if step == "shared" else {}
    ref, A, _ = lc.decode(Q, K, V, h, lengths, h_kv, **kw)
    bad = {(0, 0, 0): np.nan, (1, 0, 3): -np.inf, (2, Tq - 1, 1): -np.inf, (3, 0, 2): np.inf}
    for (b, t, i), x in bad.items():
        Q[b, t, i * d] = x
    layer = _layer(dtype, h, d, h_kv)
    t = [to_device(x, dtype) for x in (Q, K, V)]
    if step == "window":
        got = layer.decode_window(*t, _lens(lengths), 333, 4)
    elif step == "shared":
        got = layer.decode_shared(t[0], t[1][0], t[2][0], t[1], t[2], _lens(lengths))
    else:
        got = layer.decode_weights(*t, _lens(lengths), torch.zeros((B, h_kv, Tmax), device="cuda"))
    got = to_host(got)
    want = np.zeros((B, Tq, h), bool)
    for b, n, i in bad:
        want[b, n, i] = True
    nan = np.isnan(got).reshape(B, Tq, h, d)
    assert (nan.all(-1) == want).all() and (nan.any(-1) == want).all()
    keep = ~np.repeat(want, d, -1)
    _check(np.where(keep, got, 0), np.where(keep, ref, 0), np.where(keep, A, 0), dtype, "beside NaN rows")
    assert layer.status() == 0


@pytest.mark.parametrize("code", [_lib.MHA_ERR_TIMEOUT, _lib.MHA_ERR_BAD_LENGTH])
@pytest.mark.parametrize("d", [64, 128])
def test_status_resets_what_a_timed_out_step_left(code, d):
    """Arrivals, generation and unit counter as an aborted step leaves them (written here by the host; the status
    may be that of an earlier error): reading the status makes the workspace whole again."""
    h, h_kv = 8, 2
    cases = _step_cases("bf16", d, 850)
    layer = _layer("bf16", h, d, h_kv)
    for t, lens, _, w, *_ in cases:
        layer.decode_weights(*t, lens, w)
    assert layer.status() == 0
    layer._ws[:16].view(torch.int32).copy_(torch.tensor([code, 77, 5, 901], dtype=torch.int32))
    assert layer.status() == code
    for t, lens, lengths, w, ref, A, W in cases:
        w.zero_()
        _check(to_host(layer.decode_weights(*t, lens, w)), ref, A, "bf16", "after an error")
        for b, n in enumerate(lengths):
            _check_weights(to_host(w)[b, :, :n], W[b, :, :n], "after an error")
    assert layer.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_status_of_replays_is_kept(dtype):
    """An error of one replay is there to read after later ones, in a workspace attached under capture too."""
    h, h_kv, d, B, T = 4, 2, 64, 2, 300
    Q, K, V = _cache(950, dtype, B, 1, T, h, h_kv, d, d)
    t, lens = [to_device(x, dtype) for x in (Q, K, V)], _lens([T, 100])
    _layer(dtype, h, d, h_kv).decode_window(*t, lens, 50)
    torch.cuda.synchronize()
    for _ in range(40):  # from whichever of torch's streams comes next, the capture's own among them
        layer = _layer(dtype, h, d, h_kv)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            torch.full((1 << 22,), 1, dtype=torch.uint8, device="cuda")  # a temporary, where its pool may hand out memory
            out = layer.decode_window(*t, lens, 50)
    ref, A, _ = lc.decode(Q, K, V, h, [T, 100], h_kv, 50)
    for bad in (False, True, False, False):
        lens.copy_(_lens([T, T + 1 if bad else 100]))
        g.replay()
        got = to_host(out)
        assert np.isnan(got[1]).all() == bad
        _check(got[:1], ref[:1], A[:1], dtype, "replayed")
    assert layer.status() == _lib.MHA_ERR_BAD_LENGTH and layer.status() == 0
    g.replay()
    _check(to_host(out), ref, A, dtype, "replayed")
    assert layer.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("op", ["attention", "linear", "linear_segments", "linear_pair"])
def test_single_steps_hold_the_status_word(dtype, op):
    """The layer's single steps use an attached workspace's status word: a captured one stays theirs, and the
    allocator knows of the stream."""
    h, d, B, T = 4, 64, 2, 128
    layer = _layer(dtype, h, d, h)
    x = [to_device(_rand((B, T, h * d), s, dtype), dtype) for s in (51, 52, 53)]
    W, rows = to_device(_rand((h * d, h * d), 54, dtype), dtype), x[0].view(B * T, h * d)
    lens = _lens([T, T + 1])  # the second is invalid

    def call():
        if op == "attention":
            return layer.attention(*x, kv_lengths=lens)
        if op == "linear":
            return layer.linear(rows, W)
        if op == "linear_segments":
            return layer.linear_segments(rows, W, None, _lens_ok, T)
        return layer.linear_pair(rows, W, None, rows, W, None)
    _lens_ok = _lens([T, 50])
    call()                                                   # none attached: no status, no workspace
    assert layer._ws is None
    layer.ensure_workspace(0, 0, 0, need=256)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    assert side.cuda_stream in layer._ws_streams
    torch.cuda.synchronize()
    assert layer.status() == (_lib.MHA_ERR_BAD_LENGTH if op == "attention" else 0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    old = layer._ws
    layer.ensure_workspace(0, 0, 0, need=1 << 20)
    assert layer._ws is not old and any(w is old for w in layer._kept_ws)
    g.replay()
    torch.cuda.synchronize()
    assert int(old[:4].view(torch.int32).item()) == (_lib.MHA_ERR_BAD_LENGTH if op == "attention" else 0)
    assert layer.status() == 0
