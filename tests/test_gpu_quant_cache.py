"""The quantised key/value cache -- writing, reading back, the decode step -- against its 64-bit definition
(oracle/quant_cache.py).

Codes, steps and lowest values are those of the real numbers and are compared for equality.  Values read back are
s code + m rounded once to fp32 (equal), or to bf16 (half a step, 2^-8 of the value, and 2^-24 for the sum in fp32).

Tolerances of the decode step.  fp32: the normwise 1e-5 every fp32 parity test uses.  bf16 outputs, element by
element: the output is rounded once, by at most 2^-8 |o|.  A value is s code + m; the products w s of softmax weight
and step are rounded to fp16, each by at most 2^-11 of itself (11 significant bits), before they meet the codes:
|sum_j fl(w_j s_j) code_j - sum_j w_j s_j code_j| <= 2^-11 sum_j w_j s_j code_j = 2^-11 S, whatever the m are, as
those meet w in fp32.  (A bound with the codes' distance from their middle in S's place, which these tests first had,
holds only for a kernel that takes the middle off the codes before the product: with code = middle it would be 0.)
Everything else is fp32 and bounded by 1e-4 A, A = sum_j w_j |v_j| (scores of a few units, off by at most (d + 8)
2^-23 sum |q||k| / sqrt(d) each), and 1e-4 S for values that are small beside the two parts they are the sum of.
"""
import numpy as np
import pytest

from gpu_util import F32_NORMWISE, errors, to_device, to_host, torch_dtype

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import quant_cache as qc  # noqa: E402
from transformer_head_scaled_02_gb300 import Mha, _lib  # noqa: E402
from transformer_head_scaled_02_gb300 import workloads as wl  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build_library()
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)


def _layer(dtype, h, d, h_kv, d_v=None):
    return Mha(h * d, h, d, d if d_v is None else d_v, dtype=torch_dtype(dtype), h_kv=h_kv)


def _rand(shape, seed, dtype):
    """Channels of different size and mean."""
    x = wl.random_tensor(shape, seed, "f32")
    r = np.random.default_rng(seed + 1000)
    x = x * np.exp(0.5 * r.standard_normal(shape[-1])) + 0.5 * r.standard_normal(shape[-1])
    x = x.astype(np.float32)
    return wl.bf16_to_f32(wl.bf16_bits(x)) if dtype == "bf16" else x


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _poison(cache):
    """Every byte of the cache set: codes all ones, parameters NaN."""
    cache.data.fill_(0xFF)


def _held(cache, which):
    """(codes, params) of a cache's keys or values in 64 bits."""
    codes, params = (cache.K_codes, cache.K_params) if which == "K" else (cache.V_codes, cache.V_params)
    d = cache.heads[1] if which == "K" else cache.heads[2]
    return qc.unpack(codes.cpu().numpy(), cache.bits, d), params.double().cpu().numpy()


SHAPES = [
    # dtype, d, d_v, h, h_kv
    ("bf16", 64, 64, 4, 4), ("bf16", 64, 64, 8, 1), ("bf16", 128, 128, 4, 2), ("f32", 64, 64, 4, 2),
    ("f32", 128, 128, 4, 4), ("f32", 20, 37, 6, 2), ("f32", 80, 130, 2, 1), ("f32", 9, 256, 8, 2)]


def _expect(x, h_kv, bits):
    """Codes and params (B, h_kv, T, ...) of rows (B, T, h_kv d)."""
    return qc.quantise(qc.heads(x, h_kv), bits)


# ------------------------------------------------------------------ writing and reading back

@pytest.mark.parametrize("dtype,d,dv,h,h_kv", SHAPES)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,B", [(1, 3), (5, 1), (61, 4)])
def test_write_and_read(dtype, d, dv, h, h_kv, bits, T, B):
    """Ragged counts at ragged places: the tokens' codes are the definition's, every other byte stays."""
    rng = np.random.default_rng(T + bits)
    counts = [T] + [int(x) for x in rng.integers(0, T + 1, B - 1)]
    layer = _layer(dtype, h, d, h_kv, dv)
    cache = layer.quant_cache(B, 2 * T + 9, bits)
    _poison(cache)
    before = cache.data.clone()
    lengths = [int(rng.integers(n, cache.T_max + 1)) for n in counts]
    lengths[-1] = cache.T_max
    K, V = _rand((B, T, h_kv * d), 3 * T, dtype), _rand((B, T, h_kv * dv), 3 * T + 1, dtype)
    K[:, T // 2] = 0.75                                              # a constant row
    V[0, T - 1] = np.round(V[0, T - 1] * 4) / 4                      # many ties
    layer.quant_write(cache, to_device(K, dtype), to_device(V, dtype), _ints(lengths), _ints(counts))
    assert layer.status() == 0
    tokens = np.zeros((B, cache.T_max), bool)
    for which, x in (("K", K), ("V", V)):
        codes, params = _held(cache, which)
        want_c, want_p = _expect(x, h_kv, bits)
        for b in range(B):
            rows = slice(lengths[b] - counts[b], lengths[b])
            tokens[b, rows] = True
            assert (codes[b, :, rows] == want_c[b, :, :counts[b]]).all()
            assert (params[b, :, rows] == want_p[b, :, :counts[b]]).all()
    # nothing else was written, but for the padding of the written rows
    for now, old in zip((cache.K_codes, cache.K_params, cache.V_codes, cache.V_params),
                        (x for x in _views(cache, before))):
        mask = torch.from_numpy(tokens).cuda()[:, None, :].expand(now.shape[:3])
        assert (now.view(torch.uint8)[~mask] == old.view(torch.uint8)[~mask]).all()
    # and back, into column views of one buffer with guard bands
    w = h_kv * (d + dv)
    buf = torch.full((B, T, w + 24), 7.0, dtype=torch_dtype(dtype), device="cuda")
    Ko, Vo = layer.quant_read(cache, _ints(lengths), _ints(counts), K_out=buf[..., 8:8 + h_kv * d],
                              V_out=buf[..., 8 + h_kv * d:8 + w])
    got = to_host(buf)
    for which, x, c0 in (("K", K, 8), ("V", V, 8 + h_kv * d)):
        want = qc.values(*_expect(x, h_kv, bits))
        want = np.moveaxis(want, 1, 2).reshape(B, T, -1)
        for b in range(B):
            n = counts[b]
            g, v = got[b, :n, c0:c0 + x.shape[-1]], want[b, :n]
            if dtype == "f32":
                assert (g == v.astype(np.float32)).all()
            else:
                assert (np.abs(g - v) <= (2.0 ** -8 + 2.0 ** -24) * np.abs(v)).all()
            assert (got[b, n:, c0:c0 + x.shape[-1]] == 7).all()
    assert (got[..., :8] == 7).all() and (got[..., 8 + w:] == 7).all()


def _views(cache, data):
    off = 0
    for x in (cache.K_codes, cache.K_params, cache.V_codes, cache.V_params):
        off = x.data_ptr() - cache.data.data_ptr()
        n = x.numel() * x.element_size()
        yield data[off:off + n].view(x.dtype).view(x.shape)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
def test_codes_at_borders(dtype, bits):
    """Groups whose values lie on and next to the borders between codes, of every size, against fractions."""
    rng = np.random.default_rng(bits)
    n, rows = 2 ** bits - 1, []
    f32 = np.float32
    for i in range(160):
        low = f32(wl.bf16_to_f32(wl.bf16_bits(np.array([rng.standard_normal() * 10.0 ** rng.integers(-3, 4)], f32)))[0])
        step = f32(wl.bf16_to_f32(wl.bf16_bits(np.array([abs(rng.standard_normal()) * 10.0 ** rng.integers(-3, 3) + 1e-6], f32)))[0])
        k = rng.integers(0, n, 64)
        x = (low.astype(np.float64) + (k + 0.5) * step.astype(np.float64)).astype(f32)
        for j in range(0, 64, 3):
            x[j] = np.nextafter(x[j], f32(np.inf if j % 2 else -np.inf), dtype=f32)
        x[0], x[1] = low, f32(low + n * np.float64(step))
        rows.append(x)
    rows += [np.full(64, v, f32) for v in (0.0, -0.0, 1.5, 1e-40, -1e-40, 3.3895313892515355e38, -3.3895313892515355e38)]
    rows.append(np.linspace(-3.3895313892515355e38, 3.3895313892515355e38, 64).astype(f32))
    rows.append(np.r_[np.full(32, -1e38, f32), np.linspace(0, 3.38e38, 32).astype(f32)])
    rows.append(np.r_[f32(1.0), np.full(62, 1e-40, f32), f32(0)])
    rows.append((np.arange(64) * 1e-41).astype(f32))
    rows.append(np.r_[-np.logspace(-38, 0, 32), np.logspace(-30, 5, 32)].astype(f32))
    x = np.stack(rows)
    if dtype == "bf16":
        x = wl.bf16_to_f32(wl.bf16_bits(x))
        x = np.clip(x, -3.3895313892515355e38, 3.3895313892515355e38)
    layer = _layer(dtype, 1, 64, 1)
    cache = layer.quant_cache(1, len(x), bits)
    t = to_device(x[None], dtype)
    layer.quant_write(cache, t, t, _ints([len(x)]))
    for which in "KV":
        codes, params = _held(cache, which)
        for i in range(len(x)):
            c, s, m = qc.quantise_exact(x[i], bits)
            assert params[0, 0, i, 0, 0] == s and params[0, 0, i, 0, 1] == m, (i, x[i], params[0, 0, i], s, m)
            assert (codes[0, 0, i] == c).all(), (i, s, m, x[i][codes[0, 0, i] != c])
    back = to_host(layer.quant_read(cache, _ints([len(x)]), T_out=len(x))[0])[0]
    assert np.isfinite(back).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 70)])
@pytest.mark.parametrize("bits", [4, 8])
def test_values_that_are_not_finite(dtype, d, bits):
    """A group with NaN, infinity or (fp32) a value above bf16's range reads back as NaN, its neighbours do not;
    a step that sees it gives NaN, a step that does not is as without."""
    layer = _layer(dtype, 2, d, 1)
    T = 40
    K, V = _rand((1, T, d), 1, dtype), _rand((1, T, d), 2, dtype)
    Kn, Vn = K.copy(), V.copy()
    Kn[0, 30, 2], Vn[0, 33, d - 1] = np.nan, -np.inf
    if dtype == "f32":
        Kn[0, 31, d - 1] = 3.4e38
    Q = to_device(_rand((1, 1, 2 * d), 3, dtype), dtype)
    clean, dirty = layer.quant_cache(1, T, bits), layer.quant_cache(1, T, bits)
    layer.quant_write(clean, to_device(K, dtype), to_device(V, dtype), _ints([T]))
    layer.quant_write(dirty, to_device(Kn, dtype), to_device(Vn, dtype), _ints([T]))
    a, b = (to_host(x) for x in layer.quant_read(clean, _ints([T]), T_out=T))
    c, e = (to_host(x) for x in layer.quant_read(dirty, _ints([T]), T_out=T))
    assert np.isnan(c[0, 30, :64]).all() and np.isnan(e[0, 33, 64:]).all()
    keep = np.isfinite(c)
    assert (c[keep] == a[keep]).all() and (~keep).sum() == 64 + (d - 64 if dtype == "f32" else 0)
    keep = np.isfinite(e)
    assert (e[keep] == b[keep]).all() and (~keep).sum() == d - 64
    assert np.isnan(to_host(layer.decode_quant(Q, dirty, _ints([T])))).all()
    assert (to_host(layer.decode_quant(Q, dirty, _ints([30]))) == to_host(layer.decode_quant(Q, clean, _ints([30])))).all()
    assert np.isfinite(to_host(layer.decode_quant(Q, dirty, _ints([30])))).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 24)])
def test_invalid_lengths_and_counts(dtype, d):
    """Batches whose numbers do not fit are not touched and reported; the others are served."""
    layer = _layer(dtype, 2, d, 2)
    T, B = 8, 7
    cache = layer.quant_cache(B, 32)
    T_max = cache.T_max
    _poison(cache)
    before = cache.data.clone()
    lengths, counts = [T_max + 1, 4, -1, 8, 8, T_max, 0], [8, 5, 0, 9, -1, 8, 0]
    x = to_device(_rand((B, T, 2 * d), 1, dtype), dtype)
    layer.quant_write(cache, x, x, _ints(lengths), _ints(counts))
    assert layer.status() == _lib.MHA_ERR_BAD_LENGTH and layer.status() == 0
    changed = (cache.K_params.view(torch.int32) != next(v for i, v in enumerate(_views(cache, before)) if i == 1).view(torch.int32))
    assert changed.flatten(1).any(1).tolist() == [False] * 5 + [True, False]
    out = torch.full((B, T, 2 * d), 7.0, dtype=torch_dtype(dtype), device="cuda")
    layer.quant_read(cache, _ints(lengths), _ints(counts), K_out=out, V_out=out.clone())
    assert layer.status() == _lib.MHA_ERR_BAD_LENGTH
    assert ((out == 7).flatten(1).all(1).tolist()) == [True] * 5 + [False, True]


# ------------------------------------------------------------------ the decode step

def _filled(layer, seed, dtype, B, T, bits):
    """A cache of random tokens, written by the library, and its contents in 64 bits; past nothing yet."""
    h_kv, d, dv = layer.h_kv, layer.d_k, layer.d_v
    cache = layer.quant_cache(B, T, bits)
    _poison(cache)
    K, V = _rand((B, T, h_kv * d), seed, dtype), _rand((B, T, h_kv * dv), seed + 1, dtype)
    layer.quant_write(cache, to_device(K, dtype), to_device(V, dtype), _ints([T] * B))
    return cache, _held(cache, "K") + _held(cache, "V")


def _spoil(cache, lengths):
    """Tokens at or past the lengths hold anything: NaN parameters, codes all ones."""
    for b, L in enumerate(lengths):
        if 0 <= L < cache.T_max:
            for x in (cache.K_codes, cache.K_params, cache.V_codes, cache.V_params):
                x[b, :, L:].view(torch.uint8).fill_(0xFF)


def _check(got, ref, A, S, dtype, what=""):
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    if dtype == "f32":
        assert errors(got, ref)["normwise"] <= F32_NORMWISE, f"{what}: {errors(got, ref)}"
    else:
        over = np.abs(got - ref) - (2.0 ** -8 * np.abs(ref) + 2.0 ** -11 * S + 1e-4 * (A + S))
        assert over.max() <= 0, f"{what}: {over.max()} over the bound; {errors(got, ref)}"


def _step(layer, cache, held, Q, lengths, dtype, what=""):
    got = to_host(layer.decode_quant(to_device(Q, dtype), cache, _ints(lengths)))
    O, A, S = qc.decode(Q, *held, layer.h, lengths)
    _check(got, O, A, S, dtype, what)
    return got


@pytest.mark.parametrize("dtype,d,dv,h,h_kv", SHAPES)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Tq,T,lengths", [
    (1, 1, [1, 1]), (1, 40, [40, 1, 17]), (3, 70, [3, 70, 64, 33]), (1, 130, [130, 97, 128, 2]), (5, 900, [900, 5, 257, 513]),
    (2, 1300, [1300, 600])])
def test_decode(dtype, d, dv, h, h_kv, bits, Tq, T, lengths):
    layer = _layer(dtype, h, d, h_kv, dv)
    cache, held = _filled(layer, T + bits, dtype, len(lengths), T, bits)
    _spoil(cache, lengths)
    Q = wl.random_tensor((len(lengths), Tq, h * d), T + 7, dtype)
    _step(layer, cache, held, Q, lengths, dtype, "decode")
    assert layer.status() == 0


@pytest.mark.parametrize("dtype,d,h,h_kv,Tq", [("bf16", 128, 16, 1, 5), ("bf16", 64, 16, 1, 9), ("bf16", 64, 24, 2, 1),
                                               ("bf16", 128, 9, 1, 1), ("f32", 64, 16, 1, 5), ("f32", 128, 16, 1, 3),
                                               ("f32", 40, 33, 1, 1), ("bf16", 64, 2, 1, 150)])
@pytest.mark.parametrize("bits", [4, 8])
def test_decode_many_rows(dtype, d, h, h_kv, Tq, bits):
    """Query rows in several row blocks, the last one partly filled; new tokens spread over several tiles."""
    lengths = [400, Tq, 161]
    layer = _layer(dtype, h, d, h_kv)
    cache, held = _filled(layer, d + h, dtype, 3, 400, bits)
    _spoil(cache, lengths)
    _step(layer, cache, held, wl.random_tensor((3, Tq, h * d), 5, dtype), lengths, dtype, "many rows")


@pytest.mark.parametrize("d", [1, 31, 32, 33, 65, 80, 96, 97, 127])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("h,h_kv,Tq,lengths", [
    (2, 2, 1, [300, 1, 129]), (4, 1, 2, [700, 2, 128, 65]), (8, 1, 2, [513, 100]), (6, 3, 2, [9000]),
    (4, 2, 1, [3000, 20, 2999, 1, 1500, 700, 64, 2048])])
def test_decode_fp32_head_sizes(d, bits, h, h_kv, Tq, lengths):
    """Heads of any number of channels up to 128: rows of 32, 64, 96 and 128 of them, outputs that end inside a piece of
    four, beside a guard band."""
    layer = _layer("f32", h, d, h_kv)
    T = max(lengths)
    cache, held = _filled(layer, d + T, "f32", len(lengths), T, bits)
    _spoil(cache, lengths)
    Q = wl.random_tensor((len(lengths), Tq, h * d), 5, "f32")
    big = torch.full((len(lengths), Tq, h * d + 9), 7.0, device="cuda")
    layer.decode_quant(to_device(Q, "f32"), cache, _ints(lengths), out=big[..., 5:5 + h * d])
    got = to_host(big)
    assert (got[..., :5] == 7).all() and (got[..., 5 + h * d:] == 7).all()
    O, A, S = qc.decode(Q, *held, h, lengths)
    _check(got[..., 5:5 + h * d], O, A, S, "f32", "head sizes")
    assert layer.status() == 0


@pytest.mark.parametrize("d,h,h_kv,B,Tq,T", [(61, 64, 4, 8, 7, 5400), (64, 16, 1, 2, 1, 30000), (128, 8, 8, 2, 1, 20000),
                                             (128, 2, 1, 2, 2, 9000), (32, 64, 16, 2, 1, 16000)])
@pytest.mark.parametrize("bits", [4, 8])
def test_decode_fp32_long_means(d, h, h_kv, B, Tq, T, bits):
    """Sums over thousands of tokens in an fp32 layer: the codes' are far larger than what they leave in the output."""
    layer = _layer("f32", h, d, h_kv)
    cache, held = _filled(layer, 3, "f32", B, T, bits)
    _step(layer, cache, held, wl.random_tensor((B, Tq, h * d), 5, "f32"), [T] * B, "f32", "means")


@pytest.mark.parametrize("d,h,h_kv,Tq,lengths", [
    (128, 2, 1, 130, [400, 130, 257]), (64, 4, 1, 65, [65, 700, 129]), (128, 4, 2, 200, [1500]),
    (64, 8, 1, 100, [128, 100, 640, 127, 384]), (128, 1, 1, 256, [256, 300])])
@pytest.mark.parametrize("bits", [4, 8])
def test_decode_prompt_pieces(d, h, h_kv, Tq, lengths, bits):
    """Hundreds of query rows of a cached head: blocks of 128 rows, the last one partly filled, whole warps of it idle;
    groups of one tile, of several, and shared by CTAs; an invalid length between them."""
    layer = _layer("bf16", h, d, h_kv)
    T = max(lengths)
    cache, held = _filled(layer, d + h, "bf16", len(lengths) + 1, T, bits)
    lengths = lengths[:1] + [Tq - 1] + lengths[1:]
    _spoil(cache, lengths)
    Q = wl.random_tensor((len(lengths), Tq, h * d), 5, "bf16")
    first = layer.decode_quant(to_device(Q, "bf16"), cache, _ints(lengths))
    assert layer.status() == _lib.MHA_ERR_BAD_LENGTH
    got = to_host(first)
    O, A, S = qc.decode(Q, *held, h, lengths)
    assert np.isnan(got[1]).all()
    keep = np.arange(len(lengths)) != 1
    _check(got[keep], O[keep], A[keep], S[keep], "bf16", "prompt pieces")
    again = layer.decode_quant(to_device(Q, "bf16"), cache, _ints(lengths))
    assert torch.equal(again[torch.from_numpy(keep).cuda()], first[torch.from_numpy(keep).cuda()])


def test_decode_prompt_pieces_large_scores_and_scales():
    """The same with scores that rise along the keys and steps that differ by 2^40: references and scales move."""
    d, Tq, T = 128, 256, 700
    layer = _layer("bf16", 1, d, 1)
    Q, K, V = (wl.random_tensor((1, n, d), 70 + i, "bf16") for i, n in enumerate((Tq, T, T)))
    rnd = lambda x: wl.bf16_to_f32(wl.bf16_bits(x.astype(np.float32)))  # noqa: E731
    ramp = np.linspace(0.1, 6.0, T)[None, :, None]
    powers = 2.0 ** np.random.default_rng(3).integers(-20, 20, T)[None, :, None]
    for q, k, v in ((Q * 4, K * ramp, V), (Q, K, V * powers), (Q * 2.0 ** 60, K * 2.0 ** -60, V * 2.0 ** 100)):
        q, k, v = rnd(q), rnd(k), rnd(v)
        cache = layer.quant_cache(1, T, 4)
        layer.quant_write(cache, to_device(k, "bf16"), to_device(v, "bf16"), _ints([T]))
        held = _held(cache, "K") + _held(cache, "V")
        got = to_host(layer.decode_quant(to_device(q, "bf16"), cache, _ints([T])))
        O, A, S = qc.decode(q, *held, 1, [T])
        assert np.isfinite(got).all()
        p = np.repeat(held[1], 64, -2)[0, :, :T]
        s = np.max(np.abs(q[0]) @ np.moveaxis(np.abs(p[..., 1]) + p[..., 0] * 15, -1, -2)[0]) / np.sqrt(d)
        w = 2 * s * (d + 8) * 2.0 ** -23
        assert (np.abs(got - O) <= 2.0 ** -8 * np.abs(O) + 2.0 ** -11 * S + (w + 1e-5) * (A + S)).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 48)])
@pytest.mark.parametrize("bits", [4, 8])
def test_decode_long(dtype, d, bits):
    """A few sequences of very different length: parts of every size, and joins of many."""
    lengths = [20000, 300, 1, 9999]
    layer = _layer(dtype, 4, d, 2)
    cache, held = _filled(layer, 11, dtype, 4, 20000, bits)
    _spoil(cache, lengths)
    _step(layer, cache, held, wl.random_tensor((4, 1, 4 * d), 5, dtype), lengths, dtype, "long")


@pytest.mark.parametrize("dtype,d,h,h_kv", [("bf16", 64, 8, 4), ("bf16", 128, 4, 4), ("bf16", 64, 64, 4), ("f32", 64, 4, 4), ("f32", 48, 4, 4)])
@pytest.mark.parametrize("B,T", [(13, 700), (40, 300), (70, 257)])
def test_decode_many_sequences(dtype, d, h, h_kv, B, T):
    """More groups than CTAs, and nearly as many, with lengths of every size, none at all among them: groups shared by
    two CTAs, CTAs with many groups, batches beyond a warp's lanes."""
    rng = np.random.default_rng(B + T)
    lengths = [int(x) for x in rng.integers(1, T + 1, B)]
    lengths[0], lengths[5], lengths[-1], lengths[7] = T, 1, T, 0
    layer = _layer(dtype, h, d, h_kv)
    cache, held = _filled(layer, 11, dtype, B, T, 4)
    _spoil(cache, lengths)
    Q = wl.random_tensor((B, 1, h * d), 5, dtype)
    got = to_host(layer.decode_quant(to_device(Q, dtype), cache, _ints(lengths)))
    O, A, S = qc.decode(Q, *held, h, lengths)
    assert np.isnan(got[7]).all() and layer.status() == _lib.MHA_ERR_BAD_LENGTH
    keep = np.arange(B) != 7
    _check(got[keep], O[keep], A[keep], S[keep], dtype, "many sequences")


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 16)])
@pytest.mark.parametrize("bits", [4, 8])
def test_decode_large_scores_and_scales(dtype, d, bits):
    """Scores of hundreds that rise or fall along the keys, steps that differ by 2^40 between tokens, queries of
    2^-60 and 2^60, and values of 2^-100 and 2^100: the references have to follow."""
    T, h = 700, 2
    layer = _layer(dtype, h, d, 1)
    Q, K, V = (wl.random_tensor((1, n, w), 60 + i, dtype) for i, (n, w) in enumerate(((1, h * d), (T, d), (T, d))))
    ramp = np.linspace(0.1, 12.0, T)[None, :, None]
    powers = 2.0 ** np.random.default_rng(3).integers(-20, 20, T)[None, :, None]
    rnd = (lambda x: wl.bf16_to_f32(wl.bf16_bits(x.astype(np.float32)))) if dtype == "bf16" else (lambda x: x.astype(np.float32))
    # (scores: how far fp32 sums of products let them be off, twice that for the weights, relative)
    for q, k, v in ((Q * 4, K * ramp, V), (Q * 4, K * ramp[:, ::-1], V), (Q, K, V * powers), (Q * 2.0 ** -60, K * 2.0 ** 60, V),
                    (Q * 2.0 ** 60, K * 2.0 ** -60, V * 2.0 ** 100), (Q, K, V * 2.0 ** -100), (Q, K, V * powers * 2.0 ** 80)):
        q, k, v = rnd(q), rnd(k), rnd(v)
        cache = layer.quant_cache(1, T, bits)
        layer.quant_write(cache, to_device(k, dtype), to_device(v, dtype), _ints([T]))
        held = _held(cache, "K") + _held(cache, "V")
        got = to_host(layer.decode_quant(to_device(q, dtype), cache, _ints([T])))
        O, A, S = qc.decode(q, *held, h, [T])
        assert np.isfinite(got).all()
        # (rows past T are unset memory) a score sums d products of q and the parts s code and m of a key, which may cancel
        Kv, p = qc.values(held[0], held[1]), np.repeat(held[1], 64, -2)[..., :d, :]
        parts = np.abs(p[..., 1]) + p[..., 0] * (2 ** bits - 1)
        s = np.max(np.abs(qc.heads(q, h)[0]) @ np.moveaxis(parts[0, :, :T], -1, -2)) / np.sqrt(d)
        w = 2 * s * (d + 8) * 2.0 ** -23
        rounding = 2.0 ** -8 * np.abs(O) + 2.0 ** -11 * S if dtype == "bf16" else 0.0
        assert (np.abs(got - O) <= rounding + (w + 1e-5) * (A + S)).all(), (np.abs(got - O) / (A + S)).max()
        assert Kv.shape[-1] == d


def _bound(q, held, h, d, bits, O, A, S, dtype):
    """_check's bound for scores of any size: a score sums d products of q and the parts s code and m of a key, which may
    cancel, in fp32; its weight is off by twice as much, relatively."""
    parts = np.abs(held[1][..., 1]) + held[1][..., 0] * (2 ** bits - 1)
    parts = np.repeat(parts, 64, -1)[..., :d]
    per = h // parts.shape[1]
    s = np.max(np.abs(qc.heads(q, h)) @ np.moveaxis(np.repeat(parts, per, 1), -1, -2)) / np.sqrt(d)
    w = 2 * s * (d + 8) * 2.0 ** -23
    return (2.0 ** -8 * np.abs(O) + 2.0 ** -11 * S if dtype == "bf16" else 0.0) + (w + 1e-5) * (A + S)


@pytest.mark.parametrize("dtype,d,Tq", [("bf16", 64, 3), ("bf16", 128, 2), ("bf16", 64, 1), ("f32", 64, 3), ("f32", 128, 2),
                                        ("f32", 24, 3), ("bf16", 64, 150), ("bf16", 128, 130)])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("where", ["first", "last", "spread"])
def test_decode_values_that_matter_to_some_rows(dtype, d, Tq, bits, where):
    """Values 2^70 times as large as the others at tokens that only the first of two heads gives any weight, and at new
    tokens that the earlier ones do not see: the other rows' outputs are as accurate as without them."""
    h, T = 2, 700
    layer = _layer(dtype, h, d, 1)
    rnd = (lambda x: wl.bf16_to_f32(wl.bf16_bits(x.astype(np.float32)))) if dtype == "bf16" else (lambda x: x.astype(np.float32))
    Q, K, V = (wl.random_tensor((1, n, w), 80 + i, dtype) for i, (n, w) in enumerate(((Tq, h * d), (T, d), (T, d))))
    way = np.sign(wl.random_tensor((d,), 9, "f32"))
    Q[..., :d] = np.abs(Q[..., :d]) * way  # of the first head towards those keys, of the second one away from them
    Q[..., d:] = -np.abs(Q[..., d:]) * way
    at = {"first": slice(0, 3), "last": slice(T - Tq - 3, T - Tq), "spread": slice(5, T - Tq, 97)}[where]
    K[:, at] = 60 * way
    V[:, at] *= 2.0 ** 70
    V[:, T - Tq + 1:] *= 2.0 ** 60
    Q, K, V = rnd(Q), rnd(K), rnd(V)
    cache = layer.quant_cache(1, T, bits)
    layer.quant_write(cache, to_device(K, dtype), to_device(V, dtype), _ints([T]))
    held = tuple(x[:, :, :T] for x in _held(cache, "K") + _held(cache, "V"))
    got = to_host(layer.decode_quant(to_device(Q, dtype), cache, _ints([T])))
    O, A, S = qc.decode(Q, *held, h, [T])
    assert np.abs(O[0, 0, d:]).max() < 2 ** 10  # (the oracle: it does not see them either)
    assert np.isfinite(got).all()
    assert (np.abs(got - O) <= _bound(Q, held, h, d, bits, O, A, S, dtype)).all(), (np.abs(got - O) / (A + S)).max((0, 1))


@pytest.mark.parametrize("dtype,d,Tq", [("bf16", 64, 1), ("bf16", 128, 3), ("bf16", 64, 300), ("f32", 64, 2), ("f32", 128, 1), ("f32", 20, 1)])
def test_decode_huge_queries(dtype, d, Tq):
    """Queries of 2^110: a row's largest score, 1e-3 or more above the next one, has all the weight."""
    T = 400
    layer = _layer(dtype, 1, d, 1)
    Q = wl.random_tensor((1, Tq, d), 21, dtype) * np.float32(2.0 ** 110)
    K, V = (wl.random_tensor((1, T, d), 22 + i, dtype) for i in range(2))
    # the key that a row is closest to by far: its own direction, doubled
    K[0, :Tq] = 2 * Q[0] * np.float32(2.0 ** -110)
    cache = layer.quant_cache(1, T, 8)
    layer.quant_write(cache, to_device(K, dtype), to_device(V, dtype), _ints([T]))
    held = tuple(x[:, :, :T] for x in _held(cache, "K") + _held(cache, "V"))
    x = np.sort(qc.heads(Q, 1)[0, 0].astype(np.float64) @ qc.values(*held[:2])[0, 0].T, -1)
    assert (x[:, -1] - x[:, -2] > 1e-3 * np.abs(x).max(-1)).all()
    got = to_host(layer.decode_quant(to_device(Q, dtype), cache, _ints([T])))
    O, A, S = qc.decode(Q, *held, 1, [T])
    _check(got, O, A, S, dtype, "huge queries")


def test_decode_invalid_lengths():
    for dtype, d in (("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 24)):
        layer = _layer(dtype, 4, d, 2)
        lengths = [200, 1, 0, 201, 90, -5]
        cache, held = _filled(layer, 2, dtype, 6, 192, 4)
        lengths[3] = cache.T_max + 1
        lengths[0] = cache.T_max
        Q = wl.random_tensor((6, 2, 4 * d), 5, dtype)
        big = torch.full((6, 2, 4 * d + 16), 7.0, dtype=torch_dtype(dtype), device="cuda")
        layer.decode_quant(to_device(Q, dtype), cache, _ints(lengths), out=big[..., 8:8 + 4 * d])
        assert layer.status() == _lib.MHA_ERR_BAD_LENGTH and layer.status() == 0
        got = to_host(big)
        assert (got[..., :8] == 7).all() and (got[..., 8 + 4 * d:] == 7).all()
        got = got[..., 8:8 + 4 * d]
        O, A, S = qc.decode(Q, *held, 4, lengths)
        for b in range(6):
            if 2 <= lengths[b] <= cache.T_max:
                _check(got[b], O[b], A[b], S[b], dtype)
            else:
                assert np.isnan(got[b]).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 128)])
def test_decode_views_and_results_that_repeat(dtype, d):
    """Query rows inside wider ones; the same call gives the same bits, alone or beside other batches."""
    h, h_kv, B, T = 8, 2, 3, 3000
    layer = _layer(dtype, h, d, h_kv)
    cache, held = _filled(layer, 4, dtype, B, T, 4)
    x = wl.random_tensor((B, 2, h * d + 32), 6, dtype)
    t = to_device(x, dtype)[..., 16:16 + h * d]
    lengths = [3000, 77, 1501]
    first = layer.decode_quant(t, cache, _ints(lengths))
    O, A, S = qc.decode(x[..., 16:16 + h * d], *held, h, lengths)
    _check(to_host(first), O, A, S, dtype)
    for _ in range(5):
        assert torch.equal(layer.decode_quant(t, cache, _ints(lengths)), first)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_offsets_past_32_bits(dtype, d):
    """A cache of more than 4 GB of codes: the last sequence's tokens are written, read and attended over in place."""
    layer = _layer(dtype, 16, d, 16)
    B, T_max = 512 * 128 // d, 9216
    cache = layer.quant_cache(B, T_max, 4)
    assert cache.K_codes.numel() > 2 ** 32
    n = 600
    K, V = _rand((1, n, 16 * d), 1, dtype), _rand((1, n, 16 * d), 2, dtype)
    big = torch.zeros((B, n, 16 * d), dtype=torch_dtype(dtype), device="cuda")
    vig = torch.zeros_like(big)
    big[-1], vig[-1] = to_device(K[0], dtype), to_device(V[0], dtype)
    lengths = [T_max] * B
    layer.quant_write(cache, big, vig, _ints(lengths))
    Ko, Vo = layer.quant_read(cache, _ints(lengths), K_out=big, V_out=vig)
    small = layer.quant_cache(1, n, 4)
    layer.quant_write(small, to_device(K, dtype), to_device(V, dtype), _ints([n]))
    Ks, Vs = layer.quant_read(small, _ints([n]), T_out=n)
    assert torch.equal(Ko[-1], Ks[0]) and torch.equal(Vo[-1], Vs[0]) and not Ko[-2].any()
    # the tokens before them: keys far from the queries, so that only the last ones count
    del big, vig, Ko, Vo
    at = T_max - n
    cache.K_params[-1, :, :at].zero_()
    cache.K_codes[-1, :, :at].zero_()
    cache.V_params[-1, :, :at].zero_()
    cache.V_codes[-1, :, :at].zero_()
    held = tuple(x.copy() for x in _held(small, "K") + _held(small, "V"))
    Q = wl.random_tensor((1, 1, 16 * d), 9, dtype)
    q = torch.zeros((B, 1, 16 * d), dtype=torch_dtype(dtype), device="cuda")
    q[-1] = to_device(Q, dtype)[0]
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    lens[-1] = T_max
    cache.K_params[:-1, :, 0].zero_()
    cache.V_params[:-1, :, 0].zero_()
    out = to_host(layer.decode_quant(q, cache, lens)[-1:])
    pad = [np.concatenate((np.zeros(x.shape[:2] + (at,) + x.shape[3:]), x[:, :, :n]), 2) for x in held]
    O, A, S = qc.decode(Q, *pad, 16, [T_max])
    _check(out, O, A, S, dtype, "past 32 bits")


# ------------------------------------------------------------------ together, as they are used

@pytest.mark.parametrize("dtype,d,h,h_kv", [("bf16", 64, 8, 2), ("bf16", 128, 4, 4), ("f32", 64, 4, 1), ("f32", 30, 4, 2)])
@pytest.mark.parametrize("bits", [4, 8])
def test_generation(dtype, d, h, h_kv, bits):
    """Prompts of several lengths are projected, attended and written; then tokens are generated one by one and
    three at a time, each written before its step; at the end the whole cache is read back and decoded over."""
    D, B, T = h * d, 3, 150
    layer = _layer(dtype, h, d, h_kv)
    width = layer.proj_width
    W = to_device((wl.random_tensor((D, width), 1, "f32") * 0.1).astype(np.float32), dtype)
    cut = (h * d, (h + h_kv) * d)
    cache = layer.quant_cache(B, 400, bits)
    _poison(cache)
    lengths = np.array([150, 1, 67], np.int32)
    x = to_device(_rand((B, T, D), 2, dtype), dtype)
    lens = _ints(lengths.tolist())
    p = layer.linear(x.view(-1, D), W).view(B, T, width)
    layer.quant_write(cache, p[..., cut[0]:cut[1]], p[..., cut[1]:], lens, lens)
    Ks, Vs = ([_expect(to_host(p[..., a:b]), h_kv, bits) for a, b in ((cut[0], cut[1]), (cut[1], width))])
    want = [[[y[b, :, :lengths[b]] for y in side] for b in range(B)] for side in (Ks, Vs)]
    for step, n in enumerate((1, 1, 3, 1)):
        x = to_device(_rand((B, n, D), 10 + step, dtype), dtype)
        p = layer.linear(x.view(-1, D), W).view(B, n, width)
        lens += n
        lengths += n
        layer.quant_write(cache, p[..., cut[0]:cut[1]], p[..., cut[1]:], lens)
        got = to_host(layer.decode_quant(p[..., :cut[0]], cache, lens))
        for side, (a, e) in zip(want, ((cut[0], cut[1]), (cut[1], width))):
            new = _expect(to_host(p[..., a:e]), h_kv, bits)
            for b in range(B):
                side[b] = [np.concatenate((old, y[b]), 1) for old, y in zip(side[b], new)]
        for b in range(B):
            held = [y[None] for y in want[0][b] + want[1][b]]
            O, A, S = qc.decode(to_host(p[b:b + 1, :, :cut[0]]), *held, h, [lengths[b]])
            _check(got[b:b + 1], O, A, S, dtype, f"step {step}")
    assert layer.status() == 0
    Ko, Vo = layer.quant_read(cache, lens, lens, K_out=torch.zeros((B, 400, h_kv * d), dtype=torch_dtype(dtype), device="cuda"),
                              V_out=torch.zeros((B, 400, h_kv * d), dtype=torch_dtype(dtype), device="cuda"))
    a, b = to_host(layer.decode(p[..., :cut[0]], Ko, Vo, lens)), got
    e = errors(a, b)
    # the values read back are rounded once more, and bf16 layers' plain decode rounds its weights
    assert e["rel_fro"] <= (2e-2 if dtype == "bf16" else 1e-5), e


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 128), ("f32", 20)])
def test_captured_steps_share_a_workspace(dtype, d):
    """Two captured graphs (a write and a step each) and eager calls in between, on another stream than the
    default: every replay is right, with lengths and inputs changed in between."""
    h, h_kv, B, T = 4, 2, 2, 900
    layer = _layer(dtype, h, d, h_kv)
    cache, _ = _filled(layer, 3, dtype, B, T, 4)
    tdt = torch_dtype(dtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for n in (1, 3):
            s = {"q": torch.zeros((B, n, h * d), dtype=tdt, device="cuda"), "k": torch.zeros((B, n, h_kv * d), dtype=tdt, device="cuda"),
                 "v": torch.zeros((B, n, h_kv * d), dtype=tdt, device="cuda"), "len": _ints([n] * B)}
            s["out"] = torch.zeros_like(s["q"])
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                layer.quant_write(cache, s["k"], s["v"], s["len"])
                layer.decode_quant(s["q"], cache, s["len"], out=s["out"])
            graphs.append((g, s, n))
        for round_, lengths in enumerate(([900, 20], [5, 899], [600, 601])):
            for g, s, n in graphs:
                for name in "qkv":
                    s[name].copy_(to_device(_rand(tuple(s[name].shape), 50 + 7 * round_ + n, dtype), dtype))
                s["len"].copy_(_ints(lengths))
                g.replay()
                got = to_host(s["out"])
                held = _held(cache, "K") + _held(cache, "V")
                O, A, S = qc.decode(to_host(s["q"]), *held, h, lengths)
                _check(got, O, A, S, dtype, f"replay {round_}")
                eager = layer.decode_quant(s["q"], cache, s["len"])
                assert torch.equal(eager, s["out"])
    torch.cuda.current_stream().wait_stream(side)
    assert layer.status() == 0


def test_empty_calls():
    layer = _layer("bf16", 2, 64, 1)
    cache = layer.quant_cache(0, 64)
    z = torch.zeros((0, 3, 64), dtype=torch.bfloat16, device="cuda")
    lens = torch.zeros(0, dtype=torch.int32, device="cuda")
    layer.quant_write(cache, z, z, lens)
    assert layer.quant_read(cache, lens, T_out=2)[0].shape == (0, 2, 64)
    assert layer.decode_quant(torch.zeros((0, 1, 128), dtype=torch.bfloat16, device="cuda"), cache, lens).shape == (0, 1, 128)
    cache = layer.quant_cache(2, 64)
    z = torch.zeros((2, 0, 64), dtype=torch.bfloat16, device="cuda")
    layer.quant_write(cache, z, z, _ints([0, 0]))
    assert layer.decode_quant(torch.zeros((2, 0, 128), dtype=torch.bfloat16, device="cuda"), cache, _ints([1, 1])).shape == (2, 0, 128)
