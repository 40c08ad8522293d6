"""The decode step over a quantised cache at the ends of its number range, against the 64-bit definition
(oracle/quant_cache.py).

Weighted sums are held before the division by the weights' sum, in fp32: they are finite as long as
2^8 T max |v| is below 2^128 (no weight is above 2^8), or for scores that are all alike, whose weights are 1,
T max |v|.  Tolerances are those of test_gpu_quant_cache.py.
"""
import numpy as np
import pytest

import test_gpu_quant_cache as base
from gpu_util import to_device, to_host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import quant_cache as qc  # noqa: E402
from transformer_head_scaled_02_gb300 import workloads as wl  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build_library()
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)


def _round(x, dtype):
    x = np.asarray(x, np.float32)
    return wl.bf16_to_f32(wl.bf16_bits(x)) if dtype == "bf16" else x


def _written(layer, K, V, dtype, bits):
    """A cache that holds the rows K and V (B, T, ..) and its contents in 64 bits."""
    B, T = K.shape[:2]
    cache = layer.quant_cache(B, T, bits)
    layer.quant_write(cache, to_device(K, dtype), to_device(V, dtype), base._ints([T] * B))
    return cache, tuple(x[:, :, :T] for x in base._held(cache, "K") + base._held(cache, "V"))


# query heads over one cached head, new tokens: 1, 2, 4, 8, 16 rows and hundreds
ROWS = [("bf16", 64, 1, 1), ("bf16", 64, 8, 1), ("bf16", 64, 16, 1), ("bf16", 128, 1, 1), ("bf16", 128, 4, 1), ("bf16", 128, 16, 1),
        ("bf16", 64, 1, 256), ("bf16", 128, 2, 140), ("f32", 64, 1, 1), ("f32", 64, 16, 1), ("f32", 128, 1, 1), ("f32", 40, 3, 1)]


@pytest.mark.parametrize("dtype,d,h,Tq", ROWS)
@pytest.mark.parametrize("bits", [4, 8])
def test_decode_values_near_the_top(dtype, d, h, Tq, bits):
    """Values of 2^108 under ordinary scores, and of 2^116 under scores that are nearly alike: 300 of them, times 5 and
    the weights, stay below 2^128."""
    T = 300
    layer = base._layer(dtype, h, d, 1)
    Q, K, V = (wl.random_tensor((1, n, w), 30 + i, dtype) for i, (n, w) in enumerate(((Tq, h * d), (T, d), (T, d))))
    assert np.abs(V).max() < 5
    for q, v in ((Q, V * np.float32(2.0 ** 108)), (Q * np.float32(2.0 ** -12), V * np.float32(2.0 ** 116))):
        cache, held = _written(layer, K, v, dtype, bits)
        got = to_host(layer.decode_quant(to_device(q, dtype), cache, base._ints([T])))
        O, A, S = qc.decode(q, *held, h, [T])
        base._check(got, O, A, S, dtype, "values near the top")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_references_that_move_slowly(dtype):
    """Two heads of one cached head: the first one's scores rise by 9 powers of two of a weight with each quantum, so that
    its reference always moves, and the second one's by 0.9, so that its first tokens, of values 2^30 times the others',
    fade slowly.  The last tokens' values count in full."""
    d, h, B, T, bits = 128, 2, 300, 8192, 8          # (a CTA has a sequence to itself, or nearly)
    layer = base._layer(dtype, h, d, 1)
    V = np.exp(1.5 * wl.random_tensor((1, T, d), 5, dtype))  # (most codes low)
    V[0, :128] *= 2.0 ** 30
    V = _round(V, dtype)
    one, _ = _written(layer, np.zeros((1, T, d), np.float32), V, dtype, bits)
    # keys: 9 j in channel 0, j in channel 64, j the quantum
    one.K_codes.zero_()
    one.K_codes[..., 0], one.K_codes[..., 64] = 9, 1
    one.K_params.zero_()
    one.K_params[..., 0] = (torch.arange(T, device="cuda") // 128)[:, None]
    held = base._held(one, "K") + base._held(one, "V")
    Q = np.zeros((1, 1, h * d), np.float32)
    Q[..., 0] = np.sqrt(d) / np.log2(np.e)
    Q[..., d + 64] = 0.9 * Q[..., 0]
    Q = _round(Q, dtype)
    cache = layer.quant_cache(B, T, bits)
    for to, x in ((cache.K_codes, one.K_codes), (cache.K_params, one.K_params), (cache.V_codes, one.V_codes),
                  (cache.V_params, one.V_params)):
        to.copy_(x.expand_as(to))
    got = to_host(layer.decode_quant(to_device(np.repeat(Q, B, 0), dtype), cache, base._ints([T] * B)))
    O, A, S = qc.decode(Q, *held, h, [T])
    bound = base._bound(Q, held, h, d, bits, O, A, S, dtype)
    assert np.isfinite(got).all()
    assert (np.abs(got - O) <= bound).all(), (np.abs(got - O) / (A + S)).max((0, 1))


@pytest.mark.parametrize("dtype,d,h,Tq", [("bf16", 64, 1, 1), ("bf16", 128, 8, 1), ("bf16", 64, 16, 1), ("bf16", 128, 2, 128),
                                          ("f32", 64, 1, 1), ("f32", 70, 1, 1)])
def test_decode_scores_a_step_of_fp32_apart(dtype, d, h, Tq):
    """Scores so large that fp32 holds them in steps of 4 to 16 powers of two of a weight, each quantum's a step above the
    last one's, over values that grow: outputs are means of the values, whatever the weights' rounding."""
    B, T, bits = 8, 4096, 8
    layer = base._layer(dtype, h, d, 1)
    j = np.arange(T) // 128
    V = _round(wl.random_tensor((1, T, d), 5, dtype) * 2.0 ** (4 * (j % 4)[None, :, None]), dtype)
    K = np.zeros((1, T, d), np.float32)
    K[0, :, 0], K[0, :, 1] = 255, j                            # codes of a step of 1
    cache, held = _written(layer, np.repeat(K, B, 0), np.repeat(V, B, 0), dtype, bits)
    assert (held[1][..., 0, 0] == 1).all()
    for power in np.arange(25.0, 29.01, 0.25):                 # of the log2 of a weight
        Q = np.zeros((1, Tq, h * d), np.float32)
        Q[..., 0::d] = 2.0 ** power * np.sqrt(d) / np.log2(np.e) / 255
        Q[..., 1::d] = Q[..., 0::d] * 255 * 2.0 ** -23
        got = to_host(layer.decode_quant(to_device(np.repeat(_round(Q, dtype), B, 0), dtype), cache, base._ints([T] * B)))
        assert np.isfinite(got).all(), power
        assert np.abs(got).max() <= np.abs(qc.values(*held[2:])).max() * (1 + 2.0 ** -7), power


@pytest.mark.parametrize("dtype,d,h,Tq", ROWS)
@pytest.mark.parametrize("bits", [4, 8])
def test_decode_small_queries_and_values(dtype, d, h, Tq, bits):
    """Queries of 2^-95 and 2^-113 under keys as large as that makes ordinary scores, and values of 2^-112: no bits are lost."""
    T = 300
    layer = base._layer(dtype, h, d, 1)
    Q, K, V = (wl.random_tensor((1, n, w), 30 + i, dtype) for i, (n, w) in enumerate(((Tq, h * d), (T, d), (T, d))))
    for qk, v in ((-95, 0), (-113, 0), (0, -112)):
        q, k, v = (x * np.float32(2.0 ** p) for x, p in ((Q, qk), (K, -qk), (V, v)))
        cache, held = _written(layer, k, v, dtype, bits)
        got = to_host(layer.decode_quant(to_device(q, dtype), cache, base._ints([T])))
        O, A, S = qc.decode(q, *held, h, [T])
        base._check(got, O, A, S, dtype, f"2^{qk}")


def test_write_borders_of_the_widest_ranges():
    """A range beyond fp32's largest number, and values of the smallest one on either side of a border between two codes."""
    s = 1.25 * 2.0 ** 124
    tiny = 2.0 ** -149
    rows = []
    for k in (6, 7):
        x = np.zeros(64, np.float32)
        x[:6] = -(k + 0.5) * s, (14.5 - k) * s, -tiny, tiny, 3 * tiny, -3 * tiny
        rows.append(x)
    x = np.stack(rows)
    layer = base._layer("f32", 1, 64, 1)
    cache = layer.quant_cache(1, len(x), 4)
    t = to_device(x[None], "f32")
    layer.quant_write(cache, t, t, base._ints([len(x)]))
    codes, params = base._held(cache, "K")
    for i in range(len(x)):
        c, step, low = qc.quantise_exact(x[i], 4)
        assert params[0, 0, i, 0, 0] == step and params[0, 0, i, 0, 1] == low
        assert (codes[0, 0, i] == c).all(), (i, codes[0, 0, i][:8], c[:8])


@pytest.mark.parametrize("dtype,d,Tq", [("bf16", 64, 1), ("bf16", 128, 3), ("bf16", 64, 256), ("f32", 64, 1), ("f32", 128, 2)])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("alike", [True, False])
def test_decode_one_token_far_above_many(dtype, d, Tq, bits, alike):
    """One token of nearly all the weight before thousands of equal small ones, down to 2^-24 of it each, whose values are
    alike (so that their products with the steps are all rounded the same way) or not.  A product is off by 2^-11 (fp32:
    2^-22) of itself and by 2^-23 of the row's largest besides; it meets a code (fp32: less half its range)."""
    B, T = (300, 4096) if Tq < 100 else (3, 4096)     # (a CTA has a sequence to itself, or nearly; rows: some tiles each)
    layer = base._layer(dtype, 1, d, 1)
    V = wl.random_tensor((1, T, d), 5, dtype)
    if alike:
        V[0, 1:] = V[0, 1]
    one, _ = _written(layer, np.zeros((1, T, d), np.float32), V, dtype, bits)
    one.K_codes.zero_()
    one.K_params.zero_()
    one.K_codes[0, 0, 0, 0] = 1                       # (the first token's key: 1 in channel 0; the others': 0)
    one.K_params[0, 0, 0, :, 0] = 1
    held = base._held(one, "K") + base._held(one, "V")
    cache = layer.quant_cache(B, T, bits)
    for to, x in ((cache.K_codes, one.K_codes), (cache.K_params, one.K_params), (cache.V_codes, one.V_codes),
                  (cache.V_params, one.V_params)):
        to.copy_(x.expand_as(to))
    step = np.repeat(held[3][0, 0, :, :, 0], 64, -1)[:, :d]
    code = np.abs(held[2][0, 0] - (0 if dtype == "bf16" else 2 ** (bits - 1)))
    for power in (8, 13, 16, 19, 21, 24):
        Q = np.zeros((1, Tq, d), np.float32)
        Q[..., 0] = power * np.sqrt(d) / np.log2(np.e)
        Q = _round(Q, dtype)
        got = to_host(layer.decode_quant(to_device(np.repeat(Q, B, 0), dtype), cache, base._ints([T] * B)))
        O, A, S = qc.decode(Q, *held, 1, [T])
        w = np.exp(Q[0, 0, 0] / np.sqrt(d) * (np.arange(T) == 0))
        w /= w[:T - Tq + 1].sum()                     # (the first new token sees fewest)
        part, most = (w[:, None] * step * code).sum(0), (w[:, None] * step).max()
        # scores are one product, off by some 2^-23 of up to 17, and sums of fp32 numbers: 2e-5
        bound = 2.0 ** -8 * np.abs(O) + 2.0 ** -11 * S if dtype == "bf16" else 2.0 ** -22 * part
        bound = bound + 2.0 ** -23 * most * code.sum(0) + 2e-5 * (A + S)
        assert (np.abs(got - O) <= bound).all(), (power, (np.abs(got - O) / bound).max())
