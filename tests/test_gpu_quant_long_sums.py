"""Decode steps of bf16 layers whose CTAs each take tens of thousands of tokens of a quantised cache: values around zero
under nearly even weights, where the outputs are a thousandth of the sums of codes that they come from.

The outputs' distance from the 64-bit definition, as a norm: 2^-8 of the outputs' (their rounding); sqrt(sum_j (w_j s_j
code_j)^2) 2^-11, as the products of weights and steps are rounded to 11 bits independently of each other; and `cut` of
sum_j w_j s_j code_j: n additions to a sum that grows evenly, each cut off by less than 2^-23 of it, take less than
n 2^-24.  n is 32 for a few rows (the bound allows for 64) and 128 for hundreds.  A sum of all the tokens' products that is
cut off with every product (512 of a warp, 2048 of a row) lies outside.
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


def _check_even_weights(B, T, h, h_kv, d, bits, Tq, cut):
    layer = base._layer("bf16", h, d, h_kv)
    g = torch.Generator(device="cuda").manual_seed(3)
    one, cache = layer.quant_cache(1, T, bits), layer.quant_cache(B, T, bits)
    K, V = (torch.randn((1, T, h_kv * d), generator=g, device="cuda").bfloat16() for _ in "KV")
    layer.quant_write(one, 0.25 * K, V, base._ints([T]))
    del K, V
    for name in ("K_codes", "K_params", "V_codes", "V_params"):
        to = getattr(cache, name)
        to.copy_(getattr(one, name).expand_as(to))
    Q = torch.randn((B, Tq, h * d), generator=g, device="cuda").bfloat16()
    got = layer.decode_quant(Q, cache, base._ints([T] * B))
    assert layer.status() == 0

    def plane(x):
        codes, params = (getattr(one, f"{x}_{y}")[0] for y in ("codes", "params"))
        if bits == 4:
            codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
        s, m = (params[..., i].double().repeat_interleave(64, -1) for i in range(2))
        return codes.double() * s, m

    (ks, km), (vs, vm) = plane("K"), plane("V")
    per = h // h_kv
    for b in (0, B // 2, B - 1):
        q = Q[b].double().view(Tq, h_kv, per, d).permute(1, 2, 0, 3).reshape(h_kv, per * Tq, d)
        x = q @ (ks + km).mT / np.sqrt(d)
        t = torch.arange(Tq, device="cuda").repeat(per)
        w = torch.softmax(x.masked_fill(torch.arange(T, device="cuda") > (T - Tq + t)[:, None], -np.inf), -1)
        want = w @ (vs + vm)
        have = got[b].double().view(Tq, h_kv, per, d).permute(1, 2, 0, 3).reshape(h_kv, per * Tq, d)
        bound = 2.0 ** -8 * want.norm() + 2.0 ** -11 * ((w * w) @ (vs * vs)).sum().sqrt() + cut * (w @ vs).norm()
        assert (have - want).norm() <= bound, ((have - want).norm() / want.norm()).item()


@pytest.mark.parametrize("h,h_kv,d,bits,Tq", [(2, 2, 128, 8, 1), (2, 2, 64, 8, 8), (4, 2, 128, 4, 4), (2, 2, 128, 4, 1)])
def test_even_weights_of_long_sequences(h, h_kv, d, bits, Tq):
    _check_even_weights(152, 65536, h, h_kv, d, bits, Tq, 2.0 ** -18)


@pytest.mark.parametrize("h,h_kv,d,bits,Tq", [(4, 2, 128, 4, 128), (4, 2, 64, 8, 128), (4, 2, 128, 8, 150), (2, 1, 64, 4, 129)])
def test_even_weights_under_many_rows(h, h_kv, d, bits, Tq):
    """Hundreds of query rows of a cached head."""
    _check_even_weights(40 if h_kv == 2 else 60, 32768, h, h_kv, d, bits, Tq, 2.0 ** -17)


@pytest.mark.parametrize("d,Tq,bits", [(64, 257, 4), (128, 300, 8)])
def test_moving_references_under_many_rows(d, Tq, bits):
    """The same paths with scores that rise along the keys and steps that differ by 2^40, blocks of rows partly filled, and
    pieces that begin and end inside a sequence."""
    B, T = 60, 6000
    layer = base._layer("bf16", 1, d, 1)
    rnd = lambda x: wl.bf16_to_f32(wl.bf16_bits(x.astype(np.float32)))  # noqa: E731
    Q, K, V = (wl.random_tensor((1, n, d), 70 + i, "bf16") for i, n in enumerate((Tq, T, T)))
    powers = 2.0 ** np.random.default_rng(3).integers(-20, 20, T)[None, :, None]
    K, V = rnd(K * np.linspace(0.1, 3.0, T)[None, :, None]), rnd(V * powers)
    one, cache = layer.quant_cache(1, T, bits), layer.quant_cache(B, T, bits)
    layer.quant_write(one, to_device(K, "bf16"), to_device(V, "bf16"), base._ints([T]))
    for name in ("K_codes", "K_params", "V_codes", "V_params"):
        to = getattr(cache, name)
        to.copy_(getattr(one, name).expand_as(to))
    held = tuple(x[:, :, :T] for x in base._held(one, "K") + base._held(one, "V"))
    got = to_host(layer.decode_quant(to_device(np.repeat(Q, B, 0), "bf16"), cache, base._ints([T] * B)))
    O, A, S = qc.decode(Q, *held, 1, [T])
    assert layer.status() == 0 and np.isfinite(got).all()
    assert (np.abs(got - O) <= base._bound(Q, held, 1, d, bits, O, A, S, "bf16")).all()
