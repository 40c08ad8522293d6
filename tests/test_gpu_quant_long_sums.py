"""Decode steps of bf16 layers whose CTAs each take tens of thousands of tokens of a quantised cache: values around zero
under nearly even weights, where the outputs are a thousandth of the sums of codes that they come from.

The outputs' distance from the 64-bit definition, as a norm: 2^-8 of the outputs' (their rounding); sqrt(sum_j (w_j s_j
code_j)^2) 2^-11, as the products of weights and steps are rounded to 11 bits independently of each other; and 2^-18 of
sum_j w_j s_j code_j, for at most 2^6 fp32 additions to sums that grow evenly, each cut off by less than 2^-23 of its sum.
A sum of all the tokens' products that is cut off with every product (512 of a warp) lies
outside.
"""
import numpy as np
import pytest

import test_gpu_quant_cache as base

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build_library()
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)


def _check_even_weights(B, T, h, h_kv, d, bits, Tq):
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
        bound = 2.0 ** -8 * want.norm() + 2.0 ** -11 * ((w * w) @ (vs * vs)).sum().sqrt() + 2.0 ** -18 * (w @ vs).norm()
        assert (have - want).norm() <= bound, ((have - want).norm() / want.norm()).item()


@pytest.mark.parametrize("h,h_kv,d,bits,Tq", [(2, 2, 128, 8, 1), (2, 2, 64, 8, 8), (4, 2, 128, 4, 4), (2, 2, 128, 4, 1)])
def test_even_weights_of_long_sequences(h, h_kv, d, bits, Tq):
    _check_even_weights(152, 65536, h, h_kv, d, bits, Tq)
