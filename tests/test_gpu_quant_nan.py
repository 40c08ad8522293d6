"""Values and queries that are not finite, in a decode step over a quantised cache: a row that sees a token of NaN is NaN
however the step is cut, and so is a row whose query has a NaN or an infinity; other sequences are as without.
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


# (dtype, d_k, d_v, query heads of a cached head, new tokens): every kernel and number of rows of a block
LAYERS = [("bf16", 64, 64, 1, 1), ("bf16", 64, 64, 2, 3), ("bf16", 128, 128, 1, 1), ("bf16", 128, 128, 3, 1), ("bf16", 128, 128, 5, 3),
          ("bf16", 64, 64, 2, 128), ("bf16", 128, 128, 2, 129), ("f32", 64, 64, 1, 1), ("f32", 128, 128, 2, 2), ("f32", 24, 24, 9, 1),
          ("f32", 20, 37, 1, 1), ("f32", 130, 130, 2, 2)]
# (sequences, capacity, the first one's length, its tokens of NaN): clusters whose last CTA has one token, or whose first has
# nothing else; several clusters of one sequence; sequences cut evenly
CUTS = [(1, 400, 385, (384, 385)), (1, 1024, 1024, (0, 128)), (2, 1024, 1024, (896, 1024)), (1, 20000, 20000, (0, 128)),
        (1, 20000, 20000, (0, 2500)), (1, 20000, 129, (128, 129)), (40, 1500, 1500, (0, 256)), (40, 1500, 1409, (1408, 1409)),
        (3, 500, 500, (0, 500))]


@pytest.mark.parametrize("dtype,d,dv,per,Tq", LAYERS)
@pytest.mark.parametrize("B,T,L,where", CUTS)
@pytest.mark.parametrize("bits", [4, 8])
def test_tokens_of_nan_are_seen(dtype, d, dv, per, Tq, B, T, L, where, bits):
    h_kv = 2
    layer = base._layer(dtype, h_kv * per, d, h_kv, dv)
    clean = layer.quant_cache(B, T, bits)
    g = torch.Generator(device="cuda").manual_seed(3)
    K, V = (torch.randn((B, T, h_kv * w), generator=g, device="cuda").to(layer.dtype) for w in (d, dv))
    layer.quant_write(clean, K, V, base._ints([T] * B))
    lengths = [max(L, Tq)] + [max(Tq, T - 7 * b) for b in range(1, B)]
    Q = to_device(wl.random_tensor((B, Tq, h_kv * per * d), 4, dtype), dtype)
    want = layer.decode_quant(Q, clean, base._ints(lengths))
    assert torch.isfinite(want).all()
    for side in ("K_params", "V_params"):
        cache = layer.quant_cache(B, T, bits)
        cache.data.copy_(clean.data)
        getattr(cache, side)[0, 1, where[0]:where[1]] = float("nan")  # the second cached head's
        got = layer.decode_quant(Q, cache, base._ints(lengths))
        first = torch.arange(Tq, device="cuda") + lengths[0] - Tq >= where[0]  # rows that see one
        heads = got[0].view(Tq, h_kv, per, dv)
        assert torch.isnan(heads[first, 1]).all()
        assert torch.equal(heads[:, 0], want[0].view(Tq, h_kv, per, dv)[:, 0])
        assert torch.equal(got[1:], want[1:])
    assert layer.status() == 0


@pytest.mark.parametrize("dtype,d,dv,per,Tq", LAYERS)
@pytest.mark.parametrize("B,T", [(1, 300), (1, 8000), (30, 700)])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_queries_that_are_not_finite(dtype, d, dv, per, Tq, B, T, bad):
    """Such a query head's output is NaN, every other one's stays within its bound."""
    h_kv, bits = 2, 4
    h = h_kv * per
    layer = base._layer(dtype, h, d, h_kv, dv)
    cache, held = base._filled(layer, 3, dtype, B, T, bits)
    lengths = [max(Tq, T - 7 * b) for b in range(B)]
    Q = wl.random_tensor((B, Tq, h * d), 4, dtype)
    hurt = Q.copy()
    hurt[0, Tq - 1, d - 1] = bad                                     # the first head's, of the last new token
    got = to_host(layer.decode_quant(to_device(hurt, dtype), cache, base._ints(lengths)))
    assert np.isnan(got[0, Tq - 1, :dv]).all()
    held = tuple(x[:1] for x in held)
    O, A, S = qc.decode(Q[:1], *held, h, lengths[:1])
    keep = np.ones(O.shape, bool)
    keep[0, Tq - 1, :dv] = False
    base._check(got[:1][keep], O[keep], A[keep], S[keep], dtype, "beside a query that is not finite")
    assert np.isfinite(got[1:]).all()
