"""Decode steps over a quantised cache give the same bits every time, whatever ran before them on the same multiprocessors
(shared memory keeps what the last kernel left), and as part of whatever batch of equal steps."""
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


@pytest.mark.parametrize("dtype,d,per,Tq", [("bf16", 64, 4, 130), ("bf16", 128, 3, 100), ("bf16", 64, 8, 70), ("bf16", 128, 5, 3),
                                            ("bf16", 64, 3, 1), ("f32", 64, 3, 3), ("f32", 128, 3, 1), ("f32", 50, 1, 1)])
@pytest.mark.parametrize("bits", [4, 8])
def test_the_same_bits_after_other_steps(dtype, d, per, Tq, bits):
    """Steps of values 2^40 apart, whose rows' scales move all the time, in blocks that rows fill in part."""
    h_kv, B, T = 2, 100, 3000
    layer = base._layer(dtype, h_kv * per, d, h_kv)
    g = torch.Generator(device="cuda").manual_seed(4)
    K, V, W = (torch.randn((B, T, h_kv * d), generator=g, device="cuda") for _ in range(3))
    V *= torch.exp2(torch.randint(-20, 20, (B, T, 1), generator=g, device="cuda").float())
    lens = torch.randint(Tq, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    cache, other = layer.quant_cache(B, T, bits), layer.quant_cache(B, T, bits)
    for c, v in ((cache, V), (other, W)):
        layer.quant_write(c, K.to(layer.dtype), v.to(layer.dtype), base._ints([T] * B))
    Q = torch.randn((B, Tq, h_kv * per * d), generator=g, device="cuda").to(layer.dtype)
    full = torch.randn((B, max(128, Tq), h_kv * per * d), generator=g, device="cuda").to(layer.dtype)
    outs = []
    for scale in (0.0, 2.0 ** -20, 1.0, 2.0 ** 30, np.nan):
        layer.decode_quant(full * scale, other, base._ints([T] * B))  # blocks that are filled
        layer.decode_quant(Q * scale, other, lens)
        outs.append(layer.decode_quant(Q, cache, lens))
    assert torch.isfinite(outs[0]).all()
    for x in outs[1:]:
        assert torch.equal(x, outs[0])
    assert layer.status() == 0
