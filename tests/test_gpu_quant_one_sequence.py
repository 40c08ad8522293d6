"""A decode step over one long sequence of a quantised cache: every group has several clusters of CTAs, whose records a
second launch joins, and at lengths far below the capacity most of them have nothing."""
import numpy as np
import pytest

import test_gpu_quant_cache as base
from gpu_util import to_device, to_host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from transformer_head_scaled_02_gb300 import _lib  # noqa: E402
from transformer_head_scaled_02_gb300 import workloads as wl  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build_library()
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 100)])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("per,Tq", [(1, 1), (2, 1), (2, 4), (8, 2)])
def test_lengths_of_one_long_sequence(dtype, d, bits, per, Tq):
    h_kv, T = 2, 20000
    layer = base._layer(dtype, h_kv * per, d, h_kv)
    cache, held = base._filled(layer, 5, dtype, 1, T, bits)
    held = tuple(x[:, :, :T] for x in held)
    Q = wl.random_tensor((1, Tq, h_kv * per * d), 6, dtype)
    for L in (T, 9001, 4097, 129, 128, Tq):
        base._step(layer, cache, held, Q, [L], dtype, f"length {L}")
    assert layer.status() == 0
    for L in (Tq - 1, cache.T_max + 1):
        assert np.isnan(to_host(layer.decode_quant(to_device(Q, dtype), cache, base._ints([L])))).all()
        assert layer.status() == _lib.MHA_ERR_BAD_LENGTH
