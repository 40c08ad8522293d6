"""Copies of a quantised cache (a sequence that forks, a cache that is stored) have a buffer of their own, which their views
and every call of theirs use."""
import copy
import pickle

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from transformer_head_scaled_02_gb300 import Mha, _lib  # noqa: E402

VIEWS = ("K_codes", "K_params", "V_codes", "V_params")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build_library()


def _stored(cache):
    return pickle.loads(pickle.dumps(cache))


@pytest.mark.parametrize("fork", [copy.deepcopy, _stored])
def test_a_copy_has_a_buffer_of_its_own(fork, monkeypatch):
    layer = Mha(192, 3, 64, dtype=torch.float32, device="cpu")
    cache = layer.quant_cache(2, 20, 8)
    for i, name in enumerate(VIEWS):
        getattr(cache, name).fill_(i + 1)
    other = fork(cache)
    assert (other.B, other.T_max, other.bits) == (2, 32, 8)
    # the views are of the copy's buffer, with what the original held
    for i, name in enumerate(VIEWS):
        a, b = getattr(cache, name), getattr(other, name)
        assert torch.equal(a, b) and a.data_ptr() - cache.data.data_ptr() == b.data_ptr() - other.data.data_ptr()
        b.fill_(9)
        assert (getattr(cache, name) == i + 1).all() and (getattr(other, name) == 9).all()
    # and the calls get its address (no GPU: the entry points are replaced, and the check of devices)
    seen = []
    layer._c_quant = tuple(lambda *a, i=i: seen.append(a[4 if i < 2 else 7]) or _lib.MHA_OK for i in range(3))
    monkeypatch.setattr(layer, "_quant_ready", lambda *a: 0)
    monkeypatch.setattr(_lib, "mha_decode_quant_workspace_size", lambda *a: 256)
    x, lens = torch.zeros((2, 3, 192)), torch.full((2,), 3, dtype=torch.int32)
    for c in (cache, other):
        layer.quant_write(c, x, x, lens)
        layer.quant_read(c, lens, T_out=3)
        layer.decode_quant(x, c, lens)
        assert seen == [c.data.data_ptr()] * 3
        seen.clear()
    assert cache.data.data_ptr() != other.data.data_ptr()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 64), (torch.float32, 40)])
def test_forked_sequences(dtype, d):
    """A cache is forked, each copy takes another next token, and the original goes: both go on from the common tokens."""
    torch.cuda.set_device(0)
    h, T = 4, 50
    layer = Mha(h * d, h, d, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    K, V, Q, k, v, k2, v2 = (torch.randn((2, n, h * d), generator=g, device="cuda").to(dtype) for n in (T, T, 1, 1, 1, 1, 1))
    lens = torch.full((2,), T, dtype=torch.int32, device="cuda")

    def alone(a, b):
        c = layer.quant_cache(2, 80)
        layer.quant_write(c, torch.cat((K, a), 1), torch.cat((V, b), 1), lens + 1)
        return layer.decode_quant(Q, c, lens + 1)

    cache = layer.quant_cache(2, 80)
    layer.quant_write(cache, K, V, lens)
    forks = [copy.deepcopy(cache), copy.deepcopy(cache)]
    before = layer.decode_quant(Q, cache, lens)
    for f, a, b in zip(forks, (k, k2), (v, v2)):
        layer.quant_write(f, a, b, lens + 1)
    assert torch.equal(layer.decode_quant(Q, cache, lens), before)
    del cache
    for f, a, b in zip(forks, (k, k2), (v, v2)):
        assert torch.equal(layer.decode_quant(Q, f, lens + 1), alone(a, b))
    assert np.all(layer.status() == 0)
