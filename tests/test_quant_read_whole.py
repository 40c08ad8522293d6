"""quant_read without counts, rows or outputs reads whole sequences of any lengths."""
import pytest

torch = pytest.importorskip("torch")

from transformer_head_scaled_02_gb300 import Mha, _lib  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build_library()


def test_counts_of_a_whole_read(monkeypatch):
    """(No GPU: the entry point is replaced.)  Counts are the lengths, and T_out of them where T_out or outputs are given."""
    layer = Mha(64, 1, 64, dtype=torch.float32, device="cpu")
    cache = layer.quant_cache(2, 32)
    calls = []
    layer._c_quant = (None, lambda *a: calls.append(a) or _lib.MHA_OK, None)
    monkeypatch.setattr(layer, "_quant_ready", lambda *a: 0)
    lens, x = torch.tensor([3, 20], dtype=torch.int32), torch.zeros((2, 5, 64))
    layer.quant_read(cache, lens)
    layer.quant_read(cache, lens, T_out=3)
    layer.quant_read(cache, lens, K_out=x, V_out=x.clone())
    layer.quant_read(cache, lens, lens, K_out=x, V_out=x.clone())
    p = lens.data_ptr()
    assert [(a[5], a[10], a[11]) for a in calls] == [(32, p, p), (3, p, None), (5, p, None), (5, p, p)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_whole_read(dtype):
    torch.cuda.set_device(0)
    layer = Mha(128, 2, 64, dtype=dtype)
    lengths = [1, 30, 48, 0, 17]
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    K, V = (torch.randn((5, 48, 128), generator=g, device="cuda").to(dtype) for _ in "KV")
    cache = layer.quant_cache(5, 48, 8)
    layer.quant_write(cache, K, V, lens, lens)
    Ko, Vo = layer.quant_read(cache, lens)
    assert layer.status() == 0
    # within half a step of what was written, and half a step of bf16: steps and lowest values are rounded outwards by
    # at most 2^-7 of themselves
    for got, x in ((Ko, K), (Vo, V)):
        assert got.shape == x.shape
        for b, n in enumerate(lengths):
            y, z = (t[b, :n].float().view(n, 2, 64) for t in (got, x))
            if n:
                low, high = z.amin(-1, keepdim=True), z.amax(-1, keepdim=True)
                step = (high - low + low.abs() * 2.0 ** -7) / 255 * (1 + 2.0 ** -7)
                assert ((y - z).abs() <= step / 2 + 2.0 ** -8 * (z.abs() + step)).all()
