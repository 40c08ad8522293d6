"""The quantised-cache calls allocate no device memory: free memory is the same before and after each of them, once its
kernels have been loaded.  Named to be collected last, as allocations of other tests would count."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from transformer_head_scaled_02_gb300 import Mha  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build_library()
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)


# clusters, several of one sequence, an even cut with its join, hundreds of rows, heads on CUDA cores
@pytest.mark.parametrize("dtype,d,dv,h,h_kv,B,T,Tq", [
    (torch.bfloat16, 64, 64, 4, 2, 2, 1000, 1), (torch.bfloat16, 128, 128, 8, 2, 1, 20000, 1),
    (torch.bfloat16, 128, 128, 4, 4, 40, 1500, 1), (torch.bfloat16, 64, 64, 4, 1, 2, 700, 100),
    (torch.float32, 20, 37, 4, 2, 3, 900, 2)])
@pytest.mark.parametrize("bits", [4, 8])
def test_no_device_memory_is_allocated(dtype, d, dv, h, h_kv, B, T, Tq, bits):
    layer = Mha(h * d, h, d, dv, dtype=dtype, h_kv=h_kv)
    cache = layer.quant_cache(B, T, bits)
    K, V = (torch.randn((B, T, h_kv * w), device="cuda").to(dtype) for w in (d, dv))
    Q = torch.randn((B, Tq, h * d), device="cuda").to(dtype)
    out = torch.empty((B, Tq, h * dv), device="cuda", dtype=dtype)
    lens = torch.full((B,), T, dtype=torch.int32, device="cuda")

    def calls():
        layer.quant_write(cache, K, V, lens)
        yield "write"
        layer.decode_quant(Q, cache, lens, out=out)
        yield "decode"
        layer.quant_read(cache, lens, K_out=K, V_out=V)
        yield "read"

    for _ in calls():
        torch.cuda.synchronize()
    torch_held = torch.cuda.memory_reserved()
    free = torch.cuda.mem_get_info()[0]
    for name in calls():
        torch.cuda.synchronize()
        assert torch.cuda.mem_get_info()[0] == free, name
    assert torch.cuda.memory_reserved() == torch_held
    assert layer.status() == 0
