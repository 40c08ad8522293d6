"""The quantised cache without a GPU: host refusals of the C entry points and of the Python front end, sizes and
layout, and the oracle's own pins."""
import numpy as np
import pytest

from oracle import quant_cache as qc
from transformer_head_scaled_02_gb300 import _lib as L


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build_library()
    return L.load()


FAKE = 1 << 40  # never dereferenced: rejected earlier
G = 1 << 30


@pytest.fixture
def handles(lib):
    hs = {"bf": L.mha_create_ex(512, 8, 2, 64, 64, 0, L.MHA_BF16), "odd": L.mha_create(96, 3, 32, 32, L.MHA_BF16),
          "f32": L.mha_create_ex(96, 4, 2, 24, 80, 0, L.MHA_F32), "wide": L.mha_create(600, 2, 300, 300, L.MHA_F32),
          "many": L.mha_create(8, 600000, 1, 1, L.MHA_F32)}
    yield hs
    for h in hs.values():
        L.mha_destroy(h)


def test_cache_size(handles):
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    for name, h_kv, dk, dv in (("bf", 2, 64, 64), ("f32", 2, 24, 80)):
        for bits in (4, 8):
            for B, T in ((1, 16), (3, 48), (2, 1040)):
                size, off = L.mha_quant_cache_size(handles[name], bits, B, T)
                n, want, at = B * h_kv * T, [], 0
                for d in (dk, dv):
                    for part in (n * ((d + 31) // 32 * 32) * bits // 8, n * ((d + 63) // 64) * 4):
                        want.append(at)
                        at += up(part)
                assert off == tuple(want) and size == at
    for bad in ((5, 1, 16), (0, 1, 16), (4, -1, 16), (4, 1, -16), (4, 1, 17), (4, 1 << 16, 1 << 16)):
        assert L.mha_quant_cache_size(handles["bf"], *bad)[0] == 0, bad
    assert L.mha_quant_cache_size(None, 4, 1, 16)[0] == 0
    assert L.load().mha_quant_cache_size(handles["bf"], 4, 1, 16, None) == L.mha_quant_cache_size(handles["bf"], 4, 1, 16)[0]


@pytest.mark.parametrize("call_of", ["write", "read"])
def test_copy_refusals(handles, call_of):
    def call(h="bf", **kw):
        a = dict(bits=4, B=2, T_max=112, cache=FAKE, K=FAKE + G, ldk=128, V=FAKE + 2 * G, ldv=128,
                 cache_lengths=FAKE + 3 * G, counts=FAKE + 3 * G + 64, stream=None)
        a["T_new" if call_of == "write" else "T_out"] = 10
        a.update(kw)
        return getattr(L, f"mha_quant_{call_of}")(None if h is None else handles[h], check=False, **a)
    bad = L.MHA_ERR_INVALID_ARG
    T = "T_new" if call_of == "write" else "T_out"
    cases = [dict(h=None), dict(bits=3), dict(bits=0), dict(B=-1), dict(T_max=-16), dict(T_max=100), dict(T_max=0), {T: -1},
             dict(cache=None), dict(cache=FAKE + 128), dict(K=None), dict(V=None), dict(ldk=64), dict(ldv=120), dict(ldk=132),
             dict(K=FAKE + G + 8), dict(cache_lengths=None), dict(K=FAKE + 4096), dict(V=FAKE + 2 * 2 * 112 * 36 - 512),
             dict(B=1 << 16, T_max=1 << 16), {"B": 1 << 16, "T_max": 16, T: 1 << 16}]
    if call_of == "write":
        cases += [dict(cache_lengths=FAKE), dict(counts=FAKE + 256)]
    else:
        cases += [dict(V=FAKE + G), dict(V=FAKE + G + 128), dict(ldk=256, ldv=256, V=FAKE + G + 128),
                  dict(ldk=384, ldv=256, V=FAKE + G + 256), dict(cache_lengths=FAKE + G), dict(counts=FAKE + 2 * G + 16)]
    for kw in cases:
        assert call(**kw) == bad, kw
    assert call("odd", ldk=96, ldv=96) == L.MHA_ERR_UNSUPPORTED
    assert call("wide", ldk=600, ldv=600) == L.MHA_ERR_UNSUPPORTED
    assert call("many", B=1, T_max=1 << 17, ldk=600000, ldv=600000, V=FAKE + (1 << 43), cache=FAKE + (1 << 44),
                cache_lengths=FAKE + (1 << 45), counts=None, **{T: 1 << 17}) == L.MHA_ERR_UNSUPPORTED
    assert call(B=0) == L.MHA_OK and call(**{T: 0}) == L.MHA_OK


def test_decode_refusals(handles):
    def call(h="bf", **kw):
        a = dict(bits=4, B=2, T_q=1, T_max=112, Q=FAKE + G, ldq=512, cache=FAKE, cache_lengths=FAKE + 3 * G, O=FAKE + 2 * G,
                 ldo=512, stream=None)
        a.update(kw)
        return L.mha_decode_quant(None if h is None else handles[h], check=False, **a)
    for kw in (dict(h=None), dict(bits=16), dict(B=-1), dict(T_q=-1), dict(T_max=-16), dict(T_max=111), dict(T_q=113),
               dict(T_max=0), dict(Q=None), dict(O=None), dict(cache=None), dict(cache=FAKE + 16), dict(cache_lengths=None),
               dict(ldq=504), dict(ldq=516), dict(ldo=256), dict(O=FAKE + 2 * G + 4), dict(O=FAKE + G + 512), dict(O=FAKE),
               dict(O=FAKE + 3 * G - 16), dict(B=1 << 20, T_q=1 << 12, T_max=1 << 12)):
        assert call(**kw) == L.MHA_ERR_INVALID_ARG, kw
    assert call("odd", ldq=96, ldo=96) == L.MHA_ERR_UNSUPPORTED
    assert call("wide", ldq=600, ldo=600) == L.MHA_ERR_UNSUPPORTED
    assert call() == L.MHA_ERR_WORKSPACE and call("f32", ldo=320) == L.MHA_ERR_WORKSPACE
    assert call(B=0) == L.MHA_OK and call(T_q=0) == L.MHA_OK


def test_decode_workspace_size(handles):
    size = L.mha_decode_quant_workspace_size
    for name in ("bf", "f32"):
        assert 256 <= size(handles[name], 1, 1, 16) <= size(handles[name], 1, 1, 65536)
        assert size(handles[name], 0, 1, 16) == size(handles[name], 1, 0, 16) == 256
        for bad in ((-1, 1, 16), (1, -1, 16), (1, 1, -16), (1, 1, 17), (1 << 16, 1, 1 << 16)):
            assert size(handles[name], *bad) == 0, bad
    assert size(None, 1, 1, 16) == 0
    # the records stay small beside the caches they belong to
    assert size(handles["bf"], 64, 1, 8192) < 64 << 20 and size(handles["bf"], 1, 4096, 8192) < 256 << 20


@pytest.mark.parametrize("bits", [4, 8])
def test_oracle_against_fractions(bits):
    rng = np.random.default_rng(bits)
    n = 2 ** bits - 1
    groups = [rng.standard_normal(64), rng.standard_normal(17) * 1e-3 + 5, np.full(64, -2.5), np.arange(64.0) / 4,
              np.r_[np.arange(0, n + 0.5, 0.5)[:64], n] * 0.375, np.r_[0.0, 1e-30, 1.0], -np.arange(9.0) * 3, np.zeros(1),
              rng.standard_normal(64) * 1e30]
    for x in groups:
        x = np.asarray(x, np.float32)[:64]
        codes, params = qc.quantise(x[None], bits)
        c, s, m = qc.quantise_exact(x, bits)
        assert (codes[0] == c).all() and params[0, 0, 0] == s and params[0, 0, 1] == m
        assert codes.max() <= n and codes.min() >= 0
        # every value within half a step
        assert (np.abs(qc.values(codes, params)[0] - x) <= s / 2 * (1 + 2.0 ** -40)).all()
        assert (qc.unpack(qc.pack(codes, bits), bits, x.size) == codes).all()
    bad = np.array([[1.0, np.nan, 2.0], [1.0, np.inf, 0.0], [1.0, 3.4e38, 0.0]])
    assert np.isnan(qc.quantise(bad, bits)[1]).all()


def test_front_end_refusals():
    torch = pytest.importorskip("torch")
    from transformer_head_scaled_02_gb300 import Mha
    layer = Mha(64, 1, 64, dtype=torch.bfloat16, device="cpu")  # (no CUDA call is made before the refusals)
    for bad in ((1, 16, 3), (1, 16, 16)):
        with pytest.raises(ValueError):
            layer.quant_cache(*bad)
    for bad in ((-1, 16), (1, -1), (1 << 16, 1 << 16), (1, 2 ** 31)):
        with pytest.raises(ValueError):
            layer.quant_cache(*bad)
    cache = layer.quant_cache(2, 20)
    assert (cache.B, cache.T_max, cache.bits) == (2, 32, 4)
    assert cache.K_codes.shape == (2, 1, 32, 32) and cache.V_params.shape == (2, 1, 32, 1, 2)
    x, lens = torch.zeros((2, 3, 64), dtype=torch.bfloat16), torch.tensor([3, 3], dtype=torch.int32)
    cases = [lambda: layer.quant_write(cache, x, x, lens),                       # not on a CUDA device
             lambda: layer.quant_write(cache, x[:1], x, lens), lambda: layer.quant_write(cache, x, x.float(), lens),
             lambda: layer.quant_write(cache, x, x[:, :2], lens), lambda: layer.quant_write(cache, x, x, lens.long()),
             lambda: layer.quant_write(cache, x, x, lens[:1]), lambda: layer.quant_write(cache, x, x, lens, lens[:1]),
             lambda: layer.quant_write(cache, x.transpose(0, 1), x, lens),
             lambda: layer.quant_read(cache, lens, T_out=3), lambda: layer.quant_read(cache, lens, K_out=x, V_out=x[:, :1]),
             lambda: layer.quant_read(cache, lens, lens.float(), K_out=x, V_out=x),
             lambda: layer.decode_quant(x, cache, lens), lambda: layer.decode_quant(x[:1], cache, lens),
             lambda: layer.decode_quant(x[..., :32], cache, lens), lambda: layer.decode_quant(x, cache, lens, out=x.float()),
             lambda: Mha(128, 2, 64, dtype=torch.bfloat16, device="cpu").decode_quant(x, cache, lens)]
    for call in cases:
        with pytest.raises(ValueError):
            call()
