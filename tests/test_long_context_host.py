"""The long-context operators without a GPU: host refusals of the C entry points and of the Python front
end, workspace sizes, and the oracle's own pins."""
import numpy as np
import pytest

from oracle import long_context as lc
from transformer_head_scaled_02_gb300 import _lib as L


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build_library()
    return L.load()


FAKE = 1 << 40  # never dereferenced: rejected earlier


@pytest.fixture
def handles(lib):
    hs = {"bf": L.mha_create_ex(512, 8, 2, 64, 64, 0, L.MHA_BF16), "odd": L.mha_create(96, 3, 32, 32, L.MHA_BF16),
          "f32": L.mha_create_ex(96, 4, 2, 24, 40, 0, L.MHA_F32), "wide": L.mha_create(600, 2, 300, 300, L.MHA_F32)}
    yield hs
    for h in hs.values():
        L.mha_destroy(h)


def test_attention_window_refusals(handles):
    def call(h="bf", **kw):
        a = dict(B=2, T=100, Q=FAKE, ldq=512, K=FAKE + (1 << 30), ldk=128, V=FAKE + (2 << 30), ldv=128, G=None, ldg=0,
                 window=16, sinks=4, kv_lengths=None, O=FAKE + (3 << 30), ldo=512, stream=None)
        a.update(kw)
        return L.mha_attention_window(None if h is None else handles[h], check=False, **a)
    bad = L.MHA_ERR_INVALID_ARG
    assert call(None) == bad
    for kw in (dict(B=-1), dict(T=-1), dict(window=0), dict(window=-5), dict(sinks=-1), dict(Q=None), dict(O=None),
               dict(ldq=511), dict(ldq=504), dict(ldk=120), dict(ldv=100), dict(ldo=100), dict(ldq=516), dict(Q=FAKE + 2),
               dict(G=FAKE + 8, ldg=512), dict(G=FAKE + (4 << 30), ldg=8), dict(O=FAKE + 512), dict(O=FAKE + (1 << 30)),
               dict(O=FAKE + (2 << 30)), dict(B=1 << 20, T=1 << 20)):
        assert call(**kw) == bad, kw
    assert call("odd") == L.MHA_ERR_UNSUPPORTED
    assert call("wide", ldq=600, ldk=600, ldv=600, ldo=600) == L.MHA_ERR_UNSUPPORTED
    assert call(B=0) == L.MHA_OK and call(T=0) == L.MHA_OK


def test_forward_window_refusals(handles):
    def call(h="bf", **kw):
        a = dict(X=FAKE, B=2, T=100, W_qkv=FAKE + (1 << 30), b_qkv=None, W_o=FAKE + (2 << 30), b_o=None, window=16,
                 sinks=4, kv_lengths=None, residual=None, out=FAKE + (3 << 30), stream=None)
        a.update(kw)
        return L.mha_forward_window(None if h is None else handles[h], check=False, **a)
    for kw in (dict(h=None), dict(window=0), dict(sinks=-1), dict(X=None), dict(out=FAKE), dict(B=-1)):
        assert call(**kw) == L.MHA_ERR_INVALID_ARG, kw
    assert call("odd") == L.MHA_ERR_UNSUPPORTED
    assert call() == L.MHA_ERR_WORKSPACE
    assert call(B=0) == L.MHA_OK


@pytest.mark.parametrize("step", ["window", "shared", "weights"])
def test_step_refusals(handles, step):
    def call(h="bf", **kw):
        a = dict(B=2, T_q=1, T_max=100, Q=FAKE, ldq=512, K_cache=FAKE + (1 << 30), ldk=128, V_cache=FAKE + (2 << 30),
                 ldv=128, cache_lengths=FAKE + 4, O=FAKE + (3 << 30), ldo=512, stream=None)
        if step == "window":
            a.update(window=16, sinks=2)
        if step == "shared":
            a.update(T_prefix=50, K_prefix=FAKE + (4 << 30), ldkp=128, V_prefix=FAKE + (5 << 30), ldvp=128)
        if step == "weights":
            a.update(weights=FAKE + (6 << 30))
        a.update(kw)
        return getattr(L, f"mha_decode_{step}")(None if h is None else handles[h], check=False, **a)
    bad = L.MHA_ERR_INVALID_ARG
    cases = [dict(h=None), dict(B=-1), dict(T_q=-1), dict(T_max=-1), dict(T_q=101), dict(T_max=0), dict(cache_lengths=None),
             dict(Q=None), dict(K_cache=None), dict(V_cache=None), dict(O=None), dict(ldq=500), dict(ldk=64), dict(ldv=64),
             dict(ldo=500), dict(ldk=132), dict(K_cache=FAKE + (1 << 30) + 8), dict(O=FAKE), dict(O=FAKE + (1 << 30)),
             dict(O=FAKE + (2 << 30)), dict(B=1 << 16, T_max=1 << 16)]
    if step == "window":
        cases += [dict(window=0), dict(sinks=-1)]
    if step == "shared":
        cases += [dict(T_prefix=-1), dict(K_prefix=None), dict(V_prefix=None), dict(ldkp=8), dict(ldvp=130),
                  dict(O=FAKE + (4 << 30))]
    if step == "weights":
        cases += [dict(weights=None), dict(weights=FAKE), dict(weights=FAKE + (1 << 30)), dict(weights=FAKE + (3 << 30))]
    for kw in cases:
        assert call(**kw) == bad, kw
    assert call("odd", ldq=96, ldk=96, ldv=96, ldo=96) == L.MHA_ERR_UNSUPPORTED
    assert call("wide", ldq=600, ldk=600, ldv=600, ldo=600) == L.MHA_ERR_UNSUPPORTED
    assert call() == L.MHA_ERR_WORKSPACE                     # none attached
    assert call("f32", ldk=48, ldv=80, **(dict(ldkp=48, ldvp=80) if step == "shared" else {})) == L.MHA_ERR_WORKSPACE
    assert call(B=0) == L.MHA_OK and call(T_q=0) == L.MHA_OK


def test_evict_refusals(handles):
    G = 1 << 30

    def call(h="bf", **kw):
        a = dict(B=2, T_max=100, keep=40, recent=8, K_cache=FAKE, ldk=128, V_cache=FAKE + G, ldv=128,
                 cache_lengths=FAKE + 9 * G, weights=FAKE + 2 * G, T_out=40, K_out=FAKE + 3 * G, ldko=128,
                 V_out=FAKE + 4 * G, ldvo=128, weights_out=FAKE + 5 * G, kept=FAKE + 6 * G,
                 new_lengths=FAKE + 7 * G, stream=None)
        a.update(kw)
        return L.mha_cache_evict(None if h is None else handles[h], check=False, **a)
    for kw in (dict(h=None), dict(B=-1), dict(T_max=-1), dict(T_max=0), dict(keep=0), dict(recent=-1), dict(recent=41),
               dict(T_out=39), dict(K_cache=None), dict(V_out=None), dict(weights=None), dict(weights_out=None),
               dict(kept=None), dict(new_lengths=None), dict(cache_lengths=None), dict(ldk=64), dict(ldko=132),
               dict(K_out=FAKE + 3 * G + 4), dict(K_out=FAKE),                   # in place, but V and weights are not
               dict(K_out=FAKE, V_out=FAKE + G, weights_out=FAKE + 2 * G),       # in place, but T_out != T_max
               dict(K_out=FAKE, V_out=FAKE + G, weights_out=FAKE + 2 * G, T_out=100, ldko=256),
               dict(K_out=FAKE + 256), dict(V_out=FAKE), dict(weights_out=FAKE + 2 * G), dict(V_out=FAKE + 3 * G),
               dict(kept=FAKE), dict(kept=FAKE + 2 * G), dict(new_lengths=FAKE + 6 * G),
               dict(new_lengths=FAKE + 9 * G + 4), dict(B=1 << 16, T_max=1 << 16)):
        assert call(**kw) == L.MHA_ERR_INVALID_ARG, kw
    assert call("odd", ldk=96, ldv=96, ldko=96, ldvo=96) == L.MHA_ERR_UNSUPPORTED
    assert call(B=70000, T_max=40) == L.MHA_ERR_UNSUPPORTED
    assert call(B=0) == L.MHA_OK


def test_row_counts_next_to_32_bits_are_refused(lib):
    """The kernels step past the last row in 32 bits.  One head of one element: such sizes fit a GPU's memory."""
    most, G = 2 ** 31 - 2 ** 16, 1 << 38
    one, many = L.mha_create(1, 1, 1, 1, L.MHA_F32), L.mha_create(1 << 12, 1 << 12, 1, 1, L.MHA_F32)
    bad = L.MHA_ERR_INVALID_ARG
    try:
        def step(name, h=one, T_q=1, T_max=100, ld=1, **kw):
            a = dict(B=1, T_q=T_q, T_max=T_max, Q=FAKE, ldq=ld, K_cache=FAKE + G, ldk=ld, V_cache=FAKE + 2 * G, ldv=ld,
                     cache_lengths=FAKE + 8 * G, O=FAKE + 3 * G, ldo=ld, stream=None)
            a.update(kw)
            return getattr(L, f"mha_decode_{name}")(h, check=False, **a)

        def window(T):
            return L.mha_attention_window(one, 1, T, FAKE, 1, FAKE + G, 1, FAKE + 2 * G, 1, None, 0, 8, 0, None, FAKE + 3 * G,
                                          1, None, check=False)

        def evict(T_max, keep, T_out):
            return L.mha_cache_evict(one, 1, T_max, keep, 0, FAKE, 1, FAKE + G, 1, FAKE + 8 * G, FAKE + 2 * G, T_out,
                                     FAKE + 3 * G, 1, FAKE + 4 * G, 1, FAKE + 5 * G, FAKE + 6 * G, FAKE + 7 * G, None,
                                     check=False)
        prefix = dict(K_prefix=FAKE + 4 * G, ldkp=1, V_prefix=FAKE + 5 * G, ldvp=1)
        for n in (most + 1, 2 ** 31 - 1):
            assert step("window", T_max=n, window=5, sinks=0) == bad
            assert step("weights", T_max=n, weights=FAKE + 6 * G) == bad
            assert step("shared", T_max=n, T_prefix=5, **prefix) == bad
            assert step("shared", T_prefix=n, **prefix) == bad
            assert window(n) == bad
            assert evict(n, 10, 10) == bad and evict(100, 10, n) == bad and evict(100, n, n) == bad
            assert L.mha_cache_step_workspace_size(one, 1, 1, 0, n, 0) == 0
            assert L.mha_cache_step_workspace_size(one, 1, 1, n, 100, 0) == 0
        # query rows: 2^12 heads of 2^19 new tokens
        assert step("window", many, T_q=1 << 19, T_max=1 << 19, ld=1 << 12, window=5, sinks=0) == bad
        # indices of kept tokens past 2^32: into new buffers only
        wide = dict(cache_lengths=FAKE + 8 * G, T_out=1 << 20, ldko=1 << 12, ldvo=1 << 12, kept=FAKE + 6 * G,
                    new_lengths=FAKE + 7 * G, stream=None, check=False)
        assert L.mha_cache_evict(many, 1, 100, 1 << 20, 0, FAKE, 1 << 12, FAKE + G, 1 << 12, weights=FAKE + 2 * G,
                                 K_out=FAKE + 3 * G, V_out=FAKE + 4 * G, weights_out=FAKE + 5 * G,
                                 **wide) == L.MHA_ERR_UNSUPPORTED
        # a step whose join would need more blocks than a grid has, before its units are launched
        heads = L.mha_create(1, 1 << 11, 1, 1, L.MHA_F32)
        B = (1 << 20) - 40
        assert step("weights", heads, B=B, T_max=1, ld=1 << 11, weights=FAKE + 6 * G) == L.MHA_ERR_UNSUPPORTED
        assert step("window", heads, B=B, T_max=1, ld=1 << 11, window=5, sinks=0) == L.MHA_ERR_WORKSPACE
        L.mha_destroy(heads)
        # the layer refuses what its attention refuses before the projection is launched
        f = dict(X=FAKE, W_qkv=FAKE + G, b_qkv=None, W_o=FAKE + 2 * G, b_o=None, window=8, sinks=0, kv_lengths=None,
                 residual=None, out=FAKE + 3 * G, stream=None, check=False)
        assert most < 2048 * 1048560 < 2 ** 31
        assert L.mha_forward_window(one, B=2048, T=1048560, **f) == bad
        assert L.mha_forward_window(one, B=1, T=2097121, **f) == L.MHA_ERR_UNSUPPORTED
        assert L.mha_forward_window(one, B=2047, T=1048560, **f) == L.MHA_ERR_WORKSPACE
        # the largest are taken (no workspace is attached)
        assert step("window", T_max=most, window=5, sinks=0) == L.MHA_ERR_WORKSPACE
        assert step("shared", T_prefix=most, **prefix) == L.MHA_ERR_WORKSPACE
        assert window(most) == L.MHA_ERR_UNSUPPORTED         # fp32 windows end at 2097120 tokens
    finally:
        L.mha_destroy(one)
        L.mha_destroy(many)


def test_workspace_sizes(handles):
    f = L.mha_cache_step_workspace_size
    assert f(None, 1, 1, 0, 1, 0) == 0 and f(handles["bf"], -1, 1, 0, 1, 0) == 0 and f(handles["bf"], 1, 1, -1, 1, 0) == 0
    assert f(handles["bf"], 0, 1, 0, 100, 0) == 256
    for h in ("bf", "f32"):
        base = f(handles[h], 3, 2, 0, 1000, 0)
        scores = f(handles[h], 3, 2, 0, 1000, 1) - base
        assert scores >= 3 * 2 * (4 if h == "bf" else 2) * 2 * 1000 * 4      # B * h_kv * rows * T_max floats
        assert f(handles[h], 3, 2, 70, 1000, 0) > base > 256


def test_python_refusals(lib):
    torch = pytest.importorskip("torch")
    from transformer_head_scaled_02_gb300 import Mha
    layer = Mha(256, 4, 64, dtype=torch.bfloat16, h_kv=2, device="cpu")
    B, T = 2, 10

    def z(*s, dt=torch.bfloat16):
        return torch.zeros(s, dtype=dt)
    q, k = z(B, 1, 256), z(B, T, 128)
    lens, w = torch.ones(B, dtype=torch.int32), torch.zeros((B, 2, T))
    bad = [lambda: layer.decode_window(q, k, k, lens, 4),                         # host tensors
           lambda: layer.decode_window(z(B, 1, 255), k, k, lens, 4),
           lambda: layer.decode_window(q.float(), k, k, lens, 4),
           lambda: layer.decode_window(q, k[:, ::2], k, lens, 4),
           lambda: layer.decode_window(q, k.transpose(0, 1).contiguous().transpose(0, 1), k, lens, 4),
           lambda: layer.decode_window(q, k, k, lens.long(), 4),
           lambda: layer.decode_window(q, k, k, lens[:1], 4),
           lambda: layer.decode_shared(q, z(5, 64), z(5, 128), k, k, lens),
           lambda: layer.decode_shared(q, z(5, 128), z(6, 128), k, k, lens),
           lambda: layer.decode_weights(q, k, k, lens, w.double()),
           lambda: layer.decode_weights(q, k, k, lens, w[..., :9]),
           lambda: layer.attention_window(z(B, T, 256), k, z(B, T + 1, 128), 4),
           lambda: layer.evict(k, k, lens, w, 0, 0),
           lambda: layer.evict(k, k, lens, w, 4, 1, K_out=z(B, 4, 64)),
           lambda: layer.forward(z(B, T, 256), z(256, 512), None, z(256, 256), None, sinks=3),
           lambda: layer.forward(z(B, T, 256), z(256, 512), None, z(256, 256), None, window=3)]
    for f in bad:
        with pytest.raises(ValueError):
            f()


def test_sizes_past_32_bits_are_refused(lib):
    """ctypes would cut them to 32 bits."""
    torch = pytest.importorskip("torch")
    from transformer_head_scaled_02_gb300 import Mha
    layer = Mha(256, 4, 64, dtype=torch.bfloat16, h_kv=2, device="cpu")
    q, k = torch.zeros((2, 1, 256), dtype=torch.bfloat16), torch.zeros((2, 10, 128), dtype=torch.bfloat16)
    x, lens = torch.zeros((2, 10, 256), dtype=torch.bfloat16), torch.ones(2, dtype=torch.int32)
    w = torch.zeros((2, 2, 10))
    wq, wo = torch.zeros((256, 512), dtype=torch.bfloat16), torch.zeros((256, 256), dtype=torch.bfloat16)
    big = 2 ** 32 + 5
    for f in (lambda: layer.decode_window(q, k, k, lens, big), lambda: layer.decode_window(q, k, k, lens, 4, big),
              lambda: layer.attention_window(x, k, k, big), lambda: layer.attention_window(x, k, k, 4, -big),
              lambda: layer.forward(x, wq, None, wo, None, causal=True, window=big),
              lambda: layer.evict(k, k, lens, w, 4, big), lambda: layer.evict(k, k, lens, w, big, 0)):
        with pytest.raises(ValueError, match="out of range"):
            f()


# ------------------------------------------------------------------ the oracle's pins

def test_oracle_agrees_with_the_c_oracle():
    import oracle
    rng = np.random.default_rng(0)
    B, T, h, h_kv, d = 2, 23, 4, 2, 8
    Q, K, V = (rng.standard_normal((B, T, n * d)) for n in (h, h_kv, h_kv))
    lens = [23, 11]
    a, A = lc.attention_window(Q, K, V, h, T, 0, h_kv, lens)
    ref = oracle.attention(Q, np.repeat(K.reshape(B, T, h_kv, d), 2, 2).reshape(B, T, -1),
                           np.repeat(V.reshape(B, T, h_kv, d), 2, 2).reshape(B, T, -1), h, causal=True, kv_lengths=lens)
    assert np.abs(a - ref).max() < 1e-12 and (A >= np.abs(a) - 1e-12).all()
    q = Q[:, :3]
    o, _, W = lc.decode(q, K, V, h, lens, h_kv, weights=np.zeros((B, h_kv, T)))
    assert np.abs(o - oracle.decode(q, K, V, h, lens, h_kv=h_kv)).max() < 1e-12
    assert np.allclose(W.sum(-1), h // h_kv * 3)             # every softmax row sums to 1
    # a prefix is a cache that starts earlier
    Kc, Vc = K[:, 5:], V[:, 5:]
    s, _, _ = lc.decode(q[:1], Kc[:1], Vc[:1], h, [18], h_kv, K_prefix=K[0, :5], V_prefix=V[0, :5])
    assert np.abs(s - o[:1]).max() < 1e-12
    # windows: brute force over the mask
    w, _ = lc.attention_window(Q, K, V, h, 4, 2, h_kv)
    i, j = np.arange(T)[:, None], np.arange(T)
    see = (j <= i) & ((i - j < 4) | (j < 2))
    x = np.where(see, Q[0, :, :d] @ K[0, :, :d].T / np.sqrt(d), -np.inf)
    e = np.exp(x - x.max(1, keepdims=True))
    assert np.abs(w[0, :, :d] - e / e.sum(1, keepdims=True) @ V[0, :, :d]).max() < 1e-12
    last, _, _ = lc.decode(Q[:, -1:], K, V, h, [T, T], h_kv, 4, 2)
    assert np.abs(last - w[:, -1:]).max() < 1e-12


def test_oracle_evict():
    w = np.array([[[3.0, 1.0, np.nan, 3.0, 2.0, 9.0, 9.0]]])
    assert lc.evict(w, [7], 4, 2) == [[[0, 3, 5, 6]]]
    assert lc.evict(w, [7], 7, 2) == [[list(range(7))]]
    assert lc.evict(w, [6], 5, 1) == [[[0, 1, 3, 4, 5]]]
    assert lc.evict(w, [5], 1, 0) == [[[0]]]
    assert lc.evict(w, [8], 1, 0) == [[None]]


# ------------------------------------------------------------------ workspaces

def test_set_workspace_on_refusals(handles):
    def call(h="bf", ptr=FAKE, n=4096, stream=None):
        return L.mha_set_workspace_on(None if h is None else handles[h], ptr, n, stream, check=False)
    for kw in (dict(h=None), dict(ptr=FAKE + 128), dict(n=255), dict(n=0)):
        assert call(**kw) == L.MHA_ERR_INVALID_ARG, kw
    assert call(ptr=None, n=0) == L.MHA_OK                   # detaches
    for mode in (-1, 3):
        with pytest.raises(L.MhaError, match="invalid argument"):
            L.mha_exchange_capture_mode(mode)


class _Side:
    """A stream that knows of no GPU."""
    def __init__(self, number, current, log):
        self.cuda_stream, self.current, self.log = number, current, log

    def __enter__(self):
        self.before, self.current[0] = self.current[0], self.cuda_stream

    def __exit__(self, *a):
        self.current[0] = self.before

    def synchronize(self):
        self.log.append("waited")


def test_workspace_is_zeroed_in_the_order_of_the_calls_stream(lib, monkeypatch):
    """The status block holds the cache steps' counters: its zeros have to come before the call that follows
    the attach, which on another stream they need not.  Under capture they must not wait for the replays."""
    torch = pytest.importorskip("torch")
    from transformer_head_scaled_02_gb300 import Mha, mha
    calls, captured, current, given = [], set(), [55], iter([55, 56, 77])
    monkeypatch.setattr(mha, "_stream", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: current[0] in captured)
    monkeypatch.setattr(torch.cuda, "Stream", lambda: _Side(next(given), current, calls))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    monkeypatch.setattr(L, "mha_set_workspace", lambda *a: calls.append(("unordered",)))
    monkeypatch.setattr(L, "mha_set_workspace_on", lambda h, p, n, stream: calls.append((p, n, stream)), raising=False)
    monkeypatch.setattr(L, "mha_exchange_capture_mode", lambda m: calls.append(m) or 7, raising=False)
    layer = Mha(256, 4, 64, dtype=torch.bfloat16, device="cpu")

    def ensure(need, capturing=False):
        captured.clear()
        captured.update((55, 56) if capturing else ())       # torch may give out streams of the capture
        ws, n = layer._ws, len(calls)
        got = layer.ensure_workspace(1, 1, 1, need=need)
        assert got.numel() >= need and got is layer._ws
        if got is ws:
            assert len(calls) == n
        elif capturing:
            assert calls[n:] == [L.CAPTURE_RELAXED, (got.data_ptr(), got.numel(), 77), "waited", 7]
        else:
            assert calls[n:] == [(got.data_ptr(), got.numel(), 55)]
        return got
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: None)
    a = ensure(1000)
    assert ensure(500) is a and ensure(1000, True) is a      # captured: outlives its replacement
    b = ensure(5000)
    assert b is not a and layer._kept_ws == [a]
    c = ensure(9000, True)
    assert ensure(9000, True) is c and ensure(9000) is c     # eager calls may share it
    d = ensure(20000)
    assert d is not c and any(x is c for x in layer._kept_ws)


def test_workspace_used_on_another_stream_is_recorded_there(lib, monkeypatch):
    """Its memory must not go to another owner while calls on that stream are under way."""
    torch = pytest.importorskip("torch")
    from transformer_head_scaled_02_gb300 import Mha, mha
    now, recorded = [1], []
    monkeypatch.setattr(mha, "_stream", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: now[0])
    monkeypatch.setattr(L, "mha_set_workspace_on", lambda *a: 0)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)), raising=False)
    layer = Mha(256, 4, 64, dtype=torch.bfloat16, device="cpu")
    a = layer.ensure_workspace(1, 1, 1, need=1000).data_ptr()
    for now[0] in (1, 2, 1, 2, 3):
        layer.ensure_workspace(1, 1, 1, need=1000)
    assert recorded == [(a, 2), (a, 3)]
    old = layer._ws                                          # (keeps its address from being given out again)
    layer.ensure_workspace(1, 1, 1, need=5000)               # on 3: its own
    now[0] = 1
    layer.ensure_workspace(1, 1, 1, need=5000)
    assert recorded[2:] == [(layer._ws.data_ptr(), 1)] and old is not layer._ws


def test_remembered_workspace_sizes_are_bounded(lib):
    torch = pytest.importorskip("torch")
    from transformer_head_scaled_02_gb300 import Mha
    layer = Mha(256, 4, 64, dtype=torch.bfloat16, h_kv=2, device="cpu")
    for again in range(2):
        for Tp in range(1000):
            assert layer._step_need(3, 1, 64 * Tp, 500, 0) == L.mha_cache_step_workspace_size(layer.handle, 3, 1, 64 * Tp, 500, 0)
    assert len(layer._step_bytes) <= 64
