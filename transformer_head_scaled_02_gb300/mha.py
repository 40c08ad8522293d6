"""Torch-tensor front end of libmha.so.

torch supplies device memory and the current CUDA stream; every step of the
forward runs in the library's kernels.  This module only checks tensor
properties, allocates the caller-side buffers (output and workspace) and
passes raw pointers through the C ABI (see ``_lib``).
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib

_DTYPES = {torch.float32: _lib.MHA_F32, torch.bfloat16: _lib.MHA_BF16}


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream() -> int:
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


class Mha:
    """One multi-head attention layer shape: width D, h heads of d_k / d_v.

    ``forward`` computes MultiHead(X_q, X_kv) = Concat(head_1..head_h) W_o + b_o
    with head_i = softmax(Q_i K_i^T / sqrt(d_k) [+ mask]) V_i, the fused
    [Q|K|V] projection X W_qkv + b_qkv feeding it (itwiki.kr "멀티 헤드 어텐션",
    수식 and the tensor-shape table).  Variants (same page, 추론 비용과 변형):
    ``h_kv`` K/V heads shared by groups of query heads (MQA/GQA), ``gated`` sigmoid
    output gate (a fourth projection block [Q|K|V|G]); ``forward(residual=...)`` adds
    a residual in the output projection; ``decode`` attends new tokens to a KV cache.
    """

    def __init__(self, D: int, h: int, d_k: int, d_v: Optional[int] = None,
                 dtype: torch.dtype = torch.bfloat16, device=None, h_kv: Optional[int] = None,
                 gated: bool = False):
        if dtype not in _DTYPES:
            raise TypeError(f"dtype must be one of {list(_DTYPES)}")
        self.D, self.h, self.d_k = D, h, d_k
        self.d_v = d_k if d_v is None else d_v
        self.h_kv = h if h_kv is None else h_kv
        self.gated = bool(gated)
        self.dtype = dtype
        self.device = torch.device("cuda") if device is None else torch.device(device)
        self.handle = _lib.mha_create_ex(D, h, self.h_kv, d_k, self.d_v, int(self.gated),
                                         _DTYPES[dtype])
        self._ws: Optional[torch.Tensor] = None
        self._ws_captured = False
        self._ws_streams: set = set()  # streams that the allocator knows to use the workspace
        self._kept_ws: list = []
        self._step_bytes: dict = {}  # workspace bytes of the cache steps, by their sizes

    @property
    def proj_width(self) -> int:
        """Columns of the fused projection [Q | K | V (| G)]."""
        return (self.h * self.d_k + self.h_kv * (self.d_k + self.d_v)
                + (self.h * self.d_v if self.gated else 0))

    def __del__(self):
        h = getattr(self, "handle", None)
        if h:
            _lib.mha_destroy(h)
            self.handle = None

    # ------------------------------------------------------------ workspace
    def workspace_size(self, B: int, T_q: int, T_kv: int) -> int:
        return _lib.mha_workspace_size(self.handle, B, T_q, T_kv)

    def ensure_workspace(self, B: int, T_q: int, T_kv: int, need: Optional[int] = None) -> torch.Tensor:
        need = self.workspace_size(B, T_q, T_kv) if need is None else need
        capturing = torch.cuda.is_current_stream_capturing()
        if self._ws is None or self._ws.numel() < need:
            if self._ws_captured:  # a captured graph still launches into the one it was captured with
                self._kept_ws.append(self._ws)
                self._ws_captured = False
            self._ws, home = (self._new_workspace_in_capture if capturing else self._new_workspace)(max(need, 256))
            self._ws_streams = {home}
        if capturing:
            self._ws_captured = True
        elif _stream() not in self._ws_streams:
            # calls on this stream may still be under way when a larger workspace replaces it
            self._ws.record_stream(torch.cuda.current_stream())
            self._ws_streams.add(_stream())
        return self._ws

    def _new_workspace(self, nbytes: int):
        """A workspace, attached, and the stream it belongs to: the current one, in whose order its status
        block (with the counters of the cache steps) is zeroed, as the memory comes from there and the call
        goes there."""
        ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        _lib.mha_set_workspace_on(self.handle, ws.data_ptr(), nbytes, _stream())
        return ws, _stream()

    def _new_workspace_in_capture(self, nbytes: int):
        """The same while a graph is being captured: neither the memory nor the zeros may be the graph's.  It
        writes its temporaries over memory of its own at every replay, and eager calls may come before the
        first.  So both come from another stream, and the zeros are waited for."""
        mode = _lib.mha_exchange_capture_mode(_lib.CAPTURE_RELAXED)
        try:
            while True:  # torch gives out a few streams in turn, those under capture among them
                side = torch.cuda.Stream()
                with torch.cuda.stream(side):
                    if torch.cuda.is_current_stream_capturing():
                        continue
                    ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
                    _lib.mha_set_workspace_on(self.handle, ws.data_ptr(), nbytes, side.cuda_stream)
                break
            side.synchronize()
        finally:
            _lib.mha_exchange_capture_mode(mode)
        return ws, side.cuda_stream

    def _hold_status(self) -> None:
        """For calls that use an attached workspace for its status word alone: it has to outlive them, and the
        graphs that they are captured in, too."""
        if self._ws is not None:
            self.ensure_workspace(0, 0, 0, need=256)

    def status(self) -> int:
        """Read and clear the device status word, and reset what a step that timed out may have left in
        the workspace's counters (synchronises the current stream)."""
        return _lib.mha_get_status(self.handle, _stream())

    # ------------------------------------------------------------ checks
    def _check(self, name, t, shape=None):
        if t is None:
            return
        if not t.is_cuda or t.dtype != self.dtype or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {self.dtype} CUDA tensor")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")

    # ------------------------------------------------------------ the layer
    def forward(self, X_q: torch.Tensor, W_qkv: torch.Tensor, b_qkv: Optional[torch.Tensor],
                W_o: torch.Tensor, b_o: Optional[torch.Tensor], X_kv: Optional[torch.Tensor] = None,
                causal: bool = False, kv_lengths: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None,
                residual: Optional[torch.Tensor] = None, window: Optional[int] = None,
                sinks: int = 0) -> torch.Tensor:
        """The whole layer.  With ``window`` (self-attention, causal=True): row i sees only the last
        ``window`` keys and the first ``sinks`` of its sequence (see attention_window)."""
        B, T_q, D = X_q.shape
        T_kv = T_q if X_kv is None else X_kv.shape[1]
        if window is None and sinks:
            raise ValueError("sinks need a window")
        if window is not None and (X_kv is not None or not causal):
            raise ValueError("a window needs causal self-attention")
        if window is not None:
            self._int32("window", window, 1)
            self._int32("sinks", sinks, 0)
        ncols = self.proj_width
        self._check("X_q", X_q, (B, T_q, self.D))
        self._check("X_kv", X_kv, None if X_kv is None else (B, T_kv, self.D))
        self._check("W_qkv", W_qkv, (self.D, ncols))
        self._check("b_qkv", b_qkv, None if b_qkv is None else (ncols,))
        self._check("W_o", W_o, (self.h * self.d_v, self.D))
        self._check("b_o", b_o, None if b_o is None else (self.D,))
        if kv_lengths is not None and (kv_lengths.dtype != torch.int32 or not kv_lengths.is_cuda
                                       or kv_lengths.numel() != B):
            raise ValueError("kv_lengths must be a CUDA int32 tensor of length B")
        if out is None:
            out = torch.empty((B, T_q, self.D), dtype=self.dtype, device=X_q.device)
        self._check("out", out, (B, T_q, self.D))
        self._check("residual", residual, None if residual is None else (B, T_q, self.D))
        self.ensure_workspace(B, T_q, T_kv)
        if window is not None:
            _lib.mha_forward_window(self.handle, _ptr(X_q), B, T_q, _ptr(W_qkv), _ptr(b_qkv), _ptr(W_o),
                                    _ptr(b_o), window, sinks, _ptr(kv_lengths), _ptr(residual),
                                    _ptr(out), _stream())
            return out
        _lib.mha_forward_ex(self.handle, _ptr(X_q), _ptr(X_kv), B, T_q, T_kv, _ptr(W_qkv),
                            _ptr(b_qkv), _ptr(W_o), _ptr(b_o), causal, _ptr(kv_lengths),
                            _ptr(residual), _ptr(out), _stream())
        return out

    __call__ = forward

    def forward_host(self, X_q: torch.Tensor, W_qkv: torch.Tensor, b_qkv: Optional[torch.Tensor],
                     W_o: torch.Tensor, b_o: Optional[torch.Tensor], out: torch.Tensor,
                     X_kv: Optional[torch.Tensor] = None, causal: bool = False,
                     kv_lengths: Optional[torch.Tensor] = None,
                     residual: Optional[torch.Tensor] = None, chunks: int = 4) -> torch.Tensor:
        """forward() with X_q, X_kv, residual and out in (pinned) host memory and the weights on
        the device: the batch goes through in chunks whose copies overlap the kernels.  Enqueued
        on the current stream; synchronise it before reading ``out``."""
        B, T_q, D = X_q.shape
        T_kv = T_q if X_kv is None else X_kv.shape[1]
        for name, t, T in (("X_q", X_q, T_q), ("X_kv", X_kv, T_kv), ("residual", residual, T_q),
                           ("out", out, T_q)):
            if t is None:
                continue
            if t.is_cuda or t.dtype != self.dtype or not t.is_contiguous() or tuple(t.shape) != (B, T, self.D):
                raise ValueError(f"{name} must be a contiguous host {self.dtype} tensor of shape "
                                 f"{(B, T, self.D)}")
        self._check("W_qkv", W_qkv, (self.D, self.proj_width))
        self._check("b_qkv", b_qkv, None if b_qkv is None else (self.proj_width,))
        self._check("W_o", W_o, (self.h * self.d_v, self.D))
        self._check("b_o", b_o, None if b_o is None else (self.D,))
        if kv_lengths is not None and (kv_lengths.dtype != torch.int32 or not kv_lengths.is_cuda
                                       or kv_lengths.numel() != B):
            raise ValueError("kv_lengths must be a CUDA int32 tensor of length B")
        need = _lib.mha_forward_host_workspace_size(self.handle, B, T_q, T_kv, chunks)
        if need == 0:
            raise ValueError("invalid size or chunk count")
        self.ensure_workspace(B, T_q, T_kv, need=need)
        _lib.mha_forward_host(self.handle, _ptr(X_q), _ptr(X_kv), B, T_q, T_kv, _ptr(W_qkv),
                              _ptr(b_qkv), _ptr(W_o), _ptr(b_o), causal, _ptr(kv_lengths),
                              _ptr(residual), _ptr(out), chunks, _stream())
        return out

    # ------------------------------------------------------------ single steps
    def linear(self, A: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None,
               residual: Optional[torch.Tensor] = None) -> torch.Tensor:
        """C = A W + bias (+ residual) for 2-D A (M, K), W (K, N), residual (M, N) (row strides
        may exceed the width)."""
        M, K = A.shape
        N = W.shape[1]
        if out is None:
            out = torch.empty((M, N), dtype=self.dtype, device=A.device)
        mats = [("A", A), ("W", W), ("out", out)] + ([("residual", residual)] if residual is not None else [])
        for name, t in mats:
            if not t.is_cuda or t.dtype != self.dtype or t.stride(1) != 1:
                raise ValueError(f"{name} must be a row-major {self.dtype} CUDA matrix")
        self._check("bias", bias, None if bias is None else (N,))
        self._hold_status()
        _lib.mha_linear_ex(self.handle, _ptr(A), A.stride(0), M, K, _ptr(W), W.stride(0), N,
                           _ptr(bias), _ptr(residual), 0 if residual is None else residual.stride(0),
                           _ptr(out), out.stride(0), _stream())
        return out

    def linear_segments(self, A: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor],
                        seg_len: torch.Tensor, seg_rows: int,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """C = A W + bias where only the rows that whole 128-row tiles up to each segment's
        length need are guaranteed: the key/value projection of cross-attention with key
        lengths seg_len (CUDA int32, one per segment of seg_rows rows)."""
        M, K = A.shape
        N = W.shape[1]
        if out is None:
            out = torch.empty((M, N), dtype=self.dtype, device=A.device)
        for name, t in (("A", A), ("W", W), ("out", out)):
            if not t.is_cuda or t.dtype != self.dtype or t.stride(1) != 1:
                raise ValueError(f"{name} must be a row-major {self.dtype} CUDA matrix")
        self._check("bias", bias, None if bias is None else (N,))
        if seg_len.dtype != torch.int32 or not seg_len.is_cuda:
            raise ValueError("seg_len must be a CUDA int32 tensor")
        self._hold_status()
        _lib.mha_linear_segments(self.handle, _ptr(A), A.stride(0), M, K, _ptr(W), W.stride(0), N,
                                 _ptr(bias), _ptr(seg_len), seg_rows, _ptr(out), out.stride(0),
                                 _stream())
        return out

    def linear_pair(self, A: torch.Tensor, W: torch.Tensor, bias: Optional[torch.Tensor],
                    A2: torch.Tensor, W2: torch.Tensor, bias2: Optional[torch.Tensor],
                    seg_len: Optional[torch.Tensor] = None, seg_rows: int = 0,
                    out: Optional[torch.Tensor] = None,
                    out2: Optional[torch.Tensor] = None):
        """(A W + bias, A2 W2 + bias2) in one launch where possible (the cross-attention key /
        value and query projections); with seg_len, rows of the first past each segment's
        length may be left unwritten as in linear_segments.  Returns (out, out2)."""
        M, K = A.shape
        M2, K2 = A2.shape
        N, N2 = W.shape[1], W2.shape[1]
        if K2 != K or W.shape[0] != K or W2.shape[0] != K:
            raise ValueError("both projections need the same inner dimension")
        if out is None:
            out = torch.empty((M, N), dtype=self.dtype, device=A.device)
        if out2 is None:
            out2 = torch.empty((M2, N2), dtype=self.dtype, device=A.device)
        for name, t in (("A", A), ("W", W), ("out", out), ("A2", A2), ("W2", W2), ("out2", out2)):
            if not t.is_cuda or t.dtype != self.dtype or t.stride(1) != 1:
                raise ValueError(f"{name} must be a row-major {self.dtype} CUDA matrix")
        self._check("bias", bias, None if bias is None else (N,))
        self._check("bias2", bias2, None if bias2 is None else (N2,))
        if seg_len is not None and (seg_len.dtype != torch.int32 or not seg_len.is_cuda):
            raise ValueError("seg_len must be a CUDA int32 tensor")
        self._hold_status()
        _lib.mha_linear_pair(self.handle, _ptr(A), A.stride(0), M, _ptr(W), W.stride(0), N, _ptr(bias),
                             _ptr(seg_len), seg_rows, _ptr(out), out.stride(0), _ptr(A2), A2.stride(0),
                             M2, _ptr(W2), W2.stride(0), N2, _ptr(bias2), _ptr(out2), out2.stride(0), K,
                             _stream())
        return out, out2

    def attention(self, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, causal: bool = False,
                  kv_lengths: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None,
                  G: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Attention of all heads over (B, T, width) views whose last dim is contiguous;
        head i uses columns [i*d, (i+1)*d) of Q (and of the gate pre-activations G), K/V
        head i // (h // h_kv).  Returns Ocat (B, T_q, h*d_v)."""
        B, T_q, _ = Q.shape
        T_kv = K.shape[1]
        views = [("Q", Q), ("K", K), ("V", V)] + ([("G", G)] if G is not None else [])
        for name, t in views:
            if not t.is_cuda or t.dtype != self.dtype or t.stride(2) != 1 \
                    or t.stride(0) != t.shape[1] * t.stride(1):
                raise ValueError(f"{name} must be a (B,T,*) {self.dtype} CUDA view with "
                                 "contiguous rows and batches")
        if out is None:
            out = torch.empty((B, T_q, self.h * self.d_v), dtype=self.dtype, device=Q.device)
        if kv_lengths is not None and (kv_lengths.dtype != torch.int32 or not kv_lengths.is_cuda):
            raise ValueError("kv_lengths must be a CUDA int32 tensor")
        self._hold_status()
        _lib.mha_attention_ex(self.handle, B, T_q, T_kv, _ptr(Q), Q.stride(1), _ptr(K), K.stride(1),
                              _ptr(V), V.stride(1), _ptr(G), 0 if G is None else G.stride(1), causal,
                              _ptr(kv_lengths), _ptr(out), out.stride(1), _stream())
        return out

    def decode(self, Q: torch.Tensor, K_cache: torch.Tensor, V_cache: torch.Tensor,
               cache_lengths: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """One decode step: the T_q new tokens' queries Q (B, T_q, h*d_k view) over the cache
        K_cache (B, T_max, h_kv*d_k view), V_cache (B, T_max, h_kv*d_v view); cache_lengths
        (int32, B) count the cached tokens including the new ones.  Returns (B, T_q, h*d_v)."""
        B, T_q, _ = Q.shape
        T_max = K_cache.shape[1]
        for name, t in (("Q", Q), ("K_cache", K_cache), ("V_cache", V_cache)):
            if not t.is_cuda or t.dtype != self.dtype or t.stride(2) != 1 \
                    or t.stride(0) != t.shape[1] * t.stride(1):
                raise ValueError(f"{name} must be a (B,T,*) {self.dtype} CUDA view with "
                                 "contiguous rows and batches")
        if cache_lengths.dtype != torch.int32 or not cache_lengths.is_cuda or cache_lengths.numel() != B:
            raise ValueError("cache_lengths must be a CUDA int32 tensor of length B")
        if out is None:
            out = torch.empty((B, T_q, self.h * self.d_v), dtype=self.dtype, device=Q.device)
        self.ensure_workspace(B, T_q, T_max,
                              need=_lib.mha_decode_workspace_size(self.handle, B, T_q, T_max))
        _lib.mha_decode(self.handle, B, T_q, T_max, _ptr(Q), Q.stride(1), _ptr(K_cache),
                        K_cache.stride(1), _ptr(V_cache), V_cache.stride(1), _ptr(cache_lengths),
                        _ptr(out), out.stride(1), _stream())
        return out

    # ------------------------------------------------------------ long contexts
    def _rows(self, name: str, t: torch.Tensor, B: int, T: int, width: int) -> int:
        """Check a (B, T, width) view whose rows lie one stride apart throughout; returns the stride."""
        if t.shape != (B, T, width):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(B, T, width)}")
        s0, s1, s2 = t.stride()
        if t.dtype != self.dtype or s2 != 1 or (B > 1 and T > 1 and s0 != T * s1):
            raise ValueError(f"{name} must be a (B,T,*) {self.dtype} view with contiguous rows and "
                             "batches")
        if B * T > 1:
            return s0 if T == 1 else s1
        return max(s1, width)  # one row (or none): any stride of at least a row will do

    def _prefix(self, name: str, t: torch.Tensor, T: int, width: int) -> int:
        """_rows for the (T, width) view of a shared prefix."""
        if t.shape != (T, width):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(T, width)}")
        s0, s1 = t.stride()
        if t.dtype != self.dtype or s1 != 1:
            raise ValueError(f"{name} must be a (T,*) {self.dtype} view with contiguous rows")
        return s0 if T > 1 else max(s0, width)

    @staticmethod
    def _device(first: torch.Tensor, *others: Optional[torch.Tensor]) -> int:
        """All on one CUDA device, the current one; returns its current stream."""
        dev = first.get_device()
        if dev < 0:
            raise ValueError("the tensors must be on a CUDA device")
        for t in others:
            if t is not None and t.get_device() != dev:
                raise ValueError("all tensors must be on one CUDA device")
        if dev != torch._C._cuda_getDevice():
            raise ValueError(f"the tensors are on cuda:{dev}, which is not the current device")
        return torch._C._cuda_getCurrentRawStream(dev)

    @staticmethod
    def _int32(name: str, x: int, least: int) -> int:
        """A size as a C int (ctypes would cut it to 32 bits)."""
        if not least <= x <= 0x7FFFFFFF:
            raise ValueError(f"{name} = {x} is out of range")
        return x

    @staticmethod
    def _ints(name: str, t: torch.Tensor, B: int) -> int:
        if t.dtype != torch.int32 or t.shape != (B,) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA int32 tensor of length {B}")
        return t.data_ptr()

    @staticmethod
    def _weights(name: str, t: torch.Tensor, shape) -> int:
        if t.dtype != torch.float32 or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA float32 tensor of shape {shape}")
        return t.data_ptr()

    def attention_window(self, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, window: int,
                         sinks: int = 0, kv_lengths: Optional[torch.Tensor] = None,
                         out: Optional[torch.Tensor] = None,
                         G: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Causal sliding-window attention over (B, T, width) views: row i sees key j iff j <= i,
        j < L_b and (i - j < window or j < sinks); rows that see nothing (padding only) are zero.
        Heads, gate and views as in attention().  Returns Ocat (B, T, h*d_v)."""
        B, T, _ = Q.shape
        self._int32("window", window, 1)
        self._int32("sinks", sinks, 0)
        ldq = self._rows("Q", Q, B, T, self.h * self.d_k)
        ldk = self._rows("K", K, B, T, self.h_kv * self.d_k)
        ldv = self._rows("V", V, B, T, self.h_kv * self.d_v)
        if out is None:
            out = torch.empty((B, T, self.h * self.d_v), dtype=self.dtype, device=Q.device)
        ldo = self._rows("out", out, B, T, self.h * self.d_v)
        ldg = 0 if G is None else self._rows("G", G, B, T, self.h * self.d_v)
        lens = None if kv_lengths is None else self._ints("kv_lengths", kv_lengths, B)
        stream = self._device(Q, K, V, out, G, kv_lengths)
        self._hold_status()
        _lib.mha_attention_window(self.handle, B, T, Q.data_ptr(), ldq, K.data_ptr(), ldk, V.data_ptr(),
                                  ldv, _ptr(G), ldg, window, sinks, lens, out.data_ptr(), ldo, stream)
        return out

    def _step_need(self, *sizes: int) -> int:
        """mha_cache_step_workspace_size, remembered for the sizes at hand."""
        need = self._step_bytes.get(sizes)
        if need is None:
            if len(self._step_bytes) >= 64:  # (a prefix length that varies would fill it without end)
                self._step_bytes.clear()
            need = self._step_bytes[sizes] = _lib.mha_cache_step_workspace_size(self.handle, *sizes)
        return need

    def _cache_step(self, Q, K_cache, V_cache, cache_lengths, out, T_prefix, weights, *others):
        """Checks and workspace that the cache steps share: (out, the arguments they have in common)."""
        B, T_q, _ = Q.shape
        T_max = K_cache.shape[1]
        ldq = self._rows("Q", Q, B, T_q, self.h * self.d_k)
        ldk = self._rows("K_cache", K_cache, B, T_max, self.h_kv * self.d_k)
        ldv = self._rows("V_cache", V_cache, B, T_max, self.h_kv * self.d_v)
        if out is None:
            out = torch.empty((B, T_q, self.h * self.d_v), dtype=self.dtype, device=Q.device)
        ldo = self._rows("out", out, B, T_q, self.h * self.d_v)
        lens = self._ints("cache_lengths", cache_lengths, B)
        stream = self._device(Q, K_cache, V_cache, cache_lengths, out, *others)
        need = self._step_need(B, T_q, T_prefix, T_max, weights)
        self.ensure_workspace(B, T_q, T_max, need=need)
        cache = (Q.data_ptr(), ldq, K_cache.data_ptr(), ldk, V_cache.data_ptr(), ldv)
        return out, (B, T_q, T_max), cache, lens, (out.data_ptr(), ldo, stream)

    def decode_window(self, Q: torch.Tensor, K_cache: torch.Tensor, V_cache: torch.Tensor,
                      cache_lengths: torch.Tensor, window: int, sinks: int = 0,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """decode() under a sliding window: the new token at position p of its cache sees keys j <= p
        with p - j < window or j < sinks, and only those are read."""
        self._int32("window", window, 1)
        self._int32("sinks", sinks, 0)
        out, sizes, cache, lens, tail = self._cache_step(Q, K_cache, V_cache, cache_lengths, out, 0, 0)
        _lib.mha_decode_window(self.handle, *sizes, *cache, window, sinks, lens, *tail)
        return out

    def decode_shared(self, Q: torch.Tensor, K_prefix: torch.Tensor, V_prefix: torch.Tensor,
                      K_cache: torch.Tensor, V_cache: torch.Tensor, cache_lengths: torch.Tensor,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """One decode step of a batch that shares its first tokens: K_prefix (T_prefix, h_kv*d_k view)
        and V_prefix (T_prefix, h_kv*d_v view) are stored and read once for the whole batch; the
        caches and cache_lengths hold each sequence's own tokens after them, the new ones included."""
        T_p = K_prefix.shape[0]
        ldkp = self._prefix("K_prefix", K_prefix, T_p, self.h_kv * self.d_k)
        ldvp = self._prefix("V_prefix", V_prefix, T_p, self.h_kv * self.d_v)
        out, (B, T_q, T_max), cache, lens, tail = self._cache_step(
            Q, K_cache, V_cache, cache_lengths, out, T_p, 0, K_prefix, V_prefix)
        _lib.mha_decode_shared(self.handle, B, T_q, T_p, K_prefix.data_ptr(), ldkp, V_prefix.data_ptr(),
                               ldvp, T_max, *cache, lens, *tail)
        return out

    def decode_weights(self, Q: torch.Tensor, K_cache: torch.Tensor, V_cache: torch.Tensor,
                       cache_lengths: torch.Tensor, weights: torch.Tensor,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """decode() that also adds, to ``weights`` (float32 (B, h_kv, T_max)), the softmax weight each
        cached token receives from the step, summed over its group's query heads and the new tokens;
        the new tokens' own entries are written, not added to."""
        w = self._weights("weights", weights, (Q.shape[0], self.h_kv, K_cache.shape[1]))
        out, sizes, cache, lens, tail = self._cache_step(Q, K_cache, V_cache, cache_lengths, out, 0, 1,
                                                         weights)
        _lib.mha_decode_weights(self.handle, *sizes, *cache, lens, w, *tail)
        return out

    def evict(self, K_cache: torch.Tensor, V_cache: torch.Tensor, cache_lengths: torch.Tensor,
              weights: torch.Tensor, keep: int, recent: int, K_out: Optional[torch.Tensor] = None,
              V_out: Optional[torch.Tensor] = None, weights_out: Optional[torch.Tensor] = None,
              lengths_out: Optional[torch.Tensor] = None):
        """Cut every sequence to at most ``keep`` tokens per K/V head: the last ``recent`` and the
        earlier ones of largest ``weights`` (decode_weights accumulates them), in their order.  The
        outputs may be new buffers of T_out >= keep rows (the default: exactly keep, rows past the new
        length unset) or, all three, the inputs themselves (in place).  Returns (K_out, V_out,
        lengths_out, weights_out, kept): kept (int32 (B, h_kv, keep)) holds the kept tokens' indices,
        then -1."""
        B, T_max, _ = K_cache.shape
        wk, wv = self.h_kv * self.d_k, self.h_kv * self.d_v
        ldk = self._rows("K_cache", K_cache, B, T_max, wk)
        ldv = self._rows("V_cache", V_cache, B, T_max, wv)
        w = self._weights("weights", weights, (B, self.h_kv, T_max))
        lens = self._ints("cache_lengths", cache_lengths, B)
        self._int32("keep", keep, 1)
        self._int32("recent", recent, 0)
        dev = K_cache.device
        T_out = keep if K_out is None else K_out.shape[1]
        if K_out is None:
            K_out = torch.empty((B, T_out, wk), dtype=self.dtype, device=dev)
        if V_out is None:
            V_out = torch.empty((B, T_out, wv), dtype=self.dtype, device=dev)
        if weights_out is None:
            weights_out = torch.empty((B, self.h_kv, T_out), dtype=torch.float32, device=dev)
        if lengths_out is None:
            lengths_out = torch.empty_like(cache_lengths)
        kept = cache_lengths.new_empty((B, self.h_kv, keep))
        ldko = self._rows("K_out", K_out, B, T_out, wk)
        ldvo = self._rows("V_out", V_out, B, T_out, wv)
        wo = self._weights("weights_out", weights_out, (B, self.h_kv, T_out))
        lo = self._ints("lengths_out", lengths_out, B)
        stream = self._device(K_cache, V_cache, cache_lengths, weights, K_out, V_out, weights_out, lengths_out)
        self.ensure_workspace(0, 0, 0, need=256)  # the status word
        _lib.mha_cache_evict(self.handle, B, T_max, keep, recent, K_cache.data_ptr(), ldk,
                             V_cache.data_ptr(), ldv, lens, w, T_out, K_out.data_ptr(), ldko,
                             V_out.data_ptr(), ldvo, wo, kept.data_ptr(), lo, stream)
        return K_out, V_out, lengths_out, weights_out, kept
