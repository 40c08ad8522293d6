"""Measured cases of the long-context serving operators: sliding-window attention with sinks
(whole sequences and decode steps), the decode step of a batch that shares a prefix, the decode
step that accumulates attention weights, and the eviction that goes by them.

``own`` chooses between the operators' plain form (elementary torch operations in 32 bits, rounded
once at the end) and the calls a user makes of the package.  ``exact`` states the definitions in 64
bits, one sequence at a time.

Formulas (query head i reads K/V head i // (h // h_kv); s = q . k / sqrt(d)):
  window   row i sees key j iff j <= i, j < L_b and (i - j < window or j < sinks);
           o_i = sum_j softmax_j(s_ij) v_j, zeros where nothing is visible; times sigmoid(G) if gated
  decode   new token t of T_q sits at p = L_b - T_q + t of its cache and sees keys j <= p
           (decode_window: and (p - j < window or j < sinks))
  shared   every row sees the whole prefix and, of its own cache, keys j <= p
  weights  w[b, g, j] (+)= sum over the group's query heads and new tokens of softmax_j, the new
           tokens' own entries starting at zero
  evict    per (b, g) with L_b > keep: the last `recent` tokens and the keep - recent earlier ones of
           largest weight (ties: lowest index), in their order; all L_b tokens otherwise
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_OPS = ("window", "decode_window", "shared", "weights", "evict")


def _case(name, op, dtype="bf16", B=1, Tq=1, T=1024, h=16, hkv=16, d=64, window=0, sinks=0, prefix=0,
          keep=0, recent=0, ragged=False, gated=False):
    c = {"op": op, "dtype": dtype, "B": B, "Tq": Tq, "T": T, "h": h, "hkv": hkv, "d": d, "window": window,
         "sinks": sinks, "prefix": prefix, "keep": keep, "recent": recent, "ragged": ragged, "gated": gated}
    return dict(c, name=name) if name else c


def listed():
    return [
        # prompt of the bf16 causal layer (B = 4, T = 2048, d = 64) with grouped heads, short window
        _case("window_prompt", "window", B=4, T=2048, h=16, hkv=4, d=64, window=256, sinks=4),
        # the long-sequence layer (T = 16384, d = 128) under a window of an eighth of it
        _case("window_long", "window", B=1, T=16384, h=16, hkv=16, d=128, window=2048, sinks=16),
        # fp32 layer, ragged padded batch, odd length, no sinks, gated
        _case("window_ragged_f32", "window", "f32", B=8, T=1001, h=8, hkv=2, d=64, window=128, ragged=True,
              gated=True),
        # one user's next token: latency
        _case("decode_window_one", "decode_window", B=1, T=4096, h=16, hkv=4, d=64, window=1000, sinks=4),
        # the decode benchmark's batch and cache (32 x 8192, d = 128), half of it inside the window
        _case("decode_window_batch", "decode_window", B=32, T=8192, h=16, hkv=16, d=128, window=4096, sinks=4,
              ragged=True),
        # fp32, a few new tokens at once (speculative decoding), odd sizes
        _case("decode_window_tokens_f32", "decode_window", "f32", B=3, Tq=5, T=2000, h=8, hkv=4, d=64, window=300,
              sinks=10, ragged=True),
        # a handful of users behind one system prompt
        _case("shared_few", "shared", B=8, T=256, h=16, hkv=16, d=64, prefix=1000, ragged=True),
        # many samples of one long prompt
        _case("shared_many", "shared", B=64, T=1024, h=16, hkv=4, d=128, prefix=32768, ragged=True),
        # fp32, short caches
        _case("weights_few_f32", "weights", "f32", B=2, T=1024, h=8, hkv=8, d=64, ragged=True),
        # the decode benchmark's grouped-head cache
        _case("weights_batch", "weights", B=32, T=8192, h=16, hkv=4, d=128, ragged=True),
        # one small cache cut to a quarter
        _case("evict_few", "evict", B=2, T=1000, h=8, hkv=8, d=64, keep=250, recent=50),
        # the decode benchmark's batch, cut from about 8192 tokens to 2048
        _case("evict_batch", "evict", B=32, T=8192, h=16, hkv=16, d=128, keep=2048, recent=256, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(_OPS)
    dtype = rng.choice(("bf16", "bf16", "f32"))
    hkv = rng.choice((1, 2, 4, 8, 16))
    per = rng.choice([p for p in (1, 2, 4, 8) if p * hkv <= 16])
    d = rng.choice((64, 128)) if dtype == "bf16" else rng.choice((32, 64, 80, 128))
    c = dict(dtype=dtype, h=hkv * per, hkv=hkv, d=d, ragged=rng.random() < 0.7)
    if op == "window":
        T = _log_int(rng, 100, 8192 if dtype == "bf16" else 2048)
        B = _log_int(rng, 1, max(1, min(8, (1 << 25) // (T * T))))
        return _case(None, op, B=B, T=T, window=_log_int(rng, 16, T), sinks=rng.choice((0, 1, 4, 16, 130)),
                     gated=rng.random() < 0.3, **c)
    B = _log_int(rng, 1, 32)
    T = _log_int(rng, 128, 8192)
    Tq = rng.choice((1, 1, 1, 2, 5))
    if op == "decode_window":
        return _case(None, op, B=B, Tq=Tq, T=T, window=_log_int(rng, 16, T), sinks=rng.choice((0, 1, 4, 64, 130)), **c)
    if op == "shared":
        return _case(None, op, B=B, Tq=Tq, T=_log_int(rng, 16, 1024), prefix=_log_int(rng, 64, 32768), **c)
    if op == "weights":
        return _case(None, op, B=B, Tq=Tq, T=T, **c)
    keep = _log_int(rng, 16, T)
    return _case(None, op, B=B, T=T, keep=keep, recent=rng.randint(0, keep), **c)


def _lowest(c):
    """Least cached (or valid) length of a ragged batch."""
    return max(c["Tq"], c["T"] // 2)


def prepare(case, seed):
    c = dict(case)
    dt, dev = _DT[c["dtype"]], "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    B, T, Tq, h, hkv, d = c["B"], c["T"], c["Tq"], c["h"], c["hkv"], c["d"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    s = {"c": c}
    if c["ragged"]:
        s["len"] = torch.randint(_lowest(c), T + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    else:
        s["len"] = torch.full((B,), T, device=dev, dtype=torch.int32)
    if c["op"] == "window":
        # the projection's fused [Q | K | V (| G)] rows, read as column views
        width = (h + 2 * hkv) * d + (h * d if c["gated"] else 0)
        x = normal(B, T, width)
        s["Q"], s["K"], s["V"] = x[..., :h * d], x[..., h * d:(h + hkv) * d], x[..., (h + hkv) * d:(h + 2 * hkv) * d]
        s["G"] = x[..., (h + 2 * hkv) * d:] if c["gated"] else None
        s["out"] = torch.empty((B, T, h * d), device=dev, dtype=dt)
    else:
        s["K"], s["V"] = normal(B, T, hkv * d), normal(B, T, hkv * d)
        if c["op"] != "evict":
            s["Q"] = normal(B, Tq, h * d)
            s["out"] = torch.empty((B, Tq, h * d), device=dev, dtype=dt)
    if c["op"] == "shared":
        s["Kp"], s["Vp"] = normal(c["prefix"], hkv * d), normal(c["prefix"], hkv * d)
    if c["op"] in ("weights", "evict"):
        # weights that earlier steps left: a few heavy tokens, many light ones, some exactly zero
        w = torch.exp(2.0 * torch.randn((B, hkv, T), generator=g, device=dev)) / 64.0
        s["w"] = torch.where(w < 0.004, torch.zeros_like(w), w)
    if c["op"] == "evict":
        n = c["keep"]
        s["Ko"], s["Vo"] = torch.zeros((B, n, hkv * d), device=dev, dtype=dt), torch.zeros((B, n, hkv * d), device=dev, dtype=dt)
        s["wo"] = torch.zeros((B, hkv, n), device=dev)
    if own:
        from transformer_head_scaled_02_gb300 import Mha
        s["layer"] = Mha(h * d, h, d, d, dtype=dt, h_kv=hkv, gated=c["gated"])
    return s


# ------------------------------------------------------------------ the plain forms

def _softmax(x):
    """Weights of the last axis; rows without a visible entry (all -inf) weigh nothing."""
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def _grouped(x, n, d):
    """(B, T, n d) -> (B, n, T, d) in 32 bits."""
    return x.float().reshape(x.shape[0], x.shape[1], n, d).transpose(1, 2)


def _queries(s):
    """(B, h_kv, per T_q, d): the rows that share a K/V head."""
    c = s["c"]
    q = _grouped(s["Q"], c["h"], c["d"])
    return q.reshape(c["B"], c["hkv"], -1, c["d"])


def _merged(o, s):
    """(B, h_kv, per T_q, d) -> (B, T_q, h d) in the storage type."""
    c = s["c"]
    return o.reshape(c["B"], c["h"], -1, c["d"]).transpose(1, 2).reshape(c["B"], -1, c["h"] * c["d"]).to(_DT[c["dtype"]])


def _new_rows(c, length):
    """Position (B, per T_q) in its cache of each query row."""
    t = torch.arange(c["Tq"], device=length.device).repeat(c["h"] // c["hkv"])
    return length.long()[:, None] - c["Tq"] + t


def _plain_window(s):
    c = s["c"]
    T, per = c["T"], c["h"] // c["hkv"]
    q, k, v = _queries(s), _grouped(s["K"], c["hkv"], c["d"]), _grouped(s["V"], c["hkv"], c["d"])
    x = (q / math.sqrt(c["d"])) @ k.transpose(-1, -2)
    i, j = torch.arange(T, device=x.device)[:, None], torch.arange(T, device=x.device)
    seen = (j <= i) & ((i - j < c["window"]) | (j < c["sinks"]))
    seen = seen & (j < s["len"][:, None, None])
    x = x.reshape(c["B"], c["hkv"], per, T, T).masked_fill_(~seen[:, None, None], -math.inf)
    o = (_softmax(x).reshape(c["B"], c["hkv"], per * T, T) @ v)
    if c["gated"]:
        o = o / (1 + torch.exp(-_grouped(s["G"], c["h"], c["d"]).reshape(o.shape)))
    return _merged(o, s)


def _plain_decode_window(s):
    c = s["c"]
    L, W, S = s["len"].long(), c["window"], c["sinks"]
    n = min(c["T"], S + W + c["Tq"] - 1)
    p = torch.arange(n, device=L.device)
    first = (L - c["Tq"] - W + 1).clamp(min=S)[:, None]
    key = torch.where(p < S, p, first + p - S)                      # (B, n): sinks, then the window
    at = key.clamp(max=c["T"] - 1)[..., None].expand(-1, -1, c["hkv"] * c["d"])
    k, v = _grouped(s["K"].gather(1, at), c["hkv"], c["d"]), _grouped(s["V"].gather(1, at), c["hkv"], c["d"])
    x = (_queries(s) / math.sqrt(c["d"])) @ k.transpose(-1, -2)
    row = _new_rows(c, L)[..., None]
    seen = (key[:, None] <= row) & ((row - key[:, None] < W) | (key[:, None] < S))
    return _merged(_softmax(x.masked_fill(~seen[:, None], -math.inf)) @ v, s)


def _plain_shared(s):
    c = s["c"]
    q = _queries(s) / math.sqrt(c["d"])
    kp, vp = _grouped(s["Kp"][None], c["hkv"], c["d"]), _grouped(s["Vp"][None], c["hkv"], c["d"])
    k, v = _grouped(s["K"], c["hkv"], c["d"]), _grouped(s["V"], c["hkv"], c["d"])
    rows = q.shape[2]
    qa = q.transpose(0, 1).reshape(c["hkv"], c["B"] * rows, c["d"])  # all sequences' rows at once
    xp = (qa @ kp[0].transpose(-1, -2)).reshape(c["hkv"], c["B"], rows, -1).transpose(0, 1)
    seen = torch.arange(c["T"], device=q.device) <= _new_rows(c, s["len"])[..., None]
    x = (q @ k.transpose(-1, -2)).masked_fill(~seen[:, None], -math.inf)
    w = _softmax(torch.cat((xp, x), -1))
    wp, w = w[..., :c["prefix"]], w[..., c["prefix"]:]
    op = wp.transpose(0, 1).reshape(c["hkv"], c["B"] * rows, -1) @ vp[0]
    return _merged(op.reshape(c["hkv"], c["B"], rows, -1).transpose(0, 1) + w @ v, s)


def _plain_weights(s):
    c = s["c"]
    k, v = _grouped(s["K"], c["hkv"], c["d"]), _grouped(s["V"], c["hkv"], c["d"])
    x = (_queries(s) / math.sqrt(c["d"])) @ k.transpose(-1, -2)
    j = torch.arange(c["T"], device=x.device)
    seen = j <= _new_rows(c, s["len"])[..., None]
    w = _softmax(x.masked_fill(~seen[:, None], -math.inf))
    L = s["len"][:, None, None]
    old, total = s["w"], w.sum(2)
    s["w"].copy_(torch.where(j < L - c["Tq"], old + total, torch.where(j < L, total, old)))
    return {"out": _merged(w @ v, s), "weights": s["w"]}


def _plain_evict(s):
    c = s["c"]
    B, T, n, hkv, d = c["B"], c["T"], c["keep"], c["hkv"], c["d"]
    L = s["len"].long()[:, None, None]
    j = torch.arange(T, device=L.device)
    # the kept recent tokens rank above every weight, tokens past the length below
    rank = torch.where(j >= L - c["recent"], math.inf, s["w"])
    rank = torch.where(j < L, rank, -math.inf)
    order = rank.sort(dim=-1, descending=True, stable=True).indices[..., :n]
    order = order.masked_fill(torch.arange(n, device=L.device) >= L, T).sort(-1).values
    valid = order < T
    at = order.clamp(max=T - 1)
    rows = at.transpose(1, 2)[..., None].expand(-1, -1, -1, d)      # (B, n, h_kv, d)
    k = s["K"].reshape(B, T, hkv, d).gather(1, rows).reshape(B, n, hkv * d)
    v = s["V"].reshape(B, T, hkv, d).gather(1, rows).reshape(B, n, hkv * d)
    new = s["len"].clamp(max=n)
    inside = torch.arange(n, device=L.device)[:, None] < new[:, None, None]
    s["Ko"].copy_(torch.where(inside, k, s["Ko"]))
    s["Vo"].copy_(torch.where(inside, v, s["Vo"]))
    s["wo"].copy_(torch.where(valid, s["w"].gather(2, at), s["wo"]))
    return {"K": s["Ko"], "V": s["Vo"], "lengths": new, "weights": s["wo"],
            "kept": order.masked_fill(~valid, -1).int()}


# ------------------------------------------------------------------ the package's calls

def _own(s):
    c, layer = s["c"], s["layer"]
    if c["op"] == "window":
        return layer.attention_window(s["Q"], s["K"], s["V"], c["window"], c["sinks"], kv_lengths=s["len"],
                                      out=s["out"], G=s["G"])
    if c["op"] == "decode_window":
        return layer.decode_window(s["Q"], s["K"], s["V"], s["len"], c["window"], c["sinks"], out=s["out"])
    if c["op"] == "shared":
        return layer.decode_shared(s["Q"], s["Kp"], s["Vp"], s["K"], s["V"], s["len"], out=s["out"])
    if c["op"] == "weights":
        out = layer.decode_weights(s["Q"], s["K"], s["V"], s["len"], s["w"], out=s["out"])
        return {"out": out, "weights": s["w"]}
    K, V, lengths, w, kept = layer.evict(s["K"], s["V"], s["len"], s["w"], c["keep"], c["recent"],
                                         K_out=s["Ko"], V_out=s["Vo"], weights_out=s["wo"])
    return {"K": K, "V": V, "lengths": lengths, "weights": w, "kept": kept}


def run(state):
    if own:
        return _own(state)
    return {"window": _plain_window, "decode_window": _plain_decode_window, "shared": _plain_shared,
            "weights": _plain_weights, "evict": _plain_evict}[state["c"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    size = 2 if c["dtype"] == "bf16" else 4
    B, T, Tq, h, hkv, d = c["B"], c["T"], c["Tq"], c["h"], c["hkv"], c["d"]
    L = (_lowest(c) + T) / 2 if c["ragged"] else T                  # mean length
    rows = B * Tq * h * d * size                                    # queries, or outputs
    if c["op"] == "window":
        W, S = min(c["window"], T), c["sinks"]
        pairs = sum(min(i + 1, L, W + min(S, max(0, i + 1 - W))) for i in range(T))
        return {"bytes": B * T * (2 * h + (h if c["gated"] else 0)) * d * size + 2 * B * L * hkv * d * size,
                "flops": 4 * B * h * d * pairs}
    if c["op"] == "decode_window":
        n = min(L, c["window"] + c["sinks"] + Tq - 1)
        return {"bytes": 2 * rows + 2 * B * n * hkv * d * size, "flops": 4 * B * h * Tq * n * d}
    if c["op"] == "shared":
        return {"bytes": 2 * rows + 2 * (B * L + c["prefix"]) * hkv * d * size,
                "flops": 4 * B * h * Tq * (L + c["prefix"]) * d}
    if c["op"] == "weights":
        return {"bytes": 2 * rows + 2 * B * L * hkv * d * size + 8 * B * hkv * L, "flops": 4 * B * h * Tq * L * d}
    n = min(L, c["keep"])
    return {"bytes": 4 * B * hkv * L + 4 * B * hkv * n * d * size + 8 * B * hkv * n, "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_attend(q, keys, values, visible):
    """q (R, d) over keys / values (n, d) where visible (R, n): the outputs and the weights."""
    score = torch.matmul(q.double(), keys.double().mT).div_(float(q.shape[-1]) ** 0.5)
    score[~visible] = -math.inf
    top = score.max(dim=1, keepdim=True).values.nan_to_num(neginf=0.0)
    e = score.sub_(top).exp_()
    total = e.sum(dim=1, keepdim=True)
    w = torch.where(total > 0, e / total, 0.0)
    return w @ values.double(), w


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    B, T, Tq, h, hkv, d = c["B"], c["T"], c["Tq"], c["h"], c["hkv"], c["d"]
    per, lens = h // hkv, s["len"].tolist()
    dev = s["len"].device
    if c["op"] == "evict":
        K, V, wo = s["Ko"].double(), s["Vo"].double(), s["wo"].double()
        for b in range(B):
            for g in range(hkv):
                L, n = lens[b], c["keep"]
                w = s["w"][b, g]
                if L <= n:
                    keep = list(range(L))
                else:
                    early = w[:L - c["recent"]].tolist()
                    heavy = sorted(range(len(early)), key=lambda t: (-early[t], t))[:n - c["recent"]]
                    keep = sorted(heavy) + list(range(L - c["recent"], L))
                at = torch.tensor(keep, device=dev, dtype=torch.long)
                cols = slice(g * d, (g + 1) * d)
                K[b, :len(keep), cols] = s["K"][b, at, cols].double()
                V[b, :len(keep), cols] = s["V"][b, at, cols].double()
                wo[b, g, :len(keep)] = w[at].double()
        return {"K": K, "V": V, "lengths": None, "weights": wo, "kept": None}
    out = torch.zeros((B, T if c["op"] == "window" else Tq, h * d), device=dev, dtype=torch.float64)
    weights = s["w"].double() if c["op"] == "weights" else None
    for b in range(B):
        L = lens[b]
        for i in range(h):
            g = i // per
            qc, kc = slice(i * d, (i + 1) * d), slice(g * d, (g + 1) * d)
            if c["op"] == "window":
                for r0 in range(0, T, 1024):                        # rows in blocks, keys they can reach
                    row = torch.arange(r0, min(T, r0 + 1024), device=dev)
                    lo = max(0, r0 - c["window"] + 1)
                    key = torch.cat((torch.arange(0, min(c["sinks"], lo), device=dev),
                                     torch.arange(lo, min(T, r0 + 1024), device=dev)))
                    back = row[:, None] - key
                    see = (back >= 0) & (key < L) & ((back < c["window"]) | (key < c["sinks"]))
                    o, _ = _exact_attend(s["Q"][b, row, qc], s["K"][b, key, kc], s["V"][b, key, kc], see)
                    if c["gated"]:
                        o = o * torch.sigmoid(s["G"][b, row, qc].double())
                    out[b, row, qc] = o
                continue
            keys, values = s["K"][b, :L, kc], s["V"][b, :L, kc]
            back = torch.arange(L - Tq, L, device=dev)[:, None] - torch.arange(L, device=dev)
            see = back >= 0
            if c["op"] == "decode_window":
                see &= (back < c["window"]) | (torch.arange(L, device=dev) < c["sinks"])
            if c["op"] == "shared":
                keys, values = torch.cat((s["Kp"][:, kc], keys)), torch.cat((s["Vp"][:, kc], values))
                see = torch.cat((see.new_ones((Tq, c["prefix"])), see), 1)
            o, w = _exact_attend(s["Q"][b, :, qc], keys, values, see)
            out[b, :, qc] = o
            if c["op"] == "weights":
                if i % per == 0:
                    weights[b, g, L - Tq:L] = 0.0
                weights[b, g, :L] += w.sum(0)
    if c["op"] == "weights":
        return {"out": out, "weights": weights}
    return out
