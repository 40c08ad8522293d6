"""Measured cases of the quantised key/value cache: keys and values quantised to 4 or 8 bits as they are
written, read back as the values the cache holds, and the decode step that attends over the cache as it is.

``own`` chooses between the operators' plain form (elementary torch operations: 64 bits where a value may
lie next to a border, else 32, rounded once at the end) and the calls a user makes of the package.
``exact`` states the definitions in 64 bits, written apart from the plain form.

The cache holds, per (sequence, K/V head, token), the codes of the head's d channels and, per group of 64
channels (the last one may be shorter), a step s and a lowest value m, both bf16; n = 2^bits - 1:
  m     the largest bf16 not above the group's minimum
  s     the smallest bf16 with n s >= maximum - m, at least 2^-126
  code  (x - m) / s rounded to the nearest whole number, ties to even;  it stands for  s code + m
A group with a value that is not finite in bf16 has s = m = NaN.  4-bit codes: channel 2i in the low half
of byte i, channel 2i + 1 in the high half; rows are padded to 32 channels.

  write   rows 0 .. n_b - 1 of K and V become tokens L_b - n_b .. L_b - 1 of sequence b
  read    the values of the same tokens, into rows 0 .. n_b - 1
  decode  new token t of T_q sits at p = L_b - T_q + t and sees keys j <= p; query head i reads K/V head
          i // (h // h_kv):  o = sum_j softmax_j(q . k_j / sqrt(d)) v_j  over the values that are held
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_GROUP = 64
_BF16_MAX = 3.3895313892515355e38


def _case(name, op, dtype="bf16", bits=4, B=1, Tq=1, T=1024, h=16, hkv=16, d=64, new=0, ragged=False):
    """new: rows a write brings at most, or a read takes (0: the whole cache)."""
    c = {"op": op, "dtype": dtype, "bits": bits, "B": B, "Tq": Tq, "T": T, "h": h, "hkv": hkv, "d": d,
         "new": new or T, "ragged": ragged}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the decode benchmark's batch writes its next token: latency
        _case("write_step", "write", B=32, T=1024, hkv=16, d=128, new=1, ragged=True),
        # prompts of the bf16 causal layer (B = 4, T = 2048, d = 64), padded to one length
        _case("write_prompt", "write", B=4, T=2048, hkv=16, d=64, ragged=True),
        # a few prompts of an fp32 layer, odd length, 8 bits
        _case("write_prompt_f32", "write", "f32", bits=8, B=3, T=1001, hkv=8, d=64, ragged=True),
        # a batch of long prompts at once
        _case("write_long", "write", B=8, T=8192, hkv=16, d=128),
        # two short caches of an fp32 layer back to 32 bits
        _case("read_few_f32", "read", "f32", bits=8, B=2, T=1000, hkv=8, d=64),
        # the decode benchmark's grouped-head caches back to bf16
        _case("read_batch", "read", B=32, T=8192, hkv=4, d=128, ragged=True),
        # one user's next token: latency
        _case("decode_one", "decode", B=1, T=4096, h=16, hkv=4, d=64),
        # the decode benchmark: a K/V head for each query head
        _case("decode_batch", "decode", B=32, T=8192, h=16, hkv=16, d=128, ragged=True),
        # the same with grouped heads
        _case("decode_grouped", "decode", B=32, T=8192, h=16, hkv=4, d=128, ragged=True),
        # one user with a very long context, 8 bits, two K/V heads
        _case("decode_long", "decode", bits=8, B=1, T=131072, h=16, hkv=2, d=128),
        # a few new tokens at once (speculative decoding) over one K/V head: 80 query rows share a cache
        _case("decode_tokens", "decode", B=8, Tq=5, T=8192, h=16, hkv=1, d=128, ragged=True),
        # fp32 layer, a few new tokens, odd sizes
        _case("decode_tokens_f32", "decode", "f32", B=3, Tq=5, T=2000, h=8, hkv=4, d=64, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("write", "read", "decode", "decode"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    hkv = rng.choice((1, 2, 4, 8, 16))
    per = rng.choice([p for p in (1, 2, 4, 8, 16) if p * hkv <= 16])
    d = rng.choice((64, 128)) if dtype == "bf16" else rng.choice((32, 64, 80, 128))
    c = dict(dtype=dtype, bits=rng.choice((4, 4, 8)), h=hkv * per, hkv=hkv, d=d, ragged=rng.random() < 0.7)
    B = _log_int(rng, 1, 32)
    T = _log_int(rng, 64, 8192)
    if op == "decode":
        return _case(None, op, B=B, T=T, Tq=rng.choice((1, 1, 1, 2, 5)), **c)
    B = min(B, 8)
    return _case(None, op, B=B, T=T, new=rng.choice((1, 0, _log_int(rng, 1, T))), **c)


def _lowest(c):
    """Least cached length of a ragged batch."""
    return max(c["Tq"], c["T"] // 2)


# ------------------------------------------------------------------ the plain forms

def _bf16_down(x):
    """The largest bf16 values not above x (fp32), as fp32."""
    i = x.contiguous().view(torch.int32)
    cut = i & -65536
    return torch.where((i < 0) & (cut != i), cut + 65536, cut).view(torch.float32)


def _quantise(x, bits):
    """x (..., d): codes (..., d) uint8 and [step, lowest] (..., groups, 2) bf16."""
    n = 2 ** bits - 1
    codes, params = [], []
    for y in x.split(_GROUP, dim=-1):
        y = y.double()
        bad = ~(y.abs() <= _BF16_MAX).all(-1, keepdim=True)
        y = y.masked_fill(bad, 0.0)
        low = _bf16_down(y.amin(-1, keepdim=True).float())
        span = y.amax(-1, keepdim=True) - low.double()
        # the smallest bf16 step whose n-fold covers the span, from a candidate just below it
        step = _bf16_down((span / n).float() * (1 - 2.0 ** -7))
        for _ in range(4):
            up = (step.view(torch.int32) + 65536).view(torch.float32)
            step = torch.where(step.double() * n < span, up, step)
        step = step.clamp(min=2.0 ** -126)
        codes.append(torch.round((y - low.double()) / step.double()).clamp(max=n).to(torch.uint8))
        params.append(torch.cat((step, low), -1).masked_fill(bad, math.nan).to(torch.bfloat16))
    return torch.cat(codes, -1), torch.stack(params, -2)


def _pack(codes, bits):
    """Codes (..., d) as the bytes of a cache row."""
    d = codes.shape[-1]
    row = codes.new_zeros(codes.shape[:-1] + ((d + 31) // 32 * 32,))
    row[..., :d] = codes
    return row if bits == 8 else row[..., 0::2] | (row[..., 1::2] << 4)


def _values(codes, params, bits, d):
    """What a cache's rows stand for, (..., d) fp32."""
    if bits == 4:
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    p = params.float().repeat_interleave(_GROUP, dim=-2)[..., :d, :]
    return codes[..., :d].float() * p[..., 0] + p[..., 1]


def _heads(x, n, d):
    """(B, T, n d) -> (B, n, T, d)."""
    return x.reshape(x.shape[0], x.shape[1], n, d).transpose(1, 2)


def _tokens(s):
    """Cache row (B, new) of each row of a write or read, and whether it is one of the n_b."""
    i = torch.arange(s["c"]["new"], device=s["len"].device)
    n = s["count"].long()[:, None]
    return (s["len"].long()[:, None] - n + i).clamp(0, s["T"] - 1), i < n


def _plain_read(s):
    c = s["c"]
    at, valid = _tokens(s)
    b, g = torch.arange(c["B"], device=at.device)[:, None, None], torch.arange(c["hkv"], device=at.device)[:, None]
    for x in "KV":
        held = _values(s[x + "c"][b, g, at[:, None]], s[x + "p"][b, g, at[:, None]], c["bits"], c["d"])
        rows = held.transpose(1, 2).flatten(2).to(_DT[c["dtype"]])
        s[x + "o"].copy_(torch.where(valid[..., None], rows, s[x + "o"]))
    return {"K": s["Ko"], "V": s["Vo"]}


def _plain_write(s):
    c = s["c"]
    at, valid = _tokens(s)
    b, t = valid.nonzero(as_tuple=True)
    for x in "KV":
        codes, params = _quantise(_heads(s[x], c["hkv"], c["d"]), c["bits"])
        s[x + "c"][b, :, at[b, t]] = _pack(codes, c["bits"])[b, :, t]
        s[x + "p"][b, :, at[b, t]] = params[b, :, t]
    return _plain_read(s)


def _plain_decode(s):
    c = s["c"]
    B, hkv, d, Tq = c["B"], c["hkv"], c["d"], c["Tq"]
    q = _heads(s["Q"].float(), c["h"], d).reshape(B, hkv, -1, d)
    x = (q / math.sqrt(d)) @ _values(s["Kc"], s["Kp"], c["bits"], d).transpose(-1, -2)
    t = torch.arange(Tq, device=x.device).repeat(c["h"] // hkv)
    row = (s["len"].long()[:, None] - Tq + t)[:, None, :, None]
    x = x.masked_fill(torch.arange(s["T"], device=x.device) > row, -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    v = _values(s["Vc"], s["Vp"], c["bits"], d)
    v = v.masked_fill((torch.arange(s["T"], device=x.device) >= s["len"][:, None])[:, None, :, None], 0.0)
    o = (e @ v) / e.sum(-1, keepdim=True)
    return o.reshape(B, c["h"], Tq, d).transpose(1, 2).flatten(2).to(_DT[c["dtype"]])


# ------------------------------------------------------------------ inputs, and the package's calls

def prepare(case, seed):
    c = dict(case)
    dt, dev = _DT[c["dtype"]], "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    B, T, Tq, h, hkv, d, bits = c["B"], c["T"], c["Tq"], c["h"], c["hkv"], c["d"], c["bits"]
    cap = (T + 15) // 16 * 16                                       # a cache holds whole sixteens of tokens
    row, groups = (d + 31) // 32 * 32 * bits // 8, (d + _GROUP - 1) // _GROUP

    # keys and values of real layers: channels of different size and mean
    size = torch.exp(0.5 * torch.randn((hkv * d,), generator=g, device=dev))
    mean = 0.5 * torch.randn((hkv * d,), generator=g, device=dev)

    def rows(n):
        return torch.randn((B, n, hkv * d), generator=g, device=dev).mul_(size).add_(mean).to(dt)

    s = {"c": c, "T": cap}
    if c["ragged"]:
        s["len"] = torch.randint(_lowest(c), T + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    else:
        s["len"] = torch.full((B,), T, device=dev, dtype=torch.int32)
    s["count"] = s["len"].clamp(max=c["new"])
    if own:
        from transformer_head_scaled_02_gb300 import Mha
        s["layer"] = Mha(h * d, h, d, d, dtype=dt, h_kv=hkv)
        cache = s["cache"] = s["layer"].quant_cache(B, T, bits)
        s.update(Kc=cache.K_codes, Kp=cache.K_params, Vc=cache.V_codes, Vp=cache.V_params)
    else:
        for x in "KV":
            s[x + "c"] = torch.empty((B, hkv, cap, row), device=dev, dtype=torch.uint8)
            s[x + "p"] = torch.empty((B, hkv, cap, groups, 2), device=dev, dtype=torch.bfloat16)
    for x in "KV":
        s[x + "c"].zero_()
        s[x + "p"].zero_()
    if c["op"] == "write":
        s["K"], s["V"] = rows(c["new"]), rows(c["new"])
    else:
        for x in "KV":                                              # sequence by sequence: it is large
            held = rows(T)
            for b in range(B):
                codes, params = _quantise(_heads(held[b:b + 1], hkv, d), bits)
                s[x + "c"][b:b + 1, :, :T] = _pack(codes, bits)
                s[x + "p"][b:b + 1, :, :T] = params
    if c["op"] == "decode":
        s["Q"] = torch.randn((B, Tq, h * d), generator=g, device=dev).to(dt)
        s["out"] = torch.empty((B, Tq, h * d), device=dev, dtype=dt)
    else:
        s["Ko"], s["Vo"] = (torch.zeros((B, c["new"], hkv * d), device=dev, dtype=dt) for _ in "KV")
    return s


def _own(s):
    layer, cache = s["layer"], s["cache"]
    if s["c"]["op"] == "decode":
        return layer.decode_quant(s["Q"], cache, s["len"], out=s["out"])
    if s["c"]["op"] == "write":
        layer.quant_write(cache, s["K"], s["V"], s["len"], s["count"])
    K, V = layer.quant_read(cache, s["len"], s["count"], K_out=s["Ko"], V_out=s["Vo"])
    return {"K": K, "V": V}


def run(state):
    if own:
        return _own(state)
    return {"write": _plain_write, "read": _plain_read, "decode": _plain_decode}[state["c"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    size = 2 if c["dtype"] == "bf16" else 4
    B, T, Tq, h, hkv, d = c["B"], c["T"], c["Tq"], c["h"], c["hkv"], c["d"]
    L = (_lowest(c) + T) / 2 if c["ragged"] else T                  # mean length
    held = hkv * (d * c["bits"] / 8 + 4 * ((d + _GROUP - 1) // _GROUP))  # bytes of a token's keys (or values)
    if c["op"] == "decode":
        return {"bytes": 2 * B * Tq * h * d * size + 2 * B * L * held, "flops": 4 * B * h * Tq * L * d}
    n = min(L, c["new"])
    return {"bytes": 2 * B * n * (hkv * d * size * (2 if c["op"] == "write" else 1) + held), "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_grid(x, up):
    """x to 8 significant bits, upwards or downwards."""
    power = (x.contiguous().view(torch.int64) & 0x7FF0000000000000).view(torch.float64)  # of two, not above |x|
    unit = power.clamp_min(2.0 ** -200) * 2.0 ** -7
    return (torch.ceil(x / unit) if up else torch.floor(x / unit)) * unit


def _exact_held(x, bits):
    """The values that stand for one group's channels x (..., channels) in a cache."""
    x = x.double()
    lowest = _exact_grid(x.min(dim=-1, keepdim=True).values, False)
    span = x.max(dim=-1, keepdim=True).values - lowest
    # (divided by a tensor: by a number it would be a product with the number's rounded reciprocal)
    step = _exact_grid(span / torch.full_like(span, 2 ** bits - 1), True).clamp_min(2.0 ** -126)
    return ((x - lowest) / step).round() * step + lowest


def _exact_cached(s, x, b, g, L):
    """Keys or values (L, d) of one sequence and K/V head."""
    c = s["c"]
    byte = s[x + "c"][b, g, :L].long()
    out = torch.empty((L, c["d"]), device=byte.device, dtype=torch.float64)
    for i in range(c["d"]):
        code = byte[:, i] if c["bits"] == 8 else (byte[:, i // 2] >> (4 * (i % 2))) % 16
        step, lowest = s[x + "p"][b, g, :L, i // _GROUP].double().unbind(-1)
        out[:, i] = code * step + lowest
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    B, Tq, h, hkv, d = c["B"], c["Tq"], c["h"], c["hkv"], c["d"]
    lens, counts = s["len"].tolist(), s["count"].tolist()
    if c["op"] == "decode":
        out = torch.zeros((B, Tq, h * d), device=s["len"].device, dtype=torch.float64)
        for b in range(B):
            L = lens[b]
            hidden = torch.ones((Tq, L), device=out.device, dtype=torch.bool).triu(L - Tq + 1)
            for g in range(hkv):
                k, v = _exact_cached(s, "K", b, g, L), _exact_cached(s, "V", b, g, L)
                for i in range(g * (h // hkv), (g + 1) * (h // hkv)):
                    cols = slice(i * d, (i + 1) * d)
                    score = (s["Q"][b, :, cols].double() @ k.mT) / d ** 0.5
                    out[b, :, cols] = torch.softmax(score.masked_fill(hidden, -math.inf), -1) @ v
        return out
    out = {"K": s["Ko"].double(), "V": s["Vo"].double()}
    for b in range(B):
        L, n = lens[b], counts[b]
        for x in "KV":
            for g in range(hkv):
                if c["op"] == "read":
                    out[x][b, :n, g * d:(g + 1) * d] = _exact_cached(s, x, b, g, L)[L - n:]
                    continue
                for i in range(0, d, _GROUP):
                    cols = slice(g * d + i, g * d + min(d, i + _GROUP))
                    out[x][b, :n, cols] = _exact_held(s[x][b, :n, cols], c["bits"])
    return out
