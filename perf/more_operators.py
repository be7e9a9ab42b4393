"""Cases of the K/V cache held in 4 or 8 bits: written, read back, and attended to.

A cached row of a K/V head is a K and a V vector of 128 channels. Each group of 32 channels has a bf16 scale
s = bf16(max |x| / m), m = 7 (4 bits) or 127 (8 bits), and a whole number for each channel, n = x / s rounded to the
nearest, ties away from zero; n * s is the value that the cache holds. (A group whose largest magnitude is below 2^-100
is held as zeros.)

Three kinds of pass, each through the public calls of long_context_causal_blockwise_gb300:

  write   kv_cache_write, then kv_cache_read of the rows written: K and V of new tokens go into the cache, and come back
          as the values that it holds
  read    kv_cache_read: rows of the cache as bf16 K and V, as a chunk of a prompt wants them that attends in bf16
  attn    attn_cache_decode: attention of the newest tokens of each sequence over the cached values; a query at position
          p sees the keys j <= p with p - j < window, and the first `sinks` keys

With `own` false every kind is computed in its plain form: elementary operations in 32 bits, rounded once at the end.
"""

import math

import torch

own = False

D = 128
GROUP = 32
BF16 = torch.bfloat16
FULL = 1 << 30  # a window that hides nothing


def listed():
    return [
        # one new token of one sequence: what every layer of a decoding step writes, where the launch counts
        dict(name="write_token", kind="write", bits=4, B=1, Hkv=32, T=1, Smax=4096, ragged=False),
        # a batch of prompts of unequal length, padded on the left
        dict(name="write_ragged_b3", kind="write", bits=8, B=3, Hkv=8, T=1777, Smax=2000, ragged=True),
        # a long prompt through a layer with 32 K/V heads
        dict(name="write_prompt_32k", kind="write", bits=4, B=1, Hkv=32, T=32768, Smax=32768, ragged=False),
        # part of two cached contexts, from the middle of a cache
        dict(name="read_b2_8bit", kind="read", bits=8, B=2, Hkv=8, n=2001, start=4099, Smax=8192),
        # a 64K context as bf16, for the next chunk of its prompt
        dict(name="read_64k", kind="read", bits=4, B=1, Hkv=8, n=65536, start=0, Smax=65536),
        # a short conversation: the smallest call of serving
        dict(name="attn_b1_777", kind="attn", bits=4, B=1, H=32, Hkv=32, T=1, Smax=777, window=FULL, sinks=0),
        # one token against a window with sinks
        dict(name="attn_b1_w2048", kind="attn", bits=4, B=1, H=32, Hkv=32, T=1, Smax=8192, window=2048, sinks=4),
        # a batch of sequences of unequal length, shared K/V heads, two new tokens each
        dict(name="attn_b8_t2_gqa", kind="attn", bits=4, B=8, H=32, Hkv=8, T=2, Smax=20001, window=FULL, sinks=0),
        # a batch of long contexts with 40 heads, every key of a wide window read once
        dict(name="attn_b4_w32k", kind="attn", bits=4, B=4, H=40, Hkv=40, T=1, Smax=40000, window=32768, sinks=4),
        # one long context in 8 bits
        dict(name="attn_128k_8bit", kind="attn", bits=8, B=1, H=32, Hkv=8, T=1, Smax=131072, window=FULL, sinks=0),
        # the longest context: 512K tokens, one new one
        dict(name="attn_512k", kind="attn", bits=4, B=1, H=32, Hkv=8, T=1, Smax=524288, window=FULL, sinks=0),
        # sixteen drafted tokens checked at once against a 64K context
        dict(name="attn_t16_64k", kind="attn", bits=4, B=1, H=32, Hkv=8, T=16, Smax=65536, window=FULL, sinks=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        case = _draw_once(rng)
        w = work(case)
        if w["bytes"] > 7.0e8 or w["flops"] > 1.7e10 or case["B"] * case["Hkv"] * case["Smax"] > 6.4e6:
            continue
        return case


def _draw_once(rng):
    kind = rng.choice(["write", "read", "attn", "attn"])
    bits = rng.choice([4, 4, 8])
    H = rng.choice([4, 8, 16, 32, 40])
    Hkv = H // rng.choice([1, 1, 2, 4, 8] if H != 4 else [1, 2, 4])
    B = _log_int(rng, 1, 16)
    if kind == "write":
        T = _log_int(rng, 1, 32768)
        return dict(kind=kind, bits=bits, B=B, Hkv=Hkv, T=T, Smax=T + _log_int(rng, 1, 4096) - 1, ragged=rng.random() < 0.4)
    Smax = _log_int(rng, 16, 524288)
    if kind == "read":
        n = _log_int(rng, 1, min(Smax, 65536))
        return dict(kind=kind, bits=bits, B=B, Hkv=Hkv, n=n, start=rng.randrange(Smax - n + 1), Smax=Smax)
    window = FULL if rng.random() < 0.6 else _log_int(rng, 16, 65536)
    return dict(kind=kind, bits=bits, B=B, H=H, Hkv=Hkv, T=rng.choice([1, 1, 1, 2, 3, 4, 7, 16]), Smax=Smax,
                window=window, sinks=rng.choice([0, 1, 4, 16, 128]) if window < FULL else 0)


def _lens(case):
    """Rows in each sequence's cache after the newest tokens."""
    B, Smax = case["B"], case["Smax"]
    if case["kind"] == "read":
        return [Smax] * B
    T = case["T"]
    if case["kind"] == "write":
        # a prompt from the cache's first row on, padded on the left where the batch is ragged; or the cache's end
        return [max(1, T - (b * T) // (2 * B) - (b % 3)) if b else T for b in range(B)] if case["ragged"] else [Smax] * B
    return [max(min(T, Smax), Smax - (b * Smax) // (2 * B) - (b % 3)) for b in range(B)]


def _rows_written(case):
    """(first row, rows) that a write pass reads back."""
    return (0, case["T"]) if case["ragged"] else (case["Smax"] - case["T"], case["T"])


def _inputs(case, seed):
    """q (None without one), k and v: those of the new tokens, or of every row of the cache."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    B, Hkv = case["B"], case["Hkv"]
    T = case["T"] if case["kind"] == "write" else case["Smax"]
    # some channels of K are larger than the others in every token
    k = (normal(B, T, Hkv, D) * torch.where(normal(Hkv, D) > 1.5, 3.0, 1.0)).to(BF16)
    v = normal(B, T, Hkv, D).to(BF16)
    q = normal(B, case["T"], case["H"], D).to(BF16) if case["kind"] == "attn" else None
    return q, k, v


def prepare(case, seed):
    st = dict(case)
    B, Hkv, Smax = case["B"], case["Hkv"], case["Smax"]
    st["q"], st["k"], st["v"] = _inputs(case, seed)
    st["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    if own:
        import long_context_causal_blockwise_gb300 as lcb

        st["cache"] = lcb.kv_cache_empty(B, Hkv, Smax, bits=case["bits"], device="cuda")
        if case["kind"] != "write":
            full = torch.full((B,), Smax, dtype=torch.int32, device="cuda")
            lcb.kv_cache_write(st["cache"], st.pop("k"), st.pop("v"), full)
    else:
        for name in ("k", "v"):
            st[name + "_codes"] = torch.zeros(B, Smax, Hkv, D * case["bits"] // 8, dtype=torch.uint8, device="cuda")
            st[name + "_scale"] = torch.zeros(B, Smax, Hkv, D // GROUP, dtype=BF16, device="cuda")
            if case["kind"] != "write":
                x = st.pop(name)
                for b in range(B):
                    st[name + "_codes"][b], st[name + "_scale"][b] = _plain_quant(x[b], case["bits"])
    return st


def run(st):
    if own:
        import long_context_causal_blockwise_gb300 as lcb

        if st["kind"] == "write":
            lcb.kv_cache_write(st["cache"], st["k"], st["v"], st["lens"])
            start, n = _rows_written(st)
            return lcb.kv_cache_read(st["cache"], n, start=start, lens=st["lens"])
        if st["kind"] == "read":
            return lcb.kv_cache_read(st["cache"], st["n"], start=st["start"])
        return lcb.attn_cache_decode(st["q"], st["cache"], st["lens"], window=st["window"], sinks=st["sinks"])
    if st["kind"] == "write":
        return _plain_write(st)
    if st["kind"] == "read":
        rows = slice(st["start"], st["start"] + st["n"])
        return tuple(_plain_values(st[x + "_codes"][:, rows], st[x + "_scale"][:, rows], st["bits"]).to(BF16) for x in "kv")
    return _plain_attn(st)


# ------------------------------------------------------------------ plain forms


def _plain_quant(x, bits):
    """(codes, scales) of x [..., 128]: bytes of one number (8 bits) or two (4 bits, the even channel in the low half)."""
    x = x.float().unflatten(-1, (D // GROUP, GROUP))
    top = x.abs().amax(dim=-1, keepdim=True)
    top = torch.where(top < 2.0 ** -100, 0.0, top)
    s = (top / (7.0 if bits == 4 else 127.0)).to(BF16)
    n = torch.floor(x.abs() / torch.where(s == 0, 1.0, s.float()) + 0.5)
    n = (torch.where(s == 0, 0.0, n) * x.sign()).flatten(-2).to(torch.int32)
    n = n + (8 if bits == 4 else 128)
    if bits == 4:
        n = n[..., 0::2] | (n[..., 1::2] << 4)
    return n.to(torch.uint8), s.squeeze(-1)


def _plain_values(codes, scale, bits):
    """fp32 [..., 128]"""
    if bits == 4:
        n = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).float() - 8.0
    else:
        n = codes.float() - 128.0
    return (n.unflatten(-1, (D // GROUP, GROUP)) * scale.float()[..., None]).flatten(-2)


def _plain_write(st):
    B, T = st["B"], st["T"]
    lens = st["lens"].long()
    dev = lens.device
    start, n = _rows_written(st)
    at = lens[:, None] - T + torch.arange(T, device=dev)[None]  # [B, T]: the row of each token
    # rows of the cache that the pass reads back, and the token that each of them gets
    row = start + torch.arange(n, device=dev)
    tok = row[None] - (lens[:, None] - T)
    has = (row[None] < lens[:, None]) & (tok >= 0)
    b = torch.arange(B, device=dev)[:, None].expand(B, T)
    keep = at >= 0
    out = []
    for name in ("k", "v"):
        codes, scale = _plain_quant(st[name], st["bits"])
        if st["ragged"]:
            st[name + "_codes"][b[keep], at[keep]] = codes[keep]
            st[name + "_scale"][b[keep], at[keep]] = scale[keep]
        else:
            st[name + "_codes"][:, start:start + n] = codes
            st[name + "_scale"][:, start:start + n] = scale
        x = _plain_values(st[name + "_codes"][:, start:start + n], st[name + "_scale"][:, start:start + n], st["bits"])
        out.append(torch.where(has[:, :, None, None], x, 0.0).to(BF16))
    return tuple(out)


def _plain_attn(st):
    q, lens, W, N = st["q"].float(), st["lens"].long(), st["window"], st["sinks"]
    B, T, H, _ = q.shape
    Smax, Hkv = st["Smax"], st["Hkv"]
    dev = q.device
    n_win = min(Smax, W + T - 1)
    # columns: the sinks, then the last n_win keys of each sequence
    win = lens[:, None] - n_win + torch.arange(n_win, device=dev)[None]
    sink = torch.arange(min(N, Smax), device=dev)[None].expand(B, -1)
    p = (lens[:, None] - T + torch.arange(T, device=dev)[None])[:, :, None]  # [B, T, 1]
    in_win = (win[:, None] >= 0) & (win[:, None] <= p) & (p - win[:, None] < W)
    in_sink = (sink[:, None] <= p) & (p - sink[:, None] >= W)
    vis = torch.cat([in_sink, in_win], dim=2)  # [B, T, n]
    j = torch.cat([sink, win.clamp(min=0)], dim=1)
    row = torch.arange(B, device=dev)[:, None]
    kk, vv = (_plain_values(st[x + "_codes"][row, j], st[x + "_scale"][row, j], st["bits"]).transpose(1, 2) for x in "kv")
    qq = q.view(B, T, Hkv, H // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    s = torch.matmul(qq, kk.transpose(2, 3)).mul_(D ** -0.5)
    vis = vis[:, None, :, None].expand(B, Hkv, T, H // Hkv, -1).reshape(s.shape)
    s.masked_fill_(~vis, float("-inf"))
    m = s.amax(dim=-1, keepdim=True)
    s.sub_(m.masked_fill(m == float("-inf"), 0.0)).exp_()
    z = s.sum(dim=-1, keepdim=True)
    s.div_(z.masked_fill(z == 0, 1.0))
    lse = (m + torch.log(z)).masked_fill(z == 0, float("-inf")).squeeze(-1)
    o = torch.matmul(s, vv).view(B, Hkv, T, H // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, T, H, D)
    lse = lse.view(B, Hkv, T, H // Hkv).permute(0, 1, 3, 2).reshape(B, H, T)
    return o.to(BF16), lse.contiguous()


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    rec = 2 * (D * case["bits"] // 8 + 2 * D // GROUP)  # bytes of a cached row of a head, K and V
    B, Hkv = case["B"], case["Hkv"]
    if case["kind"] == "write":
        # K and V in, the cache's rows out, their values out
        rows = sum(min(n, case["T"]) for n in _lens(case)) * Hkv
        return {"bytes": rows * (4 * D + rec) + 4 * B * case["T"] * Hkv * D, "flops": 8 * rows * D}
    if case["kind"] == "read":
        rows = B * case["n"] * Hkv
        return {"bytes": rows * (rec + 4 * D), "flops": 2 * rows * D}
    H, T, W, N = case["H"], case["T"], case["window"], case["sinks"]
    keys = pairs = 0
    for n in _lens(case):
        lo = max(0, n - T - W + 1)  # the oldest key in any window
        keys += n - lo + min(N, lo)
        for p in range(max(0, n - T), n):
            first = max(0, p - W + 1)
            pairs += p + 1 - first + min(N, first)
    return {"bytes": keys * Hkv * rec + B * T * H * (4 * D + 4) + 4 * B, "flops": 4 * D * H * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits


def _held(x, bits):
    """The values that the cache holds for x [..., 128], in 64 bits."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for c in range(0, D, GROUP):
        g = x[..., c:c + GROUP].double()
        top = torch.max(g.abs(), dim=-1, keepdim=True).values
        s = (top / (2 ** (bits - 1) - 1)).to(BF16).double()
        s = torch.where(top >= 2.0 ** -100, s, torch.full_like(s, math.inf))  # a group of zeros: every quotient is 0
        n = torch.trunc(g / s + torch.copysign(torch.full_like(g, 0.5), g))
        out[..., c:c + GROUP] = torch.where(n == 0, 0.0, n * s)
    return out


def exact(case, seed):
    B, Hkv, bits = case["B"], case["Hkv"], case["bits"]
    q, k, v = _inputs(case, seed)
    if case["kind"] == "read":
        rows = slice(case["start"], case["start"] + case["n"])
        return _held(k[:, rows], bits), _held(v[:, rows], bits)
    if case["kind"] == "write":
        start, n = _rows_written(case)
        out = [torch.zeros(B, n, Hkv, D, dtype=torch.float64, device="cuda") for _ in "kv"]
        for b, length in enumerate(_lens(case)):
            for r, x in zip(out, (k, v)):
                new = min(case["T"], length)  # the tokens that stand at a row
                r[b, length - start - new:length - start] = _held(x[b, case["T"] - new:], bits)
        return tuple(out)
    Tq, H, W, N = case["T"], case["H"], case["window"], case["sinks"]
    G = H // Hkv
    o = torch.zeros(B, Tq, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, Tq), -math.inf, dtype=torch.float64, device="cuda")
    for b, length in enumerate(_lens(case)):
        for h in range(Hkv):
            kd, vd = _held(k[b, :length, h], bits), _held(v[b, :length, h], bits)
            for t in range(Tq):
                p = length - Tq + t
                if p < 0:
                    continue
                first = max(0, p - W + 1)
                js = torch.cat([torch.arange(min(N, first)), torch.arange(first, p + 1)]).to("cuda") if N and first else \
                    slice(first, p + 1)
                s = q[b, t, h * G:(h + 1) * G].double() @ kd[js].T / math.sqrt(D)
                L = torch.logsumexp(s, dim=-1)
                lse[b, h * G:(h + 1) * G, t] = L
                o[b, t, h * G:(h + 1) * G] = torch.exp(s - L[:, None]) @ vd[js]
    return o, lse
