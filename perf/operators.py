"""Cases of the windowed-attention operators and of the rotary embedding with several position axes.

Four kinds of pass, each through the public calls of long_context_causal_blockwise_gb300:

  fwd     attn_window_fwd: attention whose query at position p sees the keys j <= p with p - j < window, and the
          first `sinks` keys whatever their distance (sinks), over [B, S, H, 128] tensors with shared K/V heads
  train   attn_window_fwd, then attn_window_bwd: one layer's forward and backward
  decode  attn_window_decode: the newest tokens of each sequence against its K/V cache
  rope    rope_axes: rotary positions with several axes (time, height, width), or the transpose of that rotation

With `own` false every kind is computed in its plain form: elementary operations in 32 bits (rotation angles in 64),
rounded once at the end.
"""

import math

import torch

own = False

D = 128
BF16 = torch.bfloat16


def listed():
    return [
        # a short conversation's prompt: one small forward, where the launch counts
        dict(name="fwd_prompt_777", kind="fwd", B=1, H=32, Hkv=32, Sq=777, Sk=777, window=256, sinks=4),
        # a prompt of ordinary length through a layer with 32 heads
        dict(name="fwd_8k_w1024", kind="fwd", B=1, H=32, Hkv=32, Sq=8192, Sk=8192, window=1024, sinks=4),
        # chunked prefill: the last 1000 tokens of a 64K context, K/V heads shared by four query heads
        dict(name="fwd_chunk_64k", kind="fwd", B=1, H=32, Hkv=8, Sq=1000, Sk=65536, window=16384, sinks=64),
        # training of a small batch of odd-length sequences, no sinks
        dict(name="train_b2_2001", kind="train", B=2, H=8, Hkv=8, Sq=2001, Sk=2001, window=512, sinks=0),
        # training with shared K/V heads and a sink region of a whole tile
        dict(name="train_16k_gqa", kind="train", B=1, H=32, Hkv=8, Sq=16384, Sk=16384, window=2048, sinks=128),
        # the long-context training layer: 32 heads, 32K tokens
        dict(name="train_32k_w4096", kind="train", B=1, H=32, Hkv=32, Sq=32768, Sk=32768, window=4096, sinks=4),
        # one token of one sequence: the smallest call of serving
        dict(name="decode_b1_w2048", kind="decode", B=1, H=32, Hkv=32, T=1, Smax=8192, window=2048, sinks=4),
        # a batch of sequences of unequal length with shared K/V heads, two new tokens each
        dict(name="decode_b8_t2_gqa", kind="decode", B=8, H=32, Hkv=8, T=2, Smax=20001, window=8192, sinks=16),
        # a batch of long contexts, every key of a wide window read once
        dict(name="decode_b4_w32k", kind="decode", B=4, H=40, Hkv=40, T=1, Smax=40000, window=32768, sinks=4),
        # one image's patches between text, K of a layer with shared heads
        dict(name="rope_image", kind="rope", B=1, H=8, S=1031, sections="16,24,24", interleaved=False, theta=1e6,
             inverse=False, per_batch=False),
        # a batch with positions of its own for every sequence, dQ turned back
        dict(name="rope_b2_inverse", kind="rope", B=2, H=32, S=4099, sections="24,20,20", interleaved=True, theta=1e4,
             inverse=True, per_batch=True),
        # an hour of video at 32 heads
        dict(name="rope_video_128k", kind="rope", B=1, H=32, S=131072, sections="16,24,24", interleaved=False,
             theta=1e6, inverse=False, per_batch=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        case = _draw_once(rng)
        w = work(case)
        if case["kind"] in ("fwd", "train"):
            # scores that the plain form holds, and the floating operations
            width = case["window"] + _block(case["window"]) + case["sinks"]
            if case["B"] * case["H"] * case["Sq"] * width > 5.0e9 or w["flops"] > 7.0e12:
                continue
        elif w["bytes"] > 2.5e9 or case.get("Smax", 0) * case.get("Hkv", 0) * case["B"] > 6.6e6:
            continue
        return case


def _draw_once(rng):
    kind = rng.choice(["fwd", "train", "decode", "rope"])
    H = rng.choice([4, 8, 16, 32, 40])
    if kind == "rope":
        a = rng.randrange(4, 41)
        b = rng.randrange(4, 61 - a)
        sections = rng.choice(["%d,%d,%d" % (a, b, 64 - a - b), "%d,%d" % (a, 64 - a), "16,24,24"])
        return dict(kind=kind, B=rng.choice([1, 1, 2, 3]), H=H, S=_log_int(rng, 1, 131072), sections=sections,
                    interleaved=rng.random() < 0.5, theta=rng.choice([1e4, 5e5, 1e6]), inverse=rng.random() < 0.5,
                    per_batch=rng.random() < 0.5)
    G = rng.choice([1, 1, 2, 4, 8] if H != 4 else [1, 2, 4])
    sinks = rng.choice([0, 1, 4, 4, 16, 64, 128, 200])
    B = rng.choice([1, 1, 2, 3])
    if kind == "decode":
        return dict(kind=kind, B=_log_int(rng, 1, 16), H=H, Hkv=H // G, T=rng.choice([1, 1, 1, 2, 3, 4]),
                    Smax=_log_int(rng, 16, 131072), window=_log_int(rng, 16, 65536), sinks=sinks)
    Sq = _log_int(rng, 16 if kind == "train" else 1, 32768)
    Sk = Sq + (0 if rng.random() < 0.6 else _log_int(rng, 1, 65536))
    return dict(kind=kind, B=B, H=H, Hkv=H // G, Sq=Sq, Sk=Sk, window=_log_int(rng, 16, 16384), sinks=sinks)


def _lens(case):
    """Keys in each sequence's cache: the first one full, the others shorter by odd amounts."""
    B, Smax, T = case["B"], case["Smax"], case["T"]
    return [max(min(T, Smax), Smax - (b * Smax) // (2 * B) - (b % 3)) for b in range(B)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(BF16)

    st = dict(case)
    B, H = case["B"], case["H"]
    if case["kind"] == "rope":
        S, axes = case["S"], len(case["sections"].split(","))
        st["x"] = normal(B, S, H, D)
        start = torch.randint(0, 100000, (B if case["per_batch"] else 1, 1), generator=gen, device="cuda")
        # an eighth of the tokens is text (all axes count together), then frames of 24 x 24 patches
        i = torch.arange(S, device="cuda")[None]
        text = S // 8
        patch = (i - text).clamp(min=0)
        grid = [torch.div(patch, 576, rounding_mode="floor"), torch.div(patch, 24, rounding_mode="floor") % 24, patch % 24]
        pos = torch.stack([start + torch.where(i < text, i, text + g) for g in grid[:axes]])
        pos = pos.to(torch.int32)
        st["pos"] = pos if case["per_batch"] else pos[:, 0].contiguous()
        st["sections"] = tuple(int(n) for n in case["sections"].split(","))
        return st
    Hkv = case["Hkv"]
    if case["kind"] == "decode":
        st["q"] = normal(B, case["T"], H, D) * 1.5
        st["k"] = normal(B, case["Smax"], Hkv, D)
        st["v"] = normal(B, case["Smax"], Hkv, D)
        st["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
        return st
    st["q"] = normal(B, case["Sq"], H, D) * 1.5
    st["k"] = normal(B, case["Sk"], Hkv, D)
    st["v"] = normal(B, case["Sk"], Hkv, D)
    if case["kind"] == "train":
        st["do"] = normal(B, case["Sq"], H, D)
    return st


def run(st):
    if own:
        import long_context_causal_blockwise_gb300 as lcb

        if st["kind"] == "rope":
            x = st["x"]
            return lcb.rope_axes(x, st["theta"], st["pos"], st["sections"], inverse=st["inverse"],
                                 interleaved=st["interleaved"], out=torch.empty_like(x))
        if st["kind"] == "decode":
            return lcb.attn_window_decode(st["q"], st["k"], st["v"], st["lens"], st["window"], st["sinks"])
        o, lse = lcb.attn_window_fwd(st["q"], st["k"], st["v"], st["window"], st["sinks"])
        if st["kind"] == "fwd":
            return o, lse
        dq, dk, dv = lcb.attn_window_bwd(st["q"], st["k"], st["v"], o, lse, st["do"], st["window"], st["sinks"])
        return o, lse, dq, dk, dv
    if st["kind"] == "rope":
        return _plain_rope(st)
    if st["kind"] == "decode":
        return _plain_decode(st)
    return _plain_window(st)


# ------------------------------------------------------------------ plain forms


def _pair_axes(sections, interleaved):
    """The axis of each of the 64 feature pairs."""
    if not interleaved:
        return sum(([a] * n for a, n in enumerate(sections)), [])
    turns = [(i, a) for a, n in enumerate(sections) for i in range(n)]
    return [a for _, a in sorted(turns)]


def _plain_rope(st):
    x, pos = st["x"].float(), st["pos"]
    pos = pos[:, None] if pos.dim() == 2 else pos  # [axes, 1 or B, S]
    axis = torch.tensor(_pair_axes(st["sections"], st["interleaved"]), device=x.device)
    freq = st["theta"] ** (-2.0 * torch.arange(D // 2, device=x.device, dtype=torch.float64) / D)
    ang = pos.double()[axis].permute(1, 2, 0) * freq  # [1 or B, S, 64]
    c, s = torch.cos(ang).float()[:, :, None], torch.sin(ang).float()[:, :, None]
    if st["inverse"]:
        s = -s
    lo, hi = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([lo * c - hi * s, hi * c + lo * s], dim=-1).to(BF16)


def _softmax(s, vis):
    """In place over scores s: (P, LSE); a row with nothing visible has P = 0 and LSE = -inf."""
    s.masked_fill_(~vis, float("-inf"))
    m = s.amax(dim=-1, keepdim=True)
    m0 = m.masked_fill(m == float("-inf"), 0.0)
    s.sub_(m0).exp_()
    z = s.sum(dim=-1, keepdim=True)
    s.div_(z.masked_fill(z == 0, 1.0))
    return s, (m + torch.log(z)).masked_fill(z == 0, float("-inf")).squeeze(-1)


def _plain_decode(st):
    q, lens, W, N = st["q"].float(), st["lens"].long(), st["window"], st["sinks"]
    k, v = st["k"], st["v"]
    B, T, H, _ = q.shape
    Smax, Hkv = k.shape[1], k.shape[2]
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
    kk, vv = (t[row, j].float().transpose(1, 2) for t in (k, v))  # [B, Hkv, n, D]
    qq = q.view(B, T, Hkv, H // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    s = torch.matmul(qq, kk.transpose(2, 3)).mul_(D ** -0.5)
    vis = vis[:, None, :, None].expand(B, Hkv, T, H // Hkv, -1).reshape(s.shape)
    pr, lse = _softmax(s, vis)
    o = torch.matmul(pr, vv).view(B, Hkv, T, H // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, T, H, D)
    lse = lse.view(B, Hkv, T, H // Hkv).permute(0, 1, 3, 2).reshape(B, H, T)
    return o.to(BF16), lse.contiguous()


def _block(window):
    return 64 if window <= 64 else min(512, 1 << (window - 1).bit_length())


def _plain_window(st):
    """Queries in blocks of `blk`; a block sees the sinks and the m + 1 key blocks that its windows touch."""
    q, k, v, W = st["q"], st["k"], st["v"], st["window"]
    B, Sq, H, _ = q.shape
    Sk, Hkv = k.shape[1], k.shape[2]
    G, dev = H // Hkv, q.device
    N = min(st["sinks"], Sk)
    blk = _block(W)
    m = -(-(W - 1) // blk)
    off = Sk - Sq  # position of the first query
    first = off // blk  # its block
    lead = off - first * blk  # rows of padding before it
    nb = -(-(lead + Sq) // blk)
    tail = nb * blk - lead - Sq
    scale = D ** -0.5

    def q_blocks(x):  # [B, Sq, H, D] -> [B, Hkv, nb, G * blk, D]
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, lead, tail))
        return x.view(B, nb, blk, Hkv, G, D).permute(0, 3, 1, 4, 2, 5).reshape(B, Hkv, nb, G * blk, D)

    def from_q_blocks(x, d):  # back to [B, Sq, H, d]
        x = x.view(B, Hkv, nb, G, blk, d).permute(0, 2, 4, 1, 3, 5).reshape(B, nb * blk, H, d)
        return x[:, lead:lead + Sq]

    at = first - m + torch.arange(nb + m, device=dev)  # key blocks touched at all
    touch = torch.arange(nb, device=dev)[:, None] + torch.arange(m + 1, device=dev)[None]  # [nb, m + 1], into `at`
    pos_k = at[:, None] * blk + torch.arange(blk, device=dev)[None]  # [nb + m, blk]
    inside = ((pos_k >= 0) & (pos_k < Sk)).view(-1)
    take = pos_k.view(-1).clamp(0, Sk - 1)

    def k_blocks(x):  # [B, Sk, Hkv, D] -> [B, Hkv, nb, N + (m + 1) * blk, D]
        w = x[:, take].float() * inside[None, :, None, None]
        w = w.transpose(1, 2).reshape(B, Hkv, nb + m, blk, D)[:, :, touch].reshape(B, Hkv, nb, -1, D)
        s = x[:, :N].float().transpose(1, 2)[:, :, None].expand(B, Hkv, nb, N, D)
        return torch.cat([s, w], dim=3)

    def from_k_blocks(x):  # the adjoint of k_blocks
        s, w = x[:, :, :, :N].sum(dim=2), x[:, :, :, N:].reshape(B, Hkv, nb * (m + 1), blk, D)
        acc = torch.zeros(B, Hkv, nb + m, blk, D, device=dev).index_add_(2, touch.reshape(-1), w)
        acc = acc.view(B, Hkv, -1, D) * inside[None, None, :, None]
        full = torch.zeros(B, Hkv, Sk, D, device=dev).index_add_(2, take, acc)
        full[:, :, :N] += s
        return full.transpose(1, 2)

    p = (first * blk + torch.arange(nb * blk, device=dev)).view(nb, blk, 1)
    j = pos_k[touch].reshape(nb, 1, -1)
    in_win = (j >= 0) & (j < Sk) & (j <= p) & (p - j < W)
    j = torch.arange(N, device=dev)[None, None]
    in_sink = (j <= p) & (p - j >= W)
    vis = torch.cat([in_sink, in_win], dim=2)[:, None].expand(nb, G, blk, -1).reshape(nb, G * blk, -1)

    qb, kb, vb = q_blocks(q), k_blocks(k), k_blocks(v)
    pr, lse = _softmax(torch.matmul(qb, kb.transpose(3, 4)).mul_(scale), vis)
    ob = torch.matmul(pr, vb)
    o = from_q_blocks(ob, D).to(BF16)
    lse = from_q_blocks(lse, 1).view(B, Sq, H).transpose(1, 2).contiguous()
    if st["kind"] == "fwd":
        return o, lse
    dob = q_blocks(st["do"])
    dv = from_k_blocks(torch.matmul(pr.transpose(3, 4), dob)).to(BF16)
    ds = torch.matmul(dob, vb.transpose(3, 4)).sub_((dob * ob).sum(dim=-1, keepdim=True)).mul_(pr).mul_(scale)
    dq = from_q_blocks(torch.matmul(ds, kb), D).to(BF16)
    dk = from_k_blocks(torch.matmul(ds.transpose(3, 4), qb)).to(BF16)
    return o, lse, dq, dk, dv


# ------------------------------------------------------------------ what a pass cannot do without


def _seen(p, Sk, W, N):
    """Keys that the query at position p sees."""
    if p < 0:
        return 0
    lo, hi = max(0, p - W + 1), min(p, Sk - 1)
    return max(0, hi - lo + 1) + max(0, min(N, lo, Sk))


def work(case):
    B, H = case["B"], case["H"]
    if case["kind"] == "rope":
        n = B * case["S"] * H * D
        axes = len(case["sections"].split(","))
        return {"bytes": 4 * n + 4 * axes * case["S"] * (B if case["per_batch"] else 1), "flops": 3 * n}
    W, N, Hkv = case["window"], case["sinks"], case["Hkv"]
    if case["kind"] == "decode":
        T, keys, pairs = case["T"], 0, 0
        for n in _lens(case):
            lo = max(0, n - T - W + 1)  # the oldest key in any window
            keys += n - lo + min(N, lo)
            pairs += sum(_seen(n - T + t, n, W, N) for t in range(T))
        return {"bytes": 4 * keys * Hkv * D + B * T * H * (4 * D + 4) + 4 * B, "flops": 4 * D * H * pairs}
    Sq, Sk = case["Sq"], case["Sk"]
    pairs = B * H * sum(_seen(Sk - Sq + i, Sk, W, N) for i in range(Sq))
    lo = max(0, Sk - Sq - W + 1)
    keys = Sk - lo + min(N, lo)
    q_bytes, kv_bytes = 2 * B * Sq * H * D, 2 * B * keys * Hkv * D
    if case["kind"] == "fwd":
        return {"bytes": 2 * q_bytes + 2 * kv_bytes + 4 * B * H * Sq, "flops": 4 * D * pairs}
    # q, do in; o, dq out; k, v in; dk, dv out (every row of them)
    return {"bytes": 4 * q_bytes + 2 * kv_bytes + 4 * B * Sk * Hkv * D + 4 * B * H * Sq, "flops": 14 * D * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "rope":
        return _exact_rope(st)
    if case["kind"] == "decode":
        out = [_exact_rows(st["q"][b:b + 1], st["k"][b:b + 1, :n], st["v"][b:b + 1, :n], None, n - case["T"],
                           case["window"], case["sinks"]) for b, n in enumerate(_lens(case))]
        return torch.cat([r[0] for r in out]), torch.cat([r[1] for r in out])
    out = _exact_rows(st["q"], st["k"], st["v"], st.get("do"), case["Sk"] - case["Sq"], case["window"], case["sinks"])
    return out if case["kind"] == "train" else out[:2]


def _exact_rope(st):
    out = torch.empty(st["x"].shape, dtype=torch.float64, device="cuda")
    start = 0
    order = [[] for _ in st["sections"]]  # the pairs of each axis
    if st["interleaved"]:
        left, k = list(st["sections"]), 0
        while k < D // 2:
            for a in range(len(left)):
                if left[a]:
                    order[a].append(k)
                    left[a] -= 1
                    k += 1
    else:
        for a, n in enumerate(st["sections"]):
            order[a] = list(range(start, start + n))
            start += n
    for a, pairs in enumerate(order):
        for k in pairs:
            ang = st["pos"][a].double() * st["theta"] ** (-k / 64.0)
            ang = (ang if ang.dim() == 2 else ang[None])[:, :, None] * (-1.0 if st["inverse"] else 1.0)
            z = torch.polar(torch.ones_like(ang), ang) * torch.complex(st["x"][..., k].double(), st["x"][..., k + 64].double())
            out[..., k], out[..., k + 64] = z.real, z.imag
    return out


def _exact_rows(q, k, v, do, pos0, W, N):
    """Panels of query rows against every key that one of them sees."""
    B, Sq, H, _ = q.shape
    Sk, Hkv = k.shape[1], k.shape[2]
    G = H // Hkv
    f8 = dict(dtype=torch.float64, device=q.device)
    o, lse = torch.zeros(B, Sq, H, D, **f8), torch.full((B, H, Sq), -math.inf, **f8)
    grads = [torch.zeros(t.shape, **f8) for t in (q, k, v)] if do is not None else None
    step = max(16, min(512, W // 4))
    for b in range(B):
        for h in range(Hkv):
            kd, vd = k[b, :, h].double(), v[b, :, h].double()
            for r in range(0, Sq, step):
                e = min(Sq, r + step)
                p = pos0 + torch.arange(r, e, device=q.device)
                lo, hi = max(0, pos0 + r - W + 1), max(0, min(Sk, pos0 + e))
                js = torch.cat([torch.arange(0, min(N, lo, Sk)), torch.arange(min(lo, hi), hi)]).to(q.device)
                if not js.numel():
                    continue
                seen = (js[None] <= p[:, None]) & ((p[:, None] - js[None] < W) | (js[None] < N))
                qd = q[b, r:e, h * G:(h + 1) * G].double().transpose(0, 1)  # [G, rows, D]
                s = torch.where(seen, qd @ kd[js].T / math.sqrt(D), -math.inf)
                L = torch.logsumexp(s, dim=-1)
                pr = torch.exp(s - torch.where(L == -math.inf, 0.0, L)[..., None])
                oo = pr @ vd[js]
                o[b, r:e, h * G:(h + 1) * G] = oo.transpose(0, 1)
                lse[b, h * G:(h + 1) * G, r:e] = L
                if do is not None:
                    dd = do[b, r:e, h * G:(h + 1) * G].double().transpose(0, 1)
                    ds = pr * (dd @ vd[js].T - (dd * oo).sum(-1, keepdim=True)) / math.sqrt(D)
                    grads[0][b, r:e, h * G:(h + 1) * G] = (ds @ kd[js]).transpose(0, 1)
                    grads[1][b, :, h].index_add_(0, js, torch.einsum("grn,grd->nd", ds, qd))
                    grads[2][b, :, h].index_add_(0, js, torch.einsum("grn,grd->nd", pr, dd))
    return (o, lse) if do is None else (o, lse, *grads)
