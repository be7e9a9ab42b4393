"""GPU tests of the K/V cache in 4 or 8 bits: what is written and read back
equals the fp64 oracle's values to the bit; attention over it is checked
element by element against the fp64 oracle on the held values, within the
bounds of window_bounds.py: the kernel's products take the held whole numbers
exactly, its scores are fp32 sums of 128 terms, and it rounds the weights
(times V's scale) and O to bf16, as the other windowed kernels do.

The form for many query rows ("tiles") also rounds what it multiplies:
  V, where sixteen keys' scales allow it, to fp16 over 2^12: by 2^-12 |v|, or below fp16's normal numbers by 2^-25 times
    2^12. There the scales are 2^-7 or more in 4 bits, 2^-11 in 8, so a group's largest value `top` is 7 * 2^-7 or
    127 * 2^-11 at least, but for the half a step by which bf16 may have rounded its scale up, and 2^-13 is at most
    top / 400. Otherwise to bf16, by U |v|. Either way by dv = max(U |v|, min(2^-13, top / 400)) at most.
  the weights to fp16 with them: 2^-12 of each, or 2^-25 over the 2^7 by which they are raised, of a sum that is 1 at
    least: 2^-32 of each key's |v| more. So O is within U |O| + (U + E) (P |V|) + P dV + 2^-32 sum |v|.
  K in 8 bits, of which the magnitude's lower 4 bits times the scale go to fp16:
    by 2^-12 * 15 s <= 2^-12 * 15 / 127 * (the group's largest |k|) (1 + 2^-8) a
    value, so a score by scale * sum_G (sum |q|) top_G 2^-12 * 15 / 127 (1 + 2^-8),
    which is added to E twice, as the score's other error is.
"""

import numpy as np
import pytest
import torch

import oracle
import long_context_causal_blockwise_gb300 as lcb
from parity import to64
from window_bounds import check_attn

pytestmark = pytest.mark.gpu
D = 128
SCALE = D ** -0.5
BF16 = torch.bfloat16


def _rand(seed, *shapes):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(s, generator=g, device="cuda").to(BF16) for s in shapes]


def _lens(*n):
    return torch.tensor(n, dtype=torch.int32, device="cuda")


def _held(x, bits):
    return oracle.cache_values(to64(x), bits)


def _same(got, want):
    """bf16 tensor against fp64 values: equal after their one rounding (a zero's sign aside; NaN where NaN)."""
    want = torch.from_numpy(np.ascontiguousarray(want)).to(BF16).double().numpy()
    got = to64(got)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


def _filled(seed, B, Hkv, Smax, bits, scale=1.0):
    """A full cache and the fp64 K and V that it holds."""
    k, v = _rand(seed, (B, Smax, Hkv, D), (B, Smax, Hkv, D))
    k, v = k * scale, v * scale
    cache = lcb.kv_cache_empty(B, Hkv, Smax, bits=bits)
    lcb.kv_cache_write(cache, k, v, _lens(*[Smax] * B))
    return cache, _held(k, bits), _held(v, bits)


def _check_tiles(q, kd, vd, window, sinks, pos0, o, lse, bits, name):
    """window_bounds.check_attn's comparison with the roundings of the form for many rows; one sequence."""
    r = oracle.window_attn(q, kd, vd, window, sinks, pos0, SCALE)
    G = q.shape[2] // kd.shape[2]
    assert np.isfinite(o).all(), name
    seen = np.isfinite(r["lse"])
    assert np.array_equal(np.isfinite(lse), seen) and (lse[~seen] == -np.inf).all(), name
    for h in range(q.shape[2]):
        kh, vh, qh = np.abs(kd[0, :, h // G]), np.abs(vd[0, :, h // G]), np.abs(q[0, :, h])
        p = r["p"][0, h]
        err = 2 * 128 * 2.0 ** -24 * SCALE * (qh @ kh.T)
        if bits == 8:
            top = kh.reshape(-1, 4, 32).max(axis=2)
            err = err + SCALE * (qh.reshape(-1, 4, 32).sum(axis=2) @ top.T) * 2.0 ** -12 * 15 / 127 * (1 + 2.0 ** -8)
        E = (err * (p > 0)).max(axis=1, initial=0.0)[:, None] * 2 + 2.0 ** -20
        rows = seen[0, h]
        ltol = E[rows, 0] + 2.0 ** -21 * (1 + np.abs(r["lse"][0, h][rows]))
        assert (np.abs(lse[0, h][rows] - r["lse"][0, h][rows]) <= ltol).all(), f"{name} LSE"
        want = r["o"][0, :, h]
        top = np.repeat(vh.reshape(-1, 4, 32).max(axis=2), 32, axis=1)
        dv = np.maximum(2.0 ** -8 * vh, np.minimum(2.0 ** -13, top / 400))
        bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + E) * (p @ vh) + p @ dv + 2.0 ** -32 * vh.sum(axis=0) + 1e-30
        ratio = np.abs(o[0, :, h] - want) / bound
        assert (ratio <= 1).all(), f"{name} O: off by {ratio.max():.2f} bounds"


def _check(q, cache, kd, vd, lens, window, sinks, name="", **kw):
    o, lse = lcb.attn_cache_decode(q, cache, _lens(*lens), window, sinks, **kw)
    torch.cuda.synchronize()
    W = 1 << 30 if window is None else window
    B, T, H, _ = q.shape
    bits = 4 if cache.shape[3] == 144 else 8
    form = lcb.attn_cache_decode_form(B, H, cache.shape[1], T, cache.shape[2], bits, window, sinks)
    for b, n in enumerate(lens):
        n = min(max(n, 0), kd.shape[1])
        if form == "tiles":
            _check_tiles(to64(q[b:b + 1]), kd[b:b + 1, :n], vd[b:b + 1, :n], W, sinks, n - T, to64(o[b:b + 1]),
                         to64(lse[b:b + 1]), bits, f"{name} sequence {b}")
            continue
        check_attn(to64(q[b:b + 1]), kd[b:b + 1, :n], vd[b:b + 1, :n], W, sinks, n - q.shape[1], SCALE,
                   to64(o[b:b + 1]), to64(lse[b:b + 1]), name=f"{name} sequence {b}")
    return o, lse


# ------------------------------------------------------------------ written and read back


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("B,T,Hkv,Smax,lens", [
    (1, 1, 1, 1, (1,)),
    (1, 1, 32, 40, (17,)),
    (2, 9, 3, 30, (9, 30)),
    (3, 33, 5, 64, (64, 40, 33)),
    (3, 20, 2, 50, (7, 0, 20)),        # padded on the left: 13 tokens dropped, all, none
    (2, 20, 2, 30, (35, 60)),          # past the cache: the last five dropped, all
    (2, 40, 1, 16, (20, 30)),          # both ends
    (2, 5, 2, 16, (-3, 2 ** 31 - 1)),  # nothing
    (1, 3, 2, 16, (-2 ** 31,)),
])
def test_write_and_read(bits, B, T, Hkv, Smax, lens):
    k, v = _rand(T + Smax, (B, T, Hkv, D), (B, T, Hkv, D))
    cache = lcb.kv_cache_empty(B, Hkv, Smax, bits=bits).fill_(0xA5)
    before = cache.clone()
    assert lcb.kv_cache_write(cache, k, v, _lens(*lens)) is cache
    kr, vr = lcb.kv_cache_read(cache, Smax)
    torch.cuda.synchronize()
    kd, vd = _held(k, bits), _held(v, bits)
    for b, n in enumerate(lens):
        at = [(n - T + t, t) for t in range(T) if 0 <= n - T + t < Smax]
        rows, toks = [r for r, _ in at], [t for _, t in at]
        _same(kr[b, rows], kd[b, toks])
        _same(vr[b, rows], vd[b, toks])
        others = [r for r in range(Smax) if r not in rows]
        assert torch.equal(cache[b][:, others], before[b][:, others])


@pytest.mark.parametrize("bits", [4, 8])
def test_values_where_rounding_is_tight(bits):
    """Ties, every pair of significands, tiny and huge groups, zeros, and groups with infinities or NaN."""
    m = 7 if bits == 4 else 127
    x = torch.zeros(512, D, dtype=torch.float64)
    S = torch.arange(128, 256, dtype=torch.float64)
    for i in range(128):  # scale S[i] (as near as bf16 has it): ties (j + 1/2) S and the significands around them
        x[i, 0] = m * S[i]
        x[i, 1:32] = (torch.arange(31) % m + 0.5) * S[i] * (-1) ** i
        x[i, 32] = -m * 128.0
        x[i, 33:64] = 128.0 * (i / 128.0) + torch.arange(31)
        x[i, 64] = m * 2.0
        x[i, 65:96] = (torch.arange(31) + 0.5) / 4
        x[i, 96:] = S.roll(i)[:32] * 2.0 ** (i % 9)
    g = torch.Generator().manual_seed(bits)
    x[128:384] = torch.randn(256, D, generator=g, dtype=torch.float64) * 2.0 ** torch.randint(-140, 120, (256, 1), generator=g)
    x[384:448] = torch.randn(64, D, generator=g, dtype=torch.float64) * 2.0 ** -100
    x[448, 5] = float("inf")
    x[449, 40] = float("-inf")
    x[450, 127] = float("nan")
    x[451, 0] = torch.finfo(BF16).min
    x[452] = torch.finfo(BF16).max
    x[453:500] = torch.randn(47, D, generator=g, dtype=torch.float64).sign() * 2.0 ** torch.arange(47)[:, None]
    x = x.to(BF16).cuda()
    k, v = x.view(1, 512, 1, D), x.flip(0).view(1, 512, 1, D)
    cache = lcb.kv_cache_write(lcb.kv_cache_empty(1, 1, 512, bits=bits), k, v, _lens(512))
    kr, vr = lcb.kv_cache_read(cache, 512)
    torch.cuda.synchronize()
    _same(kr, _held(k, bits))
    _same(vr, _held(v, bits))


@pytest.mark.parametrize("bits", [4, 8])
def test_views(bits):
    """K and V as slices of a fused projection, part of a larger cache, and outputs between other rows."""
    B, T, Hkv, Smax = 3, 21, 4, 37
    qkv, = _rand(0, (B, T + 2, 3 * Hkv, D))
    k, v = qkv[:, 1:-1, Hkv:2 * Hkv], qkv[:, 1:-1, 2 * Hkv:]
    big = lcb.kv_cache_empty(B + 2, Hkv + 3, Smax, bits=bits).fill_(7)
    cache = big[1:-1, 2:-1]
    lcb.kv_cache_write(cache, k, v, _lens(30, 21, 37))
    out = torch.full((B, 2 * T, 2 * Hkv + 1, D), 3.0, device="cuda", dtype=BF16)
    ko, vo = out[:, :T, :Hkv], out[:, T:, Hkv:2 * Hkv]
    lcb.kv_cache_read(cache, T, start=9, lens=_lens(30, 21, 37), k=ko, v=vo)
    torch.cuda.synchronize()
    kd, vd = np.zeros((B, Smax, Hkv, D)), np.zeros((B, Smax, Hkv, D))
    for b, n in enumerate((30, 21, 37)):
        kd[b, n - T:n], vd[b, n - T:n] = _held(k[b], bits), _held(v[b], bits)
    # sequence 2 begins at row 16: what lies before is the filling
    _same(ko[:2], kd[:2, 9:9 + T])
    _same(vo[:2], vd[:2, 9:9 + T])
    _same(ko[2, 7:], kd[2, 16:9 + T])
    _same(vo[2, 7:], vd[2, 16:9 + T])
    assert (out[:, :T, Hkv:] == 3).all() and (out[:, T:, :Hkv] == 3).all() and (out[:, T:, 2 * Hkv:] == 3).all()
    untouched = torch.ones(B + 2, Hkv + 3, dtype=torch.bool, device="cuda")
    untouched[1:-1, 2:-1] = False
    assert (big[untouched] == 7).all()
    q, = _rand(1, (B, 1, 2 * Hkv, D))
    _check(q[:2], cache[:2], kd[:2], vd[:2], (30, 21), 12, 0)  # the windows lie within what was written


def test_read_past_the_end_is_zero():
    cache, kd, vd = _filled(3, 3, 2, 50, 4)
    k, v = torch.full((2, 3, 40, 2, D), float("nan"), device="cuda", dtype=BF16)
    lcb.kv_cache_read(cache, 40, start=5, lens=_lens(0, 20, 99), k=k, v=v)
    torch.cuda.synchronize()
    assert (k[0] == 0).all() and (v[0] == 0).all() and (k[1, 15:] == 0).all() and (v[1, 15:] == 0).all()
    _same(k[1, :15], kd[1, 5:20])
    _same(v[2], vd[2, 5:45])
    lcb.kv_cache_read(cache, 40, start=5, lens=_lens(-7, -2 ** 31, 2 ** 31 - 1), k=k, v=v)
    torch.cuda.synchronize()
    assert (k[:2] == 0).all() and torch.equal(torch.isnan(v), torch.zeros_like(v, dtype=torch.bool))
    _same(k[2], kd[2, 5:45])


# ------------------------------------------------------------------ attention

# B, H, Hkv, T, Smax, lens, window, sinks
CASES = [
    (1, 1, 1, 1, 1, (1,), None, 0),
    (1, 2, 2, 1, 300, (300,), None, 0),
    (2, 4, 1, 1, 100, (16, 17), None, 0),         # at and past a step of 16 keys
    (3, 2, 2, 1, 100, (31, 32, 33), None, 0),     # around a unit of 32
    (3, 8, 2, 2, 500, (1, 2, 500), 40, 3),        # a token before the first row; a window with sinks
    (2, 4, 4, 3, 64, (0, -5), None, 0),           # nothing in the cache
    (2, 4, 2, 1, 64, (1000, 64), None, 2),        # lengths past the cache
    (1, 8, 1, 1, 1111, (1050,), None, 0),         # eight query rows
    (1, 9, 1, 1, 1111, (1111,), None, 0),         # nine
    (1, 16, 1, 1, 700, (650,), 1, 0),             # every row sees itself alone
    (1, 16, 2, 2, 700, (699,), 300, 17),
    (2, 8, 1, 7, 400, (400, 5), 100, 30),         # rows of several tiles, the second sequence's first two see nothing
    (1, 40, 8, 16, 900, (900,), None, 0),         # tiles that begin inside a token's group of heads
    (1, 4, 4, 70, 300, (290,), 33, 5),            # many tokens
    (1, 32, 8, 1, 5000, (4999,), None, 0),
    (2, 2, 1, 4, 3001, (3001, 1777), 2000, 129),  # sinks over several units
    (1, 2, 2, 2, 600, (600,), 10, 10 ** 9),       # every key a sink
    (5, 40, 40, 1, 257, (257, 1, 100, 33, 16), 2 ** 31 - 1, 0),
]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("B,H,Hkv,T,Smax,lens,window,sinks", CASES)
def test_attention_vs_oracle(bits, B, H, Hkv, T, Smax, lens, window, sinks):
    cache, kd, vd = _filled(Smax + T, B, Hkv, Smax, bits)
    q, = _rand(H, (B, T, H, D))
    _check(q, cache, kd, vd, lens, window, sinks)
    _check(4 * q, cache, kd, vd, lens, window, sinks, "sharp")


# Sizes that take each form on a GB300: B, H, Hkv, T, Smax, lens, window, sinks
FORMS = [
    ("cluster", 1, 32, 32, 1, 777, (777,), None, 0),
    ("cluster", 3, 12, 4, 5, 700, (700, 650, 3), 333, 40),      # 15 rows
    ("line", 1, 1, 1, 1, 60000, (59999,), None, 0),             # one head: 152 CTAs share it
    ("line", 2, 8, 2, 1, 30000, (30000, 1), None, 0),
    ("line", 2, 12, 2, 1, 30011, (30011, 17000), 29000, 300),   # six rows; sinks over several units
    ("line", 1, 16, 1, 1, 80000, (80000,), None, 0),            # sixteen rows
    ("line", 3, 4, 1, 2, 30000, (12345, 0, 30000), None, 0),    # eight rows; a sequence without keys
    ("line", 5, 2, 1, 2, 30000, (30000, 100, 7, 9000, 1), 25000, 3),
    ("tiles", 1, 8, 2, 32, 12000, (11999,), None, 0),           # 128 rows
    ("tiles", 2, 8, 1, 9, 20000, (20000, 1501), None, 0),       # 72
    ("tiles", 2, 4, 2, 200, 3000, (3000, 150), 2000, 129),      # four row tiles, tokens before the first row
    ("tiles", 3, 3, 3, 130, 3500, (3500, 0, 129), None, 5),     # two, the second with two rows; a sequence without keys
    ("tiles", 1, 24, 1, 2, 150000, (149999,), None, 0),         # 48 rows, many keys
    ("line", 3, 8, 2, 1, 30000, (40000, -7, 29000), None, 0),   # lengths past the cache and below zero
    ("line", 2, 8, 2, 1, 30000, (2 ** 31 - 1, 30000), None, 0),
    ("tiles", 3, 8, 1, 9, 20000, (30000, -2 ** 31, 19000), None, 0),
    ("tiles", 1, 2, 1, 3500, 3600, (5000,), 300, 7),            # more row tiles than a warp has lanes
]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("form,B,H,Hkv,T,Smax,lens,window,sinks", FORMS)
def test_each_form_vs_oracle(form, bits, B, H, Hkv, T, Smax, lens, window, sinks):
    assert lcb.attn_cache_decode_form(B, H, Hkv, T, Smax, bits, window, sinks) == form
    cache, kd, vd = _filled(Smax + T, B, Hkv, Smax, bits)
    q, = _rand(H, (B, T, H, D))
    a = _check(q, cache, kd, vd, lens, window, sinks)
    for _ in range(3):
        b = lcb.attn_cache_decode(q, cache, _lens(*lens), window, sinks)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    _check(6 * q, cache, kd, vd, lens, window, sinks, "sharp")
    # a given workspace, of any contents
    n = lcb.attn_cache_decode_workspace_bytes(B, H, Hkv, T, Smax, bits, window, sinks)
    assert (n > 0) == (form != "cluster")
    ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    b = lcb.attn_cache_decode(q, cache, _lens(*lens), window, sinks, workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    if n:
        with pytest.raises(lcb.AttnError):
            lcb.attn_cache_decode(q, cache, _lens(*lens), window, sinks, workspace=ws[:n - 16])


@pytest.mark.parametrize("bits", [4, 8])
def test_attention_does_not_read_what_is_hidden(bits):
    """Rows past the end, before the window, or of positions after a query's: any bytes there change nothing."""
    B, H, Hkv, T, Smax = 2, 8, 2, 3, 777
    cache, kd, vd = _filled(5, B, Hkv, Smax, bits)
    q, = _rand(6, (B, T, H, D))
    for lens, window, sinks in (((700, 401), 300, 5), ((640, 33), None, 0), ((2, 700), 50, 40)):
        want = _check(q, cache, kd, vd, lens, window, sinks)
        dirty = cache.clone()
        for b, n in enumerate(lens):
            dirty[b, :, n:] = 0xFF  # scales of NaN
            if window:
                dirty[b, :, min(sinks, max(0, n - T - window + 1)):max(0, n - T - window + 1)] = 0xFF
        got = lcb.attn_cache_decode(q, dirty, _lens(*lens), window, sinks)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        # NaN in the newest row: the last token sees it, the others do not; NaN in the oldest row of the first token's
        # window: the others do not see it
        for b, n in enumerate(lens):
            if n > T:
                dirty[b, 0, n - 1] = 0xFF
        o, lse = lcb.attn_cache_decode(q, dirty, _lens(*lens), window, sinks)
        for b, n in enumerate(lens):
            if n <= T:
                continue
            G = H // Hkv
            assert torch.isnan(o[b, -1, :G]).all() and torch.isnan(lse[b, :G, -1]).all()
            assert torch.equal(o[b, :-1], want[0][b, :-1]) and torch.equal(o[b, -1, G:], want[0][b, -1, G:])
            assert torch.equal(lse[b, :, :-1], want[1][b, :, :-1])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("kscale,vscale", [(1.0, 2.0 ** -90), (1.0, 2.0 ** 100), (2.0 ** -60, 1.0), (2.0 ** 60, 1.0)])
def test_attention_over_the_range_of_values(bits, kscale, vscale):
    """K and V far from 1 (Q makes up for K): nothing overflows or loses its precision on the way."""
    B, H, Hkv, T, Smax = 1, 6, 2, 2, 900
    k, v, q = _rand(9, (B, Smax, Hkv, D), (B, Smax, Hkv, D), (B, T, H, D))
    k, v, q = k * kscale, v * vscale, q / kscale
    cache = lcb.kv_cache_write(lcb.kv_cache_empty(B, Hkv, Smax, bits=bits), k, v, _lens(Smax))
    _check(q, cache, _held(k, bits), _held(v, bits), (Smax,), 700, 4)


SOME = [("line", 2, 12, 2, 1, 30011), ("line", 1, 2, 1, 1, 40000), ("tiles", 1, 8, 2, 32, 12000), ("tiles", 2, 8, 1, 9, 20000)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("which", ["small V", "large V", "small K", "large K", "V of all sizes", "V grows", "small groups"])
@pytest.mark.parametrize("form,B,H,Hkv,T,Smax", SOME)
def test_each_form_over_the_range_of_values(form, B, H, Hkv, T, Smax, which, bits):
    """As above in the other forms, and V whose sizes change from key to key, along the keys, and among channels."""
    assert lcb.attn_cache_decode_form(B, H, Hkv, T, Smax, bits) == form
    k, v, q = _rand(10, (B, Smax, Hkv, D), (B, Smax, Hkv, D), (B, T, H, D))
    g = torch.Generator(device="cuda").manual_seed(11)
    if which == "small V":
        v = v * 2.0 ** -90
    elif which == "large V":
        v = v * 2.0 ** 95
    elif which in ("small K", "large K"):
        f = 2.0 ** (-60 if which == "small K" else 60)
        k, q = k * f, q / f
    elif which == "V of all sizes":
        v = v * torch.exp2(torch.randint(-30, 30, (B, Smax, Hkv, 1), generator=g, device="cuda").float()).to(BF16)
    elif which == "V grows":
        v = v * torch.exp2((torch.arange(Smax, device="cuda") * 80 // Smax - 40).float()).to(BF16)[None, :, None, None]
    else:
        v = v * torch.exp2(-torch.arange(D, device="cuda") // 32 * 5.0).to(BF16)
    cache = lcb.kv_cache_write(lcb.kv_cache_empty(B, Hkv, Smax, bits=bits), k, v, _lens(*[Smax] * B))
    _check(q, cache, _held(k, bits), _held(v, bits), [Smax] * B, None, 0, which)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("form,B,H,Hkv,T,Smax,lens,window,sinks", [
    ("line", 2, 12, 2, 2, 30011, (29000, 17001), 20000, 300),
    ("line", 1, 16, 1, 1, 80000, (79990,), 70001, 5),
    ("tiles", 1, 8, 2, 32, 12000, (11500,), 9001, 3),
    ("tiles", 2, 8, 1, 9, 20000, (19999, 19001), 18000, 129),
    ("tiles", 2, 4, 2, 200, 4000, (3900, 2500), 2000, 0),
])
def test_each_form_reads_nothing_hidden(form, bits, B, H, Hkv, T, Smax, lens, window, sinks):
    """Rows that no token sees hold NaN; then the newest row does, which the last token alone sees."""
    assert lcb.attn_cache_decode_form(B, H, Hkv, T, Smax, bits, window, sinks) == form
    cache, kd, vd = _filled(7, B, Hkv, Smax, bits)
    q, = _rand(8, (B, T, H, D))
    want = _check(q, cache, kd, vd, lens, window, sinks)
    for b, n in enumerate(lens):
        cache[b, :, n:] = 0xFF
        cache[b, :, sinks:max(sinks, n - T - window + 1)] = 0xFF
    got = lcb.attn_cache_decode(q, cache, _lens(*lens), window, sinks)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for b, n in enumerate(lens):
        cache[b, 0, n - 1, -16:-8] = 0xFF  # K's scales
    o, lse = lcb.attn_cache_decode(q, cache, _lens(*lens), window, sinks)
    G = H // Hkv
    assert torch.isnan(o[:, -1, :G]).all() and torch.isnan(lse[:, :G, -1]).all()
    assert torch.equal(o[:, :-1], want[0][:, :-1]) and torch.equal(o[:, -1, G:], want[0][:, -1, G:])
    assert torch.equal(lse[:, :, :-1], want[1][:, :, :-1]) and torch.equal(lse[:, G:], want[1][:, G:])
    for b, n in enumerate(lens):
        cache[b, 0, n - 1] = 0xFF
    o, lse = lcb.attn_cache_decode(q, cache, _lens(*lens), window, sinks)
    assert torch.isnan(o[:, -1, :G]).all() and torch.isnan(lse[:, :G, -1]).all()
    assert torch.equal(o[:, :, G:], want[0][:, :, G:]) and torch.equal(lse[:, :, :-1], want[1][:, :, :-1])
    assert torch.equal(o[:, :-1], want[0][:, :-1])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("form,B,H,Hkv,T,Smax", [("cluster", 1, 16, 2, 2, 600), ("line", 1, 8, 2, 2, 40000),
                                                 ("tiles", 1, 8, 2, 32, 12000), ("tiles", 2, 8, 1, 9, 20000)])
def test_nan_in_v_stays_in_its_channels_and_rows(form, B, H, Hkv, T, Smax, bits):
    """A NaN among one key's V makes NaN of its group of channels, for the tokens that see the key."""
    assert lcb.attn_cache_decode_form(B, H, Hkv, T, Smax, bits) == form
    k, v = _rand(80, (B, Smax, Hkv, D), (B, Smax, Hkv, D))
    q, = _rand(81, (B, T, H, D))
    lens = _lens(*[Smax] * B)
    cache = lcb.kv_cache_write(lcb.kv_cache_empty(B, Hkv, Smax, bits=bits), k, v, lens)
    want = lcb.attn_cache_decode(q, cache, lens)
    G = H // Hkv
    for key, channel, first in ((Smax - T + 1, 70, 1), (Smax - 1, 0, T - 1), (Smax // 2 + 3, 127, 0)):
        bad = v.clone()
        bad[0, key, -1, channel] = float("inf") if channel else float("nan")
        lcb.kv_cache_write(cache, k, bad, lens)
        o, lse = lcb.attn_cache_decode(q, cache, lens)
        nan = torch.zeros_like(o, dtype=torch.bool)
        nan[0, first:, -G:, channel // 32 * 32:channel // 32 * 32 + 32] = True
        assert torch.equal(torch.isnan(o), nan) and not torch.isnan(lse).any()
        # (the step's other V are rounded to bf16 then, in the form for many rows)
        torch.testing.assert_close(o[~nan].float(), want[0][~nan].float(), rtol=2.0 ** -6, atol=2.0 ** -8)
        torch.testing.assert_close(lse, want[1], rtol=0, atol=2.0 ** -20)


def test_more_sequences_than_the_line_holds():
    """Above 1024 sequences of any length: checked against the same sequences in calls of their own."""
    B, H, Hkv, T, Smax = 1300, 4, 2, 2, 260
    cache, kd, vd = _filled(23, B, Hkv, Smax, 4)
    q, = _rand(24, (B, T, H, D))
    lens = [(37 * b) % (Smax + 20) for b in range(B)]
    o, lse = lcb.attn_cache_decode(q, cache, _lens(*lens), 200, 3)
    for b in (0, 1, 511, 1024, 1299):
        _check(q[b:b + 1], cache[b:b + 1], kd[b:b + 1], vd[b:b + 1], [lens[b]], 200, 3)
    for s in range(0, B, 1000):
        a = lcb.attn_cache_decode(q[s:s + 1000], cache[s:s + 1000], _lens(*lens[s:s + 1000]), 200, 3)
        torch.testing.assert_close(o[s:s + 1000].float(), a[0].float(), rtol=2 ** -6, atol=2 ** -6)


def test_infinite_and_nan_queries_stay_in_their_rows():
    cache, kd, vd = _filled(11, 1, 2, 200, 4)
    q, = _rand(12, (1, 3, 8, D))
    want = lcb.attn_cache_decode(q, cache, _lens(200))
    q[0, 1, 3, 7] = float("inf")
    q[0, 2, 5, 100] = float("nan")
    o, lse = lcb.attn_cache_decode(q, cache, _lens(200))
    keep = torch.ones(3, 8, dtype=torch.bool, device="cuda")
    keep[1, 3] = keep[2, 5] = False
    assert torch.equal(o[0][keep], want[0][0][keep]) and torch.equal(lse[0].T[keep], want[1][0].T[keep])


def test_views_of_queries_and_outputs():
    B, H, Hkv, T, Smax = 2, 8, 4, 3, 150
    cache, kd, vd = _filled(13, B, Hkv, Smax, 4)
    qkv, = _rand(14, (B, T, 3 * H, D))
    q = qkv[:, :, H:2 * H]
    out = torch.full((B, T, 2 * H, D), 5.0, device="cuda", dtype=BF16)
    st = torch.full((B, 2 * H, T + 4), 5.0, device="cuda")
    o, lse = lcb.attn_cache_decode(q, cache, _lens(150, 77), o=out[:, :, :H], lse=st[:, H:, :T])
    want = _check(q.contiguous(), cache, kd, vd, (150, 77), None, 0)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert (out[:, :, H:] == 5).all() and (st[:, :H] == 5).all() and (st[:, :, T:] == 5).all()


@pytest.mark.parametrize("bits", [4, 8])
def test_rows_beyond_32_bits(bits):
    """A cache of more than 4 GB, its last rows written, read and attended to."""
    Smax, T, n = (1 << 25) + 5, 40, (1 << 25) + 1
    cache = torch.empty((1, 1, Smax, 144 if bits == 4 else 272), dtype=torch.uint8, device="cuda")
    k, v, q = _rand(15, (1, T, 1, D), (1, T, 1, D), (1, 2, 3, D))
    lcb.kv_cache_write(cache, k, v, _lens(n))
    kr, vr = lcb.kv_cache_read(cache, T, start=n - T)
    torch.cuda.synchronize()
    kd, vd = _held(k, bits), _held(v, bits)
    _same(kr, kd)
    _same(vr, vd)
    o, lse = lcb.attn_cache_decode(q, cache, _lens(n), window=30)
    check_attn(to64(q), kd, vd, 30, 0, T - 2, SCALE, to64(o), to64(lse))


# ------------------------------------------------------------------ the calls together


@pytest.mark.parametrize("bits", [4, 8])
def test_prompt_then_decoding(bits):
    """Prompts of unequal length, padded on the left; then tokens one at a time; each step against the oracle."""
    B, H, Hkv, Smax, T = 3, 8, 4, 120, 50
    first = [50, 31, 1]
    k, v, q = _rand(17, (B, T + 6, Hkv, D), (B, T + 6, Hkv, D), (B, T + 6, H, D))
    cache = lcb.kv_cache_empty(B, Hkv, Smax, bits=bits).fill_(0xFF)
    kd, vd = np.zeros((B, Smax, Hkv, D)), np.zeros((B, Smax, Hkv, D))
    lens = _lens(*first)
    lcb.kv_cache_write(cache, k[:, :T], v[:, :T], lens)
    for b, n in enumerate(first):
        kd[b, :n], vd[b, :n] = _held(k[b, T - n:T], bits), _held(v[b, T - n:T], bits)
    _check(q[:, :T].contiguous(), cache, kd, vd, first, 40, 4, "prompt")
    for i in range(6):
        lens += 1
        new = slice(T + i, T + i + 1)
        lcb.kv_cache_write(cache, k[:, new], v[:, new], lens)
        now = [n + i + 1 for n in first]
        for b, n in enumerate(now):
            kd[b, n - 1], vd[b, n - 1] = _held(k[b, T + i], bits), _held(v[b, T + i], bits)
        _check(q[:, new].contiguous(), cache, kd, vd, now, 40, 4, f"token {i}")


def test_chunked_prompt_through_the_cache():
    """A prompt's chunks: written, the rows so far read back, and attention in bf16 over them; the same queries over the
    cache itself differ by the rounding of the held values to bf16, at most half a step of each score's terms and V."""
    B, H, Hkv, S, chunk = 1, 8, 2, 700, 256
    k, v, q = _rand(19, (B, S, Hkv, D), (B, S, Hkv, D), (B, S, H, D))
    cache = lcb.kv_cache_empty(B, Hkv, S, bits=8)
    for s in range(0, S, chunk):
        e = min(S, s + chunk)
        lcb.kv_cache_write(cache, k[:, s:e], v[:, s:e], _lens(e))
        kk, vv = lcb.kv_cache_read(cache, e)
        o, lse = lcb.attn_window_fwd(q[:, s:e].contiguous(), kk, vv, window=300, sinks=4)
        torch.cuda.synchronize()
        check_attn(to64(q[:, s:e]), to64(kk), to64(vv), 300, 4, s, SCALE, to64(o), to64(lse))
        _check(q[:, s:e].contiguous(), cache, _held(k, 8), _held(v, 8), (e,), 300, 4)


@pytest.mark.parametrize("B,H,Hkv,Smax", [(2, 8, 2, 900), (1, 1, 1, 60000), (1, 8, 8, 20000), (1, 64, 2, 20000)])
def test_repeated_captured_and_on_another_stream(B, H, Hkv, Smax):
    """The same bits every time; a captured step replays with the lengths and tokens of the moment."""
    cache, kd, vd = _filled(21, B, Hkv, Smax, 4)
    q, k, v = _rand(22, (B, 1, H, D), (B, 1, Hkv, D), (B, 1, Hkv, D))
    lens = _lens(*[Smax // 2] * B)
    o, lse = torch.empty_like(q), torch.empty(B, H, 1, device="cuda")

    def step():
        lens.add_(1)
        lcb.kv_cache_write(cache, k, v, lens)
        lcb.attn_cache_decode(q, cache, lens, o=o, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    kd[:, Smax // 2], vd[:, Smax // 2] = _held(k[:, 0], 4), _held(v[:, 0], 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        q.copy_(_rand(30 + i, q.shape)[0])
        k.copy_(_rand(40 + i, k.shape)[0])
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone(), lse.clone()
        for _ in range(2):
            again = lcb.attn_cache_decode(q, cache, lens)
            assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
        n = Smax // 2 + 2 + i
        kd[:, n - 1] = _held(k[:, 0], 4)
        vd[:, n - 1] = _held(v[:, 0], 4)
        _check(q, cache, kd, vd, [n] * B, None, 0)
    assert lens.tolist() == [Smax // 2 + 4] * B


@pytest.mark.parametrize("H", [4, 64])
def test_two_calls_at_once(H):
    """Calls that overlap on two streams, each with buffers of its own; then two captured ones, replayed together."""
    sets = []
    for i in range(2):
        cache, kd, vd = _filled(50 + i, 1, 2, 40000, 4)
        q, = _rand(60 + i, (1, 2, H, D))
        sets.append((cache, kd, vd, q, torch.cuda.Stream(), []))
    assert lcb.attn_cache_decode_form(1, H, 2, 2, 40000) == ("line" if H == 4 else "tiles")
    lens = _lens(40000)
    torch.cuda.synchronize()
    for _ in range(10):
        for cache, _, _, q, stream, out in sets:
            with torch.cuda.stream(stream):
                out.append(lcb.attn_cache_decode(q, cache, lens))
    torch.cuda.synchronize()
    graphs = []
    for cache, _, _, q, stream, out in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out.append(lcb.attn_cache_decode(q, cache, lens))
        graphs.append(graph)
    for _ in range(10):
        for graph, (_, _, _, _, stream, _) in zip(graphs, sets):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for cache, kd, vd, q, _, out in sets:
        want = _check(q, cache, kd, vd, (40000,), None, 0)
        assert all(torch.equal(o, want[0]) and torch.equal(lse, want[1]) for o, lse in out)


def test_wrong_devices():
    cache, _, _ = _filled(70, 1, 2, 64, 4)
    k, v, q = _rand(71, (1, 3, 2, D), (1, 3, 2, D), (1, 3, 4, D))
    lens = _lens(64)
    for call in (lambda: lcb.kv_cache_write(cache, k.cpu(), v, lens), lambda: lcb.kv_cache_write(cache, k, v, lens.cpu()),
                 lambda: lcb.kv_cache_write(cache.cpu(), k, v, lens), lambda: lcb.kv_cache_read(cache.cpu(), 3),
                 lambda: lcb.kv_cache_read(cache, 3, lens=lens.cpu()), lambda: lcb.attn_cache_decode(q.cpu(), cache, lens),
                 lambda: lcb.attn_cache_decode(q, cache, lens.cpu()), lambda: lcb.attn_cache_decode(q, cache.cpu(), lens),
                 lambda: lcb.attn_cache_decode(q, cache, lens, o=q.cpu())):
        with pytest.raises((ValueError, lcb.AttnError)):
            call()
