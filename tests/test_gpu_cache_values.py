"""GPU tests of attn_cache_decode over the range of values, in each of its forms
and each of their layouts (4, 8 and 16 query rows a tile, 128 in the form for many
rows): K whose sizes differ from key to key and among channels, zeros, very large
Q, K and V, and values that a row does not see.

Bounds. A pair's score is off by at most d = 2 * 128 * 2^-24 * scale * |q| |k|
(window_bounds.py; in 8 bits in the form for many rows 2^-12 of K's lower four bits
more, test_gpu_kv_cache.py; and scale * 2^-36 max |q| sum |k|, as Q goes to fp16 with
its largest element at 2^15, or 2^11 for half of the channels), so its weight by a factor between e^-d and e^d. With
w = e^d - 1 and z = sum p w + 2^-20 (ex2.approx and the sums), the sum of weights is
off by z at most, and where z <= 1/2
  |dLSE| <= 2 z + 2^-21 (1 + |LSE|)
  |dO| <= U |O| + U (p |V|) + 2 z (p |V|) + (1 + 2 z) (p w |V|)
plus, in the form for many rows, its p dV and 2^-32 of each visible |v|. Of rows with a
larger z (a key whose score is in the thousands) O has to be finite, and the LSE off
by the largest d at most. Rows that do not see what was changed keep their bits.
The references are the oracle's formulas in fp64 on the GPU (the host takes seconds
for each of these sizes).
"""

import numpy as np
import pytest
import torch

import oracle
import long_context_causal_blockwise_gb300 as lcb
from parity import to64

pytestmark = pytest.mark.gpu
D = 128
SCALE = D ** -0.5
BF16 = torch.bfloat16
U = 2.0 ** -8

# form, B, H, Hkv, T, Smax: T * H / Hkv rows a K/V head
FORMS = [
    ("cluster", 1, 8, 8, 3, 700),      # 3
    ("cluster", 1, 8, 4, 3, 700),      # 6
    ("cluster", 1, 16, 2, 2, 600),     # 16
    ("line", 1, 2, 1, 2, 40000),       # 4
    ("line", 1, 8, 2, 2, 40000),       # 8
    ("line", 1, 8, 1, 2, 80000),       # 16
    ("tiles", 1, 8, 2, 32, 12000),     # 128
    ("tiles", 2, 8, 1, 9, 20000),      # 72
]
each_form = pytest.mark.parametrize("form,B,H,Hkv,T,Smax", FORMS)
both_bits = pytest.mark.parametrize("bits", [4, 8])


def _rand(seed, *shapes):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(s, generator=g, device="cuda") for s in shapes]


def _lens(*n):
    return torch.tensor(n, dtype=torch.int32, device="cuda")


def _cache(k, v, bits):
    B, Smax, Hkv, _ = k.shape
    return lcb.kv_cache_write(lcb.kv_cache_empty(B, Hkv, Smax, bits=bits), k, v, _lens(*[Smax] * B))


def _held(x, bits):
    """The values that the cache holds for finite x [..., 128], fp64 on the GPU (the oracle's definition)."""
    g = x.double().unflatten(-1, (4, 32))
    top = g.abs().amax(dim=-1, keepdim=True)
    s = torch.where(top < 2.0 ** -100, 0.0, (top / (2 ** (bits - 1) - 1)).to(BF16).double())
    n = torch.floor(g.abs() / torch.where(s == 0, 1.0, s) + 0.5) * g.sign()
    return (torch.where(s == 0, 0.0, n) * s).flatten(-2)


def _attn(q, k, v, window, sinks, pos0, scale):
    """(o, lse, p) of one head, fp64: q [T, 128], k and v [n, 128]."""
    p, j = pos0 + torch.arange(len(q), device="cuda")[:, None], torch.arange(len(k), device="cuda")[None]
    x = (scale * (q @ k.T)).masked_fill(~((j <= p) & ((p - j < window) | (j < sinks))), -torch.inf)
    lse = torch.logsumexp(x, dim=1)
    p = torch.exp(x - lse[:, None].masked_fill(lse[:, None].isinf(), 0.0))
    return p @ v, lse, p


def test_these_are_the_oracles():
    q, k, v = [x.to(BF16) for x in _rand(0, (1, 5, 1, D), (1, 50, 1, D), (1, 50, 1, D))]
    k[0, 3, 0, 32:64] = 0
    for bits in (4, 8):
        kd, vd = _held(k, bits), _held(v, bits)
        assert np.array_equal(kd.cpu().numpy(), oracle.cache_values(to64(k), bits))
        r = oracle.window_attn(to64(q), kd.cpu().numpy(), vd.cpu().numpy(), 20, 3, -2, SCALE)
        o, lse, p = [x.cpu().numpy() for x in _attn(q[0, :, 0].double(), kd[0, :, 0], vd[0, :, 0], 20, 3, -2, SCALE)]
        assert np.allclose(o, r["o"][0, :, 0], atol=1e-12) and np.allclose(lse, r["lse"][0, 0], atol=1e-12)
        assert np.allclose(p, r["p"][0, 0], atol=1e-12)


def _compare(q, kd, vd, window, sinks, pos0, scale, o, lse, bits, form, name):
    """One sequence, all fp64; the rows compared."""
    T, H = q.shape[:2]
    G = H // kd.shape[1]
    compared = 0
    for h in range(H):
        qh, kh, vh = q[:, h], kd[:, h // G], vd[:, h // G]
        want, ref, p = _attn(qh, kh, vh, window, sinks, pos0, scale)
        seen = torch.isfinite(ref)
        assert torch.isfinite(o[:, h]).all(), f"{name} O: non-finite"
        assert torch.equal(torch.isfinite(lse[h]), seen) and (lse[h][~seen] == -torch.inf).all(), f"{name} LSE: empty rows"
        assert (o[:, h][~seen] == 0).all(), f"{name} O: empty rows"
        qh, kh, vh = qh.abs(), kh.abs(), vh.abs()
        d = 2 * 128 * 2.0 ** -24 * scale * (qh @ kh.T) + scale * 2.0 ** -36 * qh.amax(dim=1)[:, None] * kh.sum(dim=1)
        if bits == 8 and form == "tiles":
            top = kh.unflatten(1, (4, 32)).amax(dim=2)
            d = d + scale * (qh.unflatten(1, (4, 32)).sum(dim=2) @ top.T) * 2.0 ** -12 * 15 / 127 * (1 + U)
        w = torch.where(p > 0, torch.expm1(d.clamp(max=100.0)), 0.0)
        z = (p * w).sum(dim=1) + 2.0 ** -20
        use = seen & (z <= 0.5)
        compared += int(use.sum())
        l_tol = torch.where(use, 2 * z, (d * (p > 0)).amax(dim=1) + 2.0 ** -20) + 2.0 ** -21 * (1 + ref.abs())
        l_off = ((lse[h] - ref).abs() / l_tol)[seen]
        assert (l_off <= 1).all(), f"{name} LSE: off by {l_off.max():.2f} bounds"
        want, p, w, z = want[use], p[use], w[use], z[use, None]
        pv = p @ vh
        bound = U * want.abs() + (U + 2 * z) * pv + (1 + 2 * z) * ((p * w) @ vh) + 1e-30
        if form == "tiles":
            top = vh.unflatten(1, (4, 32)).amax(dim=2).repeat_interleave(32, dim=1)
            dv = torch.maximum(U * vh, (top / 400).clamp(max=2.0 ** -13))
            bound += p @ dv + 2.0 ** -32 * ((p > 0).double() @ vh)
        off = (o[:, h][use] - want).abs() / bound
        assert (off <= 1).all(), f"{name} O: off by {off.max():.2f} bounds"
    return compared


def _check(form, bits, q, k, v, lens=None, window=None, sinks=0, scale=SCALE, name="", all_rows=True):
    """The call on a cache of k and v, compared with the oracle on what it holds; its (o, lse)."""
    B, T, H, _ = q.shape
    Smax, Hkv = k.shape[1:3]
    assert lcb.attn_cache_decode_form(B, H, Hkv, T, Smax, bits, window, sinks) == form
    lens = [Smax] * B if lens is None else lens
    cache = _cache(k, v, bits)
    o, lse = lcb.attn_cache_decode(q, cache, _lens(*lens), window, sinks, scale=scale)
    torch.cuda.synchronize()
    kd, vd = _held(k, bits), _held(v, bits)
    W = 1 << 30 if window is None else window
    for b, n in enumerate(lens):
        rows = _compare(q[b].double(), kd[b, :n], vd[b, :n], W, sinks, n - T, scale, o[b].double(), lse[b].double(), bits,
                        form, f"{name} sequence {b}")
        assert rows == H * min(T, n) or not all_rows
    return o, lse


# ------------------------------------------------------------------ K of all sizes


@both_bits
@each_form
def test_large_keys_that_the_queries_turn_away_from(form, B, H, Hkv, T, Smax, bits):
    """Every eighth key is 2^4 to 2^20 times the others, its score far below theirs: the others' weights are what they are
    without it. (Queries of one direction, and large keys of the opposite one.)"""
    k, v, q = _rand(1, (B, Smax, Hkv, D), (B, Smax, Hkv, D), (B, T, H, D))
    base, = _rand(2, (D,))
    q = base + 0.3 * q
    g = torch.Generator(device="cuda").manual_seed(3)
    size = torch.exp2(torch.randint(4, 21, (B, Smax, Hkv, 1), generator=g, device="cuda").float())
    large = torch.arange(Smax, device="cuda")[None, :, None, None] % 8 == 5
    k = torch.where(large, -size * (base + 0.1 * k), k)
    _check(form, bits, q.to(BF16), k.to(BF16), v.to(BF16))


@both_bits
@each_form
def test_a_huge_key_that_only_the_last_token_sees(form, B, H, Hkv, T, Smax, bits):
    """The other tokens' rows keep their bits, whatever stands in the newest key."""
    k, v, q = [x.to(BF16) for x in _rand(4, (B, Smax, Hkv, D), (B, Smax, Hkv, D), (B, T, H, D))]
    want = _check(form, bits, q, k, v)
    lens = _lens(*[Smax] * B)
    for e in (6, 11, 20, 60, 120):
        huge = k.clone()
        huge[:, -1] = (huge[:, -1].float() * 2.0 ** e).to(BF16)
        o, lse = lcb.attn_cache_decode(q, _cache(huge, v, bits), lens)
        assert torch.equal(o[:, :-1], want[0][:, :-1]) and torch.equal(lse[:, :, :-1], want[1][:, :, :-1]), e
    for e in (-9, -30):
        tiny = k.clone()
        tiny[:, -1] = (tiny[:, -1].float() * 2.0 ** e).to(BF16)
        o, lse = lcb.attn_cache_decode(q, _cache(tiny, v, bits), lens)
        assert torch.equal(o[:, :-1], want[0][:, :-1]) and torch.equal(lse[:, :, :-1], want[1][:, :, :-1]), e


@both_bits
@pytest.mark.parametrize("e", [7, 9, 14, 20])
@each_form
def test_a_large_group_of_channels(form, B, H, Hkv, T, Smax, e, bits):
    """K's second group 2^e times the others, where the queries have next to nothing."""
    k, v, q = _rand(5, (B, Smax, Hkv, D), (B, Smax, Hkv, D), (B, T, H, D))
    k[..., 32:64] *= 2.0 ** e
    q[..., 32:64] *= 2.0 ** (-2 * e)
    _check(form, bits, q.to(BF16), k.to(BF16), v.to(BF16))


@both_bits
@each_form
def test_k_and_its_channels_of_all_sizes(form, B, H, Hkv, T, Smax, bits):
    """Powers of two by key and by channel group, the queries' the inverse of the groups', and the keys' below 1."""
    k, v, q = _rand(6, (B, Smax, Hkv, D), (B, Smax, Hkv, D), (B, T, H, D))
    g = torch.Generator(device="cuda").manual_seed(7)
    groups = torch.exp2(torch.tensor([0.0, 6.0, -6.0, 3.0], device="cuda")).repeat_interleave(32)
    k = k * torch.exp2(-torch.randint(0, 16, (B, Smax, Hkv, 1), generator=g, device="cuda").float()) * groups
    _check(form, bits, (q / groups).to(BF16), k.to(BF16), v.to(BF16), lens=[Smax - 5 * b - 3 for b in range(B)],
           window=Smax - 99, sinks=5)


# ------------------------------------------------------------------ very large K, Q and V


@both_bits
@pytest.mark.parametrize("e", [100, 119, 123])
@each_form
def test_very_large_keys(form, B, H, Hkv, T, Smax, e, bits):
    """K up to 2^125, and Q that makes up for it."""
    k, v, q = _rand(8, (B, Smax, Hkv, D), (B, Smax, Hkv, D), (B, T, H, D))
    _check(form, bits, (q * 2.0 ** -e).to(BF16), (k * 2.0 ** e).to(BF16), v.to(BF16))


# ------------------------------------------------------------------ zeros


@both_bits
@pytest.mark.parametrize("zero", ["q", "k", "both", "a row", "small q", "some k"])
@each_form
def test_zeros(form, B, H, Hkv, T, Smax, zero, bits):
    """Queries, keys or both of zeros: every visible key has the same weight. Lengths that end inside sixteen keys, and a
    window that begins inside."""
    k, v, q = _rand(9, (B, Smax, Hkv, D), (B, Smax, Hkv, D), (B, T, H, D))
    if zero in ("q", "both"):
        q.zero_()
    if zero in ("k", "both", "small q"):
        k.zero_()
    if zero == "a row":
        q[:, 0].zero_()
        k.zero_()
    if zero == "small q":
        q *= 2.0 ** -100
    if zero == "some k":
        q[:, :, ::2].zero_()
        k[:, ::3].zero_()
        k[:, -40:].zero_()
    lens = [Smax - 7 - 20 * b for b in range(B)]
    for window, sinks in ((None, 0), (Smax - 77, 3)):
        _check(form, bits, q.to(BF16), k.to(BF16), v.to(BF16), lens, window, sinks)


@both_bits
@each_form
def test_a_scale_next_to_nothing(form, B, H, Hkv, T, Smax, bits):
    """scale = 2^-120, with which the scores are zeros in fp32: equal weights, for zero queries too."""
    k, v, q = _rand(10, (B, Smax, Hkv, D), (B, Smax, Hkv, D), (B, T, H, D))
    q[:, 0].zero_()
    _check(form, bits, q.to(BF16), k.to(BF16), v.to(BF16), [Smax - 5] * B, scale=2.0 ** -120)


@both_bits
@pytest.mark.parametrize("e", [100, 112, 118, 124])
@each_form
def test_very_large_queries(form, B, H, Hkv, T, Smax, e, bits):
    """Q up to 2^126: over K of 2^-95, with a scale that makes up for the rest; then K such that a row's largest score
    takes it all; one such row among ordinary ones leaves those as they are."""
    k, v, q = _rand(11, (B, Smax, Hkv, D), (B, Smax, Hkv, D), (B, T, H, D))
    small, large, v = (k * 2.0 ** -95).to(BF16), (q * 2.0 ** e).to(BF16), v.to(BF16)
    lens = [Smax - 3 - 30 * b for b in range(B)]
    _check(form, bits, large, small, v, lens, Smax - 99, 5, scale=SCALE * 2.0 ** (95 - e))
    _check(form, bits, large, small, v, lens, all_rows=False)
    k, q = k.to(BF16), q.to(BF16)
    want = _check(form, bits, q, k, v, lens)
    mixed = q.clone()
    mixed[:, -1, 1] = (mixed[:, -1, 1].float() * 2.0 ** (e - 2)).to(BF16)  # scores below 2^127 for e = 124 too
    o, lse = _check(form, bits, mixed, k, v, lens, all_rows=False)
    keep = torch.ones(T, H, dtype=torch.bool, device="cuda")
    keep[-1, 1] = False
    assert torch.equal(o[:, keep], want[0][:, keep])
    assert torch.equal(lse.transpose(1, 2)[:, keep], want[1].transpose(1, 2)[:, keep])


def _values_that_the_last_token_sees(form, B, H, Hkv, T, Smax, bits):
    """V up to bf16's largest number, and far below 1, in the newest key: the other tokens' rows keep their bits."""
    k, v, q = [x.to(BF16) for x in _rand(12, (B, Smax, Hkv, D), (B, Smax, Hkv, D), (B, T, H, D))]
    want = _check(form, bits, q, k, v)
    for x in (2.0 ** -30, 2.0 ** 10, 2.0 ** 100, 2.0 ** 120, torch.finfo(BF16).max):
        other = v.clone()
        other[:, -1] = x
        o, lse = lcb.attn_cache_decode(q, _cache(k, other, bits), _lens(*[Smax] * B))
        assert torch.equal(o[:, :-1], want[0][:, :-1]), x
        assert torch.equal(lse, want[1]), x


@both_bits
@pytest.mark.parametrize("form,B,H,Hkv,T,Smax", FORMS[:6])
def test_a_huge_value_that_only_the_last_token_sees(form, B, H, Hkv, T, Smax, bits):
    _values_that_the_last_token_sees(form, B, H, Hkv, T, Smax, bits)


@both_bits
@pytest.mark.parametrize("which", ["large", "all sizes", "grows"])
@each_form
def test_values_of_all_sizes(form, B, H, Hkv, T, Smax, which, bits):
    """V whose sizes change at once, from key to key, and along the keys, in every layout."""
    k, v, q = _rand(13, (B, Smax, Hkv, D), (B, Smax, Hkv, D), (B, T, H, D))
    g = torch.Generator(device="cuda").manual_seed(14)
    if which == "large":
        v = v * 2.0 ** 95
    elif which == "all sizes":
        v = v * torch.exp2(torch.randint(-30, 30, (B, Smax, Hkv, 1), generator=g, device="cuda").float())
    else:
        v = v * torch.exp2((torch.arange(Smax, device="cuda") * 130 // Smax - 40).float())[None, :, None, None]
    _check(form, bits, q.to(BF16), k.to(BF16), v.to(BF16), [Smax - 3 - 30 * b for b in range(B)], Smax - 99, 5)


@both_bits
@pytest.mark.parametrize("form,B,H,Hkv,T,Smax", FORMS[6:])
def test_a_huge_value_that_only_the_last_token_sees_tiles(form, B, H, Hkv, T, Smax, bits):
    _values_that_the_last_token_sees(form, B, H, Hkv, T, Smax, bits)


@both_bits
@each_form
def test_rows_before_the_last_token_are_those_without_it(form, B, H, Hkv, T, Smax, bits):
    """The newest key's V at any distance from a multiple of sixteen: the other rows keep their bits."""
    k, v, q = [x.to(BF16) for x in _rand(15, (B, Smax, Hkv, D), (B, Smax, Hkv, D), (B, T, H, D))]
    for back in (0, 1, 7, 15, 16):
        n, lens = Smax - back, _lens(*[Smax - back] * B)
        want = lcb.attn_cache_decode(q, _cache(k, v, bits), lens)
        other = v.clone()
        other[:, n - 1, :, ::3] = 2.0 ** 9
        o, lse = lcb.attn_cache_decode(q, _cache(k, other, bits), lens)
        assert torch.equal(o[:, :-1], want[0][:, :-1]) and torch.equal(lse, want[1]), back


# ------------------------------------------------------------------ Q whose sizes differ among channels


@both_bits
@pytest.mark.parametrize("form,B,H,Hkv,T,Smax,e", [(*f, e) for f in FORMS for e in (14, 22)] + [(*f, 27) for f in FORMS[:6]])
def test_small_channels_of_q_over_large_ones_of_k(form, B, H, Hkv, T, Smax, e, bits):
    """K's second group 2^e times the others, Q's the same below them: all groups count alike."""
    k, v, q = _rand(16, (B, Smax, Hkv, D), (B, Smax, Hkv, D), (B, T, H, D))
    k[..., 32:64] *= 2.0 ** e
    q[..., 32:64] *= 2.0 ** -e
    _check(form, bits, q.to(BF16), k.to(BF16), v.to(BF16))


# ------------------------------------------------------------------ bf16's end


@both_bits
def test_the_largest_number_reads_as_infinity(bits):
    """A group whose largest magnitude is bf16's largest number holds m s = 7 * 146 * 2^118 or 127 * 129 * 2^114, which
    bf16 rounds to infinity when it is read; attention takes the held number. The next smaller one reads as a number,
    the held one rounded as any other is."""
    end = torch.finfo(BF16).max
    below = (2.0 - 2.0 ** -6) * 2.0 ** 127
    x = torch.zeros(1, 4, 1, D, device="cuda", dtype=BF16)
    x[0, 0, 0, 5], x[0, 1, 0, 40], x[0, 2, 0, 127], x[0, 3, 0, 64] = end, -end, below, -below
    cache = _cache(x, torch.ones_like(x), bits)
    k, v = lcb.kv_cache_read(cache, 4)
    assert k[0, 0, 0, 5] == torch.inf and k[0, 1, 0, 40] == -torch.inf and (v == 1).all()
    assert k[0, 2, 0, 127] == _held(x, bits)[0, 2, 0, 127].to(BF16) and torch.isfinite(k[0, 2:]).all()
    assert k[0, 3, 0, 64] == _held(x, bits)[0, 3, 0, 64].to(BF16)
    held = 7 * 146 * 2.0 ** 118 if bits == 4 else 127 * 129 * 2.0 ** 114
    q = torch.zeros(1, 1, 1, D, device="cuda", dtype=BF16)
    q[..., 5] = 2.0 ** -126
    o, lse = lcb.attn_cache_decode(q, cache, _lens(1))
    assert (o == 1).all() and abs(lse.item() - SCALE * held * 2.0 ** -126) <= 2.0 ** -21
