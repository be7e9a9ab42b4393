"""GPU tests of rows of windowed attention at the ends of their range and beside
one another, in each form of the forward (keys split over a cluster, a block of
rows shared by a cluster, 128-row tiles) and in the decode call."""

import numpy as np
import pytest
import torch

import long_context_causal_blockwise_gb300 as lcb
from parity import to64
from window_bounds import U, check_attn

pytestmark = pytest.mark.gpu
D = 128
SCALE = D ** -0.5
LOG2E = 1.4426950408889634
# H, Hkv, Sq, Sk, window: one of each form (16 rows at most: split; 16 blocks and many keys: cluster; 40 heads: tiles)
FORMS = [(4, 4, 4, 700, 600), (8, 8, 300, 4000, 3500), (40, 40, 400, 600, 500)]


def _rand(seed, *shapes):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(s, generator=g, device="cuda").to(torch.bfloat16) for s in shapes]


def _climbing(seed, H, Hkv, Sq, Sk):
    """q, k, v whose scores are small but for every 331st key's, which are higher by 0 to 60 in base 2, growing with the
    row and with the key: most tiles have none, and a running maximum has to follow by small steps and by large ones."""
    q, k, v = _rand(seed, (1, Sq, H, D), (1, Sk, Hkv, D), (1, Sk, Hkv, D))
    q *= 0.25
    q[..., 1] = (torch.arange(Sq, device="cuda") % 61 / LOG2E / SCALE / 8)[None, :, None].to(q.dtype)
    far = torch.arange(Sk, device="cuda") % 331 == 330
    k[..., 1] = torch.where(far, 4 + 4 * torch.arange(Sk, device="cuda") / Sk, 0.0)[None, :, None].to(k.dtype)
    return q, k, v


@pytest.mark.parametrize("H,Hkv,Sq,Sk,window", FORMS)
def test_large_values_stay_finite(H, Hkv, Sq, Sk, window):
    """O is finite where |v| stays below 2^120 / (keys + 512): before the division by l a weight is at most 2^8, or 2^15
    for one key of a tile. Here the largest |v| is 2^118 / keys."""
    q, k, v = _climbing(Sk, H, Hkv, Sq, Sk)
    v = v.float()
    v *= 2.0 ** 118 / window / v.abs().max()
    v = v.to(torch.bfloat16)
    o, lse = lcb.attn_window_fwd(q, k, v, window)
    torch.cuda.synchronize()
    check_attn(to64(q), to64(k), to64(v), window, 0, Sk - Sq, SCALE, to64(o), to64(lse))
    lens = torch.tensor([Sk], dtype=torch.int32, device="cuda")
    o, lse = lcb.attn_window_decode(q[:, :3], k, v, lens, window)
    torch.cuda.synchronize()
    check_attn(to64(q[:, :3]), to64(k), to64(v), window, 0, Sk - 3, SCALE, to64(o), to64(lse))


@pytest.mark.parametrize("H,Hkv,Sq,Sk,window", FORMS)
def test_small_values_keep_their_precision(H, Hkv, Sq, Sk, window):
    """v times 2^-100 gives O times 2^-100. The weights reach down to 2^-16 below a row's largest, so that O before the
    division holds products of 2^-116 |v|, subnormal in fp32: off by 2^-149 each, 2^-149 * 2^16 * 2^100 = 2^-33 of v's
    unit after it, for at most 2^12 of them. Each O is then rounded once more."""
    q, k, v = _rand(Sk + 2, (1, Sq, H, D), (1, Sk, Hkv, D), (1, Sk, Hkv, D))
    want = lcb.attn_window_fwd(q, k, v, window)[0].double()
    got = lcb.attn_window_fwd(q, k, (v.float() * 2.0 ** -100).to(torch.bfloat16), window)[0].double() * 2.0 ** 100
    torch.cuda.synchronize()
    assert ((got - want).abs() <= 2 * U * want.abs() + 2.0 ** -21).all()


@pytest.mark.parametrize("H,Hkv,Sq,Sk,window", FORMS)
def test_rows_beside_one_that_has_seen_nothing_yet(H, Hkv, Sq, Sk, window):
    """A row's bits are its own: they do not change when another row's scores of the first two thirds of the keys are
    all -inf (a product past the fp32 range), so that it takes its maximum later."""
    q, k, v = _climbing(Sk + 1, H, Hkv, Sq, Sk)
    q[..., 0] = 0
    k[..., 0] = 0
    k[:, :2 * Sk // 3, :, 0] = -3e38
    want = lcb.attn_window_fwd(q, k, v, Sk)
    rows = torch.arange(1, Sq, 32, device="cuda")
    q[:, rows, :, 0] = 3e38  # times -3e38: -inf
    got = lcb.attn_window_fwd(q, k, v, Sk)
    torch.cuda.synchronize()
    others = torch.ones(Sq, dtype=torch.bool, device="cuda")
    others[rows] = False
    assert torch.equal(got[0][:, others], want[0][:, others])
    assert torch.equal(got[1][:, :, others], want[1][:, :, others])
    assert torch.isfinite(got[0]).all() and not torch.equal(got[1][:, :, rows], want[1][:, :, rows])


@pytest.mark.parametrize("B,H,Hkv,Sq,Sk,window,sinks", [
    (1, 48, 48, 1000, 9000, 8000, 4),  # 19 heads' windows fit the L2 share: groups of 19, 19 and 10
    (1, 48, 24, 1000, 9000, 8000, 0),  # of 38 and 10
    (2, 20, 20, 1100, 9001, 8000, 130),  # of 19, 19 and 2, a group over both sequences
])
def test_more_than_one_group_of_heads(B, H, Hkv, Sq, Sk, window, sinks):
    """Heads whose windows' K and V exceed what a group of heads keeps in L2, a last group that is smaller: every row of
    every head is written (outputs start as NaN) and right."""
    q, k, v = _rand(Sq, (B, Sq, H, D), (B, Sk, Hkv, D), (B, Sk, Hkv, D))
    o = torch.full_like(q, float("nan"))
    lse = torch.full((B, H, Sq), float("nan"), device="cuda")
    lcb.attn_window_fwd(q, k, v, window, sinks, o=o, lse=lse)
    p = (Sk - Sq + torch.arange(Sq, device="cuda"))[:, None]
    j = torch.arange(Sk, device="cuda")[None]
    hidden = ~((j <= p) & ((p - j < window) | (j < sinks)))
    for b in range(B):
        for h in range(H):
            qd, kd, vd = q[b, :, h].double(), k[b, :, h * Hkv // H].double(), v[b, :, h * Hkv // H].double()
            s = (qd @ kd.T * SCALE).masked_fill(hidden, float("-inf"))
            want = torch.logsumexp(s, dim=1)
            pr = torch.exp(s - want[:, None])
            # the bounds of window_bounds.py
            E = (2 * 2 * 128 * 2.0 ** -24 * SCALE * (qd.abs() @ kd.abs().T)).amax(dim=1, keepdim=True) + 2.0 ** -20
            err = (o[b, :, h].double() - pr @ vd).abs()
            assert (err <= U * (pr @ vd).abs() + (U + E) * (pr @ vd.abs())).all(), (b, h)
            assert ((lse[b, h].double() - want).abs() <= E[:, 0] + 2.0 ** -21 * (1 + want.abs())).all(), (b, h)
