"""GPU tests of rows of windowed attention at the ends of their range and beside
one another, in each form of the forward (keys split over a cluster, a block of
rows shared by a cluster, 128-row tiles) and in the decode call."""

import pytest
import torch

import long_context_causal_blockwise_gb300 as lcb
from parity import to64
from window_bounds import check_attn

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
