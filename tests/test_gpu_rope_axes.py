"""GPU parity of rotary positions with several axes against the fp64 oracle.

Bound: the output's one rounding to bf16 (half a step, 2^-8 of the value) and
the rotation in fp32: sin and cos of an angle that is off by at most pi 2^-24
plus the frequency's own rounding, |pos| 2^-53 of a turn at most, and their
last bits, under 1e-6 of the pair's size together for |pos| < 2^30."""

import numpy as np
import pytest
import torch

import oracle
import long_context_causal_blockwise_gb300 as lcb
from parity import to64

pytestmark = pytest.mark.gpu
D = 128


def _check(got, x, theta, pos, sections, interleaved=False, inverse=False):
    want = oracle.rope_axes(x, theta, pos.cpu().numpy(), lcb.rope_pair_axes(sections, interleaved), inverse)
    pair = np.abs(x[..., :64]) + np.abs(x[..., 64:])
    bound = 2.0 ** -8 * np.abs(want) + 1e-6 * np.concatenate([pair, pair], axis=-1)
    err = np.abs(to64(got) - want)
    assert (err <= bound).all(), float((err / bound).max())


def _x(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("B,S,H,sections,interleaved,theta,dtype,far", [
    (1, 1, 1, (64,), False, 1e4, torch.int32, 10), (2, 77, 3, (16, 24, 24), False, 1e6, torch.int32, 1000),
    (1, 300, 8, (16, 24, 24), True, 1e4, torch.int64, 10 ** 9), (3, 50, 11, (20, 44), True, 5e5, torch.int32, 2 ** 30),
    (1, 40, 40, (1, 2, 3, 58), False, 1e9, torch.int64, 500_000), (2, 33, 32, (0, 64), False, 0.5, torch.int32, 900)])
@pytest.mark.parametrize("per_batch,inverse", [(False, False), (True, True)])
def test_rope_axes_vs_oracle(B, S, H, sections, interleaved, theta, dtype, far, per_batch, inverse):
    """Positions of either sign, near and far, shared and per sequence, both directions, all head batches."""
    x = _x(S + H, B, S, H, D)
    shape = (len(sections), B, S) if per_batch else (len(sections), S)
    g = torch.Generator(device="cuda").manual_seed(S)
    pos = torch.randint(-far, far, shape, generator=g, device="cuda").to(dtype)
    x0 = to64(x)
    y = lcb.rope_axes(x, theta, pos, sections, inverse=inverse, interleaved=interleaved, out=torch.empty_like(x))
    torch.cuda.synchronize()
    _check(y, x0, theta, pos, sections, interleaved, inverse)
    lcb.rope_axes(x, theta, pos, sections, inverse=inverse, interleaved=interleaved)  # in place
    assert torch.equal(x, y)


def test_equal_axes_match_rope():
    """All axes at the token's index: the single-axis kernel's rotation, within one bf16 step."""
    x = _x(1, 2, 300, 4, D)
    pos = torch.arange(300, dtype=torch.int32, device="cuda").expand(3, 300)  # axis stride 0
    y = lcb.rope_axes(x, 1e6, pos, (16, 24, 24), out=torch.empty_like(x))
    z = lcb.rope(x, 1e6, 0, out=torch.empty_like(x))
    torch.cuda.synchronize()
    assert (to64(y) != to64(z)).mean() < 1e-3 and np.abs(to64(y) - to64(z)).max() <= 2.0 ** -7 * np.abs(to64(x)).max() * 2


def test_strided_views_in_place_on_a_side_stream():
    """A K slice of a packed buffer (4-byte aligned rows), positions read through strides; its neighbours untouched."""
    buf = _x(2, 2, 90, 5 * D + 2)
    k = buf[:, :, 2 * D + 2:4 * D + 2].unflatten(2, (2, D))
    before, rest = to64(k), buf.clone()
    pos = torch.randint(0, 5000, (90, 2, 3), device="cuda").permute(2, 1, 0)  # [3, 2, 90], last stride 6
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lcb.rope_axes(k, 1e6, pos, (16, 24, 24))
    side.synchronize()
    _check(k, before, 1e6, pos, (16, 24, 24))
    assert torch.equal(buf[:, :, :2 * D + 2], rest[:, :, :2 * D + 2]) and torch.equal(buf[:, :, 4 * D + 2:], rest[:, :, 4 * D + 2:])


def test_rope_axes_graph_replay_with_new_positions():
    x = _x(3, 1, 64, 2, D)
    out = torch.empty_like(x)
    pos = torch.zeros(2, 64, dtype=torch.int32, device="cuda")
    lcb.rope_axes(x, 1e4, pos, (32, 32), out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lcb.rope_axes(x, 1e4, pos, (32, 32), out=out)
    for add in (3, 40):
        pos += add
        graph.replay()
        torch.cuda.synchronize()
        _check(out, to64(x), 1e4, pos, (32, 32))


def test_rope_axes_large_offsets():
    """Rows past 2^31 elements from the base."""
    rows = torch.empty(2, (1 << 30) + 4096, dtype=torch.bfloat16, device="cuda")
    x = rows[:, :8 * D].unflatten(1, (4, 2, D))  # batch stride 2^30 + 4096: two batches; then a row stride of that size
    y = rows[:, :2 * D].unflatten(1, (2, D))[None]  # [1, 2, 2, D]
    for t in (x, y):
        t.copy_(_x(4, *t.shape))
        before = to64(t)
        pos = torch.arange(t.shape[1], dtype=torch.int32, device="cuda")[None]
        lcb.rope_axes(t, 1e4, pos, (64,))
        torch.cuda.synchronize()
        _check(t, before, 1e4, pos, (64,))


def test_rope_axes_python_refusals():
    x = _x(5, 2, 8, 2, D)
    pos = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    for a, kw in (((x, 1e4, pos, (64,)), {}), ((x, 1e4, pos.float(), (32, 32)), {}), ((x, 1e4, pos[:, :4], (32, 32)), {}),
                  ((x, 1e4, pos, (32, 31)), {}), ((x, 1e4, pos.cpu(), (32, 32)), {}),
                  ((x, 1e4, pos, (32, 32)), dict(out=torch.empty(2, 8, 4, D, dtype=torch.bfloat16, device="cuda")[:, :, :2])),
                  ((x.float(), 1e4, pos, (32, 32)), {})):
        with pytest.raises(ValueError):
            lcb.rope_axes(*a, **kw)
    with pytest.raises(lcb.AttnError):
        lcb.rope_axes(x, 0.0, pos, (32, 32))
