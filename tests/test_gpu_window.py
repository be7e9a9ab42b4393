"""GPU parity of windowed attention (forward, backward, decode) against the
fp64 oracle, element by element within bounds derived from the kernels'
roundings (window_bounds.py); and the calls around it: strides, streams, graph
capture, repeated calls, rows left alone, long caches."""

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


def _rand(seed, *shapes):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(s, generator=g, device="cuda").to(torch.bfloat16) for s in shapes]


def _check(q, k, v, window, sinks, pos0, do=None, name=""):
    """Forward (and backward) of the given tensors against the oracle; returns the kernel's outputs."""
    o, lse = lcb.attn_window_fwd(q, k, v, window, sinks, pos0)
    grads = None if do is None else lcb.attn_window_bwd(q, k, v, o, lse, do, window, sinks, pos0)
    torch.cuda.synchronize()
    p0 = k.shape[1] - q.shape[1] if pos0 is None else pos0
    check_attn(to64(q), to64(k), to64(v), window, sinks, p0, SCALE, to64(o), to64(lse), None if do is None else to64(do),
               None if do is None else [to64(g) for g in grads], name)
    return (o, lse) if do is None else (o, lse, *grads)


# B, H, Hkv, Sq, Sk, window, sinks, q_pos0
CASES = [
    (1, 1, 1, 1, 1, 1, 0, None),         # one token that sees itself
    (2, 2, 1, 300, 300, 1, 0, None),     # every row sees itself alone
    (1, 2, 2, 513, 513, 64, 4, None),
    (1, 2, 2, 384, 384, 128, 0, None),   # a window of exactly one tile
    (1, 2, 2, 385, 385, 129, 1, None),
    (1, 2, 1, 640, 640, 127, 128, None),  # a whole tile of sinks
    (2, 4, 2, 257, 700, 130, 129, None),  # a chunk after earlier keys, not on a tile boundary
    (1, 2, 1, 200, 900, 128, 300, None),  # more sinks than window
    (1, 2, 1, 130, 1000, 10, 5, None),
    (1, 8, 1, 150, 150, 40, 3, None),    # eight query heads of one K/V head
    (1, 2, 2, 300, 100, 50, 4, None),    # more queries than keys: the first 200 see nothing
    (1, 2, 1, 400, 300, 100, 0, 150),    # queries past the keys: the last rows see nothing
    (1, 2, 1, 400, 300, 100, 5, 150),    # ... but the sinks
    (1, 2, 2, 300, 1000, 100, 1000, 1100),  # no key in any window, all keys sinks
    (1, 2, 2, 300, 1000, 100, 0, 2000),  # nothing at all
    (1, 2, 2, 300, 300, 2 ** 31 - 1, 2 ** 31 - 1, None),  # causal
    (3, 3, 3, 17, 17, 5, 2, None),
    (1, 10, 5, 129, 400, 200, 64, 100),  # a block of queries in the middle of the keys
]


@pytest.mark.parametrize("B,H,Hkv,Sq,Sk,window,sinks,pos0", CASES)
def test_fwd_bwd_vs_oracle(B, H, Hkv, Sq, Sk, window, sinks, pos0):
    q, k, v, do = _rand(Sq + Sk + window % 1000, (B, Sq, H, D), (B, Sk, Hkv, D), (B, Sk, Hkv, D), (B, Sq, H, D))
    _check(q, k, v, window, sinks, pos0, do)


@pytest.mark.parametrize("B,H,Hkv,Sq,Sk,window,sinks,pos0", [c for c in CASES if c[3] * c[1] // c[2] > 16])
def test_forward_in_128_row_tiles(B, H, Hkv, Sq, Sk, window, sinks, pos0):
    """The same with so many heads (more than 608 tiles of 16 rows) that the keys are not split over a cluster."""
    n = 608 // (B * Hkv * ((Sq * (H // Hkv) + 15) // 16)) + 1
    q, k, v = _rand(Sq + Sk + window % 1000, (B, Sq, n * H, D), (B, Sk, n * Hkv, D), (B, Sk, n * Hkv, D))
    _check(q, k, v, window, sinks, pos0)


@pytest.mark.parametrize("B,H,Hkv,Sq,Sk,window,sinks,pos0", [
    (1, 8, 8, 300, 4000, 3500, 4, None),      # 16 blocks, clusters of nine or so
    (2, 16, 2, 130, 5000, 4500, 300, None),
    (1, 12, 12, 513, 2600, 2200, 0, 2000),    # a last block of one row
    (1, 16, 4, 257, 3000, 2900, 0, 2990),     # later rows past the keys
    (1, 16, 16, 400, 2500, 2300, 200, -150),  # rows that see nothing; so few keys that a block is one CTA's
    (1, 5, 1, 700, 1500, 1400, 130, None),
    (1, 10, 10, 100, 6000, 5900, 0, None),    # one query tile alone
    (2, 6, 6, 200, 2300, 100, 2000, None),    # sinks in most parts, the window in the last
])
def test_forward_blocks_shared_by_a_cluster(B, H, Hkv, Sq, Sk, window, sinks, pos0):
    """Few blocks of query rows and many keys: a cluster of CTAs shares a block, joined through shared memory."""
    q, k, v = _rand(Sq + window, (B, Sq, H, D), (B, Sk, Hkv, D), (B, Sk, Hkv, D))
    a = _check(q, k, v, window, sinks, pos0)
    b = lcb.attn_window_fwd(q, k, v, window, sinks, pos0)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    # scores of hundreds, the largest anywhere; a key of -inf towards q has no weight, nor has a NaN key past the diagonal
    q = 4 * q.abs()
    k *= (0.1 + 6 * (torch.arange(Sk, device="cuda") * 617 % Sk) / Sk)[None, :, None, None].to(k.dtype)
    k[:, Sk // 3] = torch.finfo(torch.bfloat16).min
    _check(q, k, v, window, sinks, pos0)
    want = lcb.attn_window_fwd(q, k, v, window, sinks, pos0)
    k[:, Sk // 3] = float("-inf")
    half = Sq // 64 * 32  # a warp's rows share the choice of how a tile is done
    first = (Sk - Sq if pos0 is None else pos0) + half
    if 0 <= first < Sk:
        k[:, first:] = float("nan")  # rows of the first half do not see them
    o, lse = lcb.attn_window_fwd(q, k, v, window, sinks, pos0)
    assert torch.equal(o[:, :half], want[0][:, :half]) and torch.equal(lse[:, :, :half], want[1][:, :, :half])


@pytest.mark.parametrize("H,Hkv,Sq,Sk,window", [(32, 8, 5, 9000, 8000), (8, 1, 33, 5000, 4000), (2, 2, 500, 3000, 2000),
                                                (3, 1, 7, 2000, 1500), (40, 8, 30, 700, 700)])
def test_forward_split_over_row_tiles(H, Hkv, Sq, Sk, window):
    """More query rows than one 16-row tile, few enough heads that their keys are split over clusters all the same:
    row tiles that begin inside a token's group of heads, a last tile with rows missing."""
    q, k, v = _rand(Sk, (1, Sq, H, D), (1, Sk, Hkv, D), (1, Sk, Hkv, D))
    a = _check(q, k, v, window, 3, None)
    b = lcb.attn_window_fwd(q, k, v, window, 3)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    _check(q, k, v, window, 0, Sk - 2 * Sq)  # the chunk before the last keys
    _check(q, k, v, 20, 3, Sk + 5)  # its window past the keys for the last rows


@pytest.mark.parametrize("H,Hkv,Sq", [(1, 1, 1), (1, 1, 16), (8, 1, 2), (8, 8, 16), (16, 1, 1), (12, 1, 1), (6, 2, 5)])
def test_few_rows_forward(H, Hkv, Sq):
    """Up to 16 query rows a K/V head: the keys split over a cluster of CTAs."""
    for Sk, window, sinks, pos0 in ((1, 5, 0, None), (37, 5, 3, None), (5000, 3000, 4, None), (5000, 900, 1200, None),
                                    (700, 100, 0, 690), (700, 100, 9, 900), (40, 10, 0, -8)):
        q, k, v = _rand(Sk, (2, Sq, H, D), (2, Sk, Hkv, D), (2, Sk, Hkv, D))
        _check(q, k, v, window, sinks, pos0, name=f"Sk {Sk} window {window}")


@pytest.mark.parametrize("H,Hkv,S", [(2, 1, 300), (48, 24, 420), (8, 8, 3)])
def test_row_of_one_key_gives_its_v(H, Hkv, S):
    """Weight 1 of a single key: O is its v to the bit (so Delta cancels dP), in every form of the call."""
    q, k, v = _rand(H, (2, S, H, D), (2, S, Hkv, D), (2, S, Hkv, D))
    o, _ = lcb.attn_window_fwd(q, k, v, 1)
    assert torch.equal(o, v.repeat_interleave(H // Hkv, dim=2))
    o, _ = lcb.attn_window_fwd(q, k, v, S)
    assert torch.equal(o[:, 0], v[:, 0].repeat_interleave(H // Hkv, dim=1))
    lens = torch.tensor([S, 1], dtype=torch.int32, device="cuda")
    o, _ = lcb.attn_window_decode(q[:, :1], k, v, lens, 1)
    assert torch.equal(o[:, 0], torch.stack([v[0, S - 1], v[1, 0]]).repeat_interleave(H // Hkv, dim=1))


@pytest.mark.parametrize("H", [2, 20])
def test_large_scores_and_sharp_rows(H):
    """Scores of hundreds (the running maximum moves by more than 2^8 between tiles), and one key that takes all."""
    q, k, v, do = _rand(5, *[(1, 500, H, D)] * 4)
    k *= torch.linspace(0.1, 6, 500, device="cuda")[None, :, None, None].to(k.dtype)
    q *= 4
    _check(q, k, v, 200, 4, None, do)


@pytest.mark.parametrize("H", [1, 33])  # keys split over a cluster; 128-row tiles
def test_scores_of_minus_infinity_and_hidden_nan_keys(H):
    """k = -inf towards a positive q gives visible scores of -inf (weight 0), the type's lowest value gives a score that
    no other key's weight survives next to; NaN in a hidden key's k touches no row."""
    q, k, v = _rand(6, *[(1, 300, H, D)] * 3)
    q[:] = q.abs() + 0.1
    ref, lse = lcb.attn_window_fwd(q, k, v, 50)  # the same tiles: equal bits where nothing hidden gets in
    k2 = k.clone()
    k2[:, :100] = float("nan")  # rows from 150 on do not see them
    o2, lse2 = lcb.attn_window_fwd(q, k2, v, 50)
    assert torch.equal(o2[:, 150:], ref[:, 150:]) and torch.equal(lse2[:, :, 150:], lse[:, :, 150:])
    k3 = k.clone()
    k3[:, 200] = float("-inf")
    o3, lse3 = lcb.attn_window_fwd(q, k3, v, 50)
    k4 = k.clone()
    k4[:, 200] = torch.finfo(torch.bfloat16).min
    o4, lse4 = lcb.attn_window_fwd(q, k4, v, 50)
    torch.cuda.synchronize()
    assert torch.isfinite(o3).all() and torch.equal(o3, o4) and torch.equal(lse3, lse4)
    assert torch.equal(o3[:, :200], lcb.attn_window_fwd(q, k, v, 50)[0][:, :200])
    # a query that sees only such a key: no weight at all
    o5, lse5 = lcb.attn_window_fwd(q[:, :20], k3[:, 200:220], v[:, :20], 1)
    assert lse5[0, 0, 0] == float("-inf") and (o5[0, 0] == 0).all()


def test_views_of_a_packed_buffer_and_rows_left_alone():
    """q, k, v as slices of one packed [S, B, ...] buffer (batch inside the row), o, dq, dk, dv into slices of padded
    ones, o and do sharing strides; what lies beside the outputs stays as it was."""
    B, S, H, Hkv = 2, 333, 4, 2
    packed, dob = _rand(7, (S + 3, B, H + 2 * Hkv, D), (B, S, H + 1, D))
    x = packed.transpose(0, 1)[:, 1:S + 1]
    q, k, v = x[:, :, :H], x[:, :, H:H + Hkv], x[:, :, H + Hkv:]
    ob, dqb, dkb, dvb = (torch.full((B, S + 2, n + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
                         for n in (H, H, Hkv, Hkv))
    ob = ob[:, :S].contiguous()
    o, dq, dk, dv = ob[:, :, :H], dqb[:, :S, :H], dkb[:, 1:S + 1, 1:], dvb[:, 1:S + 1, 1:]
    lse = torch.empty(B, H, S + 5, device="cuda")[:, :, :S]
    lcb.attn_window_fwd(q, k, v, 70, 6, o=o, lse=lse)
    do = dob[:, :, :H]
    lcb.attn_window_bwd(q, k, v, o, lse, do, 70, 6, dq=dq, dk=dk, dv=dv)
    torch.cuda.synchronize()
    check_attn(to64(q), to64(k), to64(v), 70, 6, 0, SCALE, to64(o), to64(lse), to64(do), [to64(t) for t in (dq, dk, dv)])
    assert (ob[:, :, H:] == 7).all() and (dqb[:, S:] == 7).all() and (dqb[:, :, H:] == 7).all()
    for b in (dkb, dvb):
        assert (b[:, 0] == 7).all() and (b[:, S + 1:] == 7).all() and (b[:, :, 0] == 7).all()


def test_split_gradient_runs():
    """Key tiles whose queries are dealt to several CTAs: sinks that a long sequence sees, and a single K/V head under
    eight query heads; dK and dV come from fp32 partials, deterministic."""
    for B, H, Hkv, S, window, sinks in ((1, 2, 1, 2500, 64, 4), (1, 8, 1, 1100, 500, 130), (1, 8, 1, 700, 700, 0)):
        assert lcb.attn_window_bwd_workspace_bytes(B, H, Hkv, S, S, window, sinks) \
            > B * H * (S + 127) // 128 * (65536 + 1024) + 65536
        q, k, v, do = _rand(S, (B, S, H, D), (B, S, Hkv, D), (B, S, Hkv, D), (B, S, H, D))
        o, lse, dq, dk, dv = _check(q, k, v, window, sinks, None, do, f"S {S}")
        for _ in range(3):
            _, dk2, dv2 = lcb.attn_window_bwd(q, k, v, o, lse, do, window, sinks)
            assert torch.equal(dk, dk2) and torch.equal(dv, dv2)
            o2, lse2 = lcb.attn_window_fwd(q, k, v, window, sinks)
            assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_gradient_against_differences():
    """d(sum o * do) along random directions of q, k, v against the bf16 gradients: the forward at fp64 (the oracle) on
    inputs moved by a finite step, so only the gradients' own bounds enter."""
    q, k, v, do = _rand(8, (1, 200, 2, D), (1, 260, 1, D), (1, 260, 1, D), (1, 200, 2, D))
    _, _, dq, dk, dv = _check(q, k, v, 60, 3, None, do)
    x = [to64(t) for t in (q, k, v)]
    rng = np.random.default_rng(0)

    def loss(q, k, v):
        return (oracle.window_attn(q, k, v, 60, 3, 60, SCALE)["o"] * to64(do)).sum()
    for i, g in enumerate((dq, dk, dv)):
        d = rng.standard_normal(x[i].shape)
        moved = [[y + (s * 1e-4 * d if n == i else 0) for n, y in enumerate(x)] for s in (1, -1)]
        diff = (loss(*moved[0]) - loss(*moved[1])) / 2e-4
        got = (to64(g) * d).sum()
        # each gradient value is off by at most a few half steps of its own size, in directions that d signs at random:
        # the sum of n such errors stays under eight standard deviations of 3 * 2^-8 |g| |d|
        assert abs(got - diff) <= 8 * 3 * 2.0 ** -8 * np.sqrt((to64(g) ** 2 * d ** 2).sum()) + 1e-5 * abs(diff)


@pytest.mark.parametrize("B,H,Hkv,Sq,Sk,window,sinks,pos0", [
    (2, 40, 8, 300, 300, 90, 4, None),     # 160 blocks of 256 query rows: some CTAs walk over two
    (1, 64, 64, 600, 500, 64, 3, -200),    # ... and some of their blocks see nothing
    (1, 48, 16, 1030, 700, 200, 0, 400),   # a last block of six rows, rows past every key
])
def test_more_blocks_than_sms(B, H, Hkv, Sq, Sk, window, sinks, pos0):
    """A CTA's second and third block: barrier phases carried over, blocks without keys in between."""
    q, k, v, do = _rand(Sq, (B, Sq, H, D), (B, Sk, Hkv, D), (B, Sk, Hkv, D), (B, Sq, H, D))
    _check(q, k, v, window, sinks, pos0, do)


def test_broadcast_keys_of_a_batch():
    """One K/V for every sequence of the batch (batch stride 0): as with copies, gradients per sequence."""
    q, k, v, do = _rand(12, (3, 300, 4, D), (1, 300, 2, D), (1, 300, 2, D), (3, 300, 4, D))
    kx, vx = k.expand(3, -1, -1, -1), v.expand(3, -1, -1, -1)
    a = _check(q, kx, vx, 100, 4, None, do)
    b = _check(q, kx.contiguous(), vx.contiguous(), 100, 4, None, do)
    assert all(torch.equal(x, y) for x, y in zip(a[:2] + a[3:], b[:2] + b[3:]))
    lens = torch.tensor([300, 17, 0], dtype=torch.int32, device="cuda")
    _decode_check(q[:, :1], kx, vx, lens, 100, 4)


def test_wide_window_agrees_with_attn_fwd():
    """A window over everything is causal attention: the two kernels within both their roundings."""
    q, k, v = _rand(13, (1, 1000, 3, D), (1, 1000, 3, D), (1, 1000, 3, D))
    o, lse = lcb.attn_window_fwd(q, k, v, 1000)
    o2, lse2 = lcb.attn_fwd(q, k, v)
    torch.cuda.synchronize()
    assert (lse - lse2).abs().max() <= 1e-5 * lse.abs().max()
    assert (o.float() - o2.float()).abs().max() <= 4 * 2.0 ** -8 * v.float().abs().max()


def test_two_captured_graphs_interleaved():
    """Two graphs of the whole training pass, each with buffers of its own, replayed in turn and on two streams."""
    runs = []
    for seed in (14, 15):
        t = _rand(seed, (1, 500, 4, D), (1, 500, 2, D), (1, 500, 2, D), (1, 500, 4, D))
        ws = torch.empty(lcb.attn_window_bwd_workspace_bytes(1, 4, 2, 500, 500, 70, 4), dtype=torch.uint8, device="cuda")

        def step(t=t, ws=ws):
            o, lse = lcb.attn_window_fwd(*t[:3], 70, 4)
            return (o, lse, *lcb.attn_window_bwd(*t[:3], o, lse, t[3], 70, 4, workspace=ws))
        want = [x.clone() for x in step()]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        runs.append((graph, out, want, torch.cuda.Stream(), step))  # step keeps its inputs alive
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, _, _, stream, _ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, out, want, _, _ in runs:
        for i, (x, y) in enumerate(zip(out, want)):
            if i == 2:  # dQ: an fp32 sum in no fixed order, then one rounding: within one bf16 step of either
                assert (x.float() - y.float()).abs().max() <= 2.0 ** -7 * y.float().abs().max()
            else:
                assert torch.equal(x, y)


def test_side_stream_and_graph_replay():
    """On a stream of its own; then forward and backward captured once and replayed with other inputs."""
    q, k, v, do = _rand(9, (1, 300, 4, D), (1, 300, 2, D), (1, 300, 2, D), (1, 300, 4, D))
    want = _check(q, k, v, 90, 4, None, do)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, lse = lcb.attn_window_fwd(q, k, v, 90, 4)
        dq, dk, dv = lcb.attn_window_bwd(q, k, v, o, lse, do, 90, 4)
    side.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(dk, want[3]) and torch.equal(dv, want[4])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = lcb.attn_window_fwd(q, k, v, 90, 4)
        dq, dk, dv = lcb.attn_window_bwd(q, k, v, o, lse, do, 90, 4)
    for seed in (10, 11):
        for t, new in zip((q, k, v, do), _rand(seed, q.shape, k.shape, v.shape, do.shape)):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        check_attn(to64(q), to64(k), to64(v), 90, 4, 0, SCALE, to64(o), to64(lse), to64(do),
                   [to64(t) for t in (dq, dk, dv)])


# ------------------------------------------------------------------ decode

def _decode_check(q, k, v, lens, window, sinks, name=""):
    o, lse = lcb.attn_window_decode(q, k, v, lens, window, sinks)
    torch.cuda.synchronize()
    T = q.shape[1]
    for b, n in enumerate(lens.tolist()):
        n = min(max(n, 0), k.shape[1])
        check_attn(to64(q[b:b + 1]), to64(k[b:b + 1, :n]), to64(v[b:b + 1, :n]), window, sinks, n - T, SCALE,
                   to64(o[b:b + 1]), to64(lse[b:b + 1]), name=f"{name} b {b} len {n}")
    return o, lse


@pytest.mark.parametrize("H,Hkv,T,window,sinks", [
    (4, 4, 1, 100, 4), (4, 4, 1, 1, 0), (8, 1, 1, 500, 16), (16, 2, 2, 64, 0), (32, 2, 1, 300, 200), (8, 1, 4, 300, 3),
    (40, 8, 1, 5000, 0), (6, 2, 7, 33, 2), (2, 1, 40, 90, 5)])
def test_decode_vs_oracle(H, Hkv, T, window, sinks):
    """Lengths from zero to a full cache, with NaN in every cache row at or past each length (never read)."""
    Smax = 1500
    lens = torch.tensor([0, 1, T, 2, 77, 128, 1000, Smax, Smax + 9, -3], dtype=torch.int32, device="cuda")
    B = lens.numel()
    q, k, v = _rand(H + T, (B, T, H, D), (B, Smax, Hkv, D), (B, Smax, Hkv, D))
    for b, n in enumerate(lens.tolist()):
        k[b, max(0, n):] = float("nan")
        v[b, max(0, n):] = float("nan")
    _decode_check(q, k, v, lens, window, sinks)


@pytest.mark.parametrize("B,H,Hkv,T,Smax", [(37, 32, 32, 1, 70), (37, 32, 32, 1, 1500), (90, 16, 8, 5, 1100)])
def test_decode_more_tiles_than_fit(B, H, Hkv, T, Smax):
    """Batches whose tiles run in several waves, with short caches and with long ones."""
    lens = Smax - 3 * torch.arange(B, dtype=torch.int32, device="cuda")
    q, k, v = _rand(Smax, (B, T, H, D), (B, Smax, Hkv, D), (B, Smax, Hkv, D))
    _decode_check(q, k, v, lens, 1400, 2)


def test_decode_graph_follows_the_lengths():
    """One captured call replayed while the sequences grow, each step equal to an eager call."""
    B, H, Hkv, Smax = 3, 8, 2, 700
    q, k, v = _rand(3, (B, 1, H, D), (B, Smax, Hkv, D), (B, Smax, Hkv, D))
    lens = torch.tensor([1, 300, 650], dtype=torch.int32, device="cuda")
    lcb.attn_window_decode(q, k, v, lens, 128, 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = lcb.attn_window_decode(q, k, v, lens, 128, 4)
    for step in range(4):
        lens += 7
        graph.replay()
        want = lcb.attn_window_decode(q, k, v, lens, 128, 4)
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), step
    _decode_check(q, k, v, lens, 128, 4)


def test_decode_long_cache_past_32_bit_offsets():
    """A cache of more than 2^31 elements: the window at its end and the sinks at its start."""
    Smax, H = 530_000, 32
    k = torch.zeros(1, Smax, H, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    assert k.numel() > 2 ** 31
    q, ends = _rand(4, (1, 1, H, D), (4, 1, 300, H, D))
    k[:, :300], v[:, :300], k[:, -300:], v[:, -300:] = ends[0], ends[1], ends[2], ends[3]
    lens = torch.tensor([Smax], dtype=torch.int32, device="cuda")
    o, lse = lcb.attn_window_decode(q, k, v, lens, 300, 300)
    o2, lse2 = lcb.attn_window_fwd(q, k, v, 300, 300)
    qq = q.expand(1, 129, H, D).contiguous()  # the tiled forward, every row but the last before the end
    o3, lse3 = lcb.attn_window_fwd(qq, k, v, 300, 300)
    torch.cuda.synchronize()
    ke, ve = torch.cat([k[:, :300], k[:, -300:]], 1), torch.cat([v[:, :300], v[:, -300:]], 1)
    args = (to64(q), to64(ke), to64(ve), 600, 0, 599, SCALE)
    check_attn(*args, to64(o), to64(lse))
    check_attn(*args, to64(o2), to64(lse2))
    check_attn(*args, to64(o3[:, -1:]), to64(lse3[:, :, -1:]))


# ------------------------------------------------------------------ together

def test_video_layer_prefill_then_decode():
    """rope_axes on q and k, windowed attention forward and backward, rope_axes^T on dq and dk; then one more token:
    its q and k turned to their positions, k and v put into the cache, and the decode call. Each step against the
    oracle on the values that it was given."""
    B, S, H, Hkv, Smax, window, sinks, theta = 2, 400, 4, 2, 512, 150, 4, 1e6
    sections = (16, 24, 24)
    axis = lcb.rope_pair_axes(sections)
    q, do, k, v = _rand(20, (B, S + 1, H, D), (B, S, H, D), (B, Smax, Hkv, D), (B, Smax, Hkv, D))
    t = torch.arange(S + 1, device="cuda")
    pos = torch.stack([100 + t // 64, 100 + t // 8 % 8, 100 + t % 8]).to(torch.int32)
    raw_q, raw_k = to64(q), to64(k)
    lcb.rope_axes(q[:, :S], theta, pos[:, :S], sections)
    lcb.rope_axes(k[:, :S], theta, pos[:, :S], sections)
    torch.cuda.synchronize()
    for got, raw in ((q, raw_q), (k, raw_k)):
        want = oracle.rope_axes(raw[:, :S], theta, pos[:, :S].cpu().numpy(), axis)
        assert np.abs(to64(got[:, :S]) - want).max() <= 2.0 ** -8 * np.abs(want).max() + 1e-5
    o, lse, dq, dk, dv = _check(q[:, :S].contiguous(), k[:, :S], v[:, :S], window, sinks, None, do)
    turned = to64(dq), to64(dk)
    lcb.rope_axes(dq, theta, pos[:, :S], sections, inverse=True)
    lcb.rope_axes(dk, theta, pos[:, :S], sections, inverse=True)
    torch.cuda.synchronize()
    for got, t0 in zip((dq, dk), turned):
        want = oracle.rope_axes(t0, theta, pos[:, :S].cpu().numpy(), axis, inverse=True)
        assert np.abs(to64(got) - want).max() <= 2.0 ** -8 * np.abs(want).max() + 1e-5
    lcb.rope_axes(q[:, S:], theta, pos[:, S:], sections)
    lcb.rope_axes(k[:, S:S + 1], theta, pos[:, S:], sections)
    lens = torch.full((B,), S + 1, dtype=torch.int32, device="cuda")
    _decode_check(q[:, S:], k, v, lens, window, sinks)
    # the last token of the prompt through the decode call: the forward's last row, within both calls' bounds
    od, _ = lcb.attn_window_decode(q[:, S - 1:S], k, v, lens - 1, window, sinks)
    check_attn(to64(q[:, S - 1:S]), to64(k[:, :S]), to64(v[:, :S]), window, sinks, S - 1, SCALE, to64(od),
               to64(lse[:, :, S - 1:]))


def test_long_sequence_sampled_rows():
    """32768 tokens, window 4096: sampled query rows and sampled keys' gradients against the oracle on the keys and
    queries that reach them."""
    B, S, H, Hkv, window, sinks = 1, 32768, 2, 1, 4096, 4
    q, k, v, do = _rand(30, (B, S, H, D), (B, S, Hkv, D), (B, S, Hkv, D), (B, S, H, D))
    o, lse = lcb.attn_window_fwd(q, k, v, window, sinks)
    dq, dk, dv = lcb.attn_window_bwd(q, k, v, o, lse, do, window, sinks)
    torch.cuda.synchronize()
    for r in (0, 5000, 16383, 32767):
        lo = max(0, r - window + 1)
        keep = torch.cat([torch.arange(0, min(sinks, lo)), torch.arange(lo, r + 1)]).cuda()
        n = keep.numel()
        args = (to64(q[:, r:r + 1]), to64(k[:, keep]), to64(v[:, keep]), n, 0, n - 1, SCALE)
        check_attn(*args, to64(o[:, r:r + 1]), to64(lse[:, :, r:r + 1]), to64(do[:, r:r + 1]),
                   (to64(dq[:, r:r + 1]), None, None), f"row {r}")
    # keys 20000 .. 20007 are seen by rows 20000 .. 24102: those rows with all that they see, on the GPU in fp64
    rows = torch.arange(20000, 20008 + window - 1, device="cuda")
    lo, hi = 20000 - window + 1, int(rows[-1]) + 1
    keys = torch.cat([torch.arange(0, sinks, device="cuda"), torch.arange(lo, hi, device="cuda")])
    kd, vd = k[0, keys, 0].double(), v[0, keys, 0].double()
    vis = (keys[None] <= rows[:, None]) & ((rows[:, None] - keys[None] < window) | (keys[None] < sinks))
    at = sinks + 20000 - lo
    rdk, rdv = torch.zeros(8, D, dtype=torch.float64, device="cuda"), torch.zeros(8, D, dtype=torch.float64, device="cuda")
    for h in range(H):
        qd, dd = q[0, rows, h].double(), do[0, rows, h].double()
        p = torch.softmax((qd @ kd.T * SCALE).masked_fill(~vis, float("-inf")), dim=1)
        dp = dd @ vd[at:at + 8].T - (dd * (p @ vd)).sum(1, keepdim=True)
        p = p[:, at:at + 8]
        rdv += p.T @ dd
        rdk += SCALE * (p * dp).T @ qd
    # sums of some 8000 terms rounded to bf16 one by one: their errors add at random, a few half steps of the whole
    for got, want in ((dk, rdk), (dv, rdv)):
        err = (got[0, 20000:20008, 0].double() - want).norm() / want.norm()
        assert err < 2.0 ** -7, float(err)


# ------------------------------------------------------------------ refusals

def test_python_refusals():
    q, k, v = _rand(1, (2, 8, 4, D), (2, 8, 2, D), (2, 8, 2, D))
    for bad in (dict(window=0), dict(window=4, sinks=-1), dict(window=4, scale=0.0), dict(window=4, q_pos0=1 << 29)):
        with pytest.raises(lcb.AttnError):
            lcb.attn_window_fwd(q, k, v, **bad)
    for a in ((q, k[:1], v[:1]), (q, k[:, :, :1].expand(2, 8, 3, D), v), (q[..., :64], k[..., :64], v[..., :64]),
              (q.float(), k, v), (q, k.cpu(), v.cpu()), (q, k, v[:, ::2])):
        with pytest.raises((ValueError, lcb.AttnError)):
            lcb.attn_window_fwd(*a, 4)
    o, lse = lcb.attn_window_fwd(q, k, v, 4)
    with pytest.raises(ValueError):
        lcb.attn_window_bwd(q, k, v, o, lse, q[:, :4], 4)
    with pytest.raises(lcb.AttnError):
        lcb.attn_window_bwd(q, k, v, o, lse, q, 4, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(lcb.AttnError):  # one row for both batches
        lcb.attn_window_fwd(q, k, v, 4, o=torch.empty_like(q[:1]).expand(2, 8, 4, D))
    with pytest.raises(ValueError):
        lcb.attn_window_decode(q, k, v, torch.tensor([8, 8], device="cuda"), 4)  # int64 lengths


def test_empty_sides():
    """No keys: zeros and -inf; no queries: zero dK, dV."""
    q, k = _rand(2, (2, 8, 4, D), (2, 40, 2, D))
    o, lse = lcb.attn_window_fwd(q, k[:, :0], k[:, :0], 4)
    assert (o == 0).all() and (lse == float("-inf")).all()
    dq, dk, dv = lcb.attn_window_bwd(q, k[:, :0], k[:, :0], o, lse, q, 4)
    assert (dq == 0).all() and dk.numel() == 0
    none = q[:, :0]
    o, lse = lcb.attn_window_fwd(none, k, k, 4)
    dq, dk, dv = lcb.attn_window_bwd(none, k, k, o, lse, none, 4)
    torch.cuda.synchronize()
    assert (dk == 0).all() and (dv == 0).all() and dq.numel() == 0
    o, lse = lcb.attn_window_decode(q[:, :1], k[:, :0], k[:, :0], torch.zeros(2, dtype=torch.int32, device="cuda"), 4)
    assert (o == 0).all() and (lse == float("-inf")).all()
