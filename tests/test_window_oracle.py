"""Pins of the windowed-attention and several-axes RoPE oracle (CPU), and the
host side of the new calls: refusals, workspace sizes, pair axes."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
import long_context_causal_blockwise_gb300 as lcb
from long_context_causal_blockwise_gb300 import _lib


def _qkv(rng, B, H, Hkv, Sq, Sk, D=16):
    return rng.standard_normal((B, Sq, H, D)), rng.standard_normal((B, Sk, Hkv, D)), rng.standard_normal((B, Sk, Hkv, D))


def test_visible_by_hand():
    """Window 2, one sink, queries at positions 1 .. 4 over five keys; and a query before the first key."""
    got = oracle.window_visible(4, 5, 2, 1, 1).astype(int)
    assert got.tolist() == [[1, 1, 0, 0, 0], [1, 1, 1, 0, 0], [1, 0, 1, 1, 0], [1, 0, 0, 1, 1]]
    assert not oracle.window_visible(2, 5, 3, 2, -2).any()


def test_wide_window_is_causal_attention():
    rng = np.random.default_rng(0)
    q, k, v = _qkv(rng, 2, 3, 3, 20, 20)
    do = rng.standard_normal(q.shape)
    r = oracle.window_attn(q, k, v, 20, 0, 0, 0.3, do)
    w = oracle.attn_bwd(q, k, v, do, True, 0.3)
    for n in ("o", "lse", "dq", "dk", "dv"):
        assert np.allclose(r[n], w[n], rtol=0, atol=1e-12), n


def test_shared_heads_equal_repeated_heads():
    rng = np.random.default_rng(1)
    q, k, v = _qkv(rng, 1, 4, 2, 9, 30)
    do = rng.standard_normal(q.shape)
    r = oracle.window_attn(q, k, v, 7, 2, 21, 0.25, do)
    w = oracle.window_attn(q, k.repeat(2, axis=2), v.repeat(2, axis=2), 7, 2, 21, 0.25, do)
    assert np.allclose(r["o"], w["o"]) and np.allclose(r["dq"], w["dq"])
    for n in ("dk", "dv"):
        assert np.allclose(r[n], w[n].reshape(1, 30, 2, 2, -1).sum(axis=3))


def test_gradients_by_differences():
    rng = np.random.default_rng(2)
    q, k, v = _qkv(rng, 1, 2, 1, 6, 10, D=4)
    do = rng.standard_normal(q.shape)
    args = (3, 2, 4, 0.5)
    r = oracle.window_attn(q, k, v, *args, do)
    loss = lambda q, k, v: (oracle.window_attn(q, k, v, *args)["o"] * do).sum()  # noqa: E731
    for n, x in (("dq", q), ("dk", k), ("dv", v)):
        for idx in np.ndindex(*x.shape):
            hi, lo = x.copy(), x.copy()
            hi[idx] += 1e-5
            lo[idx] -= 1e-5
            f = [loss(*[y if z is x else z for z in (q, k, v)]) for y in (hi, lo)]
            assert abs((f[0] - f[1]) / 2e-5 - r[n][idx]) < 1e-8, (n, idx)


def test_empty_rows():
    rng = np.random.default_rng(3)
    q, k, v = _qkv(rng, 1, 1, 1, 8, 5)
    r = oracle.window_attn(q, k, v, 2, 0, -2, 0.3, rng.standard_normal(q.shape))
    assert np.isneginf(r["lse"][0, 0]).tolist() == [True, True, False, False, False, False, False, False]
    r = oracle.window_attn(q, k, v, 2, 0, 3, 0.3, rng.standard_normal(q.shape))
    assert np.isneginf(r["lse"][0, 0]).tolist() == [False] * 3 + [True] * 5
    assert (r["o"][0, 3:] == 0).all() and (r["dq"][0, 3:] == 0).all()


def test_rope_axes_with_one_position_is_rope():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((2, 7, 3, 128))
    pos = np.broadcast_to(50 + np.arange(7), (3, 7))
    y = oracle.rope_axes(x, 1e6, pos, [k % 3 for k in range(64)])
    assert np.allclose(y, oracle.rope(x, 1e6, 50), rtol=0, atol=1e-12)
    assert np.allclose(oracle.rope_axes(y, 1e6, pos, [k % 3 for k in range(64)], inverse=True), x, rtol=0, atol=1e-12)


def test_pair_axes():
    assert lcb.rope_pair_axes((16, 24, 24)) == [0] * 16 + [1] * 24 + [2] * 24
    assert lcb.rope_pair_axes((2, 62), interleaved=True) == [0, 1, 0, 1] + [1] * 60
    assert lcb.rope_pair_axes((20, 22, 22), interleaved=True)[:7] == [0, 1, 2, 0, 1, 2, 0]
    assert lcb.rope_pair_axes((0, 64)) == [1] * 64
    for bad in ((), (64, 1), (63,), (65, -1)):
        with pytest.raises(ValueError):
            lcb.rope_pair_axes(bad)


# ------------------------------------------------------------------ refusals, before any CUDA call

NUL, FAKE = ctypes.c_void_p(0), ctypes.c_void_p(1 << 20)
ARG, UNSUP = _lib.LCB_ERR_ARG, _lib.LCB_ERR_UNSUPPORTED


def _fwd(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, B=2, H=4, Hkv=2, Sq=64, Sk=64, D=128, window=8, sinks=0, pos0=0,
         scale=0.1, qs=(512, 512 * 64), ks=(256, 256 * 64), os=(512, 512 * 64), ls=(64, 256)):
    return _lib.load().attn_window_fwd(q, k, v, o, lse, B, H, Hkv, Sq, Sk, D, window, sinks, pos0, scale, *qs, *ks, *os,
                                       *ls, NUL)


def _bwd(dq=FAKE, dk=FAKE, dv=FAKE, o=FAKE, do=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 40, B=2, H=4, Hkv=2, Sq=64, Sk=64,
         D=128, window=8, sinks=0, pos0=0, scale=0.1, os=(512, 512 * 64), dqs=(512, 512 * 64), dks=(256, 256 * 64)):
    return _lib.load().attn_window_bwd(FAKE, FAKE, FAKE, o, lse, do, dq, dk, dv, B, H, Hkv, Sq, Sk, D, window, sinks,
                                       pos0, scale, 512, 512 * 64, 256, 256 * 64, *os, 64, 256, *dqs, *dks, ws, ws_bytes,
                                       NUL)


def _dec(lens=FAKE, B=2, H=4, Hkv=2, T=2, Smax=64, D=128, window=8, sinks=0, o=FAKE, os=(512, 1024)):
    return _lib.load().attn_window_decode(FAKE, FAKE, FAKE, lens, o, FAKE, B, H, Hkv, T, Smax, D, window, sinks, 0.1,
                                          512, 1024, 256, 256 * 64, *os, T, 4 * T, NUL)


@pytest.mark.parametrize("kw,want", [
    (dict(D=64), UNSUP), (dict(Hkv=3), ARG), (dict(Hkv=0), ARG), (dict(B=0), ARG), (dict(Sq=-1), ARG),
    (dict(window=0), ARG), (dict(sinks=-1), ARG), (dict(scale=-0.1), ARG), (dict(scale=float("nan")), ARG),
    (dict(pos0=(1 << 28) + 1), ARG), (dict(pos0=-(1 << 28) - 1), ARG), (dict(Sk=(1 << 28) + 1), ARG),
    (dict(q=NUL), ARG), (dict(k=NUL), ARG), (dict(v=NUL), ARG), (dict(o=NUL), ARG), (dict(lse=NUL), ARG),
    (dict(q=ctypes.c_void_p(8)), ARG), (dict(o=ctypes.c_void_p(8)), ARG), (dict(qs=(510, 512 * 64)), ARG),
    (dict(ks=(128, 256 * 64)), ARG), (dict(os=(256, 512 * 64)), ARG), (dict(os=(512, 0)), ARG),
    (dict(os=(512, 512)), ARG), (dict(ls=(-1, 0)), ARG), (dict(Sq=0), _lib.LCB_OK)])
def test_fwd_refusals(kw, want):
    assert _fwd(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(D=64), UNSUP), (dict(Hkv=3), ARG), (dict(window=0), ARG), (dict(scale=0.0), ARG), (dict(dq=NUL), ARG),
    (dict(dk=NUL), ARG), (dict(dv=ctypes.c_void_p(8)), ARG), (dict(o=NUL), ARG), (dict(do=NUL), ARG),
    (dict(lse=NUL), ARG), (dict(ws=NUL), ARG), (dict(ws=ctypes.c_void_p(8)), ARG), (dict(ws_bytes=100), ARG),
    (dict(dqs=(512, 0)), ARG), (dict(dks=(256, 0)), ARG), (dict(dks=(250, 256 * 64)), ARG),
    (dict(os=(500, 512 * 64)), ARG), (dict(Sq=0, Sk=0), _lib.LCB_OK)])
def test_bwd_refusals(kw, want):
    assert _bwd(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(lens=NUL), ARG), (dict(lens=ctypes.c_void_p(2)), ARG), (dict(T=-1), ARG), (dict(window=0), ARG),
    (dict(Hkv=3), ARG), (dict(D=96), UNSUP), (dict(os=(512, 512)), ARG), (dict(o=ctypes.c_void_p(4)), ARG),
    (dict(T=0), _lib.LCB_OK)])
def test_decode_refusals(kw, want):
    assert _dec(**kw) == want


def test_rope_axes_refusals():
    lib = _lib.load()
    axes = (ctypes.c_int * 64)(*([0] * 32 + [1] * 32))

    def call(x=FAKE, S=8, D=128, theta=1e6, pos=FAKE, pb=4, n=2, arr=axes, ps=(8, 0, 1), inverse=0, rs=256, bs=0, B=1):
        return lib.lcb_rope_axes(x, FAKE, B, S, 2, D, theta, pos, pb, n, arr, *ps, inverse, rs, bs, NUL)
    assert call(D=64) == UNSUP and call(pb=2) == UNSUP
    for kw in (dict(theta=0.0), dict(theta=1e-310), dict(theta=float("inf")), dict(n=1), dict(n=0), dict(n=65), dict(arr=None),
               dict(pos=NUL), dict(pos=ctypes.c_void_p(6)), dict(pos=ctypes.c_void_p(12), pb=8), dict(ps=(-1, 0, 1)),
               dict(inverse=2), dict(rs=255), dict(rs=128), dict(x=ctypes.c_void_p(2)), dict(B=2, bs=0),
               dict(B=2, bs=256)):
        assert call(**kw) == ARG, kw
    assert call(S=0) == _lib.LCB_OK


def test_workspace_covers_statistics_dq_and_partials():
    n = lcb.attn_window_bwd_workspace_bytes
    tile = 65536 + 1024  # an fp32 dQ tile and two row statistics
    assert n(1, 2, 2, 300, 300, 64) == 2 * 3 * tile
    # a sink tile seen by all of a long sequence: its list is cut into runs, each with an fp32 dK and dV
    base = 4 * 512 * tile
    assert n(1, 4, 1, 65536, 65536, 128, 0) == base
    more = n(1, 4, 1, 65536, 65536, 128, 4) - base
    assert more > 0 and more % (2 * 65536) == 0
    assert n(1, 2, 2, 0, 300, 64) == 0 and n(1, 2, 2, 300, 300, 0) == 0 and n(1, 3, 2, 300, 300, 64) == 0


def test_python_refusals_without_a_gpu():
    q = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        lcb.attn_window_fwd(q, q, q, 4)
    with pytest.raises(ValueError, match="CUDA"):
        lcb.rope_axes(q, 1e4, torch.zeros(1, 4, dtype=torch.int32), (64,))
    with pytest.raises(ValueError, match="sections"):
        lcb.rope_axes(q, 1e4, torch.zeros(1, 4, dtype=torch.int32), (63,))
