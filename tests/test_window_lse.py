"""LSE outputs whose rows share an element are refused, as such O outputs are,
before any CUDA call; layouts that keep them apart are not."""

import ctypes

import pytest

from long_context_causal_blockwise_gb300 import _lib

NUL, FAKE = ctypes.c_void_p(0), ctypes.c_void_p(1 << 20)
ARG = _lib.LCB_ERR_ARG
B, H, S, D = 2, 4, 64, 128
# (head stride, batch stride)
SHARED = [(0, 256), (64, 0), (63, 256), (64, 255), (64, 64), (128, 63), (0, 0)]


def _fwd(ls, sk=64):
    return _lib.load().attn_window_fwd(FAKE, FAKE, FAKE, FAKE, FAKE, B, H, 2, S, sk, D, 8, 0, 0, 0.1, 512, 512 * S, 256,
                                       256 * 64, 512, 512 * S, *ls, NUL)


def _decode(ls):
    return _lib.load().attn_window_decode(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, B, H, 2, S, 64, D, 8, 0, 0.1, 512, 512 * S,
                                          256, 256 * 64, 512, 512 * S, *ls, NUL)


@pytest.mark.parametrize("ls", SHARED)
def test_shared_rows_are_refused(ls):
    assert [_fwd(ls), _fwd(ls, sk=0), _decode(ls)] == [ARG] * 3


@pytest.mark.gpu
@pytest.mark.parametrize("S,order", [(1, (0, 1, 2)), (1, (1, 0, 2)), (1, (0, 2, 1)), (64, (0, 1, 2)), (64, (1, 0, 2))])
def test_rows_apart_are_not(S, order):
    """lse as a view of [B, H, S], [H, B, S] and (one row) [B, S, H] buffers with gaps: the values of a fresh one, and
    the gaps left alone."""
    import torch

    import long_context_causal_blockwise_gb300 as lcb

    g = torch.Generator(device="cuda").manual_seed(S)
    q, k, v = (torch.randn(B, n, h, D, generator=g, device="cuda").to(torch.bfloat16) for n, h in ((S, H), (64, 2), (64, 2)))
    _, want = lcb.attn_window_fwd(q, k, v, 20)
    lens = torch.full((B,), 64, dtype=torch.int32, device="cuda")
    for call in (lambda x: lcb.attn_window_fwd(q, k, v, 20, lse=x), lambda x: lcb.attn_window_decode(q, k, v, lens, 20, lse=x)):
        buf = torch.full([(B, H, S)[i] + 1 for i in order], 7.0, device="cuda")
        lse = buf.permute(*(order.index(i) for i in range(3)))[:B, :H, :S]
        call(lse)
        torch.cuda.synchronize()
        assert (lse - want).abs().max() <= 2e-5
        lse.fill_(7.0)
        assert (buf == 7.0).all()
