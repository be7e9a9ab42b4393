"""The cache in 4 or 8 bits without a GPU: the oracle pinned, the arithmetic
that the write kernel relies on, and the refusals of the entry points."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
import long_context_causal_blockwise_gb300 as lcb
from long_context_causal_blockwise_gb300 import _lib


def test_round_bf16_is_torchs():
    x = np.random.default_rng(0).standard_normal(4000) * 2.0 ** np.random.default_rng(1).integers(-60, 60, 4000)
    x = np.concatenate([x, (2 * np.arange(128, 256) + 1) / 512.0])  # midpoints between neighbours
    assert np.array_equal(oracle.round_bf16(x), torch.from_numpy(x).to(torch.bfloat16).double().numpy())


@pytest.mark.parametrize("bits", [4, 8])
def test_oracle_by_hand(bits):
    m = 7 if bits == 4 else 127
    x = np.zeros((1, 128))
    x[0, :4] = [m, -m, 2.5, -0.5]         # scale 1: ties go away from zero
    x[0, 32:35] = [2.0 * m, 3.0, 2.9]     # scale 2
    x[0, 64:66] = [2.0 ** -101, -2.0 ** -120]
    x[0, 96] = np.inf
    n, s = oracle.cache_codes(x, bits)
    assert s[0, 0, 0] == 1 and s[0, 1, 0] == 2 and s[0, 2, 0] == 0 and np.isnan(s[0, 3, 0])
    assert n[0, 0, :4].tolist() == [m, -m, 3, -1] and n[0, 1, :3].tolist() == [m, 2, 1]
    v = oracle.cache_values(x, bits)
    assert v[0, 32:35].tolist() == [2 * m, 4, 2] and (v[0, 64:96] == 0).all() and np.isnan(v[0, 96:]).all()


@pytest.mark.parametrize("bits", [4, 8])
def test_oracle_error_bound(bits):
    x = np.random.default_rng(bits).standard_normal((500, 128))
    x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    n, s = oracle.cache_codes(x, bits)
    m = 2 ** (bits - 1) - 1
    assert np.abs(n).max() == m  # the scale's rounding never lifts a number past m
    err = np.abs(oracle.cache_values(x, bits) - x).reshape(500, 4, 32)
    top = np.abs(x).reshape(500, 4, 32).max(axis=-1, keepdims=True)
    assert (err <= s / 2 + 2.0 ** -8 * top).all()


@pytest.mark.parametrize("m", [7, 127])
def test_one_multiplication_rounds_as_the_division(m):
    """x * inv with inv = fp32(r * (1 + 2^-20)), rounded to the nearest whole number, is x / s rounded with ties away from
    zero, for every pair of bf16 significands at every distance that a group has, and r = 1 / s to two steps either way."""
    S = np.arange(128, 256, dtype=np.float64)[:, None]
    for off in (-2, -1, 0, 1, 2):
        r = (np.float32(1) / S.astype(np.float32)).astype(np.float32)
        r = (r.view(np.int32) + off).view(np.float32)
        inv = (r * np.float32(1 + 2.0 ** -20)).astype(np.float64)
        for e in range(-3, 9):
            x = np.arange(128, 256, dtype=np.float64)[None, :] * 2.0 ** e
            q = x / S
            want = np.floor(q + 0.5)
            got = np.rint(x * inv)  # 8 by 24 bits: the product is exact in fp64, as inside the fused multiply-add
            use = q <= m * (1 + 2.0 ** -8)
            assert np.array_equal(got[use], want[use])
            assert (want[use] <= m).all()


def test_scales_are_one_rounding():
    """fp32(max * fp32(1 / m)) rounded to bf16 is max / m rounded to bf16: no quotient lies next to a midpoint."""
    X = np.arange(128, 256, dtype=np.float32)
    for m in (7, 127):
        q32 = (X * (np.float32(1) / np.float32(m))).astype(np.float64)
        assert np.array_equal(oracle.round_bf16(q32), oracle.round_bf16(X.astype(np.float64) / m))


NUL, FAKE = ctypes.c_void_p(0), ctypes.c_void_p(1 << 20)  # aligned, never dereferenced
ERR_ARG, ERR_UNSUPPORTED, OK = _lib.LCB_ERR_ARG, _lib.LCB_ERR_UNSUPPORTED, _lib.LCB_OK


def test_row_bytes():
    lib = _lib.load()
    for bits, n in _lib._ROW_BYTES.items():
        assert lib.lcb_kv_cache_row_bytes(bits) == n
    assert lib.lcb_kv_cache_row_bytes(5) == ERR_UNSUPPORTED


def test_write_and_read_refusals_need_no_gpu():
    lib = _lib.load()

    def write(cache=FAKE, k=FAKE, v=FAKE, lens=FAKE, B=2, Hkv=2, T=4, Smax=10, D=128, bits=4, cb=2880, ch=1440, rs=256,
              bs=1024):
        return lib.lcb_kv_cache_write(cache, k, v, lens, B, Hkv, T, Smax, D, bits, cb, ch, rs, bs, NUL)

    def read(cache=FAKE, k=FAKE, v=FAKE, lens=NUL, B=2, Hkv=2, n=4, start=0, Smax=10, D=128, bits=4, cb=2880, ch=1440,
             rs=256, bs=1024):
        return lib.lcb_kv_cache_read(cache, k, v, lens, B, Hkv, n, start, Smax, D, bits, cb, ch, rs, bs, NUL)

    for call in (write, read):
        assert call(D=64) == ERR_UNSUPPORTED and call(bits=5) == ERR_UNSUPPORTED
        for bad in (dict(B=0), dict(Hkv=0), dict(Smax=-1), dict(cache=NUL), dict(k=NUL), dict(v=NUL),
                    dict(cache=ctypes.c_void_p(8)), dict(k=ctypes.c_void_p((1 << 20) + 8)), dict(ch=1448), dict(cb=-16),
                    dict(rs=128), dict(rs=260), dict(lens=ctypes.c_void_p((1 << 20) + 2)), dict(Smax=(1 << 28) + 1)):
            assert call(**bad) == ERR_ARG, bad
    assert write(lens=NUL) == ERR_ARG and write(T=-1) == ERR_ARG
    assert write(ch=1424) == ERR_ARG and write(cb=1440) == ERR_ARG  # heads, or sequences, of the output overlap
    for B, Hkv in ((2 ** 31 - 1, 2), (2, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 1)):  # strides times counts past 64 bits
        assert write(B=B, Hkv=Hkv, ch=2 ** 39, cb=2 ** 39, rs=2 ** 38 - 8, bs=2 ** 38 - 8) == ERR_ARG
    assert write(T=0, cache=NUL) == OK and write(Smax=0, cache=NUL) == OK
    assert read(start=7) == ERR_ARG and read(start=-1) == ERR_ARG and read(n=11) == ERR_ARG and read(n=-1) == ERR_ARG
    assert read(bs=512) == ERR_ARG  # sequences of the output overlap
    assert read(n=0, cache=NUL) == OK


def test_attention_refusals_need_no_gpu():
    lib = _lib.load()

    def call(q=FAKE, cache=FAKE, lens=FAKE, o=FAKE, lse=FAKE, B=2, H=4, Hkv=2, T=1, Smax=10, D=128, bits=4, window=5,
             sinks=1, scale=0.1, qr=512, qb=512, cb=2880, ch=1440, orr=512, ob=512, lh=1, lb=4):
        return lib.attn_cache_decode(q, cache, lens, o, lse, B, H, Hkv, T, Smax, D, bits, window, sinks, scale, qr, qb,
                                     cb, ch, orr, ob, lh, lb, NUL, 0, NUL)

    assert call(D=64) == ERR_UNSUPPORTED and call(bits=3) == ERR_UNSUPPORTED
    for bad in (dict(B=0), dict(H=3), dict(Hkv=0), dict(T=-1), dict(window=0), dict(sinks=-1), dict(scale=0.0),
                dict(scale=float("nan")), dict(q=NUL), dict(cache=NUL), dict(lens=NUL), dict(o=NUL), dict(lse=NUL),
                dict(ch=1448), dict(qr=500), dict(ob=0), dict(lh=0), dict(cache=ctypes.c_void_p(8)),
                dict(lens=ctypes.c_void_p((1 << 20) + 1)), dict(Smax=(1 << 28) + 1), dict(T=(1 << 28) + 1)):
        assert call(**bad) == ERR_ARG, bad
    assert call(T=0, q=NUL) == OK
    assert lib.attn_cache_decode_workspace_bytes(1, 3, 2, 1, 10, 128, 4, 5, 0) == 0  # a refused size
    assert lib.attn_cache_decode_form(1, 3, 2, 1, 10, 128, 4, 5, 0) == ERR_ARG
    assert lib.attn_cache_decode_form(1, 4, 2, 1, 10, 64, 4, 5, 0) == ERR_UNSUPPORTED
    assert lib.attn_cache_decode_form(1, 4, 2, 1, 10, 128, 5, 5, 0) == ERR_UNSUPPORTED
    assert lib.attn_cache_decode_form(1, 4, 2, 0, 10, 128, 4, 5, 0) == 0
    with pytest.raises(lcb.AttnError):
        lcb.attn_cache_decode_form(1, 4, 2, 1, 10, 4, window=-3)
    assert lib.attn_cache_decode_workspace_bytes(1, 4, 2, 1, 0, 128, 4, 5, 0) == 0


def test_python_refusals():
    cache = lcb.kv_cache_empty(2, 2, 16, device="cpu")
    assert cache.shape == (2, 2, 16, 144) and lcb.kv_cache_empty(1, 1, 4, bits=8, device="cpu").shape[3] == 272
    k = torch.zeros(2, 3, 2, 128, dtype=torch.bfloat16)
    lens = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        lcb.kv_cache_empty(1, 1, 4, bits=3)
    for bad in (cache.float(), cache[0], cache[..., :100], cache[:, :, ::2],
                torch.zeros(2, 2, 16, 288, dtype=torch.uint8)[..., ::2]):
        with pytest.raises(ValueError):
            lcb.kv_cache_write(bad, k, k, lens)
        with pytest.raises(ValueError):
            lcb.kv_cache_read(bad, 1)
        with pytest.raises(ValueError):
            lcb.attn_cache_decode(k, bad, lens)
    for kk, vv, ll in ((k[:1], k[:1], lens), (k[:, :, :1], k[:, :, :1], lens), (k.float(), k, lens), (k, k[:, :2], lens),
                       (k, k.transpose(0, 1).contiguous().transpose(0, 1), lens), (k, k, lens.long()), (k, k, lens[:1]),
                       (k[..., :64], k[..., :64], lens)):
        with pytest.raises(ValueError):
            lcb.kv_cache_write(cache, kk, vv, ll)
    for n, start in ((-1, 0), (17, 0), (1, 16), (1, -1)):
        with pytest.raises(ValueError):
            lcb.kv_cache_read(cache, n, start)
    with pytest.raises(ValueError):
        lcb.kv_cache_read(cache, 3, k=k[:, :2])
    for q in (k[:1], torch.zeros(2, 1, 3, 128, dtype=torch.bfloat16), k.float(), k[..., :64]):
        with pytest.raises(ValueError):
            lcb.attn_cache_decode(q, cache, lens)
    with pytest.raises(ValueError):  # everything in order, but not on a GPU
        lcb.kv_cache_write(cache, k, k, lens)
    with pytest.raises(ValueError):
        lcb.kv_cache_read(cache, 2)


class _Library:
    """Answers as the library does in one device context, whose calls need `need` bytes; queries listed in `says` answer
    that instead (one that failed: 0)."""

    def __init__(self, need, says=()):
        self.need, self.says, self.given = need, list(says), []
        self.attn_status_string = _lib.load().attn_status_string

    def attn_cache_decode_workspace_bytes(self, *sizes):
        return self.says.pop(0) if self.says else self.need

    def attn_cache_decode(self, *args):
        self.given.append(args[-2])
        return OK if args[-2] >= self.need else ERR_ARG


def test_a_workspace_size_that_is_out_of_date_is_asked_for_again(monkeypatch):
    cache = lcb.kv_cache_empty(1, 2, 16, device="cpu")
    q, lens = torch.zeros(1, 1, 4, 128, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    monkeypatch.setattr(_lib, "_raw_stream", lambda *args: 0)
    _lib._cache_decode_workspace.cache_clear()

    def calls(lib, n, **kw):
        monkeypatch.setattr(_lib, "_LIB", lib)
        for _ in range(n):
            lcb.attn_cache_decode(q, cache, lens, **kw)
        return lib.given

    assert calls(_Library(64, says=[0]), 2) == [0, 64, 64]  # the first query failed
    assert calls(_Library(128), 2) == [64, 128, 128]        # a context with more SMs
    assert calls(_Library(96), 1) == [128]                  # and one with fewer
    assert lcb.attn_cache_decode_workspace_bytes(1, 4, 2, 1, 16) == 96  # what is said to the caller is never kept
    with pytest.raises(lcb.AttnError):                      # a size of the caller's own is refused as it is
        calls(_Library(256), 1, workspace=torch.empty(128, dtype=torch.uint8))
    with pytest.raises(lcb.AttnError):
        calls(_Library(1 << 40, says=[64, 64]), 1)          # still too little: an error, no second attempt
    _lib._cache_decode_workspace.cache_clear()
