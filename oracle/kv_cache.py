"""fp64 oracle for the K/V cache held in 4 or 8 bits.

TEST INFRASTRUCTURE (see the package header): only tests/ may call this module.

A row of 128 channels is held in groups of 32: with m = 2^(bits - 1) - 1, the
group's scale is s = max |x| / m rounded to bf16, and channel c is held as
n_c s, n_c = x_c / s rounded to the nearest whole number, ties away from zero.
A group whose largest magnitude is below 2^-100 holds zeros, one with an
infinity or a NaN holds NaN.
"""

import numpy as np

GROUP = 32


def round_bf16(x):
    """fp64 -> the nearest number of 8 significant bits, ties to even (no overflow, no subnormals)."""
    m, e = np.frexp(np.asarray(x, dtype=np.float64))
    return np.ldexp(np.rint(m * 256.0) / 256.0, e)


def cache_codes(x, bits):
    """(n, s) of x [..., 128]: whole numbers [..., 4, 32] and scales [..., 4, 1]; s is NaN in a non-finite group."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    bad = ~np.isfinite(g).all(axis=-1, keepdims=True)
    g = np.where(bad, 0.0, g)
    top = np.abs(g).max(axis=-1, keepdims=True)
    s = np.where(top < 2.0 ** -100, 0.0, round_bf16(top / (2 ** (bits - 1) - 1)))
    n = np.floor(np.abs(g) / np.where(s == 0, 1.0, s) + 0.5) * np.sign(g)
    return np.where(s == 0, 0.0, n), np.where(bad, np.nan, s)


def cache_values(x, bits):
    """The values that the cache holds for x [..., 128]."""
    n, s = cache_codes(x, bits)
    return (n * s).reshape(np.shape(x))
