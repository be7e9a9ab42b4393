"""fp64 oracle for attention with a sliding window and sinks, and for rotary
positions with several axes.

TEST INFRASTRUCTURE (see the package header): only tests/, the smoke check and
the bench's CPU-baseline leg may call this module.

Window and sinks: the query of row i stands at position p = q_pos0 + i; key j
is visible to it iff j <= p and (p - j < window or j < sinks). Query head h
reads K/V head h // (H // Hkv). Everything else is the textbook attention of
attention.py: softmax over the visible keys, a row without any gives O = 0,
LSE = -inf and takes no part in a gradient; dK and dV sum over the query heads
that share a K/V head. The whole mask and the whole probability matrix are
written out.

Several axes: feature pair k (features k and k + D/2) turns by
pos[axis[k]][token] * theta^(-2k/D).
"""

import numpy as np


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def window_visible(Sq, Sk, window, sinks, q_pos0):
    """Boolean [Sq, Sk]."""
    p = q_pos0 + np.arange(Sq)[:, None]
    j = np.arange(Sk)[None, :]
    return (j <= p) & ((p - j < window) | (j < sinks))


def window_attn(q, k, v, window, sinks, q_pos0, scale, do=None):
    """Returns a dict: o [B,Sq,H,D], lse [B,H,Sq], p [B,H,Sq,Sk] and, with do, ds (scale included) [B,H,Sq,Sk],
    dq [B,Sq,H,D], dk and dv [B,Sk,Hkv,D]."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, Sq, H, D = q.shape
    Sk, Hkv = k.shape[1], k.shape[2]
    G = H // Hkv
    vis = window_visible(Sq, Sk, window, sinks, q_pos0)
    r = dict(o=np.zeros((B, Sq, H, D)), lse=np.full((B, H, Sq), -np.inf), p=np.zeros((B, H, Sq, Sk)))
    if do is not None:
        do = _f64(do)
        r.update(ds=np.zeros((B, H, Sq, Sk)), dq=np.zeros((B, Sq, H, D)), dk=np.zeros((B, Sk, Hkv, D)),
                 dv=np.zeros((B, Sk, Hkv, D)))
    some = vis.any(axis=1)
    for b in range(B):
        for h in range(H):
            kh, vh = k[b, :, h // G], v[b, :, h // G]
            s = scale * (q[b, :, h] @ kh.T)
            for i in np.nonzero(some)[0]:
                x = s[i, vis[i]]
                m = x.max()
                e = np.exp(x - m)
                r["lse"][b, h, i] = m + np.log(e.sum())
                r["p"][b, h, i, vis[i]] = e / e.sum()
            p = r["p"][b, h]
            r["o"][b, :, h] = o = p @ vh
            if do is None:
                continue
            dh = do[b, :, h]
            ds = p * (dh @ vh.T - (dh * o).sum(axis=1, keepdims=True)) * scale
            r["ds"][b, h] = ds
            r["dq"][b, :, h] = ds @ kh
            r["dk"][b, :, h // G] += ds.T @ q[b, :, h]
            r["dv"][b, :, h // G] += p.T @ dh
    return r


def rope_axes(x, theta, pos, axis, inverse=False):
    """x [B, S, H, D]; pos [axes, S] or [axes, B, S]; axis: one axis number per feature pair."""
    x, pos = _f64(x), np.asarray(pos)
    B, S, H, D = x.shape
    if pos.ndim == 2:
        pos = np.broadcast_to(pos[:, None], (pos.shape[0], B, S))
    y = np.empty_like(x)
    for k in range(D // 2):
        a = pos[axis[k]].astype(np.float64) * float(theta) ** (-2.0 * k / D) * (-1.0 if inverse else 1.0)
        z = (x[..., k] + 1j * x[..., k + D // 2]) * np.exp(1j * a)[:, :, None]
        y[..., k], y[..., k + D // 2] = z.real, z.imag
    return y
