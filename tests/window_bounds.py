"""How far the windowed-attention kernels may be from the fp64 oracle, element
by element, derived from what they round and nothing else.

U = 2^-8 is half a bf16 step relative to the value. E covers the fp32 parts:
a score is a 128-term fp32 sum, off by at most 128 * 2^-24 * scale * sum |q k|
(with a margin of two for its products with log2 e), which moves P by that much
relatively; ex2.approx and the row sums add under 2^-20.

  O  = round(sum_j round(P_j) v_j / l):  U |O| + (U + E) (P |V|)
  dV = round(sum_i round(P_i) dO_i):     U |dV| + (U + E) (P^T |dO|)
  Delta_i = dO_i . round(O_i):           |dO_i| . (bound of O_i) =: dD_i
  dS = round(scale P (dP - Delta)):      |dS| (U + E) + scale P (dD + E |dO||v|) =: dS'
  dQ = round(sum_j dS_j k_j):            U |dQ| + dS' |K|
  dK = round(sum_i dS_i q_i):            U |dK| + dS'^T |Q|
"""

import numpy as np

import oracle

U = 2.0 ** -8


def check_attn(q, k, v, window, sinks, q_pos0, scale, o, lse, do=None, grads=None, name=""):
    """All arguments fp64 numpy; o, lse, grads (dq, dk, dv; None: not checked) are what the kernels gave."""
    r = oracle.window_attn(q, k, v, window, sinks, q_pos0, scale, do)
    B, Sq, H, D = q.shape
    G = H // k.shape[2]
    assert np.isfinite(o).all(), f"{name} O: non-finite"
    seen = np.isfinite(r["lse"])
    assert np.array_equal(np.isfinite(lse), seen) and (lse[~seen] == -np.inf).all(), f"{name} LSE: empty rows differ"
    b_o = np.zeros_like(r["o"])
    b_dq = np.zeros_like(r["o"])
    b_dk, b_dv = np.zeros(k.shape), np.zeros(k.shape)
    for b in range(B):
        for h in range(H):
            kh, vh, qh = np.abs(k[b, :, h // G]), np.abs(v[b, :, h // G]), np.abs(q[b, :, h])
            p = r["p"][b, h]
            ds_score = 2 * 128 * 2.0 ** -24 * scale * (qh @ kh.T)
            E = (ds_score * (p > 0)).max(axis=1, initial=0.0)[:, None] * 2 + 2.0 ** -20
            lerr = np.abs(lse[b, h][seen[b, h]] - r["lse"][b, h][seen[b, h]])
            ltol = (E[:, 0] + 2.0 ** -21 * (1 + np.abs(r["lse"][b, h], where=seen[b, h], out=np.zeros(Sq))))[seen[b, h]]
            assert (lerr <= ltol).all(), f"{name} LSE: off by {(lerr / ltol).max():.2f} bounds"
            b_o[b, :, h] = U * np.abs(r["o"][b, :, h]) + (U + E) * (p @ vh)
            if do is None:
                continue
            dh = np.abs(do[b, :, h])
            dd = (dh * b_o[b, :, h]).sum(axis=1, keepdims=True)
            ds = np.abs(r["ds"][b, h]) * (U + E) + scale * p * (dd + E * (dh @ vh.T))
            b_dq[b, :, h] = U * np.abs(r["dq"][b, :, h]) + ds @ kh
            b_dk[b, :, h // G] += ds.T @ qh
            b_dv[b, :, h // G] += ((U + E) * p).T @ dh
    todo = [("O", o, r["o"], b_o)]
    if do is not None:
        b_dk += U * np.abs(r["dk"])
        b_dv += U * np.abs(r["dv"])
        todo += [("dQ", grads[0], r["dq"], b_dq), ("dK", grads[1], r["dk"], b_dk), ("dV", grads[2], r["dv"], b_dv)]
    for n, got, want, bound in todo:
        if got is None:
            continue
        assert np.isfinite(got).all(), f"{name} {n}: non-finite"
        err = np.abs(got - want)
        bad = err > bound + 1e-30
        assert not bad.any(), (f"{name} {n}: {int(bad.sum())} of {bad.size} values off by up to "
                               f"{(err / (bound + 1e-30)).max():.2f} bounds, first at {np.argwhere(bad)[0]}")
    return r
