"""Float64 causal attention over packed sequences with grouped heads, and its
gradients, with the element-wise magnitudes that rounding bounds are made of.

Plain NumPy, one (sequence, query head) at a time, from the formulas: within a
sequence S = scale q k^T for j <= i, P = exp(S - lse), o = P v; with
delta = rowsum(dO * o), dS = P (dO v^T - delta): dv = P^T dO,
dk = scale dS^T q, dq = scale dS k, the sums of dk and dv over the query
heads of a K/V head.  Shares no code with the CUDA path.
"""

import numpy as np


def starts(lengths):
    return np.concatenate([[0], np.cumsum(np.asarray(lengths, dtype=np.int64))])


def _scores(q, k, scale):
    n = q.shape[0]
    s = scale * (q @ k.T)
    s[np.triu_indices(n, 1)] = -np.inf
    return s


def forward(q, k, v, lengths, scale=None):
    """q [T, Hq, D], k, v [T, Hkv, D] float64 -> o, lse [Hq, T], and sum_j P_ij |v_j| (of o's shape).
    Rows behind the last sequence are zero."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    o, mag, lse = np.zeros_like(q), np.zeros_like(q), np.zeros((Hq, T))
    c = starts(lengths)
    for a, b in zip(c[:-1], c[1:]):
        if a == b:
            continue
        for h in range(Hq):
            s = _scores(q[a:b, h], k[a:b, h // G], scale)
            m = s.max(-1, keepdims=True)
            e = np.exp(s - m)
            z = e.sum(-1, keepdims=True)
            lse[h, a:b] = (m + np.log(z))[:, 0]
            o[a:b, h] = e @ v[a:b, h // G] / z
            mag[a:b, h] = e @ np.abs(v[a:b, h // G]) / z
    return o, lse, mag


def backward(q, k, v, o, lse, dO, lengths, scale=None):
    """dq, dk, dv from the given o and lse, and a dict of magnitudes: for dq ``scale sum |dS| |k|`` and
    ``scale sum P |k|``, the same for dk with |q|, and ``sum P |dO|`` and ``sum |dO|`` for dv."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(k)
    mag = {n: np.zeros_like(x) for n, x in (("dq_ds", q), ("dq_p", q), ("dq_n", q), ("dk_ds", k), ("dk_p", k),
                                            ("dk_n", k), ("dv_p", k), ("dv_n", k))}
    c = starts(lengths)
    for a, b in zip(c[:-1], c[1:]):
        if a == b:
            continue
        for h in range(Hq):
            g = h // G
            qq, kk, vv, gg = q[a:b, h], k[a:b, g], v[a:b, g], dO[a:b, h]
            p = np.exp(_scores(qq, kk, scale) - lse[h, a:b, None])
            keep = np.tril(np.ones_like(p))
            ds = p * (gg @ vv.T - (gg * o[a:b, h]).sum(-1, keepdims=True))
            dq[a:b, h] = scale * (ds @ kk)
            dk[a:b, g] += scale * (ds.T @ qq)
            dv[a:b, g] += p.T @ gg
            mag["dq_ds"][a:b, h] = scale * (np.abs(ds) @ np.abs(kk))
            mag["dq_p"][a:b, h] = scale * (p @ np.abs(kk))
            mag["dq_n"][a:b, h] = scale * (keep @ np.abs(kk))
            mag["dk_ds"][a:b, g] += scale * (np.abs(ds).T @ np.abs(qq))
            mag["dk_p"][a:b, g] += scale * (p.T @ np.abs(qq))
            mag["dk_n"][a:b, g] += scale * (keep.T @ np.abs(qq))
            mag["dv_p"][a:b, g] += p.T @ np.abs(gg)
            mag["dv_n"][a:b, g] += keep.T @ np.abs(gg)
    return dq, dk, dv, mag
