"""Float64 NumPy oracle of the attention sublayer: per-head RMSNorm of queries
and keys with the position rotation (forward and backward), and causal
attention of new tokens over a cache.  Written from the formulas, one sequence
and one head at a time; it shares no code with the CUDA library.
"""

from __future__ import annotations

import numpy as np


def rotation(cos_sin, positions, rot, dh, adjacent):
    """The rotation of each token as a matrix [T, dh, dh] (y = R z)."""
    T = len(positions)
    R = np.zeros((T, dh, dh))
    R[:, np.arange(dh), np.arange(dh)] = 1.0
    half = rot // 2
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if adjacent else (j, j + half)
        c = np.asarray(cos_sin, np.float64)[positions, j]
        s = np.asarray(cos_sin, np.float64)[positions, half + j]
        R[:, a, a], R[:, a, b] = c, -s
        R[:, b, b], R[:, b, a] = c, s
    return R


def norm_rope(x, w, R, eps):
    """x [T, H, dh] -> R (x w / sqrt(mean(x^2) + eps))."""
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    return np.einsum("tij,thj->thi", R, x * r * np.asarray(w, np.float64))


def norm_rope_bwd(g, x, w, R, eps):
    """Gradients (dx, dw) of <g, norm_rope(x, w)>."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    dh = x.shape[-1]
    r = 1.0 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    h = np.einsum("tji,thj->thi", R, np.asarray(g, np.float64))
    u = h * w
    dx = r * u - x * r ** 3 * (u * x).sum(-1, keepdims=True) / dh
    return dx, (h * x * r).sum((0, 1))


def attention(q, k, v, scale, window=0, softcap=0.0):
    """Causal attention of the n rows of q [n, Hq, dh], the newest of the m
    cached tokens k, v [m, Hk, dh].  Returns o [n, Hq, dh], lse [n, Hq], and for
    error bounds sum_j p_j |v_j| (as o) and max_j scale sum_d |q_d k_d| (as lse)
    over the keys a row sees."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    n, hq, dh = q.shape
    m, hk, _ = k.shape
    o, pabs = np.zeros((n, hq, dh)), np.zeros((n, hq, dh))
    lse, size = np.full((n, hq), -np.inf), np.zeros((n, hq))
    for i in range(n):
        last = m - n + i
        first = max(0, last - window + 1) if window else 0
        if last < first:
            continue
        for h in range(hq):
            kk, vv = k[first:last + 1, h // (hq // hk)], v[first:last + 1, h // (hq // hk)]
            z = kk @ q[i, h] * scale
            if softcap > 0:
                z = softcap * np.tanh(z / softcap)
            top = z.max()
            e = np.exp(z - top)
            lse[i, h] = top + np.log(e.sum())
            p = e / e.sum()
            o[i, h] = p @ vv
            pabs[i, h] = p @ np.abs(vv)
            size[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * scale
    return o, lse, pabs, size
