"""Float64 definitions of what stands in front of a mixer and of the linear attention with a decay for
each head: the norms of queries and keys with the rotation by position, and the recurrence token by
token, with their exact gradients.

Each function takes one sequence as numpy float64 and shares nothing with the CUDA library.  With
`absolute=True` every term of every sum is taken by its absolute value, so that a result bounds the
magnitude that the rounding errors of the same sum are relative to.
"""
from __future__ import annotations

import numpy as np


def _identity(v):
    return v


# --------------------------------------------------------------------------------- rotation


def angles(positions, freqs, sections):
    """[L, rot / 2] from positions [L, axes], freqs [rot / 2] and the pairs of each axis."""
    axis = np.repeat(np.arange(len(sections)), sections)
    return positions.astype(np.float64)[:, axis] * freqs


def _pairs(d, rot, neighbours):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if neighbours else (i, i + rot // 2)


def rotate(n, a, neighbours, sign=1.0, absolute=False):
    """The pairs of n [L, H, d] turned by sign a [L, rot / 2].  The errors of cosine and sine are relative
    to 1, whatever the angle: with absolute=True both count as 1."""
    m = np.abs if absolute else _identity
    one, two = _pairs(n.shape[-1], 2 * a.shape[1], neighbours)
    c, s = np.cos(a)[:, None], sign * np.sin(a)[:, None]
    if absolute:
        c, s = np.ones_like(c), -np.ones_like(s)
    y = m(n).copy()
    n1, n2 = m(n[..., one]), m(n[..., two])
    y[..., one] = n1 * c - n2 * s
    y[..., two] = n2 * c + (n1 * -s if absolute else n1 * s)
    return y


def _norm(x, eps):
    rs = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * rs, rs


def rope_fwd(x, w, a, neighbours, norm, eps, absolute=False):
    """y [L, H, d] of x [L, H, d], w [d], angles a."""
    n = _norm(x, eps)[0] * w if norm else x
    return rotate(n, a, neighbours, absolute=absolute)


def rope_bwd(x, w, a, neighbours, norm, eps, dy, absolute=False):
    """dx, dw."""
    m = np.abs if absolute else _identity
    dn = rotate(dy, a, neighbours, -1.0, absolute)
    if not norm:
        return dn, np.zeros_like(w)
    xh, rs = _norm(x, eps)
    t, xh = dn * m(w), m(xh)
    c = (t * xh).mean(-1, keepdims=True)
    return rs * (t + xh * c if absolute else t - xh * c), (dn * xh).sum((0, 1))


# ----------------------------------------------------------------------------------- decays


def decay_fwd(q, k, v, log_decay, s0, scale, absolute=False):
    """o [L, Hq, dv] and the last state [Hkv, dk, dv] of q [L, Hq, dk], k [L, Hkv, dk], v [L, Hkv, dv]."""
    m = np.abs if absolute else _identity
    L, Hq, _ = q.shape
    Hkv, dv = v.shape[1:]
    keep = np.exp(log_decay)[:, None, None]
    S, o = m(s0).copy(), np.zeros((L, Hq, dv))
    for t in range(L):
        S = keep * S + m(k[t])[:, :, None] * m(v[t])[:, None, :]
        o[t] = m(scale) * np.einsum("hgi,hij->hgj", m(q[t]).reshape(Hkv, Hq // Hkv, -1), S).reshape(Hq, dv)
    return o, S


def decay_bwd(q, k, v, log_decay, s0, scale, do, ds_out, absolute=False):
    """dq, dk, dv, ds0."""
    m = np.abs if absolute else _identity
    L, Hq, _ = q.shape
    Hkv = v.shape[1]
    keep = np.exp(log_decay)[:, None, None]
    heads = (Hkv, Hq // Hkv, -1)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    S = m(s0).copy()
    for t in range(L):
        S = keep * S + m(k[t])[:, :, None] * m(v[t])[:, None, :]
        dq[t] = m(scale) * np.einsum("hgj,hij->hgi", m(do[t]).reshape(heads), S).reshape(Hq, -1)
    D = m(ds_out).copy()
    for t in range(L - 1, -1, -1):
        D = D + m(scale) * np.einsum("hgi,hgj->hij", m(q[t]).reshape(heads), m(do[t]).reshape(heads))
        dk[t] = np.einsum("hij,hj->hi", D, m(v[t]))
        dv[t] = np.einsum("hij,hi->hj", D, m(k[t]))
        D = keep * D
    return dq, dk, dv, D
