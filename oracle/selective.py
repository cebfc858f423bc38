"""Float64 definitions of the selective state space block's operators, token by token: the short
causal convolution, the selective scan, and the norms, gate and residual around a block, with
their exact gradients.

Each function takes one sequence (tokens x channels) as numpy float64 and shares nothing with the
CUDA library.  With `absolute=True` every term of every sum is taken by its absolute value, so
that a result bounds the magnitude that the rounding errors of the same sum are relative to.
"""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    return np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def silu(v):
    return v * sigmoid(v)


def dsilu(v, absolute=False):
    s = sigmoid(v)
    return s + s * (1 - s) * (np.abs(v) if absolute else v)


def _identity(v):
    return v


# ------------------------------------------------------------------------------ convolution


def conv_fwd(x, w, bias, state, act: bool, absolute: bool = False):
    """y [L, C], final state [K-1, C], pre-activation [L, C] of x [L, C], w [C, K], bias [C],
    state [K-1, C]."""
    m = np.abs if absolute else _identity
    L, K = x.shape[0], w.shape[1]
    line = np.concatenate([state, x])
    pre = np.zeros_like(x)
    for t in range(L):
        pre[t] = m(bias)
        for j in range(K):
            pre[t] += m(w[:, j]) * m(line[t + j])
    y = pre * (1 if absolute else sigmoid(pre)) if act else pre
    return y, line[len(line) - (K - 1):], pre


def conv_bwd(x, w, bias, state, act: bool, dy, dstate_out, absolute: bool = False):
    """dx, dw, dbias, dstate_in."""
    m = np.abs if absolute else _identity
    L, K = x.shape[0], w.shape[1]
    line = np.concatenate([state, x])
    _, _, pre = conv_fwd(x, w, bias, state, act)
    dp = m(dy) * dsilu(pre, absolute) if act else m(dy)
    dline, dw = np.zeros_like(line), np.zeros_like(w)
    for t in range(L):
        for j in range(K):
            dline[t + j] += m(w[:, j]) * dp[t]
            dw[:, j] += dp[t] * m(line[t + j])
    if K > 1:
        dline[len(line) - (K - 1):] += m(dstate_out)
    return dline[K - 1:], dw, dp.sum(0), dline[:K - 1]


# ------------------------------------------------------------------------------------- scan


def _spread(v, C):  # [L, G, N] -> [L, C, N]
    return np.repeat(v, C // v.shape[1], axis=1)


def scan_fwd(x, dt, A, B, Cm, D, z, dt_bias, h0, use_softplus: bool = True, absolute: bool = False):
    """y [L, C] and the states after each token [L + 1, C, N] (entry 0 is h0)."""
    m = np.abs if absolute else _identity
    L, C = x.shape
    d = softplus(dt + dt_bias) if use_softplus else dt + dt_bias
    Bc, Cc = m(_spread(B, C)), m(_spread(Cm, C))
    h = [m(h0)]
    y = np.zeros_like(x)
    for t in range(L):
        h.append(np.exp(d[t][:, None] * A) * h[-1] + m(d[t] * x[t])[:, None] * Bc[t])
        y[t] = (Cc[t] * h[-1]).sum(-1) + m(D * x[t])
        if z is not None:
            y[t] *= m(silu(z[t]))
    return y, np.stack(h)


def scan_bwd(x, dt, A, B, Cm, D, z, dt_bias, h0, dy, dh_out, use_softplus: bool = True,
             absolute: bool = False):
    """A dict of dx, ddt, dA, dB, dC, dD, dz (None without z), ddt_bias, dh0."""
    m = np.abs if absolute else _identity
    L, C = x.shape
    G, N = B.shape[1:]
    raw = dt + dt_bias
    d = softplus(raw) if use_softplus else raw
    _, h = scan_fwd(x, dt, A, B, Cm, D, None, dt_bias, h0, use_softplus, absolute)
    Bc, Cc = m(_spread(B, C)), m(_spread(Cm, C))
    g = m(dh_out).copy()  # reaches the state from later tokens
    o = dict(dx=np.zeros_like(x), ddt=np.zeros_like(x), dz=None if z is None else np.zeros_like(x),
             dB=np.zeros_like(B), dC=np.zeros_like(Cm), dA=np.zeros_like(A), dD=np.zeros(C))
    for t in range(L - 1, -1, -1):
        e = m(dy[t] * silu(z[t]) if z is not None else dy[t])
        md, mx = m(d[t]), m(x[t])
        if z is not None:
            o["dz"][t] = m(dy[t]) * dsilu(z[t], absolute) * ((Cc[t] * h[t + 1]).sum(-1) + m(D * x[t]))
        g = g + Cc[t] * e[:, None]
        gb = (g * Bc[t]).sum(-1)
        o["dB"][t] = (g * (md * mx)[:, None]).reshape(G, C // G, N).sum(1)
        o["dC"][t] = (h[t + 1] * e[:, None]).reshape(G, C // G, N).sum(1)
        g = g * np.exp(d[t][:, None] * A)
        q = g * h[t]
        o["dx"][t] = md * gb + m(D) * e
        o["ddt"][t] = (mx * gb + (q * m(A)).sum(-1)) * (sigmoid(raw[t]) if use_softplus else 1)
        o["dA"] += q * md[:, None]
        o["dD"] += e * mx
    o["ddt_bias"] = o["ddt"].sum(0)
    o["dh0"] = g
    return o


# ------------------------------------------------------------------------------------- norm


def _gate(act: str, v):
    return silu(v) if act == "silu" else sigmoid(v)


def _dgate(act: str, v):
    return dsilu(v) if act == "silu" else sigmoid(v) * (1 - sigmoid(v))


def norm_fwd(o, gate, r, w_post, scale, w_pre, groups: int, act: str, gate_first: bool, eps: float):
    """r_out, n_out (None without w_pre); absent inputs are None."""
    T, D = o.shape
    n = o.copy()
    if gate is not None and gate_first:
        n = n * _gate(act, gate)
    if w_post is not None:
        for t in range(T):
            for k in range(groups):
                s = slice(k * D // groups, (k + 1) * D // groups)
                n[t, s] = w_post[s] * n[t, s] / np.sqrt(np.mean(n[t, s] ** 2) + eps)
    if gate is not None and not gate_first:
        n = n * _gate(act, gate)
    rr = n if scale is None else scale * n
    rr = rr if r is None else r + rr
    if w_pre is None:
        return rr, None
    return rr, np.stack([w_pre * v / np.sqrt(np.mean(v ** 2) + eps) for v in rr])


def norm_bwd(o, gate, r, w_post, scale, w_pre, groups: int, act: str, gate_first: bool, eps: float,
             dr_out, dn_out):
    """A dict of do, dgate, dr, dw_post, dscale, dw_pre (None for absent inputs)."""
    T, D = o.shape
    one = np.ones(D)
    first, last = gate is not None and gate_first, gate is not None and not gate_first
    a = _gate(act, gate) if gate is not None else np.ones_like(o)
    da = _dgate(act, gate) if gate is not None else None
    wp, sc = one if w_post is None else w_post, one if scale is None else scale
    out = dict(do=np.zeros_like(o), dgate=None if gate is None else np.zeros_like(o),
               dr=np.zeros_like(o), dw_post=np.zeros(D), dscale=np.zeros(D), dw_pre=np.zeros(D))
    for t in range(T):
        u = o[t] * a[t] if first else o[t]
        unit, root = u.copy(), np.ones(D)
        if w_post is not None:
            for k in range(groups):
                s = slice(k * D // groups, (k + 1) * D // groups)
                root[s] = np.sqrt(np.mean(u[s] ** 2) + eps)
            unit = u / root
        n = unit * wp * (a[t] if last else 1)
        rr = sc * n + (r[t] if r is not None else 0)
        g = dr_out[t].copy() if dr_out is not None else np.zeros(D)
        if w_pre is not None:
            q = np.sqrt(np.mean(rr ** 2) + eps)
            out["dw_pre"] += dn_out[t] * rr / q
            v = dn_out[t] * w_pre
            g += v / q - rr * np.mean(v * rr) / q ** 3
        out["dr"][t] = g
        out["dscale"] += g * n
        g = g * sc
        if last:
            out["dgate"][t] = g * unit * wp * da[t]
            g = g * a[t]
        out["dw_post"] += g * unit
        g = g * wp
        if w_post is not None:
            for k in range(groups):
                s = slice(k * D // groups, (k + 1) * D // groups)
                g[s] = (g[s] - unit[s] * np.mean(g[s] * unit[s])) / root[s]
        if first:
            out["dgate"][t] = g * o[t] * da[t]
            g = g * a[t]
        out["do"][t] = g
    for k, v in (("dr", r), ("dw_post", w_post), ("dscale", scale), ("dw_pre", w_pre)):
        if v is None:
            out[k] = None
    return out
