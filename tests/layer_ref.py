"""Plain 64-bit implementations (numpy) of the layer's steps around the scan,
written from their formulas: the reference of the GPU tests.  Their gradients
are checked against differences of their forward passes in
tests/test_layer_ref.py."""
import math

import numpy as np

E4M3_MAX = 448.0


def sigmoid(v):
    v = np.asarray(v, dtype=np.float64)
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def silu(v):
    return v * sigmoid(v)


def silu_slope(v):
    s = sigmoid(v)
    return s * (1.0 + v * (1.0 - s))


_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(p, name):
    p = np.asarray(p, dtype=np.float64)
    if name == "silu":
        return silu(p)
    if name == "gelu":
        return 0.5 * p * (1.0 + _erf(p / math.sqrt(2.0))) if p.size else p
    if name == "relu":
        return np.maximum(p, 0.0)
    return p


def act_slope(p, name):
    p = np.asarray(p, dtype=np.float64)
    if name == "silu":
        return silu_slope(p)
    if name == "gelu":
        if not p.size:
            return p
        return 0.5 * (1.0 + _erf(p / math.sqrt(2.0))) + p * np.exp(-0.5 * p * p) / math.sqrt(2 * math.pi)
    if name == "relu":
        return (p > 0).astype(np.float64)
    return np.ones_like(p)


# ----------------------------------------------------------------------- norm
def norm_fwd(x, r, w, eps):
    """(y, s, rstd)"""
    s = x if r is None else x + r
    rstd = 1.0 / np.sqrt((s * s).mean(axis=-1) + eps)
    return s * rstd[..., None] * w, s, rstd


def norm_bwd(dy, s, w, rstd, dres):
    """(ds, dw) at the rstd given."""
    e = dy * w
    v = s * rstd[..., None]
    ds = rstd[..., None] * (e - v * (e * v).mean(axis=-1, keepdims=True))
    if dres is not None:
        ds = ds + dres
    return ds, (dy * v).reshape(-1, s.shape[-1]).sum(axis=0)


# -------------------------------------------------------------------- product
def linear_fwd(x, w, bias=None, residual=None, activation="none", x_scale=None, w_scale=None):
    """(y, p)"""
    p = x @ w.T
    if x_scale is not None:
        p = p * x_scale[:, None] * w_scale[None, :]
    if bias is not None:
        p = p + bias
    y = act(p, activation)
    return (y if residual is None else y + residual), p


def linear_bwd(dy, x, w, preact=None, activation="none"):
    """(dx, dw, dbias)"""
    dp = dy if preact is None else dy * act_slope(preact, activation)
    return dp @ w, dp.T @ x, dp.sum(axis=0)


# ----------------------------------------------------------------- recurrence
def gated_fwd(x, g, z, init, cu):
    """x, g, z [T, D] (z may be None), init [nseq, D], offsets cu.  Returns
    (y, h, final, before): before[t] is the state that token t starts from."""
    h_all, before = np.empty_like(x), np.empty_like(x)
    final = np.array(init, dtype=np.float64)
    for s in range(len(cu) - 1):
        h = final[s].copy()
        for t in range(cu[s], cu[s + 1]):
            before[t] = h
            h = sigmoid(g[t]) * h + sigmoid(-g[t]) * x[t]
            h_all[t] = h
        final[s] = h
    return (h_all if z is None else h_all * silu(z)), h_all, final, before


def gated_bwd(dy, x, g, z, init, dfinal, cu):
    """(dx, dg, dz or None, dinit)"""
    _, h, _, before = gated_fwd(x, g, z, init, cu)
    dz = None if z is None else dy * h * silu_slope(z)
    dh = dy if z is None else dy * silu(z)
    dx, dg = np.empty_like(x), np.empty_like(x)
    dinit = np.array(dfinal, dtype=np.float64)
    for s in range(len(cu) - 1):
        lam = dinit[s].copy()
        for t in range(cu[s + 1] - 1, cu[s] - 1, -1):
            lam = lam + dh[t]
            f, d = sigmoid(g[t]), sigmoid(-g[t])
            dx[t] = d * lam
            dg[t] = lam * (before[t] - x[t]) * f * d
            lam = f * lam
        dinit[s] = lam
    return dx, dg, dz, dinit
