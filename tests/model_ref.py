"""Plain 64-bit implementations (numpy) of the embedding, the layer norm and the gated
delta rule, written from their formulas: the reference of the GPU tests.  Their
gradients are checked against differences of their forward passes in
tests/test_model_ref.py."""
import numpy as np


# ----------------------------------------------------------------- layer norm
def layernorm_fwd(x, r, w, b, eps):
    """(y, s, mean, rstd)"""
    s = x if r is None else x + r
    mean = s.mean(axis=-1)
    away = s - mean[..., None]
    rstd = 1.0 / np.sqrt((away * away).mean(axis=-1) + eps)
    y = away * rstd[..., None] * w
    return (y if b is None else y + b), s, mean, rstd


def layernorm_bwd(dy, s, w, mean, rstd, dres):
    """(ds, dw, db) at the mean and rstd given."""
    v = (s - mean[..., None]) * rstd[..., None]
    e = dy * w
    ds = rstd[..., None] * (e - e.mean(axis=-1, keepdims=True) - v * (e * v).mean(axis=-1, keepdims=True))
    if dres is not None:
        ds = ds + dres
    flat = lambda t: t.reshape(-1, s.shape[-1]).sum(axis=0)   # noqa: E731
    return ds, flat(dy * v), flat(dy)


# ------------------------------------------------------------------ embedding
def embedding_fwd(tokens, table, scale):
    real = (tokens >= 0) & (tokens < len(table))
    return np.where(real[..., None], table[np.where(real, tokens, 0)] * scale, 0.0)


def embedding_bwd(dy, tokens, vocab, scale):
    out = np.zeros((vocab, dy.shape[-1]))
    for t, row in zip(tokens.reshape(-1), dy.reshape(-1, dy.shape[-1])):
        if 0 <= t < vocab:
            out[t] += row * scale
    return out


# ----------------------------------------------------------------- delta rule
def delta_fwd(q, k, v, g, beta, init, cu, scale):
    """q, k [T, G, N], v [T, H, P], g, beta [T, H], init [nseq, H, P, N], offsets cu.
    Returns (o [T, H, P], final, before): before[t] is the state that token t starts from."""
    heads, wide = v.shape[1], v.shape[1] // q.shape[1]
    o = np.zeros(v.shape)
    before = np.zeros((v.shape[0], heads) + init.shape[2:])
    final = np.array(init, dtype=np.float64)
    for s in range(len(cu) - 1):
        state = final[s].copy()
        for t in range(cu[s], cu[s + 1]):
            before[t] = state
            kt, qt = np.repeat(k[t], wide, axis=0), np.repeat(q[t], wide, axis=0)
            state = np.exp(g[t])[:, None, None] * state
            u = beta[t][:, None] * (v[t] - np.einsum("hpn,hn->hp", state, kt))
            state = state + u[:, :, None] * kt[:, None, :]
            o[t] = scale * np.einsum("hpn,hn->hp", state, qt)
        final[s] = state
    return o, final, before


def delta_bwd(do, q, k, v, g, beta, init, dfinal, cu, scale):
    """(dq, dk, dv, dg, dbeta, dinit)"""
    heads, groups = v.shape[1], q.shape[1]
    wide = heads // groups
    _, _, before = delta_fwd(q, k, v, g, beta, init, cu, scale)
    dq, dk, dv = np.zeros(q.shape), np.zeros(q.shape), np.zeros(v.shape)
    dg, dbeta = np.zeros(g.shape), np.zeros(g.shape)
    dinit = np.array(dfinal, dtype=np.float64)
    for s in range(len(cu) - 1):
        d = dinit[s].copy()
        for t in range(cu[s + 1] - 1, cu[s] - 1, -1):
            kt, qt = np.repeat(k[t], wide, axis=0), np.repeat(q[t], wide, axis=0)
            faded = np.exp(g[t])[:, None, None] * before[t]
            miss = v[t] - np.einsum("hpn,hn->hp", faded, kt)
            u = beta[t][:, None] * miss
            state = faded + u[:, :, None] * kt[:, None, :]
            d = d + scale * do[t][:, :, None] * qt[:, None, :]
            w = np.einsum("hpn,hn->hp", d, kt)
            dvt = beta[t][:, None] * w
            back = d - dvt[:, :, None] * kt[:, None, :]
            dqt = scale * np.einsum("hpn,hp->hn", state, do[t])
            dkt = np.einsum("hpn,hp->hn", d, u) - np.einsum("hpn,hp->hn", faded, dvt)
            dq[t] = dqt.reshape(groups, wide, -1).sum(axis=1)
            dk[t] = dkt.reshape(groups, wide, -1).sum(axis=1)
            dv[t] = dvt
            dbeta[t] = (w * miss).sum(axis=-1)
            dg[t] = (back * faded).sum(axis=(-2, -1))
            d = np.exp(g[t])[:, None, None] * back
        dinit[s] = d
    return dq, dk, dv, dg, dbeta, dinit


def delta_kept(before, cu, every=64):
    """(place, state) of the states that the forward pass keeps."""
    for s in range(len(cu) - 1):
        for c in range(-(-(cu[s + 1] - cu[s]) // every)):
            yield cu[s] // every + s + c, before[cu[s] + c * every]
