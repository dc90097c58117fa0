"""What stands around a block's products, in fp64: the linear layer's epilogue
and gradient, the norms before and after a block, and a mixture-of-experts
layer.  NumPy only."""

import numpy as np

from . import ffn


def act(z, kind):
    """(act(z), act'(z), s): s the sigmoid's argument, 0 without one."""
    if kind == "none":
        return z, np.ones_like(z), np.zeros_like(z)
    if kind == "relu":
        return np.where(z <= 0, 0.0, z), np.where(z <= 0, 0.0, 1.0), np.zeros_like(z)
    return ffn.act(z, kind)


def linear(x, w, bias=None, kind="none", residual=None):
    """(y, z) of y = residual + act(z), z = x w + bias."""
    z = x @ w + (0.0 if bias is None else bias)
    y = act(z, kind)[0]
    return (y if residual is None else y + residual), z


def linear_grad(dy, x, w, z, kind="none"):
    """(dx, dw, db, dz)."""
    dz = dy * act(z, kind)[1]
    return dz @ w.T, x.T @ dz, dz.sum(axis=0), dz


def rms_norm(v, w, eps):
    """(v / rms * w, 1 / rms) of rows v."""
    r = 1.0 / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)
    return v * r * w, r


def rms_norm_grad(d, v, w, eps):
    """(dv, dw) for the gradient d of the normed rows."""
    _, r = rms_norm(v, w, eps)
    e = d * w
    dot = np.sum(e * v, axis=1, keepdims=True) / v.shape[1]
    return r * e - v * r ** 3 * dot, np.sum(d * v * r, axis=0)


def spread(gate, M):
    """gate [G, K] as one row per token: each for M / G consecutive tokens."""
    return np.repeat(gate, M // gate.shape[0], axis=0)


def block_norm(y, h, w, post=None, gate=None, scale=1.0, eps=1e-6):
    """(n, s, p): p = post-norm(y), s = h + scale gate p, n = norm(s)."""
    p = y if post is None else rms_norm(y, post, eps)[0]
    s = h + scale * (p if gate is None else spread(gate, y.shape[0]) * p)
    return rms_norm(s, w, eps)[0], s, p


def block_norm_grad(dn, y, h, w, post=None, gate=None, scale=1.0, eps=1e-6, ds=None):
    """(dh, dy, dw, dpost, dgate) for the gradients dn of n and ds of s."""
    _, s, p = block_norm(y, h, w, post, gate, scale, eps)
    dh, dw = rms_norm_grad(dn, s, w, eps)
    if ds is not None:
        dh = dh + ds
    dp, dgate, dpost = scale * dh, None, None
    if gate is not None:
        G = gate.shape[0]
        dgate = (dp * p).reshape(G, -1, y.shape[1]).sum(axis=1)
        dp = dp * spread(gate, y.shape[0])
    dy = dp
    if post is not None:
        dy, dpost = rms_norm_grad(dp, y, post, eps)
    return dh, dy, dw, dpost, dgate


def route(x, router, top, renormalize=True, scale=1.0):
    """(ids [M, top], weights, logits) of the ``top`` largest logits x router,
    the first of equals: softmax over the chosen, or over all experts."""
    logits = x @ router
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top]
    e = np.exp(logits - logits.max(axis=1, keepdims=True))
    p = np.take_along_axis(e, ids, axis=1)
    total = p.sum(axis=1, keepdims=True) if renormalize else e.sum(axis=1, keepdims=True)
    return ids, scale * p / total, logits


def experts(x, ids, weights, w_gate_up, w_down, kind="silu", h=None):
    """sum_j weights[m, j] (act(g) u) W_down[ids[m, j]], [g | u] = x
    W_gate_up[ids[m, j]].  ids outside the experts add nothing.  ``h``
    [M, top, F] takes the place of act(g) u."""
    M, F = x.shape[0], w_down.shape[1]
    y = np.zeros((M, w_down.shape[2]))
    for m in range(M):
        for j, e in enumerate(ids[m]):
            if not 0 <= e < w_gate_up.shape[0]:
                continue
            if h is None:
                gu = x[m] @ w_gate_up[e]
                a = ffn.act(gu[:F], kind)[0] * gu[F:]
            else:
                a = h[m, j]
            y[m] += weights[m, j] * (a @ w_down[e])
    return y
