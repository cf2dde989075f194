"""Float64 numpy oracle of the operators around the block: norms with gate and
scaled residual, their gradients, the gradient norm with clipping.

TEST INFRASTRUCTURE, written from the formulas and sharing no code with the
CUDA path.  Gradients are the chain rule, checked against differences of the
forward functions by the tests.
"""
from __future__ import annotations

import numpy as np


def norm(x, kind, eps=0.0, weight=None, bias=None):
    """N(x) over the last axis: kind "rms", "layer" or "none"."""
    x = np.asarray(x, dtype=np.float64)
    if kind == "none":
        return x
    m = x.mean(axis=1, keepdims=True) if kind == "layer" else 0.0
    out = (x - m) / np.sqrt(((x - m) ** 2).mean(axis=1, keepdims=True) + eps)
    if weight is not None:
        out = out * weight
    return out if bias is None else out + bias


def combine(y_slots, inv, T, k, S):
    """The block's slot rows in token order, summed."""
    y_slots = np.asarray(y_slots, dtype=np.float64)
    y = np.zeros((T, y_slots.shape[1]))
    inv = np.asarray(inv).reshape(T, k).astype(np.int64)
    for t in range(T):
        for j in range(k):
            if 0 <= inv[t, j] < T * k:
                y[t] += y_slots[inv[t, j]]
        for s in range(S):
            y[t] += y_slots[T * k + s * T + t]
    return y


def residual_norm(y, residual, post, gate, scale, nxt):
    """(h, xn): h = residual + scale gate N_post(y), xn = N_next(h); post and
    nxt are norm()'s keyword arguments, nxt None for no next norm."""
    z = norm(y, **post)
    h = scale * (z if gate is None else z * gate)
    if residual is not None:
        h = h + np.asarray(residual, dtype=np.float64)
    return h, None if nxt is None else norm(h, **nxt)


def norm_backward(x, dout, kind, eps=0.0, weight=None, bias=None, gate=None, scale=1.0,
                  dadd=None):
    """Gradients of scale * gate * N(x): dict of x, weight, bias, gate."""
    x, dout = np.asarray(x, dtype=np.float64), np.asarray(dout, dtype=np.float64)
    H = x.shape[1]
    w = np.ones(H) if weight is None else np.asarray(weight, dtype=np.float64)
    b = np.zeros(H) if bias is None else np.asarray(bias, dtype=np.float64)
    g = 1.0 if gate is None else np.asarray(gate, dtype=np.float64)
    D = scale * g * dout
    if kind == "none":
        xhat, dx = x, D
    else:
        xc = x - x.mean(axis=1, keepdims=True) if kind == "layer" else x
        sigma = np.sqrt((xc ** 2).mean(axis=1, keepdims=True) + eps)
        xhat = xc / sigma
        wD = w * D
        dx = wD - xhat * (wD * xhat).mean(axis=1, keepdims=True)
        if kind == "layer":
            dx = dx - wD.mean(axis=1, keepdims=True)
        dx = dx / sigma
    out = {"weight": (D * xhat).sum(axis=0), "bias": D.sum(axis=0), "gate": None,
           "x": dx if dadd is None else dx + np.asarray(dadd, dtype=np.float64)}
    if gate is not None:
        dz = scale * dout * (xhat * w + b)
        out["gate"] = dz.sum(axis=1, keepdims=True) if g.shape[-1] == 1 and H != 1 or \
            g.ndim == 2 and g.shape[0] != 1 else dz.sum(axis=0)
    return out


def clip(grads, max_norm):
    """(norm, clipped gradients)."""
    grads = [np.asarray(g, dtype=np.float64) for g in grads]
    n = np.sqrt(sum((g ** 2).sum() for g in grads))
    c = min(1.0, max_norm / (n + 1e-6))
    return n, [g * c for g in grads]
