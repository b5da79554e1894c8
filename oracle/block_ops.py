"""CPU oracle of the feed-forward block around the products: activations and
the dense epilogue, the norms between blocks, a mixture-of-experts layer, with
their gradients -- TEST INFRASTRUCTURE ONLY (same rules as the rest of
``oracle``).  Plain numpy in 64 bits, written from the operators' definitions.
"""
from __future__ import annotations

import numpy as np
from scipy import special

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_C = np.sqrt(2 / np.pi)


def act(name, z):
    z = np.asarray(z, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        if name == "none":
            return z.copy()
        if name == "relu":
            return np.where(z < 0, 0.0, z)
        if name == "silu":
            p = special.expit(z)
        elif name == "gelu":
            p = special.ndtr(z)
        else:
            p = special.expit(2 * _C * (z + 0.044715 * z ** 3))
        return np.where(z == -np.inf, 0.0, z * p)  # the limit


def act_grad(name, z):
    z = np.asarray(z, np.float64)
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return np.where(np.isnan(z), z, (z > 0).astype(np.float64))
    b = np.clip(z, -1e4, 1e4)  # beyond, every derivative is 0 or 1
    with np.errstate(over="ignore", under="ignore"):
        if name == "gelu":
            return special.ndtr(b) + b * np.exp(-b * b / 2) / np.sqrt(2 * np.pi)
        v, dv = (b, 1.0) if name == "silu" else (2 * _C * (b + 0.044715 * b ** 3), 2 * _C * (1 + 3 * 0.044715 * b * b))
        p, q = special.expit(v), special.expit(-v)
        return p + b * dv * p * q


def epilogue(sums, bias, name, residual):
    """(z, out) of FP64 sums [m][n]."""
    z = sums if bias is None else sums + np.asarray(bias, np.float64)
    out = act(name, z)
    return z, out if residual is None else out + np.asarray(residual, np.float64)


def norm(v, layer, eps):
    """(norm(v), 1 / sqrt(..) [rows][1])."""
    v = np.asarray(v, np.float64)
    if layer:
        v = v - v.mean(-1, keepdims=True)
    r = 1 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    return v * r, r


def _or(p, other):
    return other if p is None else np.asarray(p, np.float64)


def norm_residual(x, residual, post_norm, post_weight, gate, scale, pre_weight, layer, eps):
    """(h, y) in FP64."""
    u = norm(x, layer, eps)[0] * _or(post_weight, 1.0) if post_norm else np.asarray(x, np.float64)
    h = u * _or(gate, 1.0)
    if residual is not None:
        h = scale * np.asarray(residual, np.float64) + h
    return h, norm(h, layer, eps)[0] * _or(pre_weight, 1.0)


def _through(b, v, layer, eps):
    """Gradient of v through norm(v) for the gradient b of the norm."""
    n, r = norm(v, layer, eps)
    d = b - n * (b * n).mean(-1, keepdims=True)
    return r * (d - b.mean(-1, keepdims=True) if layer else d)


def norm_residual_grads(grad_h, grad_y, x, h, post_norm, post_weight, gate, scale, pre_weight, layer, eps):
    """dict of the gradients (of a gate per row where the gate is [rows][n])."""
    f64 = lambda t: np.asarray(t, np.float64)
    gh = 0.0 if grad_h is None else f64(grad_h)
    out = {}
    if grad_y is not None:
        out["pre_weight"] = (f64(grad_y) * norm(h, layer, eps)[0]).sum(0)
        gh = gh + _through(f64(grad_y) * _or(pre_weight, 1.0), h, layer, eps)
    n = None if x is None else norm(x, layer, eps)[0] if post_norm else f64(x)
    w = _or(post_weight, 1.0) if post_norm else 1.0
    if gate is not None:
        g = gh * (n * w)
        out["gate"] = g if np.ndim(gate) == 2 and np.shape(gate)[0] == g.shape[0] > 1 else g.sum(0).reshape(np.shape(gate))
    du = gh * _or(gate, 1.0)
    if post_norm:
        out["post_weight"] = (du * n).sum(0)
        out["x"] = _through(du * w, x, layer, eps)
    else:
        out["x"] = du
    out["residual"] = scale * gh
    return out


def block_matrix(values, scales):
    """values [n][k] (decoded codes) times a scale per 128 x 128 block."""
    n, k = values.shape
    return np.asarray(values, np.float64) * np.repeat(np.repeat(np.asarray(scales, np.float64), 128, 0)[:n], 128, 1)[:, :k]


def moe_layer(x, expert_idx, weights, up, down, name):
    """out [T][hidden] of FP64 matrices up [E][2 inter][hidden], down [E][hidden][inter]."""
    x = np.asarray(x, np.float64)
    out = np.zeros((x.shape[0], down.shape[1]))
    inter = down.shape[2]
    for t in range(x.shape[0]):
        for j, e in enumerate(expert_idx[t]):
            if 0 <= e < up.shape[0]:
                both = up[e] @ x[t]
                mid = act(name, both[:inter]) * both[inter:]
                out[t] += (1.0 if weights is None else float(weights[t, j])) * (down[e] @ mid)
    return out
