"""CPU oracle of expert routing, of the weighted combine with their gradients,
and of the 4-bit products -- TEST INFRASTRUCTURE ONLY (same rules as the rest
of ``oracle``).  Plain numpy in 64 bits, one row at a time, written from the
operators' definitions.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], np.float64)


def route_scores(logits, sigmoid: bool) -> np.ndarray:
    """FP64 scores of every expert (0 where the logit is -inf or NaN)."""
    l = np.asarray(logits, np.float64)
    out = np.zeros_like(l)
    for t in range(l.shape[0]):
        on = l[t] > -np.inf
        x = l[t][on]
        if not x.size:
            continue
        if sigmoid:
            out[t][on] = np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))
        else:
            top = x.max()
            p = np.exp(np.where(x == top, 0.0, x - np.where(np.isinf(top), 0.0, top)) if np.isfinite(top)
                       else np.where(x == top, 0.0, -np.inf))
            out[t][on] = p / p.sum()
    return out


def _best(values, count):
    """Indices of the `count` largest values above -inf, best first, ties to
    the lowest index; the smallest gap between a chosen value and a lower one
    it is told from."""
    left = np.array(values, np.float64)
    picks, gap = [], np.inf
    for _ in range(count):
        i = int(np.argmax(left))  # the first of equal values
        if left[i] == -np.inf:
            break
        top = left[i]
        left[i] = -np.inf
        picks.append(i)
        lower = left[left < top]
        if lower.size and lower.max() > -np.inf:
            gap = min(gap, top - lower.max())
    return picks, gap


def route(logits, topk, sigmoid=False, bias=None, groups=1, topk_groups=1, top2=False, renormalize=False, scale=1.0):
    """(expert_idx [T][topk], weights [T][topk] FP64, gap [T]: the smallest
    difference between two selection scores that decided something)."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    s = route_scores(l, sigmoid)
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    idx = np.full((T, topk), -1, np.int32)
    w = np.zeros((T, topk))
    gaps = np.full(T, np.inf)
    for t in range(T):
        with np.errstate(invalid="ignore"):
            sel = np.where((l[t] > -np.inf) & (b > -np.inf), s[t] + b, -np.inf)
        if groups > 1:
            parts = np.sort(sel.reshape(groups, -1), axis=1)[:, ::-1]
            gscore = parts[:, 0].copy()
            if top2 and parts.shape[1] > 1:
                two = parts[:, 1] > -np.inf
                gscore[two] += parts[two, 1]
            keep, _ = _best(gscore, topk_groups)  # the order of the kept groups decides nothing
            dropped = [gscore[g] for g in range(groups) if g not in keep and gscore[g] > -np.inf]
            if keep and dropped and gscore[keep].min() > max(dropped):
                gaps[t] = gscore[keep].min() - max(dropped)
            for g in range(groups):
                if g not in keep:
                    sel[g * (E // groups):(g + 1) * (E // groups)] = -np.inf
        picks, gap = _best(sel, topk)
        gaps[t] = min(gaps[t], gap)
        idx[t, :len(picks)] = picks
        w[t, :len(picks)] = _weights(l[t], s[t], picks, sigmoid, renormalize) * scale
    return idx, w, gaps


def _weights(l, s, picks, sigmoid, renormalize):
    """Weights of the picks before the scale; the renormalised ones through
    logarithms, so that scores too small for 64 bits keep their ratios."""
    if not picks:
        return np.zeros(0)
    if not renormalize:
        return s[picks]
    x = l[picks]
    log = np.where(x >= 0, -np.log1p(np.exp(-np.abs(x))), x - np.log1p(np.exp(-np.abs(x)))) if sigmoid else x
    top = log.max()
    p = np.where(log == top, 1.0, np.exp(np.where(log == top, 0.0, log - top)))
    return p / p.sum()


def route_backward(logits, expert_idx, grad_weights, sigmoid=False, renormalize=False, scale=1.0):
    """(grad_logits [T][E], the same sum with every term's absolute value)."""
    l = np.asarray(logits, np.float64)
    g = np.asarray(grad_weights, np.float64)
    s = route_scores(l, sigmoid)
    out, mag = np.zeros_like(l), np.zeros_like(l)
    for t in range(l.shape[0]):
        on = [j for j in range(expert_idx.shape[1]) if 0 <= expert_idx[t, j] < l.shape[1]]
        picks = [int(expert_idx[t, j]) for j in on]
        if not picks:
            continue
        w = _weights(l[t], s[t], picks, sigmoid, renormalize)
        # dw_j / dl_e = w_j (d log s_j / dl_e - [renormalised] the w-weighted mean over the picks)
        for j, e in zip(on, picks):
            for e2, w2 in zip(picks, w):
                own = 1.0 if e2 == e else 0.0
                coef = w[picks.index(e)] * (own - w2) if renormalize else w[picks.index(e)] * own
                cmag = w[picks.index(e)] * (own + w2) if renormalize else abs(coef)
                slope = (1.0 - s[t, e2]) if sigmoid else 1.0
                out[t, e2] += scale * g[t, j] * coef * slope
                mag[t, e2] += abs(scale * g[t, j]) * cmag * slope
        if not sigmoid and not renormalize:
            total = float(np.sum(g[t, on] * w))
            out[t] -= scale * s[t] * total
            mag[t] += abs(scale) * s[t] * float(np.sum(np.abs(g[t, on]) * w))
    return out, mag


def combine(y, dst_row, weights):
    """(FP64 sums [T][n], the sums of absolute terms)."""
    y = np.asarray(y, np.float64)
    T, k = weights.shape
    out, mag = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            d = int(dst_row[t, j])
            if 0 <= d < y.shape[0]:
                out[t] += float(weights[t, j]) * y[d]
                mag[t] += abs(float(weights[t, j])) * np.abs(y[d])
    return out, mag


def combine_backward(grad_out, y, dst_row, weights, grad_y):
    """(grad_y with the named rows replaced, grad_weights, its absolute sums)."""
    go, y = np.asarray(grad_out, np.float64), np.asarray(y, np.float64)
    gy = np.array(grad_y, np.float64)
    gw, mag = np.zeros(weights.shape), np.zeros(weights.shape)
    for t in range(weights.shape[0]):
        for j in range(weights.shape[1]):
            d = int(dst_row[t, j])
            if 0 <= d < y.shape[0]:
                gy[d] = float(weights[t, j]) * go[t]
                gw[t, j] = np.dot(go[t], y[d])
                mag[t, j] = np.dot(np.abs(go[t]), np.abs(y[d]))
    return gy, gw, mag


def w4_codes(packed) -> np.ndarray:
    """[..][k / 2] bytes -> [..][k] codes, the even column in the low 4 bits."""
    packed = np.asarray(packed, np.uint8)
    out = np.empty(packed.shape[:-1] + (packed.shape[-1] * 2,), np.uint8)
    out[..., 0::2], out[..., 1::2] = packed % 16, packed // 16
    return out


def w4_parts(packed, scales, zeros, e2m1: bool):
    """(code values, zero points, scales), each [n][k] FP64."""
    codes = w4_codes(packed)
    g = codes.shape[-1] // scales.shape[-1] if scales.shape[-1] else 1
    wide = lambda a: np.repeat(np.asarray(a, np.float64), g, axis=-1)
    s = wide(scales)
    if e2m1:
        return E2M1[codes], np.zeros_like(s), s
    z = np.full_like(s, 8.0) if zeros is None else wide(zeros)
    return codes.astype(np.float64), z, s


def w4_matvec(x, packed, scales, zeros=None, e2m1=False):
    """(FP64 products [m][n], the same sums over absolute values of codes,
    zero points and inputs)."""
    v, z, s = w4_parts(packed, scales, zeros, e2m1)
    x = np.asarray(x, np.float64)
    return x @ ((v - z) * s).T, np.abs(x) @ ((np.abs(v) + np.abs(z)) * np.abs(s)).T


def w4_matvec_experts(x, expert_idx, packed, scales, zeros=None, e2m1=False):
    e = np.asarray(expert_idx).reshape(-1)
    per = e.size // x.shape[0] if x.shape[0] else 1
    out = np.zeros((e.size, packed.shape[1]))
    mag = np.zeros_like(out)
    for g in sorted(set(e.tolist())):
        if 0 <= g < packed.shape[0]:
            p = np.nonzero(e == g)[0]
            out[p], mag[p] = w4_matvec(x[p // per], packed[g], scales[g], None if zeros is None else zeros[g], e2m1)
    return out, mag
