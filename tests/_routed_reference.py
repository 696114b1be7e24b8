"""64-bit references of moe_topk_route, its backward pass and moe_combine_topk,
from their definitions in include/moe.h, in numpy."""

import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)


def scores(logits, kind):
    """(cleaned logits, masked, scores) in 64 bits."""
    l = np.array(logits, dtype=np.float64)
    l[np.isnan(l)] = -np.inf
    l = np.minimum(l, FLT_MAX)
    masked = np.isneginf(l)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            s = 1 / (1 + np.exp(-l))
        else:
            m = l.max(axis=1, keepdims=True)
            s = np.exp(l - np.where(np.isneginf(m), 0, m))
            s[masked] = 0
            z = s.sum(axis=1, keepdims=True)
            s = s / np.where(z > 0, z, 1)
    s[masked] = 0
    return l, masked, s


def log_scores(l, kind):
    """Logarithm of the scores up to a term that a row shares."""
    with np.errstate(over="ignore"):
        return l if kind == "softmax" else np.where(l > 0, -np.log1p(np.exp(-np.abs(l))), l - np.log1p(np.exp(-np.abs(l))))


def route(logits, k, kind="softmax", bias=None, groups=1, keep=1, rule="max", renorm=False, scale=1.0, n=None):
    T, E = logits.shape
    n = T if n is None else min(max(n, 0), T)
    l, masked, s = scores(logits, kind)
    idx = np.full((T, k), -1, dtype=np.int64)
    w = np.zeros((T, k))
    s[n:] = 0
    for t in range(n):
        c = l[t].copy()
        v = s[t] if bias is None else s[t] + bias.astype(np.float64)
        if bias is not None:
            c = np.where(masked[t] | np.isnan(v), -np.inf, v)
        if groups > 1:
            gs = E // groups
            gv = []
            for g in range(groups):
                run = slice(g * gs, (g + 1) * gs)
                ok = ~np.isneginf(c[run])
                top = np.sort((c if rule == "max" else v)[run][ok])[::-1]
                gv.append(-np.inf if top.size == 0 else top[:1 if rule == "max" else 2].sum())
            for g in sorted(range(groups), key=lambda g: (-gv[g], g))[keep:]:
                c[g * gs:(g + 1) * gs] = -np.inf
        order = sorted(range(E), key=lambda e: (-c[e], e))[:k]
        idx[t, :k] = [e if not np.isneginf(c[e]) else -1 for e in order]
        has = idx[t] >= 0
        if has.any():
            if renorm:
                a = log_scores(l[t, idx[t][has]], kind)
                x = np.exp(a - a.max())
                w[t, has] = x / x.sum()
            else:
                w[t, has] = s[t, idx[t][has]]
    w *= scale
    out = {"idx": idx, "weights": w, "scores": s}
    out.update(dispatch(idx, w, E))
    return out


def dispatch(idx, w, E):
    T, k = idx.shape
    token, slot = np.nonzero(idx >= 0)
    order = np.lexsort((token, idx[token, slot]))
    token, slot = token[order], slot[order]
    counts = np.bincount(idx[idx >= 0], minlength=E)
    d = {"counts": counts, "offsets": np.concatenate([[0], np.cumsum(counts)]), "perm_token": np.full(T * k, -1),
         "perm_slot": np.full(T * k, -1), "slot_pos": np.full((T, k), -1), "gate_perm": np.zeros(T * k)}
    m = token.size
    d["perm_token"][:m], d["perm_slot"][:m], d["gate_perm"][:m] = token, slot, w[token, slot]
    d["slot_pos"][token, slot] = np.arange(m)
    return d


def weights_of(logits, idx, kind, renorm, scale):
    """Weights of a given choice and all scores, differentiable by differences."""
    l, _, s = scores(logits, kind)
    has = (idx >= 0) & (idx < logits.shape[1])
    at = np.where(has, idx, 0)
    if renorm:
        a = np.where(has, np.take_along_axis(log_scores(l, kind), at, 1), -np.inf)
        m = a.max(axis=1, keepdims=True)
        x = np.where(has, np.exp(a - np.where(np.isneginf(m), 0, m)), 0)
        z = x.sum(axis=1, keepdims=True)
        return scale * x / np.where(z > 0, z, 1), s
    return scale * np.where(has, np.take_along_axis(s, at, 1), 0), s


def route_backward(logits, idx, gw, kind, renorm, scale, gs=None, n=None):
    T, E = logits.shape
    n = T if n is None else min(max(n, 0), T)
    l, masked, s = scores(logits, kind)
    has = (idx >= 0) & (idx < E)
    w, _ = weights_of(logits, idx, kind, renorm, 1.0)
    grad = np.zeros((T, E))
    ds = np.zeros((T, E)) if gs is None else gs.astype(np.float64)
    with np.errstate(over="ignore"):
        rest = 1 / (1 + np.exp(l))  # 1 - sigmoid
    for t in range(n):
        g = np.where(has[t], gw[t].astype(np.float64), 0) * scale
        if renorm:
            p = w[t]
            d = p * (g - (g * p).sum())
            for j in np.nonzero(has[t])[0]:
                e = idx[t, j]
                grad[t, e] += d[j] * (rest[t, e] if kind == "sigmoid" else 1)
        else:
            for j in np.nonzero(has[t])[0]:
                ds[t, idx[t, j]] += g[j]
        if kind == "sigmoid":
            grad[t] += s[t] * rest[t] * ds[t]
        else:
            grad[t] += s[t] * (ds[t] - (s[t] * ds[t]).sum())
    grad[masked] = 0
    grad[n:] = 0
    return grad


def combine(y, pos, weights=None, residual=None):
    T, k = pos.shape
    out = np.zeros((T, y.shape[1])) if residual is None else residual.astype(np.float64)
    size = np.abs(out)
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < y.shape[0]:
                part = y[pos[t, j]].astype(np.float64) * (1 if weights is None else float(weights[t, j]))
                out[t] += part
                size[t] += np.abs(part)
    return out, size
