"""CPU oracle of the expert and head operators: routing, dispatch, combination, and the norm and
rotation of heads, with their gradients.

TEST INFRASTRUCTURE ONLY, like fp8_gemm_oracle.py; it shares no code with the HIP path. FP64
numpy from the formulas, one token at a time where that is plainest. Beside a result comes, where
an error bound needs it, the sum of the magnitudes it is made of.
"""
from __future__ import annotations

import numpy as np

from .layer_oracle import rotate

TINY = 1e-20


def scores(x, scoring):
    """[T, E]; a row without any expert has scores 0."""
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if scoring == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        top = x.max(axis=1, keepdims=True)
        top = np.where(np.isneginf(top), 0.0, top)
        e = np.exp(x - top)
        total = e.sum(axis=1, keepdims=True)
        return np.where(total == 0, 0.0, e / np.where(total == 0, 1.0, total))


def route(x, top_k, bias=None, scoring="softmax", groups=1, top_groups=1, group_best=1, renormalize=True, scale=1.0):
    """(ids [T, top_k], weights, scores). Finite logits or -inf."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    s = scores(x, scoring)
    ids, weights = np.full((T, top_k), -1, np.int64), np.zeros((T, top_k))
    size = E // groups
    for t in range(T):
        key = s[t] + (0.0 if bias is None else np.asarray(bias, np.float64))
        gone = np.isneginf(x[t]) | np.isneginf(key)
        rank = x[t] if bias is None else key  # the scores rise with the logits
        left = [e for e in range(E) if not gone[e]]
        if top_groups < groups:
            total = []
            for g in range(groups):
                live = sorted((key[e] for e in left if e // size == g), reverse=True)
                total.append(sum(live[:group_best]) if live else -np.inf)
            best = sorted(range(groups), key=lambda g: (-total[g], g))[:top_groups]
            left = [e for e in left if e // size in best]
        first = sorted(left, key=lambda e: (-rank[e], e))[:top_k]
        ids[t, :len(first)] = first
        w = s[t, first]
        weights[t, :len(first)] = scale * (w / (w.sum() + TINY) if renormalize else w)
    return ids, weights, s


def route_backward(dw, x, ids, scoring="softmax", renormalize=True, scale=1.0, dscores=None):
    """(dx [T, E], magnitudes). ids as int arrays; those outside the experts have no part."""
    x, dw = np.asarray(x, np.float64), np.asarray(dw, np.float64)
    T, E = x.shape
    s = scores(x, scoring)
    ds = np.zeros((T, E)) if dscores is None else np.asarray(dscores, np.float64).copy()
    mag = np.abs(ds)
    for t in range(T):
        at = [i for i in range(ids.shape[1]) if 0 <= ids[t, i] < E]
        chosen = s[t, ids[t, at]]
        g = scale * dw[t, at]
        m = np.abs(g)
        if renormalize:
            total = chosen.sum() + TINY
            g, m = (g - (g * chosen).sum() / total) / total, (m + (m * chosen).sum() / total) / total
        np.add.at(ds[t], ids[t, at], g)
        np.add.at(mag[t], ids[t, at], m)
    if scoring == "sigmoid":
        return ds * s * (1 - s), mag * s * (1 - s)
    return s * (ds - (ds * s).sum(axis=1, keepdims=True)), s * (mag + (mag * s).sum(axis=1, keepdims=True))


def layout(ids, E, max_m=0, rows=None):
    """(positions, sources, m_indices, counts) of choices ids [T, top_k]."""
    T, k = ids.shape
    of = [[] for _ in range(E)]
    for c, e in enumerate(ids.reshape(-1)):
        if 0 <= e < E:
            of[e].append(c)
    if max_m:
        rows = E * max_m
    elif rows is None:
        n = T * k
        rows = (n + min(n, E) * 127) // 128 * 128
    positions, sources, m_indices = np.full(T * k, -1, np.int64), np.full(rows, -1, np.int64), np.full(rows, -1, np.int64)
    counts, at = np.zeros(E, np.int64), 0
    for e in range(E):
        begin = e * max_m if max_m else at
        for i, c in enumerate(of[e]):
            if (i < max_m) if max_m else (begin + i < rows):
                positions[c], sources[begin + i], m_indices[begin + i] = begin + i, c, e
                counts[e] += 1
        at += -(-len(of[e]) // 128) * 128
    return positions.reshape(T, k), sources, m_indices, counts


def combine(y, positions, weights=None, c=None):
    """(out [T, N], magnitudes) of rows y [rows, N]."""
    y = np.asarray(y, np.float64)
    T, k = positions.shape
    w = np.ones((T, k)) if weights is None else np.asarray(weights, np.float64)
    out = np.zeros((T, y.shape[1])) if c is None else np.asarray(c, np.float64).copy()
    mag = np.abs(out)
    for t in range(T):
        for j in range(k):
            if 0 <= positions[t, j] < len(y):
                out[t] += w[t, j] * y[positions[t, j]]
                mag[t] += np.abs(w[t, j] * y[positions[t, j]])
    return out, mag


def combine_backward(do, y, positions, weights):
    """(rows' gradients as {row: [N]}, dweights, magnitudes)."""
    do, y, w = (np.asarray(a, np.float64) for a in (do, y, weights))
    T, k = positions.shape
    dy, dw, mag = {}, np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = int(positions[t, j])
            if 0 <= p < len(y):
                dy[p] = w[t, j] * do[t]
                dw[t, j], mag[t, j] = do[t] @ y[p], np.abs(do[t]) @ np.abs(y[p])
    return dy, dw, mag


def _turns(x, cos_sin, positions):
    if cos_sin is None:
        return np.zeros((x.shape[0], 1, 0)), np.zeros((x.shape[0], 1, 0))
    at = np.clip(np.arange(x.shape[0]) if positions is None else positions, 0, len(cos_sin) - 1)
    half = cos_sin.shape[1] // 2
    rows = np.asarray(cos_sin, np.float64)[at][:, None, :]
    return rows[..., :half], rows[..., half:]


def qk_norm_rope(x, w, cos_sin=None, positions=None, eps=1e-6, interleaved=False):
    """(out, magnitudes) of heads x [T, H, D]."""
    x = np.asarray(x, np.float64)
    n = x / np.sqrt((x * x).mean(axis=2, keepdims=True) + eps) * np.asarray(w, np.float64)
    cos, sin = _turns(x, cos_sin, positions)
    return rotate(n, cos, sin, interleaved)


def qk_norm_rope_backward(dy, x, w, cos_sin=None, positions=None, eps=1e-6, interleaved=False):
    """(dx, dw, magnitudes of both)."""
    dy, x, w = (np.asarray(a, np.float64) for a in (dy, x, w))
    rstd = 1.0 / np.sqrt((x * x).mean(axis=2, keepdims=True) + eps)
    xh = x * rstd
    cos, sin = _turns(x, cos_sin, positions)
    dn, turned = rotate(dy, cos, -sin, interleaved)
    g, m = dn * w, turned * np.abs(w)
    dx = rstd * (g - xh * (g * xh).mean(axis=2, keepdims=True))
    mag = rstd * (m + np.abs(xh) * (m * np.abs(xh)).mean(axis=2, keepdims=True))
    return dx, (dn * xh).sum(axis=(0, 1)), mag, (turned * np.abs(xh)).sum(axis=(0, 1))
