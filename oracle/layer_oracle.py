"""CPU oracle of the operators around the GEMMs of a transformer layer: the residual RMS
norm with its quantisation and gradients, the rotation and append to a paged 8-bit cache,
and causal attention over that cache.

TEST INFRASTRUCTURE ONLY, like fp8_gemm_oracle.py; it shares no code with the HIP path.
Everything is FP64 numpy, straight from the formulas, one sequence and head at a time. Where
a result is rounded by definition (codes), the functions return the value before rounding,
and where it helps, the sum of magnitudes that an error bound is made of.
"""
from __future__ import annotations

import numpy as np

from .fp8_gemm_oracle import decode_e4m3

E4M3_MAX = 448.0


def rmsnorm(h, w, eps):
    """y [M, K] = h / sqrt(mean(h^2) + eps) * w and rstd [M]."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h * rstd[:, None] * w, rstd


def block_scales(y):
    """amax / 448 of each 128 columns of y [M, K] (1 where that is 0), as [K / 128, M]."""
    a = np.abs(y).reshape(y.shape[0], -1, 128).max(axis=2) / E4M3_MAX
    return np.where(a > 0, a, 1.0).T


def rmsnorm_backward(dy, h, rstd, w, dh=None):
    """(dX, dW, bound_dx, bound_dw): gradients of sum(dy * y), and the sums of magnitudes
    of their terms. rstd is taken as given."""
    dy, h, rstd, w = (np.asarray(a, np.float64) for a in (dy, h, rstd, w))
    K = h.shape[1]
    xhat = h * rstd[:, None]
    g = dy * w
    mean = (g * xhat).sum(axis=1) / K
    dx = rstd[:, None] * (g - xhat * mean[:, None])
    mag = rstd[:, None] * (np.abs(g) + np.abs(xhat) * (np.abs(g * xhat).sum(axis=1) / K)[:, None])
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
        mag = mag + np.abs(dh)
    return dx, (dy * xhat).sum(axis=0), mag, np.abs(dy * xhat).sum(axis=0)


def rotate(x, cos, sin, interleaved=False):
    """x [..., D] with the first 2 len(cos) columns turned; also the magnitudes |x1 cos| + |x2 sin|."""
    x, cos, sin = (np.asarray(a, np.float64) for a in (x, cos, sin))
    half = cos.shape[-1]
    y, mag = x.copy(), np.abs(x)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = cos[..., i], sin[..., i]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
        mag[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
    return y, mag


def fit_scale(amax):
    """The smallest power of two, 2^-126 at least, by which amax fits 448."""
    e = -126
    if amax > 0:
        e = int(np.ceil(np.log2(amax / E4M3_MAX)))
        while E4M3_MAX * 2.0 ** e < amax:
            e += 1
        while E4M3_MAX * 2.0 ** (e - 1) >= amax:
            e -= 1
    return 2.0 ** max(e, -126)


def append(codes, scales, x, table, seq_lens, cu_q, page_size):
    """The cache after rows x [T, H, D] are appended: (value, scale, written). value [N, H,
    P, D] is what each code stands for over its page's new scale, before rounding; written
    marks the slots that hold a new token (True). Earlier codes of a touched page are
    decoded and taken over the new scale; all others as they are."""
    value = decode_e4m3(codes)
    scale = np.asarray(scales, np.float64).copy()
    written = np.zeros(codes.shape[:3], bool)
    N, H, P, _ = codes.shape
    for b in range(len(seq_lens)):
        rows = range(cu_q[b], cu_q[b + 1])
        start = seq_lens[b] - len(rows)
        by_page = {}
        for i, r in enumerate(rows):
            if start + i >= 0:
                by_page.setdefault((start + i) // P, []).append(((start + i) % P, r))
        for j, new in by_page.items():
            page = table[b][j]
            if not 0 <= page < N:
                continue
            for h in range(H):
                finite = np.abs([x[r, h] for _, r in new])
                fit = fit_scale(np.max(np.where(np.isfinite(finite), finite, 0.0)))
                first = new[0][0]
                if first > 0:
                    fit = max(fit, scale[page, h])
                    value[page, h, :first] *= scale[page, h] / fit
                scale[page, h] = fit
                for slot, r in new:
                    value[page, h, slot] = x[r, h] / fit
                    written[page, h, slot] = True
    return value, scale, written


def attention(q, k_codes, k_scale, v_codes, v_scale, table, seq_lens, cu_q, softmax_scale, window=0):
    """(out, lse, spread, depth): out [T, Hq, D] and lse [T, Hq]; spread = sum_j p_j |v_j|
    and depth = max_j softmax_scale sum_d |q_d k_jd| over the keys a row sees, for error
    bounds."""
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    N, Hkv, P, _ = k_codes.shape
    g = Hq // Hkv
    out, spread = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, depth = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for b in range(len(seq_lens)):
        n, m = cu_q[b + 1] - cu_q[b], seq_lens[b]
        if n == 0 or m == 0:
            continue
        pages = np.array([table[b][j] for j in range(-(-m // P))])
        there = np.repeat((pages >= 0) & (pages < N), P)[:m]
        pages = np.where((pages >= 0) & (pages < N), pages, 0)
        key, pos = np.arange(m), m - n + np.arange(n)
        sees = (key[None] <= pos[:, None]) & there[None]
        if window:
            sees &= key[None] > pos[:, None] - window
        used = sees.any(axis=0)  # what no row sees may hold anything
        for h in range(Hkv):
            k = (decode_e4m3(k_codes[pages, h]) * np.asarray(k_scale, np.float64)[pages, h][:, None, None]).reshape(-1, D)[:m]
            v = (decode_e4m3(v_codes[pages, h]) * np.asarray(v_scale, np.float64)[pages, h][:, None, None]).reshape(-1, D)[:m]
            k, v = np.where(used[:, None], k, 0.0), np.where(used[:, None], v, 0.0)
            for i in range(h * g, h * g + g):
                rows = q[cu_q[b]:cu_q[b + 1], i]
                s = np.where(sees, rows @ k.T * softmax_scale, -np.inf)
                top = np.max(s, axis=1, keepdims=True)
                top = np.where(np.isfinite(top), top, 0.0)
                p = np.exp(s - top)
                total = p.sum(axis=1, keepdims=True)
                any_key = total[:, 0] > 0
                p = p / np.where(total > 0, total, 1.0)
                at = slice(cu_q[b], cu_q[b + 1])
                out[at, i] = p @ v
                spread[at, i] = p @ np.abs(v)
                with np.errstate(divide="ignore"):
                    lse[at, i] = np.where(any_key, top[:, 0] + np.log(total[:, 0]), -np.inf)
                depth[at, i] = np.max(np.where(sees, np.abs(rows) @ np.abs(k).T * abs(softmax_scale), 0.0), axis=1)
    return out, lse, spread, depth
