"""The layer operators' CPU oracle against independent evaluations: finite differences,
plain loops in extended precision, closed forms and invariants. No GPU needed."""
import math

import numpy as np
import pytest

import oracle
from oracle import layer_oracle as lo


@pytest.mark.parametrize("M,K", [(1, 128), (3, 256)])
def test_norm_gradients_against_central_differences(M, K):
    rng = np.random.default_rng(M + K)
    h, w, dy = rng.standard_normal((M, K)), 1 + 0.3 * rng.standard_normal(K), rng.standard_normal((M, K))
    eps = 1e-3

    def loss(h, w):
        return float((lo.rmsnorm(h, w, eps)[0] * dy).sum())

    _, rstd = lo.rmsnorm(h, w, eps)
    dx, dw, mag, magw = lo.rmsnorm_backward(dy, h, rstd, w)
    step = 1e-5  # truncation ~ step^2, cancellation ~ 1e-16 |loss| / step
    for i, j in [(0, 0), (M - 1, K - 1), (0, K // 2), (M // 2, 17)]:
        d = np.zeros_like(h)
        d[i, j] = step
        assert abs((loss(h + d, w) - loss(h - d, w)) / (2 * step) - dx[i, j]) < 1e-8
        e = np.zeros_like(w)
        e[j] = step
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * step) - dw[j]) < 1e-8
    assert np.all(mag >= np.abs(dx) - 1e-15) and np.all(magw >= np.abs(dw) - 1e-15)
    extra = rng.standard_normal((M, K))
    assert np.allclose(lo.rmsnorm_backward(dy, h, rstd, w, extra)[0], dx + extra, rtol=0, atol=1e-15)


def test_norm_closed_forms():
    y, rstd = lo.rmsnorm(np.full((2, 128), 3.0), np.ones(128), 0.0)
    assert np.allclose(y, 1.0, rtol=1e-15) and np.allclose(rstd, 1 / 3, rtol=1e-15)
    y, rstd = lo.rmsnorm(np.zeros((1, 128)), np.ones(128), 0.25)
    assert np.all(y == 0) and rstd[0] == 2.0
    assert np.all(lo.block_scales(y) == 1.0)
    assert lo.block_scales(np.eye(1, 256, 130) * 448)[1, 0] == 1.0


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_rotation_of_pairs(interleaved):
    rng = np.random.default_rng(5)
    x, ang = rng.standard_normal((4, 3, 64)), rng.uniform(-7, 7, (4, 1, 16))
    y, mag = lo.rotate(x, np.cos(ang), np.sin(ang), interleaved)
    z = x[..., 0:32:2] + 1j * x[..., 1:32:2] if interleaved else x[..., :16] + 1j * x[..., 16:32]
    u = z * np.exp(1j * ang)
    want = x.copy()
    if interleaved:
        want[..., 0:32:2], want[..., 1:32:2] = u.real, u.imag
    else:
        want[..., :16], want[..., 16:32] = u.real, u.imag
    assert np.allclose(y, want, rtol=0, atol=1e-14) and np.array_equal(y[..., 32:], x[..., 32:])
    assert np.all(mag >= np.abs(y) - 1e-15)


def test_fit_scale_is_the_smallest_power():
    assert lo.fit_scale(0.0) == 2.0 ** -126 and lo.fit_scale(448.0) == 1.0 and lo.fit_scale(np.nextafter(448.0, 500)) == 2.0
    for a in np.random.default_rng(1).lognormal(0, 20, 200):
        s = lo.fit_scale(a)
        assert math.frexp(s)[0] == 0.5 and 448 * s >= a and (448 * s / 2 < a or s == 2.0 ** -126)


def test_append_places_tokens_and_grows_scales():
    rng = np.random.default_rng(2)
    N, H, P, D = 5, 2, 4, 64
    codes = np.full((N, H, P, D), 0x38, np.uint8)  # 1.0
    scales = np.full((N, H), 0.5)
    x = rng.uniform(1, 2, (7, H, D))
    x[:, 1] *= 1000
    table = [[3, 1], [4, 9]]
    # sequence 0: 3 new tokens from slot 3 to 5; sequence 1: 4 from slot 2 on, of which slots 4.. have no page
    value, scale, written = lo.append(codes, scales, x, table, [6, 6], [0, 3, 7], P)
    assert written.sum() == H * (1 + 2 + 2)
    assert scale[3, 0] == 0.5 and np.all(value[3, 0, :3] == 1.0)      # the old scale fits
    assert scale[3, 1] > 0.5 and np.allclose(value[3, 1, :3] * scale[3, 1], 0.5)  # it does not: the same values at a larger one
    assert scale[1, 0] == lo.fit_scale(x[1:3, 0].max())                # a fresh page
    assert np.allclose(value[1, :, 0] * scale[1][:, None], x[1]) and np.allclose(value[3, :, 3] * scale[3][:, None], x[0])
    assert np.allclose(value[4, :, 2] * scale[4][:, None], x[3]) and np.all(scale[[0, 2]] == 0.5)


def _attention_by_loops(q, k, v, pages, n, m, P, scale, window, i, h, t):
    pos = m - n + t
    logits, rows = [], []
    for j in range(m):
        if j <= pos and (not window or j > pos - window) and 0 <= pages[j // P] < k.shape[0]:
            logits.append(math.fsum(float(a) * float(b) for a, b in zip(q[t, i], k[pages[j // P], h, j % P])) * scale)
            rows.append(v[pages[j // P], h, j % P])
    if not logits:
        return np.zeros(q.shape[2]), -math.inf
    top = max(logits)
    w = [math.exp(s - top) for s in logits]
    return sum(a * r for a, r in zip(w, rows)) / math.fsum(w), top + math.log(math.fsum(w))


@pytest.mark.parametrize("window", [0, 3])
def test_attention_against_loops(window):
    rng = np.random.default_rng(3)
    N, Hkv, P, D, Hq = 6, 2, 16, 64, 4
    kc, vc = (rng.integers(0, 0x7F, (N, Hkv, P, D)).astype(np.uint8) for _ in range(2))
    ks, vs = (2.0 ** rng.integers(-9, -6, (N, Hkv)).astype(float) for _ in range(2))
    q = rng.standard_normal((6, Hq, D)) * 0.1
    # the last sequence has more new tokens than it has keys: its first row sees none
    lens, cu, table = [19, 0, 17, 1], [0, 2, 2, 4, 6], [[2, 0], [-1, -1], [5, -1], [1, -1]]
    out, lse, spread, depth = lo.attention(q, kc, ks, vc, vs, table, lens, cu, 0.3, window)
    k = oracle.decode_e4m3(kc) * ks[:, :, None, None]
    v = oracle.decode_e4m3(vc) * vs[:, :, None, None]
    for b in range(4):
        for t in range(cu[b + 1] - cu[b]):
            for i in range(Hq):
                o, s = _attention_by_loops(q[cu[b]:cu[b + 1]], k, v, table[b], cu[b + 1] - cu[b], lens[b], P, 0.3, window, i, i // 2, t)
                assert np.allclose(out[cu[b] + t, i], o, rtol=1e-12, atol=1e-14)
                assert lse[cu[b] + t, i] == pytest.approx(s, rel=1e-12)
    assert np.all(out[4] == 0) and np.all(np.isneginf(lse[4])) and np.all(spread >= np.abs(out) - 1e-14)
