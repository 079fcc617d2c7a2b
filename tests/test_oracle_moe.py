"""The oracle of the expert and head operators against hand-made cases and against differences."""
import numpy as np
import pytest

from oracle import moe_oracle as mo


def test_route_by_hand():
    x = np.log(np.array([[1.0, 4.0, 2.0, 1.0]]))  # scores 1/8, 1/2, 1/4, 1/8
    ids, w, s = mo.route(x, 3)
    assert ids.tolist() == [[1, 2, 0]] and np.allclose(s, [[0.125, 0.5, 0.25, 0.125]])
    assert np.allclose(w, [[4 / 7, 2 / 7, 1 / 7]])
    ids, w, _ = mo.route(x, 2, bias=np.array([0.0, 0.0, 0.0, 1.0]), renormalize=False, scale=2.0)
    assert ids.tolist() == [[3, 1]] and np.allclose(w, [[0.25, 1.0]])
    # two groups of two: {1/8, 1/2} and {1/4, 1/8}: the best one decides, or the sum of two
    assert mo.route(x, 2, groups=2, top_groups=1)[0].tolist() == [[1, 0]]
    near = np.log(np.array([[5.0, 0.01, 4.0, 4.0]]))
    assert mo.route(near, 1, groups=2, top_groups=1)[0].tolist() == [[0]]
    assert mo.route(near, 1, groups=2, top_groups=1, group_best=2)[0].tolist() == [[2]]


def test_route_ties_and_none_left():
    ids, w, s = mo.route(np.zeros((1, 5)), 2)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, 0.5)
    x = np.array([[-np.inf, 0.0, -np.inf], [-np.inf] * 3])
    ids, w, s = mo.route(x, 2)
    assert ids.tolist() == [[1, -1], [-1, -1]] and w.tolist() == [[1.0, 0.0], [0.0, 0.0]] and s[1].tolist() == [0, 0, 0]
    ids, _, _ = mo.route(x, 2, scoring="sigmoid", bias=np.array([9.0, -np.inf, 0.0]))
    assert (ids == -1).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_is_that_of_differences(scoring, renormalize):
    rng = np.random.default_rng(1)
    T, E, k, h = 3, 7, 3, 1e-5
    x, dw, ds = rng.normal(size=(T, E)), rng.normal(size=(T, k)), rng.normal(size=(T, E))
    ids = mo.route(x, k, scoring=scoring)[0]

    def loss(x):
        s = mo.scores(x, scoring)
        c = np.take_along_axis(s, ids, 1)
        w = 1.7 * (c / (c.sum(1, keepdims=True) + mo.TINY) if renormalize else c)
        return (w * dw).sum() + (s * ds).sum()

    dx, _ = mo.route_backward(dw, x, ids, scoring, renormalize, 1.7, ds)
    for t in range(T):
        for e in range(E):
            d = np.zeros_like(x)
            d[t, e] = h
            assert abs((loss(x + d) - loss(x - d)) / (2 * h) - dx[t, e]) < 1e-8  # h^2 and rounding over h


def test_layouts_by_hand():
    ids = np.array([[1, 0], [1, 2], [0, -1], [7, 1]])
    positions, sources, m_indices, counts = mo.layout(ids, 3)
    assert counts.tolist() == [2, 3, 1] and positions.tolist() == [[128, 0], [129, 256], [1, -1], [-1, 130]]
    assert len(sources) == (8 + 3 * 127) // 128 * 128 and sources[[0, 1, 2, 128, 129, 130, 131, 256]].tolist() == [1, 4, -1, 0, 2, 7, -1, 3]
    assert m_indices[[0, 1, 2, 128, 130, 131, 256, 257]].tolist() == [0, 0, -1, 1, 1, -1, 2, -1]
    positions, sources, _, counts = mo.layout(ids, 3, max_m=2)
    assert counts.tolist() == [2, 2, 1] and positions.tolist() == [[2, 0], [3, 4], [1, -1], [-1, -1]]
    assert sources.tolist() == [1, 4, 0, 2, 3, -1]
    assert mo.layout(ids, 3, rows=128)[3].tolist() == [2, 0, 0]


def test_combination_and_its_gradient():
    rng = np.random.default_rng(2)
    y, w, c, do = rng.normal(size=(5, 4)), rng.normal(size=(3, 2)), rng.normal(size=(3, 4)), rng.normal(size=(3, 4))
    at = np.array([[0, 3], [-1, 2], [9, -1]])
    out, mag = mo.combine(y, at, w, c)
    assert np.allclose(out, [c[0] + w[0, 0] * y[0] + w[0, 1] * y[3], c[1] + w[1, 1] * y[2], c[2]]) and (mag >= np.abs(out) - 1e-12).all()
    dy, dw, _ = mo.combine_backward(do, y, at, w)
    assert sorted(dy) == [0, 2, 3] and np.allclose(dw, [[do[0] @ y[0], do[0] @ y[3]], [0, do[1] @ y[2]], [0, 0]])
    assert np.allclose(dy[3], w[0, 1] * do[0])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotated", [0, 4, 8])
def test_head_gradients_are_those_of_differences(interleaved, rotated):
    rng = np.random.default_rng(3)
    T, H, D, h = 2, 2, 8, 1e-5
    x, w, dy = rng.normal(size=(T, H, D)), 1 + 0.2 * rng.normal(size=D), rng.normal(size=(T, H, D))
    angle = rng.normal(size=(5, rotated // 2))
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1) if rotated else None
    at = np.array([3, 99])

    def loss(x, w):
        return (mo.qk_norm_rope(x, w, table, at, 1e-6, interleaved)[0] * dy).sum()

    dx, dw, _, _ = mo.qk_norm_rope_backward(dy, x, w, table, at, 1e-6, interleaved)
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = h
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * h) - dx[i]) < 1e-7
    for i in range(D):
        d = np.zeros_like(w)
        d[i] = h
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * h) - dw[i]) < 1e-7
    if rotated:  # a rotation keeps the length of what it turns
        n = mo.qk_norm_rope(x, w)[0]
        y = mo.qk_norm_rope(x, w, table, at, 1e-6, interleaved)[0]
        assert np.allclose((y * y).sum(2), (n * n).sum(2)) and not np.allclose(y, n)
