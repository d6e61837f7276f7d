"""Pins of the oracles of the operators around the layers to things other than themselves (CPU): hand-worked values, closed
forms, central differences, brute force."""
import numpy as np
import pytest

from oracle import around_layers as A


def test_embedding_by_hand():
    E = np.array([[1.0, 2.0], [3.0, -4.0], [0.5, 0.25]])
    out = A.embedding_fwd(E, [2, -1, 0, 3, 2], 2.0, width=3)
    np.testing.assert_array_equal(out, [[1, .5, 0], [0, 0, 0], [2, 4, 0], [0, 0, 0], [1, .5, 0]])
    g, a, n = A.embedding_bwd(np.array([[1., 2, 9], [7, 7, 9], [3, 4, 9], [5, 5, 9], [-2, 1, 9]]), [2, -1, 0, 3, 2], 3, 2, 2.0)
    np.testing.assert_array_equal(g, [[6, 8], [0, 0], [-2, 6]])
    np.testing.assert_array_equal(a[2], [6, 6])
    np.testing.assert_array_equal(n, [1, 0, 2])


def test_embedding_gradient_by_differences():
    rng = np.random.default_rng(0)
    E, ids, up = rng.normal(size=(5, 3)), [1, 4, 1, 0, -1, 1], rng.normal(size=(6, 3))
    g = A.embedding_bwd(up, ids, 5, 3, 1.5)[0]
    f = lambda t: float((A.embedding_fwd(t, ids, 1.5) * up).sum())
    for i in range(5):
        for j in range(3):
            d = np.zeros_like(E)
            d[i, j] = 1e-3
            assert abs((f(E + d) - f(E - d)) / 2e-3 - g[i, j]) < 1e-9


def test_norm_closed_forms():
    # two values a +- s: LayerNorm gives +-1 (eps 0); RMS of (3, 4) is 5 / sqrt 2
    m, r = A.stats("layer", np.array([[7.0, 3.0]]), 0.0)
    assert m[0, 0] == 5 and r[0, 0] == 0.5
    m, r = A.stats("rms", np.array([[3.0, 4.0]]), 0.0)
    assert m[0, 0] == 0 and abs(r[0, 0] - np.sqrt(2) / 5) < 1e-15
    m, r = A.stats("layer", np.array([[4.0, 4.0]]), 0.25)
    assert r[0, 0] == 2
    np.testing.assert_allclose(A.act("silu", np.array([0.0, 1.0]))[0], [0, 1 / (1 + np.exp(-1))])
    np.testing.assert_allclose(A.act("sigmoid", np.array([0.0]))[1], [0.25])


def test_block_by_hand():
    # b = (7, 3): normalised (1, -1); gamma 2, beta 1: (3, -1); gate (none) (2, 2): (6, -2); s = .5: + x
    cfg = {"post": "layer", "pre": "rms", "gate": None}
    p = {"post_gamma": np.array([2.0, 2]), "post_beta": np.array([1.0, 1]), "res_scale": np.array([.5, .5]), "pre_gamma": np.array([1.0, 3])}
    y, _, _ = A.block_y(cfg, p, np.array([[0.0, 5]]), np.array([[7.0, 3]]), np.array([[2.0, 2]]), 0.0)
    np.testing.assert_array_equal(y, [[3, 4]])
    h, _, r = A.block_h(cfg, p, y, 0.0)
    np.testing.assert_allclose(h, np.array([[3, 12]]) * np.sqrt(2) / 5, rtol=1e-15)


@pytest.mark.parametrize("post,pre,gate", [("layer", "layer", "silu"), ("rms", "layer", "sigmoid"), ("layer", "rms", None),
                                           (None, "rms", "silu"), ("rms", None, "none")])
def test_block_gradients_by_differences(post, pre, gate):
    rng = np.random.default_rng(3)
    T, d, eps = 3, 6, 1e-3
    cfg = {"post": post, "pre": pre, "gate": gate}
    v = {n: rng.normal(size=(T, d)) for n in ("x", "b", "gate")}
    p = {n: rng.normal(size=d) for n in ("post_gamma", "post_beta", "res_scale", "pre_gamma", "pre_beta")}
    if gate is None:
        v["gate"] = None
    wy, wh = rng.normal(size=(T, d)), rng.normal(size=(T, d))

    def loss(v, p):
        y, _, _ = A.block_y(cfg, p, v["x"], v["b"], v["gate"], eps)
        return float((wy * y).sum() + (wh * A.block_h(cfg, p, y, eps)[0]).sum())

    y, m1, r1 = A.block_y(cfg, p, v["x"], v["b"], v["gate"], eps)
    _, m2, r2 = A.block_h(cfg, p, y, eps)
    got = A.block_bwd(cfg, p, y, v["b"], v["gate"], np.concatenate([m1, r1, m2, r2], 1), wy, wh)
    where = {"x": "dx", "b": "db", "gate": "dgate"}
    for name, a in [*v.items(), *p.items()]:
        g = got.get(where.get(name, name))
        if a is None:
            continue
        if g is None:                       # a parameter of a norm that is not there
            assert name.split("_")[0] in ("post", "pre") and cfg[name.split("_")[0]] is None
            continue
        for i in np.ndindex(a.shape):
            old, h = a[i], 1e-5
            a[i] = old + h
            up = loss(v, p)
            a[i] = old - h
            down = loss(v, p)
            a[i] = old
            assert abs((up - down) / (2 * h) - g[i]) < 1e-6 * max(1, abs(g[i])), (name, i)


def test_e4m3_table():
    # smallest subnormal, largest subnormal, smallest normal, 1, largest
    for code, v in ((1, 2.0 ** -9), (7, 7 * 2.0 ** -9), (8, 2.0 ** -6), (56, 1.0), (126, 448.0)):
        assert A.E4M3[code] == v
    assert np.all(np.diff(A.E4M3) > 0)


@pytest.mark.parametrize("fmt,top", [("int8", 127.0), ("e4m3", 448.0)])
def test_hold_scales_and_roundings(fmt, top):
    x = np.zeros((1, 32))
    # the group's largest value on, just above and just below top 2^k
    for big, k in ((top, 0), (top * (1 + 1e-9), 1), (top / 2, -1), (top * 2 ** 10, 10), (0.0, -126), (2.0 ** -140, -126)):
        x[0, 5] = big
        q, e, back = A.hold(fmt, x)
        assert e[0, 0] == k, big
        assert np.all(np.abs(q) <= top)
    rng = np.random.default_rng(1)
    x = rng.normal(size=(20, 64)) * np.exp(rng.normal(size=(20, 64)) * 3)
    q, e, back = A.hold(fmt, x)
    unit = np.repeat(2.0 ** e, 32, axis=1)
    half = 0.5 * unit if fmt == "int8" else np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10 * unit)
    assert np.all(np.abs(back - x) <= half)
    # brute force: no code is nearer
    codes = np.arange(-127, 128) if fmt == "int8" else np.concatenate([-A.E4M3, A.E4M3])
    for i, j in ((0, 0), (3, 40), (7, 63), (19, 20)):
        assert abs(back[i, j] - x[i, j]) <= np.min(np.abs(codes * unit[i, j] - x[i, j])) * (1 + 1e-12)


def test_hold_ties_go_to_even():
    x = np.zeros((1, 32))
    x[0, :6] = [127.0, 2.5, 3.5, -2.5, 0.5, 126.5]
    np.testing.assert_array_equal(A.hold("int8", x)[0][0, :6], [127, 2, 4, -2, 0, 126])
    x[0, :5] = [448.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10]
    np.testing.assert_array_equal(A.hold("e4m3", x)[0][0, :5], [448, 16, 20, 0, 2 * 2.0 ** -9])


def test_hold_marks_non_finite_groups():
    for bad in (np.nan, np.inf, -np.inf):
        x = np.ones((1, 64))
        x[0, 40] = bad
        _, k, back = A.hold("int8", x)
        assert k[0, 1] == 128 and np.all(np.isnan(back[0, 32:])) and np.all(back[0, :32] == 1)
