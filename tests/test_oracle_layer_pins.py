"""The fp64 reference of the layer (`oracle/layer.py`) against closed forms and, for the
gradients, against central differences of its forward.

Differences: with step s the central difference of a smooth f is off by f''' s^2 / 6 and by
rounding of about 2^-52 |f| / s; s = 1e-5 on values of order 1 leaves both below 1e-9, and the
bound taken is 1e-7.
"""
import numpy as np
import pytest

from oracle import layer as ol

STEP, TOL = 1e-5, 1e-7


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def differences(f, x):
    """Gradient of the scalar f by central differences over the entries of x (in place)."""
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        v = x[i]
        x[i] = v + STEP
        a = f()
        x[i] = v - STEP
        b = f()
        x[i] = v
        g[i] = (a - b) / (2 * STEP)
    return g


def test_closed_forms():
    assert np.allclose(ol.act("gelu", np.array([0.0, 30.0, -30.0])), [0, 30, 0], atol=1e-15)
    assert np.allclose(ol.act("silu", np.array([0.0, 800.0, -800.0])), [0, 800, 0], atol=1e-15)
    # a constant row has root mean square |c|
    y, h = ol.residual_norm(np.full((2, 5), -3.0), np.arange(5.0), eps=1e-30)
    assert np.allclose(y, -np.arange(5.0)) and np.array_equal(h, np.full((2, 5), -3.0))
    # a zero row stays zero
    assert not ol.residual_norm(np.zeros((1, 4)), np.ones(4))[0].any()
    # one-hot rows: z picks a weight row
    w = rng(0).standard_normal((3, 4))
    assert np.array_equal(ol.linear(np.eye(4), w)[0], w.T)


@pytest.mark.parametrize("kind", ["none", "silu", "gelu", "sigmoid"])
def test_linear_gradients(kind):
    r = rng(1)
    x, w, b = r.standard_normal((4, 5)), r.standard_normal((3, 5)), r.standard_normal(3)
    dy = r.standard_normal((4, 3))

    def f():
        return float((ol.linear(x, w, b, kind, None, 0.7)[0] * dy).sum())
    z = ol.linear(x, w, b, kind, None, 0.7)[1]
    dx, dw, db, _ = ol.linear_bwd(x, w, dy, z, kind, 0.7)
    for got, arr in ((dx, x), (dw, w), (db, b)):
        assert np.max(np.abs(got - differences(f, arr))) <= TOL


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_residual_norm_gradients(post, gate):
    r = rng(2)
    T, N = 3, 6
    x, res, w = r.standard_normal((T, N)), r.standard_normal((T, N)), r.standard_normal(N)
    pw = r.standard_normal(N) if post else None
    g = {"none": None, "channel": r.standard_normal(N), "token": r.standard_normal((T, N))}[gate]
    dy, dh = r.standard_normal((T, N)), r.standard_normal((T, N))

    def f():
        y, h = ol.residual_norm(x, w, res, pw, g, 0.5)
        return float((y * dy).sum() + (h * dh).sum())
    h = ol.residual_norm(x, w, res, pw, g, 0.5)[1]
    dx, dr, dw, dpw, dg = ol.residual_norm_bwd(x, h, w, dy, dh, pw, g, 0.5)
    pairs = [(dx, x), (dr, res), (dw, w)]
    if post:
        pairs.append((dpw, pw))
    if gate != "none":
        pairs.append((dg.sum(0) if gate == "channel" else dg, g))
    for got, arr in pairs:
        assert np.max(np.abs(got - differences(f, arr))) <= TOL


@pytest.mark.parametrize("kind", ["sigmoid", "silu", "none"])
def test_gated_norm_gradients(kind):
    r = rng(3)
    o, g, w = r.standard_normal((2, 3, 5)), r.standard_normal((2, 3, 5)), r.standard_normal(5)
    dy = r.standard_normal((2, 3, 5))

    def f():
        return float((ol.gated_norm(o, g, w, kind) * dy).sum())
    for got, arr in zip(ol.gated_norm_bwd(o, g, w, dy, kind), (o, g, w)):
        assert np.max(np.abs(got - differences(f, arr))) <= TOL
