"""Pins of the float64 oracle of the operators around the recurrence (CPU): every gradient against
central differences of the forward, and cases worked by hand."""
import math

import numpy as np
import pytest

from oracle import layer as L


def _diff(f, x, upstream, h=1e-5):
    """Central differences of <f(x), upstream> in every element of x."""
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        old = x[i]
        x[i] = old + h
        up = f()
        x[i] = old - h
        dn = f()
        x[i] = old
        g[i] = sum(((a - b) * u).sum() for a, b, u in zip(up, dn, upstream)) / (2 * h)
    return g


def _near(a, b, tol=1e-7):
    return np.max(np.abs(a - b)) <= tol * max(1.0, np.max(np.abs(b)))


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (2, 4)])
def test_scan_gradients_are_differences(Hk, Hv):
    rng = np.random.default_rng(3)
    cu, Dk, Dv = [0, 3, 3, 7], 3, 2
    T, N = cu[-1], 3
    v = dict(x=rng.standard_normal((T, Hv, Dv)), b=rng.standard_normal((T, Hk, Dk)), c=rng.standard_normal((T, Hk, Dk)),
             dt=rng.standard_normal((T, Hv)), a_log=rng.standard_normal(Hv) * 0.5, dt_bias=rng.standard_normal(Hv),
             d_skip=rng.standard_normal(Hv), S0=rng.standard_normal((N, Hv, Dk, Dv)))
    dy, dST = rng.standard_normal((T, Hv, Dv)), rng.standard_normal((N, Hv, Dk, Dv))
    got = L.ssm_bwd(cu, *v.values(), dy, dST)
    f = lambda: L.ssm_fwd(cu, *v.values())
    for name in v:
        want = _diff(f, v[name], (dy, dST))
        assert _near(got["d" + name], want), name


def test_scan_by_hand():
    """One head, Dk = Dv = 1, softplus(dt) = ln 2 at dt = 0, a_log = 0: a = 1/2. x = 1, b = 2, c = 3:
    S = ln 4, then ln 4 / 2 + ln 4; y = 3 S + x with d_skip = 1."""
    one = np.ones((2, 1, 1))
    y, ST = L.ssm_fwd([0, 2], one, 2 * one, 3 * one, np.zeros((2, 1)), np.zeros(1), None, np.ones(1), None)
    s = math.log(4.0)
    assert np.allclose(y.ravel(), [3 * s + 1, 3 * 1.5 * s + 1], rtol=1e-15) and np.allclose(ST.ravel(), [1.5 * s], rtol=1e-15)


def test_conv_by_hand():
    """K = 3, weights 1, 2, 3: rows 1, 2 behind carried rows 5, 7; z = 5 + 14 + 3 and 7 + 2 + 6, plus the
    bias -1; the window moves on to (1, 2), and to (7, 1) after one row only."""
    x, w, first = np.array([[1.0], [2.0]]), np.array([[1.0, 2.0, 3.0]]), np.array([[[5.0], [7.0]]])
    silu = lambda z: z / (1 + math.exp(-z))
    y, last = L.conv_prompt([0, 2], x, w, np.array([-1.0]), first)
    assert np.allclose(y.ravel(), [silu(21.0), silu(14.0)]) and np.array_equal(last.ravel(), [1.0, 2.0])
    assert np.array_equal(L.conv_prompt([0, 1], x[:1], w, None, first)[1].ravel(), [7.0, 1.0])
    assert np.array_equal(L.conv_prompt([0, 0], x[:0], w, None, first)[1].ravel(), [5.0, 7.0])


@pytest.mark.parametrize("gate_first", [False, True])
def test_gated_norm_gradients_are_differences(gate_first):
    rng = np.random.default_rng(4)
    x, z, dy = (rng.standard_normal((3, 2, 4)) for _ in range(3))
    w = rng.standard_normal((2, 4))
    got = L.gated_norm_bwd(x, z, w, 1e-2, gate_first, dy)
    f = lambda: (L.gated_norm(x, z, w, 1e-2, gate_first),)
    for g, v in zip(got, (x, z, w)):
        assert _near(g, _diff(f, v, (dy,)))


def test_norm_by_hand():
    """(3, 4): mean square 12.5; with eps 0 the norm is (3, 4) / sqrt(12.5)."""
    v = np.array([[[3.0, 4.0]]])
    big = np.full_like(v, 40.0)  # silu(40) = 40 to 1e-16
    assert np.allclose(L.gated_norm(v, big, np.ones((1, 2)), 0.0, False), 40 * v / math.sqrt(12.5), rtol=1e-14)
    assert np.allclose(L.gated_norm(v, big, np.ones((1, 2)), 0.0, True), v / math.sqrt(12.5), rtol=1e-14)


def test_add_norm_gradients_are_differences():
    rng = np.random.default_rng(5)
    h, y, dout, dres = (rng.standard_normal((3, 5)) for _ in range(4))
    s, w, scale, eps = rng.standard_normal(5), rng.standard_normal(5), 0.7, 1e-2

    def f():
        res = h + scale * s * y
        return res * L._rms(res, eps) * w, res

    got = L.add_norm_bwd(h + scale * s * y, y, scale * s, w, eps, dout, dres, scale)
    for g, v in zip(got, (h, y, w, s)):
        assert _near(g, _diff(f, v, (dout, dres)))
