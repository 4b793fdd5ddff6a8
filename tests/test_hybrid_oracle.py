"""Pins of the float64 oracle of the other token mixers (CPU): every gradient against central differences of
the forward, and cases worked by hand."""
import math

import numpy as np
import pytest

from oracle import hybrid as O


def _diff(f, x, upstream, h=1e-5):
    """Central differences of <f(), upstream> in every element of x."""
    g = np.zeros_like(x)
    for at in np.ndindex(*x.shape):
        old, side = x[at], []
        for d in (h, -h):
            x[at] = old + d
            side.append(sum((a * u).sum() for a, u in zip(f(), upstream)))
        x[at] = old
        g[at] = (side[0] - side[1]) / (2 * h)
    return g


def _near(a, b, tol=1e-7):
    return np.max(np.abs(a - b)) <= tol * max(1.0, np.max(np.abs(b)))


@pytest.mark.parametrize("fresh", [None, [1, 0, 1, 0], [1, 1, 1, 1]])
@pytest.mark.parametrize("init", [True, False])
def test_recurrence_gradients_are_differences(fresh, init):
    rng = np.random.default_rng(5)
    cu, C = [0, 3, 3, 4, 8], 3
    T, N = cu[-1], 4
    v = dict(x=rng.standard_normal((T, C)), r=rng.standard_normal((T, C)), i=rng.standard_normal((T, C)), lam=rng.standard_normal(C))
    h0 = rng.standard_normal((N, C)) if init else None
    dy, dhT = rng.standard_normal((T, C)), rng.standard_normal((N, C))
    f = lambda: O.glr_fwd(cu, *v.values(), 8.0, h0, fresh)
    got = O.glr_bwd(cu, *v.values(), 8.0, h0, fresh, dy, dhT)
    for name in v:
        assert _near(got["d" + name], _diff(f, v[name], (dy, dhT))), name
    if init:
        assert _near(got["dh0"], _diff(f, h0, (dy, dhT)))


def test_recurrence_by_hand():
    """r = 0: s = 1/2; lam = 0: softplus = ln 2; rate 4: L = 2 ln 2, a = 1/4, w = sqrt(15) / 4; i = ln 3: s = 3/4; x = 4: u = 3."""
    one = np.ones((2, 1))
    y, hT = O.glr_fwd([0, 2], 4 * one, 0 * one, math.log(3) * one, np.zeros(1), 4.0, np.array([[8.0]]))
    b = 3 * math.sqrt(15) / 4
    assert np.allclose(y[:, 0], [2 + b, (2 + b) / 4 + b], rtol=1e-14) and hT[0, 0] == y[1, 0]
    y, _ = O.glr_fwd([0, 2], 4 * one, 0 * one, math.log(3) * one, np.zeros(1), 4.0, np.array([[8.0]]), [1])
    assert np.allclose(y[:, 0], [3, 0.75 + b], rtol=1e-14)  # fresh: the first token as it is
    y, s = O.glr_step(4 * one, 0 * one, math.log(3) * one, np.zeros(1), 4.0, np.full((3, 1), 8.0), [2, 7])
    assert np.allclose(s[:, 0], [8, 8, 2 + b]) and np.isnan(y[1, 0])


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("R", [0, 4, 8])
def test_rotation_gradients_are_differences(adjacent, R):
    rng = np.random.default_rng(6)
    v, w, dy = rng.standard_normal((3, 2, 8)), 1 + 0.3 * rng.standard_normal(8), rng.standard_normal((3, 2, 8))
    pos, freq = np.array([0, 5, 100003]), 100.0 ** -np.arange(R // 2)
    f = lambda: (O.norm_rope(v, w, pos, freq, R, adjacent, 1e-3, 1.25),)
    dv, dw = O.norm_rope_bwd(v, w, pos, freq, R, adjacent, 1e-3, dy, 1.25)
    assert _near(dv, _diff(f, v, (dy,))) and _near(dw, _diff(f, w, (dy,)))


def test_rotation_by_hand():
    """(3, 4, 3, 4): mean square 12.5; a quarter of a turn takes (a, b) to (-b, a)."""
    v = np.array([[[3.0, 4.0, 3.0, 4.0]]])
    n = v / math.sqrt(12.5)
    quarter = np.array([math.pi / 2, math.pi / 2])
    assert np.allclose(O.norm_rope(v, np.ones(4), np.array([1]), quarter, 4, False, 0.0) * math.sqrt(12.5), [[[-3, -4, 3, 4]]])
    assert np.allclose(O.norm_rope(v, np.ones(4), np.array([1]), quarter, 4, True, 0.0) * math.sqrt(12.5), [[[-4, 3, -4, 3]]])
    assert np.allclose(O.norm_rope(v, np.ones(4), np.array([0]), quarter, 4, True, 0.0), n)


def test_attention_by_hand():
    """Scores 0 and ln 3: weights 1/4 and 3/4; the window and a page outside the pool leave one token; no token at all."""
    k = np.array([[[[0.0]], [[1.0]]], [[[1.0]], [[0.0]]]]).transpose(0, 2, 1, 3)  # 2 pages x 1 head x 2 tokens x 1
    v = np.array([[[[4.0], [8.0]]], [[[2.0], [6.0]]]])
    q = np.full((1, 1, 1), math.log(3))
    run = lambda table, n, **kw: O.paged(q, k, v, np.array([table]), [n], 1.0, **kw)[:2]
    out, lse = run([0, 1], 2)
    assert np.isclose(out[0, 0, 0], 7) and np.isclose(lse[0, 0], math.log(4))
    assert run([0, 1], 2, window=1)[0][0, 0, 0] == 8 and run([5, 1], 4, window=3)[0][0, 0, 0] == pytest.approx(3)
    out, lse = run([0, 1], 0)
    assert out[0, 0, 0] == 0 and lse[0, 0] == -math.inf
