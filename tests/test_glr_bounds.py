"""The bounds of glr_bounds.py on the CPU: narrow enough that a mistake of a thousandth, or a lost part of a sum, is outside."""
import numpy as np
import pytest

import glr_bounds as B
from oracle import hybrid as O


@pytest.fixture(scope="module", params=range(len(B.CASES)), ids=lambda k: f"{B.CASES[k][0]}-{len(B.CASES[k][1])}x{sum(B.CASES[k][1])}")
def case(request):
    dtype, lens, C, _ = B.CASES[request.param]
    v, g = B.draw(lens, C, 91 + request.param, dtype)
    names = [v[k] for k in ("cu", "x", "r", "i", "lam", "rate", "h0", "fresh")]
    return dtype, v, g, B.wanted(v, g), B.bounds(*names, *g.values(), dtype)


def outside(got, want, bound, dtype, k):
    """Where got[k] is outside."""
    return np.abs(got - want) > bound + 2.0 ** -126 + (B.HALF[dtype] * (np.abs(want) + bound) if k in B.ROWS else 0.0)


def test_bounds_are_narrow(case):
    dtype, v, g, want, bound = case
    for k in ("y", "hT", "dx", "di", "dh0"):
        assert (bound[k] <= 5e-4 * np.abs(want[k])).all(), k
    assert np.linalg.norm(bound["dr"]) <= 2e-4 * np.linalg.norm(want["dr"])
    narrow = bound["dlam"] / np.abs(want["dlam"])  # (in a channel whose states start above where they settle, tokens of both signs may cancel)
    assert np.median(narrow) <= 2e-4 and (narrow <= 5e-3).mean() > 0.9
    assert max(B.beyond(want, want, bound, dtype).values()) == 0


def test_a_lost_part_of_dlambda_is_outside(case):
    """The sum over a segment (256 tokens at most) missing, or there twice."""
    dtype, v, g, want, bound = case
    part = want["dr"] / O.sigmoid(-v["r"]) * (O.sigmoid(v["lam"]) / np.logaddexp(v["lam"], 0.0))  # of each token
    assert np.allclose(part.sum(0), want["dlam"], rtol=1e-10)
    for lo, hi in zip(v["cu"], v["cu"][1:]):
        for t in range(lo, hi, 256):
            if min(hi, t + 256) - t < 128:
                continue
            for sign in (-1, 1):
                hit = outside(want["dlam"] + sign * part[t:min(hi, t + 256)].sum(0), want["dlam"], bound["dlam"], dtype, "dlam")
                assert hit.mean() > 0.75, (lo, t)


def test_a_lost_state_or_gradient_is_outside(case):
    """A segment that starts from nothing: its first states (and the last gradients in front of it) are outside."""
    dtype, v, g, want, bound = case
    for n, (lo, hi) in enumerate(zip(v["cu"], v["cu"][1:])):
        if hi - lo < 300:
            continue
        cut = lo + 256
        rows = lambda a: a[cut:hi]
        y, _ = O.glr_fwd([0, hi - cut], *(rows(v[k]) for k in "xri"), v["lam"], v["rate"])
        assert outside(y[:8], want["y"][cut:cut + 8], bound["y"][cut:cut + 8], dtype, "y").all()
        rows = lambda a: a[lo:cut]
        alone = O.glr_bwd([0, cut - lo], *(rows(v[k]) for k in "xri"), v["lam"], v["rate"], None if v["h0"] is None else v["h0"][n:n + 1],
                          None if v["fresh"] is None else v["fresh"][n:n + 1], rows(g["dy"]), None)
        assert outside(alone["dx"][-8:], want["dx"][cut - 8:cut], bound["dx"][cut - 8:cut], dtype, "dx").all()


def test_a_thousandth_of_a_gate_is_outside(case, monkeypatch):
    """The input's weight, or the decay's exponent, a thousandth off (float32 rows; half a step of bfloat16 is four)."""
    dtype, v, g, want, bound = case
    gates = O.glr_gates
    for change in (lambda L, a, w: (L, a, w * 1.001), lambda L, a, w: (L * 1.001, np.exp(-L * 1.001), np.sqrt(-np.expm1(-2.002 * L)))):
        monkeypatch.setattr(O, "glr_gates", lambda *args: change(*gates(*args)))
        got = B.wanted(v, g)
        monkeypatch.setattr(O, "glr_gates", gates)
        off = B.beyond(got, want, bound, dtype)
        for k in ("hT", "dlam") if dtype == "bf16" else ("y", "hT", "dx", "dr", "di", "dlam"):
            assert off[k] > 1, k
