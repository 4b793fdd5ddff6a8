"""GPU: the gated linear recurrence within the bounds of glr_bounds.py, a few 1e-5 of a float32 result (rows add half a step
of their type)."""
import numpy as np
import pytest
import torch  # noqa: F401  (in front of the package, which then has torch's HIP runtime)

import glr_bounds as B
from layer_gpu import dev, host, rounded
from test_glr_gpu import run

pytestmark = pytest.mark.gpu


def check(v, g, dtype, **kw):
    out = {k: host(t) for k, t in run(v, g, dtype, **kw).items()}
    want = B.wanted(v, g)
    bound = B.bounds(*[v[k] for k in ("cu", "x", "r", "i", "lam", "rate", "h0", "fresh")], *g.values(), dtype)
    off = B.beyond(out, want, bound, dtype)
    assert max(off.values()) <= 1, off


@pytest.mark.parametrize("k", range(len(B.CASES)), ids=lambda k: f"{B.CASES[k][0]}-{len(B.CASES[k][1])}x{sum(B.CASES[k][1])}")
def test_cases(k):
    """Outputs and all gradients, of whole sequences and of ones cut into segments."""
    dtype, lens, C, table = B.CASES[k]
    check(*B.draw(lens, C, 91 + k, dtype), dtype, cu=table)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("init,fresh", [(True, "none"), (True, "all"), (False, "none")])
def test_starts(dtype, init, fresh):
    check(*B.draw([5, 0, 140, 600, 2100], 40, 89, dtype, init, fresh), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[1, 1, 1, 1], [40, 1, 0, 7, 200], [300, 777]])
def test_gradients_of_open_gates(dtype, lens):
    """Gates of up to 85, whose complements 1 - s(z) the gradients of r and i have as a factor."""
    v, g = B.draw(lens, 72, 81 + len(lens), dtype, fresh="none")
    rng = np.random.default_rng(82)
    for k in "ri":
        wide = rng.random(v[k].shape)
        v[k] = rounded(np.where(wide < 0.5, v[k], np.where(wide < 0.9, rng.uniform(5, 30, v[k].shape), rng.uniform(-85, 85, v[k].shape))), dtype)
    check(v, g, dtype)


def test_open_gates_in_place():
    """A gradient over the very rows that its complement is formed from."""
    import gated_delta_rule_34_amd as G

    v, g = B.draw([300, 77], 72, 83, "bf16", fresh="none")
    v["r"], v["i"] = rounded(6 * v["r"], "bf16"), rounded(6 * v["i"], "bf16")
    want = run(v, g, "bf16")
    p = G.make_glr_problem(2, 377, 72, lam=dev(v["lam"]), cu_seqlens=torch.tensor(v["cu"], dtype=torch.int32, device="cuda"))
    saved = G.glr_forward(p, *(dev(v[k], "bf16") for k in "xri"), dev(v["h0"]))[2]
    for order in ((0, 1, 2), (1, 2, 0), (2, 0, 1)):
        rows = [dev(v[n], "bf16") for n in "xri"]
        out = [rows[k] for k in order]
        ws = torch.empty(G.gdn_glr_bwd_workspace_bytes(p), dtype=torch.uint8, device="cuda")
        G.gdn_glr_bwd(p, *rows, saved, dev(g["dy"], "bf16"), dev(g["dhT"]), *out, None, None, ws)
        for a, n in zip(out, ("dx", "dr", "di")):
            assert torch.equal(a, want[n]), (order, n)


@pytest.mark.parametrize("z", [float("inf"), -float("inf"), 200.0, -200.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gates_without_a_complement(dtype, z):
    """Gates at their ends: no gradient of them, none that is not finite."""
    v, g = B.draw([50, 9], 16, 84, dtype, fresh="none")
    v["r"][:, :8], v["i"][:, 8:] = z, z
    out = run(v, g, dtype)
    assert all(bool(torch.isfinite(t).all()) for t in out.values())
    assert not out["dr"][:, :8].any() and not out["di"][:, 8:].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dlambda_of_very_small_rates(dtype):
    """lambda down to -92, where the softplus is a float32 below 2^-126 (off by up to 2^-149) and exp(-lambda) is none: with a rate of 1e5
    the exponents and dlambda are ordinary numbers."""
    v, g = B.draw([300, 40, 700], 24, 85, dtype, fresh="none")
    v["lam"], v["rate"] = rounded(np.repeat([-20.5, -60.0, -88.0, -89.0, -90.5, -92.0], 4), "f32"), 1e5
    got, want = host(run(v, g, dtype)["dlam"]), B.wanted(v, g)["dlam"]
    bound = B.bounds(*[v[k] for k in ("cu", "x", "r", "i", "lam", "rate", "h0", "fresh")], *g.values(), dtype)["dlam"]
    step = 2.0 ** -149 * np.exp(-v["lam"])  # of the softplus, relative
    assert (np.abs(want) > 2.0 ** -100).all() and (bound < 1e-3 * np.abs(want)).all() and (step < 1e-4).all()
    assert (np.abs(got - want) <= bound + step * np.abs(want)).all()
