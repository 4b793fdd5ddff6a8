"""GPU: the selective state space scan (prompts, gradients, single tokens) against the float64
oracle's token-by-token recurrence.

Tolerances (2-norm relative). bfloat16 outputs: the result's own rounding and that of the two
bfloat16 operands behind it, each at most 2^-8 of a value and so at most 2^-8 / sqrt(3) in the mean
square: together 2^-8. float32 outputs: the operands keep 24 bits; a decay over the few units of
log2 that matter carries some 8 2^-23, and sums of up to some thousand terms of either sign some
sqrt(4096) 2^-24: together below 1e-5."""
import numpy as np
import pytest

from layer_gpu import cu_of, dev, host, rel, rounded, torch_dtype

pytestmark = pytest.mark.gpu

TOL = {"bf16": 2.0 ** -8, "f32": 1e-5}
GRADS = ("dx", "db", "dc", "ddt", "da_log", "ddt_bias", "dd_skip", "dS0")


def make(lens, Hk, Hv, Dk, Dv, dtype, seed=0, bias=True, skip=True, init=True, dt=None, a_log=None):
    rng = np.random.default_rng(seed)
    T, N = sum(lens), len(lens)
    a = dict(x=rounded(rng.standard_normal((T, Hv, Dv)), dtype), b=rounded(rng.standard_normal((T, Hk, Dk)), dtype),
             c=rounded(rng.standard_normal((T, Hk, Dk)), dtype),
             dt=rounded(rng.standard_normal((T, Hv)) - 2 if dt is None else np.broadcast_to(dt, (T, Hv)), "f32"),
             a_log=rounded(rng.uniform(-1, 2, Hv) if a_log is None else np.full(Hv, a_log), "f32"),
             dt_bias=rounded(rng.standard_normal(Hv), "f32") if bias else None,
             d_skip=rounded(rng.standard_normal(Hv), "f32") if skip else None,
             S0=rounded(0.5 * rng.standard_normal((N, Hv, Dk, Dv)), "f32") if init else None)
    up = dict(dy=rounded(rng.standard_normal((T, Hv, Dv)), dtype), dST=rounded(0.3 * rng.standard_normal((N, Hv, Dk, Dv)), "f32"))
    return a, up, cu_of(lens)


def place(a, up, cu, dtype, packed=True, varlen=True, lens=None):
    """Device tensors and the problem; packed: x | b | c are views of one row, padded to 16 more values."""
    import torch
    import gated_delta_rule_34_amd as G

    T, Hv, Dv = a["x"].shape
    Hk, Dk = a["b"].shape[1:]
    flat = {k: a[k].reshape(T, a[k].shape[1] * a[k].shape[2]) for k in ("x", "b", "c")}
    if packed:
        row = torch.full((T, Hv * Dv + 2 * Hk * Dk + 16), float("nan"), dtype=torch_dtype(dtype), device="cuda")
        d, at = {}, 0
        for k, v in flat.items():
            d[k] = row[:, at:at + v.shape[1]]
            d[k].copy_(dev(v, dtype))
            at += v.shape[1]
    else:
        d = {k: dev(v, dtype) for k, v in flat.items()}
    for k in ("dt", "a_log", "dt_bias", "d_skip", "S0"):
        d[k] = dev(a[k])
    d["dy"], d["dST"] = dev(up["dy"].reshape(T, Hv * Dv), dtype), dev(up["dST"])
    kw = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda")) if varlen else dict(T=lens[0])
    p = G.make_ssm_problem(len(cu) - 1, T, Hk, Hv, Dk, Dv, a_log=d["a_log"], dt_bias=d["dt_bias"], d_skip=d["d_skip"], dtype=dtype, **kw)
    return p, d


def run(p, d, backward=True, dST=True):
    import gated_delta_rule_34_amd as G

    y, ST, sv = G.ssm_forward(p, d["x"], d["b"], d["c"], d["dt"], d["S0"], save=backward)
    out = dict(y=y, S_T=ST)
    if backward:
        out.update(G.ssm_backward(p, d["x"], d["b"], d["c"], d["dt"], d["S0"], sv, d["dy"], d["dST"] if dST else None))
    return out


def check(a, up, cu, dtype, out, dST=True, more=0.0):
    """``more``: what a test's decays add to the float32 tolerance. Values below 1e-30 are beneath float32."""
    from oracle import layer as L

    y, ST = L.ssm_fwd(cu, *a.values())
    want = dict(y=y, S_T=ST)
    if "dx" in out:
        want.update(L.ssm_bwd(cu, *a.values(), up["dy"], up["dST"] if dST else None))
    errs = {k: rel(host(out[k]), v) if np.linalg.norm(host(out[k]).reshape(-1) - v.reshape(-1)) > 1e-30 * v.size ** 0.5 else 0.0
            for k, v in want.items() if out.get(k) is not None}
    assert all(np.isfinite(host(v)).all() for v in out.values() if v is not None)
    bad = {k: e for k, e in errs.items() if not e <= TOL[dtype if k in ("y", "dx", "db", "dc") else "f32"] + more}
    assert not bad, (bad, errs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Dk", [16, 32, 64, 128])
@pytest.mark.parametrize("Dv", [16, 32, 64, 128])
def test_scan_all_sizes(dtype, Dk, Dv):
    """Lengths around the chunk, one token, none; three heads to a group; padded packed rows."""
    a, up, cu = make([1, 0, 63, 64, 65, 130], 2, 6, Dk, Dv, dtype, seed=Dk + Dv)
    check(a, up, cu, dtype, run(*place(a, up, cu, dtype)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[1], [3000], [1500, 700], [0, 0, 1000, 0]])
def test_scan_few_long_sequences(dtype, lens):
    """One head and few sequences: the long axis is cut into segments."""
    a, up, cu = make(lens, 1, 2, 32, 64, dtype, seed=7)
    check(a, up, cu, dtype, run(*place(a, up, cu, dtype, packed=False)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("r,lens", [(7, [1000]), (9, [2500, 100]), (17, [70, 20])])
def test_scan_groups_of_many_heads(dtype, r, lens):
    """A group's heads by several workgroups with an uneven share, by one workgroup over more than it
    takes at a time, and by one workgroup each."""
    a, up, cu = make(lens, 4, 4 * r, 16, 32, dtype, seed=r)
    check(a, up, cu, dtype, run(*place(a, up, cu, dtype)))


@pytest.mark.parametrize("r", [1, 7])
def test_scan_equal_lengths_and_missing_parts(r):
    """No cu_seqlens, no bias, no skip, no initial state, no dS_T; the gradients nobody asks for are skipped."""
    import torch
    import gated_delta_rule_34_amd as G

    a, up, cu = make([100, 100], 2, 2 * r, 64, 32, "bf16", seed=9, bias=False, skip=False, init=False)
    p, d = place(a, up, cu, "bf16", varlen=False, lens=[100, 100])
    out = run(p, d, dST=False)
    assert out["ddt_bias"] is None and out["dd_skip"] is None
    check(a, up, cu, "bf16", out, dST=False)
    y, ST, sv = G.ssm_forward(p, d["x"], d["b"], d["c"], d["dt"], None)
    g = {k: torch.empty_like(out[k]) for k in ("dx", "db", "dc", "ddt")}
    G.ssm_backward(p, d["x"], d["b"], d["c"], d["dt"], None, sv, d["dy"], None, grads=g)
    assert all(torch.equal(g[k], out[k]) for k in g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dt,a_log", [(-60.0, 0.0), (30.0, 3.0), (-3.0, -20.0), (2.0, 2.7)])
def test_scan_extreme_steps(dtype, dt, a_log):
    """Steps that vanish (nothing is written), decays that leave nothing, decays of one, and strong
    decays whose exponents reach thousands within a chunk. One token's decay e^-m carries some
    m 4 2^-23 (the exponent is a float32 product of four factors), and m up to 80 can be seen in a float32."""
    a, up, cu = make([200, 33], 1, 2, 32, 32, dtype, seed=11, dt=dt, a_log=a_log, bias=False)
    m = np.exp(a_log) * np.logaddexp(dt, 0)
    check(a, up, cu, dtype, run(*place(a, up, cu, dtype)), more=min(m, 80) * 4 * 2.0 ** -23)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dt,a_log", [(2.0, 100.0), (-200.0, 100.0), (1e6, 20.0), (0.0, -200.0)])
def test_scan_rates_past_float32(dtype, dt, a_log):
    """Rates exp(a_log) and exponents beyond float32: nothing is left of a state, or (a step of zero, a
    rate of zero) all of it; prompts, gradients and single tokens alike. In the second case the step is zero in
    float32 and 1e-87 in the oracle, and 3e43 of it is still nothing."""
    import torch
    import gated_delta_rule_34_amd as G

    a, up, cu = make([130, 33], 1, 2, 32, 32, dtype, seed=12, dt=dt, a_log=a_log, bias=False)
    a["dt"][[40, 100, 150]] = -200.0  # steps of zero between the others
    p, d = place(a, up, cu, dtype)
    check(a, up, cu, dtype, run(p, d))
    from oracle import layer as L

    one, up, cu = make([1, 1], 1, 2, 32, 32, dtype, seed=14, dt=dt, a_log=a_log, bias=False)
    p, d = place(one, up, cu, dtype, varlen=False, lens=[1])
    y, state = torch.empty(2, 64, dtype=torch_dtype(dtype), device="cuda"), d["S0"].clone()
    G.gdn_ssm_decode(p, d["x"], d["b"], d["c"], d["dt"], state, None, y)
    yr, STr = L.ssm_fwd(cu, *one.values())
    assert rel(host(y), yr) <= TOL[dtype] and rel(host(state), STr) <= 1e-5


def test_scan_forward_is_the_same_with_and_without_saving_and_on_every_run():
    import torch

    a, up, cu = make([300, 41], 2, 4, 128, 64, "bf16", seed=13)
    p, d = place(a, up, cu, "bf16")
    first, second, only = run(p, d), run(p, d), run(p, d, backward=False)
    for k in first:
        assert torch.equal(first[k], second[k]), k
    assert torch.equal(first["y"], only["y"]) and torch.equal(first["S_T"], only["S_T"])


def test_scan_leaves_rows_of_no_sequence_alone():
    """cu_seqlens that end before T_total and start behind 0 (a caller's error): rows outside keep
    their values, and what stands there (NaN) reaches nothing."""
    import torch
    import gated_delta_rule_34_amd as G

    a, up, cu = make([70, 50, 30], 1, 2, 32, 32, "bf16", seed=15)
    p, d = place(a, up, cu, "bf16")
    for k in ("x", "b", "c", "dt", "dy"):
        d[k][120:] = float("nan")
    want = run(p, d)
    short = torch.tensor([0, 70, 120], dtype=torch.int32, device="cuda")
    q = G.make_ssm_problem(2, 150, 1, 2, 32, 32, cu_seqlens=short, a_log=d["a_log"], dt_bias=d["dt_bias"], d_skip=d["d_skip"])
    y = torch.full_like(want["y"], 7.0)
    _, ST, sv = G.ssm_forward(q, d["x"], d["b"], d["c"], d["dt"], d["S0"][:2].contiguous(), y=y)
    assert torch.equal(y[:120], want["y"][:120]) and bool((y[120:] == 7.0).all()) and torch.equal(ST, want["S_T"][:2])
    g = {k: torch.full_like(want[k], 7.0) for k in ("dx", "db", "dc", "ddt", "da_log")}
    G.ssm_backward(q, d["x"], d["b"], d["c"], d["dt"], None, sv, d["dy"], d["dST"][:2].contiguous(), grads=g)
    for k in ("dx", "db", "dc", "ddt"):
        assert torch.equal(g[k][:120], want[k][:120]) and bool((g[k][120:] == 7.0).all()), k
    assert bool(torch.isfinite(g["da_log"]).all())


def test_scan_malformed_tables_stay_inside():
    """Negative, decreasing and overlong offsets complete without touching rows outside the buffers."""
    import torch
    import gated_delta_rule_34_amd as G

    a, up, cu = make([100, 60], 1, 2, 32, 32, "bf16", seed=16)
    p, d = place(a, up, cu, "bf16")
    for table in ([0, 500, 160], [90, 20, 160], [-5, 100, 160], [0, 160, 90], [160, 0, -160]):
        q = G.make_ssm_problem(2, 160, 1, 2, 32, 32, cu_seqlens=torch.tensor(table, dtype=torch.int32, device="cuda"), a_log=d["a_log"])
        _, _, sv = G.ssm_forward(q, d["x"], d["b"], d["c"], d["dt"], d["S0"])
        G.ssm_backward(q, d["x"], d["b"], d["c"], d["dt"], d["S0"], sv, d["dy"], d["dST"])
        torch.cuda.synchronize()


def test_scan_nan_stays_in_its_sequence_and_head():
    import torch

    a, up, cu = make([70, 40, 130], 1, 2, 32, 32, "bf16", seed=17)
    p, d = place(a, up, cu, "bf16")
    clean = run(p, d)
    d["x"][80, :32] = float("nan")  # sequence 1, head 0
    out = run(p, d)
    assert bool(out["y"][80, :32].isnan().all())
    for k in ("y", "dx"):
        assert torch.equal(out[k][:70], clean[k][:70]) and torch.equal(out[k][110:], clean[k][110:])
        assert torch.equal(out[k][70:110, 32:], clean[k][70:110, 32:])
    assert torch.equal(out["dS0"][[0, 2]], clean["dS0"][[0, 2]])


def test_scan_graph_replays_and_streams():
    """Captured on a side stream and replayed with eager work between; two graphs side by side."""
    import torch
    import gated_delta_rule_34_amd as G

    graphs = []
    for lens, seed in (([300, 0, 77], 19), ([2000], 20)):
        a, up, cu = make(lens, 1, 2, 64, 64, "bf16", seed=seed)
        p, d = place(a, up, cu, "bf16")
        eager = run(p, d)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            on_side = run(p, d)
        side.synchronize()
        assert all(torch.equal(on_side[k], eager[k]) for k in eager)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(p, d)
        graphs.append((graph, out, eager, p, d))
    for rep in range(3):
        for graph, out, eager, p, d in graphs:
            for t in out.values():
                t.fill_(float("nan"))
            graph.replay()
        torch.cuda.synchronize()
        for graph, out, eager, p, d in graphs:
            assert all(torch.equal(out[k], eager[k]) for k in eager), rep
            run(p, d)


def test_scan_empty_batches():
    import torch
    import gated_delta_rule_34_amd as G

    a, up, cu = make([0, 0], 1, 2, 32, 32, "bf16", seed=21)
    p, d = place(a, up, cu, "bf16", packed=False)
    out = run(p, d)
    assert torch.equal(out["S_T"], d["S0"]) and torch.equal(out["dS0"], d["dST"])
    assert all(bool((out[k] == 0).all()) for k in ("da_log", "ddt_bias", "dd_skip"))
    q = G.make_ssm_problem(0, 0, 1, 2, 32, 32, a_log=d["a_log"])
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    y, ST, sv = G.ssm_forward(q, e(0, 64), e(0, 32), e(0, 32), torch.empty(0, 2, device="cuda"))
    g = G.ssm_backward(q, e(0, 64), e(0, 32), e(0, 32), torch.empty(0, 2, device="cuda"), None, sv, e(0, 64))
    assert y.shape[0] == 0 and ST.shape[0] == 0 and bool((g["da_log"] == 0).all())


def test_scan_offsets_past_32_bits():
    """Sequences behind nine million rows of none: rows, gradients and steps past 2^32 bytes."""
    import torch
    import gated_delta_rule_34_amd as G

    T, width = 9_000_000, 128
    a, up, cu = make([100, 64], 1, 2, 16, 16, "f32", seed=29)
    first = T - cu[-1]
    rows = torch.empty(2, T, width, device="cuda")  # inputs (x, b, c, dy) and outputs (dx, db, dc, y)
    cols = dict(x=(0, 32), b=(32, 16), c=(48, 16), dy=(64, 32))
    d = {k: rows[0, :, at:at + n] for k, (at, n) in cols.items()}
    outs = {k: rows[1, :, at:at + n] for k, (at, n) in zip(("dx", "db", "dc", "y"), cols.values())}
    for k in d:
        src = up["dy"] if k == "dy" else a[k]
        d[k][first:] = dev(src.reshape(cu[-1], cols[k][1]), "f32")
    dt = torch.empty(T, 2, device="cuda")
    dt[first:] = dev(a["dt"])
    p = G.make_ssm_problem(2, T, 1, 2, 16, 16, a_log=(al := dev(a["a_log"])), dt_bias=dev(a["dt_bias"]), d_skip=dev(a["d_skip"]),
                           cu_seqlens=torch.tensor([first + c for c in cu], dtype=torch.int32, device="cuda"), dtype="f32")
    y, ST, sv = G.ssm_forward(p, d["x"], d["b"], d["c"], dt, dev(a["S0"]), y=outs["y"])
    g = dict(dx=outs["dx"], db=outs["db"], dc=outs["dc"], ddt=torch.empty_like(dt), da_log=torch.empty_like(al),
             ddt_bias=torch.empty_like(al), dd_skip=torch.empty_like(al), dS0=torch.empty_like(ST))
    G.ssm_backward(p, d["x"], d["b"], d["c"], dt, None, sv, d["dy"], dev(up["dST"]), grads=g)
    out = dict(g, y=y, S_T=ST)
    for k in ("y", "dx", "db", "dc", "ddt"):
        out[k] = out[k][first:]
    check(a, up, cu, "f32", out)


@pytest.mark.parametrize("Dk,Dv", [(16, 16), (32, 128), (64, 32), (128, 64)])
@pytest.mark.parametrize("lens", [[130, 70], [1500]])
def test_scan_rows_carry_no_rounding_but_their_own(Dk, Dv, lens):
    """Every element of y and dx in bfloat16, where a carried state dominates and terms cancel: half a step of
    the row's type, and the operands' remainder. The state and the weights between tokens enter as two bfloat16
    terms, which leave at most 2^-8 of 2^-8 of each; the sums of float32 products and the decays add some 2^-17:
    together below 2^-15 of the sum of the terms' sizes."""
    from oracle import layer as L

    a, up, cu = make(lens, 1, 3, Dk, Dv, "bf16", seed=Dk + len(lens), skip=False, a_log=-3.0)
    out = run(*place(a, up, cu, "bf16"))
    size = {k: v if k in ("dt", "a_log", "dt_bias") or v is None else np.abs(v) for k, v in a.items()}
    absup = [np.abs(up["dy"]), np.abs(up["dST"])]
    for k, want, most in (("y", L.ssm_fwd(cu, *a.values())[0], L.ssm_fwd(cu, *size.values())[0]),
                          ("dx", L.ssm_bwd(cu, *a.values(), up["dy"], up["dST"])["dx"], L.ssm_bwd(cu, *size.values(), *absup)["dx"])):
        off = np.abs(host(out[k]).reshape(want.shape) - want) / (2.0 ** -8 * np.abs(want) + 2.0 ** -15 * most + 1e-30)
        assert off.max() <= 1, (k, float(off.max()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64)])
def test_scan_gradients_of_many_heads_in_one_workgroup(dtype, Dk, Dv):
    """Two groups of nine heads over more chunks than half the compute units: a workgroup's heads come in a second
    batch (float32: in five), with one and two slabs of a head."""
    lens = [70, 0, 1, 2] + [1, 0, 2] * 21
    a, up, cu = make(lens, 2, 18, Dk, Dv, dtype, seed=Dk)
    check(a, up, cu, dtype, run(*place(a, up, cu, dtype)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,T,Hk,r", [(9, 70, 4, 5), (5, 700, 2, 2)])
def test_scan_groups_dealt_to_one_xcd(dtype, N, T, Hk, r):
    """Groups whose heads go to one XCD, their number no multiple of eight; sequences whole, and in segments."""
    a, up, cu = make([T] * N, Hk, Hk * r, 16, 16, dtype, seed=T)
    check(a, up, cu, dtype, run(*place(a, up, cu, dtype, varlen=False, lens=[T])))


# ------------------------------------------------------------------------------------ single tokens


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Dk,Dv", [(16, 16), (16, 128), (32, 64), (64, 32), (128, 16), (128, 64), (128, 128)])
def test_decode_against_oracle(dtype, Dk, Dv):
    """Slots in no order, two rows skipped (their rows and every other state keep their bits)."""
    import torch
    import gated_delta_rule_34_amd as G
    from oracle import layer as L

    N, slots = 13, 17
    a, up, cu = make([1] * N, 2, 6, Dk, Dv, dtype, seed=Dk * 3 + Dv)
    rng = np.random.default_rng(1)
    pool = rounded(rng.standard_normal((slots, 6, Dk, Dv)), "f32")
    idx = rng.permutation(slots)[:N]
    use = idx.copy()
    use[3], use[8] = -1, slots
    _, d = place(a, up, cu, dtype)
    p = G.make_ssm_problem(N, N, 2, 6, Dk, Dv, T=1, a_log=d["a_log"], dt_bias=d["dt_bias"], d_skip=d["d_skip"], dtype=dtype)
    state = dev(pool)
    y = torch.full((N, 6 * Dv), 7.0, dtype=torch_dtype(dtype), device="cuda")
    G.gdn_ssm_decode(p, d["x"], d["b"], d["c"], d["dt"], state, torch.from_numpy(use.astype(np.int32)).cuda(), y)
    a["S0"] = pool[idx]
    yr, STr = L.ssm_fwd(cu, *a.values())
    live = [i for i in range(N) if i not in (3, 8)]
    assert rel(host(y)[live], yr[live]) <= (2.0 ** -8 if dtype == "bf16" else 1e-5)
    assert bool((y[[3, 8]] == 7.0).all())
    assert rel(host(state)[idx[live]], STr[live]) <= 1e-5
    rest = [s for s in range(slots) if s not in set(idx[live])]
    assert np.array_equal(host(state)[rest], pool[rest])


def test_decode_continues_a_prompt():
    """A prompt of 70 tokens, then 5 single tokens, is the prompt of 75."""
    import torch
    import gated_delta_rule_34_amd as G

    a, up, cu = make([75, 75], 1, 3, 64, 64, "f32", seed=23)
    p, d = place(a, up, cu, "f32", packed=False)
    whole = run(p, d, backward=False)
    rows = [list(range(0, 70)) + list(range(75, 145))] + [[70 + t, 145 + t] for t in range(5)]
    kw = dict(a_log=d["a_log"], dt_bias=d["dt_bias"], d_skip=d["d_skip"], dtype="f32")
    take = lambda i: [d[k][rows[i]] for k in ("x", "b", "c", "dt")]
    y, state, _ = G.ssm_forward(G.make_ssm_problem(2, 140, 1, 3, 64, 64, T=70, **kw), *take(0), d["S0"], save=False)
    assert rel(host(y), host(whole["y"][rows[0]])) <= 1e-6
    for t in range(1, 6):
        y = torch.empty(2, 3 * 64, device="cuda")
        G.gdn_ssm_decode(G.make_ssm_problem(2, 2, 1, 3, 64, 64, T=1, **kw), *take(t), state, None, y)
        assert rel(host(y), host(whole["y"][rows[t]])) <= 1e-5
    assert rel(host(state), host(whole["S_T"])) <= 1e-5


def test_decode_slots_past_32_bits():
    """A pool of 1100 slots of 4 MiB: the last slot's state is behind 2^32 bytes."""
    import torch
    import gated_delta_rule_34_amd as G

    a, up, cu = make([1, 1], 1, 64, 128, 128, "bf16", seed=31)
    _, d = place(a, up, cu, "bf16")
    p = G.make_ssm_problem(2, 2, 1, 64, 128, 128, T=1, a_log=d["a_log"], dt_bias=d["dt_bias"], d_skip=d["d_skip"], dtype="bf16")
    pool, small = torch.empty(1100, 64, 128, 128, device="cuda"), d["S0"].clone()
    idx = torch.tensor([1099, 3], dtype=torch.int32, device="cuda")
    pool[idx.long()] = small
    y, want = (torch.empty(2, 64 * 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    G.gdn_ssm_decode(p, d["x"], d["b"], d["c"], d["dt"], pool, idx, y)
    G.gdn_ssm_decode(p, d["x"], d["b"], d["c"], d["dt"], small, None, want)
    assert torch.equal(y, want) and torch.equal(pool[idx.long()], small)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_in_place_of_x(dtype):
    """y as the very view of x, inside a packed row beside b and c."""
    import torch
    import gated_delta_rule_34_amd as G

    a, up, cu = make([1] * 5, 2, 6, 64, 128, dtype, seed=33)
    p, d = place(a, up, cu, dtype, varlen=False, lens=[1])
    state, y = d["S0"].clone(), torch.empty(5, 6 * 128, dtype=torch_dtype(dtype), device="cuda")
    G.gdn_ssm_decode(p, d["x"], d["b"], d["c"], d["dt"], state, None, y)
    G.gdn_ssm_decode(p, d["x"], d["b"], d["c"], d["dt"], d["S0"], None, d["x"])
    assert torch.equal(d["x"], y) and torch.equal(d["S0"], state)
