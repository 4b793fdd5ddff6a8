"""GPU: the gated linear recurrence (prompts, gradients, single tokens) against the float64 oracle.

Tolerances. Every float32 step rounds by at most 2^-24 of its terms; a token's gate costs some 24 such
roundings (two sigmoids with the hardware's exponential and reciprocal for bfloat16 rows, whose argument of up to 6 in
the drawn gates counts once more per unit, 1 - a, w), a composition of maps 4, and a token's contribution
passes through at most as many gates as tokens lie behind it and a dozen compositions; h - e h rounds by 2^-24 of h. The
oracle's sizes sum absolute terms, counted once more for each later step, so 64 2^-24 of them bounds a float32 result; rows add half a step of
their type. dlambda: each term has such a size. Below 2^-126 a result may come out as 0. An exponent L below 2^-126
counts as 0 in float32, and w = sqrt(2 L) is then up to 2^-62.5 off: each token's u (and with a gradient, its du) may move
every result of its sequence and channel by 2^-62 of it at the most: 2^-62 times the sum of |u| and |h0| there, and for gradients
times the sum of |dy| and |dhT| (`tiny`)."""
import math

import numpy as np
import pytest
import torch  # noqa: F401  (in front of the package, which then has torch's HIP runtime)

from layer_gpu import HALF, cu_of, dev, host, rounded, torch_dtype

pytestmark = pytest.mark.gpu
U = 64 * 2.0 ** -24
RATE = 8.0


def near(got, want, size, half=0.0, what="", tiny=0.0):
    tol = half * (np.abs(want) + U * size) + U * size + 2.0 ** -126 + 2.0 ** -62 * tiny
    got = host(got)
    assert got.shape == want.shape, what
    off = np.abs(got - want) / tol
    assert (off <= 1).all(), (what, float(np.nanmax(off)), int(np.isnan(got).sum()))


def view(a, dtype, pad=8):
    """a [rows, cols] as a view of wider rows, NaN around it."""
    import torch

    wide = torch.full((a.shape[0], a.shape[1] + 2 * pad), float("nan"), dtype=torch_dtype(dtype), device="cuda")
    wide[:, pad:pad + a.shape[1]] = dev(a, dtype)
    return wide[:, pad:pad + a.shape[1]]


def case(lens, C, dtype, seed, init=True, fresh="some"):
    rng = np.random.default_rng(seed)
    T, N = sum(lens), len(lens)
    v = dict(cu=cu_of(lens), x=rounded(rng.standard_normal((T, C)), dtype), r=rounded(1.5 * rng.standard_normal((T, C)), dtype),
             i=rounded(1.5 * rng.standard_normal((T, C)), dtype),
             lam=rounded(np.log(np.expm1(-np.log(rng.uniform(0.9, 0.999, C)) / RATE)), "f32"), rate=RATE,
             h0=rounded(rng.standard_normal((N, C)), "f32") if init else None,
             fresh={"none": None, "all": np.ones(N), "some": np.arange(N) % 2}[fresh])
    g = dict(dy=rounded(rng.standard_normal((T, C)), dtype), dhT=rounded(rng.standard_normal((N, C)), "f32"))
    return v, g


def i32(a):
    import torch

    return None if a is None else torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def run(v, g, dtype, cu=True, pad=8):
    import gated_delta_rule_34_amd as G

    N, (T, C) = len(v["cu"]) - 1, v["x"].shape
    p = G.make_glr_problem(N, T, C, lam=dev(v["lam"]), rate=v["rate"], fresh=i32(v["fresh"]), cu_seqlens=i32(v["cu"]) if cu else None, dtype=dtype)
    x, r, i = (view(v[k], dtype, pad) for k in "xri")
    h0 = dev(v["h0"])
    y, hT, saved = G.glr_forward(p, x, r, i, h0, save=g is not None)
    if g is None:
        return dict(y=y, hT=hT)
    return dict(y=y, hT=hT, **G.glr_backward(p, x, r, i, saved, view(g["dy"], dtype, pad), dev(g["dhT"])))


def check(v, g, dtype, **kw):
    from oracle import hybrid as O

    out = run(v, g, dtype, **kw)
    names = [v[k] for k in ("cu", "x", "r", "i", "lam", "rate", "h0", "fresh")]
    size = O.glr_sizes(*names, *(() if g is None else g.values()))
    y, hT = O.glr_fwd(*names)
    tiny = np.abs(v["x"]).sum(0) + (0 if v["h0"] is None else np.abs(v["h0"]).sum(0))
    near(out["y"], y, size["y"], HALF[dtype], "y", tiny)
    near(out["hT"], hT, size["hT"], 0.0, "hT", tiny)
    if g is not None:
        want = O.glr_bwd(*names, *g.values())
        tiny = (1 + tiny) * (np.abs(g["dy"]).sum(0) + np.abs(g["dhT"]).sum(0))
        for k in ("dx", "dr", "di"):
            near(out[k], want[k], size[k], HALF[dtype], k, tiny)
        near(out["dlam"], want["dlam"], size["dlam"], 0.0, "dlam", tiny)
        near(out["dh0"], want["dh0"], size["dh0"], 0.0, "dh0", tiny)
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[1], [2, 1, 0, 3], [127, 128, 129], [0, 64, 0, 300, 1, 0], [515, 1, 130]])
@pytest.mark.parametrize("C", [8, 72, 256])
def test_against_oracle(dtype, lens, C):
    v, g = case(lens, C, dtype, 10 + C + len(lens))
    check(v, g, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("init,fresh", [(True, "none"), (True, "all"), (False, "none"), (False, "all"), (False, "some")])
def test_starts(dtype, init, fresh):
    v, g = case([5, 0, 140, 33], 40, dtype, 21, init, fresh)
    check(v, g, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_lengths_without_table(dtype):
    v, g = case([200, 200, 200], 136, dtype, 22)
    check(v, g, dtype, cu=False)


@pytest.mark.parametrize("dtype,lens,C,cu", [("bf16", [5000], 16, False), ("f32", [3000, 2999], 24, True), ("bf16", [40, 2600, 0, 1500, 511, 513], 72, True),
                                             ("f32", [9000, 30, 4400], 8, True)])
def test_sequences_cut_into_segments(dtype, lens, C, cu):
    import gated_delta_rule_34_amd as G
    import torch

    v, g = case(lens, C, dtype, 23)
    p = G.make_glr_problem(len(lens), sum(lens), C, lam=torch.zeros(C, device="cuda"), cu_seqlens=i32(v["cu"]) if cu else None, dtype=dtype)
    assert G.gdn_glr_fwd_workspace_bytes(p) > 0  # (several segments)
    check(v, g, dtype, cu=cu)


def test_many_sequences():
    """More than 256 of them, two long enough to be cut."""
    rng = np.random.default_rng(36)
    lens = [int(v) for v in rng.integers(0, 12, 300)]
    lens[40], lens[299] = 2100, 1500
    v, g = case(lens, 16, "f32", 37)
    check(v, g, "f32")


def test_forward_without_backward_and_parts_skipped():
    import torch
    import gated_delta_rule_34_amd as G

    v, g = case([300, 77], 64, "bf16", 24)
    both = run(v, g, "bf16")
    alone = run(v, None, "bf16")
    assert torch.equal(both["y"], alone["y"]) and torch.equal(both["hT"], alone["hT"])
    p = G.make_glr_problem(2, 377, 64, lam=dev(v["lam"]), fresh=i32(v["fresh"]), cu_seqlens=i32(v["cu"]))
    x, r, i, dy = (dev(a, "bf16") for a in (v["x"], v["r"], v["i"], g["dy"]))
    y, hT, saved = G.glr_forward(p, x, r, i, dev(v["h0"]), want_final=False)
    assert hT is None and torch.equal(y, both["y"])
    d = [torch.empty_like(x) for _ in range(3)]
    ws = torch.empty(G.gdn_glr_bwd_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    G.gdn_glr_bwd(p, x, r, i, saved, dy, dev(g["dhT"]), *d, None, None, ws)
    for a, k in zip(d, ("dx", "dr", "di")):
        assert torch.equal(a, both[k])
    want = run(v, dict(dy=g["dy"], dhT=np.zeros_like(g["dhT"])), "bf16")  # no gradient of the final state
    G.gdn_glr_bwd(p, x, r, i, saved, dy, None, *d, None, None, ws)
    for a, k in zip(d, ("dx", "dr", "di")):
        assert torch.equal(a, want[k])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(dtype):
    import torch
    import gated_delta_rule_34_amd as G

    v, g = case([700, 90], 72, dtype, 25)
    want = run(v, g, dtype)
    p = G.make_glr_problem(2, 790, 72, lam=dev(v["lam"]), fresh=i32(v["fresh"]), cu_seqlens=i32(v["cu"]), dtype=dtype)
    saved = G.glr_forward(p, *(dev(v[k], dtype) for k in "xri"), dev(v["h0"]))[2]
    for k in range(3):
        rows = [dev(v[n], dtype) for n in "xri"]
        G.glr_forward(p, *rows, dev(v["h0"]), y=rows[k], save=False)
        assert torch.equal(rows[k], want["y"])
    for order in ((0, 1, 2), (3, 0, 1), (2, 3, 0)):
        rows = [dev(v[n], dtype) for n in "xri"] + [dev(g["dy"], dtype)]
        out = [rows[k] for k in order]
        ws = torch.empty(G.gdn_glr_bwd_workspace_bytes(p), dtype=torch.uint8, device="cuda")
        G.gdn_glr_bwd(p, *rows[:3], saved, rows[3], dev(g["dhT"]), *out, None, None, ws)
        for a, n in zip(out, ("dx", "dr", "di")):
            assert torch.equal(a, want[n]), (order, n)


def test_long_memory_and_closed_gates():
    """Decays next to one (lambda -40: an exponent of 3e-17), next to zero, and gates of +-60 (a bfloat16 sigmoid's
    exponential is then some 60 2^-24 off, within the 64)."""
    rng = np.random.default_rng(26)
    for dtype in ("bf16", "f32"):
        v, g = case([400, 20], 32, dtype, 27)
        v["lam"] = rounded(np.repeat([-40.0, -12.0, 4.0, 30.0], 8), "f32")
        v["r"][rng.random(v["r"].shape) < 0.2] = 60.0
        v["r"][rng.random(v["r"].shape) < 0.2] = -60.0
        check(v, g, dtype)


def test_zero_exponents_are_finite():
    """No exponent at all (lambda -200, or a gate of -infinity): nothing enters, nothing is lost, no gradient of the gate;
    an exponent beyond float32 (rate 1e38): nothing is kept."""
    import torch

    v, g = case([50], 16, "f32", 28, fresh="none")
    v["lam"][:8] = -200.0
    v["r"][:, 8:] = -np.inf
    out = run(v, g, "f32")
    assert torch.equal(out["hT"], dev(v["h0"])) and all(bool(torch.isfinite(t).all()) for t in out.values())
    assert not out["dr"].any() and not out["dlam"].any()
    v, g = case([50], 16, "f32", 28, fresh="none")
    v.update(rate=1e38, lam=np.full(16, 5.0))
    out = run(v, g, "f32")
    u = v["x"] / (1 + np.exp(-v["i"]))
    assert np.allclose(host(out["y"]), u, rtol=1e-6) and all(bool(torch.isfinite(t).all()) for t in out.values())


def test_nan_stays_in_its_sequence_and_channel():
    import torch

    for lens in ([300, 200, 100], [3000, 40, 10]):
        v, g = case(lens, 24, "bf16", 29, fresh="none")
        clean = run(v, g, "bf16")
        t, c = lens[0] + 30, 5
        v["x"][t, c] = np.nan
        out = run(v, g, "bf16")
        hit = np.zeros((sum(lens), 24), bool)
        hit[t:lens[0] + lens[1], c] = True
        assert (np.isnan(host(out["y"])) == hit).all()
        for k in ("y", "dx", "di"):
            same = torch.from_numpy(~hit).cuda()
            assert torch.equal(out[k][same], clean[k][same]), k
        assert np.isnan(host(out["hT"])[1, 5]) and np.isnan(host(out["hT"])).sum() == 1


def test_a_fresh_sequences_start_is_not_read():
    import torch

    v, g = case([5, 200], 16, "bf16", 30, fresh="all")
    want = run(v, g, "bf16")
    v["h0"][:] = np.nan
    out = run(v, g, "bf16")
    assert all(torch.equal(out[k], want[k]) for k in want)


def test_rows_of_no_sequence_stay():
    """Rows in front of the first and behind the last offset are left as they were; a table that points past the rows
    or falls stays inside."""
    import torch
    import gated_delta_rule_34_amd as G

    for C, T in ((64, 300), (8, 5000)):
        x, r, i, dy = (torch.randn(T, C, device="cuda") for _ in range(4))
        lam = torch.zeros(C, device="cuda")
        for cu, touched in (([40, 100, T - 50], (40, T - 50)), ([0, T // 2, T * 4], None), ([0, T, 5], None), ([-7, T // 3, -9], None), ([0, T, 5, T, 0, T], None)):
            p = G.make_glr_problem(len(cu) - 1, T, C, lam=lam, cu_seqlens=i32(cu), dtype="f32")
            outs = [torch.full((T, C), 7.0, device="cuda") for _ in range(4)]
            saved = torch.zeros(G.gdn_glr_state_bytes(p), dtype=torch.uint8, device="cuda")
            ws = torch.zeros(max(G.gdn_glr_fwd_workspace_bytes(p), G.gdn_glr_bwd_workspace_bytes(p)), dtype=torch.uint8, device="cuda")
            G.gdn_glr_fwd(p, x, r, i, None, outs[0], torch.empty(p.N, C, device="cuda"), saved, ws)
            G.gdn_glr_bwd(p, x, r, i, saved, dy, None, *outs[1:], torch.empty(C, device="cuda"), torch.empty(p.N, C, device="cuda"), ws)
            torch.cuda.synchronize()
            if touched:
                for o in outs:
                    assert (o[:touched[0]] == 7).all() and (o[touched[1]:] == 7).all() and not (o[touched[0]:touched[1]] == 7).any()


def test_no_tokens():
    import torch
    import gated_delta_rule_34_amd as G

    x = torch.empty(0, 16, device="cuda")
    for N in (0, 3):
        p = G.make_glr_problem(N, 0, 16, lam=torch.zeros(16, device="cuda"), fresh=torch.tensor([0, 1, 0][:N], dtype=torch.int32, device="cuda"), dtype="f32")
        h0, dhT = torch.randn(N, 16, device="cuda"), torch.randn(N, 16, device="cuda")
        y, hT, saved = G.glr_forward(p, x, x, x, h0)
        g = G.glr_backward(p, x, x, x, saved, x, dhT)
        keep = torch.tensor([1, 0, 1][:N], device="cuda")[:, None]
        assert torch.equal(hT, h0 * keep) and torch.equal(g["dh0"], dhT * keep) and not g["dlam"].any()
        if N == 0:  # without a workspace
            dlam = torch.full((16,), 3.0, device="cuda")
            G.gdn_glr_bwd(p, x, x, x, None, x, None, x, x, x, dlam, None, None)
            assert not dlam.any()


def test_continued_prompt_and_tokens_follow_the_whole():
    """A prompt in two parts, then token by token, against the whole: the same recurrence up to its roundings."""
    import torch
    import gated_delta_rule_34_amd as G
    from oracle import hybrid as O

    for dtype in ("bf16", "f32"):
        v, _ = case([400], 40, dtype, 31, fresh="all")
        args = [v[k] for k in ("cu", "x", "r", "i", "lam", "rate", "h0", "fresh")]
        want, size = O.glr_fwd(*args)[0], O.glr_sizes(*args)["y"]
        x, r, i = (dev(v[k], dtype) for k in "xri")
        lam, one = dev(v["lam"]), torch.ones(1, dtype=torch.int32, device="cuda")
        part = lambda lo, hi, h, **kw: G.glr_forward(G.make_glr_problem(1, hi - lo, 40, lam=lam, dtype=dtype, **kw), x[lo:hi], r[lo:hi], i[lo:hi], h, save=False)
        ya, h, _ = part(0, 150, None, fresh=one)
        yb, h, _ = part(150, 370, h)
        state = torch.full((3, 40), float("nan"), device="cuda")
        state[2] = h[0]
        ys, p = [ya, yb], G.make_glr_problem(1, 1, 40, T=1, lam=lam, dtype=dtype)
        for t in range(370, 400):
            y = torch.empty(1, 40, dtype=x.dtype, device="cuda")
            G.gdn_glr_decode(p, x[t:t + 1], r[t:t + 1], i[t:t + 1], state, torch.tensor([2], dtype=torch.int32, device="cuda"), y)
            ys.append(y)
        near(torch.cat(ys), want, size, HALF[dtype])
        assert torch.isnan(state[:2]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,C", [(1, 8), (5, 520), (70, 72)])
def test_tokens(dtype, N, C):
    import torch
    import gated_delta_rule_34_amd as G
    from oracle import hybrid as O

    v, _ = case([1] * N, C, dtype, 32)
    rng = np.random.default_rng(33)
    pool = rounded(rng.standard_normal((N + 6, C)), "f32")
    slots = rng.permutation(N + 6)[:N]
    if N > 2:
        slots[1], slots[2] = -1, N + 6
    want, after = O.glr_step(v["x"], v["r"], v["i"], v["lam"], RATE, pool, slots, v["fresh"])
    p = G.make_glr_problem(N, N, C, T=1, lam=dev(v["lam"]), fresh=i32(v["fresh"]), dtype=dtype)
    state, y = dev(pool), torch.full((N, C + 16), 5.0, dtype=torch_dtype(dtype), device="cuda")[:, 8:8 + C]
    G.gdn_glr_decode(p, view(v["x"], dtype), view(v["r"], dtype), view(v["i"], dtype), state, i32(slots), y)
    skipped = np.isnan(want[:, 0])
    size = 4 * np.abs(pool).max() + 4 * np.abs(v["x"])
    assert (host(y)[skipped] == 5).all()
    near(y[torch.from_numpy(~skipped).cuda()], want[~skipped], size[~skipped], HALF[dtype])
    near(state, after, 4 * np.abs(pool).max() + 4 * np.abs(v["x"]).max() + 0 * after)
    untouched = [s for s in range(N + 6) if s not in set(slots)]
    assert (host(state)[untouched] == pool[untouched]).all()
    rows, state = [dev(v[k], dtype) for k in "xri"], dev(pool)  # in place, rows in order
    p2 = G.make_glr_problem(N, N, C, T=1, lam=dev(v["lam"]), fresh=i32(v["fresh"]), dtype=dtype)
    want = O.glr_step(v["x"], v["r"], v["i"], v["lam"], RATE, pool, range(N), v["fresh"])[0]
    G.gdn_glr_decode(p2, *rows, state, None, rows[1])
    near(rows[1], want, size, HALF[dtype])


def test_rows_past_2_31_bytes_and_elements():
    """Rows 2^20 elements apart: offsets pass 2^31 elements."""
    import torch
    import gated_delta_rule_34_amd as G

    T, C, wide = 2200, 64, 1 << 20
    v, g = case([900, 1300], C, "bf16", 34)
    buf = torch.empty(T, wide, dtype=torch.bfloat16, device="cuda")
    at = lambda k: buf[:, wide - (k + 1) * C: wide - k * C]
    names = ("x", "r", "i")
    for k, n in enumerate(names):
        at(k).copy_(dev(v[n], "bf16"))
    at(3).copy_(dev(g["dy"], "bf16"))
    p = G.make_glr_problem(2, T, C, lam=dev(v["lam"]), fresh=i32(v["fresh"]), cu_seqlens=i32(v["cu"]))
    y, hT, saved = G.glr_forward(p, at(0), at(1), at(2), dev(v["h0"]), y=at(4))
    ws = torch.empty(G.gdn_glr_bwd_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    G.gdn_glr_bwd(p, at(0), at(1), at(2), saved, at(3), dev(g["dhT"]), at(5), at(6), at(7), None, None, ws)
    want = run(v, g, "bf16")
    for k, n in ((4, "y"), (5, "dx"), (6, "dr"), (7, "di")):
        assert torch.equal(at(k), want[n]), n
    assert torch.equal(hT, want["hT"])


def test_same_bits_twice_on_streams_and_replayed():
    """Two runs, a run on another stream, and a captured forward and backward replayed between eager ones."""
    import torch
    import gated_delta_rule_34_amd as G

    v, g = case([1500, 0, 700, 64], 72, "bf16", 35)
    want = run(v, g, "bf16")
    again = run(v, g, "bf16")
    assert all(torch.equal(want[k], again[k]) for k in want)
    N, T, C = 4, 2264, 72
    p = G.make_glr_problem(N, T, C, lam=dev(v["lam"]), fresh=i32(v["fresh"]), cu_seqlens=i32(v["cu"]))
    x, r, i, dy = (dev(a, "bf16") for a in (v["x"], v["r"], v["i"], g["dy"]))
    h0, dhT = dev(v["h0"]), dev(g["dhT"])
    rows = [torch.empty_like(x) for _ in range(4)]
    f32 = [torch.empty(N, C, device="cuda"), torch.empty(C, device="cuda"), torch.empty(N, C, device="cuda")]
    saved = torch.empty(G.gdn_glr_state_bytes(p), dtype=torch.uint8, device="cuda")
    ws = torch.empty(max(G.gdn_glr_fwd_workspace_bytes(p), G.gdn_glr_bwd_workspace_bytes(p)), dtype=torch.uint8, device="cuda")

    def step():
        G.gdn_glr_fwd(p, x, r, i, h0, rows[0], f32[0], saved, ws)
        G.gdn_glr_bwd(p, x, r, i, saved, dy, dhT, *rows[1:], *f32[1:], ws)

    names = ("y", "dx", "dr", "di", "hT", "dlam", "dh0")

    def equal():
        torch.cuda.synchronize()
        for t, n in zip(rows + f32, names):
            assert torch.equal(t, want[n]), n
            t.fill_(float("nan"))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    equal()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        graph.replay()
        equal()
        step()
        equal()
