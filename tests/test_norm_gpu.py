"""GPU: the gated RMS norm and the residual addition with its norm, forward and backward, against the
float64 oracle.

Tolerances. Row outputs, per element: half a step of the type, plus float32 roundings: a norm's
sum of squares carries at most some 32 2^-24 relative (partial sums of 8 to 64 values in a tree),
its root and the factors some 8 more, the backward's difference of two terms the same of each term:
64 2^-24 of the terms' size. What is below the smallest normal float32, 2^-126, may come out as 0
(the gate of -100 is 100 e^-100 = 4e-42). Sums over rows (dw, ds): 64 2^-24 of the sum of the terms' sizes."""
import numpy as np
import pytest

from layer_gpu import HALF, dev, host, rounded, torch_dtype

pytestmark = pytest.mark.gpu
U = 64 * 2.0 ** -24
WIDTHS = [8, 16, 24, 128, 136, 512, 520, 1024, 2048, 2056, 4096, 6144, 6152, 9000, 12296, 16384]


def near(got, want, size, dtype):
    tol = HALF[dtype] * (np.abs(want) + U * size) + U * size + 2.0 ** -126
    assert got.shape == want.shape and (np.abs(got - want) <= tol).all(), float(np.max(np.abs(got - want) / tol))


def view(a, dtype, pad=8):
    """a [rows, cols] as a view of wider rows, NaN around it."""
    import torch

    wide = torch.full((a.shape[0], a.shape[1] + 2 * pad), float("nan"), dtype=torch_dtype(dtype), device="cuda")
    wide[:, pad:pad + a.shape[1]] = dev(a, dtype)
    return wide[:, pad:pad + a.shape[1]]


def gate_case(rows, groups, W, shared, dtype, seed):
    rng = np.random.default_rng(seed)
    x, z, dy = (rounded(rng.standard_normal((rows, groups, W)), dtype) for _ in range(3))
    w = rounded(1 + 0.3 * rng.standard_normal((1 if shared else groups, W)), "f32")
    return x, z, w, dy


def gate_run(x, z, w, dy, shared, gate_first, dtype, eps=1e-5):
    import gated_delta_rule_34_amd as G

    rows, groups, W = x.shape
    p = G.make_norm_problem(rows, W, groups=groups, shared=shared, eps=eps, gate_first=gate_first, dtype=dtype)
    f = lambda a: view(a.reshape(rows, -1), dtype)
    y = G.gated_norm_forward(p, f(x), f(z), dev(w))
    g = G.gated_norm_backward(p, f(x), f(z), dev(w), f(dy))
    return y, g


def gate_check(x, z, w, dy, shared, gate_first, dtype, eps=1e-5):
    from oracle import layer as L

    y, g = gate_run(x, z, w, dy, shared, gate_first, dtype, eps)
    shape = x.shape
    s = 1 / (1 + np.exp(-z))
    gate = np.abs(z * s)
    v = x * z * s if gate_first else x
    rs = L._rms(v, eps)
    n = np.abs(v * rs)
    near(host(y).reshape(shape), L.gated_norm(x, z, w, eps, gate_first), n * np.abs(w) * (1 if gate_first else gate), dtype)
    dx, dz, dw = L.gated_norm_bwd(x, z, w, eps, gate_first, dy)
    dn = np.abs(dy) * (1 if gate_first else gate)
    t = dn * np.abs(w)
    dv = rs * (t + n * (t * n).mean(-1, keepdims=True))  # sizes of the terms
    dg = s * (1 + np.abs(z) * (1 - s))
    near(host(g["dx"]).reshape(shape), dx, dv * (gate if gate_first else 1), dtype)
    near(host(g["dz"]).reshape(shape), dz, (dv * np.abs(x) if gate_first else np.abs(dy) * n * np.abs(w)) * dg, dtype)
    size = (dn * n).sum(0)
    if shared:
        dw, size = dw.sum(0, keepdims=True), size.sum(0, keepdims=True)
    near(host(g["dw"]).reshape(dw.shape), dw, size, "f32")


@pytest.mark.parametrize("W", WIDTHS)
@pytest.mark.parametrize("dtype,gate_first", [("bf16", False), ("f32", True)])
def test_gated_norm_widths(W, dtype, gate_first):
    gate_check(*gate_case(5, 2, W, False, dtype, W), False, gate_first, dtype)


@pytest.mark.parametrize("rows,groups,W", [(1, 1, 128), (3, 48, 128), (700, 3, 64), (70, 5, 1000), (1025, 1, 8), (9, 300, 8), (600, 2, 2056)])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("dtype,gate_first", [("bf16", True), ("f32", False)])
def test_gated_norm_layouts(rows, groups, W, shared, dtype, gate_first):
    """One row, rows and groups that fill no workgroup, more rows than workgroups, weights shared or not."""
    gate_check(*gate_case(rows, groups, W, shared, dtype, rows + W), shared, gate_first, dtype)


def test_gated_norm_zero_rows_and_large_gates():
    """A zero row (the epsilon alone), gates of +-100 and of 0."""
    x, z, w, dy = gate_case(6, 2, 64, False, "f32", 1)
    x[0] = 0
    z[1], z[2], z[3] = 100, -100, 0
    for gate_first in (False, True):
        gate_check(x, z, w, dy, False, gate_first, "f32")


def test_gated_norm_in_place_and_no_rows():
    import torch
    import gated_delta_rule_34_amd as G

    x, z, w, dy = (dev(a.reshape(a.shape[0], -1), t) for a, t in zip(gate_case(40, 4, 72, False, "bf16", 2), ("bf16", "bf16", "f32", "bf16")))
    p = G.make_norm_problem(40, 72, groups=4)
    y = G.gated_norm_forward(p, x, z, w.view(-1))
    g = G.gated_norm_backward(p, x, z, w.view(-1), dy)
    x2, z2 = x.clone(), z.clone()
    G.gdn_gated_norm_bwd(p, x2, z2, w.view(-1), dy, x2, z2, None, None)
    assert torch.equal(x2, g["dx"]) and torch.equal(z2, g["dz"])
    x3 = x.clone()
    G.gdn_gated_norm_fwd(p, x3, z, w.view(-1), x3)
    assert torch.equal(x3, y)
    q = G.make_norm_problem(0, 72, groups=4)
    e = x[:0]
    assert G.gated_norm_forward(q, e, e, w.view(-1)).shape == (0, 288)
    assert bool((G.gated_norm_backward(q, e, e, w.view(-1), e)["dw"] == 0).all())


def add_check(rows, W, dtype, vector, with_dres, seed, scale=0.7, eps=1e-5):
    import torch
    import gated_delta_rule_34_amd as G
    from oracle import layer as L

    rng = np.random.default_rng(seed)
    h, y, dout, dres = (rounded(rng.standard_normal((rows, W)), dtype) for _ in range(4))
    s = rounded(rng.standard_normal(W), "f32") if vector else None
    w = rounded(1 + 0.3 * rng.standard_normal(W), "f32")
    p = G.make_norm_problem(rows, W, eps=eps, scale=scale, dtype=dtype)
    scale = float(np.float32(scale))
    f = scale * (np.ones(W) if s is None else s)
    th, ty = view(h, dtype), view(y, dtype)
    res, out = G.add_norm_forward(p, th, ty, dev(s), dev(w))
    near(host(res), h + f * y, np.abs(h) + np.abs(f * y), dtype)
    r64 = host(res)  # the norm is of the stored residual
    n = r64 * L._rms(r64, eps)
    near(host(out), n * w, np.abs(n * w), dtype)
    dr = view(dres, dtype) if with_dres else None
    g = G.add_norm_backward(p, res, ty, dev(s), dev(w), view(dout, dtype), dr)
    dh, dy, dw, ds = L.add_norm_bwd(r64, y, f, w, eps, dout, dres if with_dres else None, scale)
    t, na = np.abs(dout * w), np.abs(n)
    size = L._rms(r64, eps) * (t + na * (t * na).mean(-1, keepdims=True)) + (np.abs(dres) if with_dres else 0)
    near(host(g["dh"]), dh, size, dtype)
    near(host(g["dy"]), dy, size * np.abs(f), dtype)
    near(host(g["dw"]), dw, np.abs(dout * n).sum(0), "f32")
    assert ("ds" in g) == vector
    if vector:
        near(host(g["ds"]), ds, scale * (size * np.abs(y)).sum(0), "f32")
    # in place, and without what nobody asks for
    th2 = th.clone()
    out2 = torch.empty_like(out)
    G.gdn_add_norm_fwd(p, th2, ty, dev(s), dev(w), th2, out2)
    assert torch.equal(th2, res) and torch.equal(out2, out)
    dh2 = torch.empty_like(g["dh"]) if dr is None else dr.contiguous()
    G.gdn_add_norm_bwd(p, res, None, dev(s), dev(w), dev(dout, dtype), None if dr is None else dh2, dh2, None, None, None, None)
    assert torch.equal(dh2, g["dh"])


@pytest.mark.parametrize("W", WIDTHS)
@pytest.mark.parametrize("dtype,vector", [("bf16", True), ("f32", False)])
def test_add_norm_widths(W, dtype, vector):
    add_check(7, W, dtype, vector, True, W)


@pytest.mark.parametrize("rows", [1, 3, 513, 2100])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_add_norm_rows(rows, dtype):
    add_check(rows, 520, dtype, True, False, rows)
    add_check(rows, 40, dtype, False, True, rows)


def test_norms_offsets_past_32_bits():
    import torch
    import gated_delta_rule_34_amd as G

    rows, wide = 55000, 40000
    big = torch.ones(rows, wide, dtype=torch.bfloat16, device="cuda")
    big[-9:, :128] = torch.randn(9, 128, device="cuda")
    w = torch.ones(64, device="cuda")
    p, q = G.make_norm_problem(rows, 64), G.make_norm_problem(9, 64)
    y, y9 = G.gated_norm_forward(p, big[:, :64], big[:, 64:128], w), G.gated_norm_forward(q, big[-9:, :64], big[-9:, 64:128], w)
    assert torch.equal(y[-9:], y9)


def test_norm_graph_replays():
    import torch
    import gated_delta_rule_34_amd as G

    x, z, w, dy = gate_case(300, 3, 128, True, "bf16", 8)
    f = lambda a, t="bf16": dev(a.reshape(-1, a.shape[-1] * (3 if t == "bf16" else 1)), t)
    x, z, dy, w = f(x), f(z), f(dy), dev(w).view(-1)
    p = G.make_norm_problem(300, 128, groups=3, shared=True)
    q = G.make_norm_problem(300, 384)
    wide = torch.ones(384, device="cuda")

    def step():
        out = dict(y=G.gated_norm_forward(p, x, z, w), **G.gated_norm_backward(p, x, z, w, dy))
        res, o = G.add_norm_forward(q, x, out["y"], wide, wide)
        out.update(res=res, o=o, **{"a" + k: v for k, v in G.add_norm_backward(q, res, out["y"], wide, wide, dy, z).items()})
        return out

    eager = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(3):
        for t in out.values():
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], eager[k]) for k in eager), rep
        step()


@pytest.mark.parametrize("rows,groups,W", [(2101, 48, 128), (5001, 3, 512), (1201, 1, 2568)])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("dtype,gate_first", [("bf16", False), ("f32", True)])
def test_gated_norm_several_rows_to_a_workgroup(rows, groups, W, shared, dtype, gate_first):
    """More passes than row splits: the weights' gradients add up over a workgroup's rows, and some workgroups
    have one row more than others."""
    gate_check(*gate_case(rows, groups, W, shared, dtype, rows + W), shared, gate_first, dtype)


@pytest.mark.parametrize("rows,W", [(9001, 520), (1201, 2568), (140001, 24)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_add_norm_several_rows_to_a_workgroup(rows, W, dtype):
    add_check(rows, W, dtype, True, True, rows)


def test_norms_nan_and_infinities_stay_in_their_groups():
    """A NaN or an infinity in a group reaches that group's values and the column sums, nothing else."""
    import torch
    import gated_delta_rule_34_amd as G

    for width, groups in ((64, 3), (2056, 2)):
        x, z, w, dy = (dev(a.reshape(a.shape[0], -1), t) for a, t in zip(gate_case(9, groups, width, False, "bf16", 6), ("bf16", "bf16", "f32", "bf16")))
        w = w.view(-1)
        p = G.make_norm_problem(9, width, groups=groups)
        run = lambda: dict(y=G.gated_norm_forward(p, x, z, w), **G.gated_norm_backward(p, x, z, w, dy))
        clean = run()
        x[1, 0], x[4, width], z[6, 2], dy[7, width + 1] = float("nan"), float("inf"), float("nan"), float("-inf")
        out = run()
        hit = torch.zeros(9, groups, dtype=torch.bool, device="cuda")
        hit[1, 0], hit[4, 1], hit[6, 0], hit[7, 1] = True, True, True, True
        for k in ("y", "dx", "dz"):
            a, b = (v[k].view(9, groups, width)[~hit] for v in (out, clean))
            assert torch.equal(a, b), k
        assert bool(out["y"].view(9, groups, width)[1, 0].isnan().all())
        q = G.make_norm_problem(9, width * groups)
        h, y = clean["y"].clone(), clean["dx"]
        wide = torch.ones(width * groups, device="cuda")
        res, o = G.add_norm_forward(q, h, y, wide, wide)
        g = G.add_norm_backward(q, res, y, wide, wide, dy.nan_to_num(0, 0, 0), None)
        h[3, 5] = float("inf")
        res2, o2 = G.add_norm_forward(q, h, y, wide, wide)
        g2 = G.add_norm_backward(q, res2, y, wide, wide, dy.nan_to_num(0, 0, 0), None)
        rest = [0, 1, 2, 4, 5, 6, 7, 8]
        for a, b in ((res, res2), (o, o2), (g["dh"], g2["dh"]), (g["dy"], g2["dy"])):
            assert torch.equal(a[rest], b[rest])

