"""GPU: the norm of query and key heads with the rotation of positions, forward, gradients and into the pages of
a cache, against the float64 oracle.

Tolerances, per element: half a step of the type, plus float32 roundings of the terms' sizes: a sum of up to 256 squares
in a tree and its root some 32 2^-24, the weight, the cosine and sine (their series and the angle's rounding, 4
2^-24 of one) and the turn some 12 more, the backward's difference of two terms the same of each: 64 2^-24 of the sum of the
absolute terms. Sums over rows (dwq, dwk): 64 2^-24 of the sum of the terms' sizes."""
import numpy as np
import pytest
import torch  # noqa: F401  (in front of the package, which then has torch's HIP runtime)

from layer_gpu import HALF, dev, host, rounded, torch_dtype
from test_glr_gpu import i32, view

pytestmark = pytest.mark.gpu
U = 64 * 2.0 ** -24
EPS = 1e-5


def near(got, want, size, half, what=""):
    tol = half * (np.abs(want) + U * size) + U * size + 2.0 ** -126
    got = host(got).reshape(want.shape)
    off = np.abs(got - want) / tol
    assert (off <= 1).all(), (what, float(np.nanmax(off)))


def case(rows, Hq, Hk, D, dtype, seed, far=1 << 20):
    rng = np.random.default_rng(seed)
    v = {k: rounded(rng.standard_normal((rows, h, D)) * rng.uniform(0.1, 3, (rows, h, 1)), dtype)
         for k, h in (("q", Hq), ("k", Hk), ("v", Hk), ("dqo", Hq), ("dko", Hk))}
    v.update({w: rounded(1 + 0.3 * rng.standard_normal(D), "f32") for w in ("wq", "wk")})
    pos = rng.integers(0, far, rows)
    pos[: rows // 4] = [0, 1, far - 1, 2 ** 31 - 1, -3][: rows // 4] if rows // 4 <= 5 else pos[: rows // 4]
    v["pos"] = pos
    return v


def problem(v, R, adjacent, dtype, scale=1.0, weights=True):
    import torch
    import gated_delta_rule_34_amd as G

    (rows, Hq, D), Hk = v["q"].shape, v["k"].shape[1]
    freq = 10000.0 ** (-np.arange(0, R, 2) / max(R, 1))
    p = G.make_qk_rope_problem(rows, Hq, Hk, D, rot=R, adjacent=adjacent, positions=i32(v["pos"]), eps=EPS, rope_scale=scale, dtype=dtype,
                               freq=torch.from_numpy(freq).cuda() if R else None, wq=dev(v["wq"]) if weights else None, wk=dev(v["wk"]) if weights else None)
    return p, freq


def sizes(v, w, pos, freq, R, adjacent, scale):
    """Sum of the absolute terms of a normed and turned head."""
    from oracle import hybrid as O

    n = np.abs(v / np.sqrt(np.mean(v * v, -1, keepdims=True) + EPS) * w)
    return spread(n, R, adjacent, scale)


def spread(n, R, adjacent, scale):
    """|a| + |b| at both places of each pair."""
    from oracle import hybrid as O

    if R == 0:
        return n
    z = O._pairs(n, R, adjacent)
    s = abs(scale) * (z.real + z.imag)
    return O._flat(s + 1j * s, n[..., R:], adjacent)


def flat(a):
    return a.reshape(a.shape[0], -1)


def check(v, R, adjacent, dtype, scale=1.0, weights=True):
    import gated_delta_rule_34_amd as G
    from oracle import hybrid as O

    p, freq = problem(v, R, adjacent, dtype, scale, weights)
    q, k, dqo, dko = (view(flat(v[n]), dtype) for n in ("q", "k", "dqo", "dko"))
    outs = dict(zip(("q", "k"), G.qk_rope_forward(p, q, k)))
    g = G.qk_rope_backward(p, q, k, dqo, dko)
    for n in ("q", "k"):
        w = v["w" + n] if weights else np.ones(v["q"].shape[2])
        near(outs[n], O.norm_rope(v[n], w, v["pos"], freq, R, adjacent, EPS, scale), sizes(v[n], w, v["pos"], freq, R, adjacent, scale), HALF[dtype], n)
        dv, dw = O.norm_rope_bwd(v[n], w, v["pos"], freq, R, adjacent, EPS, v[f"d{n}o"], scale)
        rs = 1 / np.sqrt(np.mean(v[n] ** 2, -1, keepdims=True) + EPS)
        t, nn = spread(np.abs(v[f"d{n}o"]), R, adjacent, scale), np.abs(v[n] * rs)
        near(g["d" + n], dv, rs * (t * np.abs(w) + nn * np.mean(t * np.abs(w) * nn, -1, keepdims=True)), HALF[dtype], "d" + n)
        if weights:
            near(g["dw" + n], dw, (t * nn).sum((0, 1)), 0.0, "dw" + n)
        else:
            assert g["dw" + n] is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("D,R", [(16, 16), (16, 0), (32, 16), (48, 32), (64, 64), (80, 80), (96, 48), (128, 32), (128, 128), (192, 192), (256, 64), (256, 256)])
def test_against_oracle(dtype, adjacent, D, R):
    check(case(19, 5, 2, D, dtype, D + R), R, adjacent, dtype)


@pytest.mark.parametrize("rows", [1, 3, 4, 1030, 4099])
def test_rows(rows):
    check(case(rows, 3, 1, 64, "bf16", rows, far=5000), 32, False, "bf16")


def test_scale_and_no_weights():
    check(case(21, 2, 2, 64, "f32", 50), 64, False, "f32", scale=-1.5)
    check(case(21, 7, 1, 96, "bf16", 51), 96, True, "bf16", scale=0.5, weights=False)


def test_far_positions():
    """Angles of 2^31 turns' worth keep their places: float64 products, as the oracle's."""
    v = case(8, 1, 1, 32, "f32", 52)
    v["pos"] = np.array([2**31 - 1, -2**31, 2**30 + 1, 123456789, 7, -1, 0, 2**24 + 1])
    check(v, 32, False, "f32")


def test_in_place_and_zero_rows():
    import torch
    import gated_delta_rule_34_amd as G

    v = case(37, 4, 2, 128, "bf16", 53)
    p, _ = problem(v, 64, False, "bf16")
    new = lambda n: dev(flat(v[n]), "bf16")
    qo, ko = G.qk_rope_forward(p, new("q"), new("k"))
    q, k = new("q"), new("k")
    G.gdn_qk_rope_fwd(p, q, k, q, k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    g = G.qk_rope_backward(p, new("q"), new("k"), new("dqo"), new("dko"))
    for over_grad in (False, True):
        a = [new(n) for n in ("q", "k", "dqo", "dko")]
        out = a[2:] if over_grad else a[:2]
        G.gdn_qk_rope_bwd(p, *a, *out, None, None, None)
        assert torch.equal(out[0], g["dq"]) and torch.equal(out[1], g["dk"])
    only = torch.empty(128, device="cuda")  # one weight's gradient alone
    ws = torch.empty(G.gdn_qk_rope_bwd_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    G.gdn_qk_rope_bwd(p, new("q"), new("k"), new("dqo"), new("dko"), torch.empty_like(qo), torch.empty_like(ko), None, only, ws)
    assert torch.equal(only, g["dwk"])
    z = {n: a[:0] for n, a in v.items() if n not in ("wq", "wk")}
    p, _ = problem({**v, **z}, 64, False, "bf16")
    empty = lambda h: torch.empty(0, h * 128, dtype=torch.bfloat16, device="cuda")
    assert G.qk_rope_forward(p, empty(4), empty(2))[0].shape == (0, 512)
    g = G.qk_rope_backward(p, empty(4), empty(2), empty(4), empty(2))
    assert not g["dwq"].any() and not g["dwk"].any()


def test_zero_and_nonfinite_heads():
    """A head of zeros stays zero (epsilon 0: NaN, as 0 / 0); NaN and infinity stay in their head."""
    import torch
    import gated_delta_rule_34_amd as G

    v = case(6, 3, 2, 64, "f32", 54)
    v["q"][0, 1] = 0.0
    p, _ = problem(v, 32, False, "f32")
    new = lambda n: dev(flat(v[n]))
    clean = G.qk_rope_forward(p, new("q"), new("k")) + tuple(G.qk_rope_backward(p, new("q"), new("k"), new("dqo"), new("dko")).values())
    assert not clean[0].view(6, 3, 64)[0, 1].any()
    v["q"][2, 1, 5], v["k"][4, 0, 40], v["dqo"][5, 2, 3] = np.nan, np.inf, np.nan
    out = G.qk_rope_forward(p, new("q"), new("k")) + tuple(G.qk_rope_backward(p, new("q"), new("k"), new("dqo"), new("dko")).values())
    for a, b, H, bad in ((out[0], clean[0], 3, [(2, 1)]), (out[1], clean[1], 2, [(4, 0)]), (out[2], clean[2], 3, [(2, 1), (5, 2)]), (out[3], clean[3], 2, [(4, 0)])):
        a, b = a.view(6, H, 64), b.view(6, H, 64)
        for row in range(6):
            for h in range(H):
                assert ((row, h) in bad and not torch.isfinite(a[row, h]).all()) or torch.equal(a[row, h], b[row, h]), (row, h)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,Hq,Hk,D,R,page,pages", [(1, 1, 1, 16, 16, 1, 1), (13, 6, 3, 80, 32, 5, 4), (70, 4, 1, 256, 64, 16, 6), (4100, 2, 2, 64, 64, 24, 200)])
def test_into_pages(dtype, rows, Hq, Hk, D, R, page, pages):
    import torch
    import gated_delta_rule_34_amd as G

    v = case(rows, Hq, Hk, D, dtype, rows + D)
    rng = np.random.default_rng(rows)
    where = rng.permutation(page * pages)[:rows]
    if rows > 4:
        where[[1, 2, 3]] = [-1, page * pages, -2**31]  # not cached
    p, _ = problem(v, R, False, dtype)
    q, k, vv = (view(flat(v[n]), dtype) for n in ("q", "k", "v"))
    qo, ko = G.qk_rope_forward(p, q, k)
    kp, vp = (torch.full((pages, Hk, page, D), 9.0, dtype=torch_dtype(dtype), device="cuda") for _ in range(2))
    out = torch.empty_like(qo)
    G.gdn_qk_rope_cache(p, q, k, vv, out, kp, vp, i32(where))
    assert torch.equal(out, qo)
    wk, wv = torch.full_like(kp, 9.0), torch.full_like(vp, 9.0)
    ok = (where >= 0) & (where < page * pages)
    at, rows_ok = torch.from_numpy(where[ok]).cuda(), torch.from_numpy(np.flatnonzero(ok)).cuda()
    wk[at // page, :, at % page] = ko.view(rows, Hk, D)[rows_ok]
    wv[at // page, :, at % page] = dev(v["v"], dtype)[rows_ok]
    assert torch.equal(kp, wk) and torch.equal(vp, wv)  # the very keys of the other form, the values as they were


def test_pages_past_2_31_bytes():
    import torch
    import gated_delta_rule_34_amd as G

    v = case(6, 2, 2, 128, "bf16", 55)
    p, _ = problem(v, 128, False, "bf16")
    q, k, vv = (dev(flat(v[n]), "bf16") for n in ("q", "k", "v"))
    pages, page = 70000, 128  # 4.6 GB each
    kp, vp = (torch.empty(pages, 2, page, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    where = torch.tensor([0, pages * page - 1, 8388608, 8388607, 4194304, 5], dtype=torch.int32, device="cuda")
    qo, ko = G.qk_rope_forward(p, q, k)
    G.gdn_qk_rope_cache(p, q, k, vv, qo, kp, vp, where)
    at = where.long()
    assert torch.equal(kp[at // page, :, at % page], ko.view(6, 2, 128)) and torch.equal(vp[at // page, :, at % page], vv.view(6, 2, 128))


def test_same_bits_twice_and_replayed():
    import torch
    import gated_delta_rule_34_amd as G

    v = case(5000, 4, 2, 64, "bf16", 56, far=9000)
    p, _ = problem(v, 64, True, "bf16")
    new = lambda n: dev(flat(v[n]), "bf16")
    a = [new(n) for n in ("q", "k", "dqo", "dko")]
    want = list(G.qk_rope_forward(p, a[0], a[1])) + list(G.qk_rope_backward(p, *a).values())
    outs = [torch.empty_like(t) for t in want]
    ws = torch.empty(G.gdn_qk_rope_bwd_workspace_bytes(p), dtype=torch.uint8, device="cuda")

    def step():
        G.gdn_qk_rope_fwd(p, a[0], a[1], outs[0], outs[1])
        G.gdn_qk_rope_bwd(p, *a, *outs[2:], ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        if k:
            graph.replay()
        torch.cuda.synchronize()
        for t, w in zip(outs, want):
            assert torch.equal(t, w)
            t.fill_(float("nan"))
