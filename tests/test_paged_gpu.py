"""GPU: attention of one new token over a paged cache against the float64 oracle.

Tolerances, per element: half a step of the type, plus what float32 moves the weights by. A score of D terms, and its
product with the scale, is off by at most (D + 4) 2^-24 of the sum of its absolute terms (`dot`), the exponential's
argument by 4 2^-24 of the largest |score| (`top`, in both units), the exponential and each sum's terms by a few more: a weight is off by
w = (2 (D + 4) dot + 8 top + 64) 2^-24 of itself, and so is the output, of the sum of the weights times |v|; lse
by w, and by its own rounding."""
import math

import numpy as np
import pytest
import torch  # noqa: F401  (in front of the package, which then has torch's HIP runtime)

from layer_gpu import HALF, dev, host, rounded, torch_dtype
from test_glr_gpu import i32, view

pytestmark = pytest.mark.gpu


def case(lens, Hq, Hk, D, page, dtype, seed, extra=3, width=None, scale=1.5):
    rng = np.random.default_rng(seed)
    N, used = len(lens), [-(-max(0, n) // page) for n in lens]
    pages = sum(used) + extra
    width = max(max(used), 1) if width is None else width
    order, at = rng.permutation(pages), 0
    table = rng.integers(0, pages, (N, width))  # entries behind a length point anywhere
    for n, u in enumerate(used):
        table[n, :u] = order[at:at + u]
        at += u
    return dict(q=rounded(scale * rng.standard_normal((N, Hq, D)), dtype), k=rounded(rng.standard_normal((pages, Hk, page, D)), dtype),
                v=rounded(rng.standard_normal((pages, Hk, page, D)), dtype), table=table, lens=np.array(lens), page=page)


def run(c, dtype, poison=True, **kw):
    """out and lse; NaN in every place of the pool that no sequence holds."""
    import torch
    import gated_delta_rule_34_amd as G

    N, Hq, D = c["q"].shape
    Hk, page = c["k"].shape[1], c["page"]
    kp, vp = dev(c["k"], dtype), dev(c["v"], dtype)
    if poison:
        held = np.zeros((len(c["k"]), page), bool)
        for n in range(N):
            for t in range(max(0, min(int(c["lens"][n]), c["table"].shape[1] * page))):
                if 0 <= c["table"][n][t // page] < len(held):
                    held[c["table"][n][t // page], t % page] = True
        free = torch.from_numpy(~held).cuda()
        for t in (kp, vp):
            t.permute(0, 2, 1, 3)[free] = float("nan")
    p = G.make_paged_problem(i32(c["table"]), i32(c["lens"]), Hq, Hk, D, page_size=page, dtype=dtype, **kw)
    q = view(c["q"].reshape(N, -1), dtype)
    out, lse = G.paged_attention(p, q, kp, vp, want_lse=True)
    bits = torch.int16 if dtype == "bf16" else torch.int32  # (NaN are equal too)
    assert torch.equal(G.paged_attention(p, q, kp, vp)[0].view(bits), out.view(bits))
    return out.view(N, Hq, D), lse, p


def check(c, dtype, window=0, scale=None, max_len=None, **kw):
    from oracle import hybrid as O

    out, lse, p = run(c, dtype, window=window, scale=scale, max_len=max_len, **kw)
    D = c["q"].shape[2]
    want, wl, size, top, dot = O.paged(c["q"], c["k"], c["v"], c["table"], c["lens"], D ** -0.5 if scale is None else scale, window, max_len)
    w = (2 * (D + 4) * dot + 8 * top + 64) * 2.0 ** -24
    tol = HALF[dtype] * (np.abs(want) + w[..., None] * size) + w[..., None] * size + 2.0 ** -126
    got, gl = host(out), host(lse)
    off = np.abs(got - want) / tol
    assert (off <= 1).all(), float(np.nanmax(off))
    none = np.isinf(wl)
    assert (gl[none] == wl[none]).all() and (np.abs(gl[~none] - wl[~none]) <= (w[~none] + 2.0 ** -23 * np.abs(wl[~none]))).all()
    assert (got[none] == 0).all()
    return out, lse, p


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("page", [1, 8, 16, 24, 64])
def test_sizes(dtype, D, page):
    check(case([0, 1, 2, 15, 16, 17, 64, 65, 130, 300], 6, 2, D, page, dtype, D + page), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (7, 7), (4, 1), (10, 1), (16, 1), (17, 1), (24, 3), (40, 1), (64, 2)])
def test_heads(dtype, Hq, Hk):
    check(case([70, 1, 33], Hq, Hk, 64, 16, dtype, Hq + Hk), dtype)
    check(case([40, 9], Hq, Hk, 32, 5, dtype, Hq + Hk), dtype)


@pytest.mark.parametrize("dtype,D,page", [("bf16", 128, 16), ("bf16", 64, 7), ("f32", 64, 32), ("f32", 256, 24), ("bf16", 256, 48)])
def test_long_ones_are_split_and_joined(dtype, D, page):
    import gated_delta_rule_34_amd as G

    c = case([3000, 0, 257, 256, 1], 4, 2, D, page, dtype, D)
    _, _, p = check(c, dtype)
    assert G.gdn_paged_attn_workspace_bytes(p) > 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_chunk_or_several(dtype):
    """At the longest cache that one chunk takes, and one token behind it."""
    import gated_delta_rule_34_amd as G

    for D, most in ((64, 512), (256, 256)):
        for more in (0, 1):
            _, _, p = check(case([most + more, 3, most - 1], 3, 1, D, 1, dtype, D + more), dtype)
            assert (G.gdn_paged_attn_workspace_bytes(p) > 0) == bool(more)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences(dtype):
    """More than 256 of them: all of one chunk, and of several."""
    import gated_delta_rule_34_amd as G

    lens = [int(v) for v in np.random.default_rng(68).integers(0, 90, 300)]
    _, _, p = check(case(lens, 3, 1, 32, 16, dtype, 68), dtype)
    assert G.gdn_paged_attn_workspace_bytes(p) == 0
    lens[7], lens[299], lens[130] = 700, 650, 256
    c = case(lens, 3, 1, 32, 16, dtype, 69)
    _, _, p = check(c, dtype)
    assert G.gdn_paged_attn_workspace_bytes(p) > 0
    check(c, dtype, window=300)
    check(case(lens, 2, 2, 64, 20, dtype, 69), dtype)


@pytest.mark.parametrize("window", [1, 15, 16, 17, 100, 255, 512, 5000])
def test_window(window):
    for page in (16, 10):
        check(case([700, 99, 0, 1, 17], 4, 1, 64, page, "bf16", window), "bf16", window=window)


def test_bounds_of_lengths():
    """Lengths past the bound count as the bound, negative ones as nothing; a looser bound changes nothing but roundings."""
    c = case([300, 40, 170], 2, 1, 64, 16, "bf16", 70)
    check(c, "bf16", max_len=100)
    check({**c, "lens": np.array([10**9, -5, 170])}, "bf16", max_len=304, poison=False)
    wide = case([300, 40, 170], 2, 1, 64, 16, "bf16", 70, width=4000)
    check(wide, "bf16")


def test_pages_outside_the_pool_are_left_out():
    for page in (16, 12):
        c = case([200, 100, 30], 4, 2, 64, page, "bf16", 71)
        c["table"][0, 3], c["table"][0, 5], c["table"][1, 0] = -1, len(c["k"]), 2**31 - 1
        c["table"][2, :] = -7  # nothing is left
        check(c, "bf16")


def test_scores_far_apart():
    """Scores that grow along the sequence move the maximum again and again; equal ones, and ones so large that all but one weigh nothing."""
    for dtype in ("bf16", "f32"):
        c = case([900, 300], 3, 1, 64, 16, dtype, 72, scale=1.0)
        check(c, dtype, scale=8.0)
        ramp = np.linspace(-40, 40, 900)
        for t in range(900):
            c["k"][c["table"][0][t // 16], 0, t % 16] = rounded(np.full(64, ramp[t] / 8), dtype)
        c["q"][0] = rounded(np.full((3, 64), 1.0), dtype)
        check(c, dtype, scale=0.125)
        c["q"][:] = 0.0
        check(c, dtype)
        check(c, dtype, scale=0.0)


def test_infinite_scores():
    """Keys of minus infinity weigh nothing, like masked ones; where all are, nothing is left."""
    c = case([100, 40], 2, 1, 32, 16, "f32", 73)
    c["q"][:] = np.abs(c["q"])
    for t in range(20, 70):
        c["k"][c["table"][0][t // 16], 0, t % 16] = -np.inf
    for t in range(40):
        c["k"][c["table"][1][t // 16], 0, t % 16] = -np.inf
    out, lse, _ = run(c, "f32", poison=False)
    kept = {**c, "table": c["table"].copy()}
    keep = [t for t in range(100) if not 20 <= t < 70]
    k = np.stack([c["k"][c["table"][0][t // 16], 0, t % 16] for t in keep])
    v = np.stack([c["v"][c["table"][0][t // 16], 0, t % 16] for t in keep])
    z = c["q"][0] @ k.T / math.sqrt(32)
    e = np.exp(z - z.max(1, keepdims=True))
    assert np.allclose(host(out)[0], e @ v / e.sum(1, keepdims=True), atol=1e-5)
    assert (host(out)[1] == 0).all() and (host(lse)[1] == -np.inf).all()


def test_nan_stays_in_its_sequence_and_heads():
    import torch

    c = case([600, 300, 50], 8, 2, 64, 16, "bf16", 74)
    clean = run(c, "bf16", poison=False)[:2]
    c["k"][c["table"][1][3], 1, 5] = np.nan
    out, lse, _ = run(c, "bf16", poison=False)
    hit = torch.zeros(3, 8, dtype=torch.bool, device="cuda")
    hit[1, 4:] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])


def test_nothing():
    import torch
    import gated_delta_rule_34_amd as G

    none = torch.empty(0, 2, 16, 32, dtype=torch.bfloat16, device="cuda")
    for N, width in ((0, 4), (3, 4), (3, 0)):
        lens = torch.zeros(N, dtype=torch.int32, device="cuda")
        p = G.make_paged_problem(torch.zeros(N, width, dtype=torch.int32, device="cuda"), lens + 9, 4, 2, 32, page_size=16)
        out, lse = G.paged_attention(p, torch.randn(N, 128, device="cuda").bfloat16(), none, none, want_lse=True)
        assert out.shape == (N, 128) and not out.any() and bool((lse == -math.inf).all())


def test_cache_past_2_32_bytes():
    """Pages at both ends of a pool of 9 GB (keys and values each), pages of 16 and of 24 tokens."""
    import torch
    import gated_delta_rule_34_amd as G

    for page, pages in ((16, 1200000), (24, 800000)):
        c = case([500], 4, 4, 64, page, "bf16", 75)
        N = len(c["k"])
        kp, vp = (torch.empty(pages, 4, page, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        place = (np.arange(N) * 104729 + pages - 1) % pages
        place[0] = pages - 1
        assert len(set(place)) == N
        at = torch.from_numpy(place).cuda()
        kp[at], vp[at] = dev(c["k"], "bf16"), dev(c["v"], "bf16")
        small = run(c, "bf16", poison=False)[0]
        far = {**c, "table": place[c["table"]]}
        p = G.make_paged_problem(i32(far["table"]), i32(c["lens"]), 4, 4, 64, page_size=page)
        out, _ = G.paged_attention(p, dev(c["q"].reshape(1, -1), "bf16"), kp, vp)
        assert torch.equal(out.view(1, 4, 64), small)
        del kp, vp


def test_same_bits_twice_and_replayed_as_the_cache_grows():
    """A captured call reads lengths and tables anew at every replay; two graphs share a workspace in turn."""
    import torch
    import gated_delta_rule_34_amd as G

    c = case([2000, 900, 3], 8, 2, 64, 16, "bf16", 76)
    kp, vp, q = dev(c["k"], "bf16"), dev(c["v"], "bf16"), dev(c["q"].reshape(3, -1), "bf16")
    table, lens = i32(c["table"]), i32(c["lens"])
    p = G.make_paged_problem(table, lens, 8, 2, 64, page_size=16)
    p2 = G.make_paged_problem(table, lens, 8, 2, 64, page_size=16, window=700)
    ws = torch.empty(max(G.gdn_paged_attn_workspace_bytes(p), G.gdn_paged_attn_workspace_bytes(p2)), dtype=torch.uint8, device="cuda")
    out, out2 = torch.empty_like(q), torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        G.gdn_paged_attn_decode(p, q, kp, vp, out, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, G.paged_attention(p, q, kp, vp)[0])
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        G.gdn_paged_attn_decode(p, q, kp, vp, out, None, ws)
    with torch.cuda.graph(graphs[1]):
        G.gdn_paged_attn_decode(p2, q, kp, vp, out2, None, ws)
    for n in ([2000, 900, 3], [1, 0, 48], [1999, 901, 2]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        out.fill_(float("nan"))
        out2.fill_(float("nan"))
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(out, G.paged_attention(p, q, kp, vp)[0]) and torch.equal(out2, G.paged_attention(p2, q, kp, vp)[0])
