"""GPU: the operators of a hybrid model's layers together, as they are used: a recurrent block (conv, gated linear
recurrence), the residual addition with its norm, an attention block (norm and rotation into the pages, attention over
them). Prompts in one call per operator, then tokens from a captured graph whose buffers are updated between replays;
and a training step through the same blocks. Each operator's outputs are held to the oracle's on the very inputs that it got
(so the tolerances are those of the operators' own tests). Then what the binding refuses."""
import numpy as np
import pytest
import torch  # noqa: F401  (in front of the package, which then has torch's HIP runtime)

from layer_gpu import dev, host, rounded
from test_glr_gpu import i32
from test_glr_gpu import near as near_glr

pytestmark = pytest.mark.gpu
C, Hq, Hk, D, R, PAGE, EPS, RATE = 64, 4, 2, 32, 16, 8, 1e-5, 8.0
U = 64 * 2.0 ** -24
QKV = (Hq + 2 * Hk) * D


class Model:
    """One recurrent and one attention block in float32, the projections by torch."""

    def __init__(self, seed):
        import torch

        rng = np.random.default_rng(seed)
        f = lambda *s, scale=1.0: dev(rounded(scale * rng.standard_normal(s), "f32"))
        self.conv_w, self.conv_b = f(C, 4, scale=0.4), f(C, scale=0.1)
        self.gates, self.qkv = f(C, 2 * C, scale=C ** -0.5 * 1.5), f(C, QKV, scale=C ** -0.5)
        self.lam = dev(rounded(np.log(np.expm1(-np.log(rng.uniform(0.9, 0.999, C)) / RATE)), "f32"))
        self.norm_w, self.wq, self.wk = (1 + 0.2 * f(n) for n in (C, D, D))
        self.freq = torch.from_numpy(1000.0 ** (-np.arange(0, R, 2) / R)).cuda()


def oracle_attention(m, q, kp, vp, table, lens, out, lse):
    from oracle import hybrid as O

    N = q.shape[0]
    want, wl, size, top, dot = O.paged(host(q).reshape(N, Hq, D), host(kp), host(vp), table.cpu().numpy(), lens.cpu().numpy(), D ** -0.5)
    w = (2 * (D + 4) * dot + 8 * top + 64) * 2.0 ** -24
    assert (np.abs(host(out).reshape(want.shape) - want) <= (w[..., None] + 2.0 ** -23) * (size + np.abs(want))).all()
    assert (np.abs(host(lse) - wl) <= w + 2.0 ** -23 * np.abs(wl)).all()


def oracle_rope(m, qkv, pos, qo, kp, vp, where):
    from oracle import hybrid as O

    rows = qkv.shape[0]
    q, k, v = np.split(host(qkv).reshape(rows, -1, D), [Hq, Hq + Hk], 1)
    freq = m.freq.cpu().numpy()
    tol = lambda x: 8 * U * (1 + np.abs(x).max())  # (a head's normed values add up pairwise: at most some three apart)
    want = O.norm_rope(q, host(m.wq), pos, freq, R, False, EPS)
    assert (np.abs(host(qo).reshape(want.shape) - want) <= tol(want)).all()
    want = O.norm_rope(k, host(m.wk), pos, freq, R, False, EPS)
    assert (np.abs(host(kp)[where // PAGE, :, where % PAGE] - want) <= tol(want)).all()
    assert (host(vp)[where // PAGE, :, where % PAGE] == v).all()


def test_prompts_then_tokens():
    import torch
    import gated_delta_rule_34_amd as G
    from oracle import hybrid as O

    m, lens, N = Model(1), [37, 1, 20], 3
    T, cu = sum(lens), np.concatenate([[0], np.cumsum(lens)])
    rng = np.random.default_rng(2)
    x = dev(rounded(rng.standard_normal((T, C)), "f32"))
    width, pages = 8, 30
    table = i32(rng.permutation(pages)[: N * width].reshape(N, width))
    kp, vp = (torch.zeros(pages, Hk, PAGE, D, device="cuda") for _ in range(2))
    pos = np.concatenate([np.arange(n) for n in lens])
    seq = np.repeat(np.arange(N), lens)
    where = table.cpu().numpy()[seq, pos // PAGE] * PAGE + pos % PAGE

    # prompts: every sequence new
    fresh = torch.ones(N, dtype=torch.int32, device="cuda")
    y, window = torch.empty_like(x), torch.empty(N, 3, C, device="cuda")
    G.gdn_conv1d_silu_prompt(G.make_conv_problem(N, T, C, 4, cu_seqlens=i32(cu), dtype="f32"), x, m.conv_w, m.conv_b, None, y, window)
    g = y @ m.gates
    h, state, _ = G.glr_forward(G.make_glr_problem(N, T, C, lam=m.lam, fresh=fresh, cu_seqlens=i32(cu), dtype="f32"), y, g[:, :C], g[:, C:], save=False)
    args = [host(t) for t in (y, g[:, :C], g[:, C:], m.lam)]
    want, end = O.glr_fwd(cu, *args, RATE, None, np.ones(N))
    size = O.glr_sizes(cu, *args, RATE, None, np.ones(N))
    near_glr(h, want, size["y"], 2.0 ** -24)
    near_glr(state, end, size["hT"])
    res, n = G.add_norm_forward(G.make_norm_problem(T, C, eps=EPS, dtype="f32"), x, h, None, m.norm_w)
    qkv = n @ m.qkv
    q, k, v = qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hk) * D], qkv[:, (Hq + Hk) * D:]
    p = G.make_qk_rope_problem(T, Hq, Hk, D, rot=R, positions=i32(pos), freq=m.freq, wq=m.wq, wk=m.wk, eps=EPS, dtype="f32")
    qo = torch.empty(T, Hq * D, device="cuda")
    G.gdn_qk_rope_cache(p, q, k, v, qo, kp, vp, i32(where))
    oracle_rope(m, qkv, pos, qo, kp, vp, where)
    last = torch.from_numpy(cu[1:] - 1).cuda()
    out, lse = G.paged_attention(G.make_paged_problem(table, i32(lens), Hq, Hk, D, page_size=PAGE, dtype="f32"), qo[last], kp, vp, want_lse=True)
    oracle_attention(m, qo[last], kp, vp, table, i32(lens), out, lse)

    # tokens: one captured step for all of them; the program moves inputs, lengths, positions and places on between replays
    b = dict(x=torch.empty(N, C, device="cuda"), y=torch.empty(N, C, device="cuda"), h=torch.empty(N, C, device="cuda"),
             res=torch.empty(N, C, device="cuda"), n=torch.empty(N, C, device="cuda"), g=torch.empty(N, 2 * C, device="cuda"),
             qkv=torch.empty(N, QKV, device="cuda"), q=torch.empty(N, Hq * D, device="cuda"), out=torch.empty(N, Hq * D, device="cuda"),
             lse=torch.empty(N, Hq, device="cuda"))
    slots = i32([2, 0, 4])
    windows, states = torch.zeros(5, 3, C, device="cuda"), torch.zeros(5, C, device="cuda")
    windows[slots.long()], states[slots.long()] = window, state
    count, at, place = i32(lens), i32(lens), i32(np.zeros(N))
    pc = G.make_conv_problem(N, N, C, 4, T=1, dtype="f32")
    pg = G.make_glr_problem(N, N, C, T=1, lam=m.lam, dtype="f32")
    pn = G.make_norm_problem(N, C, eps=EPS, dtype="f32")
    pr = G.make_qk_rope_problem(N, Hq, Hk, D, rot=R, positions=at, freq=m.freq, wq=m.wq, wk=m.wk, eps=EPS, dtype="f32")
    pp = G.make_paged_problem(table, count, Hq, Hk, D, page_size=PAGE, dtype="f32")
    ws = torch.empty(max(1, G.gdn_paged_attn_workspace_bytes(pp)), dtype=torch.uint8, device="cuda")

    def step():
        G.gdn_conv1d_silu_decode(pc, b["x"], m.conv_w, m.conv_b, windows, slots, b["y"])
        torch.matmul(b["y"], m.gates, out=b["g"])
        G.gdn_glr_decode(pg, b["y"], b["g"][:, :C], b["g"][:, C:], states, slots, b["h"])
        G.gdn_add_norm_fwd(pn, b["x"], b["h"], None, m.norm_w, b["res"], b["n"])
        torch.matmul(b["n"], m.qkv, out=b["qkv"])
        G.gdn_qk_rope_cache(pr, b["qkv"][:, :Hq * D], b["qkv"][:, Hq * D:(Hq + Hk) * D], b["qkv"][:, (Hq + Hk) * D:], b["q"], kp, vp, place)
        G.gdn_paged_attn_decode(pp, b["q"], kp, vp, b["out"], b["lse"], ws)

    keep = [t.clone() for t in (windows, states, kp, vp)]
    place.fill_(-1)
    b["x"].zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # (libraries make their handles outside the capture)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, old in zip((windows, states, kp, vp), keep):
        t.copy_(old)
    now = np.array(lens)
    for _ in range(12):
        before = host(states)
        b["x"].copy_(dev(rounded(rng.standard_normal((N, C)), "f32")))
        where = table.cpu().numpy()[np.arange(N), now // PAGE] * PAGE + now % PAGE
        at.copy_(i32(now))
        place.copy_(i32(where))
        count.copy_(i32(now + 1))
        graph.replay()
        torch.cuda.synchronize()
        one = [host(t) for t in (b["y"], b["g"][:, :C], b["g"][:, C:], m.lam)]
        want, after = O.glr_step(*one, RATE, before, [2, 0, 4])
        size = 4 * np.abs(before).max() + 4 * np.abs(one[0])
        near_glr(b["h"], want, size, 2.0 ** -24)
        near_glr(states, after, size.max() + 0 * after)
        oracle_rope(m, b["qkv"], now, b["q"], kp, vp, where)
        oracle_attention(m, b["q"], kp, vp, table, count, b["out"], b["lse"])
        now = now + 1


def test_training_step():
    """x -> recurrence -> + x, norm -> q, k heads normed and turned: gradients of every operator for what came down to it."""
    import torch
    import gated_delta_rule_34_amd as G
    from oracle import hybrid as O

    m, lens, N = Model(3), [150, 0, 33], 3
    T, cu = sum(lens), np.concatenate([[0], np.cumsum([150, 0, 33])])
    rng = np.random.default_rng(4)
    f = lambda *s: dev(rounded(rng.standard_normal(s), "f32"))
    x, r, i, fresh, pos = f(T, C), f(T, C), f(T, C), np.array([1, 0, 1]), np.concatenate([np.arange(n) for n in lens])
    pg = G.make_glr_problem(N, T, C, lam=m.lam, fresh=i32(fresh), cu_seqlens=i32(cu), dtype="f32")
    pn = G.make_norm_problem(T, C, eps=EPS, dtype="f32")
    pr = G.make_qk_rope_problem(T, Hq, Hk, D, rot=R, positions=i32(pos), freq=m.freq, wq=m.wq, wk=m.wk, eps=EPS, dtype="f32")
    h, _, saved = G.glr_forward(pg, x, r, i)
    res, n = G.add_norm_forward(pn, x, h, None, m.norm_w)
    qkv = n @ m.qkv
    q, k = qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hk) * D]
    G.qk_rope_forward(pr, q, k)
    dqo, dko = f(T, Hq * D), f(T, Hk * D)
    d = G.qk_rope_backward(pr, q, k, dqo, dko)
    for name, t, w, up, heads in (("q", q, m.wq, dqo, Hq), ("k", k, m.wk, dko, Hk)):
        v = host(t).reshape(T, heads, D)
        dv, dw = O.norm_rope_bwd(v, host(w), pos, m.freq.cpu().numpy(), R, False, EPS, host(up).reshape(T, heads, D))
        scale = 1 / np.sqrt(np.mean(v * v, -1, keepdims=True) + EPS)
        assert (np.abs(host(d["d" + name]).reshape(dv.shape) - dv) <= U * 40 * scale).all()  # (terms: |t w| and n mean(t w n) of at most some 8 each)
        assert (np.abs(host(d["dw" + name]) - dw) <= U * T * heads * 12).all()
    dn = torch.cat([d["dq"], d["dk"]], 1) @ m.qkv[:, :(Hq + Hk) * D].t().contiguous()
    e = G.add_norm_backward(pn, res, h, None, m.norm_w, dn)
    g = G.glr_backward(pg, x, r, i, saved, e["dy"])
    args = [host(t) for t in (x, r, i, m.lam)]
    want = O.glr_bwd(cu, *args, RATE, None, fresh, host(e["dy"]), None)
    size = O.glr_sizes(cu, *args, RATE, None, fresh, host(e["dy"]), None)
    for name in ("dx", "dr", "di"):
        near_glr(g[name], want[name], size[name], 2.0 ** -24, name)
    near_glr(g["dlam"], want["dlam"], size["dlam"])
    near_glr(g["dh0"], want["dh0"], size["dh0"])


def test_refusals():
    import torch
    import gated_delta_rule_34_amd as G

    new = lambda *s, dtype=torch.bfloat16: torch.randn(*s, device="cuda").to(dtype)
    x, lam = new(20, 64), new(64, dtype=torch.float32)
    p = G.make_glr_problem(1, 20, 64, lam=lam)
    G.glr_forward(p, x, x, x)
    for bad in (None, x.cpu(), x.float(), x[:19], x[:, :56], x.t().contiguous().t(), new(20, 128)[:, ::2]):
        for k in range(3):
            rows = [x, x, x]
            rows[k] = bad
            with pytest.raises((ValueError, AttributeError)):
                G.glr_forward(p, *rows)
    h = torch.zeros(1, 64, device="cuda")
    for bad in (h[:, :32], h.double(), h.cpu(), torch.zeros(64, 2, device="cuda").t()[:1]):
        with pytest.raises(ValueError):
            G.glr_forward(p, x, x, x, bad)
    with pytest.raises(ValueError):  # saved states too small
        G.gdn_glr_fwd(p, x, x, x, None, torch.empty_like(x), None, torch.empty(8, dtype=torch.uint8, device="cuda"), None)
    with pytest.raises(G.GdnError):  # the final state in place of the first
        G.gdn_glr_fwd(p, x, x, x, h, torch.empty_like(x), h, None, None)
    ints = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    for kw in (dict(lam=lam.cpu()), dict(lam=lam.double()), dict(lam=lam[:32]), dict(lam=lam, fresh=ints(2)), dict(lam=lam, fresh=ints(1).long()),
               dict(lam=lam, cu_seqlens=ints(3)), dict(lam=lam, cu_seqlens=ints(2).cpu())):
        with pytest.raises(ValueError):
            G.make_glr_problem(1, 20, 64, **kw)
    one = G.make_glr_problem(4, 4, 64, T=1, lam=lam)
    pool = torch.zeros(4, 64, device="cuda")
    for state, idx in ((None, None), (pool.bfloat16(), None), (pool[:, :32], None), (pool, ints(4).long()), (pool, ints(3))):
        with pytest.raises(ValueError):
            G.gdn_glr_decode(one, x[:4], x[:4], x[:4], state, idx, x[:4].clone())
    with pytest.raises(G.GdnError):  # fewer slots than rows
        G.gdn_glr_decode(one, x[:4], x[:4], x[:4], pool[:3], None, x[:4].clone())

    q, k, freq, pos = new(20, 128), new(20, 64), torch.ones(16, dtype=torch.float64, device="cuda"), ints(20)
    for kw in (dict(positions=pos.long(), freq=freq), dict(positions=pos[:19], freq=freq), dict(positions=pos, freq=freq.float()),
               dict(positions=pos, freq=freq[:8]), dict(positions=pos), dict(positions=pos, freq=freq, wq=lam), dict(positions=pos, freq=freq, wk=lam[:32].bfloat16())):
        with pytest.raises(ValueError):
            G.make_qk_rope_problem(20, 4, 2, 32, **kw)
    r = G.make_qk_rope_problem(20, 4, 2, 32, positions=pos, freq=freq)
    G.qk_rope_forward(r, q, k)
    for bad in ((q, q), (k, k), (q.float(), k), (q, k[:10]), (q[:, ::2], k), (None, k), (q, None)):
        with pytest.raises((ValueError, AttributeError)):
            G.qk_rope_forward(r, *bad)
    kp, where = new(4, 2, 8, 32), ints(20)
    for pages in ((None, kp), (kp, kp[:3]), (kp.float(), kp), (kp, kp.transpose(1, 2)), (kp[..., :16], kp), (kp.flatten(2), kp)):
        with pytest.raises(ValueError):
            G.gdn_qk_rope_cache(r, q, k, k, torch.empty_like(q), *pages, where)
    with pytest.raises(ValueError):
        G.gdn_qk_rope_cache(r, q, k, k, torch.empty_like(q), kp, kp.clone(), where.long())
    with pytest.raises(G.GdnError):  # keys and values into one pool
        G.gdn_qk_rope_cache(r, q, k, k, torch.empty_like(q), kp, kp, where)

    table, lens = ints(6).view(2, 3), ints(2)
    a = G.make_paged_problem(table, lens, 4, 2, 32, page_size=8)
    G.paged_attention(a, q[:2], kp, kp)
    for bad in ((q[:3], kp, kp), (q[:2].float(), kp, kp), (q[:2], kp[:, :1], kp), (q[:2], kp, kp[:3]), (q[:2], None, kp), (None, kp, kp)):
        with pytest.raises((ValueError, AttributeError)):
            G.paged_attention(a, *bad)
    for t, n in ((table.long(), lens), (table[:, ::2], lens), (table[0], lens), (table, lens[:1]), (table, lens.float()), (table, None)):
        with pytest.raises(ValueError):
            G.make_paged_problem(t, n, 4, 2, 32, page_size=8)
    with pytest.raises(ValueError):  # another pool than the problem's
        G.paged_attention(G.make_paged_problem(table, lens, 4, 2, 32, page_size=8, n_pages=9), q[:2], kp, kp)
    with pytest.raises(G.GdnError):  # a longer bound than the table holds
        G.paged_attention(G.make_paged_problem(table, lens, 4, 2, 32, page_size=8, max_len=25), q[:2], kp, kp)
    with pytest.raises(G.GdnError):  # no workspace
        long = G.make_paged_problem(ints(2000).view(2, 1000), lens, 4, 2, 32, page_size=8)
        G.gdn_paged_attn_decode(long, q[:2], kp, kp, torch.empty_like(q[:2]), None, None)
