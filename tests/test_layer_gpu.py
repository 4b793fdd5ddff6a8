"""GPU: the operators around the recurrence run together as a layer does: conv1d with a carried window
-> scan -> gated norm -> residual addition with the next norm; as one prompt, as a prompt in parts, token
by token, and with the whole chain of gradients.

Tolerances (2-norm relative), bfloat16 between the operators: each of the four hands on one rounding of
at most 2^-8 (2^-8 / sqrt(3) in the mean square), and the next operator's output moves by about as much:
4 2^-8. float32: the scan's 1e-5, four times. Gradients do not move by as much: a group's norm divides by
its root mean square, which falls to 0.02 here beside 1 elsewhere, and in float64 the rounding of the
conv's output alone moves the gradient of the projection by 0.076. So with bfloat16 the oracle's backward
operators take what the device's operators before them handed on."""
import numpy as np
import pytest

from layer_gpu import cu_of, dev, host, rel, rounded, torch_dtype

pytestmark = pytest.mark.gpu
Hk, Hv, Dk, Dv, K, EPS = 2, 4, 32, 64, 4, 1e-5
XW, KW = Hv * Dv, Hk * Dk
CH = XW + 2 * KW
TOL = {"bf16": 4 * 2.0 ** -8, "f32": 4e-5}


def weights(rng):
    f = lambda a: rounded(a, "f32")
    return dict(w=f(rng.uniform(-1, 1, (CH, K))), bias=f(0.2 * rng.standard_normal(CH)), a_log=f(rng.uniform(0, 2, Hv)),
                dt_bias=f(rng.standard_normal(Hv) - 2), d=f(rng.standard_normal(Hv)), gw=f(1 + 0.2 * rng.standard_normal(Dv)),
                s=f(0.5 + 0.1 * rng.standard_normal(XW)), nw=f(1 + 0.2 * rng.standard_normal(XW)))


def layer(G, W, proj, dt, z, h, first, S0, lens, dtype, save=False):
    """One prompt step; returns everything that a later step or the backward needs."""
    import torch

    T, N = proj.shape[0], len(lens)
    cu = torch.tensor(cu_of(lens), dtype=torch.int32, device="cuda")
    cp = G.make_conv_problem(N, T, CH, K, cu_seqlens=cu, dtype=dtype)
    mixed, last = torch.empty_like(proj), torch.empty_like(first)
    G.gdn_conv1d_silu_prompt(cp, proj, W["w"], W["bias"], first, mixed, last)
    x, b, c = mixed[:, :XW], mixed[:, XW:XW + KW], mixed[:, XW + KW:]
    sp = G.make_ssm_problem(N, T, Hk, Hv, Dk, Dv, a_log=W["a_log"], dt_bias=W["dt_bias"], d_skip=W["d"], cu_seqlens=cu, dtype=dtype)
    y, ST, sv = G.ssm_forward(sp, x, b, c, dt, S0, save=save)
    gp = G.make_norm_problem(T, Dv, groups=Hv, shared=True, eps=EPS, dtype=dtype)
    gated = G.gated_norm_forward(gp, y, z, W["gw"])
    ap = G.make_norm_problem(T, XW, eps=EPS, dtype=dtype)
    res, out = G.add_norm_forward(ap, h, gated, W["s"], W["nw"])
    return dict(cp=cp, cu=cu, mixed=mixed, last=last, sp=sp, x=x, b=b, c=c, y=y, ST=ST, sv=sv, gp=gp, gated=gated, ap=ap, res=res, out=out)


def inputs(dtype, lens, seed):
    rng = np.random.default_rng(seed)
    T, N = sum(lens), len(lens)
    w = weights(rng)
    a = dict(proj=rounded(rng.standard_normal((T, CH)), dtype), dt=rounded(rng.standard_normal((T, Hv)), "f32"),
             z=rounded(rng.standard_normal((T, XW)), dtype), h=rounded(rng.standard_normal((T, XW)), dtype),
             first=rounded(rng.standard_normal((N, K - 1, CH)), dtype), S0=rounded(0.3 * rng.standard_normal((N, Hv, Dk, Dv)), "f32"))
    return w, a, {k: dev(v) for k, v in w.items()}, {k: dev(v, "f32" if k in ("dt", "S0") else dtype) for k, v in a.items()}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_and_its_gradients(dtype):
    import torch
    import gated_delta_rule_34_amd as G
    from oracle import layer as L
    from oracle.conv import conv1d_silu_bwd

    lens = [70, 1, 0, 130]
    w, a, W, t = inputs(dtype, lens, 1)
    a["first"][:] = 0  # the training form of the conv starts each sequence empty
    t["first"].zero_()
    w["bias"][:] = 0
    W["bias"].zero_()
    f = layer(G, W, *t.values(), lens, dtype, save=True)
    cu, T = cu_of(lens), sum(lens)
    rng = np.random.default_rng(2)
    dout, dres = (rounded(rng.standard_normal((T, XW)), dtype) for _ in range(2))
    # the library's chain
    g = G.add_norm_backward(f["ap"], f["res"], f["gated"], W["s"], W["nw"], dev(dout, dtype), dev(dres, dtype))
    gg = G.gated_norm_backward(f["gp"], f["y"], t["z"], W["gw"], g["dy"])
    packed = torch.empty(T, CH, dtype=torch_dtype(dtype), device="cuda")
    new = lambda *s: torch.empty(*s, device="cuda")
    sg = dict(dx=packed[:, :XW], db=packed[:, XW:XW + KW], dc=packed[:, XW + KW:], ddt=new(T, Hv), da_log=new(Hv), ddt_bias=new(Hv),
              dd_skip=new(Hv), dS0=new(len(lens), Hv, Dk, Dv))
    G.ssm_backward(f["sp"], f["x"], f["b"], f["c"], t["dt"], t["S0"], f["sv"], gg["dx"], None, grads=sg)
    dproj = torch.empty_like(packed)
    G.gdn_conv1d_silu_bwd(f["cp"], t["proj"], W["w"], packed, dproj)
    # the oracle's
    mixed, _ = L.conv_prompt(cu, a["proj"], w["w"], w["bias"], a["first"])
    x, b, c = mixed[:, :XW].reshape(T, Hv, Dv), mixed[:, XW:XW + KW].reshape(T, Hk, Dk), mixed[:, XW + KW:].reshape(T, Hk, Dk)
    sa = (x, b, c, a["dt"], w["a_log"], w["dt_bias"], w["d"], a["S0"])
    y, ST = L.ssm_fwd(cu, *sa)
    z = a["z"].reshape(T, Hv, Dv)
    gated = L.gated_norm(y, z, w["gw"], EPS, False).reshape(T, XW)
    res = a["h"] + w["s"] * gated
    out = res * L._rms(res, EPS) * w["nw"]
    for k, v in (("mixed", mixed), ("y", y), ("ST", ST), ("gated", gated), ("res", res), ("out", out)):
        assert rel(host(f[k]), v) <= TOL[dtype], k
    hand = (lambda v, t: host(t).reshape(v.shape)) if dtype == "bf16" else (lambda v, t: v)
    mixed, y, gated, res = hand(mixed, f["mixed"]), hand(y, f["y"]), hand(gated, f["gated"]), hand(res, f["res"])
    x, b, c = mixed[:, :XW].reshape(T, Hv, Dv), mixed[:, XW:XW + KW].reshape(T, Hk, Dk), mixed[:, XW + KW:].reshape(T, Hk, Dk)
    sa = (x, b, c, *sa[3:])
    dh, dg, dnw, ds = L.add_norm_bwd(res, gated, w["s"], w["nw"], EPS, dout, dres, 1.0)
    dy, dz, dgw = L.gated_norm_bwd(y, z, w["gw"], EPS, False, hand(dg, g["dy"]).reshape(T, Hv, Dv))
    want = L.ssm_bwd(cu, *sa, hand(dy, gg["dx"]), None)
    dmix = hand(np.concatenate([want["dx"].reshape(T, -1), want["db"].reshape(T, -1), want["dc"].reshape(T, -1)], 1), packed)
    pairs = dict(dh=(g["dh"], dh), dnw=(g["dw"], dnw), ds=(g["ds"], ds), dz=(gg["dz"], dz), dgw=(gg["dw"], dgw.sum(0)),
                 dproj=(dproj, conv1d_silu_bwd(cu, a["proj"], w["w"], dmix)), **{k: (sg[k], want[k]) for k in sg})
    for k, (got, v) in pairs.items():
        assert rel(host(got), v) <= 2 * TOL[dtype], k  # forward and backward behind one another


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_in_parts_and_tokens(dtype):
    """Prompts of 80 and 45 tokens at once; and as a first part, an uneven second part, then single tokens
    on pools of windows and states."""
    import torch
    import gated_delta_rule_34_amd as G

    lens = [80, 45]
    w, a, W, t = inputs(dtype, lens, 3)
    whole = layer(G, W, *t.values(), lens, dtype)
    start = [0, 80]
    done, first, S0 = [0, 0], t["first"], t["S0"]
    got = torch.zeros_like(whole["out"])
    for part in ([50, 2], [27, 40]):
        rows = [start[n] + done[n] + i for n in range(2) for i in range(part[n])]
        f = layer(G, W, *(t[k][rows] for k in ("proj", "dt", "z", "h")), first, S0, part, dtype)
        got[rows] = f["out"]
        done, first, S0 = [done[n] + part[n] for n in range(2)], f["last"], f["ST"]
    assert done == [77, 42]
    slots = torch.tensor([3, 0], dtype=torch.int32, device="cuda")
    pool_w = torch.zeros(4, K - 1, CH, dtype=torch_dtype(dtype), device="cuda")
    pool_s = torch.zeros(4, Hv, Dk, Dv, device="cuda")
    pool_w[[3, 0]], pool_s[[3, 0]] = first, S0
    cp = G.make_conv_problem(2, 2, CH, K, T=1, dtype=dtype)
    sp = G.make_ssm_problem(2, 2, Hk, Hv, Dk, Dv, T=1, a_log=W["a_log"], dt_bias=W["dt_bias"], d_skip=W["d"], dtype=dtype)
    gp, ap = G.make_norm_problem(2, Dv, groups=Hv, shared=True, eps=EPS, dtype=dtype), G.make_norm_problem(2, XW, eps=EPS, dtype=dtype)
    for i in range(3):
        rows = [start[n] + done[n] + i for n in range(2)]
        mixed, y = torch.empty(2, CH, dtype=torch_dtype(dtype), device="cuda"), torch.empty(2, XW, dtype=torch_dtype(dtype), device="cuda")
        G.gdn_conv1d_silu_decode(cp, t["proj"][rows], W["w"], W["bias"], pool_w, slots, mixed)
        G.gdn_ssm_decode(sp, mixed[:, :XW], mixed[:, XW:XW + KW], mixed[:, XW + KW:], t["dt"][rows], pool_s, slots, y)
        _, got[rows] = G.add_norm_forward(ap, t["h"][rows], G.gated_norm_forward(gp, y, t["z"][rows], W["gw"]), W["s"], W["nw"])
    assert torch.equal(pool_w[[3, 0]], whole["last"])
    assert rel(host(pool_s[[3, 0]]), host(whole["ST"])) <= 1e-5 + (0 if dtype == "f32" else 2.0 ** -8)
    assert rel(host(got), host(whole["out"])) <= TOL[dtype]
