"""GPU: what the binding of the layer's operators refuses (ValueError, before anything is launched), and calls
on a raw stream."""
import pytest

pytestmark = pytest.mark.gpu


def _scan():
    import torch
    import gated_delta_rule_34_amd as G

    new = lambda *s, dtype=torch.bfloat16: torch.randn(*s, device="cuda").to(dtype)
    t = dict(x=new(100, 64), b=new(100, 32), c=new(100, 32), dt=new(100, 2, dtype=torch.float32))
    return t, G.make_ssm_problem(1, 100, 1, 2, 32, 32, a_log=torch.zeros(2, device="cuda"))


@pytest.mark.parametrize("name", ["x", "b", "c", "dt"])
def test_scan_refuses(name):
    import torch
    import gated_delta_rule_34_amd as G

    t, p = _scan()
    G.ssm_forward(p, *t.values())
    bad = [None, t[name].cpu(), t[name].double(), t[name][:99], t[name].t().contiguous().t(), t[name][:, :-1]]
    if name == "dt":
        bad.append(torch.zeros(100, 4, device="cuda")[:, ::2])
    else:
        bad.append(t[name].view(100, 2, -1).transpose(1, 2).contiguous().transpose(1, 2))
    for v in bad:
        with pytest.raises((ValueError, AttributeError)):
            G.ssm_forward(p, **{**t, name: v})


def test_problem_and_buffers_refused():
    import torch
    import gated_delta_rule_34_amd as G

    t, p = _scan()
    a = torch.zeros(2, device="cuda")
    for kw in (dict(a_log=a.cpu()), dict(a_log=a.double()), dict(a_log=a[:1]), dict(a_log=a, dt_bias=a.half()),
               dict(a_log=a, cu_seqlens=torch.zeros(2, dtype=torch.int64, device="cuda")),
               dict(a_log=a, cu_seqlens=torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            G.make_ssm_problem(1, 100, 1, 2, 32, 32, **kw)
    y = torch.empty_like(t["x"])
    with pytest.raises(ValueError):  # saved states too small
        G.gdn_ssm_fwd(p, *t.values(), None, y, None, torch.empty(100, dtype=torch.uint8, device="cuda"), None)
    with pytest.raises(G.GdnError):  # in place
        G.gdn_ssm_fwd(p, *t.values(), None, t["x"], None, None, None)
    q = G.make_ssm_problem(4, 4, 1, 2, 32, 32, T=1, a_log=a)
    row = {k: v[:4] for k, v in t.items()}
    pool = torch.zeros(4, 2, 32, 32, device="cuda")
    for bad in (None, pool.bfloat16(), pool[:, :, :, :16], pool.transpose(2, 3)):
        with pytest.raises(ValueError):
            G.gdn_ssm_decode(q, *row.values(), bad, None, y[:4])
    with pytest.raises(ValueError):
        G.gdn_ssm_decode(q, *row.values(), pool, torch.zeros(4, dtype=torch.int64, device="cuda"), y[:4])
    with pytest.raises(G.GdnError):  # fewer slots than rows
        G.gdn_ssm_decode(q, *row.values(), pool[:3], None, y[:4])


def test_conv_and_norms_refused():
    import torch
    import gated_delta_rule_34_amd as G

    x = torch.randn(8, 64, device="cuda").bfloat16()
    w, y, win = torch.randn(64, 4, device="cuda"), torch.empty_like(x), torch.zeros(2, 3, 64, device="cuda").bfloat16()
    p = G.make_conv_problem(2, 8, 64, 4, T=4)
    for bad in (dict(w=w.t().contiguous().t()), dict(w=w.bfloat16()), dict(first=win.float()), dict(first=win[:, :2]), dict(last=win[:1])):
        a = {**dict(x=x, w=w, bias=None, first=win, y=y, last=None), **bad}
        with pytest.raises(ValueError):
            G.gdn_conv1d_silu_prompt(p, *a.values())
    one = G.make_conv_problem(8, 8, 64, 1, T=1)  # a window of no rows needs no state
    G.gdn_conv1d_silu_decode(one, x, w[:, :1].contiguous(), None, None, None, y)
    n = G.make_norm_problem(8, 32, groups=2)
    for v in (torch.ones(32, device="cuda"), torch.ones(64, device="cuda").bfloat16(), torch.ones(32, 2, device="cuda"), None):
        with pytest.raises(ValueError):
            G.gated_norm_forward(n, x, x, v)
    with pytest.raises(G.GdnError):  # weights off their 16 bytes
        G.gated_norm_forward(n, x, x, torch.ones(65, device="cuda")[1:])


def test_raw_stream_and_two_streams_at_once():
    """The same scan on two streams at once, each with its own buffers, and on a stream given as a number."""
    import torch
    import gated_delta_rule_34_amd as G

    t, p = _scan()
    want, last, _ = G.ssm_forward(p, *t.values(), save=False)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(G.ssm_forward(p, *t.values(), save=False)[:2])
    y = torch.empty_like(t["x"])
    G.gdn_ssm_fwd(p, *t.values(), None, y, None, None, None, stream=streams[0].cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    for a, b in outs:
        assert torch.equal(a, want) and torch.equal(b, last)
