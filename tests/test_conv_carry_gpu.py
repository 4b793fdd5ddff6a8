"""GPU: conv1d + SiLU with a carried window (prompts and single tokens) against the float64 oracle.

Tolerance, per element: the result's rounding (half a step of the type) and some 16 float32 roundings
of the window's products (SiLU's slope is below 1.1). The carried rows are copies: equal."""
import numpy as np
import pytest

from layer_gpu import HALF, cu_of, dev, host, rel, rounded, torch_dtype

pytestmark = pytest.mark.gpu


def make(lens, ch, K, dtype, seed, bias=True, first=True):
    rng = np.random.default_rng(seed)
    T, N = sum(lens), len(lens)
    return dict(x=rounded(rng.standard_normal((T, ch)), dtype), w=rounded(rng.uniform(-1, 1, (ch, K)), "f32"),
                bias=rounded(rng.standard_normal(ch), "f32") if bias else None,
                first=rounded(rng.standard_normal((N, K - 1, ch)), dtype) if first else None)


def size_of(a, cu):
    """Sum of the window's |products| per output."""
    from oracle import layer as L

    ab = {k: None if v is None else np.abs(v) for k, v in a.items()}
    K = a["w"].shape[1]
    out = np.zeros(a["x"].shape)
    for n in range(len(cu) - 1):
        head = np.zeros((K - 1, out.shape[1])) if ab["first"] is None else ab["first"][n]
        ext = np.concatenate([head, ab["x"][cu[n]:cu[n + 1]]])
        for t in range(cu[n + 1] - cu[n]):
            out[cu[n] + t] = (ab["w"].T * ext[t:t + K]).sum(0)
    return out + (0.0 if ab["bias"] is None else ab["bias"])


def check(y, want, size, dtype):
    tol = HALF[dtype] * np.abs(want) + 16 * 2.0 ** -24 * (size + 1e-30) * 1.1
    assert (np.abs(y - want) <= tol).all(), float(np.max(np.abs(y - want) / tol))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("bias,first", [(True, True), (False, False)])
def test_prompt(dtype, K, bias, first):
    """Lengths below the window, one, none, around a thread's run of rows; 296 channels leave lanes idle;
    x and y are views of wider rows."""
    import torch
    import gated_delta_rule_34_amd as G
    from oracle import layer as L

    lens = [1, 0, 2, 3, 33, 32, 64, 70, 1]
    a, cu = make(lens, 296, K, dtype, 30 + K, bias, first), cu_of(lens)
    want, last_want = L.conv_prompt(cu, *a.values())
    wide = torch.full((sum(lens), 296 + 24), float("nan"), dtype=torch_dtype(dtype), device="cuda")
    x, y = wide[:, 8:304], torch.full_like(wide, 7.0)[:, :296]
    x.copy_(dev(a["x"], dtype))
    p = G.make_conv_problem(len(lens), sum(lens), 296, K, cu_seqlens=(t := torch.tensor(cu, dtype=torch.int32, device="cuda")), dtype=dtype)
    last = torch.empty(len(lens), K - 1, 296, dtype=torch_dtype(dtype), device="cuda")
    G.gdn_conv1d_silu_prompt(p, x, dev(a["w"]), dev(a["bias"]), dev(a["first"], dtype), y, last)
    check(host(y), want, size_of(a, cu), dtype)
    assert np.array_equal(host(last), last_want)
    again = torch.empty_like(y)
    G.gdn_conv1d_silu_prompt(p, x, dev(a["w"]), dev(a["bias"]), dev(a["first"], dtype), again, None)
    assert torch.equal(again, y) and t is not None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ch", [8, 2056])
def test_parts_and_tokens_are_the_whole(dtype, ch):
    """A prompt in three parts (the second shorter than the window), then single tokens, is the whole
    prompt, bit for bit; equal lengths without cu_seqlens."""
    import torch
    import gated_delta_rule_34_amd as G

    a = make([60, 60], ch, 4, dtype, 5)
    x, w, bias, first = dev(a["x"], dtype), dev(a["w"]), dev(a["bias"]), dev(a["first"], dtype)
    whole, end = torch.empty_like(x), torch.empty_like(first)
    G.gdn_conv1d_silu_prompt(G.make_conv_problem(2, 120, ch, 4, T=60, dtype=dtype), x, w, bias, first, whole, end)
    x2, w2 = x.view(2, 60, ch), whole.view(2, 60, ch)
    at, win = 0, first
    for n in (35, 2, 20):
        part, y, nxt = x2[:, at:at + n].reshape(-1, ch), torch.empty(2 * n, ch, dtype=x.dtype, device="cuda"), torch.empty_like(win)
        G.gdn_conv1d_silu_prompt(G.make_conv_problem(2, 2 * n, ch, 4, T=n, dtype=dtype), part, w, bias, win, y, nxt)
        assert torch.equal(y.view(2, n, ch), w2[:, at:at + n])
        at, win = at + n, nxt
    pool = torch.full((5, 3, ch), 9.0, dtype=x.dtype, device="cuda")
    slots = torch.tensor([4, 1], dtype=torch.int32, device="cuda")
    pool[[4, 1]] = win
    p = G.make_conv_problem(2, 2, ch, 4, T=1, dtype=dtype)
    for t in range(at, 60):
        y = torch.empty(2, ch, dtype=x.dtype, device="cuda")
        G.gdn_conv1d_silu_decode(p, x2[:, t].contiguous(), w, bias, pool, slots, y)
        check(host(y), host(w2[:, t]), 8.0, dtype)
    assert torch.equal(pool[[4, 1]], end) and bool((pool[[0, 2, 3]] == 9.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [1, 2, 3, 4])
def test_token(dtype, K):
    import torch
    import gated_delta_rule_34_amd as G
    from oracle import layer as L

    N, ch, slots = 11, 520, 14
    a = make([1] * N, ch, K, dtype, 60 + K)
    rng = np.random.default_rng(2)
    idx = rng.permutation(slots)[:N]
    pool = rounded(rng.standard_normal((slots, K - 1, ch)), dtype)
    a["first"] = pool[idx]
    want, last = L.conv_prompt(cu_of([1] * N), *a.values())
    use = idx.copy()
    use[2] = -3
    if K > 1:
        use[7] = slots
    state, y = dev(pool, dtype), torch.full((N, ch), 7.0, dtype=torch_dtype(dtype), device="cuda")
    p = G.make_conv_problem(N, N, ch, K, T=1, dtype=dtype)
    G.gdn_conv1d_silu_decode(p, dev(a["x"], dtype), dev(a["w"]), dev(a["bias"]), state, torch.from_numpy(use.astype(np.int32)).cuda(), y)
    live = [i for i in range(N) if use[i] == idx[i]]
    check(host(y)[live], want[live], size_of(a, cu_of([1] * N))[live], dtype)
    dead = [i for i in range(N) if i not in live]
    assert bool((y[dead] == 7.0).all())
    got = host(state)
    assert np.array_equal(got[idx[live]], last[live])
    rest = [s for s in range(slots) if s not in set(idx[live])]
    assert np.array_equal(got[rest], pool[rest])


def test_token_without_a_window():
    """K == 1: rows are skipped by their slots all the same; without a pool only negative slots are."""
    import torch
    import gated_delta_rule_34_amd as G

    x, w = torch.randn(4, 16, device="cuda"), torch.randn(16, 1, device="cuda")
    p = G.make_conv_problem(4, 4, 16, 1, T=1, dtype="f32")
    idx = torch.tensor([5, -1, 0, 6], dtype=torch.int32, device="cuda")
    for state, live in ((torch.empty(6, 0, 16, device="cuda"), [0, 2]), (None, [0, 2, 3])):
        y = torch.full((4, 16), 7.0, device="cuda")
        G.gdn_conv1d_silu_decode(p, x, w, None, state, idx, y)
        dead = [i for i in range(4) if i not in live]
        z = (x.double() * w[:, 0].double())[live]
        assert rel(host(y)[live], host(z * z.sigmoid())) <= 1e-6 and bool((y[dead] == 7.0).all())


def test_rows_of_no_sequence_and_malformed_tables():
    import torch
    import gated_delta_rule_34_amd as G

    a = make([40, 30], 64, 4, "bf16", 3)
    x, w, first = dev(a["x"], "bf16"), dev(a["w"]), dev(a["first"], "bf16")
    x[50:] = float("nan")
    cu = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    for table in (cu(0, 20, 50), cu(0, 500, 70), cu(60, 20, 70), cu(-5, 20, 50), cu(0, 70, 20), cu(70, 0, -70)):
        y, last = torch.full_like(x, 7.0), torch.empty_like(first)
        G.gdn_conv1d_silu_prompt(G.make_conv_problem(2, 70, 64, 4, cu_seqlens=table), x, w, None, first, y, last)
        if table.tolist() == [0, 20, 50]:
            assert bool(torch.isfinite(y[:50]).all()) and bool((y[50:] == 7.0).all()) and torch.equal(last[1], x[47:50])


def test_offsets_past_32_bits():
    """Rows 40000 apart over more than 2^31 elements: the last rows are those of a call on them alone."""
    import torch
    import gated_delta_rule_34_amd as G

    rows, wide = 55000, 40000
    big = torch.zeros(rows, wide, dtype=torch.bfloat16, device="cuda")
    big[-40:, :64] = torch.randn(40, 64, device="cuda")
    w = torch.randn(64, 4, device="cuda")
    G.gdn_conv1d_silu_prompt(G.make_conv_problem(1, rows, 64, 4, T=rows), big[:, :64], w, None, None, big[:, 64:128], None)
    alone = torch.empty(40, 64, dtype=torch.bfloat16, device="cuda")
    G.gdn_conv1d_silu_prompt(G.make_conv_problem(1, 40, 64, 4, T=40), big[-40:, :64].contiguous(), w, None, None, alone, None)
    assert torch.equal(big[-40:, 64:128], alone) and bool((alone != 0).any())


@pytest.mark.parametrize("decode", [False, True])
def test_silu_keeps_float32_far_from_zero(decode):
    """One tap of weight 1: y = z sigma(z) of z = x itself, relative to y: the exponential within an ulp (two
    halves), 1 + e^-z, the quotient and the product round: at most 5 2^-24, and e^-z past float32 gives 0."""
    import torch
    import gated_delta_rule_34_amd as G

    z = np.float32(np.random.default_rng(5).uniform(-87, 87, (64, 64))).astype(np.float64)
    z[0, :8] = [0, -200, 200, 1e-30, -1e-30, -103, 88.8, -88.8]
    x, w = dev(z), torch.ones(64, 1, device="cuda")
    y = torch.empty_like(x)
    if decode:
        G.gdn_conv1d_silu_decode(G.make_conv_problem(64, 64, 64, 1, T=1, dtype="f32"), x, w, None, None, None, y)
    else:
        G.gdn_conv1d_silu_prompt(G.make_conv_problem(1, 64, 64, 1, T=64, dtype="f32"), x, w, None, None, y, None)
    want = z / (1 + np.exp(-z))
    off = np.abs(host(y) - want) / (5 * 2.0 ** -24 * np.abs(want) + 100 * 2.0 ** -126)
    assert off.max() <= 1, (float(off.max()), z.reshape(-1)[off.argmax()])


def plain(a, cu):
    """y, the sum of the window's |products| and the last rows, for many rows at once: the rows of every window
    gathered from the sequences' rows and the carried ones behind them."""
    x, w, K, N = a["x"], a["w"], a["w"].shape[1], len(cu) - 1
    first = np.zeros((N, K - 1, x.shape[1])) if a["first"] is None else a["first"]
    rows = np.concatenate([x, first.reshape(N * (K - 1), x.shape[1])])
    n = np.repeat(np.arange(N), np.diff(cu))
    at = lambda t, n: np.where(t >= 0, np.asarray(cu)[n] + t, len(x) + n * (K - 1) + (K - 1) + t)  # place t of sequence n
    t = np.arange(len(x)) - np.asarray(cu)[n]
    z, size = np.zeros(x.shape), np.zeros(x.shape)
    for j in range(K):
        v = rows[at(t - (K - 1) + j, n)] * w[:, j]
        z, size = z + v, size + np.abs(v)
    b = 0.0 if a["bias"] is None else a["bias"]
    seqs = np.arange(N)[:, None]
    last = rows[at(np.diff(cu)[:, None] - (K - 1) + np.arange(K - 1)[None], seqs)]
    return (z + b) / (1 + np.exp(-(z + b))), size + np.abs(b), last


def test_plain_is_the_oracle():
    from oracle import layer as L

    lens = [1, 0, 2, 3, 9]
    a, cu = make(lens, 8, 4, "f32", 1), cu_of(lens)
    (y, size, last), (yo, lo) = plain(a, cu), L.conv_prompt(cu, *a.values())
    assert np.allclose(y, yo, rtol=1e-13, atol=0) and np.array_equal(last, lo) and np.allclose(size, size_of(a, cu), rtol=1e-13, atol=0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("rows,ch", [(8333, 520), (131111, 24)])
def test_prompt_of_many_rows(dtype, K, rows, ch):
    """Runs of 16 rows and of 64: sequences of none to three rows, others that start and end inside a run, a last
    run that is not full, with bias and carried rows; the rows behind the last sequence stay as they were."""
    import torch
    import gated_delta_rule_34_amd as G

    rng = np.random.default_rng(K)
    lens, left = [1, 0, 2, 3, 1, 64, 65, 0, 127, 16, 17], rows
    left -= sum(lens)
    while left:
        lens.append(min(left, int(rng.choice([0, 1, 3, 15, 33, 100, 700, 2500]))))
        left -= lens[-1]
    a, cu = make(lens, ch, K, dtype, K + ch), cu_of(lens)
    want, size, ends = plain(a, cu)
    x = torch.full((rows + 5, ch + 8), float("nan"), dtype=torch_dtype(dtype), device="cuda")[:, :ch]
    x[:rows] = dev(a["x"], dtype)
    y = torch.full((rows + 5, ch), 7.0, dtype=x.dtype, device="cuda")
    last = torch.empty(len(lens), K - 1, ch, dtype=x.dtype, device="cuda")
    t = torch.tensor(cu, dtype=torch.int32, device="cuda")
    p = G.make_conv_problem(len(lens), rows + 5, ch, K, cu_seqlens=t, dtype=dtype)
    G.gdn_conv1d_silu_prompt(p, x, dev(a["w"]), dev(a["bias"]), dev(a["first"], dtype), y, last)
    check(host(y[:rows]), want, size, dtype)
    assert np.array_equal(host(last), ends) and bool((y[rows:] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [1, 2, 3, 4])
def test_tokens_of_many_rows(dtype, K):
    """Four rows to a thread, the last thread's not all there, slots outside the pool at every place among the four."""
    import torch
    import gated_delta_rule_34_amd as G

    N, ch, slots = 1027, 520, 1040
    a = make([1] * N, ch, K, dtype, 70 + K)
    rng = np.random.default_rng(3)
    idx = rng.permutation(slots)[:N]
    pool = rounded(rng.standard_normal((slots, K - 1, ch)), dtype)
    a["first"] = pool[idx]
    want, size, last = plain(a, cu_of([1] * N))
    use = idx.copy()
    use[[0, 5, 10, 15, 17, 18, 20, 21, 22, 23, 500, 1026]] = [-1, slots, -7, slots, -1, -1, -1, slots, -1, -1, 2**31 - 1, -2**31]
    state, x = dev(pool, dtype), dev(a["x"], dtype)
    p = G.make_conv_problem(N, N, ch, K, T=1, dtype=dtype)
    G.gdn_conv1d_silu_decode(p, x, dev(a["w"]), dev(a["bias"]), state, torch.from_numpy(use.astype(np.int32)).cuda(), x)  # in place
    live = use == idx
    y = host(x)
    check(y[live], want[live], size[live], dtype)
    assert np.array_equal(y[~live], a["x"][~live])
    pool[idx[live]] = last[live]
    assert np.array_equal(host(state), pool)


def test_nan_and_infinities_stay_in_their_windows():
    """A carried row reaches the first K - 1 rows of its sequence and channel, a row the next K - 1."""
    import torch
    import gated_delta_rule_34_amd as G

    a, cu = make([20, 40, 20], 16, 4, "f32", 4), cu_of([20, 40, 20])
    x, w, bias, first = dev(a["x"]), dev(a["w"]), dev(a["bias"]), dev(a["first"])
    p = G.make_conv_problem(3, 80, 16, 4, cu_seqlens=(t := torch.tensor(cu, dtype=torch.int32, device="cuda")), dtype="f32")

    def go():
        y, last = torch.empty_like(x), torch.empty_like(first)
        G.gdn_conv1d_silu_prompt(p, x, w, bias, first, y, last)
        return y, last

    y, last = go()
    first[1, 2, 3], first[2, 0, 5], x[59, 7], x[30, 9] = float("nan"), float("inf"), float("-inf"), float("nan")
    y2, last2 = go()
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[20:23, 3], hit[60, 5], hit[59, 7], hit[30:34, 9] = True, True, True, True
    assert torch.equal(y2[~hit], y[~hit]) and bool(y2[20:23, 3].isnan().all()) and bool(y2[30:34, 9].isnan().all()) and t is not None
    assert last2[1, 2, 7] == float("-inf") and torch.equal(last2[[0, 2]], last[[0, 2]])

