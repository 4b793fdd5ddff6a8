"""How far float32 may take the gated linear recurrence from the float64 oracle, followed token by token, for inputs
that are nowhere negative (x, h0, dy, dhT; the gates have either sign), where no sum cancels. Then a bound is a few 1e-5 of the
value, and a lost part or a wrong factor shows.

With E = 2^-24, half a step of float32. The hardware's exponential, reciprocal and roots are off by up to a whole step, 2 E.
  s(z), 1 - s(z)   z log2(e) is rounded (of bfloat16 rows without a correction): 1.3 |z| E in the exponential, which adds 2, the sum 1,
                   the reciprocal 2, the product 1: 1.3 |z| + 10 (`gate`). A bfloat16 row's 1 - s up to z = 7 is one less the rounded s, which
                   is off by 3 E of one: 3 / (1 - s) more.
  L = c s          c = rate softplus(lambda): exponential 2, log1p 4, product 1 and slack, 8; the product: gate + 9
  e = 1 - exp(-L)  its condition in L is at most one; polynomial (5e-9, 5 roundings of ever smaller terms) or exponential and
                   difference (2 a / e + 1 for L > 1/4, at most 9): gate + 19 (`ke`)
  w = sqrt(e (1 + a))   half of that, root 2, product 2: ke / 2 + 6 (`kw`);  u = s(i) x: gate + 1;  b = w u: kw + gate + 2
                   where w^2 = 2 L < 2^-126, 1 / w ends at 2^63 and w = w^2 / w comes out as less than it is, at worst as 0 (L = 0.104 2^-126: 0.46
                   of it), so by less than itself, which is kw = 1 / E; L / w likewise. Its terms are below 2^-62 of u and G
  a                1 - e where L < 1/4 (then e / a < 0.29: 0.29 ke + 2), exp(-L) beyond: L is off by its own, so max(1, L) (gate + 12) + 4 covers both

The state. A token's own map moves h by E (ke e h + kb b), and what is there by then passes on by a. Maps of 8 tokens are composed before
they reach the carried state: 8 more roundings of each of their e and b (terms of one sign), and 2 of the state per 8 tokens, 1/4
per token. A segment's map (256 tokens at least) is composed of runs of its 64 thread rows (2 per token of a run: at most 64 for up to
8192 tokens a segment), those of 2 + 16 steps (3 each): 128 per segment, 1/2 per token. Together `R` = 3/4 per token of the state. A
composed map is applied at once: h - E h rounds, and is off, by (ke + 128) E of the state in front, however little it leaves; so
that much of the largest state so far counts without decay. The gradient from behind is the same chain in reverse, with b = a dy, whose
roundings (sum, product, 1 - e: 6 with those of 8 tokens, 12) count as kb.
"""
import numpy as np

from layer_gpu import HALF, cu_of, rounded
from oracle import hybrid as O

E = 2.0 ** -24
R = 0.75


def bounds(cu, x, r, i, lam, rate, h0, fresh, dy, dhT, dtype):
    """{y, hT, dx, dr, di, dlam, dh0}: what float32 may move each by (a row's own rounding, half a step of its type, is not in it)."""
    assert all(t is None or (t >= 0).all() for t in (x, h0, dy, dhT))
    (T, C), N = x.shape, len(cu) - 1
    L, a, w = O.glr_gates(r, lam, rate)
    e, si, cr, ci = -np.expm1(-L), O.sigmoid(i), O.sigmoid(-r), O.sigmoid(-i)
    gr, gi = 1.3 * np.abs(r) + 10, 1.3 * np.abs(i) + 10
    fr, fi = (g + (np.where(z <= 7, 3 / c, 0.0) if dtype == "bf16" else 0.0) for g, z, c in ((gr, r, cr), (gi, i, ci)))  # of 1 - s
    ke = gr + 19
    kw, ka = np.where(L < 2.0 ** -125, 1 / E, ke / 2 + 6), np.maximum(1, L) * (gr + 12) + 4
    u, first = si * x, np.zeros((T, 1), bool)
    for n, lo, hi, new in O._sequences(cu, fresh):
        first[lo:hi][:1] = new
    a, e, w = np.where(first, 0.0, a), np.where(first, 1.0, e), np.where(first, 1.0, w)
    y, _ = O.glr_fwd(cu, x, r, i, lam, rate, h0, fresh)
    out = {k: np.zeros((T, C)) for k in ("y", "dx", "dr", "di")}
    out.update({k: np.zeros((N, C)) for k in ("hT", "dh0")}, dlam=np.zeros(C))
    H, bH, G, bG = (np.zeros((T, C)) for _ in range(4))  # the state in front of a token, the gradient that reaches it, their bounds
    for n, lo, hi, new in O._sequences(cu, fresh):
        h = np.zeros(C) if h0 is None or new else h0[n]
        err, most, k = np.zeros(C), np.zeros(C), np.zeros(C)
        for t in range(lo, hi):
            H[t], bH[t] = h, err + E * ((k + 128) * most + h)
            err = a[t] * err + E * ((ke[t] + 8) * e[t] * h + R * np.maximum(h, y[t]) + (kw[t] + gi[t] + 10) * w[t] * u[t])
            most, k, h = np.maximum(most, h), np.maximum(k, ke[t]), y[t]
            out["y"][t] = err + E * ((k + 128) * most + h)
        out["hT"][n] = out["y"][hi - 1] if hi > lo else 0.0
        c = np.zeros(C) if dhT is None else dhT[n]
        err, most, k = np.zeros(C), np.zeros(C), np.zeros(C)
        for t in reversed(range(lo, hi)):
            g = dy[t] + c
            G[t], bG[t] = g, err + E * ((k + 128) * most + g)
            err = a[t] * err + E * ((ke[t] + 8) * e[t] * g + R * g + 12 * a[t] * dy[t])
            most, k, c = np.maximum(most, g), np.maximum(k, ke[t]), a[t] * g
        out["dh0"][n] = 0.0 if new or hi == lo else err + E * ((k + 128) * most + c)
    du = w * G
    bdu = w * bG + (kw + 2) * E * du
    out["dx"] = si * bdu + (gi + 1) * E * si * du
    out["di"] = u * ci * (bdu + (gi + fi + 4) * E * du)
    with np.errstate(divide="ignore", invalid="ignore"):
        T1 = np.where(first, 0.0, u * a / w)
    Q = np.where(first, 0.0, T1 - H)
    bQ = (gi + ka + kw + 4) * E * T1 + bH + E * np.abs(Q)
    LdL = np.abs(a * L * G * Q)
    bL = a * L * (G * bQ + np.abs(Q) * bG) + (ka + gr + 13) * E * LdL
    out["dr"] = cr * (bL + (fr + 1) * E * LdL)
    # sums of a thread's tokens, of 16 rows' and of 16 groups' in float32, of the segments' in float64; the factor sigmoid / softplus
    out["dlam"] = O.sigmoid(lam) / np.logaddexp(lam, 0.0) * (bL + (T / 64 + 44) * E * LdL).sum(0)
    return {k: 1.01 * v for k, v in out.items()}  # (products of two errors)


# (type, lengths, channels, table): one workgroup per sequence, sequences cut into segments of 256 tokens and more, with a table, without one,
# and more than 256 of them.
MANY = [int(n) for n in np.random.default_rng(90).integers(0, 12, 300)]
MANY[40], MANY[41], MANY[299] = 2100, 600, 1500
CASES = [("f32", [127, 128, 129], 32, True), ("bf16", [515, 1, 130], 72, True), ("f32", [3000, 2999], 24, True),
         ("bf16", [40, 2600, 0, 1500, 511, 513], 72, True), ("f32", [9000, 30, 4400], 8, True), ("bf16", [9000, 30, 4400], 8, True),
         ("bf16", [5000], 16, False), ("f32", [1300] * 3, 40, False), ("f32", MANY, 16, True), ("bf16", MANY, 16, True)]


def draw(lens, C, seed, dtype, init=True, fresh="some", gates=1.5, near_one=0.999):
    """Inputs that are nowhere negative, rounded to the type that the kernels read."""
    rng = np.random.default_rng(seed)
    T, N = sum(lens), len(lens)
    v = dict(cu=cu_of(lens), x=rounded(rng.uniform(0.1, 2, (T, C)), dtype), r=rounded(gates * rng.standard_normal((T, C)), dtype),
             i=rounded(gates * rng.standard_normal((T, C)), dtype),
             lam=rounded(np.log(np.expm1(-np.log(rng.uniform(0.9, near_one, C)) / 8.0)), "f32"), rate=8.0,
             h0=rounded(rng.uniform(0, 2, (N, C)), "f32") if init else None,
             fresh={"none": None, "all": np.ones(N), "some": np.arange(N) % 2}[fresh])
    g = dict(dy=rounded(rng.uniform(0.1, 2, (T, C)), dtype), dhT=rounded(rng.uniform(0, 2, (N, C)), "f32"))
    return v, g


def wanted(v, g):
    """The oracle's outputs and gradients."""
    names = [v[k] for k in ("cu", "x", "r", "i", "lam", "rate", "h0", "fresh")]
    y, hT = O.glr_fwd(*names)
    return dict(y=y, hT=hT, **O.glr_bwd(*names, *g.values()))


ROWS = ("y", "dx", "dr", "di")


def beyond(got, want, bound, dtype):
    """By name: the largest difference over its bound."""
    off = {}
    for k in want:
        tol = bound[k] + 2.0 ** -126
        if k in ROWS:
            tol = tol + HALF[dtype] * (np.abs(want[k]) + bound[k])
        assert got[k].shape == want[k].shape, k
        off[k] = float(np.max(np.abs(got[k] - want[k]) / tol, initial=0.0)) if np.isfinite(got[k]).all() else np.inf
    return off
