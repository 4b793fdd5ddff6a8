"""Float64 CPU oracle of the other token mixers of a hybrid model (``include/gdn_hybrid.h``).

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``; it shares no code with the HIP path. Every
function is the definition written out: the gated linear recurrence token by token, its gradients by
the adjoint of that recurrence in reverse time, norm and rotation head by head with complex factors,
attention by each sequence's own tokens. Pins (tests/test_hybrid_oracle.py): central differences of
every gradient, and cases worked by hand.

``glr_sizes`` follows the same sums with absolute terms: what a float32 rounding of every step can move a
result by is a multiple of them. A step's product with a = 1 - e is formed as h - e h and rounds by its larger term, h.
"""
from __future__ import annotations

import numpy as np


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def glr_gates(r, lam, rate):
    """L, a and w of gate rows r [T, C]."""
    L = rate * np.logaddexp(lam, 0.0) * sigmoid(r)
    return L, np.exp(-L), np.sqrt(-np.expm1(-2 * L))


def _sequences(cu, fresh):
    for n in range(len(cu) - 1):
        yield n, cu[n], cu[n + 1], fresh is not None and bool(fresh[n])


def glr_fwd(cu, x, r, i, lam, rate, h0=None, fresh=None):
    """x, r, i [T, C], lam [C] -> y [T, C], h_T [N, C]; h0 [N, C], fresh [N] may be None."""
    _, a, w = glr_gates(r, lam, rate)
    u = sigmoid(i) * x
    y, hT = np.zeros_like(u), np.zeros((len(cu) - 1, x.shape[1]))
    for n, lo, hi, new in _sequences(cu, fresh):
        h = np.zeros(x.shape[1]) if h0 is None or new else h0[n]
        for t in range(lo, hi):
            h = u[t] if new and t == lo else a[t] * h + w[t] * u[t]
            y[t] = h
        hT[n] = h
    return y, hT


def glr_bwd(cu, x, r, i, lam, rate, h0, fresh, dy, dhT):
    """Gradients of glr_fwd for dy and dhT (None: zeros): dict dx, dr, di, dlam, dh0."""
    L, a, w = glr_gates(r, lam, rate)
    si, sr, ci = sigmoid(i), sigmoid(r), sigmoid(-i)  # (one minus a sigmoid next to one would be all rounding)
    u = si * x
    y, _ = glr_fwd(cu, x, r, i, lam, rate, h0, fresh)
    g = {k: np.zeros_like(u) for k in ("dx", "dr", "di")}
    dL, dh0 = np.zeros_like(u), np.zeros((len(cu) - 1, x.shape[1]))
    for n, lo, hi, new in _sequences(cu, fresh):
        c = np.zeros(x.shape[1]) if dhT is None else dhT[n]
        for t in reversed(range(lo, hi)):
            G = dy[t] + c
            first = new and t == lo
            du = G if first else w[t] * G
            g["dx"][t] = si[t] * du
            g["di"][t] = du * x[t] * si[t] * ci[t]
            if not first:
                before = y[t - 1] if t > lo else (0.0 if h0 is None else h0[n])
                with np.errstate(divide="ignore", invalid="ignore"):
                    dL[t] = np.where(w[t] > 0, G * (u[t] * a[t] ** 2 / w[t] - a[t] * before), 0.0)
            c = np.zeros_like(G) if first else a[t] * G
        dh0[n] = 0.0 if new else c
    g["dr"] = dL * L * sigmoid(-r)
    g["dlam"] = (dL * sr).sum(0) * rate * sigmoid(lam)
    g["dh0"] = dh0
    return g


def glr_sizes(cu, x, r, i, lam, rate, h0, fresh, dy=None, dhT=None):
    """Sizes of the forward's terms (h, [N, C] at the ends) and of the backward's: sums of absolute terms,
    each step's counted once more for every later step that it passes through."""
    L, a, w = glr_gates(r, lam, rate)
    si, sr = sigmoid(i), sigmoid(r)
    u = np.abs(si * x)
    H, HT = np.zeros_like(u), np.zeros((len(cu) - 1, x.shape[1]))
    B = np.zeros_like(u)  # in front of each token
    for n, lo, hi, new in _sequences(cu, fresh):
        h = np.zeros(x.shape[1]) if h0 is None or new else np.abs(h0[n])
        m = np.zeros_like(h)
        for t in range(lo, hi):
            B[t] = h + m
            if new and t == lo:
                h, m = u[t], np.zeros_like(h)
            else:
                m = a[t] * m + h
                h = a[t] * h + w[t] * u[t]
            H[t] = h + m
        HT[n] = h + m
    out = dict(y=H, hT=HT)
    if dy is None:
        return out
    for k in ("dx", "dr", "di"):
        out[k] = np.zeros_like(u)
    S, dh0 = np.zeros_like(u), np.zeros_like(HT)
    for n, lo, hi, new in _sequences(cu, fresh):
        c = np.zeros(x.shape[1]) if dhT is None else np.abs(dhT[n])
        m = np.zeros_like(c)
        for t in reversed(range(lo, hi)):
            g, first = np.abs(dy[t]) + c, new and t == lo
            du = (g + m) * (1.0 if first else w[t])
            out["dx"][t] = si[t] * du
            out["di"][t] = du * u[t]
            if not first:
                with np.errstate(divide="ignore", invalid="ignore"):
                    S[t] = np.where(w[t] > 0, (g + m) * a[t] * (u[t] * a[t] / w[t] + B[t]), 0.0)
            c, m = (np.zeros_like(c), np.zeros_like(c)) if first else (a[t] * g, a[t] * m + g)
        dh0[n] = c + m
    out.update(dr=S * L, dlam=(S * sr).sum(0) * rate * sigmoid(lam), dh0=dh0)
    return out


def glr_step(x, r, i, lam, rate, state, slots, fresh=None):
    """One token per row [N, C] over a pool [n_slots, C]: y (NaN where a row is skipped), the pool behind it."""
    y, state = np.full_like(x, np.nan), state.copy()
    for n, s in enumerate(slots):
        if 0 <= s < len(state):
            one, _ = glr_fwd([0, 1], x[n:n + 1], r[n:n + 1], i[n:n + 1], lam, rate, state[s][None], None if fresh is None else fresh[n:n + 1])
            y[n] = state[s] = one[0]
    return y, state


# ------------------------------------------------------------------------------------ norm and rotation


def _pairs(v, R, adjacent):
    """The first R values of the last axis as complex pairs."""
    return v[..., 0:R:2] + 1j * v[..., 1:R:2] if adjacent else v[..., :R // 2] + 1j * v[..., R // 2:R]


def _flat(z, rest, adjacent):
    turned = np.stack([z.real, z.imag], -1).reshape(*z.shape[:-1], -1) if adjacent else np.concatenate([z.real, z.imag], -1)
    return np.concatenate([turned, rest], -1)


def turn(v, pos, freq, R, adjacent, scale=1.0):
    """Heads [rows, H, D] with their first R values turned by pos[row] freq[j]."""
    if R == 0:
        return v
    return _flat(_pairs(v, R, adjacent) * (scale * np.exp(1j * np.multiply.outer(pos.astype(np.float64), freq)))[:, None], v[..., R:], adjacent)


def norm_rope(v, w, pos, freq, R, adjacent, eps, scale=1.0):
    """v [rows, H, D], w [D]."""
    return turn(v / np.sqrt(np.mean(v * v, -1, keepdims=True) + eps) * w, pos, freq, R, adjacent, scale)


def norm_rope_bwd(v, w, pos, freq, R, adjacent, eps, dy, scale=1.0):
    """dv, dw of norm_rope for dy."""
    rs = 1 / np.sqrt(np.mean(v * v, -1, keepdims=True) + eps)
    n, t = v * rs, turn(dy, -pos, freq, R, adjacent, scale)
    tw = t * w
    return rs * (tw - n * np.mean(tw * n, -1, keepdims=True)), (t * n).sum((0, 1))


# ------------------------------------------------------------------------------------ paged attention


def paged(q, k_pages, v_pages, table, lens, scale, window=0, max_len=None):
    """q [N, Hq, D], pages [n_pages, Hk, page, D] -> out [N, Hq, D], lse [N, Hq], and per head the sum of weights times
    |v|, the largest |score| and the largest sum of the score's absolute terms."""
    (N, Hq, D), (n_pages, Hk, page, _) = q.shape, k_pages.shape
    out, size = np.zeros_like(q), np.zeros_like(q)
    lse, top, dot = np.full((N, Hq), -np.inf), np.zeros((N, Hq)), np.zeros((N, Hq))
    for n in range(N):
        end = max(0, int(lens[n])) if max_len is None else min(max(0, int(lens[n])), max_len)
        begin = max(0, end - window) if window else 0
        at = [(table[n][t // page], t % page) for t in range(begin, end) if 0 <= table[n][t // page] < n_pages]
        if not at:
            continue
        p, o = (np.array(v) for v in zip(*at))
        for h in range(Hq):
            k, v = (c[p, h // (Hq // Hk), o] for c in (k_pages, v_pages))
            z = scale * (k @ q[n, h])
            m = z.max()
            if m == -np.inf:
                continue
            e = np.exp(z - m)
            out[n, h], size[n, h] = e @ v / e.sum(), e @ np.abs(v) / e.sum()
            lse[n, h], top[n, h], dot[n, h] = m + np.log(e.sum()), np.abs(z).max(), (abs(scale) * (np.abs(k) @ np.abs(q[n, h]))).max()
    return out, lse, size, top, dot
