"""Float64 CPU oracle of the operators around the recurrence (``include/gdn_layer.h``).

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``; it shares no code with the HIP path. Every
function is the definition written out: the scan token by token, its gradients by the adjoint of
that recurrence in reverse time, the conv over each sequence's rows behind its carried ones, the
norms row by row. Pins (tests/test_layer_oracle.py): central differences of every gradient, and
cases worked by hand.
"""
from __future__ import annotations

import numpy as np


def _sigmoid(z):
    return 1.0 / (1.0 + np.exp(-np.clip(z, -700, 700)))


def softplus(z):
    return np.logaddexp(z, 0.0)


def ssm_fwd(cu, x, b, c, dt, a_log, dt_bias, d_skip, S0):
    """x [T, Hv, Dv], b, c [T, Hk, Dk], dt [T, Hv] -> y [T, Hv, Dv], S_T [N, Hv, Dk, Dv]. dt_bias,
    d_skip, S0 may be None."""
    N, (T, Hv, Dv), (_, Hk, Dk) = len(cu) - 1, x.shape, b.shape
    r = Hv // Hk
    step = softplus(dt + (0.0 if dt_bias is None else dt_bias))
    a = np.exp(-np.exp(a_log) * step)
    y, ST = np.zeros((T, Hv, Dv)), np.zeros((N, Hv, Dk, Dv))
    for n in range(N):
        S = np.zeros((Hv, Dk, Dv)) if S0 is None else S0[n].copy()
        for t in range(cu[n], cu[n + 1]):
            bb, cc = np.repeat(b[t], r, 0), np.repeat(c[t], r, 0)
            S = a[t][:, None, None] * S + bb[:, :, None] * (step[t][:, None] * x[t])[:, None, :]
            y[t] = np.einsum("hdp,hd->hp", S, cc)
            if d_skip is not None:
                y[t] += d_skip[:, None] * x[t]
        ST[n] = S
    return y, ST


def ssm_bwd(cu, x, b, c, dt, a_log, dt_bias, d_skip, S0, dy, dST):
    """Gradients of ssm_fwd for dy and dST (None: zeros): dict dx, db, dc, ddt, da_log, ddt_bias, dd_skip, dS0."""
    N, (T, Hv, Dv), (_, Hk, Dk) = len(cu) - 1, x.shape, b.shape
    r = Hv // Hk
    z = dt + (0.0 if dt_bias is None else dt_bias)
    step, A = softplus(z), -np.exp(a_log)
    a = np.exp(A * step)
    dx, db, dc, ddt = np.zeros_like(x), np.zeros_like(b), np.zeros_like(c), np.zeros_like(dt)
    da_log, dS0 = np.zeros(Hv), np.zeros((N, Hv, Dk, Dv))
    for n in range(N):
        S = [np.zeros((Hv, Dk, Dv)) if S0 is None else S0[n].copy()]
        for t in range(cu[n], cu[n + 1]):
            S.append(a[t][:, None, None] * S[-1] + np.repeat(b[t], r, 0)[:, :, None] * (step[t][:, None] * x[t])[:, None, :])
        dS = np.zeros((Hv, Dk, Dv)) if dST is None else dST[n].copy()
        for t in reversed(range(cu[n], cu[n + 1])):
            i = t - cu[n]
            dc[t] = np.einsum("hdp,hp->hd", S[i + 1], dy[t]).reshape(Hk, r, Dk).sum(1)
            dS = dS + np.repeat(c[t], r, 0)[:, :, None] * dy[t][:, None, :]
            db[t] = np.einsum("hdp,hp->hd", dS, step[t][:, None] * x[t]).reshape(Hk, r, Dk).sum(1)
            du = np.einsum("hdp,hd->hp", dS, np.repeat(b[t], r, 0))
            dx[t] = step[t][:, None] * du
            dlog = a[t] * (S[i] * dS).sum((1, 2))
            da_log += dlog * step[t] * A
            ddt[t] = ((du * x[t]).sum(-1) + A * dlog) * _sigmoid(z[t])
            dS = a[t][:, None, None] * dS
        dS0[n] = dS
    if d_skip is not None:
        dx = dx + d_skip[:, None] * dy
    return dict(dx=dx, db=db, dc=dc, ddt=ddt, da_log=da_log, ddt_bias=ddt.sum(0), dd_skip=(x * dy).sum((0, 2)), dS0=dS0)


def conv_prompt(cu, x, w, bias, first):
    """x [T, ch], w [ch, K], first [N, K - 1, ch] (None: zeros) -> y [T, ch], last [N, K - 1, ch]."""
    K, N = w.shape[1], len(cu) - 1
    y, last = np.zeros(x.shape), np.zeros((N, K - 1, x.shape[1]))
    for n in range(N):
        head = np.zeros((K - 1, x.shape[1])) if first is None else first[n]
        ext = np.concatenate([head, x[cu[n]:cu[n + 1]]])
        for t in range(cu[n + 1] - cu[n]):
            zt = (w.T * ext[t:t + K]).sum(0) + (0.0 if bias is None else bias)
            y[cu[n] + t] = zt * _sigmoid(zt)
        last[n] = ext[len(ext) - (K - 1):] if K > 1 else ext[:0]
    return y, last


def _rms(v, eps):
    return 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)


def gated_norm(x, z, w, eps, gate_first):
    """x, z [rows, groups, width], w [groups or 1, width] -> y."""
    gate = z * _sigmoid(z)
    v = x * gate if gate_first else x
    y = v * _rms(v, eps) * w
    return y if gate_first else y * gate


def gated_norm_bwd(x, z, w, eps, gate_first, dy):
    """dx, dz and dw [groups, width] (not yet summed over shared groups)."""
    s = _sigmoid(z)
    gate, dgate = z * s, s * (1 + z * (1 - s))
    v = x * gate if gate_first else x
    rs = _rms(v, eps)
    n = v * rs
    dn = dy if gate_first else dy * gate
    t = dn * w
    dv = rs * (t - n * (t * n).mean(-1, keepdims=True))
    dw = (dn * n).sum(0)
    if gate_first:
        return dv * gate, dv * x * dgate, dw
    return dv, dy * n * w * dgate, dw


def add_norm_bwd(res, y, f, w, eps, dout, dres, scale):
    """f: the factor of y per column. dh, dy, dw, ds."""
    rs = _rms(res, eps)
    n = res * rs
    t = dout * w
    dh = rs * (t - n * (t * n).mean(-1, keepdims=True)) + (0.0 if dres is None else dres)
    return dh, f * dh, (dout * n).sum(0), scale * (dh * y).sum(0)
