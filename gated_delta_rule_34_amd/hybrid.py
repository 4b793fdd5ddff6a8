"""The other token mixers of a hybrid model (C ABI of ``include/gdn_hybrid.h``).

The gated linear recurrence (``gdn_glr_fwd`` / ``_bwd`` / ``_decode``), the RMS norm of each query and
key head with the rotation of its position (``gdn_qk_rope_fwd`` / ``_bwd``, and ``_cache`` on the way into
the pages of a cache) and attention of one new token over such a cache (``gdn_paged_attn_decode``). As in
``layer`` the functions keep the C names and only marshal tensors; ``glr_forward`` and the like allocate
outputs and workspaces with torch. Shapes, types, devices and inner strides are checked here (ValueError),
the rest in the library (GdnError). Everything runs on the current stream of the tensors' device, which has
to be the current device; the calls that allocate nothing also take a raw ``stream`` (the caller then keeps
the tensors alive until that stream is done with them).
"""
from __future__ import annotations

import ctypes
import functools

from . import _empty_bytes
from . import layer as _l
from .layer import I32, I64, P, SZ, _V, _WS, _array, _begin, _call, _dtype, _on, _pool, _rows, _scratch, _vector, _ws_bytes

F32 = ctypes.c_float


class gdn_glr_problem(ctypes.Structure):
    _fields_ = [("N", I32), ("T", I32), ("T_total", I64), ("cu_seqlens", P), ("channels", I32), ("dtype", I32), ("rate", F32),
                ("lambda", P), ("fresh", P)]


class gdn_qk_rope_problem(ctypes.Structure):
    _fields_ = [("rows", I64), ("Hq", I32), ("Hk", I32), ("D", I32), ("rot", I32), ("adjacent", I32), ("eps", F32),
                ("rope_scale", F32), ("dtype", I32), ("positions", P), ("freq", P), ("wq", P), ("wk", P)]


class gdn_paged_problem(ctypes.Structure):
    _fields_ = [("N", I32), ("Hq", I32), ("Hk", I32), ("D", I32), ("page_size", I32), ("n_pages", I32), ("max_pages", I32),
                ("max_len", I32), ("window", I32), ("scale", F32), ("dtype", I32), ("page_table", P), ("lens", P)]


_GLR, _ROPE, _PAGED = (ctypes.POINTER(t) for t in (gdn_glr_problem, gdn_qk_rope_problem, gdn_paged_problem))

# Arguments of every function of gdn_hybrid.h; bound at first use.
SIGNATURES = {
    "gdn_glr_fwd_workspace_bytes": ([_GLR], SZ),
    "gdn_glr_bwd_workspace_bytes": ([_GLR], SZ),
    "gdn_glr_state_bytes": ([_GLR], SZ),
    "gdn_glr_fwd": ([_GLR, *_V, *_V, *_V, P, *_V, P, P, *_WS], ctypes.c_int),
    "gdn_glr_bwd": ([_GLR, *_V, *_V, *_V, P, *_V, P, *_V, *_V, *_V, P, P, *_WS], ctypes.c_int),
    "gdn_glr_decode": ([_GLR, *_V, *_V, *_V, P, I32, P, *_V, P], ctypes.c_int),
    "gdn_qk_rope_fwd": ([_ROPE, *_V, *_V, *_V, *_V, P], ctypes.c_int),
    "gdn_qk_rope_bwd_workspace_bytes": ([_ROPE], SZ),
    "gdn_qk_rope_bwd": ([_ROPE, *_V, *_V, *_V, *_V, *_V, *_V, P, P, *_WS], ctypes.c_int),
    "gdn_qk_rope_cache": ([_ROPE, *_V, *_V, *_V, *_V, P, P, I32, I32, P, P], ctypes.c_int),
    "gdn_paged_attn_workspace_bytes": ([_PAGED], SZ),
    "gdn_paged_attn_decode": ([_PAGED, *_V, P, P, *_V, P, *_WS], ctypes.c_int),
}
HYBRID_EXPORTED = tuple(SIGNATURES)
_l._signatures.update(SIGNATURES)


def _ints(t, name, shape, device):
    """Address of an int32 array, or None."""
    return None if t is None else _array(t, name, shape, device, _l._i32)


def _gpu(t, name):
    """The device of a problem's first tensor."""
    if _l._torch is None:
        _l._use_torch()
    if t is None:
        raise ValueError(f"{name}: missing")
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name}: expected a GPU tensor")
    return device


# ------------------------------------------------------------------------------------ gated linear recurrence


def make_glr_problem(N, T_total, channels, *, lam, rate=8.0, fresh=None, T=None, cu_seqlens=None, dtype="bf16"):
    """Build a gdn_glr_problem. ``lam``: device float32 [channels]; ``fresh``: device int32 [N] or None; ``cu_seqlens``:
    device int32 [N + 1] or None. The problem keeps these tensors alive."""
    device = _gpu(lam, "lam")
    if T is None:
        T = T_total // N if (cu_seqlens is None and N) else 0
    p = gdn_glr_problem(N, T, T_total, _ints(cu_seqlens, "cu_seqlens", (N + 1,), device), channels, _dtype(dtype), rate,
                        _vector(lam, "lam", channels, device), _ints(fresh, "fresh", (N,), device))
    p.device, p._keep = device, (lam, fresh, cu_seqlens)
    return p


def gdn_glr_fwd_workspace_bytes(p) -> int:
    return _ws_bytes("gdn_glr_fwd_workspace_bytes", p, gdn_glr_problem)


def gdn_glr_bwd_workspace_bytes(p) -> int:
    return _ws_bytes("gdn_glr_bwd_workspace_bytes", p, gdn_glr_problem)


def gdn_glr_state_bytes(p) -> int:
    return _ws_bytes("gdn_glr_state_bytes", p, gdn_glr_problem)


def _glr_ins(p, x, r, i, device, dtype):
    v = (p.T_total, p.channels, device, dtype)
    return (*_rows(x, "x", *v), *_rows(r, "r", *v), *_rows(i, "i", *v))


def _states(p, states, device):
    """Address of the saved states, large enough for the problem."""
    if states is None:
        return None
    (at, size), need = _scratch(states, device), gdn_glr_state_bytes(p)
    if size < need:
        raise ValueError(f"states: {need} bytes needed, got {size}")
    return at


def _final(p, t, name, device):
    return None if t is None else _array(t, name, (p.N, p.channels), device, _l._f32)


def gdn_glr_fwd(p, x, r, i, h0, y, h_T, states, workspace, stream=None):
    """Call gdn_glr_fwd: y and h_T of the recurrence over prompts (h0, h_T, states, workspace may be None)."""
    device, dtype = _begin(p, x, "x")
    _call("gdn_glr_fwd", p, *_glr_ins(p, x, r, i, device, dtype), _final(p, h0, "h0", device),
          *_rows(y, "y", p.T_total, p.channels, device, dtype), _final(p, h_T, "h_T", device), _states(p, states, device),
          *_scratch(workspace, device), _on(stream, device))


def gdn_glr_bwd(p, x, r, i, states, dy, dh_T, dx, dr, di, dlam, dh0, workspace, stream=None):
    """Call gdn_glr_bwd: the gradients of gdn_glr_fwd's inputs (dh_T, dlam, dh0 may be None)."""
    device, dtype = _begin(p, x, "x")
    v = (p.T_total, p.channels, device, dtype)
    _call("gdn_glr_bwd", p, *_glr_ins(p, x, r, i, device, dtype), _states(p, states, device), *_rows(dy, "dy", *v),
          _final(p, dh_T, "dh_T", device), *_rows(dx, "dx", *v), *_rows(dr, "dr", *v), *_rows(di, "di", *v),
          _vector(dlam, "dlam", p.channels, device), _final(p, dh0, "dh0", device), *_scratch(workspace, device), _on(stream, device))


def gdn_glr_decode(p, x, r, i, state, slot_idx, y, stream=None):
    """Call gdn_glr_decode: one token per row; ``state`` float32 [n_slots, channels] updated in place, ``slot_idx``
    int32 [N] or None (row n -> slot n)."""
    device, dtype = _begin(p, x, "x")
    _call("gdn_glr_decode", p, *_glr_ins(p, x, r, i, device, dtype), *_pool(state, slot_idx, p.N, device, (p.channels,), _l._f32),
          *_rows(y, "y", p.N, p.channels, device, dtype), _on(stream, device))


def glr_forward(p, x, r, i, h0=None, y=None, want_final=True, workspace=None, save=True):
    """Allocate y, h_T and (``save``) the states for a backward, run gdn_glr_fwd; returns (y, h_T, states),
    states None with ``save=False``."""
    import torch

    if y is None:
        y = torch.empty(p.T_total, p.channels, dtype=x.dtype, device=x.device)
    h_T = torch.empty(p.N, p.channels, dtype=torch.float32, device=x.device) if want_final else None
    states = _empty_bytes(gdn_glr_state_bytes(p), x.device) if save else None
    if workspace is None and (need := gdn_glr_fwd_workspace_bytes(p)):
        workspace = _empty_bytes(need, x.device)
    gdn_glr_fwd(p, x, r, i, h0, y, h_T, states, workspace)
    return y, h_T, states


def glr_backward(p, x, r, i, states, dy, dh_T=None, want_dh0=True, workspace=None):
    """Allocate gradients, run gdn_glr_bwd; returns dict dx, dr, di, dlam, dh0 (None with ``want_dh0=False``). h0
    itself is not read (the saved states hold what follows from it)."""
    import torch

    new = functools.partial(torch.empty, p.T_total, p.channels, dtype=x.dtype, device=x.device)
    f32 = functools.partial(torch.empty, dtype=torch.float32, device=x.device)
    grads = dict(dx=new(), dr=new(), di=new(), dlam=f32(p.channels), dh0=f32(p.N, p.channels) if want_dh0 else None)
    if workspace is None:
        workspace = _empty_bytes(gdn_glr_bwd_workspace_bytes(p), x.device)
    gdn_glr_bwd(p, x, r, i, states, dy, dh_T, *grads.values(), workspace)
    return grads


# ------------------------------------------------------------------------------------ norm and rotation


def make_qk_rope_problem(rows, Hq, Hk, D, *, rot=None, adjacent=False, positions=None, freq=None, wq=None, wk=None, eps=1e-6,
                         rope_scale=1.0, dtype="bf16"):
    """Build a gdn_qk_rope_problem. ``positions``: device int32 [rows]; ``freq``: device float64 [rot / 2]; both may be
    None when ``rot`` (by default all of D) is 0. ``wq``, ``wk``: device float32 [D], or None (ones). The problem keeps
    these tensors alive."""
    rot = D if rot is None else rot
    device, keep = None, (positions, freq, wq, wk)
    for t, name in zip(keep, ("positions", "freq", "wq", "wk")):
        if t is not None and device is None:
            device = _gpu(t, name)
    if rot and (positions is None or freq is None):
        raise ValueError(f"{'freq' if positions is not None else 'positions'}: missing")
    p = gdn_qk_rope_problem(rows, Hq, Hk, D, rot, 1 if adjacent else 0, eps, rope_scale, _dtype(dtype),
                            _ints(positions, "positions", (rows,), device),
                            None if freq is None else _array(freq, "freq", (rot // 2,), device, _l._torch.float64),
                            _vector(wq, "wq", D, device), _vector(wk, "wk", D, device))
    p._keep = keep
    if device is not None:
        p.device = device
    return p


def gdn_qk_rope_fwd(p, q, k, qo, ko, stream=None):
    """Call gdn_qk_rope_fwd: qo, ko from q, k."""
    device, dtype = _begin(p, q, "q")
    vq, vk = (p.rows, p.Hq * p.D, device, dtype), (p.rows, p.Hk * p.D, device, dtype)
    _call("gdn_qk_rope_fwd", p, *_rows(q, "q", *vq), *_rows(k, "k", *vk), *_rows(qo, "qo", *vq), *_rows(ko, "ko", *vk),
          _on(stream, device))


def gdn_qk_rope_bwd_workspace_bytes(p) -> int:
    return _ws_bytes("gdn_qk_rope_bwd_workspace_bytes", p, gdn_qk_rope_problem)


def gdn_qk_rope_bwd(p, q, k, dqo, dko, dq, dk, dwq, dwk, workspace, stream=None):
    """Call gdn_qk_rope_bwd (dwq, dwk may be None; without both no workspace is needed)."""
    device, dtype = _begin(p, q, "q")
    vq, vk = (p.rows, p.Hq * p.D, device, dtype), (p.rows, p.Hk * p.D, device, dtype)
    _call("gdn_qk_rope_bwd", p, *_rows(q, "q", *vq), *_rows(k, "k", *vk), *_rows(dqo, "dqo", *vq), *_rows(dko, "dko", *vk),
          *_rows(dq, "dq", *vq), *_rows(dk, "dk", *vk), _vector(dwq, "dwq", p.D, device), _vector(dwk, "dwk", p.D, device),
          *_scratch(workspace, device), _on(stream, device))


def _pages(k_pages, v_pages, Hk, page_size, D, device, dtype):
    """(address of the keys' pages, of the values', pages, tokens per page)."""
    for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        if t is None:
            raise ValueError(f"{name}: missing")
        if t.dim() != 4:
            raise ValueError(f"{name}: expected pages [n_pages, Hk, page_size, D], got {tuple(t.shape)}")
    n = k_pages.shape[0]
    page_size = k_pages.shape[2] if page_size is None else page_size
    shape = (n, Hk, page_size, D)
    return _array(k_pages, "k_pages", shape, device, dtype), _array(v_pages, "v_pages", shape, device, dtype), n, page_size


def gdn_qk_rope_cache(p, q, k, v, qo, k_pages, v_pages, where, stream=None):
    """Call gdn_qk_rope_cache: qo from q; k and v into the pages [n_pages, Hk, page_size, D] at the places ``where`` (int32
    [rows], page * page_size + offset; a row with a place outside the pool is not cached)."""
    device, dtype = _begin(p, q, "q")
    vq, vk = (p.rows, p.Hq * p.D, device, dtype), (p.rows, p.Hk * p.D, device, dtype)
    _call("gdn_qk_rope_cache", p, *_rows(q, "q", *vq), *_rows(k, "k", *vk), *_rows(v, "v", *vk), *_rows(qo, "qo", *vq),
          *_pages(k_pages, v_pages, p.Hk, None, p.D, device, dtype), _array(where, "where", (p.rows,), device, _l._i32), _on(stream, device))


def qk_rope_forward(p, q, k):
    """Allocate qo, ko, run gdn_qk_rope_fwd; returns (qo, ko) [rows, heads * D]."""
    qo, ko = q.new_empty(p.rows, p.Hq * p.D), k.new_empty(p.rows, p.Hk * p.D)
    gdn_qk_rope_fwd(p, q, k, qo, ko)
    return qo, ko


def qk_rope_backward(p, q, k, dqo, dko, workspace=None):
    """Allocate gradients, run gdn_qk_rope_bwd; returns dict dq, dk, dwq, dwk (None where the problem has no such weight)."""
    import torch

    f32 = functools.partial(torch.empty, p.D, dtype=torch.float32, device=q.device)
    grads = dict(dq=q.new_empty(p.rows, p.Hq * p.D), dk=k.new_empty(p.rows, p.Hk * p.D), dwq=f32() if p.wq else None,
                 dwk=f32() if p.wk else None)
    if workspace is None and (p.wq or p.wk):
        workspace = _empty_bytes(gdn_qk_rope_bwd_workspace_bytes(p), q.device)
    gdn_qk_rope_bwd(p, q, k, dqo, dko, *grads.values(), workspace)
    return grads


# ------------------------------------------------------------------------------------ paged attention


def make_paged_problem(page_table, lens, Hq, Hk, D, *, page_size, n_pages=None, max_len=None, window=0, scale=None, dtype="bf16"):
    """Build a gdn_paged_problem. ``page_table``: device int32 [N, max_pages]; ``lens``: device int32 [N]; ``max_len``: a bound
    of lens that the host knows (by default what the table's rows hold; a lower one makes smaller launches); ``n_pages``: by
    default that of the pages at the call; ``scale``: by default D ** -0.5. The problem keeps these tensors alive."""
    device = _gpu(page_table, "page_table")
    if page_table.dim() != 2:
        raise ValueError(f"page_table: expected [N, max_pages], got {tuple(page_table.shape)}")
    N, width = page_table.shape
    p = gdn_paged_problem(N, Hq, Hk, D, page_size, 0 if n_pages is None else n_pages, width, width * page_size if max_len is None else max_len,
                          window, D ** -0.5 if scale is None else scale, _dtype(dtype),
                          _ints(page_table, "page_table", (N, width), device), _array(lens, "lens", (N,), device, _l._i32))
    p.device, p._keep, p._any = device, (page_table, lens), n_pages is None
    return p


def gdn_paged_attn_workspace_bytes(p) -> int:
    return _ws_bytes("gdn_paged_attn_workspace_bytes", p, gdn_paged_problem)


def gdn_paged_attn_decode(p, q, k_pages, v_pages, out, lse, workspace, stream=None):
    """Call gdn_paged_attn_decode: one new token per row of q over the pages [n_pages, Hk, page_size, D] (lse float32 [N, Hq]
    and workspace may be None)."""
    device, dtype = _begin(p, q, "q")
    v = (p.N, p.Hq * p.D, device, dtype)
    kp, vp, n, _ = _pages(k_pages, v_pages, p.Hk, p.page_size, p.D, device, dtype)
    own = p
    if getattr(p, "_any", False):  # (a copy: calls at the same time may bring other pools)
        own = gdn_paged_problem.from_buffer_copy(p)
        own.n_pages = n
    elif p.n_pages != n:
        raise ValueError(f"k_pages: expected {p.n_pages} pages, got {n}")
    _call("gdn_paged_attn_decode", own, *_rows(q, "q", *v), kp, vp, *_rows(out, "out", *v),
          None if lse is None else _array(lse, "lse", (p.N, p.Hq), device, _l._f32), *_scratch(workspace, device), _on(stream, device))


def paged_attention(p, q, k_pages, v_pages, want_lse=False, workspace=None):
    """Allocate out (and lse), run gdn_paged_attn_decode; returns (out [N, Hq * D], lse or None)."""
    import torch

    out = q.new_empty(p.N, p.Hq * p.D)
    lse = torch.empty(p.N, p.Hq, dtype=torch.float32, device=q.device) if want_lse else None
    if workspace is None and (need := gdn_paged_attn_workspace_bytes(p)):
        workspace = _empty_bytes(need, q.device)
    gdn_paged_attn_decode(p, q, k_pages, v_pages, out, lse, workspace)
    return out, lse
