"""The operators around the recurrence (C ABI of ``include/gdn_layer.h``).

The selective state space scan (``gdn_ssm_fwd`` / ``_bwd`` / ``_decode``), the causal conv1d +
SiLU with a carried window (``gdn_conv1d_silu_prompt`` / ``_decode``), the gated RMS norm and the
residual addition with its norm (``gdn_gated_norm_*``, ``gdn_add_norm_*``). As in the package
itself the functions keep the C names and only marshal tensors; ``ssm_forward`` and the like
allocate outputs and workspaces with torch. Shapes, types, devices and inner strides are checked
here (ValueError), the rest in the library (GdnError). Everything runs on the current stream of the
tensors' device, which has to be the current device.
"""
from __future__ import annotations

import ctypes
import functools

from . import GDN_BF16, GDN_F32, GDN_OK, GdnError, _empty_bytes, _lib, gdn_conv_problem

P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class gdn_ssm_problem(ctypes.Structure):
    _fields_ = [("N", I32), ("T", I32), ("T_total", I64), ("cu_seqlens", P), ("Hk", I32), ("Hv", I32), ("Dk", I32),
                ("Dv", I32), ("dtype", I32), ("a_log", P), ("dt_bias", P), ("d_skip", P)]


class gdn_norm_problem(ctypes.Structure):
    _fields_ = [("rows", I64), ("groups", I32), ("width", I32), ("shared", I32), ("gate_first", I32),
                ("eps", ctypes.c_float), ("scale", ctypes.c_float), ("dtype", I32)]


_SSM, _CONV, _NORM = (ctypes.POINTER(t) for t in (gdn_ssm_problem, gdn_conv_problem, gdn_norm_problem))
_V = [P, I64]  # a row view: address, row stride
_WS = [P, SZ, P]  # workspace, its bytes, stream

# Arguments of every function of gdn_layer.h; bound at first use.
SIGNATURES = {
    "gdn_ssm_fwd_workspace_bytes": ([_SSM], SZ),
    "gdn_ssm_bwd_workspace_bytes": ([_SSM], SZ),
    "gdn_ssm_chunk_state_bytes": ([_SSM], SZ),
    "gdn_ssm_fwd": ([_SSM, *_V, *_V, *_V, P, P, *_V, P, P, *_WS], ctypes.c_int),
    "gdn_ssm_bwd": ([_SSM, *_V, *_V, *_V, P, P, *_V, P, *_V, *_V, *_V, P, P, P, P, P, *_WS], ctypes.c_int),
    "gdn_ssm_decode": ([_SSM, *_V, *_V, *_V, P, P, I32, P, *_V, P], ctypes.c_int),
    "gdn_conv1d_silu_prompt": ([_CONV, *_V, P, P, P, *_V, P, P], ctypes.c_int),
    "gdn_conv1d_silu_decode": ([_CONV, *_V, P, P, P, I32, P, *_V, P], ctypes.c_int),
    "gdn_gated_norm_bwd_workspace_bytes": ([_NORM], SZ),
    "gdn_add_norm_bwd_workspace_bytes": ([_NORM], SZ),
    "gdn_gated_norm_fwd": ([_NORM, *_V, *_V, P, *_V, P], ctypes.c_int),
    "gdn_gated_norm_bwd": ([_NORM, *_V, *_V, P, *_V, *_V, *_V, P, *_WS], ctypes.c_int),
    "gdn_add_norm_fwd": ([_NORM, *_V, *_V, P, P, *_V, *_V, P], ctypes.c_int),
    "gdn_add_norm_bwd": ([_NORM, *_V, *_V, P, P, *_V, *_V, *_V, *_V, P, P, *_WS], ctypes.c_int),
}
LAYER_EXPORTED = tuple(SIGNATURES)


@functools.lru_cache(maxsize=None)
def _fn(name):
    fn = getattr(_lib, name)
    fn.argtypes, fn.restype = SIGNATURES[name]
    return fn


def _call(name, p, *args):
    st = _fn(name)(ctypes.byref(p), *args)
    if st != GDN_OK:
        raise GdnError(st, name)


# ------------------------------------------------------------------------------------ checks


def _dtype_of(p):
    import torch

    return torch.bfloat16 if p.dtype == GDN_BF16 else torch.float32


class _Check:
    """Checks the tensors of one call and gives their addresses: all on one device, the current one."""

    def __init__(self, p, stream):
        import torch

        self.torch, self.dtype, self.stream, self.device = torch, _dtype_of(p), stream, None

    def _place(self, t, name):
        if not t.is_cuda:
            raise ValueError(f"{name}: expected a GPU tensor")
        if self.device is None:
            self.device = t.device
            if t.device.index != self.torch.cuda.current_device():
                raise ValueError(f"{name} is on {t.device}: make that device current")
        elif t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, other tensors on {self.device}")

    def rows(self, t, name, rows, width, optional=False):
        """(address, row stride) of a [rows, width] view, or [rows, heads, D] with contiguous heads."""
        if t is None:
            if optional:
                return None, 0
            raise ValueError(f"{name}: missing")
        self._place(t, name)
        if t.dtype != self.dtype:
            raise ValueError(f"{name}: expected {self.dtype}, got {t.dtype}")
        if t.dim() not in (2, 3) or t.shape[0] != rows or _inner(t) != width:
            raise ValueError(f"{name}: expected {rows} rows of {width}, got {tuple(t.shape)}")
        if rows == 0:
            return t.data_ptr(), width  # no row to address
        if t.stride(-1) != 1 or (t.dim() == 3 and t.shape[1] > 1 and t.stride(1) != t.shape[2]):
            raise ValueError(f"{name}: rows must be contiguous")
        return t.data_ptr(), (t.stride(0) if rows > 1 else width)

    def array(self, t, name, shape, dtype=None, optional=False):
        """Address of a contiguous tensor of `shape` (float32 unless given)."""
        if t is None:
            if optional:
                return None
            raise ValueError(f"{name}: missing")
        self._place(t, name)
        want = dtype or self.torch.float32
        if t.dtype != want or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous {want} tensor {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
        return t.data_ptr()

    def scratch(self, t):
        """(address, bytes) of a workspace, or of none."""
        if t is None:
            return None, 0
        self._place(t, "workspace")
        return t.data_ptr(), t.numel() * t.element_size()

    def on(self):
        return self.stream if self.stream is not None else self.torch.cuda.current_stream().cuda_stream


def _inner(t):
    return t.shape[1] if t.dim() == 2 else t.shape[1] * t.shape[2]


def _dtype(dtype):
    return {"f32": GDN_F32, "bf16": GDN_BF16}[dtype] if isinstance(dtype, str) else int(dtype)


def _params(p, count, **arrays):
    """Puts the addresses of float32 parameter vectors of `count` values into the problem, which keeps them alive."""
    import torch

    for name, t in arrays.items():
        if t is None:
            setattr(p, name, None)
            continue
        if not t.is_cuda or t.dtype != torch.float32 or t.dim() != 1 or t.shape[0] != count or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous float32 GPU vector of {count}")
        setattr(p, name, t.data_ptr())
    p._keep = arrays


# ------------------------------------------------------------------------------------ scan


def make_ssm_problem(N, T_total, Hk, Hv, Dk, Dv, *, a_log, dt_bias=None, d_skip=None, T=None, cu_seqlens=None, dtype="bf16"):
    """Build a gdn_ssm_problem. ``a_log`` (and optionally ``dt_bias``, ``d_skip``): device float32
    [Hv]; ``cu_seqlens``: device int32 [N + 1] or None. The problem keeps these tensors alive."""
    p = gdn_ssm_problem()
    p.N, p.T_total = int(N), int(T_total)
    p.T = int(T if T is not None else (T_total // N if (cu_seqlens is None and N) else 0))
    p.Hk, p.Hv, p.Dk, p.Dv = int(Hk), int(Hv), int(Dk), int(Dv)
    p.dtype = _dtype(dtype)
    _params(p, p.Hv, a_log=a_log, dt_bias=dt_bias, d_skip=d_skip)
    _seqs(p, cu_seqlens)
    return p


def _seqs(p, cu):
    import torch

    if cu is not None:
        if not cu.is_cuda or cu.dtype != torch.int32 or tuple(cu.shape) != (p.N + 1,) or not cu.is_contiguous():
            raise ValueError(f"cu_seqlens: expected a contiguous int32 GPU vector of {p.N + 1}")
        p._keep["cu_seqlens"] = cu
        p.cu_seqlens = cu.data_ptr()


def gdn_ssm_fwd_workspace_bytes(p) -> int:
    return int(_fn("gdn_ssm_fwd_workspace_bytes")(ctypes.byref(p)))


def gdn_ssm_bwd_workspace_bytes(p) -> int:
    return int(_fn("gdn_ssm_bwd_workspace_bytes")(ctypes.byref(p)))


def gdn_ssm_chunk_state_bytes(p) -> int:
    return int(_fn("gdn_ssm_chunk_state_bytes")(ctypes.byref(p)))


def _ssm_ins(k, p, x, b, c, dt):
    T = p.T_total
    return (*k.rows(x, "x", T, p.Hv * p.Dv), *k.rows(b, "b", T, p.Hk * p.Dk), *k.rows(c, "c", T, p.Hk * p.Dk),
            k.array(dt, "dt", (T, p.Hv)))


def _saved(k, p, states):
    """Address of the saved chunk states, large enough for the problem."""
    if states is None:
        return None
    at, size = k.scratch(states)
    if size < gdn_ssm_chunk_state_bytes(p):
        raise ValueError(f"chunk_states: {gdn_ssm_chunk_state_bytes(p)} bytes needed, got {size}")
    return at


def gdn_ssm_fwd(p, x, b, c, dt, S0, y, S_T, chunk_states, workspace, stream=None):
    """Call gdn_ssm_fwd: y and S_T of the scan over prompts. Raises GdnError on a non-OK status."""
    k = _Check(p, stream)
    st = (p.N, p.Hv, p.Dk, p.Dv)
    _call("gdn_ssm_fwd", p, *_ssm_ins(k, p, x, b, c, dt), k.array(S0, "S0", st, optional=True),
          *k.rows(y, "y", p.T_total, p.Hv * p.Dv), k.array(S_T, "S_T", st, optional=True), _saved(k, p, chunk_states),
          *k.scratch(workspace), k.on())


def gdn_ssm_bwd(p, x, b, c, dt, chunk_states, dy, dS_T, dx, db, dc, ddt, da_log, ddt_bias, dd_skip, dS0, workspace,
                stream=None):
    """Call gdn_ssm_bwd: the gradients of gdn_ssm_fwd's inputs (da_log, ddt_bias, dd_skip, dS0 may be None)."""
    k = _Check(p, stream)
    T, xw, kw, st = p.T_total, p.Hv * p.Dv, p.Hk * p.Dk, (p.N, p.Hv, p.Dk, p.Dv)
    _call("gdn_ssm_bwd", p, *_ssm_ins(k, p, x, b, c, dt), _saved(k, p, chunk_states), *k.rows(dy, "dy", T, xw),
          k.array(dS_T, "dS_T", st, optional=True), *k.rows(dx, "dx", T, xw), *k.rows(db, "db", T, kw),
          *k.rows(dc, "dc", T, kw), k.array(ddt, "ddt", (T, p.Hv)), k.array(da_log, "da_log", (p.Hv,), optional=True),
          k.array(ddt_bias, "ddt_bias", (p.Hv,), optional=True), k.array(dd_skip, "dd_skip", (p.Hv,), optional=True),
          k.array(dS0, "dS0", st, optional=True), *k.scratch(workspace), k.on())


def gdn_ssm_decode(p, x, b, c, dt, state, slot_idx, y, stream=None):
    """Call gdn_ssm_decode: one token per row; ``state`` float32 [n_slots, Hv, Dk, Dv] updated in place,
    ``slot_idx`` int32 [N] or None (row n -> slot n)."""
    k = _Check(p, stream)
    n_slots = 0 if state is None else int(state.shape[0])
    _call("gdn_ssm_decode", p, *_ssm_ins(k, p, x, b, c, dt), k.array(state, "state", (n_slots, p.Hv, p.Dk, p.Dv)), n_slots,
          k.array(slot_idx, "slot_idx", (p.N,), k.torch.int32, optional=True), *k.rows(y, "y", p.N, p.Hv * p.Dv), k.on())


def ssm_forward(p, x, b, c, dt, S0=None, y=None, want_final=True, workspace=None, stream=None, save=True):
    """Allocate y, S_T and (``save``) the chunk states for a backward, run gdn_ssm_fwd; returns
    (y, S_T, states), states None with ``save=False``."""
    import torch

    if y is None:
        y = torch.empty(p.T_total, p.Hv * p.Dv, dtype=x.dtype, device=x.device)
    S_T = torch.empty(p.N, p.Hv, p.Dk, p.Dv, dtype=torch.float32, device=x.device) if want_final else None
    states = _empty_bytes(gdn_ssm_chunk_state_bytes(p), x.device) if save else None
    if workspace is None and (need := gdn_ssm_fwd_workspace_bytes(p)):
        workspace = _empty_bytes(need, x.device)
    gdn_ssm_fwd(p, x, b, c, dt, S0, y, S_T, states, workspace, stream)
    return y, S_T, states


def ssm_backward(p, x, b, c, dt, S0, states, dy, dS_T=None, grads=None, want_dS0=True, workspace=None, stream=None):
    """Allocate gradients, run gdn_ssm_bwd; returns dict dx, db, dc, ddt, da_log, ddt_bias, dd_skip,
    dS0 (None where the problem has no dt_bias or d_skip, or with ``want_dS0=False``). S0 itself is not
    read (the saved states hold what follows from it)."""
    import torch

    if grads is None:
        new = functools.partial(torch.empty, device=x.device)
        f32 = functools.partial(new, dtype=torch.float32)
        T = p.T_total
        grads = dict(dx=new(T, p.Hv * p.Dv, dtype=x.dtype), db=new(T, p.Hk * p.Dk, dtype=x.dtype),
                     dc=new(T, p.Hk * p.Dk, dtype=x.dtype), ddt=f32(T, p.Hv), da_log=f32(p.Hv),
                     ddt_bias=f32(p.Hv) if p.dt_bias else None, dd_skip=f32(p.Hv) if p.d_skip else None,
                     dS0=f32(p.N, p.Hv, p.Dk, p.Dv) if want_dS0 else None)
    if workspace is None:
        workspace = _empty_bytes(gdn_ssm_bwd_workspace_bytes(p), x.device)
    gdn_ssm_bwd(p, x, b, c, dt, states, dy, dS_T, *(grads.get(n) for n in (
        "dx", "db", "dc", "ddt", "da_log", "ddt_bias", "dd_skip", "dS0")), workspace, stream)
    return grads


# ------------------------------------------------------------------------------------ conv


def gdn_conv1d_silu_prompt(p, x, w, bias, first, y, last, stream=None):
    """Call gdn_conv1d_silu_prompt: y = SiLU(bias + causal conv1d(x, w)) per sequence, continuing from
    ``first`` [N, K - 1, channels] (None: zeros); ``last`` (None: skip) gets the rows a continuation needs."""
    k = _Check(p, stream)
    win = (p.N, p.kernel_size - 1, p.channels)
    _call("gdn_conv1d_silu_prompt", p, *k.rows(x, "x", p.T_total, p.channels),
          k.array(w, "w", (p.channels, p.kernel_size)), k.array(bias, "bias", (p.channels,), optional=True),
          k.array(first, "first", win, k.dtype, optional=True), *k.rows(y, "y", p.T_total, p.channels),
          k.array(last, "last", win, k.dtype, optional=True), k.on())


def gdn_conv1d_silu_decode(p, x, w, bias, state, slot_idx, y, stream=None):
    """Call gdn_conv1d_silu_decode: one token per row; ``state`` [n_slots, K - 1, channels] is moved on by a
    row in place, ``slot_idx`` int32 [N] or None (row n -> slot n)."""
    k = _Check(p, stream)
    n_slots = 0 if state is None else int(state.shape[0])
    _call("gdn_conv1d_silu_decode", p, *k.rows(x, "x", p.N, p.channels), k.array(w, "w", (p.channels, p.kernel_size)),
          k.array(bias, "bias", (p.channels,), optional=True),
          k.array(state, "state", (n_slots, p.kernel_size - 1, p.channels), k.dtype), n_slots,
          k.array(slot_idx, "slot_idx", (p.N,), k.torch.int32, optional=True), *k.rows(y, "y", p.N, p.channels), k.on())


# ------------------------------------------------------------------------------------ norms


def make_norm_problem(rows, width, *, groups=1, shared=False, eps=1e-6, gate_first=False, scale=1.0, dtype="bf16"):
    """Build a gdn_norm_problem: rows of ``groups`` groups of ``width`` values."""
    p = gdn_norm_problem()
    p.rows, p.groups, p.width = int(rows), int(groups), int(width)
    p.shared, p.gate_first = 1 if shared else 0, 1 if gate_first else 0
    p.eps, p.scale, p.dtype = float(eps), float(scale), _dtype(dtype)
    return p


def _w_shape(p):
    return p.width if p.shared else p.groups * p.width


def _weight(k, p, t, name):
    """A norm's weights, flat or [groups, width]."""
    return k.array(None if t is None else t.view(-1) if t.is_contiguous() else t, name, (_w_shape(p),))


def _ws_bytes(name, p):
    return int(_fn(name)(ctypes.byref(p)))


def gdn_gated_norm_bwd_workspace_bytes(p) -> int:
    return _ws_bytes("gdn_gated_norm_bwd_workspace_bytes", p)


def gdn_add_norm_bwd_workspace_bytes(p) -> int:
    return _ws_bytes("gdn_add_norm_bwd_workspace_bytes", p)


def gdn_gated_norm_fwd(p, x, z, w, y, stream=None):
    """Call gdn_gated_norm_fwd: y = norm(x) silu(z), or norm(x silu(z)) with gate_first."""
    k, full = _Check(p, stream), p.groups * p.width
    _call("gdn_gated_norm_fwd", p, *k.rows(x, "x", p.rows, full), *k.rows(z, "z", p.rows, full), _weight(k, p, w, "w"),
          *k.rows(y, "y", p.rows, full), k.on())


def gdn_gated_norm_bwd(p, x, z, w, dy, dx, dz, dw, workspace, stream=None):
    """Call gdn_gated_norm_bwd (dw None: skipped, and then no workspace is needed)."""
    k, full = _Check(p, stream), p.groups * p.width
    _call("gdn_gated_norm_bwd", p, *k.rows(x, "x", p.rows, full), *k.rows(z, "z", p.rows, full), _weight(k, p, w, "w"),
          *k.rows(dy, "dy", p.rows, full), *k.rows(dx, "dx", p.rows, full), *k.rows(dz, "dz", p.rows, full),
          None if dw is None else _weight(k, p, dw, "dw"), *k.scratch(workspace), k.on())


def gated_norm_forward(p, x, z, w, stream=None):
    """Allocate y, run gdn_gated_norm_fwd; returns y [rows, groups * width]."""
    y = x.new_empty(p.rows, p.groups * p.width)
    gdn_gated_norm_fwd(p, x, z, w, y, stream)
    return y


def gated_norm_backward(p, x, z, w, dy, workspace=None, stream=None):
    """Allocate gradients, run gdn_gated_norm_bwd; returns dict dx, dz, dw."""
    grads = dict(dx=x.new_empty(p.rows, p.groups * p.width), dz=x.new_empty(p.rows, p.groups * p.width),
                 dw=w.new_empty(w.shape))
    if workspace is None:
        workspace = _empty_bytes(gdn_gated_norm_bwd_workspace_bytes(p), x.device)
    gdn_gated_norm_bwd(p, x, z, w, dy, grads["dx"], grads["dz"], grads["dw"], workspace, stream)
    return grads


def gdn_add_norm_fwd(p, h, y, s, w, res, out, stream=None):
    """Call gdn_add_norm_fwd: res = h + scale s y (s None: ones), out = norm(res)."""
    k, v = _Check(p, stream), (p.rows, p.width)
    _call("gdn_add_norm_fwd", p, *k.rows(h, "h", *v), *k.rows(y, "y", *v), k.array(s, "s", (p.width,), optional=True),
          k.array(w, "w", (p.width,)), *k.rows(res, "res", *v), *k.rows(out, "out", *v), k.on())


def gdn_add_norm_bwd(p, res, y, s, w, dout, dres, dh, dy, dw, ds, workspace, stream=None):
    """Call gdn_add_norm_bwd (dres, dy, dw, ds may be None; y only where ds is None)."""
    k, v = _Check(p, stream), (p.rows, p.width)
    _call("gdn_add_norm_bwd", p, *k.rows(res, "res", *v), *k.rows(y, "y", *v, optional=ds is None),
          k.array(s, "s", (p.width,), optional=True), k.array(w, "w", (p.width,)), *k.rows(dout, "dout", *v),
          *k.rows(dres, "dres", *v, optional=True), *k.rows(dh, "dh", *v), *k.rows(dy, "dy", *v, optional=True),
          k.array(dw, "dw", (p.width,), optional=True), k.array(ds, "ds", (p.width,), optional=True), *k.scratch(workspace),
          k.on())


def add_norm_forward(p, h, y, s, w, stream=None):
    """Allocate outputs, run gdn_add_norm_fwd; returns (res, out)."""
    res, out = h.new_empty(p.rows, p.width), h.new_empty(p.rows, p.width)
    gdn_add_norm_fwd(p, h, y, s, w, res, out, stream)
    return res, out


def add_norm_backward(p, res, y, s, w, dout, dres=None, workspace=None, stream=None):
    """Allocate gradients, run gdn_add_norm_bwd; returns dict dh, dy, dw and, with a scale vector, ds."""
    grads = dict(dh=res.new_empty(p.rows, p.width), dy=res.new_empty(p.rows, p.width), dw=w.new_empty(p.width))
    if s is not None:
        grads["ds"] = s.new_empty(p.width)
    if workspace is None:
        workspace = _empty_bytes(gdn_add_norm_bwd_workspace_bytes(p), res.device)
    gdn_add_norm_bwd(p, res, y, s, w, dout, dres, grads["dh"], grads["dy"], grads["dw"], grads.get("ds"), workspace, stream)
    return grads
