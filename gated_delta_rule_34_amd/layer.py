"""The operators around the recurrence (C ABI of ``include/gdn_layer.h``).

The selective state space scan (``gdn_ssm_fwd`` / ``_bwd`` / ``_decode``), the causal conv1d +
SiLU with a carried window (``gdn_conv1d_silu_prompt`` / ``_decode``), the gated RMS norm and the
residual addition with its norm (``gdn_gated_norm_*``, ``gdn_add_norm_*``). As in the package
itself the functions keep the C names and only marshal tensors; ``ssm_forward`` and the like
allocate outputs and workspaces with torch. Shapes, types, devices and inner strides are checked
here (ValueError), the rest in the library (GdnError). Everything runs on the current stream of the
tensors' device, which has to be the current device; the calls that allocate nothing also take a raw
``stream`` (the caller then keeps the tensors alive until that stream is done with them).
"""
from __future__ import annotations

import ctypes
import functools

from . import GDN_BF16, GDN_F32, GDN_OK, GdnError, _empty_bytes, _lib, gdn_conv_problem

try:
    from . import _marshal
except ImportError as e:
    class _Missing:
        """Stands in for the module, so that the rest of the package loads; a call of this file's raises."""

        def __init__(self, reason):
            self._reason = reason

        def __getattr__(self, name):
            raise ImportError(f"the binding's module _marshal cannot be loaded ({self._reason}): build the package first "
                              "(python gated_delta_rule_34_amd/build.py, or __graft_entry__.build())")

    _marshal = _Missing(str(e))

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

_signatures = dict(SIGNATURES)  # those of gdn_hybrid.h join them
_bound = {}


def _fn(name):
    fn = _bound.get(name)
    if fn is None:
        fn = getattr(_lib, name)
        fn.argtypes, fn.restype = _signatures[name]
        _bound[name] = fn
    return fn


_address = {}


def _at(name):
    at = _address.get(name)
    if at is None:
        at = _address[name] = ctypes.cast(_fn(name), ctypes.c_void_p).value
    return at


def _call(name, p, *args):
    st = _marshal.call(_at(name), p, *args)
    if st != GDN_OK:
        raise GdnError(st, name)


def _ws_bytes(name, p, kind):
    if not isinstance(p, kind):
        raise TypeError(f"{name}: expected a {kind.__name__}, got {type(p).__name__}")
    return _marshal.size(_at(name), p)


# ------------------------------------------------------------------------------------ checks
# A single token's kernels take a few microseconds, and so would checks of their ten tensors in Python:
# _marshal looks at each tensor, and what it does not accept is explained here.

_torch = _types = _f32 = _i32 = _raw_stream = None


def _use_torch():
    """Looks torch's names up (the package itself loads without torch)."""
    global _torch, _types, _f32, _i32, _raw_stream
    import torch

    _f32, _i32 = torch.float32, torch.int32
    _types = {GDN_F32: torch.float32, GDN_BF16: torch.bfloat16}
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)
    _torch = torch


def _begin(p, t, name):
    """The device of a call, that of its tensor `t`, which has to be the current one, and the type of its rows."""
    if _torch is None:
        _use_torch()
    if t is None:
        raise ValueError(f"{name}: missing")
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name}: expected a GPU tensor")
    if device != _torch.cuda.current_device():
        raise ValueError(f"{name} is on cuda:{device}: make that device current")
    if getattr(p, "device", device) != device:
        raise ValueError(f"{name} is on cuda:{device}, the problem's parameters on cuda:{p.device}")
    return device, _types.get(p.dtype, _torch.bfloat16)


def _rows(t, name, rows, width, device, dtype):
    """(address, row stride) of a [rows, width] view, or [rows, heads, D] with contiguous heads."""
    if t is None:
        raise ValueError(f"{name}: missing")
    at = _marshal.rows(t, rows, width, device, dtype)
    if at is None:
        raise ValueError(f"{name}: expected {rows} rows of {width} contiguous values of {dtype} on cuda:{device}, "
                         f"got {tuple(t.shape)} with strides {t.stride()} of {t.dtype} on {t.device}")
    return at


def _array(t, name, shape, device, dtype):
    """Address of a contiguous tensor of `shape`."""
    if t is None:
        raise ValueError(f"{name}: missing")
    at = _marshal.array(t, shape, device, dtype)
    if at is None:
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor {tuple(shape)} on cuda:{device}, "
                         f"got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")
    return at


def _scratch(t, device):
    """(address, bytes) of a workspace, or of none."""
    if t is None:
        return None, 0
    if t.get_device() != device:
        raise ValueError(f"workspace: expected a tensor on cuda:{device}, got {t.device}")
    return t.data_ptr(), t.numel() * t.element_size()


def _on(stream, device):
    return stream if stream is not None else _raw_stream(device)


def _dtype(dtype):
    return {"f32": GDN_F32, "bf16": GDN_BF16}[dtype] if isinstance(dtype, str) else int(dtype)


def _vector(t, name, count, device):
    """Address of a float32 parameter vector, or None."""
    return None if t is None else _array(t, name, (count,), device, _f32)


# ------------------------------------------------------------------------------------ scan


def make_ssm_problem(N, T_total, Hk, Hv, Dk, Dv, *, a_log, dt_bias=None, d_skip=None, T=None, cu_seqlens=None, dtype="bf16"):
    """Build a gdn_ssm_problem. ``a_log`` (and optionally ``dt_bias``, ``d_skip``): device float32
    [Hv]; ``cu_seqlens``: device int32 [N + 1] or None. The problem keeps these tensors alive."""
    if _torch is None:
        _use_torch()
    device, cu = a_log.get_device(), None
    if device < 0:
        raise ValueError("a_log: expected a GPU tensor")
    if cu_seqlens is not None:
        cu = cu_seqlens.data_ptr()
        if cu_seqlens.get_device() != device or cu_seqlens.dtype is not _i32 or cu_seqlens.shape != (N + 1,) or not cu_seqlens.is_contiguous():
            raise ValueError(f"cu_seqlens: expected a contiguous int32 vector of {N + 1} on cuda:{device}")
    if T is None:
        T = T_total // N if (cu is None and N) else 0
    p = gdn_ssm_problem(N, T, T_total, cu, Hk, Hv, Dk, Dv, _dtype(dtype), _vector(a_log, "a_log", Hv, device),
                        _vector(dt_bias, "dt_bias", Hv, device), _vector(d_skip, "d_skip", Hv, device))
    p.device, p._keep = device, (a_log, dt_bias, d_skip, cu_seqlens)
    return p


def gdn_ssm_fwd_workspace_bytes(p) -> int:
    return _ws_bytes("gdn_ssm_fwd_workspace_bytes", p, gdn_ssm_problem)


def gdn_ssm_bwd_workspace_bytes(p) -> int:
    return _ws_bytes("gdn_ssm_bwd_workspace_bytes", p, gdn_ssm_problem)


def gdn_ssm_chunk_state_bytes(p) -> int:
    return _ws_bytes("gdn_ssm_chunk_state_bytes", p, gdn_ssm_problem)


def _ssm_ins(p, x, b, c, dt, device, dtype):
    T, kw = p.T_total, p.Hk * p.Dk
    return (*_rows(x, "x", T, p.Hv * p.Dv, device, dtype), *_rows(b, "b", T, kw, device, dtype),
            *_rows(c, "c", T, kw, device, dtype), _array(dt, "dt", (T, p.Hv), device, _f32))


def _saved(p, states, device):
    """Address of the saved chunk states, large enough for the problem."""
    if states is None:
        return None
    (at, size), need = _scratch(states, device), gdn_ssm_chunk_state_bytes(p)
    if size < need:
        raise ValueError(f"chunk_states: {need} bytes needed, got {size}")
    return at


def gdn_ssm_fwd(p, x, b, c, dt, S0, y, S_T, chunk_states, workspace, stream=None):
    """Call gdn_ssm_fwd: y and S_T of the scan over prompts. Raises GdnError on a non-OK status."""
    device, dtype = _begin(p, x, "x")
    st = (p.N, p.Hv, p.Dk, p.Dv)
    _call("gdn_ssm_fwd", p, *_ssm_ins(p, x, b, c, dt, device, dtype), None if S0 is None else _array(S0, "S0", st, device, _f32),
          *_rows(y, "y", p.T_total, p.Hv * p.Dv, device, dtype), None if S_T is None else _array(S_T, "S_T", st, device, _f32),
          _saved(p, chunk_states, device), *_scratch(workspace, device), _on(stream, device))


def gdn_ssm_bwd(p, x, b, c, dt, chunk_states, dy, dS_T, dx, db, dc, ddt, da_log, ddt_bias, dd_skip, dS0, workspace,
                stream=None):
    """Call gdn_ssm_bwd: the gradients of gdn_ssm_fwd's inputs (da_log, ddt_bias, dd_skip, dS0 may be None)."""
    device, dtype = _begin(p, x, "x")
    T, xw, kw, st = p.T_total, p.Hv * p.Dv, p.Hk * p.Dk, (p.N, p.Hv, p.Dk, p.Dv)
    _call("gdn_ssm_bwd", p, *_ssm_ins(p, x, b, c, dt, device, dtype), _saved(p, chunk_states, device),
          *_rows(dy, "dy", T, xw, device, dtype), None if dS_T is None else _array(dS_T, "dS_T", st, device, _f32),
          *_rows(dx, "dx", T, xw, device, dtype), *_rows(db, "db", T, kw, device, dtype), *_rows(dc, "dc", T, kw, device, dtype),
          _array(ddt, "ddt", (T, p.Hv), device, _f32),
          *(None if v is None else _array(v, n, (p.Hv,), device, _f32)
            for v, n in ((da_log, "da_log"), (ddt_bias, "ddt_bias"), (dd_skip, "dd_skip"))),
          None if dS0 is None else _array(dS0, "dS0", st, device, _f32), *_scratch(workspace, device), _on(stream, device))


def _pool(state, slot_idx, N, device, shape, dtype):
    """(address, slots, address of the slot map) of a pool of states [n_slots, *shape]."""
    if state is None:
        if shape[0] == 0:  # a window of no rows: any slot will do
            return None, 0x7FFFFFFF, None if slot_idx is None else _array(slot_idx, "slot_idx", (N,), device, _i32)
        raise ValueError("state: missing")
    n_slots = state.shape[0]
    return (_array(state, "state", (n_slots, *shape), device, dtype), min(n_slots, 0x7FFFFFFF),  # (int32 in the C ABI)
            None if slot_idx is None else _array(slot_idx, "slot_idx", (N,), device, _i32))


def gdn_ssm_decode(p, x, b, c, dt, state, slot_idx, y, stream=None):
    """Call gdn_ssm_decode: one token per row; ``state`` float32 [n_slots, Hv, Dk, Dv] updated in place,
    ``slot_idx`` int32 [N] or None (row n -> slot n)."""
    device, dtype = _begin(p, x, "x")
    _call("gdn_ssm_decode", p, *_ssm_ins(p, x, b, c, dt, device, dtype), *_pool(state, slot_idx, p.N, device, (p.Hv, p.Dk, p.Dv), _f32),
          *_rows(y, "y", p.N, p.Hv * p.Dv, device, dtype), _on(stream, device))


def ssm_forward(p, x, b, c, dt, S0=None, y=None, want_final=True, workspace=None, save=True):
    """Allocate y, S_T and (``save``) the chunk states for a backward, run gdn_ssm_fwd; returns
    (y, S_T, states), states None with ``save=False``."""
    import torch

    if y is None:
        y = torch.empty(p.T_total, p.Hv * p.Dv, dtype=x.dtype, device=x.device)
    S_T = torch.empty(p.N, p.Hv, p.Dk, p.Dv, dtype=torch.float32, device=x.device) if want_final else None
    states = _empty_bytes(gdn_ssm_chunk_state_bytes(p), x.device) if save else None
    if workspace is None and (need := gdn_ssm_fwd_workspace_bytes(p)):
        workspace = _empty_bytes(need, x.device)
    gdn_ssm_fwd(p, x, b, c, dt, S0, y, S_T, states, workspace)
    return y, S_T, states


def ssm_backward(p, x, b, c, dt, S0, states, dy, dS_T=None, grads=None, want_dS0=True, workspace=None):
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
        "dx", "db", "dc", "ddt", "da_log", "ddt_bias", "dd_skip", "dS0")), workspace)
    return grads


# ------------------------------------------------------------------------------------ conv


def _conv_ins(p, x, w, bias, device, dtype):
    ch = p.channels
    return (*_rows(x, "x", p.T_total, ch, device, dtype), _array(w, "w", (ch, p.kernel_size), device, _f32),
            None if bias is None else _array(bias, "bias", (ch,), device, _f32))


def gdn_conv1d_silu_prompt(p, x, w, bias, first, y, last, stream=None):
    """Call gdn_conv1d_silu_prompt: y = SiLU(bias + causal conv1d(x, w)) per sequence, continuing from
    ``first`` [N, K - 1, channels] (None: zeros); ``last`` (None: skip) gets the rows a continuation needs. No
    backward: gdn_conv1d_silu_bwd is that of the form without bias and first."""
    device, dtype = _begin(p, x, "x")
    win = (p.N, p.kernel_size - 1, p.channels)
    _call("gdn_conv1d_silu_prompt", p, *_conv_ins(p, x, w, bias, device, dtype),
          None if first is None else _array(first, "first", win, device, dtype),
          *_rows(y, "y", p.T_total, p.channels, device, dtype),
          None if last is None else _array(last, "last", win, device, dtype), _on(stream, device))


def gdn_conv1d_silu_decode(p, x, w, bias, state, slot_idx, y, stream=None):
    """Call gdn_conv1d_silu_decode: one token per row; ``state`` [n_slots, K - 1, channels] is moved on by a
    row in place, ``slot_idx`` int32 [N] or None (row n -> slot n)."""
    device, dtype = _begin(p, x, "x")
    _call("gdn_conv1d_silu_decode", p, *_conv_ins(p, x, w, bias, device, dtype),
          *_pool(state, slot_idx, p.N, device, (p.kernel_size - 1, p.channels), dtype),
          *_rows(y, "y", p.N, p.channels, device, dtype), _on(stream, device))


# ------------------------------------------------------------------------------------ norms


def make_norm_problem(rows, width, *, groups=1, shared=False, eps=1e-6, gate_first=False, scale=1.0, dtype="bf16"):
    """Build a gdn_norm_problem: rows of ``groups`` groups of ``width`` values."""
    return gdn_norm_problem(rows, groups, width, 1 if shared else 0, 1 if gate_first else 0, eps, scale, _dtype(dtype))


def _weight(p, t, name, device):
    """Address of a norm's weights, flat or [groups, width] (one group when shared)."""
    groups = 1 if p.shared else p.groups
    return _array(t, name, (groups, p.width) if t is not None and t.dim() == 2 else (groups * p.width,), device, _f32)


def gdn_gated_norm_bwd_workspace_bytes(p) -> int:
    return _ws_bytes("gdn_gated_norm_bwd_workspace_bytes", p, gdn_norm_problem)


def gdn_add_norm_bwd_workspace_bytes(p) -> int:
    return _ws_bytes("gdn_add_norm_bwd_workspace_bytes", p, gdn_norm_problem)


def gdn_gated_norm_fwd(p, x, z, w, y, stream=None):
    """Call gdn_gated_norm_fwd: y = norm(x) silu(z), or norm(x silu(z)) with gate_first."""
    device, dtype = _begin(p, x, "x")
    n, full = p.rows, p.groups * p.width
    _call("gdn_gated_norm_fwd", p, *_rows(x, "x", n, full, device, dtype), *_rows(z, "z", n, full, device, dtype),
          _weight(p, w, "w", device), *_rows(y, "y", n, full, device, dtype), _on(stream, device))


def gdn_gated_norm_bwd(p, x, z, w, dy, dx, dz, dw, workspace, stream=None):
    """Call gdn_gated_norm_bwd (dw None: skipped, and then no workspace is needed)."""
    device, dtype = _begin(p, x, "x")
    v = (p.rows, p.groups * p.width, device, dtype)
    _call("gdn_gated_norm_bwd", p, *_rows(x, "x", *v), *_rows(z, "z", *v), _weight(p, w, "w", device), *_rows(dy, "dy", *v),
          *_rows(dx, "dx", *v), *_rows(dz, "dz", *v), None if dw is None else _weight(p, dw, "dw", device),
          *_scratch(workspace, device), _on(stream, device))


def gated_norm_forward(p, x, z, w):
    """Allocate y, run gdn_gated_norm_fwd; returns y [rows, groups * width]."""
    y = x.new_empty(p.rows, p.groups * p.width)
    gdn_gated_norm_fwd(p, x, z, w, y)
    return y


def gated_norm_backward(p, x, z, w, dy, workspace=None):
    """Allocate gradients, run gdn_gated_norm_bwd; returns dict dx, dz, dw."""
    grads = dict(dx=x.new_empty(p.rows, p.groups * p.width), dz=x.new_empty(p.rows, p.groups * p.width),
                 dw=w.new_empty(w.shape))
    if workspace is None:
        workspace = _empty_bytes(gdn_gated_norm_bwd_workspace_bytes(p), x.device)
    gdn_gated_norm_bwd(p, x, z, w, dy, grads["dx"], grads["dz"], grads["dw"], workspace)
    return grads


def gdn_add_norm_fwd(p, h, y, s, w, res, out, stream=None):
    """Call gdn_add_norm_fwd: res = h + scale s y (s None: ones), out = norm(res)."""
    device, dtype = _begin(p, h, "h")
    v, width = (p.rows, p.width, device, dtype), (p.width,)
    _call("gdn_add_norm_fwd", p, *_rows(h, "h", *v), *_rows(y, "y", *v), None if s is None else _array(s, "s", width, device, _f32),
          _array(w, "w", width, device, _f32), *_rows(res, "res", *v), *_rows(out, "out", *v), _on(stream, device))


def gdn_add_norm_bwd(p, res, y, s, w, dout, dres, dh, dy, dw, ds, workspace, stream=None):
    """Call gdn_add_norm_bwd (dres, dy, dw, ds may be None; y only where ds is None)."""
    device, dtype = _begin(p, res, "res")
    v, width, none = (p.rows, p.width, device, dtype), (p.width,), (None, 0)
    _call("gdn_add_norm_bwd", p, *_rows(res, "res", *v), *(none if y is None and ds is None else _rows(y, "y", *v)),
          None if s is None else _array(s, "s", width, device, _f32), _array(w, "w", width, device, _f32),
          *_rows(dout, "dout", *v), *(none if dres is None else _rows(dres, "dres", *v)), *_rows(dh, "dh", *v),
          *(none if dy is None else _rows(dy, "dy", *v)), None if dw is None else _array(dw, "dw", width, device, _f32),
          None if ds is None else _array(ds, "ds", width, device, _f32), *_scratch(workspace, device), _on(stream, device))


def add_norm_forward(p, h, y, s, w):
    """Allocate outputs, run gdn_add_norm_fwd; returns (res, out)."""
    res, out = h.new_empty(p.rows, p.width), h.new_empty(p.rows, p.width)
    gdn_add_norm_fwd(p, h, y, s, w, res, out)
    return res, out


def add_norm_backward(p, res, y, s, w, dout, dres=None, workspace=None):
    """Allocate gradients, run gdn_add_norm_bwd; returns dict dh, dy, dw and, with a scale vector, ds."""
    grads = dict(dh=res.new_empty(p.rows, p.width), dy=res.new_empty(p.rows, p.width), dw=w.new_empty(p.width))
    if s is not None:
        grads["ds"] = s.new_empty(p.width)
    if workspace is None:
        workspace = _empty_bytes(gdn_add_norm_bwd_workspace_bytes(p), res.device)
    gdn_add_norm_bwd(p, res, y, s, w, dout, dres, grads["dh"], grads["dy"], grads["dw"], grads.get("ds"), workspace)
    return grads
