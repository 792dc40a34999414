"""Binding of the gated linear recurrence and of group norm (marshalling only).

Same manner as ``_gdr``: contiguous CUDA tensors in, outputs allocated by torch when the caller
passes none, a KdaError on a non-OK status, no fallback.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from ._gdr import _IO, _add_status, _check_status, _f32, _maybe, _need, _ptr_or_none, _run
from ._lib import KdaError, KdaGlrShape, _allocators, _increment_version, _lend, _written, load_library

ACTIVATIONS = {"none": 0, "silu": 1}


@functools.lru_cache(maxsize=256)
def _shape(B, T, D, ns, io, gate):
    """The shape struct of these sizes (read-only: every caller gets the same one)."""
    return KdaGlrShape(B, T, D, ns, io, gate)


@functools.lru_cache(maxsize=256)
def _workspace_bytes(name, *sizes):
    return int(getattr(load_library(), name)(_shape(*sizes))) or 256


def _workspace(workspace, size, device, index, empty):
    """The caller's workspace, or one of size() bytes: (tensor, bytes)."""
    if workspace is None:
        n = size()
        return empty(n, dtype=torch.uint8, device=device), n
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise KdaError(1, f"workspace must be contiguous on cuda:{index}")
    return workspace, workspace.numel() * workspace.element_size()


def _glr_args(like, name, g, cu_seqlens):
    """The checks every call of the recurrence shares: (lib, sizes of the shape struct, its shape,
    address of g, states' shape, device)."""
    io = like.dtype
    if not like.is_cuda or io not in _IO or like.dim() != 3:
        raise KdaError(1, f"{name} must be an fp32 or bf16 CUDA tensor [B, T, D]")
    if g.dtype not in _IO:
        raise KdaError(1, "g must be fp32 or bf16")
    index, shape = like.get_device(), like.shape
    B, T, D = shape
    ga = _need("g", g, g.dtype, shape, index)
    ns = 0
    if cu_seqlens is not None:
        ns = cu_seqlens.numel() - 1
        _need("cu_seqlens", cu_seqlens, torch.int32, (ns + 1,), index)
    return _lib._lib or load_library(), (B, T, D, ns, _IO[io], _IO[g.dtype]), shape, ga, \
        (B if cu_seqlens is None else ns, D), index


def kda_glr_fwd_workspace_size(shape: KdaGlrShape) -> int:
    return int(load_library().kda_glr_fwd_workspace_size(ctypes.byref(shape)))


def kda_glr_fwd(x, g, initial_state=None, cu_seqlens=None, out=None, final_state=None, output_final_state=True,
                workspace=None, stream=None, status=None):
    """Forward of the gated linear recurrence h_t = e^{g_t} h_{t-1} + x_t.  x [B,T,D] bf16 or fp32; g (log
    decay, at most 0) [B,T,D] bf16 or fp32; initial_state [NS,D] fp32; cu_seqlens [N+1] int32 (packed
    sequences, B = 1).  status: a 4-byte tensor the caller has zeroed, to which the call adds the
    bits of its device status (kda_read_device_status takes either it or the workspace); the
    results of a call that reports any are not meaningful.  Returns (y like x, final_state or None)."""
    lib, sizes, shape, ga, states, index = _glr_args(x, "x", g, cu_seqlens)
    xa = _need("x", x, x.dtype, shape, index)
    _check_status(status, index)
    s0 = _maybe("initial_state", initial_state, _f32, states, index)
    empty, empty_like = _allocators(stream, index)
    given = (out, final_state)
    if out is None:
        out = empty_like(x)
    else:
        _need("out", out, x.dtype, shape, index)
    if final_state is not None:
        _need("final_state", final_state, _f32, states, index)
    elif output_final_state:
        final_state = empty(states, dtype=_f32, device=x.device)
    ws, n = _workspace(workspace, lambda: _workspace_bytes("kda_glr_fwd_workspace_size", *sizes), x.device, index, empty)
    _run(lib.kda_glr_fwd, index, stream, _shape(*sizes), xa, ga, s0, _ptr_or_none(cu_seqlens), out.data_ptr(),
         _ptr_or_none(final_state), ws.data_ptr(), n)
    if stream is not None:
        _lend(stream, index, x, g, initial_state, cu_seqlens, out, final_state, ws, status)
    _written(*given)
    if status is not None and states[0] > 0:    # (a call without sequences leaves the workspace alone)
        _add_status(status, ws, stream, index)
    return out, final_state


def kda_glr_bwd_workspace_size(shape: KdaGlrShape) -> int:
    return int(load_library().kda_glr_bwd_workspace_size(ctypes.byref(shape)))


def kda_glr_bwd(g, y, d_out, initial_state=None, cu_seqlens=None, d_final_state=None, output_d_initial_state=True,
                workspace=None, stream=None, status=None):
    """Gradients of sum <d_out, y> + <d_final_state, h_final> for kda_glr_fwd, from its g, its y and its
    initial_state (x is not needed; status likewise).  Returns (dx like y, dg like g,
    d_initial_state fp32 or None)."""
    lib, sizes, shape, ga, states, index = _glr_args(y, "y", g, cu_seqlens)
    ya, da = _need("y", y, y.dtype, shape, index), _need("d_out", d_out, y.dtype, shape, index)
    _check_status(status, index)
    s0 = _maybe("initial_state", initial_state, _f32, states, index)
    dfin = _maybe("d_final_state", d_final_state, _f32, states, index)
    empty, empty_like = _allocators(stream, index)
    dx, dg = empty_like(y), empty_like(g)
    ds0 = empty(states, dtype=_f32, device=y.device) if output_d_initial_state else None
    ws, n = _workspace(workspace, lambda: _workspace_bytes("kda_glr_bwd_workspace_size", *sizes), y.device, index, empty)
    _run(lib.kda_glr_bwd, index, stream, _shape(*sizes), ga, ya, da, s0, _ptr_or_none(cu_seqlens), dfin, dx.data_ptr(),
         dg.data_ptr(), _ptr_or_none(ds0), ws.data_ptr(), n)
    if stream is not None:
        _lend(stream, index, g, y, d_out, initial_state, cu_seqlens, d_final_state, ws, status)
    if status is not None and states[0] > 0:
        _add_status(status, ws, stream, index)
    return dx, dg, ds0


def kda_glr_step(x, g, state, slots=None, out=None, status=None, stream=None):
    """Recurrent step for serving: x [B,T,D] and g like kda_glr_fwd's; state [B,D] fp32, updated in place,
    or with slots [B] int32 a pool [num_slots,D] (a negative slot marks an empty row, whose y is 0;
    the others differ from one another).  status: a 4-byte tensor the caller has zeroed, for a
    slot out of range.  Returns y like x."""
    lib, sizes, shape, ga, states, index = _glr_args(x, "x", g, None)
    xa = _need("x", x, x.dtype, shape, index)
    if state is None or state.dim() != 2:
        raise KdaError(1, "state must be an fp32 tensor [B or num_slots, D]")
    n, at = 0, None
    if slots is not None:
        at = _need("slots", slots, torch.int32, (shape[0],), index)
        n = state.shape[0]
        states = (n, shape[2])
    st = _need("state", state, _f32, states, index)
    written = (state,)
    if out is None:
        out = _allocators(stream, index)[1](x)
    else:
        _need("out", out, x.dtype, shape, index)
        written = (state, out)
    _check_status(status, index)
    _run(lib.kda_glr_step, index, stream, _shape(*sizes), xa, ga, st, at, n, out.data_ptr(), _ptr_or_none(status))
    if stream is not None:
        _lend(stream, index, x, g, state, slots, out, status)
    _increment_version(written)
    return out


def _samples(name, x):
    """(N, L, C) of a contiguous x [N, ..., C]."""
    if not x.is_cuda or x.dtype not in _IO or x.dim() < 2 or not x.is_contiguous():
        raise KdaError(1, f"{name} must be a contiguous fp32 or bf16 CUDA tensor [N, ..., C]")
    N, C = x.shape[0], x.shape[-1]
    L = 1
    for n in x.shape[1:-1]:
        L *= n
    return N, L, C


def _activation(name):
    if name not in ACTIVATIONS:
        raise KdaError(1, f"activation must be one of {', '.join(ACTIVATIONS)}")
    return ACTIVATIONS[name]


@functools.lru_cache(maxsize=256)
def _group_norm_bytes(name, N, L, C, groups, index):
    """A workspace's size on device `index` (blocks, and with them their parts, go by the device's processors)."""
    with torch.cuda.device(index):
        return int(getattr(load_library(), name)(N, L, C, groups)) or 256


def kda_group_norm_fwd_workspace_size(N: int, L: int, C: int, groups: int) -> int:
    """Bytes for the current device."""
    return int(load_library().kda_group_norm_fwd_workspace_size(N, L, C, groups))


def kda_group_norm_fwd(x, groups, weight=None, bias=None, eps=1e-5, activation="none", out=None, output_stats=True,
                       workspace=None, stream=None):
    """Group norm of x [N, ..., C] (bf16 or fp32, channels last) over a sample's positions and C / groups
    neighbouring channels, then an activation ("none" or "silu"); weight, bias [C] fp32 or None.
    A 2-D x [N, C] is the norm of heads, row by row.  Returns (y like x, mean, rstd): both fp32
    [N, groups] (None, None without output_stats)."""
    lib = _lib._lib or load_library()
    N, L, C = _samples("x", x)
    act, index, groups = _activation(activation), x.get_device(), int(groups)
    w, b = _maybe("weight", weight, _f32, (C,), index), _maybe("bias", bias, _f32, (C,), index)
    empty, empty_like = _allocators(stream, index)
    given = out
    if out is None:
        out = empty_like(x)
    else:
        _need("out", out, x.dtype, x.shape, index)
    mean = rstd = None
    if output_stats and groups > 0:
        mean, rstd = (empty((N, groups), dtype=_f32, device=x.device) for _ in range(2))
    ws, n = _workspace(workspace, lambda: _group_norm_bytes("kda_group_norm_fwd_workspace_size", N, L, C, groups, index),
                       x.device, index, empty)
    _run(lib.kda_group_norm_fwd, index, stream, N, L, C, groups, _IO[x.dtype], act, x.data_ptr(), w, b, eps, out.data_ptr(),
         _ptr_or_none(mean), _ptr_or_none(rstd), ws.data_ptr(), n)
    if stream is not None:
        _lend(stream, index, x, weight, bias, out, ws)
    if given is not None:
        _written(given)
    return out, mean, rstd


def kda_group_norm_bwd_workspace_size(N: int, L: int, C: int, groups: int) -> int:
    """Bytes for the current device."""
    return int(load_library().kda_group_norm_bwd_workspace_size(N, L, C, groups))


def kda_group_norm_bwd(x, dy, groups, weight, bias, mean, rstd, activation="none", output_dx=True, output_dweight=True,
                       output_dbias=True, workspace=None, stream=None):
    """Gradients of kda_group_norm_fwd from its x, weight, bias, mean and rstd.  Returns (dx, dweight,
    dbias): dx like x; dweight and dbias [C] fp32; None where not asked for."""
    lib = _lib._lib or load_library()
    N, L, C = _samples("x", x)
    act, index, groups = _activation(activation), x.get_device(), int(groups)
    da = _need("dy", dy, x.dtype, x.shape, index)
    w, b = _maybe("weight", weight, _f32, (C,), index), _maybe("bias", bias, _f32, (C,), index)
    mu, rs = _need("mean", mean, _f32, (N, groups), index), _need("rstd", rstd, _f32, (N, groups), index)
    empty, empty_like = _allocators(stream, index)
    dx = empty_like(x) if output_dx else None
    dw = empty(C, dtype=_f32, device=x.device) if output_dweight else None
    db = empty(C, dtype=_f32, device=x.device) if output_dbias else None
    ws, n = _workspace(workspace, lambda: _group_norm_bytes("kda_group_norm_bwd_workspace_size", N, L, C, groups, index),
                       x.device, index, empty)
    _run(lib.kda_group_norm_bwd, index, stream, N, L, C, groups, _IO[x.dtype], act, x.data_ptr(), da, w, b, mu, rs,
         _ptr_or_none(dx), _ptr_or_none(dw), _ptr_or_none(db), ws.data_ptr(), n)
    if stream is not None:
        _lend(stream, index, x, dy, weight, bias, mean, rstd, ws)
    return dx, dw, db
