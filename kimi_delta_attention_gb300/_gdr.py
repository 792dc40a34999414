"""Binding of the gated delta rule with a scalar gate and of layer norm (marshalling only).

Same manner as ``_lib``: contiguous CUDA tensors in, outputs allocated by torch when the
caller passes none, a KdaError on a non-OK status, no fallback.  These calls also serve
single tokens, where the host's own time counts: the checks are plain attribute reads and
the device is only switched when it is not the current one.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from ._lib import KDA_BF16, KDA_F32, KdaError, KdaShape, _allocators, _check, _increment_version, _lend, _raw, _written, load_library

_IO = {torch.float32: KDA_F32, torch.bfloat16: KDA_BF16}
_f32 = torch.float32
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _bad(name, dtype, shape, index):
    raise KdaError(1, f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on cuda:{index}")


def _need(name, t, dtype, shape, index):
    """A tensor's address after its checks (`index`: its CUDA device)."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _bad(name, dtype, shape, index)
    return t.data_ptr()


def _maybe(name, t, dtype, shape, index):
    return None if t is None else _need(name, t, dtype, shape, index)


def _run(fn, index, stream, *args):
    """fn(*args, stream) on device `index` (stream None: its current one)."""
    if stream is None:
        stream = _raw_stream(index)
    if index == _current_device():
        code = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            code = fn(*args, stream)
    if code:
        _check(code)


@functools.lru_cache(maxsize=256)
def _shape(B, T, H, HV, K, V, ns, io):
    """The shape struct of these sizes (read-only: every caller gets the same one)."""
    return KdaShape(B, T, H, HV, K, V, ns, io)


def _rule_args(q, k, v, g, beta, scale, cu_seqlens):
    """The checks every delta-rule call shares; (lib, shape struct, addresses, sizes, NS, device, scale)."""
    io = q.dtype
    if not q.is_cuda or io not in _IO:
        raise KdaError(1, "q must be an fp32 or bf16 CUDA tensor")
    qs, vs = q.shape, v.shape
    if len(qs) != 4 or len(vs) != 4:
        raise KdaError(1, "q must be [B, T, H, K] and v [B, T, HV, V]")
    index = q.get_device()
    B, T, H, K = qs
    HV, V = vs[2], vs[3]
    gate = (B, T, HV)
    addr = (_need("q", q, io, qs, index), _need("k", k, io, qs, index), _need("v", v, io, (B, T, HV, V), index),
            _need("g", g, _f32, gate, index), _need("beta", beta, _f32, gate, index))
    ns = 0
    if cu_seqlens is not None:
        ns = cu_seqlens.numel() - 1
        _need("cu_seqlens", cu_seqlens, torch.int32, (ns + 1,), index)
    return _lib._lib or load_library(), _shape(B, T, H, HV, K, V, ns, _IO[io]), addr, \
        (B if cu_seqlens is None else ns, HV, K, V), index, K ** -0.5 if scale is None else scale


def _ptr_or_none(t):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=256)
def _workspace_bytes(name, *sizes):
    return int(getattr(load_library(), name)(_shape(*sizes))) or 256


def _workspace(workspace, name, shape, index, empty):
    """The caller's workspace, or one of the size that `name` gives for the shape: (tensor, bytes)."""
    if workspace is None:
        n = _workspace_bytes(name, shape.B, shape.T, shape.H, shape.HV, shape.K, shape.V, shape.num_seqs, shape.io_dtype)
        return empty(n, dtype=torch.uint8, device=torch.device("cuda", index)), n
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise KdaError(1, f"workspace must be contiguous on cuda:{index}")
    return workspace, workspace.numel() * workspace.element_size()


def _check_status(status, index):
    if status is not None and (status.get_device() != index or status.numel() * status.element_size() < 4 or
                               not status.is_contiguous()):
        raise KdaError(1, f"status must hold 4 bytes on cuda:{index}")


def _add_status(status, ws, stream, index):
    """The status bits a call leaves in its workspace's first word, added to the caller's word."""
    word = lambda t: t.view(-1).view(torch.uint8)[:4].view(torch.int32)
    if stream is None:
        word(status).bitwise_or_(word(ws))
    else:
        with torch.cuda.stream(_raw(stream, index)):
            word(status).bitwise_or_(word(ws))


def kda_gdr_fwd_workspace_size(shape: KdaShape) -> int:
    return int(load_library().kda_gdr_fwd_workspace_size(ctypes.byref(shape)))


def kda_gdr_fwd(q, k, v, g, beta, scale=None, initial_state=None, cu_seqlens=None, out=None, final_state=None,
                output_final_state=True, workspace=None, stream=None, status=None):
    """Forward of the gated delta rule with a scalar gate.  q, k [B,T,H,K]; v [B,T,HV,V];
    g (log decay), beta [B,T,HV] fp32; initial_state [NS,HV,K,V] fp32; cu_seqlens [N+1]
    int32 (packed sequences, B = 1).  status: a 4-byte tensor the caller has zeroed, to which
    the call adds the bits of its device status (kda_read_device_status takes either it or the
    workspace); the results of a call that reports any are not meaningful.  Returns
    (o [B,T,HV,V], final_state or None)."""
    lib, shape, addr, states, index, scale = _rule_args(q, k, v, g, beta, scale, cu_seqlens)
    _check_status(status, index)
    s0 = _maybe("initial_state", initial_state, _f32, states, index)
    empty, empty_like = _allocators(stream, index)
    given = (out, final_state)
    if out is None:
        out = empty_like(v)
    else:
        _need("out", out, v.dtype, v.shape, index)
    if final_state is not None:
        _need("final_state", final_state, _f32, states, index)
    elif output_final_state:
        final_state = empty(states, dtype=_f32, device=q.device)
    ws, n = _workspace(workspace, "kda_gdr_fwd_workspace_size", shape, index, empty)
    _run(lib.kda_gdr_fwd, index, stream, shape, *addr, scale, s0, _ptr_or_none(cu_seqlens), out.data_ptr(),
         _ptr_or_none(final_state), ws.data_ptr(), n)
    if stream is not None:
        _lend(stream, index, q, k, v, g, beta, initial_state, cu_seqlens, out, final_state, ws, status)
    _written(*given)
    if status is not None and states[0] > 0:    # (a call without sequences leaves the workspace alone)
        _add_status(status, ws, stream, index)
    return out, final_state


def kda_gdr_bwd_workspace_size(shape: KdaShape) -> int:
    return int(load_library().kda_gdr_bwd_workspace_size(ctypes.byref(shape)))


def kda_gdr_bwd(q, k, v, g, beta, d_out, scale=None, initial_state=None, cu_seqlens=None, d_final_state=None,
                output_d_initial_state=True, workspace=None, stream=None, status=None):
    """Gradients of sum <d_out, o> + <d_final_state, S_final> for kda_gdr_fwd with the same
    arguments (bf16; status likewise).  Returns (dq, dk, dv, dg, dbeta, d_initial_state): dq, dk, dv bf16,
    the others fp32, in the inputs' shapes."""
    lib, shape, addr, states, index, scale = _rule_args(q, k, v, g, beta, scale, cu_seqlens)
    s0 = _maybe("initial_state", initial_state, _f32, states, index)
    _check_status(status, index)
    do = _need("d_out", d_out, v.dtype, v.shape, index)
    dfin = _maybe("d_final_state", d_final_state, _f32, states, index)
    empty, empty_like = _allocators(stream, index)
    dq, dk, dv, dg, dbeta = empty_like(q), empty_like(k), empty_like(v), empty_like(g), empty_like(beta)
    ds0 = empty(states, dtype=_f32, device=q.device) if output_d_initial_state else None
    ws, n = _workspace(workspace, "kda_gdr_bwd_workspace_size", shape, index, empty)
    _run(lib.kda_gdr_bwd, index, stream, shape, *addr, scale, s0, _ptr_or_none(cu_seqlens), do, dfin, dq.data_ptr(),
         dk.data_ptr(), dv.data_ptr(), dg.data_ptr(), dbeta.data_ptr(), _ptr_or_none(ds0), ws.data_ptr(), n)
    if stream is not None:
        _lend(stream, index, q, k, v, g, beta, initial_state, cu_seqlens, d_out, d_final_state, ws, status)
    if status is not None and states[0] > 0:
        _add_status(status, ws, stream, index)
    return dq, dk, dv, dg, dbeta, ds0


def kda_gdr_step(q, k, v, g, beta, state, scale=None, slots=None, out=None, status=None, stream=None):
    """Recurrent step for serving: q, k [B,T,H,K]; v [B,T,HV,V]; g, beta [B,T,HV] fp32;
    state [B,HV,K,V] fp32, updated in place, or with slots [B] int32 a pool
    [num_slots,HV,K,V] (a negative slot marks an empty row, whose o is 0).  status: a
    4-byte tensor the caller has zeroed, for a slot out of range.  Returns o [B,T,HV,V]."""
    lib, shape, addr, states, index, scale = _rule_args(q, k, v, g, beta, scale, None)
    if state is None or state.dim() != 4:
        raise KdaError(1, "state must be an fp32 tensor [B or num_slots, HV, K, V]")
    n, at = 0, None
    if slots is not None:
        at = _need("slots", slots, torch.int32, (states[0],), index)
        n = state.shape[0]
        states = (n, *states[1:])
    st = _need("state", state, _f32, states, index)
    written = (state,)
    if out is None:
        out = _allocators(stream, index)[1](v)
    else:
        _need("out", out, v.dtype, v.shape, index)
        written = (state, out)
    _check_status(status, index)
    _run(lib.kda_gdr_step, index, stream, shape, *addr, scale, st, at, n, out.data_ptr(), _ptr_or_none(status))
    if stream is not None:
        _lend(stream, index, q, k, v, g, beta, state, slots, out, status)
    _increment_version(written)
    return out


def _rows(name, x):
    """(rows, D, row stride) of x [..., D]: contiguous, or 2-D with dense rows."""
    if not x.is_cuda or x.dtype not in _IO or x.dim() < 1 or x.shape[-1] < 1:
        raise KdaError(1, f"{name} must be an fp32 or bf16 CUDA tensor [..., D], D >= 1")
    D = x.shape[-1]
    if x.is_contiguous():
        return x.numel() // D, D, D
    if x.dim() == 2 and x.stride(1) == 1 and x.stride(0) >= D:
        return x.shape[0], D, x.stride(0)
    raise KdaError(1, f"{name} must be contiguous, or [rows, D] with dense rows")


def kda_layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, out=None, output_stats=True, stream=None):
    """Layer norm over the last dimension of x [..., D] (bf16 or fp32; a 2-D x may have a row
    stride); weight, bias [D] fp32 or None.  Returns (y, mean, rstd): y like x, contiguous;
    mean and rstd fp32 in x's leading shape (None, None without output_stats)."""
    lib = _lib._lib or load_library()
    rows, D, ld = _rows("x", x)
    index = x.get_device()
    w, b = _maybe("weight", weight, _f32, (D,), index), _maybe("bias", bias, _f32, (D,), index)
    empty, empty_like = _allocators(stream, index)
    given = out
    if out is None:
        out = empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _need("out", out, x.dtype, x.shape, index)
    mean = rstd = None
    if output_stats:
        mean = empty(x.shape[:-1], dtype=_f32, device=x.device)
        rstd = empty_like(mean)
    _run(lib.kda_layer_norm_fwd, index, stream, rows, D, _IO[x.dtype], x.data_ptr(), ld, w, b, eps, out.data_ptr(),
         _ptr_or_none(mean), _ptr_or_none(rstd))
    if stream is not None:
        _lend(stream, index, x, weight, bias, out)
    if given is not None:
        _written(given)
    return out, mean, rstd


@functools.lru_cache(maxsize=256)
def _norm_workspace_bytes(rows, D, index):
    """The size on device `index` (a part for every block, and blocks go by the device's processors)."""
    with torch.cuda.device(index):
        return int(load_library().kda_layer_norm_bwd_workspace_size(rows, D))


def kda_layer_norm_bwd_workspace_size(rows: int, D: int) -> int:
    """Bytes for the current device."""
    return int(load_library().kda_layer_norm_bwd_workspace_size(rows, D))


def kda_layer_norm_bwd(x, dy, weight, mean, rstd, output_dx=True, output_dweight=True, output_dbias=True,
                       workspace=None, stream=None):
    """Gradients of kda_layer_norm_fwd from its x, mean and rstd.  Returns (dx, dweight,
    dbias): dx like x, contiguous; dweight and dbias [D] fp32; None where not asked for."""
    lib = _lib._lib or load_library()
    rows, D, ld = _rows("x", x)
    _, _, ldy = _rows("dy", dy)
    index = x.get_device()
    if dy.shape != x.shape or dy.dtype is not x.dtype or dy.get_device() != index:
        raise KdaError(1, "dy must have x's shape, dtype and device")
    lead = x.shape[:-1]
    w = _maybe("weight", weight, _f32, (D,), index)
    mu, rs = _need("mean", mean, _f32, lead, index), _need("rstd", rstd, _f32, lead, index)
    empty, _ = _allocators(stream, index)
    dx = empty(x.shape, dtype=x.dtype, device=x.device) if output_dx else None
    dw = empty(D, dtype=_f32, device=x.device) if output_dweight else None
    db = empty(D, dtype=_f32, device=x.device) if output_dbias else None
    if workspace is None:
        n = _norm_workspace_bytes(rows, D, index)
        workspace = empty(n, dtype=torch.uint8, device=x.device)
    else:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise KdaError(1, f"workspace must be contiguous on cuda:{index}")
        n = workspace.numel() * workspace.element_size()
    _run(lib.kda_layer_norm_bwd, index, stream, rows, D, _IO[x.dtype], x.data_ptr(), ld, dy.data_ptr(), ldy, w, mu, rs,
         _ptr_or_none(dx), _ptr_or_none(dw), _ptr_or_none(db), workspace.data_ptr(), n)
    if stream is not None:
        _lend(stream, index, x, dy, weight, mean, rstd, workspace)
    return dx, dw, db
