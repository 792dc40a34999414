"""Binding of the gated delta rule with a scalar gate and of layer norm (marshalling only).

Same manner as ``_lib``: contiguous CUDA tensors in, outputs allocated by torch when the
caller passes none, a KdaError on a non-OK status, no fallback.  These calls also serve
single tokens, where the host's own time counts: the checks are plain attribute reads and
the device is only switched when it is not the current one.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import KDA_BF16, KDA_F32, KdaError, KdaShape, _check, load_library

_IO = {torch.float32: KDA_F32, torch.bfloat16: KDA_BF16}
_f32 = torch.float32


def _need(name, t, dtype, shape, device):
    """An optional tensor's address after its checks (None stays None)."""
    if t is None:
        return None
    if t.device != device or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise KdaError(1, f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on {device}")
    return t.data_ptr()


def _stream(device, stream):
    current = torch._C._cuda_getCurrentRawStream(device.index)
    return (current if stream is None else stream), current


def _keep(made, stream, current, device):
    """Blocks allocated on the current stream's pool but used on another stream must not be
    handed out again before that stream is done with them."""
    if stream != current:
        other = torch.cuda.ExternalStream(stream, device=device)
        for t in made:
            if t is not None:
                t.record_stream(other)


def _on(device):
    return torch.cuda.device(device) if device.index != torch.cuda.current_device() else _here


class _Here:
    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_here = _Here()


def _rule_args(q, k, v, g, beta, scale, cu_seqlens):
    """The checks every delta-rule call shares; (shape struct, addresses, NS, device, scale)."""
    device, io = q.device, q.dtype
    if not q.is_cuda or io not in _IO:
        raise KdaError(1, "q must be an fp32 or bf16 CUDA tensor")
    if q.dim() != 4 or v.dim() != 4:
        raise KdaError(1, "q must be [B, T, H, K] and v [B, T, HV, V]")
    B, T, H, K = q.shape
    HV, V = v.shape[2], v.shape[3]
    gate = (B, T, HV)
    addr = (_need("q", q, io, q.shape, device), _need("k", k, io, q.shape, device),
            _need("v", v, io, (B, T, HV, V), device), _need("g", g, _f32, gate, device),
            _need("beta", beta, _f32, gate, device))
    ns = 0
    if cu_seqlens is not None:
        ns = cu_seqlens.numel() - 1
        _need("cu_seqlens", cu_seqlens, torch.int32, (ns + 1,), device)
    return KdaShape(B, T, H, HV, K, V, ns, _IO[io]), addr, (B if cu_seqlens is None else ns), device, \
        (K ** -0.5 if scale is None else scale)


def _ptr_or_none(t):
    return None if t is None else t.data_ptr()


def kda_gdr_fwd_workspace_size(shape: KdaShape) -> int:
    return int(load_library().kda_gdr_fwd_workspace_size(ctypes.byref(shape)))


def kda_gdr_fwd(q, k, v, g, beta, scale=None, initial_state=None, cu_seqlens=None, out=None, final_state=None,
                output_final_state=True, workspace=None, stream=None):
    """Forward of the gated delta rule with a scalar gate.  q, k [B,T,H,K]; v [B,T,HV,V];
    g (log decay), beta [B,T,HV] fp32; initial_state [NS,HV,K,V] fp32; cu_seqlens [N+1]
    int32 (packed sequences, B = 1).  Returns (o [B,T,HV,V], final_state or None)."""
    lib = _lib._lib or load_library()
    shape, addr, ns, device, scale = _rule_args(q, k, v, g, beta, scale, cu_seqlens)
    states = (ns, shape.HV, shape.K, shape.V)
    s0 = _need("initial_state", initial_state, _f32, states, device)
    made = []
    if out is None:
        out = torch.empty_like(v)
        made.append(out)
    else:
        _need("out", out, v.dtype, v.shape, device)
    if final_state is not None:
        _need("final_state", final_state, _f32, states, device)
    elif output_final_state:
        final_state = torch.empty(states, dtype=_f32, device=device)
        made.append(final_state)
    ref = ctypes.byref(shape)
    if workspace is None:
        workspace = torch.empty(lib.kda_gdr_fwd_workspace_size(ref) or 256, dtype=torch.uint8, device=device)
        made.append(workspace)
    elif workspace.device != device or not workspace.is_contiguous():
        raise KdaError(1, f"workspace must be contiguous on {device}")
    stream, current = _stream(device, stream)
    with _on(device):
        _check(lib.kda_gdr_fwd(ref, *addr, scale, s0, _ptr_or_none(cu_seqlens), out.data_ptr(),
                               _ptr_or_none(final_state), workspace.data_ptr(),
                               workspace.numel() * workspace.element_size(), stream))
    _keep(made, stream, current, device)
    return out, final_state


def kda_gdr_bwd_workspace_size(shape: KdaShape) -> int:
    return int(load_library().kda_gdr_bwd_workspace_size(ctypes.byref(shape)))


def kda_gdr_bwd(q, k, v, g, beta, d_out, scale=None, initial_state=None, cu_seqlens=None, d_final_state=None,
                output_d_initial_state=True, workspace=None, stream=None):
    """Gradients of sum <d_out, o> + <d_final_state, S_final> for kda_gdr_fwd with the same
    arguments (bf16).  Returns (dq, dk, dv, dg, dbeta, d_initial_state): dq, dk, dv bf16,
    the others fp32, in the inputs' shapes."""
    lib = _lib._lib or load_library()
    shape, addr, ns, device, scale = _rule_args(q, k, v, g, beta, scale, cu_seqlens)
    states = (ns, shape.HV, shape.K, shape.V)
    s0 = _need("initial_state", initial_state, _f32, states, device)
    do = _need("d_out", d_out, v.dtype, v.shape, device)
    dfin = _need("d_final_state", d_final_state, _f32, states, device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, dbeta = torch.empty_like(g), torch.empty_like(beta)
    ds0 = torch.empty(states, dtype=_f32, device=device) if output_d_initial_state else None
    made = [dq, dk, dv, dg, dbeta, ds0]
    ref = ctypes.byref(shape)
    if workspace is None:
        workspace = torch.empty(lib.kda_gdr_bwd_workspace_size(ref) or 256, dtype=torch.uint8, device=device)
        made.append(workspace)
    elif workspace.device != device or not workspace.is_contiguous():
        raise KdaError(1, f"workspace must be contiguous on {device}")
    stream, current = _stream(device, stream)
    with _on(device):
        _check(lib.kda_gdr_bwd(ref, *addr, scale, s0, _ptr_or_none(cu_seqlens), do, dfin, dq.data_ptr(), dk.data_ptr(),
                               dv.data_ptr(), dg.data_ptr(), dbeta.data_ptr(), _ptr_or_none(ds0), workspace.data_ptr(),
                               workspace.numel() * workspace.element_size(), stream))
    _keep(made, stream, current, device)
    return dq, dk, dv, dg, dbeta, ds0


def kda_gdr_step(q, k, v, g, beta, state, scale=None, slots=None, out=None, status=None, stream=None):
    """Recurrent step for serving: q, k [B,T,H,K]; v [B,T,HV,V]; g, beta [B,T,HV] fp32;
    state [B,HV,K,V] fp32, updated in place, or with slots [B] int32 a pool
    [num_slots,HV,K,V] (a negative slot marks an empty row, whose o is 0).  status: a
    4-byte tensor the caller has zeroed, for a slot out of range.  Returns o [B,T,HV,V]."""
    lib = _lib._lib or load_library()
    shape, addr, ns, device, scale = _rule_args(q, k, v, g, beta, scale, None)
    if state is None or state.dim() != 4:
        raise KdaError(1, "state must be an fp32 tensor [B or num_slots, HV, K, V]")
    n = state.shape[0] if slots is not None else ns
    st = _need("state", state, _f32, (n, shape.HV, shape.K, shape.V), device)
    made = []
    if out is None:
        out = torch.empty_like(v)
        made.append(out)
    else:
        _need("out", out, v.dtype, v.shape, device)
    if status is not None and (status.device != device or status.numel() * status.element_size() < 4):
        raise KdaError(1, f"status must hold 4 bytes on {device}")
    stream, current = _stream(device, stream)
    with _on(device):
        _check(lib.kda_gdr_step(ctypes.byref(shape), *addr, scale, st,
                                _need("slots", slots, torch.int32, (ns,), device), n if slots is not None else 0,
                                out.data_ptr(), _ptr_or_none(status), stream))
    _keep(made, stream, current, device)
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
    device = x.device
    w, b = _need("weight", weight, _f32, (D,), device), _need("bias", bias, _f32, (D,), device)
    made = []
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=device)
        made.append(out)
    else:
        _need("out", out, x.dtype, x.shape, device)
    mean = rstd = None
    if output_stats:
        mean = torch.empty(x.shape[:-1], dtype=_f32, device=device)
        rstd = torch.empty(x.shape[:-1], dtype=_f32, device=device)
        made += [mean, rstd]
    stream, current = _stream(device, stream)
    with _on(device):
        _check(lib.kda_layer_norm_fwd(rows, D, _IO[x.dtype], x.data_ptr(), ld, w, b, eps, out.data_ptr(),
                                      _ptr_or_none(mean), _ptr_or_none(rstd), stream))
    _keep(made, stream, current, device)
    return out, mean, rstd


def kda_layer_norm_bwd_workspace_size(rows: int, D: int) -> int:
    return int(load_library().kda_layer_norm_bwd_workspace_size(rows, D))


def kda_layer_norm_bwd(x, dy, weight, mean, rstd, output_dx=True, output_dweight=True, output_dbias=True,
                       workspace=None, stream=None):
    """Gradients of kda_layer_norm_fwd from its x, mean and rstd.  Returns (dx, dweight,
    dbias): dx like x, contiguous; dweight and dbias [D] fp32; None where not asked for."""
    lib = _lib._lib or load_library()
    rows, D, ld = _rows("x", x)
    rows_y, D_y, ldy = _rows("dy", dy)
    device = x.device
    if dy.shape != x.shape or dy.dtype != x.dtype or dy.device != device:
        raise KdaError(1, "dy must have x's shape, dtype and device")
    lead = x.shape[:-1]
    w = _need("weight", weight, _f32, (D,), device)
    mu, rs = _need("mean", mean, _f32, lead, device), _need("rstd", rstd, _f32, lead, device)
    dx = torch.empty(x.shape, dtype=x.dtype, device=device) if output_dx else None
    dw = torch.empty(D, dtype=_f32, device=device) if output_dweight else None
    db = torch.empty(D, dtype=_f32, device=device) if output_dbias else None
    made = [dx, dw, db]
    if workspace is None:
        workspace = torch.empty(lib.kda_layer_norm_bwd_workspace_size(rows, D), dtype=torch.uint8, device=device)
        made.append(workspace)
    elif workspace.device != device or not workspace.is_contiguous():
        raise KdaError(1, f"workspace must be contiguous on {device}")
    stream, current = _stream(device, stream)
    with _on(device):
        _check(lib.kda_layer_norm_bwd(rows, D, _IO[x.dtype], x.data_ptr(), ld, dy.data_ptr(), ldy, w, mu, rs,
                                      _ptr_or_none(dx), _ptr_or_none(dw), _ptr_or_none(db), workspace.data_ptr(),
                                      workspace.numel() * workspace.element_size(), stream))
    _keep(made, stream, current, device)
    return dx, dw, db
