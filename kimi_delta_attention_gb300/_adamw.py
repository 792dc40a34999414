"""Binding of the AdamW step over many tensors (marshalling only).

Same manner as ``_gdr``.  A step may take hundreds of tensors, so the checks run over whole lists
at a time; addresses are read at every call and nothing is kept between calls.
"""
from __future__ import annotations

import itertools
import operator
import struct

import torch

from . import _lib
from ._gdr import _IO, _f32, _run
from ._lib import KdaAdamwConfig, KdaError, _increment_version, _lend, load_library

BLOCK = 256                   # values of a tensor that share a scale (KDA_ADAMW_BLOCK)
E4M3 = torch.float8_e4m3fn
_TYPES = set(_IO)


# (over whole lists these are a third faster than attribute by attribute)
_dtype, _device, _contiguous = operator.attrgetter("dtype"), torch.Tensor.get_device, torch.Tensor.is_contiguous
_numel, _address = torch.Tensor.numel, torch.Tensor.data_ptr


def _list(name, tensors, count, dtypes, index, sizes):
    """(addresses, types in use) of a list after its checks; `sizes`: how many values each has to hold."""
    if len(tensors) != count:
        raise KdaError(1, f"{name} must have one tensor for each of the {count} params")
    found = set(map(_dtype, tensors))
    if set(map(_device, tensors)) - {index} or not found <= dtypes or not all(map(_contiguous, tensors)) or \
            list(map(_numel, tensors)) != sizes:
        raise KdaError(1, f"{name} must be contiguous {' or '.join(map(str, dtypes))} tensors of the params' sizes on cuda:{index}")
    return list(map(_address, tensors)), found


def _kinds(tensors, found):
    """The kda_dtype of each tensor."""
    return itertools.repeat(_IO[next(iter(found))]) if len(found) == 1 else [_IO[t.dtype] for t in tensors]


def _word(name, t, dtype, index):
    """(host value, address of a device word): one of them."""
    if not torch.is_tensor(t):
        return t, None
    if t.get_device() != index or t.dtype is not dtype or t.numel() != 1:
        raise KdaError(1, f"{name} must be a number or one {dtype} value on cuda:{index}")
    return None, t.data_ptr()


def kda_adamw_step(params, grads, exp_avgs, exp_avg_sqs, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2,
                   masters=None, exp_avg_scales=None, exp_avg_sq_scales=None, seed=0, grad_scale=None, skip=None, stream=None):
    """One AdamW step, in place.  Lists of CUDA tensors: params and grads (bf16 or fp32 each); exp_avgs and
    exp_avg_sqs fp32, or float8_e4m3fn codes with exp_avg_scales and exp_avg_sq_scales (fp32, one
    for 256 values of a tensor); masters: fp32 copies that the step updates, params being those
    rounded (a list that may hold None, or None).  step counts from 1; seed: of the codes' rounding.  For
    captured steps: step (int32) and lr (fp32) may be device tensors, grad_scale (fp32: multiplies
    the gradients) and skip (fp32: not 0 leaves everything as it is) are device tensors or None."""
    lib = _lib._lib or load_library()
    params, grads, exp_avgs, exp_avg_sqs = list(params), list(grads), list(exp_avgs), list(exp_avg_sqs)
    masters, exp_avg_scales, exp_avg_sq_scales = (None if x is None else list(x) for x in (masters, exp_avg_scales, exp_avg_sq_scales))
    count = len(params)
    if count == 0:
        return
    index = params[0].get_device()
    if index < 0:
        raise KdaError(1, "params must be CUDA tensors")
    sizes = list(map(_numel, params))
    at_params, param_types = _list("params", params, count, _TYPES, index, sizes)
    at_grads, grad_types = _list("grads", grads, count, _TYPES, index, sizes)
    bits8 = exp_avg_scales is not None or exp_avg_sq_scales is not None
    of = {E4M3} if bits8 else {_f32}
    written = [*params, *exp_avgs, *exp_avg_sqs]
    columns = [at_params, at_grads, _list("exp_avgs", exp_avgs, count, of, index, sizes)[0],
               _list("exp_avg_sqs", exp_avg_sqs, count, of, index, sizes)[0]]
    if bits8:
        if exp_avg_scales is None or exp_avg_sq_scales is None:
            raise KdaError(1, "8-bit states need exp_avg_scales and exp_avg_sq_scales")
        blocks = [-(-n // BLOCK) for n in sizes]
        columns += [_list("exp_avg_scales", exp_avg_scales, count, {_f32}, index, blocks)[0],
                    _list("exp_avg_sq_scales", exp_avg_sq_scales, count, {_f32}, index, blocks)[0]]
        written += [*exp_avg_scales, *exp_avg_sq_scales]
    else:
        columns += [itertools.repeat(0)] * 2
    if masters is None:
        columns.append(itertools.repeat(0))
    else:
        have = [t for t in masters if t is not None]
        if len(masters) != count:
            raise KdaError(1, f"masters must have one entry for each of the {count} params")
        at = iter(_list("masters", have, len(have), {_f32}, index, [n for n, t in zip(sizes, masters) if t is not None])[0])
        columns.append([0 if t is None else next(at) for t in masters])
        written += have
    columns += [sizes, _kinds(params, param_types), _kinds(grads, grad_types)]
    table = struct.pack(f"={10 * count}q", *itertools.chain.from_iterable(zip(*columns)))
    step, step_at = _word("step", step, torch.int32, index)
    lr, lr_at = _word("lr", lr, _f32, index)
    gs, gs_at = _word("grad_scale", grad_scale, _f32, index)
    sk, sk_at = _word("skip", skip, _f32, index)
    if gs is not None or sk is not None:
        raise KdaError(1, "grad_scale and skip must be device tensors or None")
    config = KdaAdamwConfig(0.0 if lr is None else lr, betas[0], betas[1], eps, weight_decay, 0 if step is None else step,
                            seed & 0xFFFFFFFFFFFFFFFF, 8 if bits8 else 32, step_at, lr_at, gs_at, sk_at)
    _run(lib.kda_adamw_step, index, stream, table, count, config)
    if stream is not None:
        _lend(stream, index, *written, *grads, *(t for t in (step, lr, grad_scale, skip) if torch.is_tensor(t)))
    _increment_version(written)
