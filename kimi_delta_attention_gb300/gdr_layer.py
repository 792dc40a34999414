"""A pre-norm layer on the gated delta rule with a scalar gate: training and serving.

    python -m kimi_delta_attention_gb300.gdr_layer [--steps 20]

Layer norm, projections (torch matrix products), the delta rule and the output projection,
with a residual.  ``layer_norm`` and ``gated_delta_rule`` are autograd functions over the
library's forward and backward (first derivatives; a second one raises); ``GatedDeltaLayer``
trains with them, and serves with the chunked forward for a prompt and the recurrent step for
each token after it, the requests' states in one pool.  The command trains a layer with the library's
AdamW for some steps on synthetic data, then serves the same tokens and compares.
"""
from __future__ import annotations

import argparse

import torch
from torch import nn
from torch.autograd.function import once_differentiable

from . import _gdr
from ._lib import KdaError, _check, kda_read_device_status
from .adamw import AdamW


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = _gdr.kda_layer_norm_fwd(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.has_bias = bias is not None
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = _gdr.kda_layer_norm_bwd(x, dy.contiguous(), weight, mean, rstd, output_dx=need[0],
                                             output_dweight=need[1], output_dbias=ctx.has_bias and need[2])
        return dx, dw, db, None


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """Differentiable layer norm over the last dimension (x bf16 or fp32, weight and bias fp32)."""
    return _LayerNorm.apply(x, weight, bias, eps)


class _GatedDeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, scale, initial_state, cu_seqlens, status):
        o, state = _gdr.kda_gdr_fwd(q, k, v, g, beta, scale, initial_state=initial_state, cu_seqlens=cu_seqlens,
                                    status=status)
        ctx.save_for_backward(q, k, v, g, beta, initial_state, cu_seqlens)
        ctx.scale, ctx.status = scale, status
        return o, state

    @staticmethod
    @once_differentiable
    def backward(ctx, do, dstate):
        q, k, v, g, beta, s0, cu = ctx.saved_tensors
        grads = _gdr.kda_gdr_bwd(q, k, v, g, beta, do.contiguous(), ctx.scale, initial_state=s0, cu_seqlens=cu,
                                 d_final_state=dstate.contiguous(), output_d_initial_state=ctx.needs_input_grad[6],
                                 status=ctx.status)
        return (*grads[:5], None, grads[5], None, None)


def gated_delta_rule(q, k, v, g, beta, scale=None, initial_state=None, cu_seqlens=None, status=None):
    """Differentiable gated delta rule (bf16): (o, final states).  status: a zeroed 4-byte tensor
    to which the forward and the backward add the bits of their device status, read with
    kda_read_device_status(status) (which waits for the device) when the caller chooses: after a
    bounded wait that gave up or a cu_seqlens that does not end at T, results and gradients are
    not meaningful, and nothing else tells.  fp32 q, k and v have no gradients here: they
    raise where one would be recorded (kda_backward has them)."""
    if q.dtype != torch.bfloat16 and torch.is_grad_enabled() and any(
            t is not None and t.requires_grad for t in (q, k, v, g, beta, initial_state)):
        raise KdaError(2, "gradients of the gated delta rule need bf16 q, k and v")
    return _GatedDeltaRule.apply(q, k, v, g, beta, scale, initial_state, cu_seqlens, status)


class GatedDeltaLayer(nn.Module):
    """x + W_o delta_rule(W_{q,k,v,g,beta} layer_norm(x)) on bf16 activations [B, T, width].

    heads key heads serve value_heads value heads of head_dim each.  q and k are unit vectors
    per head, g = -softplus, beta = sigmoid of their projections (fp32)."""

    def __init__(self, width, heads, value_heads=None, head_dim=128, device="cuda"):
        super().__init__()
        hv = value_heads or heads
        self.heads, self.value_heads, self.head_dim = heads, hv, head_dim
        self.norm_weight = nn.Parameter(torch.ones(width, device=device))
        self.norm_bias = nn.Parameter(torch.zeros(width, device=device))
        self.split = [heads * head_dim, heads * head_dim, hv * head_dim, hv, hv]
        bf = dict(device=device, dtype=torch.bfloat16)
        self.w_in = nn.Parameter(torch.randn(width, sum(self.split), **bf) * width ** -0.5)
        self.w_out = nn.Parameter(torch.randn(hv * head_dim, width, **bf) * (hv * head_dim) ** -0.5)

    def _project(self, x):
        B, T, _ = x.shape
        h = layer_norm(x, self.norm_weight, self.norm_bias)
        q, k, v, g, b = (h @ self.w_in).split(self.split, dim=-1)
        unit = lambda t: torch.nn.functional.normalize(t.float().view(B, T, self.heads, self.head_dim), dim=-1).to(x.dtype)
        return (unit(q), unit(k), v.reshape(B, T, self.value_heads, self.head_dim).contiguous(),
                -torch.nn.functional.softplus(g.float()) / 8, torch.sigmoid(b.float()))

    def forward(self, x, initial_state=None, cu_seqlens=None, status=None):
        """(y, final states): a training pass, or a prompt's prefill under torch.no_grad();
        status as gated_delta_rule's."""
        o, state = gated_delta_rule(*self._project(x), initial_state=initial_state, cu_seqlens=cu_seqlens, status=status)
        return x + o.reshape(*x.shape[:2], -1) @ self.w_out, state

    @torch.no_grad()
    def step(self, x, pool, slots, status=None):
        """y of T new tokens (typically 1) of each request; its state is pool[slots[b]], updated
        in place (a negative slot: an empty row, y = x); status reports a slot out of range."""
        o = _gdr.kda_gdr_step(*(t.contiguous() for t in self._project(x)), pool, slots=slots, status=status)
        return x + o.reshape(*x.shape[:2], -1) @ self.w_out


def demo(width=512, heads=4, value_heads=8, B=4, T=200, steps=20, seed=0):
    """Train on a fixed batch, then serve it: returns (first loss, last loss, worst difference of
    the served outputs from the whole forward's, relative to their largest)."""
    torch.manual_seed(seed)
    layer = GatedDeltaLayer(width, heads, value_heads)
    x = torch.randn(B, T, width, device="cuda").bfloat16()
    target = torch.roll(x, 3, dims=1)                    # recall the token three back
    opt = AdamW(layer.parameters(), lr=3e-3, weight_decay=0.0)
    losses = []
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(steps):
        y, _ = layer(x, status=status)
        loss = (y.float() - target.float()).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    with torch.no_grad():
        whole, _ = layer(x, status=status)
        prompt = T - 8
        y, state = layer(x[:, :prompt].contiguous(), status=status)
        pool = torch.zeros(2 * B, *state.shape[1:], device="cuda")
        slots = torch.randperm(2 * B, device="cuda")[:B].to(torch.int32)
        pool[slots.long()] = state
        served = [y] + [layer.step(x[:, t:t + 1].contiguous(), pool, slots, status) for t in range(prompt, T)]
        _check(kda_read_device_status(status))
        off = (torch.cat(served, 1).float() - whole.float()).abs().max() / whole.float().abs().max()
    return losses[0], losses[-1], off.item()


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    from .builder import build
    build()
    first, last, off = demo(steps=a.steps)
    print(f"loss {first:.4f} -> {last:.4f} in {a.steps} steps; served against whole forward: {off:.2e} of the largest value")


if __name__ == "__main__":
    main()
