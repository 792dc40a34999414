"""A pre-norm layer on the gated linear recurrence: training and serving.

    python -m kimi_delta_attention_gb300.glr_layer [--steps 20]

Layer norm, projections (torch matrix products), the recurrence, group norm of its heads with SiLU and
the output projection, with a residual.  ``gated_linear_recurrence`` and ``group_norm`` are autograd
functions over the library's forward and backward (first derivatives; a second one raises);
``GatedRecurrentLayer`` trains with them, and serves with the forward for a prompt and the step for each
token after it, the requests' states in one pool.  The command trains a layer with the library's AdamW
for some steps on synthetic data, then serves the same tokens and compares.
"""
from __future__ import annotations

import argparse

import torch
from torch import nn
from torch.autograd.function import once_differentiable

from . import _glr
from ._lib import _check, kda_read_device_status
from .adamw import AdamW
from .gdr_layer import layer_norm


class _Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, g, initial_state, cu_seqlens, status):
        y, state = _glr.kda_glr_fwd(x, g, initial_state=initial_state, cu_seqlens=cu_seqlens, status=status)
        ctx.save_for_backward(g, y, initial_state, cu_seqlens)
        ctx.status = status
        ctx.set_materialize_grads(False)
        return y, state

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dstate):
        g, y, s0, cu = ctx.saved_tensors
        dy = torch.zeros_like(y) if dy is None else dy.contiguous()
        dx, dg, ds0 = _glr.kda_glr_bwd(g, y, dy, initial_state=s0, cu_seqlens=cu,
                                       d_final_state=None if dstate is None else dstate.contiguous(),
                                       output_d_initial_state=ctx.needs_input_grad[2], status=ctx.status)
        return dx, dg, ds0, None, None


def gated_linear_recurrence(x, g, initial_state=None, cu_seqlens=None, status=None):
    """Differentiable h_t = e^{g_t} h_{t-1} + x_t over [B, T, D]: (h in x's type, final states fp32).  x and g bf16
    or fp32; initial_state [NS, D] fp32; status: a zeroed 4-byte tensor to which the forward and the
    backward add the bits of their device status (kda_read_device_status(status)): after a
    cu_seqlens that does not end at T, results and gradients are not meaningful, and nothing else tells."""
    return _Recurrence.apply(x, g, initial_state, cu_seqlens, status)


class _GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, groups, weight, bias, eps, activation):
        y, mean, rstd = _glr.kda_group_norm_fwd(x, groups, weight, bias, eps, activation)
        ctx.save_for_backward(x, weight, bias, mean, rstd)
        ctx.groups, ctx.activation = groups, activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, bias, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = _glr.kda_group_norm_bwd(x, dy.contiguous(), ctx.groups, weight, bias, mean, rstd, ctx.activation,
                                             output_dx=need[0], output_dweight=need[2], output_dbias=need[3])
        return dx, None, dw, db, None, None


def group_norm(x, groups, weight=None, bias=None, eps=1e-5, activation="none"):
    """Differentiable group norm of x [N, ..., C], channels last, with an activation ("none" or "silu"): x bf16 or
    fp32, weight and bias fp32.  A 2-D x is the norm of heads, row by row."""
    return _GroupNorm.apply(x, groups, weight, bias, eps, activation)


class GatedRecurrentLayer(nn.Module):
    """x + W_o group_norm(recurrence(W_{u,r} layer_norm(x))) on bf16 activations [B, T, width], with heads of
    head_dim channels: g = -softplus(r + bias) / 8, the input sqrt(1 - e^{2 g}) u (so that the state keeps
    u's size), SiLU behind the norm."""

    def __init__(self, width, heads, head_dim=128, device="cuda"):
        super().__init__()
        D = heads * head_dim
        self.heads, self.channels = heads, D
        self.norm_weight = nn.Parameter(torch.ones(width, device=device))
        self.norm_bias = nn.Parameter(torch.zeros(width, device=device))
        self.gate_bias = nn.Parameter(torch.linspace(-4.0, 2.0, D, device=device))    # channels of long and of short memory
        self.head_weight = nn.Parameter(torch.ones(D, device=device))
        self.head_bias = nn.Parameter(torch.zeros(D, device=device))
        bf = dict(device=device, dtype=torch.bfloat16)
        self.w_in = nn.Parameter(torch.randn(width, 2 * D, **bf) * width ** -0.5)
        self.w_out = nn.Parameter(torch.randn(D, width, **bf) * D ** -0.5)

    def _project(self, x):
        u, r = (layer_norm(x, self.norm_weight, self.norm_bias) @ self.w_in).split(self.channels, dim=-1)
        g = -torch.nn.functional.softplus(r.float() + self.gate_bias) / 8
        # (a gate below -103 rounds to g = 0, where the root's slope is infinite: its argument stays a normal number)
        return (torch.sqrt((-torch.expm1(2 * g)).clamp_min(2.0 ** -126)) * u.float()).to(x.dtype), g

    def _finish(self, x, y):
        o = group_norm(y.reshape(-1, self.channels), self.heads, self.head_weight, self.head_bias, activation="silu")
        return x + o.view(*x.shape[:2], -1) @ self.w_out

    def forward(self, x, initial_state=None, cu_seqlens=None, status=None):
        """(y, final states [NS, heads head_dim]): a training pass, or a prompt's prefill under torch.no_grad();
        status as gated_linear_recurrence's."""
        u, g = self._project(x)
        h, state = gated_linear_recurrence(u, g, initial_state=initial_state, cu_seqlens=cu_seqlens, status=status)
        return self._finish(x, h), state

    @torch.no_grad()
    def step(self, x, pool, slots, status=None):
        """y of T new tokens (typically 1) of each request; its state is pool[slots[b]], updated in place (a negative
        slot: an empty row, whose y comes from a state of 0); status reports a slot out of range."""
        u, g = self._project(x)
        return self._finish(x, _glr.kda_glr_step(u.contiguous(), g.contiguous(), pool, slots=slots, status=status))


def demo(width=512, heads=4, B=4, T=200, steps=20, seed=0, state_bits=8):
    """Train on a fixed batch, then serve it: returns (first loss, last loss, worst difference of the served
    outputs from the whole forward's, relative to their largest)."""
    torch.manual_seed(seed)
    layer = GatedRecurrentLayer(width, heads)
    x = torch.randn(B, T, width, device="cuda").bfloat16()
    target = torch.roll(x, 1, dims=1)                    # recall the last token
    opt = AdamW(layer.parameters(), lr=3e-3, betas=(0.9, 0.95), weight_decay=0.0, state_bits=state_bits, masters=True)
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
        pool = torch.zeros(2 * B, state.shape[1], device="cuda")
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
