"""References in 64 bits for the gated delta rule with a scalar gate, and its tolerances.

The reference is the token recurrence itself (torch double on the CPU), its gradients by
autograd through that recurrence.

Tolerances, as the 2-norm of the error over the 2-norm of the reference:
  F32 = 1e-5.  The tensor-core kernels take an fp32 operand as two bf16 parts: the second
      part's rounding leaves at most 2^-18 of the value, the dropped low x low product as
      much again; six such products in a chain, uncorrelated, stay below 6 * 2^-18 / sqrt(3)
      = 1.3e-5 at worst and near 5e-6 in the mean.  The fp32 kernels are far below.
  BF16 = 2.4e-3: one rounding to bf16 is at most 2^-8 of a value, uniform in that interval
      and averaged over the mantissa 2^-8 / sqrt(3) / 1.47 = 1.54e-3 (1.7e-3 for values near
      a power of two), and the fp32 error above is nothing beside it.
Element by element: 2^-8 |ref| + 1e-3 rms(ref) for bf16, 8e-4 max(|ref|, rms(ref)) for fp32.
"""
from __future__ import annotations

import torch

F32, BF16 = 1e-5, 2.4e-3


def make(seqs, H, HV, K, V, io="bf16", seed=0, state=True, gate="soft", cu=None, grads=False):
    """CPU tensors of a packed (seqs a list of lengths) or batched (seqs = (B, T)) problem."""
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen)
    if isinstance(seqs, tuple):
        B, T = seqs
        ns, cu = B, None
    else:
        B, T, ns = 1, sum(seqs), len(seqs)
        cu = torch.tensor([0] + list(seqs)).cumsum(0).to(torch.int32)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dt)
    x = dict(q=unit(rn(B, T, H, K)), k=unit(rn(B, T, H, K)), v=rn(B, T, HV, V).to(dt))
    n = rn(B, T, HV)
    x["g"] = {"soft": torch.nn.functional.logsigmoid(n) / 8, "none": torch.zeros(B, T, HV),
              "strong": -5 * torch.sigmoid(n), "cliff": torch.where(n > 1.2, -300.0, -0.05)}[gate]
    x["beta"] = torch.sigmoid(rn(B, T, HV))
    x["s0"] = 0.1 * rn(ns, HV, K, V) if state else None
    x["cu"], x["scale"] = cu, K ** -0.5
    if grads:
        x["do"] = rn(B, T, HV, V).to(dt)
        x["ds"] = 0.1 * rn(ns, HV, K, V) if state else None
    return x


def cuda(x):
    return {n: t.cuda() if torch.is_tensor(t) else t for n, t in x.items()}


def spans(x):
    if x["cu"] is None:
        return [(b, 0, x["q"].shape[1]) for b in range(x["q"].shape[0])]
    cu = x["cu"].tolist()
    return [(0, a, b) for a, b in zip(cu, cu[1:])]


def reference(x, wrt=()):
    """(o, final states) in double; with `wrt`, the gradients of <do, o> + <ds, S> instead."""
    d = {n: (t.detach().cpu().double() if torch.is_tensor(t) and t.is_floating_point() else t) for n, t in x.items()}
    HV, V, K = x["v"].shape[2], x["v"].shape[3], x["q"].shape[3]
    sp = spans(x)
    if d["s0"] is None:
        d["s0"] = torch.zeros(len(sp), HV, K, V, dtype=torch.float64)
    for n in wrt:
        d[n].requires_grad_()
    G = HV // x["q"].shape[2]
    q, k = d["q"].repeat_interleave(G, 2), d["k"].repeat_interleave(G, 2)
    o, S_all, loss = [], [], 0.0
    for i, (b, t0, t1) in enumerate(sp):
        S = d["s0"][i]
        rows = []
        for t in range(t0, t1):
            S = S * torch.exp(d["g"][b, t])[:, None, None]
            err = d["beta"][b, t][:, None] * (d["v"][b, t] - torch.einsum("hkv,hk->hv", S, k[b, t]))
            S = S + k[b, t][:, :, None] * err[:, None, :]
            rows.append(x["scale"] * torch.einsum("hkv,hk->hv", S, q[b, t]))
        out = torch.stack(rows) if rows else torch.zeros(0, HV, V, dtype=torch.float64)
        if wrt:
            loss = loss + (out * d["do"][b, t0:t1]).sum()
            if d.get("ds") is not None:
                loss = loss + (S * d["ds"][i]).sum()
        o.append(out)
        S_all.append(S)
    if wrt:
        got = torch.autograd.grad(loss, [d[n] for n in wrt], allow_unused=True)
        return [torch.zeros_like(d[n]) if r is None else r for n, r in zip(wrt, got)]
    o = torch.cat(o).reshape(x["v"].shape) if x["cu"] is not None else torch.stack(o)
    return o.detach(), torch.stack(S_all).detach()


def check(got, ref, what):
    got = got.detach().cpu()
    bf16 = got.dtype == torch.bfloat16
    got = got.double()
    assert got.shape == ref.shape, what
    assert torch.isfinite(got).all(), f"{what}: not finite"
    if ref.numel() == 0:
        return
    norm = ref.norm().item()
    rms = norm / ref.numel() ** 0.5
    err = (got - ref).abs()
    assert err.norm().item() <= (BF16 if bf16 else F32) * norm + 1e-30, f"{what}: {err.norm().item() / max(norm, 1e-300):.3e}"
    bound = 2.0 ** -8 * ref.abs() + 1e-3 * rms if bf16 else 8e-4 * ref.abs().clamp_min(rms)
    assert (err <= bound + 1e-30).all(), f"{what}: element off by {(err - bound).max().item():.3e}"
