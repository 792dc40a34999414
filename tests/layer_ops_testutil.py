"""References in 64 bits of the gated linear recurrence, group norm and the AdamW step, and how far
an fp32 evaluation may be from them.

Recurrence, element by element: with u = 2^-24, an exponential is good to 4 u, and each token multiplies and
adds with a few roundings wherever a kernel joins its pieces: 8 u of e^g |h| and 2 u of the sum
cover them.  These errors decay and add up as the values do, so the reference carries
    B_t = e^g B_{t-1} + |x_t|,   E_t = e^g E_{t-1} + 8 u e^g B_{t-1} + 2 u B_t
beside h_t, and a result may be E_t off, rounded once to its type (bf16: 2^-8 of it).
"""
from __future__ import annotations

import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounded(err, value, dtype):
    """The bound with one rounding to dtype on top (and a subnormal's absolute step)."""
    return err + half_step(dtype) * (value.abs() + err) + 1e-37


def rows(t, lengths):
    """[longest, sequences, D] in fp64; zeros behind a sequence's end."""
    return torch.nn.utils.rnn.pad_sequence(torch.split(t.reshape(-1, t.shape[-1]).double(), lengths)) if max(lengths) else \
        torch.zeros(0, len(lengths), t.shape[-1], dtype=torch.float64, device=t.device)


def back(r, lengths, shape):
    return torch.cat([r[:n, i] for i, n in enumerate(lengths)]).reshape(shape)


def make_glr(lengths, D, io=torch.float32, gate=torch.float32, state=True, packed=True, seed=0, device="cuda", rates=(1e-3, 2.0)):
    """lengths: tokens of each sequence (all alike where not packed)."""
    gen = torch.Generator(device=device).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen, device=device)
    B, T, ns = (1, sum(lengths), len(lengths)) if packed else (len(lengths), lengths[0], len(lengths))
    lo, hi = torch.tensor(rates, device=device).log()
    rate = torch.exp(lo + (hi - lo) * torch.rand(D, generator=gen, device=device))
    d = dict(g=(-rate * torch.sigmoid(rn(B, T, D))).to(gate), x=rn(B, T, D).to(io), dy=rn(B, T, D).to(io))
    d["s0"] = rn(ns, D) if state else None
    d["ds"] = rn(ns, D) if state else None
    d["cu"] = torch.tensor([0] + list(lengths), device=device).cumsum(0).to(torch.int32) if packed else None
    return d


def glr_reference(x, g, s0, lengths):
    """(y, its bound, final states, theirs) before any rounding to the output's type."""
    xs, es = rows(x, lengths), rows(g, lengths).exp()
    n = torch.tensor(lengths, device=x.device)
    h = torch.zeros(len(lengths), x.shape[-1], dtype=torch.float64, device=x.device) if s0 is None else s0.double()
    B, E = h.abs(), torch.zeros_like(h)
    y, err = torch.empty_like(xs), torch.empty_like(xs)
    for t in range(xs.shape[0]):
        live = (t < n)[:, None]
        grown = es[t] * B + xs[t].abs()
        E = torch.where(live, es[t] * E + 8 * U * es[t] * B + 2 * U * grown, E)
        h, B = torch.where(live, es[t] * h + xs[t], h), torch.where(live, grown, B)
        y[t], err[t] = h, E
    return back(y, lengths, x.shape), back(err, lengths, x.shape), h, E


def glr_bwd_reference(g, y, dy, s0, dfin, lengths):
    """Likewise (dx, bound, dg, bound, d_initial, bound)."""
    es, ys, ds = rows(g, lengths).exp(), rows(y, lengths), rows(dy, lengths)
    n = torch.tensor(lengths, device=y.device)
    zero = torch.zeros(len(lengths), y.shape[-1], dtype=torch.float64, device=y.device)
    first = zero if s0 is None else s0.double()
    mu = zero if dfin is None else dfin.double()
    B, E = mu.abs(), torch.zeros_like(mu)
    dx, dg, ex, eg = (torch.empty_like(ds) for _ in range(4))
    for t in range(ds.shape[0] - 1, -1, -1):
        live = (t < n)[:, None]
        dx[t], ex[t] = mu + ds[t], E + 2 * U * (B + ds[t].abs())
        grown = es[t] * (B + ds[t].abs())
        E = torch.where(live, es[t] * E + 10 * U * grown, E)
        mu, B = torch.where(live, es[t] * dx[t], mu), torch.where(live, grown, B)
        before = ys[t - 1] if t else first
        dg[t], eg[t] = mu * before, (E + 2 * U * B) * before.abs()
    shape = y.shape
    return back(dx, lengths, shape), back(ex, lengths, shape), back(dg, lengths, shape), back(eg, lengths, shape), mu, E


def within(got, ref, err, what):
    """got is ref to within err and one rounding to its type."""
    assert got.shape == ref.shape, what
    off = (got.double() - ref).abs()
    bound = rounded(err, ref, got.dtype)
    bad = ~(off <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, the worst by {(off / bound)[bad].max().item():.3g} times its bound"


def gn_reference(x, groups, w, b, eps, act):
    """(y, mean, rstd) in fp64 of x [N, ..., C]."""
    N, C = x.shape[0], x.shape[-1]
    d = x.double().reshape(N, -1, groups, C // groups)
    mean = d.mean(dim=(1, 3))
    var = (d - mean[:, None, :, None]).square().mean(dim=(1, 3))
    rstd = (var + eps) ** -0.5
    z = ((d - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(x.shape)
    z = z if w is None else z * w.double()
    z = z if b is None else z + b.double()
    return z * torch.sigmoid(z) if act == "silu" else z, mean, rstd


def gn_bwd_reference(x, dy, groups, w, b, mean, rstd, act):
    """(dx, dweight, dbias) in fp64, and the sums of the terms' magnitudes of each.  The slope of silu
    s (1 + z (1 - s)) cancels where z is near -1.28: an evaluation is good to some roundings of s (1 + |z| (1 - s)),
    so the terms take the slope by that magnitude."""
    N, C = x.shape[0], x.shape[-1]
    wide = lambda s: s.double()[:, None, :, None]
    xh = (x.double().reshape(N, -1, groups, C // groups) - wide(mean)) * wide(rstd)
    wd = torch.ones(C, dtype=torch.float64, device=x.device) if w is None else w.double()
    z = xh.reshape(N, -1, C) * wd + (0 if b is None else b.double())
    s = torch.sigmoid(z)
    dz = size = dy.double().reshape(N, -1, C)
    if act == "silu":
        dz, size = dz * s * (1 + z * (1 - s)), dz * s * (1 + z.abs() * (1 - s))
    a, big = (dz * wd).reshape(xh.shape), (size * wd).reshape(xh.shape).abs()
    m = lambda t: t.mean(dim=(1, 3), keepdim=True)
    dx = wide(rstd) * (a - m(a) - xh * m(a * xh))
    terms = wide(rstd) * (big + m(big) + xh.abs() * m(big * xh.abs()))
    flat = xh.reshape(N, -1, C)
    return (dx.reshape(x.shape), (dz * flat).sum((0, 1)), dz.sum((0, 1))), \
        (terms.reshape(x.shape), (size * flat).abs().sum((0, 1)), size.abs().sum((0, 1)))
