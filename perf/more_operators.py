"""Cases, plain forms and 64-bit references of the gated linear recurrence (forward, backward,
serving step), of group norm with an activation (forward, backward) and of the AdamW step over
many tensors.

A case is a dict of plain values; ``prepare`` draws its inputs from a seed, ``run`` makes one
pass (the plain torch form, or with ``own`` the library's entry points) and ``exact`` gives the
same outputs in fp64 from the definitions.

Recurrence, per sequence and channel:   h_t = e^{g_t} h_{t-1} + x_t,   y_t = h_t
    back: mu_t = e^{g_t} lam_t, lam_t = dy_t + mu_{t+1} (the last token's: dy + d_final);
    dx = lam, dg_t = mu_t h_{t-1} (h from the forward's y), d_initial = mu of the first token.
Group norm, per sample and group over its L positions and C / groups channels:
    xh = (x - mean) rstd, z = xh weight + bias, y = z or z sigmoid(z); biased variance.
AdamW: m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2,
    p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps).
    States in 8 bits: e4m3 codes of 256 values with an fp32 scale (their largest magnitude / 448),
    rounded up or down at random in proportion, by numbers that the seed and the step give; a v
    above 0 keeps a code above 0.
"""
import itertools
import math

import torch

own = False

EPS = 1e-5
BLOCK = 256                    # values of a tensor that share a scale
B1, B2, ADAM_EPS, LR, DECAY = 0.9, 0.99, 1e-8, 1e-3, 0.01


# ------------------------------------------------------------------- cases --
def _layer(width, heads, value_heads, dim=128):
    """Sizes of a delta layer's tensors: norm's weight and bias, input and output projections."""
    return [width, width, width * (2 * heads * dim + value_heads * dim + 2 * value_heads), value_heads * dim * width]


def listed():
    return [
        # a short prompt: all latency
        dict(name="glr_prompt37", op="glr", B=1, T=37, D=1024, io="bf16", gate="f32", state=False, lengths=""),
        # one sequence at this library's headline length and width (32 heads of 128)
        dict(name="glr_T4096_D4096", op="glr", B=1, T=4096, D=4096, io="bf16", gate="f32", state=False, lengths=""),
        # continuous prefill: 16 packed sequences of 1 to 8192 tokens, states carried in
        dict(name="glr_packed16", op="glr", B=1, T=0, D=2048, io="bf16", gate="bf16", state=True,
             lengths="1 8192 777 64 3001 129 5120 6000 63 2048 7013 4097 65 1500 7999 333"),
        # 128 requests' next tokens, their states in a pool, two rows empty
        dict(name="glr_step_B128", op="glr_step", B=128, T=1, D=4096, io="bf16", gate="f32", slots=259),
        # a training step on ragged packed samples, an odd width in fp32
        dict(name="glr_bwd_packed_odd", op="glr_bwd", B=1, T=0, D=1001, io="f32", gate="f32", state=True,
             lengths="300 1 511 188"),
        # a training step at the headline length
        dict(name="glr_bwd_B4_T4096", op="glr_bwd", B=4, T=4096, D=4096, io="bf16", gate="f32", state=False, lengths=""),
        # the heads' norm and gate over a training batch's rows (one position a sample)
        dict(name="gn_rows16384", op="gn", N=16384, L=1, C=4096, groups=32, io="bf16", act="silu", affine=True),
        # whole samples, groups over all their positions
        dict(name="gn_samples4", op="gn", N=4, L=4096, C=4096, groups=32, io="bf16", act="none", affine=True),
        # the heads' norm backward
        dict(name="gn_bwd_rows16384", op="gn_bwd", N=16384, L=1, C=4096, groups=32, io="bf16", act="silu", affine=True),
        # a few positions of odd groups in fp32
        dict(name="gn_bwd_odd", op="gn_bwd", N=3, L=77, C=1001, groups=7, io="f32", act="silu", affine=True),
        # one small layer's tensors, everything in fp32
        dict(name="adamw_layer", op="adamw", sizes=" ".join(map(str, _layer(512, 4, 8))), io="f32", bits=32, master=False,
             step=7),
        # 24 layers' tensors in bf16, states in 8 bits
        dict(name="adamw8_layers24", op="adamw", sizes=" ".join(map(str, _layer(2048, 16, 16) * 24)), io="bf16", bits=8,
             master=False, step=1000),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["glr", "glr", "glr_step", "glr_bwd", "glr_bwd", "gn", "gn", "gn_bwd", "gn_bwd", "adamw", "adamw"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op == "adamw":
        # 1 to 200 tensors, from biases to projections
        sizes = [_log_int(rng, 1, 1 << 22) for _ in range(_log_int(rng, 1, 200))]
        return dict(op=op, sizes=" ".join(map(str, sizes)), io=io, bits=rng.choice([8, 32]),
                    master=io == "bf16" and rng.random() < 0.5, step=_log_int(rng, 1, 100000))
    if op in ("gn", "gn_bwd"):
        C = _log_int(rng, 8, 8192)
        groups = rng.choice([d for d in range(1, min(C, 128) + 1) if C % d == 0])
        n = _log_int(rng, 1, (1 << 25) // C)                      # positions in all
        L = rng.choice([1, _log_int(rng, 1, n)])
        return dict(op=op, N=max(1, n // L), L=L, C=C, groups=groups, io=io, act=rng.choice(["silu", "silu", "none"]),
                    affine=rng.random() < 0.8)
    gate = "bf16" if io == "bf16" and rng.random() < 0.4 else "f32"
    if op == "glr_step":
        B = _log_int(rng, 1, 256)
        return dict(op=op, B=B, T=rng.choice([1, 1, 1, 2, 3, 5]), D=_log_int(rng, 1, 8192), io=io, gate=gate,
                    slots=rng.choice([0, 2 * B + 3]))
    D = rng.choice([_log_int(rng, 1, 8192), 64 * _log_int(rng, 1, 128)])
    tokens = _log_int(rng, 1, min(131072, (1 << 25) // D))
    B, T, lengths = 1, 0, ""
    if rng.random() < 0.5:
        n = rng.choice([1, 2, 3, 5, 8, 13, 200])                  # (some of no token)
        cuts = sorted(rng.randrange(tokens + 1) for _ in range(n - 1))
        lengths = " ".join(str(b - a) for a, b in zip([0] + cuts, cuts + [tokens]))
    else:
        B = rng.choice([1, 1, 2, 3, 7])
        T = max(1, tokens // B)
    return dict(op=op, B=B, T=T, D=D, io=io, gate=gate, state=rng.random() < 0.5, lengths=lengths)


def _lengths(case):
    return [int(x) for x in case["lengths"].split()] if case.get("lengths") else [case["T"]] * case["B"]


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


# ------------------------------------------------------------------ inputs --
def prepare(case, seed):
    """The tensors a caller holds before the call."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    rn = lambda *s: torch.randn(*s, generator=gen, device=dev)
    ru = lambda *s: torch.rand(*s, generator=gen, device=dev)
    st = {"case": case}
    dt = _dtype(case["io"])
    if case["op"] in ("gn", "gn_bwd"):
        N, L, C, G = (case[n] for n in ("N", "L", "C", "groups"))
        st["x"] = (1.5 * rn(N, L, C) + 0.3).to(dt)
        st["w"] = 1.0 + 0.2 * rn(C) if case["affine"] else None
        st["b"] = 0.1 * rn(C) if case["affine"] else None
        if case["op"] == "gn_bwd":
            st["dy"] = rn(N, L, C).to(dt)
            x = st["x"].float().view(N, L, G, C // G)             # what the forward pass has kept
            st["mean"] = x.mean(dim=(1, 3))
            st["rstd"] = torch.rsqrt((x - st["mean"][:, None, :, None]).square().mean(dim=(1, 3)) + EPS)
        return st
    if case["op"] == "adamw":
        sizes = [int(n) for n in case["sizes"].split()]
        # every tensor a view into one storage, each from a multiple of 256 values on
        blocks = [-(-n // BLOCK) for n in sizes]
        *starts, total = itertools.accumulate((BLOCK * k for k in blocks), initial=0)
        split = lambda flat: [flat[a:a + n] for a, n in zip(starts, sizes)]
        real = torch.zeros(total, dtype=torch.bool, device=dev)
        for r in split(real):
            r.fill_(True)
        fill = lambda t: torch.where(real, t, torch.zeros_like(t))
        st["sizes"], st["blocks"] = sizes, blocks
        flat = st["flat"] = {}
        scale = 10.0 ** (-1 - 3 * ru(total // BLOCK)).repeat_interleave(BLOCK)     # gradients of many magnitudes
        p, g = fill(0.02 * rn(total)), fill(scale * rn(total))
        m, v = fill(0.3 * scale * rn(total)), fill(scale * scale * (0.1 + rn(total).square()))
        flat["params"], flat["grads"] = p.to(dt), g.to(dt)
        if case["master"]:
            flat["masters"] = p
        if case["bits"] == 8:
            zero = torch.full((total // BLOCK, BLOCK), 0.5, device=dev)
            flat["m"], flat["m_scale"] = _quantise(m.view(-1, BLOCK), zero, False)
            flat["v"], flat["v_scale"] = _quantise(v.view(-1, BLOCK), zero, True)
        else:
            flat["m"], flat["v"] = m, v
        st["lists"] = {n: split(flat[n].view(-1)) for n in flat if not n.endswith("scale")}
        for n in ("m_scale", "v_scale"):
            if n in flat:
                st["lists"][n] = [flat[n][a // BLOCK:a // BLOCK + k] for a, k in zip(starts, blocks)]
        st["seed"] = int(seed) * 7919 + 17
        return st
    D = case["D"]
    lengths = _lengths(case)
    packed = bool(case.get("lengths"))
    B, T = (1, sum(lengths)) if packed else (case["B"], case["T"])
    rate = torch.exp(math.log(1e-3) * ru(D))                      # channels of long and of short memory
    g = (-2 * rate * torch.sigmoid(rn(B, T, D))).to(_dtype(case["gate"]))
    x = ((1 - torch.exp(2 * g.float())).sqrt() * rn(B, T, D)).to(dt)
    st["g"] = g
    if case["op"] == "glr_step":
        n = case["slots"]
        st["x"], st["state"], st["slots"] = x, rn(n or B, D), None
        if n:
            slots = torch.randperm(n, generator=gen, device=dev)[:B].to(torch.int32)
            if B >= 4:                                            # padding rows of a fixed-size batch
                slots[B // 3] = -1
                slots[B - 1] = -1
            st["slots"] = slots
        return st
    st["cu"] = torch.tensor([0] + lengths, device=dev).cumsum(0).to(torch.int32) if packed else None
    ns = len(lengths)
    st["s0"] = rn(ns, D) if case["state"] else None
    if case["op"] == "glr":
        st["x"] = x
        return st
    st["x"] = x
    st["y"] = _plain_glr(st)["y"]                                 # what the forward pass has kept
    del st["x"]
    st["dy"] = rn(B, T, D).to(dt)
    st["dfin"] = rn(ns, D) if case["state"] else None
    return st


# --------------------------------------------------------- the plain forms --
def _ends(st):
    """First and last tokens of the sequences that have tokens, which ones those are, and the longest."""
    lengths = _lengths(st["case"])
    n = torch.tensor(lengths, device=st["g"].device)
    last = n.cumsum(0) - 1
    live = n > 0
    return (last - n + 1)[live], last[live], live.nonzero()[:, 0], max(lengths)


def _scan(a, x, longest):
    """h_t = a_t h_{t-1} + x_t along dim 0 by doubling (a is 0 where a sequence starts); in place."""
    s = 1
    while s < longest:
        x[s:] += a[s:] * x[:-s]
        a[s:] = a[s:] * a[:-s]
        s *= 2
    return x


def _plain_glr(st):
    D = st["case"]["D"]
    first, last, seqs, longest = _ends(st)
    a = torch.exp(st["g"].float().reshape(-1, D))
    h = st["x"].float().reshape(-1, D).clone()
    if st["s0"] is not None:
        h[first] += a[first] * st["s0"][seqs]
    a[first] = 0
    h = _scan(a, h, longest)
    ns = len(_lengths(st["case"]))
    state = torch.zeros(ns, D, device=h.device) if st["s0"] is None else st["s0"].clone()
    state[seqs] = h[last]
    return {"y": h.reshape(st["g"].shape).to(st["x"].dtype), "state": state}


def _plain_glr_bwd(st):
    D = st["case"]["D"]
    first, last, seqs, longest = _ends(st)
    a = torch.exp(st["g"].float().reshape(-1, D))
    dy, y = st["dy"].float().reshape(-1, D), st["y"].float().reshape(-1, D)
    end = torch.zeros(len(_lengths(st["case"])), D, device=a.device) if st["dfin"] is None else st["dfin"]
    lam_end = end[seqs]
    mu = a * dy
    mu[last] += a[last] * lam_end
    a[last] = 0
    mu = _scan(a.flip(0), mu.flip(0), longest).flip(0)
    dx = dy.clone()
    dx[:-1] += mu[1:]
    dx[last] = dy[last] + lam_end
    before = torch.zeros_like(y)
    before[1:] = y[:-1]
    before[first] = 0 if st["s0"] is None else st["s0"][seqs]
    ds0 = end.clone()
    ds0[seqs] = mu[first]
    shape = st["g"].shape
    return {"dx": dx.reshape(shape).to(st["y"].dtype), "dg": (mu * before).reshape(shape).to(st["g"].dtype), "ds0": ds0}


def _plain_glr_step(st):
    x, a = st["x"].float(), torch.exp(st["g"].float())
    rows = None
    if st["slots"] is not None:
        rows = st["slots"] >= 0
        at = torch.where(rows, st["slots"], 0).long()
        h = st["state"][at]
    else:
        h = st["state"].clone()
    y = torch.empty_like(x)
    for t in range(st["case"]["T"]):
        h = a[:, t] * h + x[:, t]
        y[:, t] = h
    if rows is None:
        st["state"].copy_(h)
    else:
        y = torch.where(rows[:, None, None], y, 0.0)
        st["state"].index_copy_(0, at[rows], h[rows])
    return {"y": y.to(st["x"].dtype), "state": st["state"]}


def _plain_gn(st):
    case = st["case"]
    N, L, C, G = (case[n] for n in ("N", "L", "C", "groups"))
    x = st["x"].float().view(N, L, G, C // G)
    mean = x.mean(dim=(1, 3), keepdim=True)
    d = x - mean
    rstd = torch.rsqrt((d * d).mean(dim=(1, 3), keepdim=True) + EPS)
    z = (d * rstd).view(N, L, C)
    if case["affine"]:
        z = z * st["w"] + st["b"]
    y = z / (1 + torch.exp(-z)) if case["act"] == "silu" else z
    return {"y": y.to(st["x"].dtype), "mean": mean.view(N, G), "rstd": rstd.view(N, G)}


def _plain_gn_bwd(st):
    case = st["case"]
    N, L, C, G = (case[n] for n in ("N", "L", "C", "groups"))
    mean, rstd = st["mean"][:, None, :, None], st["rstd"][:, None, :, None]
    xh = (st["x"].float().view(N, L, G, C // G) - mean) * rstd
    dz = st["dy"].float()
    if case["act"] == "silu":
        z = xh.view(N, L, C)
        if case["affine"]:
            z = z * st["w"] + st["b"]
        s = 1 / (1 + torch.exp(-z))
        dz = dz * s * (1 + z * (1 - s))
    a = (dz * st["w"] if case["affine"] else dz).view(N, L, G, C // G)
    dx = rstd * (a - a.mean(dim=(1, 3), keepdim=True) - xh * (a * xh).mean(dim=(1, 3), keepdim=True))
    out = {"dx": dx.view(N, L, C).to(st["x"].dtype)}
    if case["affine"]:
        out["dweight"], out["dbias"] = (dz * xh.view(N, L, C)).sum(dim=(0, 1)), dz.sum(dim=(0, 1))
    return out


_M, _C1, _C2, _C3 = 0xFFFFFFFF, 0x9E3779B1, 0x71C61315, 0x189C32BF


def _signed(c):
    return c - (1 << 32) if c >= 1 << 31 else c


def _mix(x):
    """A 32-bit mix of shifts and odd multiplications: of a Python int, or of an int32 tensor (which wraps)."""
    if torch.is_tensor(x):
        x = (x ^ ((x >> 16) & 0xFFFF)) * _signed(_C2)
        x = (x ^ ((x >> 15) & 0x1FFFF)) * _signed(_C3)
        return x ^ ((x >> 16) & 0xFFFF)
    x = (x ^ (x >> 16)) * _C2 & _M
    x = (x ^ (x >> 15)) * _C3 & _M
    return x ^ (x >> 16)


def _random(st, step):
    """Two numbers in [0, 1) for every value, [blocks, 256] each: multiples of 2^-16 from a hash of
    the seed, the step, the tensor's number and the value's place in it."""
    dev = st["flat"]["params"].device
    key = _mix((st["seed"] & _M) ^ _mix((st["seed"] >> 32 & _M) ^ _mix(step & _M)))
    blocks = torch.tensor(st["blocks"], dtype=torch.int32, device=dev)
    i32 = lambda n: torch.arange(n, dtype=torch.int32, device=dev)
    keys = _mix(_signed(key) + i32(len(st["blocks"])) * _signed(_C1))
    nb = sum(st["blocks"])
    of = torch.repeat_interleave(i32(len(st["blocks"])).long(), blocks, output_size=nb)
    block = i32(nb) - (blocks.cumsum(0).to(torch.int32) - blocks)[of]              # its number in its tensor
    h = _mix(((block[:, None] * BLOCK + i32(BLOCK)) * _signed(_C1)) ^ keys[of][:, None])
    return (h & 0xFFFF).float() * 2.0 ** -16, ((h >> 16) & 0xFFFF).float() * 2.0 ** -16


def _quantise(x, u, keep):
    """(e4m3 codes, scales) of [blocks, 256] values; u: the random numbers; keep: a value above 0
    keeps a code above 0.  Values that are not finite become NaN codes and count for no scale."""
    a = x.abs()
    top = torch.where(torch.isfinite(a), a, 0.0).amax(dim=1)
    some = top >= 2.0 ** -100
    scale = torch.where(some, top * (1.0 / 448), 0.0)
    y = a * torch.where(some, 448.0 / top, 0.0)[:, None]
    e = ((y.view(torch.int32) >> 23) - 127).clamp(-6, 8)
    up = torch.ldexp(torch.ones_like(y), 3 - e)                                     # 1 / step
    q = ((y * up + u).floor() / up).clamp(max=448.0)
    if keep:
        q = torch.where((y > 0) & (q == 0), 2.0 ** -9, q)
    q = torch.where(torch.isfinite(a), q, float("nan"))
    return torch.copysign(q, x).to(torch.float8_e4m3fn), scale


def _plain_adamw(st):
    case, flat = st["case"], st["flat"]
    step, bits8 = case["step"], case["bits"] == 8
    g = flat["grads"].float()
    if bits8:
        m, v = ((flat[n].float() * flat[n + "_scale"][:, None]).view(-1) for n in ("m", "v"))
    else:
        m, v = flat["m"], flat["v"]
    m = m * B1 + g * (1 - B1)
    v = v * B2 + (g * g) * (1 - B2)
    p = flat["masters"] if case["master"] else flat["params"].float()
    p = p * (1 - LR * DECAY) - LR / (1 - B1 ** step) * (m / (v.sqrt() / math.sqrt(1 - B2 ** step) + ADAM_EPS))
    flat["params"].copy_(p)
    if case["master"]:
        flat["masters"].copy_(p)
    if bits8:
        um, uv = _random(st, step)
        for n, x, u in (("m", m, um), ("v", v, uv)):
            codes, scale = _quantise(x.view(-1, BLOCK), u, n == "v")
            flat[n].copy_(codes)
            flat[n + "_scale"].copy_(scale)
    else:
        flat["m"].copy_(m)
        flat["v"].copy_(v)
    return {n: t for n, t in flat.items() if n != "grads"}


def run(st):
    """One pass, as a caller makes it."""
    case = st["case"]
    op = case["op"]
    if not own:
        return {"glr": _plain_glr, "glr_bwd": _plain_glr_bwd, "glr_step": _plain_glr_step, "gn": _plain_gn,
                "gn_bwd": _plain_gn_bwd, "adamw": _plain_adamw}[op](st)
    import kimi_delta_attention_gb300 as kda
    if op == "glr":
        y, state = kda.kda_glr_fwd(st["x"], st["g"], initial_state=st["s0"], cu_seqlens=st["cu"])
        return {"y": y, "state": state}
    if op == "glr_bwd":
        dx, dg, ds0 = kda.kda_glr_bwd(st["g"], st["y"], st["dy"], initial_state=st["s0"], cu_seqlens=st["cu"],
                                      d_final_state=st["dfin"])
        return {"dx": dx, "dg": dg, "ds0": ds0}
    if op == "glr_step":
        y = kda.kda_glr_step(st["x"], st["g"], st["state"], slots=st["slots"])
        return {"y": y, "state": st["state"]}
    if op == "gn":
        y, mean, rstd = kda.kda_group_norm_fwd(st["x"], case["groups"], st["w"], st["b"], eps=EPS, activation=case["act"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "gn_bwd":
        dx, dweight, dbias = kda.kda_group_norm_bwd(st["x"], st["dy"], case["groups"], st["w"], st["b"], st["mean"], st["rstd"],
                                                    activation=case["act"], output_dweight=case["affine"],
                                                    output_dbias=case["affine"])
        out = {"dx": dx}
        if case["affine"]:
            out["dweight"], out["dbias"] = dweight, dbias
        return out
    x = st["lists"]
    kda.kda_adamw_step(x["params"], x["grads"], x["m"], x["v"], case["step"], lr=LR, betas=(B1, B2), eps=ADAM_EPS,
                       weight_decay=DECAY, masters=x.get("masters"), exp_avg_scales=x.get("m_scale"),
                       exp_avg_sq_scales=x.get("v_scale"), seed=st["seed"])
    return {n: t for n, t in st["flat"].items() if n != "grads"}


# --------------------------------------------------------------- the work ---
def work(case):
    """Bytes: every input read once, every output written once.  Operations: of the definitions
    (an exponential counts as one)."""
    es = 2 if case["io"] == "bf16" else 4
    if case["op"] == "adamw":
        sizes = [int(n) for n in case["sizes"].split()]
        n, scales = sum(sizes), 2 * 4 * sum(-(-k // BLOCK) for k in sizes)
        states = 2 * 1 * n + scales if case["bits"] == 8 else 2 * 4 * n
        return {"bytes": es * n * (2 if case["master"] else 3) + 2 * states + (8 * n if case["master"] else 0), "flops": 16 * n}
    if case["op"] in ("gn", "gn_bwd"):
        n, vec = case["N"] * case["L"] * case["C"], 4 * case["C"] if case["affine"] else 0
        stats = 8 * case["N"] * case["groups"]
        back = case["op"] == "gn_bwd"
        return {"bytes": (3 if back else 2) * n * es + (4 if back else 2) * vec + stats, "flops": (20 if back else 12) * n}
    gs, D = 2 if case["gate"] == "bf16" else 4, case["D"]
    lengths = _lengths(case)
    n, state = sum(lengths) * D, 4 * len(lengths) * D
    if case["op"] == "glr_step":
        B = case["B"]
        live = B - (2 if case["slots"] and B >= 4 else 0)
        return {"bytes": n * (2 * es + gs) + 2 * state * live // B, "flops": 3 * n}
    if case["op"] == "glr":
        return {"bytes": n * (2 * es + gs) + state * (2 if case["state"] else 1), "flops": 3 * n}
    return {"bytes": n * (3 * es + 2 * gs) + state * (3 if case["state"] else 1), "flops": 5 * n}


# -------------------------------------------------------------- in 64 bits --
def _rows64(st, t):
    """[longest, sequences, D] in fp64 of a packed or batched tensor; zeros behind a sequence's end."""
    flat = t.reshape(-1, t.shape[-1]).double()
    parts = torch.split(flat, _lengths(st["case"]))
    return torch.nn.utils.rnn.pad_sequence(parts)


def _back64(st, r):
    parts = [r[:n, i] for i, n in enumerate(_lengths(st["case"]))]
    return torch.cat(parts).reshape(st["g"].shape)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("gn", "gn_bwd"):
        N, L, C, G = (case[n] for n in ("N", "L", "C", "groups"))
        x = st["x"].double()
        w = st["w"].double() if case["affine"] else torch.ones(C, dtype=torch.float64, device=x.device)
        b = st["b"].double() if case["affine"] else torch.zeros_like(w)
        wide = lambda s: s.repeat_interleave(C // G, dim=1)[:, None, :]            # [N, G] over positions and channels
        group = lambda t: t.sum(1).view(N, G, C // G).sum(2) / (L * C // G)        # mean over a group
        if case["op"] == "gn":
            mean = group(x)
            rstd = 1 / (group(x.square()) - mean.square() + EPS).sqrt()
            z = (x - wide(mean)) * wide(rstd) * w + b
            return {"y": z * torch.sigmoid(z) if case["act"] == "silu" else z, "mean": mean, "rstd": rstd}
        mean, rstd = wide(st["mean"].double()), wide(st["rstd"].double())
        xh = (x - mean) * rstd
        z = (xh * w + b).requires_grad_()
        y = z * torch.sigmoid(z) if case["act"] == "silu" else z * 1.0
        dz, = torch.autograd.grad(y, z, st["dy"].double())
        out = {"dx": (dz * w - wide(group(dz * w)) - xh * wide(group(dz * w * xh))) * rstd}
        if case["affine"]:
            out["dweight"], out["dbias"] = torch.einsum("nlc,nlc->c", dz, xh), torch.einsum("nlc->c", dz)
        return out
    if case["op"] == "adamw":
        flat, t = {n: x for n, x in st["flat"].items()}, case["step"]
        g = flat["grads"].double()
        m, v = (flat[n].double() for n in ("m", "v"))
        if case["bits"] == 8:
            m, v = (m * flat["m_scale"].double()[:, None]).view(-1), (v * flat["v_scale"].double()[:, None]).view(-1)
        m, v = m + (1 - B1) * (g - m), v + (1 - B2) * (g ** 2 - v)
        p = (flat["masters"] if case["master"] else flat["params"]).double()
        p = p - LR * (DECAY * p + (m / (1 - B1 ** t)) / ((v / (1 - B2 ** t)) ** 0.5 + ADAM_EPS))
        out = {"params": p, "masters": p, "m": m, "v": v}
        if case["bits"] == 8:                                     # (which of two codes is a matter of chance)
            top = lambda x: x.abs().view(-1, BLOCK).amax(dim=1) / 448
            out.update(m=None, v=None, m_scale=top(m), v_scale=top(v))
        return {n: out[n] for n in flat if n != "grads"}
    if case["op"] == "glr_step":
        h = st["state"].double()
        slots = list(range(case["B"])) if st["slots"] is None else st["slots"].tolist()
        live = torch.tensor([b for b, s in enumerate(slots) if s >= 0], device=h.device, dtype=torch.long)
        at = torch.tensor([s for s in slots if s >= 0], device=h.device, dtype=torch.long)
        y = torch.zeros(st["x"].shape, dtype=torch.float64, device=h.device)
        for t in range(case["T"]):
            h[at] = st["g"][live, t].double().exp() * h[at] + st["x"][live, t].double()
            y[live, t] = h[at]
        return {"y": y, "state": h}
    lengths = _lengths(case)
    if max(lengths) > 200000 or max(lengths) * len(lengths) * case["D"] > 1 << 30:
        return None
    e = _rows64(st, st["g"]).exp()
    n = torch.tensor(lengths, device=e.device)
    h = torch.zeros(len(lengths), case["D"], dtype=torch.float64, device=e.device) if st["s0"] is None else st["s0"].double()
    if case["op"] == "glr":
        x = _rows64(st, st["x"])
        y = torch.empty_like(x)
        for t in range(x.shape[0]):
            h = torch.where((t < n)[:, None], e[t] * h + x[t], h)
            y[t] = h
        return {"y": _back64(st, y), "state": h}
    y, dy = _rows64(st, st["y"]), _rows64(st, st["dy"])
    mu = torch.zeros_like(h) if st["dfin"] is None else st["dfin"].double()
    dx, dg = torch.empty_like(dy), torch.empty_like(dy)
    for t in range(dy.shape[0] - 1, -1, -1):
        live = (t < n)[:, None]
        dx[t] = mu + dy[t]
        mu = torch.where(live, e[t] * dx[t], mu)
        dg[t] = mu * (y[t - 1] if t else h)
    return {"dx": _back64(st, dx), "dg": _back64(st, dg), "ds0": mu}
