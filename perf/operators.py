"""Cases, plain forms and 64-bit references of the scalar-gate delta rule (chunked forward,
recurrent step, backward) and of layer norm (forward, backward).

A case is a dict of plain values; ``prepare`` draws its inputs from a seed, ``run`` makes one
pass (the plain torch form, or with ``own`` the library's entry points) and ``exact`` gives the
same outputs in fp64 from the definitions.

Delta rule, per sequence and value head (q, k of key head hv // (HV / H)):
    S_t = e^{g_t} S_{t-1} + beta_t k_t (v_t - e^{g_t} S_{t-1}^T k_t)^T,   o_t = scale S_t^T q_t
Layer norm, per row: y = (x - mean) rstd w + b, rstd = (var + eps)^{-1/2}, var the biased variance.
"""
import math

import torch

own = False

EPS = 1e-5
CHUNK = 64


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # a short prompt, shorter than one chunk: all latency
        dict(name="fwd_prompt37", op="fwd", B=1, T=37, H=4, HV=8, K=128, V=128, state=False, lengths=""),
        # one long sequence at this library's headline shape
        dict(name="fwd_T4096_H32", op="fwd", B=1, T=4096, H=32, HV=32, K=128, V=128, state=False, lengths=""),
        # continuous prefill: 16 packed sequences of 1 to 8192 tokens, grouped value heads, states carried in
        dict(name="fwd_packed16_gva", op="fwd", B=1, T=0, H=8, HV=32, K=128, V=128, state=True,
             lengths="1 8192 777 64 3001 129 5120 6000 63 2048 7013 4097 65 1500 7999 333"),
        # one request's next token: all latency
        dict(name="step_B1", op="step", B=1, T=1, H=16, HV=32, K=128, V=128, io="bf16", slots=0),
        # 128 requests' next tokens
        dict(name="step_B128", op="step", B=128, T=1, H=32, HV=32, K=128, V=128, io="bf16", slots=0),
        # five tokens each (drafted ahead) for 24 requests whose states lie in a pool, two rows empty
        dict(name="step_pool_f32", op="step", B=24, T=5, H=4, HV=16, K=64, V=128, io="f32", slots=40),
        # a training step on ragged packed samples of a small model
        dict(name="bwd_packed_small", op="bwd", B=1, T=0, H=4, HV=8, K=64, V=64, state=True,
             lengths="300 1 511 188"),
        # a training step at the headline shape
        dict(name="bwd_T4096_H32", op="bwd", B=1, T=4096, H=32, HV=32, K=128, V=128, state=False, lengths=""),
        # the norm before a decoding step's projections: a few rows
        dict(name="norm_rows24", op="norm", rows=24, D=4096, io="bf16", bias=True),
        # the norm over a training batch's rows
        dict(name="norm_rows16384", op="norm", rows=16384, D=4096, io="bf16", bias=True),
        # its backward pass over the same rows
        dict(name="norm_bwd_rows16384", op="norm_bwd", rows=16384, D=4096, io="bf16", bias=True),
        # an odd width in fp32, no bias
        dict(name="norm_bwd_odd_f32", op="norm_bwd", rows=4099, D=1001, io="f32", bias=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "step", "step", "bwd", "bwd", "norm", "norm_bwd"])
    if op in ("norm", "norm_bwd"):
        D = _log_int(rng, 33, 16384)
        return dict(op=op, rows=_log_int(rng, 1, max(2, 16384 * 4096 // D // 2)), D=D,
                    io=rng.choice(["bf16", "bf16", "f32"]), bias=rng.random() < 0.7)
    K, V = rng.choice([(128, 128), (128, 128), (128, 128), (64, 64), (64, 128), (128, 64)])
    H = rng.choice([1, 2, 3, 4, 8, 16, 32])
    HV = H * rng.choice([g for g in (1, 1, 2, 3, 4) if H * g <= 32])
    if op == "step":
        B = _log_int(rng, 1, 128)
        return dict(op=op, B=B, T=rng.choice([1, 1, 1, 2, 3, 5]), H=H, HV=HV, K=K, V=V,
                    io=rng.choice(["bf16", "bf16", "f32"]), slots=rng.choice([0, 2 * B + 3]))
    most = 16384 if op == "fwd" else 4096           # tokens of a pass, for 32 value heads
    tokens = _log_int(rng, 5, most * 32 // HV if HV >= 8 else most * 4)
    packed = rng.random() < 0.5
    B, T, lengths = 1, 0, ""
    if packed:
        n = min(tokens, rng.choice([1, 2, 3, 5, 8, 13]))
        cuts = sorted(rng.randrange(tokens + 1) for _ in range(n - 1))
        lengths = " ".join(str(b - a) for a, b in zip([0] + cuts, cuts + [tokens]))
    else:
        B = rng.choice([1, 1, 2, 3])
        T = max(1, tokens // B)
    return dict(op=op, B=B, T=T, H=H, HV=HV, K=K, V=V, state=rng.random() < 0.5, lengths=lengths)


def _lengths(case):
    return [int(x) for x in case["lengths"].split()] if case["lengths"] else None


# ------------------------------------------------------------------ inputs --
def prepare(case, seed):
    """The tensors a caller holds before the call.  q and k are unit vectors per (token, key
    head), g a log decay <= 0 (logsigmoid(N) / 8), beta in (0, 1), states 0.1 N."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    rn = lambda *s: torch.randn(*s, generator=gen, device=dev)
    st = {"case": case}
    if case["op"] in ("norm", "norm_bwd"):
        rows, D = case["rows"], case["D"]
        dt = torch.bfloat16 if case["io"] == "bf16" else torch.float32
        st["x"] = (1.5 * rn(rows, D) + 0.3).to(dt)
        st["w"] = 1.0 + 0.2 * rn(D)
        st["b"] = 0.1 * rn(D) if case["bias"] else None
        if case["op"] == "norm_bwd":
            st["dy"] = rn(rows, D).to(dt)
            x = st["x"].float()          # what the forward pass has kept
            st["mean"] = x.mean(dim=1)
            st["rstd"] = torch.rsqrt((x - st["mean"][:, None]).square().mean(dim=1) + EPS)
        return st
    B, T, H, HV, K, V = (case[n] for n in ("B", "T", "H", "HV", "K", "V"))
    lengths = _lengths(case) if case["op"] != "step" else None
    if lengths:
        T = sum(lengths)
        st["cu"] = torch.tensor([0] + lengths, device=dev).cumsum(0).to(torch.int32)
    else:
        st["cu"] = None
    dt = torch.float32 if case.get("io") == "f32" else torch.bfloat16
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dt)
    st["q"], st["k"], st["v"] = unit(rn(B, T, H, K)), unit(rn(B, T, H, K)), rn(B, T, HV, V).to(dt)
    st["g"] = torch.nn.functional.logsigmoid(rn(B, T, HV)) / 8
    st["beta"] = torch.sigmoid(rn(B, T, HV))
    st["scale"] = K ** -0.5
    if case["op"] == "step":
        n = case["slots"]
        st["state"] = 0.1 * rn(n or B, HV, K, V)
        st["slots"] = None
        if n:
            slots = torch.randperm(n, generator=gen, device=dev)[:B].to(torch.int32)
            if B >= 4:                       # padding rows of a fixed-size batch
                slots[B // 3] = -1
                slots[B - 1] = -1
            st["slots"] = slots
        return st
    ns = len(lengths) if lengths else B
    st["s0"] = 0.1 * rn(ns, HV, K, V) if case["state"] else None
    if case["op"] == "bwd":
        st["do"] = rn(B, T, HV, V).to(dt)
        st["ds"] = 0.1 * rn(ns, HV, K, V) if case["state"] else None
    return st


# --------------------------------------------------------- the plain forms --
def _padded(st, lengths):
    """(index, valid): packed sequences as rows of a padded [N, L] batch, L whole chunks."""
    dev = st["q"].device
    if lengths is None:
        B, T = st["q"].shape[:2]
        lengths = [T] * B
    n = torch.tensor(lengths, device=dev)
    start = n.cumsum(0) - n
    L = -(-max(max(lengths), 1) // CHUNK) * CHUNK
    t = torch.arange(L, device=dev)
    valid = t[None, :] < n[:, None]
    return torch.where(valid, start[:, None] + t[None, :], 0), valid


def _chunked(st):
    """Inputs as fp32 [chunks, N, HV, 64, ...] with the padding rows zero."""
    case = st["case"]
    index, valid = _padded(st, _lengths(case))
    G = case["HV"] // case["H"]
    N, L = index.shape

    def lay(x, rep=1):
        x = x.reshape(-1, *x.shape[2:])[index].float()                      # [N, L, heads, (dim)]
        x = torch.where(valid.reshape(N, L, *[1] * (x.dim() - 2)), x, 0.0)
        x = x.repeat_interleave(rep, dim=2) if rep > 1 else x
        x = x.reshape(N, L // CHUNK, CHUNK, *x.shape[2:])
        return x.permute(1, 0, 3, 2, *range(4, x.dim()))

    return index, valid, G, lay


def _unchunk(x, st, index, valid, like):
    """[chunks, N, heads, 64, ...] back to the packed layout of `like`."""
    N, L = index.shape
    x = x.permute(1, 0, 3, 2, *range(4, x.dim())).reshape(N, L, x.shape[2], *x.shape[4:])
    out = torch.zeros(like.shape[0] * like.shape[1], *x.shape[2:], device=x.device)
    out[index[valid]] = x[valid]
    return out.reshape(*like.shape[:2], *x.shape[2:])


def _chunk_matrices(q, k, g, beta, scale):
    """Per chunk: D (decay between rows), M, P and T = (I + M)^{-1} by doubling."""
    gc = g.cumsum(-1)
    i = torch.arange(CHUNK, device=g.device)
    low = i[:, None] >= i[None, :]
    D = torch.where(low, torch.exp(torch.where(low, gc[..., :, None] - gc[..., None, :], 0.0)), 0.0)
    Gm = k @ k.transpose(-1, -2)
    M = torch.where(i[:, None] > i[None, :], beta[..., :, None] * Gm * D, 0.0)
    P = scale * (q @ k.transpose(-1, -2)) * D
    eye = torch.eye(CHUNK, device=g.device)
    X = -M
    T = eye + X
    for _ in range(5):
        X = X @ X
        T = T + T @ X
    return gc, D, Gm, M, P, T


def _plain_fwd(st):
    index, valid, G, lay = _chunked(st)
    q, k, v, g, beta = lay(st["q"], G), lay(st["k"], G), lay(st["v"]), lay(st["g"]), lay(st["beta"])
    scale = st["scale"]
    gc, D, Gm, M, P, T = _chunk_matrices(q, k, g, beta, scale)
    row, last = torch.exp(gc)[..., None], torch.exp(gc[..., -1:, None])
    tail = torch.exp(gc[..., -1:] - gc)[..., None]
    U, W = T @ (beta[..., None] * v), T @ (beta[..., None] * row * k)
    qd, kt = scale * row * q, (tail * k).transpose(-1, -2)
    S = torch.zeros(v.shape[1], v.shape[2], k.shape[-1], v.shape[-1], device=v.device) if st["s0"] is None else st["s0"]
    o = torch.empty_like(v)
    for n in range(v.shape[0]):
        vn = U[n] - W[n] @ S
        o[n] = qd[n] @ S + P[n] @ vn
        S = last[n] * S + kt[n] @ vn
    return {"o": _unchunk(o, st, index, valid, st["v"]).to(st["v"].dtype), "state": S}


def _plain_bwd(st):
    index, valid, G, lay = _chunked(st)
    q, k, v, do = lay(st["q"], G), lay(st["k"], G), lay(st["v"]), lay(st["do"])
    g, beta, scale = lay(st["g"]), lay(st["beta"]), st["scale"]
    gc, D, Gm, M, P, T = _chunk_matrices(q, k, g, beta, scale)
    row, last = torch.exp(gc)[..., None], torch.exp(gc[..., -1:, None])
    tail, be = torch.exp(gc[..., -1:] - gc)[..., None], beta[..., None]
    kT, qT = k.transpose(-1, -2), q.transpose(-1, -2)
    nc = v.shape[0]
    zero = torch.zeros(v.shape[1], v.shape[2], k.shape[-1], v.shape[-1], device=v.device)
    S = zero if st["s0"] is None else st["s0"]
    states, Y, vn = [], torch.empty_like(v), torch.empty_like(v)
    for n in range(nc):
        states.append(S)
        Y[n] = v[n] - row[n] * (k[n] @ S)
        vn[n] = T[n] @ (be[n] * Y[n])
        S = last[n] * S + kT[n] @ (tail[n] * vn[n])
    dS = zero if st["ds"] is None else st["ds"]
    z, kd, dleaving = torch.empty_like(v), torch.empty_like(v), [None] * nc
    Pdo, qdo = P.transpose(-1, -2) @ do, qT @ (scale * row * do)
    for n in range(nc - 1, -1, -1):
        dleaving[n] = dS
        kd[n] = k[n] @ dS
        z[n] = T[n].transpose(-1, -2) @ (Pdo[n] + tail[n] * kd[n])
        dS = last[n] * dS + qdo[n] - kT[n] @ (row[n] * be[n] * z[n])
    Sn, dSn = torch.stack(states), torch.stack(dleaving)
    dv = be * z
    zv = z @ vn.transpose(-1, -2)
    i = torch.arange(CHUNK, device=g.device)
    strict = i[:, None] > i[None, :]
    dM = torch.where(strict, -zv, 0.0)                           # of M = beta_i G_ij D_ij
    dP = do @ vn.transpose(-1, -2)                               # of P, where D is not zero
    dPk = scale * dP * D                                          # of q k^T
    dG = be * dM * D                                              # of k k^T
    doS, zS, vdS = do @ Sn.transpose(-1, -2), z @ Sn.transpose(-1, -2), vn @ dSn.transpose(-1, -2)
    dq = scale * row * doS + dPk @ k
    dk = tail * vdS - row * be * zS + dPk.transpose(-1, -2) @ q + (dG + dG.transpose(-1, -2)) @ k
    dbeta = (z * Y).sum(-1) + (dM * Gm * D).sum(-1)
    W = dM * M + dP * P
    t = tail[..., 0] * (vdS * k).sum(-1)
    dgc = W.sum(-1) - W.sum(-2) - t + row[..., 0] * (scale * (doS * q).sum(-1) - beta * (zS * k).sum(-1))
    dgc[..., -1] += t.sum(-1) + last[..., 0, 0] * (Sn * dSn).sum((-1, -2))
    dg = dgc.flip(-1).cumsum(-1).flip(-1)
    if G > 1:
        group = lambda x: x.reshape(*x.shape[:2], -1, G, *x.shape[3:]).sum(3)
        dq, dk = group(dq), group(dk)
    back = lambda x, like: _unchunk(x, st, index, valid, like)
    dt = st["q"].dtype
    return {"dq": back(dq, st["q"]).to(dt), "dk": back(dk, st["k"]).to(dt), "dv": back(dv, st["v"]).to(dt),
            "dg": back(dg, st["g"]), "dbeta": back(dbeta, st["beta"]), "ds0": dS}


def _plain_step(st):
    case = st["case"]
    G = case["HV"] // case["H"]
    rows = None
    if st["slots"] is not None:
        rows = (st["slots"] >= 0)
        at = torch.where(rows, st["slots"], 0).long()
        S = st["state"][at]
    else:
        S = st["state"].clone()
    q, k = (st[n].float().repeat_interleave(G, dim=2) for n in ("q", "k"))
    v, decay, beta = st["v"].float(), torch.exp(st["g"]), st["beta"]
    o = torch.empty_like(v)
    for t in range(case["T"]):
        S = S * decay[:, t, :, None, None]
        u = (S * k[:, t, :, :, None]).sum(2)
        S = S + k[:, t, :, :, None] * (beta[:, t, :, None] * (v[:, t] - u))[:, :, None, :]
        o[:, t] = st["scale"] * (S * q[:, t, :, :, None]).sum(2)
    if rows is None:
        st["state"].copy_(S)
    else:
        o = torch.where(rows[:, None, None, None], o, 0.0)
        st["state"].index_copy_(0, at[rows], S[rows])
    return {"o": o.to(st["v"].dtype), "state": st["state"]}


def _plain_norm(st):
    x = st["x"].float()
    mean = x.mean(dim=1, keepdim=True)
    d = x - mean
    rstd = torch.rsqrt((d * d).mean(dim=1, keepdim=True) + EPS)
    y = d * rstd * st["w"]
    if st["b"] is not None:
        y = y + st["b"]
    return {"y": y.to(st["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_norm_bwd(st):
    dy = st["dy"].float()
    xh = (st["x"].float() - st["mean"][:, None]) * st["rstd"][:, None]
    a = dy * st["w"]
    dx = st["rstd"][:, None] * (a - a.mean(dim=1, keepdim=True) - xh * (a * xh).mean(dim=1, keepdim=True))
    out = {"dx": dx.to(st["x"].dtype), "dweight": (dy * xh).sum(0)}
    if st["b"] is not None:
        out["dbias"] = dy.sum(0)
    return out


def run(st):
    """One pass, as a caller makes it."""
    op = st["case"]["op"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "norm": _plain_norm,
                "norm_bwd": _plain_norm_bwd}[op](st)
    import kimi_delta_attention_gb300 as kda
    if op == "fwd":
        o, state = kda.kda_gdr_fwd(st["q"], st["k"], st["v"], st["g"], st["beta"], st["scale"],
                                   initial_state=st["s0"], cu_seqlens=st["cu"])
        return {"o": o, "state": state}
    if op == "bwd":
        dq, dk, dv, dg, dbeta, ds0 = kda.kda_gdr_bwd(st["q"], st["k"], st["v"], st["g"], st["beta"], st["do"],
                                                     st["scale"], initial_state=st["s0"], cu_seqlens=st["cu"],
                                                     d_final_state=st["ds"])
        return {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta, "ds0": ds0}
    if op == "step":
        o = kda.kda_gdr_step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["state"], st["scale"],
                             slots=st["slots"])
        return {"o": o, "state": st["state"]}
    if op == "norm":
        y, mean, rstd = kda.kda_layer_norm_fwd(st["x"], st["w"], st["b"], eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    dx, dweight, dbias = kda.kda_layer_norm_bwd(st["x"], st["dy"], st["w"], st["mean"], st["rstd"],
                                                output_dbias=st["b"] is not None)
    out = {"dx": dx, "dweight": dweight}
    if dbias is not None:
        out["dbias"] = dbias
    return out


# --------------------------------------------------------------- the work ---
def work(case):
    """Bytes: every input read once, every output written once.  Operations: of the token
    recurrence (7 K V per token and value head forward, 20 K V for the gradients, whose
    reverse step needs the forward's states) and of the norm (8 and 12 per element)."""
    if case["op"] in ("norm", "norm_bwd"):
        n, D, rows = case["rows"] * case["D"], case["D"], case["rows"]
        es = 2 if case["io"] == "bf16" else 4
        vec = 2 if case["bias"] else 1
        if case["op"] == "norm":
            return {"bytes": 2 * n * es + 4 * D * vec + 8 * rows, "flops": 8 * n}
        return {"bytes": 3 * n * es + 4 * D * (1 + vec) + 8 * rows, "flops": 12 * n}
    lengths = _lengths(case) if case["op"] != "step" else None
    tokens = sum(lengths) if lengths else case["B"] * case["T"]
    ns = len(lengths) if lengths else case["B"]
    H, HV, K, V = case["H"], case["HV"], case["K"], case["V"]
    es = 4 if case.get("io") == "f32" else 2
    qk, vv, gate, state = tokens * H * K * es, tokens * HV * V * es, tokens * HV * 4, ns * HV * K * V * 4
    if case["op"] == "step":
        live = ns - (2 if case["slots"] and ns >= 4 else 0)
        return {"bytes": 2 * qk + 2 * vv + 2 * gate + 2 * state * live // ns, "flops": 7 * tokens * HV * K * V}
    if case["op"] == "fwd":
        return {"bytes": 2 * qk + 2 * vv + 2 * gate + state * (2 if case["state"] else 1),
                "flops": 7 * tokens * HV * K * V}
    return {"bytes": 4 * qk + 3 * vv + 4 * gate + state * (3 if case["state"] else 1), "flops": 20 * tokens * HV * K * V}


# -------------------------------------------------------------- in 64 bits --
def _cost(case):
    """Values of a state touched by the token recurrence, for the limit on exact()."""
    lengths = _lengths(case) if case["op"] != "step" else None
    ns, L = (len(lengths), max(lengths)) if lengths else (case["B"], case["T"])
    return L, ns * case["HV"] * case["K"] * case["V"]


def _tokens64(st):
    """Token-major fp64 inputs [L, N, heads, ...] of the padded batch; the padding does nothing."""
    case = st["case"]
    lengths = _lengths(case) or [st["q"].shape[1]] * st["q"].shape[0]
    L, G = max(lengths), case["HV"] // case["H"]

    def rows(x):
        flat, at, out = x.reshape(-1, *x.shape[2:]).double(), 0, []
        for n in lengths:
            out.append(torch.cat([flat[at:at + n], flat.new_zeros(L - n, *flat.shape[1:])]))
            at += n
        return torch.stack(out, dim=1)

    heads = lambda x: rows(x)[:, :, torch.arange(case["HV"], device=x.device) // G]
    back = lambda y: torch.cat([y[:n, i] for i, n in enumerate(lengths)]).reshape(*st["q"].shape[:2], *y.shape[2:])
    return lengths, rows, heads, back


def exact(case, seed):
    if case["op"] not in ("norm", "norm_bwd"):
        L, values = _cost(case)
        if L * (20e-6 + values * 8 * 6 / 3e12) * (1 if case["op"] != "bwd" else 6) > 12:
            return None
    st = prepare(case, seed)
    if case["op"] == "norm":
        x = st["x"].double()
        n = x.shape[1]
        mean = x.sum(1) / n
        rstd = 1 / ((x.square().sum(1) / n - mean.square()) + EPS).sqrt()
        y = torch.einsum("rd,r,d->rd", x - mean[:, None], rstd, st["w"].double())
        return {"y": y if st["b"] is None else y + st["b"].double(), "mean": mean, "rstd": rstd}
    if case["op"] == "norm_bwd":
        # from the gradient of the whole map: dx = J^T (w dy), J = rstd (I - 1/n - xh xh^T / n)
        x, dy, w = st["x"].double(), st["dy"].double(), st["w"].double()
        mean, rstd = st["mean"].double(), st["rstd"].double()
        n = x.shape[1]
        xh = torch.einsum("rd,r->rd", x - mean[:, None], rstd)
        c0, c1 = dy @ w / n, torch.einsum("rd,rd,d->r", dy, xh, w) / n
        dx = (dy * w - c0[:, None] - c1[:, None] * xh) * rstd[:, None]
        out = {"dx": dx, "dweight": torch.einsum("rd,rd->d", dy, xh)}
        if st["b"] is not None:
            out["dbias"] = dy.sum(0)
        return out
    scale = st["scale"]
    if case["op"] == "step":
        S = st["state"].double()
        slots = list(range(case["B"])) if st["slots"] is None else st["slots"].tolist()
        live = torch.tensor([b for b, s in enumerate(slots) if s >= 0], device=S.device)
        at = torch.tensor([s for s in slots if s >= 0], device=S.device)
        G = case["HV"] // case["H"]
        hk = torch.arange(case["HV"], device=S.device) // G
        o = torch.zeros(st["v"].shape, dtype=torch.float64, device=S.device)
        cur = S[at]
        for t in range(case["T"]):
            q, k = (st[n][live, t].double()[:, hk] for n in ("q", "k"))
            v, g, b = (st[n][live, t].double() for n in ("v", "g", "beta"))
            cur = cur * g.exp()[..., None, None]
            cur = cur + torch.einsum("bh,bhk,bhv->bhkv", b, k, v - torch.einsum("bhkv,bhk->bhv", cur, k))
            o[live, t] = scale * torch.einsum("bhkv,bhk->bhv", cur, q)
        S[at] = cur
        return {"o": o, "state": S}
    lengths, rows, heads, back = _tokens64(st)
    q, k, v, e, beta = heads(st["q"]), heads(st["k"]), rows(st["v"]), rows(st["g"]).exp(), rows(st["beta"])
    N, HV, K, V = len(lengths), case["HV"], case["K"], case["V"]
    S = torch.zeros(N, HV, K, V, dtype=torch.float64, device=q.device) if st["s0"] is None else st["s0"].double()

    def advance(S, t):
        S = S * e[t][..., None, None]
        d = beta[t][..., None] * (v[t] - torch.einsum("nhkv,nhk->nhv", S, k[t]))
        return S + k[t][..., None] * d[..., None, :]

    if case["op"] == "fwd":
        o = torch.empty_like(v)
        for t in range(v.shape[0]):
            S = advance(S, t)
            o[t] = scale * torch.einsum("nhkv,nhk->nhv", S, q[t])
        return {"o": back(o), "state": S}
    # reverse mode through the token recurrence; states kept every 64 tokens and made again
    do = rows(st["do"])
    L, kept = v.shape[0], []
    for t in range(L):
        if t % 64 == 0:
            kept.append(S)
        S = advance(S, t)
    dS = torch.zeros_like(S) if st["ds"] is None else st["ds"].double()
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, dbeta = torch.empty_like(beta), torch.empty_like(beta)
    for c in range(len(kept) - 1, -1, -1):
        span = range(64 * c, min(L, 64 * c + 64))
        before = [kept[c]]
        for t in span:
            before.append(advance(before[-1], t))
        for t in reversed(span):
            Sp, Sn = before[t - 64 * c], before[t - 64 * c + 1]
            dq[t] = scale * torch.einsum("nhkv,nhv->nhk", Sn, do[t])
            dS = dS + scale * q[t][..., None] * do[t][..., None, :]
            P = Sp * e[t][..., None, None]
            err = v[t] - torch.einsum("nhkv,nhk->nhv", P, k[t])
            kdS = torch.einsum("nhkv,nhk->nhv", dS, k[t])
            dbeta[t] = (kdS * err).sum(-1)
            dv[t] = beta[t][..., None] * kdS
            dk[t] = beta[t][..., None] * torch.einsum("nhkv,nhv->nhk", dS, err) \
                - torch.einsum("nhkv,nhv->nhk", P, dv[t])
            dP = dS - k[t][..., None] * dv[t][..., None, :]
            dg[t] = (dP * P).sum((-1, -2))
            dS = dP * e[t][..., None, None]
    fold = lambda x: x.reshape(*x.shape[:2], case["H"], HV // case["H"], K).sum(3)
    return {"dq": back(fold(dq)), "dk": back(fold(dk)), "dv": back(dv), "dg": back(dg), "dbeta": back(dbeta), "ds0": dS}
