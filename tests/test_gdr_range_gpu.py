"""The scalar-gate rule over the rest of its range: thousands of tokens, keys that are no unit
vectors or all alike, beta up to 2.  The reference is the token recurrence in 64 bits on the GPU
(torch), its gradients by autograd through it.

Tolerances, as the 2-norm of the error over the 2-norm of the reference, derived as in
gdr_testutil (an fp32 operand loses 2^-18 in its two bf16 parts, six products in a chain: 1e-5):
  long sequences: the same.  Every gate forgets (mean e^g = 0.92 a token), so a token's errors are
      gone after some tens of tokens and do not add up over the sequence.
  |beta| |k|^2 up to 2: the correction beta k (v - k S) and its products are up to twice the size
      beside the state in each of two factors, 4e-5.
  keys all alike: rows of M sum to up to 64, and the inverse's block products lose 2^-20 of
      |a| |b| each: 64 * 2^-20 = 6.1e-5.
bf16 results: one rounding, 2.4e-3, with these beside it (added)."""
import pytest
import torch

import kimi_delta_attention_gb300 as kda
from gdr_testutil import BF16, F32, cuda, make

pytestmark = pytest.mark.gpu
NAMES = ("q", "k", "v", "g", "beta", "s0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.load_library()


def recurrence(x, wrt=()):
    """(o, final states) of a batch [B, T] in double; with `wrt` the gradients of <do, o> + <ds, S>."""
    d = {n: t.double() if torch.is_tensor(t) and t.is_floating_point() else t for n, t in x.items()}
    for n in wrt:
        d[n] = d[n].detach().requires_grad_()
    G = x["v"].shape[2] // x["q"].shape[2]
    q, k, S, o = d["q"].repeat_interleave(G, 2), d["k"].repeat_interleave(G, 2), d["s0"], []
    for t in range(q.shape[1]):
        S = S * torch.exp(d["g"][:, t])[..., None, None]
        err = d["beta"][:, t][..., None] * (d["v"][:, t] - torch.einsum("bhkv,bhk->bhv", S, k[:, t]))
        S = S + k[:, t][..., None] * err[..., None, :]
        o.append(x["scale"] * torch.einsum("bhkv,bhk->bhv", S, q[:, t]))
    o = torch.stack(o, 1)
    if wrt:
        return torch.autograd.grad((o * d["do"]).sum() + (S * d["ds"]).sum(), [d[n] for n in wrt])
    return o, S


def off(got, ref, tol, what):
    assert got.shape == ref.shape and torch.isfinite(got).all(), what
    e = ((got.double() - ref).norm() / ref.norm()).item()
    assert e <= (BF16 + tol if got.dtype == torch.bfloat16 else tol), f"{what}: {e:.2e}"


def forward(x, tol):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, S = kda.kda_gdr_fwd(*(x[n] for n in NAMES[:5]), x["scale"], initial_state=x["s0"], status=status)
    o_ref, S_ref = recurrence(x)
    off(o, o_ref, tol, "o")
    off(S, S_ref, tol, "state")
    assert status.item() == 0


def gradients(x, tol, names=NAMES):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = kda.kda_gdr_bwd(*(x[n] for n in NAMES[:5]), x["do"], x["scale"], initial_state=x["s0"], d_final_state=x["ds"],
                          status=status)
    for n, a, b in zip(NAMES, got, recurrence(x, NAMES)):
        if n in names:
            off(a, b, tol, "d" + n)
    assert status.item() == 0


def test_single_elements():
    """fp32 results element by element.  An element's error is the sum of a hundred and more
    uncorrelated ones, so near to Gaussian, with F32 of the elements' size as a bound of its deviation:
    6 deviations for a million elements, and heads and tokens differ from the whole in size by up to 3:
    20 F32 of max(|ref|, rms)."""
    x = cuda(make((2, 700), 2, 4, 128, 128, seed=87, grads=True))
    _, S = kda.kda_gdr_fwd(*(x[n] for n in NAMES[:5]), x["scale"], initial_state=x["s0"])
    got = kda.kda_gdr_bwd(*(x[n] for n in NAMES[:5]), x["do"], x["scale"], initial_state=x["s0"], d_final_state=x["ds"])
    ref = recurrence(x, NAMES)
    for what, a, b in (("state", S, recurrence(x)[1]), *zip(("dg", "dbeta", "ds0"), got[3:], ref[3:])):
        rms = b.square().mean().sqrt()
        worst = ((a.double() - b).abs() / b.abs().clamp_min(rms)).max().item()
        assert worst <= 20 * F32, f"{what}: {worst:.2e}"


def test_fp32_inputs_give_fp32_states():
    """A caller who wants the states to fp32 passes fp32 q, k and v: the token recurrence.  A token
    rounds a state three times to 2^-24 of its size and takes sums over 128 dims, trees of depth 11;
    the gates (0.92 a token) leave some 12 tokens' errors to add up, uncorrelated:
    (12 * (3 + 11)) ** 0.5 * 2^-24 = 7.7e-7."""
    x = cuda(make((2, 700), 2, 4, 128, 128, seed=88))
    full = {n: t.float() if n in "qkv" else t for n, t in x.items()}
    o, S = kda.kda_gdr_fwd(*(full[n] for n in NAMES[:5]), x["scale"], initial_state=x["s0"])
    o_ref, S_ref = recurrence(x)
    off(S, S_ref, 7.7e-7, "state")
    off(o, o_ref, 7.7e-7, "o")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_exact_path_for_states_and_gradients(io, monkeypatch):
    """The library's exact-precision path takes the rule too, with the gate repeated over the key dims:
    fp32 states and gradients of inputs of either type, token by token.  States as above; a gradient
    has come through the states' recurrence and its own, 2 ** 0.5 * 7.7e-7; dg is a product of both,
    twice that."""
    monkeypatch.setenv("KDA_BACKWARD", "recurrent")
    x = cuda(make((1, 500), 2, 4, 128, 128, io=io, seed=90, grads=True))
    wide = x["g"][..., None].expand(*x["g"].shape, 128).contiguous()
    args = (x["q"], x["k"], x["v"], wide, x["beta"])
    _, S = kda.kda_recurrent_fwd(*args, x["scale"], initial_state=x["s0"])
    off(S, recurrence(x)[1], 7.7e-7, "state")
    got = list(kda.kda_backward(*args, x["do"], x["scale"], initial_state=x["s0"], d_final_state=x["ds"]))
    got[3] = got[3].sum(-1)
    for n, a, b in zip(NAMES, got, recurrence(x, NAMES)):
        off(a, b, 2.2e-6 if n == "g" else 1.1e-6, "d" + n)


# thin chains, wide chains (more CTAs than processors), chains of V = 64
@pytest.mark.parametrize("B,T,H,HV,K,V", [(1, 8200, 1, 1, 128, 128), (1, 6001, 2, 4, 64, 128), (1, 5000, 10, 40, 128, 128),
                                          (2, 4500, 20, 40, 128, 64)])
def test_forward_of_thousands_of_tokens(B, T, H, HV, K, V):
    forward(cuda(make((B, T), H, HV, K, V, seed=81)), F32)


@pytest.mark.parametrize("io", ["f32"])
def test_fp32_forward_of_thousands_of_tokens(io):
    forward(cuda(make((2, 3000), 2, 4, 128, 128, io=io, seed=82)), F32)


@pytest.mark.parametrize("T,H,HV,K,V", [(4100, 1, 2, 128, 128), (2500, 4, 4, 64, 64), (3000, 2, 2, 128, 64)])
def test_gradients_of_thousands_of_tokens(T, H, HV, K, V):
    gradients(cuda(make((1, T), H, HV, K, V, seed=83, grads=True)), F32)


def other_keys(kind, T, seed, grads=False):
    x = make((2, T), 2, 4, 128, 128, seed=seed, grads=grads)
    gen = torch.Generator().manual_seed(seed + 1)
    rand = lambda *s: torch.rand(*s, generator=gen)
    if kind == "lengths":          # |k| from 0.2 to 1.4, |q| from 0 to 11
        x["k"] = (x["k"].float() * (0.2 + 1.2 * rand(2, T, 2, 1))).bfloat16()
        x["q"] = (x["q"].float() * 11 * rand(2, T, 2, 1)).bfloat16()
    elif kind == "beta2":
        x["beta"] = 2 * rand(2, T, 4)
    elif kind == "alike":          # one key, and its opposite, for every token
        k = x["k"][:, :1].expand_as(x["k"])
        x["k"] = torch.where(rand(2, T, 2, 1) < 0.2, -k, k).contiguous()
        x["beta"] = 0.5 + 0.5 * x["beta"]
    return cuda(x)


KEYS = {"lengths": 4 * F32, "beta2": 4 * F32, "alike": 64 * 2.0 ** -20}


@pytest.mark.parametrize("kind", KEYS)
def test_forward_with_other_keys(kind):
    forward(other_keys(kind, 700, 84), KEYS[kind])


@pytest.mark.parametrize("kind", KEYS)
def test_gradients_with_other_keys(kind):
    """With keys all alike dg is what is left of sums ten times its size: see the next test."""
    gradients(other_keys(kind, 500, 85, grads=True), KEYS[kind], [n for n in NAMES if n != "g" or kind != "alike"])


@pytest.mark.parametrize("kind", KEYS)
def test_gate_gradients_against_their_terms(kind):
    """dg of one chunk held against the terms that it sums up and that may cancel:
        dgc_t = scale G q . (do S^T) + q . (A k) + k . (B k) - k . (A^T q + B^T k) - G beta k . (z S^T) - E k . (vn dS'^T),
        dg_t  = sum over s >= t of dgc_s, and what the chunk's last row adds to all of them.
    A term is a product of fp32 operands in two bf16 parts (F32 of its size, as in gdr_testutil), so
    the error of dg_t is at most F32 of the 2-norm of the terms it sums up (F32 was derived for a chain
    of six such products; no term here has passed through more)."""
    x = other_keys(kind, 64, 86, grads=True)
    got = kda.kda_gdr_bwd(*(x[n] for n in NAMES[:5]), x["do"], x["scale"], initial_state=x["s0"], d_final_state=x["ds"])[3]
    ref = recurrence(x, NAMES)[3]
    h = {n: x[n].double().transpose(1, 2) for n in ("q", "k", "v", "g", "beta", "do")}       # [B, heads, T, ...]
    q, k = h["q"].repeat_interleave(2, 1), h["k"].repeat_interleave(2, 1)
    S, dS, be, scale = x["s0"].double(), x["ds"].double(), h["beta"][..., None], x["scale"]
    gc = h["g"].cumsum(-1)
    D = torch.exp(gc[..., :, None] - gc[..., None, :]).tril()
    G, E = torch.exp(gc)[..., None], torch.exp(gc[..., -1:] - gc)[..., None]
    tr = lambda t: t.transpose(-1, -2)
    eye = torch.eye(64, dtype=torch.float64, device="cuda")
    T = torch.linalg.inv(eye + (be * (k @ tr(k)) * D).tril(-1))
    P = scale * (q @ tr(k)) * D
    vn = T @ (be * (h["v"] - G * (k @ S)))
    z = tr(T) @ (E * (k @ dS)) + tr(P @ T) @ h["do"]
    A, B = (scale * (h["do"] @ tr(vn)) * D).tril(-1), (-be * (z @ tr(vn)) * D).tril(-1)
    dot = lambda a, b: (a * b).sum(-1)
    terms = [scale * G[..., 0] * dot(q, h["do"] @ tr(S)), dot(q, A @ k), dot(k, B @ k), -dot(k, tr(A) @ q + tr(B) @ k),
             -(G * be)[..., 0] * dot(k, z @ tr(S)), -E[..., 0] * dot(k, vn @ tr(dS))]
    last = -terms[5].sum(-1) + torch.exp(gc[..., -1]) * (S * dS).sum((-1, -2))
    suffix = lambda t: t.flip(-1).cumsum(-1).flip(-1)
    whole = suffix(sum(terms)) + last[..., None]
    assert (whole - tr(ref)).norm() <= 1e-10 * ref.norm()                                    # (the formula itself)
    size = (suffix(sum(t.square() for t in terms)) + terms[5].square().sum(-1, keepdim=True) +
            torch.exp(2 * gc[..., -1:]) * (S * dS).square().sum((-1, -2))[..., None]).sqrt()
    assert (got.double() - ref).norm() <= F32 * size.norm(), ((got.double() - ref).norm() / size.norm()).item()


NEIGHBOURS = [dict(H=2, HV=4, K=128, V=128), dict(H=2, HV=4, K=64, V=64), dict(H=8, HV=32, K=128, V=128),
              dict(H=8, HV=32, K=64, V=128), dict(H=16, HV=32, K=128, V=64)]


@pytest.mark.parametrize("shape", NEIGHBOURS, ids=lambda s: "-".join(str(n) for n in s.values()))
def test_neighbours_of_every_kernel(shape):
    """Packed sequences full of NaN and infinities, in every input, leave the others' bits alone: thin
    chains, wide ones, those of V = 64, and the gradients of each, behind, before and between partial chunks."""
    seqs = [70, 33, 100, 1, 64, 129]
    bad = [1, 3, 4]
    x = make(seqs, state=True, seed=89, grads=True, **shape)
    y = {n: t.clone() if torch.is_tensor(t) else t for n, t in x.items()}
    at = torch.tensor([0] + seqs).cumsum(0).tolist()
    keep = torch.ones(at[-1], dtype=torch.bool)
    for i, s in enumerate(bad):
        keep[at[s]:at[s + 1]] = False
        for n in ("q", "k", "v", "do", "g", "beta"):
            y[n][0, at[s]:at[s + 1]] = (float("nan"), float("inf"), -float("inf"))[i]
        y["s0"][s], y["ds"][s] = float("inf"), float("nan")
    rest = [s for s in range(len(seqs)) if s not in bad]

    def both(x):
        d = cuda(x)
        args = [d[n] for n in NAMES[:5]]
        o, S = kda.kda_gdr_fwd(*args, d["scale"], initial_state=d["s0"], cu_seqlens=d["cu"])
        g = kda.kda_gdr_bwd(*args, d["do"], d["scale"], initial_state=d["s0"], cu_seqlens=d["cu"], d_final_state=d["ds"])
        return [t[0, keep.cuda()] for t in (o, *g[:5])] + [S[rest], g[5][rest]]

    clean, dirty = both(x), both(y)
    assert all(torch.isfinite(t).all() for t in clean)
    assert all(torch.equal(a, b) for a, b in zip(clean, dirty))
