"""The layer that uses recurrence, group norm, their gradients, the step and the optimizer together."""
import pytest
import torch

import kimi_delta_attention_gb300 as kda
from kimi_delta_attention_gb300 import glr_layer
from kimi_delta_attention_gb300.adamw import AdamW

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.load_library()


@pytest.mark.parametrize("bits", [8, 32])
def test_train_and_serve(bits):
    first, last, off = glr_layer.demo(steps=5, state_bits=bits)
    assert torch.isfinite(torch.tensor([first, last])).all()
    # the served tokens' projections are bf16 products of other shapes: a rounding, 2^-8 of a value, in each of
    # the chain's results (norm, u, state, group norm, y)
    assert off <= 5 * 2.0 ** -8


def test_gradients_flow_through_the_layer():
    """Every parameter's gradient against the layer written out in 64 bits (autograd).  The layer rounds to
    bf16 a dozen times on the way there and back (norm, projections, u, h, group norm, y and their
    gradients), each at most 2.4e-3 of its result in the 2-norm and uncorrelated: 12 ** 0.5 * 2.4e-3 =
    8e-3, held to twice that."""
    torch.manual_seed(1)
    B, T, W, H, D = 2, 70, 256, 2, 64
    layer = glr_layer.GatedRecurrentLayer(W, H, head_dim=D)
    x = torch.randn(B, T, W, device="cuda").bfloat16()
    w = torch.randn_like(x)
    y, state = layer(x)
    ((y * w).float().sum() + 0.1 * state.sum()).backward()

    names = ("norm_weight", "norm_bias", "w_in", "gate_bias", "head_weight", "head_bias", "w_out")
    par = {n: getattr(layer, n).detach().cpu().double().requires_grad_() for n in names}
    xd = x.cpu().double()
    norm = lambda t: (t - t.mean(-1, keepdim=True)) * (t.var(-1, unbiased=False, keepdim=True) + 1e-5) ** -0.5
    u, r = ((norm(xd) * par["norm_weight"] + par["norm_bias"]) @ par["w_in"]).split(H * D, dim=-1)
    g = -torch.nn.functional.softplus(r + par["gate_bias"]) / 8
    u = torch.sqrt(-torch.expm1(2 * g)) * u
    h, hs = torch.zeros(B, H * D, dtype=torch.float64), []
    for t in range(T):
        h = torch.exp(g[:, t]) * h + u[:, t]
        hs.append(h)
    z = norm(torch.stack(hs, 1).reshape(B, T, H, D)).reshape(B, T, -1) * par["head_weight"] + par["head_bias"]
    yd = xd + (z * torch.sigmoid(z)) @ par["w_out"]
    ref = torch.autograd.grad((yd * w.cpu().double()).sum() + 0.1 * h.sum(), list(par.values()))
    for name, r in zip(names, ref):
        off = (getattr(layer, name).grad.cpu().double() - r).norm() / r.norm()
        assert off <= 1.6e-2, f"{name}: {off:.2e}"


def test_gradients_of_what_is_used():
    """Final states or outputs alone, and inputs that need no gradient."""
    x, g = torch.randn(2, 30, 40, device="cuda", requires_grad=True), (-torch.rand(2, 30, 40, device="cuda")).requires_grad_()
    s0 = torch.randn(2, 40, device="cuda", requires_grad=True)
    y, state = glr_layer.gated_linear_recurrence(x, g, initial_state=s0)
    a = torch.autograd.grad(state.sum(), (x, g, s0), retain_graph=True)
    b = torch.autograd.grad(y[:, -1].sum(), (x, g, s0))
    assert all(torch.allclose(s, t, rtol=1e-5, atol=1e-6) for s, t in zip(a, b))
    w = torch.ones(40, device="cuda", requires_grad=True)
    out = glr_layer.group_norm(x.detach()[:, 0].contiguous(), 4, w, None, activation="silu")
    out.sum().backward()
    assert torch.isfinite(w.grad).all()


def test_empty_rows_of_the_step():
    torch.manual_seed(2)
    layer = glr_layer.GatedRecurrentLayer(256, 2, head_dim=64)
    x = torch.randn(3, 1, 256, device="cuda").bfloat16()
    pool = torch.randn(4, 128, device="cuda")
    before = pool.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = layer.step(x, pool, torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda"), status)
    assert torch.equal(pool[[1, 3]], before[[1, 3]]) and torch.isfinite(y.float()).all() and status.item() == 0
    layer.step(x, pool, torch.tensor([4, -1, 0], dtype=torch.int32, device="cuda"), status)
    assert kda.kda_read_device_status(status) == 7


def test_status_of_the_trainable_path():
    x, g = torch.randn(1, 90, 40, device="cuda", requires_grad=True), -torch.rand(1, 90, 40, device="cuda")
    cu = lambda *n: torch.tensor(n, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, _ = glr_layer.gated_linear_recurrence(x, g, cu_seqlens=cu(0, 40, 90), status=status)
    y.sum().backward()
    assert status.item() == 0
    y, _ = glr_layer.gated_linear_recurrence(x, g, cu_seqlens=cu(0, 40, 80), status=status)
    assert status.item() == 2
    status.zero_()
    y.sum().backward()
    assert kda.kda_read_device_status(status) == 7


# --------------------------------------------------------------- optimizer --
def problem(seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    return [torch.nn.Parameter(rn(70, 33)), torch.nn.Parameter(rn(500).bfloat16()), torch.nn.Parameter(rn(3))], rn


@pytest.mark.parametrize("masters", [False, True])
@pytest.mark.parametrize("bits", [8, 32])
def test_state_dict_goes_on_alike(bits, masters):
    """A run that is saved and loaded takes the same steps, bit for bit, states in their own types."""
    params, rn = problem()
    kw = dict(lr=1e-2, state_bits=bits, masters=masters, seed=5)
    opt = AdamW(params, **kw)
    grads = [[rn(*p.shape).to(p.dtype) for p in params] for _ in range(6)]

    def run(opt, params, some):
        for g in some:
            for p, t in zip(params, g):
                p.grad = t.clone()
            opt.step()

    run(opt, params, grads[:3])
    twin = [torch.nn.Parameter(p.detach().clone()) for p in params]
    other = AdamW(twin, **kw)
    other.load_state_dict(opt.state_dict())
    run(opt, params, grads[3:])
    run(other, twin, grads[3:])
    assert all(torch.equal(a, b) for a, b in zip(params, twin))
    assert other.state[twin[1]]["exp_avg"].dtype == (torch.float8_e4m3fn if bits == 8 else torch.float32)
    assert ("master" in other.state[twin[1]]) == masters and "master" not in other.state[twin[0]]


def test_parameters_without_gradients_and_late_ones():
    """A parameter that has its first gradient late starts its own count, as torch's optimizer has it."""
    params, rn = problem(1)
    params = [params[0], params[2]]
    twin = [p.detach().double().requires_grad_() for p in params]
    opt, ref = AdamW(params, lr=1e-2), torch.optim.AdamW(twin, lr=1e-2)
    for k in range(6):
        for i, (p, q) in enumerate(zip(params, twin)):
            g = rn(*p.shape) if i == 0 or k >= 3 else None
            p.grad, q.grad = g, None if g is None else g.double()
        opt.step()
        ref.step()
    for p, q in zip(params, twin):
        # six steps, each off by some 20 roundings of an update of at most 3 lr and two of p
        assert (p.double() - q).abs().max() <= 6 * (20 * 0.03 + 2 * q.abs().max().item()) * 2.0 ** -24


def test_captured_training_step():
    """Forward, backward and a capturable optimizer's step in one graph: replays count on, and follow the
    learning rate that is written on the device."""
    torch.manual_seed(3)
    layer = glr_layer.GatedRecurrentLayer(128, 2, head_dim=64)
    twin = glr_layer.GatedRecurrentLayer(128, 2, head_dim=64)
    twin.load_state_dict(layer.state_dict())
    x = torch.randn(2, 50, 128, device="cuda").bfloat16()
    target = torch.randn_like(x)
    kw = dict(lr=1e-2, state_bits=8, masters=True, seed=9)

    def train(layer, opt):
        loss = (layer(x)[0].float() - target.float()).square().mean()
        loss.backward()
        opt.step()
        opt.zero_grad(set_to_none=False)

    opt, ref = AdamW(layer.parameters(), capturable=True, **kw), AdamW(twin.parameters(), **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            train(layer, opt)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        train(layer, opt)
    for _ in range(3):
        graph.replay()
    opt.param_groups[0]["lr"].fill_(2e-3)
    graph.replay()
    assert opt.param_groups[0]["step_device"].item() == 6
    for k in range(6):
        ref.param_groups[0]["lr"] = 1e-2 if k < 5 else 2e-3
        train(twin, ref)
    for (name, p), q in zip(layer.named_parameters(), twin.parameters()):
        assert torch.equal(p, q), name


def test_refusals():
    with pytest.raises(kda.KdaError):
        AdamW([torch.nn.Parameter(torch.zeros(3, device="cuda"))], state_bits=16)
    p = torch.zeros(30, device="cuda")
    for bad in (dict(grads=[p[:3]]), dict(exp_avgs=[p.bfloat16()]), dict(grads=[p.cpu()]), dict(exp_avgs=[p, p]),
                dict(masters=[p.bfloat16()]), dict(exp_avg_scales=[p[:1]]), dict(step=0), dict(skip=1.0), dict(masters=[None, None]),
                dict(step=torch.ones(1, device="cuda")), dict(grads=[torch.zeros(60, device="cuda")[::2]]), dict(exp_avgs=[p])):
        a = dict(params=[p], grads=[p.clone()], exp_avgs=[p.clone()], exp_avg_sqs=[p.clone()], step=1)
        a.update(bad)
        with pytest.raises(kda.KdaError):
            kda.kda_adamw_step(**a)
    assert (p == 0).all()


# -------------------------------------------- optimizer, counts on the device --
def follow(params, twin, opt, ref, rn, which):
    """One step of both with the same gradients for the parameters in `which`."""
    for i, (p, q) in enumerate(zip(params, twin)):
        g = rn(*p.shape) if i in which else None
        p.grad, q.grad = g, None if g is None else g.double()
    opt.step()
    ref.step()


def near(params, twin, steps, lr):
    for p, q in zip(params, twin):
        # each step off by some 20 roundings of an update of at most 3 lr and two of p
        assert (p.double() - q).abs().max() <= steps * (20 * 3 * lr + 2 * q.abs().max().item()) * 2.0 ** -24


def test_capturable_parameters_without_gradients_and_late_ones():
    """As without capturable: each parameter counts its own steps."""
    params, rn = problem(4)
    params = [params[0], params[2], torch.nn.Parameter(rn(40))]
    twin = [p.detach().double().requires_grad_() for p in params]
    opt, ref = AdamW(params, lr=1e-2, capturable=True), torch.optim.AdamW(twin, lr=1e-2)
    for k in range(8):
        follow(params, twin, opt, ref, rn, {0} | ({1} if k >= 3 else set()) | ({2} if k != 4 else set()))
    near(params, twin, 8, 1e-2)


def test_captured_step_of_parameters_with_counts_apart():
    """Replays count on for a parameter that began later, too."""
    params, rn = problem(5)
    params = [params[0], params[2]]
    twin = [p.detach().double().requires_grad_() for p in params]
    opt, ref = AdamW(params, lr=1e-2, capturable=True), torch.optim.AdamW(twin, lr=1e-2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for k in range(4):
            follow(params, twin, opt, ref, rn, {0} if k < 3 else {0, 1})
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    for _ in range(3):
        graph.replay()
        ref.step()                              # (the gradients stay as they are)
    assert [opt.state[p]["step_device"].item() for p in params] == [7, 4]
    near(params, twin, 7, 1e-2)


@pytest.mark.parametrize("bits", [8, 32])
def test_capturable_state_goes_through_a_file_on_the_host(bits):
    """Saved, read onto the host and loaded: the next steps are the same, bit for bit, and so is a captured one's."""
    import io

    params, rn = problem(6)
    twin = [torch.nn.Parameter(p.detach().clone()) for p in params]
    kw = dict(lr=1e-2, state_bits=bits, masters=True, seed=5, capturable=True)
    opt, other = AdamW(params, **kw), AdamW(twin, **kw)

    def take(opt, params, grads):
        for p, t in zip(params, grads):
            p.grad = None if t is None else t.clone()
        opt.step()

    grads = [[rn(*p.shape).to(p.dtype) if k or i else None for i, p in enumerate(params)] for k in range(4)]
    for g in grads[:3]:
        take(opt, params, g)
    opt.param_groups[0]["lr"].fill_(3e-3)
    file = io.BytesIO()
    torch.save(opt.state_dict(), file)
    file.seek(0)
    other.load_state_dict(torch.load(file, map_location="cpu", weights_only=False))
    with torch.no_grad():
        for p, q in zip(params, twin):
            q.copy_(p)
    side = torch.cuda.Stream()
    for o, ps in ((opt, params), (other, twin)):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            take(o, ps, grads[3])
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o.step()
        graph.replay()
        torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(params, twin))
    assert [other.state[p]["step_device"].item() for p in twin] == [4, 5, 5]
    assert other.param_groups[0]["lr"].item() == opt.param_groups[0]["lr"].item()


def test_captures_that_replays_would_undo_are_refused():
    p = torch.nn.Parameter(torch.ones(5, device="cuda"))
    p.grad = torch.ones_like(p)
    for opt in (AdamW([p], capturable=True), AdamW([p])):
        with pytest.raises(kda.KdaError):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                opt.step()
        assert (p == 1).all()
    opt = AdamW([p], lr=0.5, capturable=True, weight_decay=0.0)
    opt.step()
    assert torch.allclose(p, torch.full_like(p, 0.5)) and opt.state[p]["step_device"].item() == 1
