"""The layer that uses norm, delta rule, gradients and serving step together."""
import pytest
import torch

import kimi_delta_attention_gb300 as kda
from kimi_delta_attention_gb300 import gdr_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.load_library()


def test_train_and_serve():
    first, last, off = gdr_layer.demo()
    assert last < 0.9 * first
    # the served tokens' projections are bf16 products of other shapes: a rounding, 2^-8 of a
    # value, in each of the chain's results (q, k, v, o, y)
    assert off <= 5 * 2.0 ** -8


def test_gradients_flow_through_the_layer():
    """Every parameter's gradient against the layer written out in 64 bits (autograd).  The
    layer rounds to bf16 a dozen times on the way there and back (norm, projections, q, k, o, y
    and their gradients), each at most 2.4e-3 of its result in the 2-norm and uncorrelated:
    12 ** 0.5 * 2.4e-3 = 8e-3, held to twice that."""
    torch.manual_seed(1)
    B, T, W, H, D = 2, 70, 256, 2, 64
    layer = gdr_layer.GatedDeltaLayer(W, H, H, head_dim=D)
    x = torch.randn(B, T, W, device="cuda").bfloat16()
    w = torch.randn_like(x)
    y, state = layer(x)
    ((y * w).float().sum() + 0.1 * state.sum()).backward()

    par = [p.detach().cpu().double().requires_grad_() for p in (layer.norm_weight, layer.norm_bias, layer.w_in, layer.w_out)]
    xd = x.cpu().double()
    h = (xd - xd.mean(-1, keepdim=True)) * (xd.var(-1, unbiased=False, keepdim=True) + 1e-5) ** -0.5 * par[0] + par[1]
    q, k, v, g, b = (h @ par[2]).split(layer.split, dim=-1)
    unit = lambda t: torch.nn.functional.normalize(t.reshape(B, T, H, D), dim=-1)
    q, k, v = unit(q), unit(k), v.reshape(B, T, H, D)
    g, b = -torch.nn.functional.softplus(g) / 8, torch.sigmoid(b)
    S, out = torch.zeros(B, H, D, D, dtype=torch.float64), []
    for t in range(T):
        S = S * torch.exp(g[:, t])[..., None, None]
        err = b[:, t][..., None] * (v[:, t] - torch.einsum("bhkv,bhk->bhv", S, k[:, t]))
        S = S + k[:, t][..., None] * err[..., None, :]
        out.append(D ** -0.5 * torch.einsum("bhkv,bhk->bhv", S, q[:, t]))
    yd = xd + torch.stack(out, 1).reshape(B, T, -1) @ par[3]
    ref = torch.autograd.grad((yd * w.cpu().double()).sum() + 0.1 * S.sum(), par)
    for name, p, r in zip(("norm weight", "norm bias", "w_in", "w_out"),
                          (layer.norm_weight, layer.norm_bias, layer.w_in, layer.w_out), ref):
        off = (p.grad.cpu().double() - r).norm() / r.norm()
        assert off <= 1.6e-2, f"{name}: {off:.2e}"


def test_empty_rows_pass_through():
    torch.manual_seed(2)
    layer = gdr_layer.GatedDeltaLayer(256, 2, 4, head_dim=64)
    x = torch.randn(3, 1, 256, device="cuda").bfloat16()
    pool = torch.randn(4, 4, 64, 64, device="cuda")
    before = pool.clone()
    y = layer.step(x, pool, torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda"))
    assert torch.equal(y[1], x[1]) and torch.equal(pool[[1, 3]], before[[1, 3]])
    assert not torch.equal(pool[2], before[2]) and not torch.equal(y[0], x[0])


def rule_inputs(T=100):
    torch.manual_seed(3)
    unit = lambda t: torch.nn.functional.normalize(t, dim=-1).bfloat16().requires_grad_()
    q, k = unit(torch.randn(1, T, 2, 64, device="cuda")), unit(torch.randn(1, T, 2, 64, device="cuda"))
    v = torch.randn(1, T, 4, 64, device="cuda").bfloat16().requires_grad_()
    g = (-0.1 * torch.rand(1, T, 4, device="cuda")).requires_grad_()
    return q, k, v, g, torch.rand(1, T, 4, device="cuda").requires_grad_()


def test_status_of_the_trainable_path():
    """A padded batch, whose cu_seqlens ends below T, is reported by the forward and by the
    backward; sound calls leave the word alone and bits stay once they are set."""
    x = rule_inputs()
    cu = lambda *n: torch.tensor(n, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, _ = gdr_layer.gated_delta_rule(*x, cu_seqlens=cu(0, 40, 100), status=status)
    o.sum().backward()
    assert status.item() == 0 and kda.kda_read_device_status(status) == 0
    o, _ = gdr_layer.gated_delta_rule(*x, cu_seqlens=cu(0, 40, 90), status=status)
    assert status.item() == 2 and kda.kda_read_device_status(status) == 7
    status.zero_()
    o.sum().backward()
    assert kda.kda_read_device_status(status) == 7
    gdr_layer.gated_delta_rule(*x, cu_seqlens=cu(0, 40, 100), status=status)
    assert kda.kda_read_device_status(status) == 7
    none = [t[:0] for t in x]
    status.zero_()
    gdr_layer.gated_delta_rule(*none, status=status)
    assert status.item() == 0
    side, short = torch.cuda.Stream(), cu(0, 40, 90)
    torch.cuda.synchronize()
    kda.kda_gdr_fwd(*[t.detach() for t in x], cu_seqlens=short, stream=side.cuda_stream, status=status)
    side.synchronize()
    assert kda.kda_read_device_status(status) == 7
    with pytest.raises(kda.KdaError):
        gdr_layer.gated_delta_rule(*x, status=torch.zeros(1, dtype=torch.int32))


def test_status_of_a_served_layer():
    layer = gdr_layer.GatedDeltaLayer(256, 2, 4, head_dim=64)
    x = torch.randn(2, 1, 256, device="cuda").bfloat16()
    pool, status = torch.zeros(3, 4, 64, 64, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    layer.step(x, pool, torch.tensor([2, -1], dtype=torch.int32, device="cuda"), status)
    assert status.item() == 0
    layer.step(x, pool, torch.tensor([3, 0], dtype=torch.int32, device="cuda"), status)
    assert kda.kda_read_device_status(status) == 7
