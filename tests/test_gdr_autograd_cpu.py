"""The differentiable calls' part on the host (no GPU): the library's kernels are replaced by
formulas that, like the kernels, record no graph."""
import pytest
import torch

from kimi_delta_attention_gb300 import KdaError, _gdr, gdr_layer


def norm_fwd(x, weight=None, bias=None, eps=1e-5, **kw):
    with torch.no_grad():
        mean = x.mean(-1)
        rstd = (x.var(-1, unbiased=False) + eps) ** -0.5
        y = (x - mean[..., None]) * rstd[..., None]
        return (y if weight is None else y * weight) + (0 if bias is None else bias), mean, rstd


def norm_bwd(x, dy, weight, mean, rstd, output_dx=True, output_dweight=True, output_dbias=True, **kw):
    with torch.no_grad():
        xh = (x - mean[..., None]) * rstd[..., None]
        a = dy if weight is None else dy * weight
        dx = rstd[..., None] * (a - a.mean(-1, keepdim=True) - xh * (a * xh).mean(-1, keepdim=True))
        return dx if output_dx else None, (dy * xh).sum(0) if output_dweight else None, dy.sum(0) if output_dbias else None


def rule_fwd(q, k, v, g, beta, scale=None, **kw):
    with torch.no_grad():
        return v * beta[..., None], q.new_zeros(q.shape[0], v.shape[2], q.shape[3], v.shape[3])


def rule_bwd(q, k, v, g, beta, do, scale=None, **kw):
    with torch.no_grad():
        return (torch.zeros_like(q), torch.zeros_like(k), do * beta[..., None], torch.zeros_like(g), (do * v).sum(-1), None)


@pytest.fixture
def kernels(monkeypatch):
    for name, fn in (("kda_layer_norm_fwd", norm_fwd), ("kda_layer_norm_bwd", norm_bwd), ("kda_gdr_fwd", rule_fwd),
                     ("kda_gdr_bwd", rule_bwd)):
        monkeypatch.setattr(_gdr, name, fn)


def test_layer_norm_once(kernels):
    """A first derivative is right; a second one, which the kernels do not have, is refused and
    not a gradient without the terms behind it."""
    x = torch.randn(5, 16, dtype=torch.float64, requires_grad=True)
    w = torch.randn(16, dtype=torch.float64, requires_grad=True)
    b = torch.randn(16, dtype=torch.float64, requires_grad=True)
    assert torch.autograd.gradcheck(lambda *a: gdr_layer.layer_norm(*a, 1e-5), (x, w, b))
    y = x + gdr_layer.layer_norm(x, w, b)
    grad, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        grad.square().sum().backward()


def test_rule_once(kernels):
    q, k, v = (torch.randn(1, 3, 2, 4).bfloat16().requires_grad_() for _ in range(3))
    g, beta = (torch.randn(1, 3, 2, requires_grad=True) for _ in range(2))
    o, _ = gdr_layer.gated_delta_rule(q, k, v, g, beta)
    grad, = torch.autograd.grad((o * v).sum(), v, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        grad.square().sum().backward()


def test_rule_in_fp32_has_no_gradients(kernels):
    """Refused where the graph would be recorded, not in the backward pass."""
    q, k, v = (torch.randn(1, 3, 2, 4) for _ in range(3))
    g, beta = (torch.randn(1, 3, 2) for _ in range(2))
    o, _ = gdr_layer.gated_delta_rule(q, k, v, g, beta)
    assert torch.equal(o, v * beta[..., None])
    g.requires_grad_()
    with torch.no_grad():
        gdr_layer.gated_delta_rule(q, k, v, g, beta)
    with pytest.raises(KdaError) as e:
        gdr_layer.gated_delta_rule(q, k, v, g, beta)
    assert e.value.code == 2
