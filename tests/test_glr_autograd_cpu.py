"""The differentiable recurrence's and group norm's part on the host (no GPU): the library's kernels are
replaced by formulas that, like the kernels, record no graph."""
import pytest
import torch

from kimi_delta_attention_gb300 import _glr, glr_layer


def scan(x, g, initial_state=None, **kw):
    with torch.no_grad():
        h = torch.zeros_like(x[:, 0]) if initial_state is None else initial_state
        y = []
        for t in range(x.shape[1]):
            h = torch.exp(g[:, t]) * h + x[:, t]
            y.append(h)
        return torch.stack(y, 1), h


def scan_bwd(g, y, dy, initial_state=None, d_final_state=None, output_d_initial_state=True, **kw):
    with torch.no_grad():
        h0 = torch.zeros_like(y[:, 0]) if initial_state is None else initial_state
        mu = torch.zeros_like(h0) if d_final_state is None else d_final_state
        dx, dg = torch.empty_like(y), torch.empty_like(y)
        for t in reversed(range(y.shape[1])):
            dx[:, t] = dy[:, t] + mu
            mu = torch.exp(g[:, t]) * dx[:, t]
            dg[:, t] = mu * (y[:, t - 1] if t else h0)
        return dx, dg, mu if output_d_initial_state else None


def norm(x, groups, weight=None, bias=None, eps=1e-5, activation="none", **kw):
    d = x.reshape(x.shape[0], -1, groups, x.shape[-1] // groups)
    mean, var = d.mean((1, 3)), d.var((1, 3), unbiased=False)
    z = ((d - mean[:, None, :, None]) * ((var + eps) ** -0.5)[:, None, :, None]).reshape(x.shape)
    z = (z if weight is None else z * weight) + (0 if bias is None else bias)
    return z * torch.sigmoid(z) if activation == "silu" else z, mean, (var + eps) ** -0.5


def norm_fwd(*a, **kw):
    with torch.no_grad():
        return norm(*a, **kw)


def norm_bwd(x, dy, groups, weight, bias, mean, rstd, activation="none", output_dx=True, output_dweight=True, output_dbias=True, **kw):
    with torch.enable_grad():
        at = [t.detach().requires_grad_() for t in (x, weight, bias)]
        grads = torch.autograd.grad(norm(at[0], groups, at[1], at[2], activation=activation)[0], at, dy)
    return tuple(g if want else None for g, want in zip(grads, (output_dx, output_dweight, output_dbias)))


@pytest.fixture
def kernels(monkeypatch):
    for name, fn in (("kda_glr_fwd", scan), ("kda_glr_bwd", scan_bwd), ("kda_group_norm_fwd", norm_fwd), ("kda_group_norm_bwd", norm_bwd)):
        monkeypatch.setattr(_glr, name, fn)


def test_recurrence(kernels):
    x, g = (torch.randn(2, 5, 3, dtype=torch.float64, requires_grad=True) for _ in range(2))
    s0 = torch.randn(2, 3, dtype=torch.float64, requires_grad=True)
    assert torch.autograd.gradcheck(lambda *a: glr_layer.gated_linear_recurrence(*a), (x, g, s0))
    assert torch.autograd.gradcheck(lambda a, b: glr_layer.gated_linear_recurrence(a, b)[1], (x, g))
    y, _ = glr_layer.gated_linear_recurrence(x, g)
    grad, = torch.autograd.grad((y * x).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        grad.square().sum().backward()


def test_group_norm(kernels):
    x = torch.randn(3, 4, 6, dtype=torch.float64, requires_grad=True)
    w, b = (torch.randn(6, dtype=torch.float64, requires_grad=True) for _ in range(2))
    assert torch.autograd.gradcheck(lambda *a: glr_layer.group_norm(a[0], 2, a[1], a[2], activation="silu"), (x, w, b))
    grad, = torch.autograd.grad((glr_layer.group_norm(x, 2, w, b) * x).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        grad.square().sum().backward()


@pytest.mark.parametrize("bias", [-20.0, -103.0, -104.0, -200.0, 50.0])
def test_closed_gates_have_finite_gradients(monkeypatch, bias):
    """A gate so far closed that its g rounds to 0 (or so far open that e^2g does) passes gradients on, not NaN."""
    monkeypatch.setattr(glr_layer, "layer_norm", lambda x, w, b: x)
    layer = glr_layer.GatedRecurrentLayer(8, 1, head_dim=16, device="cpu")
    with torch.no_grad():
        layer.w_in.normal_()
        layer.w_in[:, 16:] *= 0.01
        layer.gate_bias[:8] = bias
    x = torch.randn(2, 3, 8).bfloat16().requires_grad_()
    u, g = layer._project(x)
    (u.float().sum() + g.sum()).backward()
    assert torch.isfinite(u).all() and torch.isfinite(g).all()
    for t in (x, layer.w_in, layer.gate_bias):
        assert torch.isfinite(t.grad).all()
