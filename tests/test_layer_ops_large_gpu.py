"""Offsets past 32 bits, and more sequences than a grid's second dimension holds."""
import pytest
import torch

import kimi_delta_attention_gb300 as kda
from layer_ops_testutil import glr_bwd_reference, glr_reference, gn_bwd_reference, gn_reference, make_glr, within

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.load_library()
    yield
    torch.cuda.empty_cache()


def test_recurrence_past_32_bits():
    """2.2e9 values: the last tokens, and the first ones' gradients, are what their neighbours' values say."""
    T, D, n = 270000, 8192, 300
    x = torch.randn(1, n, D, device="cuda").to(BF).repeat(1, T // n, 1)
    g = (-0.05 * torch.rand(1, n, D, device="cuda")).to(BF).repeat(1, T // n, 1)
    y, state = kda.kda_glr_fwd(x, g)
    _, before = kda.kda_glr_fwd(x[:, :T - n].contiguous(), g[:, :T - n].contiguous())
    ry, ey, rs, es = glr_reference(x[:, -n:], g[:, -n:], before, [n])
    within(y[:, -n:], ry, ey + 1e-4, "y")                  # (the state before it has rounding errors of its own)
    within(state, rs, es + 1e-4, "state")
    dx, dg, ds0 = kda.kda_glr_bwd(g, y, x)
    rx, ex, rg, eg, _, _ = glr_bwd_reference(g[:, -n:].contiguous(), y[:, -n:].contiguous(), x[:, -n:].contiguous(), y[:, -n - 1].float(), None, [n])
    within(dx[:, -n:], rx, ex, "dx")
    within(dg[:, -n:], rg, eg, "dg")
    k = 2 * n                                               # a gradient fades within some hundred tokens, but for 1e-6
    rx, ex, _, _, r0, e0 = glr_bwd_reference(g[:, :k].contiguous(), y[:, :k].contiguous(), x[:, :k].contiguous(), None, None, [k])
    within(dx[:, :50], rx[:, :50], ex[:, :50] + 1e-3, "dx")
    within(ds0, r0, e0 + 1e-3, "d_initial_state")


def test_group_norm_past_32_bits():
    for N, L, C, groups in ((270000, 1, 8192, 64), (3, 90001, 8192, 64)):
        x = torch.randn(1, 1, C, device="cuda").to(BF) * torch.linspace(0.5, 2, N * L, device="cuda").to(BF).view(N, L, 1)
        y, mean, rstd = kda.kda_group_norm_fwd(x, groups, activation="silu")
        tail = x[-1:, -1000:]
        if L == 1:
            ry, rm, rr = gn_reference(tail, groups, None, None, 1e-5, "silu")
        else:
            rm, rr = mean[-1:].double(), rstd[-1:].double()
            v = x[-1].double().view(L, groups, -1)
            m = v.mean((0, 2))
            assert (m - rm[0]).abs().max() <= 1e-5
            assert (((v - m[None, :, None]).square().mean((0, 2)) + 1e-5) ** -0.5 / rr[0] - 1).abs().max() <= 1e-5
            del v
            z = ((tail.double().view(1, -1, groups, C // groups) - rm[:, None, :, None]) * rr[:, None, :, None]).reshape(tail.shape)
            ry = z * torch.sigmoid(z)
        assert ((y[-1:, -1000:].double() - ry).abs() <= 2.0 ** -8 * ry.abs() + 1e-4).all()
        if L == 1:
            dx, dw, db = kda.kda_group_norm_bwd(x, x, groups, None, None, mean, rstd)
            part = kda.kda_group_norm_bwd(x[-5:], x[-5:], groups, None, None, mean[-5:], rstd[-5:])[0]
            assert torch.equal(dx[-5:], part) and torch.isfinite(dw).all()
            del dx
        del x, y
        torch.cuda.empty_cache()


def test_adamw_past_32_bits():
    """A tensor of 2.2e9 values: its last ones take the step that they take as a tensor of their own (but for the
    rounding's random numbers, which go by a value's place)."""
    n, k = 2200000000, 5000
    p = torch.full((n,), 1.0, dtype=BF, device="cuda")
    g = torch.full((n,), 0.5, dtype=BF, device="cuda")
    g[-k:] = torch.randn(k, device="cuda").to(BF)
    first = n - k - (n - k) % 256
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    sm, sv = (torch.zeros(-(-n // 256), device="cuda") for _ in range(2))
    kda.kda_adamw_step([p], [g], [m], [v], 1, lr=0.1, exp_avg_scales=[sm], exp_avg_sq_scales=[sv])
    q, h = torch.full((n - first,), 1.0, dtype=BF, device="cuda"), g[first:].clone()
    m2, v2 = (torch.zeros(n - first, device="cuda") for _ in range(2))
    kda.kda_adamw_step([q], [h], [m2], [v2], 1, lr=0.1)
    assert torch.equal(p[first:], q)
    wide = sm[first // 256:].repeat_interleave(256)[:n - first]
    assert ((m[first:].float() * wide - m2).abs() <= m2.abs() / 8 + wide * 2.0 ** -9).all()
    assert (p[:1000] == p[0]).all() and (sm[:-30] == sm[0]).all()


def test_many_sequences():
    B, D = 70001, 12
    d = make_glr([2] * B, D, F32, F32, packed=False, seed=1)
    y, s = kda.kda_glr_fwd(d["x"], d["g"], initial_state=d["s0"])
    state = d["s0"].clone()
    z = kda.kda_glr_step(d["x"], d["g"], state)
    want = torch.exp(d["g"].double()[:, 0]) * d["s0"].double() + d["x"].double()[:, 0]
    assert ((y[:, 0].double() - want).abs() <= 1e-6 * (1 + want.abs())).all()
    assert torch.allclose(y, z, rtol=1e-5, atol=1e-6) and torch.allclose(s, state, rtol=1e-5, atol=1e-6)
    cu = torch.arange(0, 2 * B + 1, 2, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y2, s2 = kda.kda_glr_fwd(d["x"].view(1, -1, D), d["g"].view(1, -1, D), initial_state=d["s0"], cu_seqlens=cu, status=status)
    assert status.item() == 0 and torch.equal(y2.view_as(y), y) and torch.equal(s2, s)
    gone = cu.clone()
    gone[1:-1] = 2 * B                                      # one sequence of everything, then empty ones
    y3, s3 = kda.kda_glr_fwd(d["x"].view(1, -1, D), d["g"].view(1, -1, D), initial_state=d["s0"], cu_seqlens=gone, status=status)
    assert status.item() == 0 and torch.equal(s3[1:], d["s0"][1:]) and torch.isfinite(y3).all()


def test_many_groups():
    x = torch.randn(70001, 2, 12, device="cuda")
    y, mean, rstd = kda.kda_group_norm_fwd(x, 3)
    ry, rm, rr = gn_reference(x, 3, None, None, 1e-5, "none")
    assert ((y.double() - ry).abs() <= 1e-5 * (1 + ry.abs())).all()
    x = torch.randn(2, 50, 60000, device="cuda")
    y, mean, rstd = kda.kda_group_norm_fwd(x, 30000)
    ry, rm, rr = gn_reference(x, 30000, None, None, 1e-5, "none")
    assert ((y.double() - ry).abs() <= 2e-5 * (1 + ry.abs())).all()


@pytest.mark.parametrize("io,L,width", [(F32, 16, 129), (BF, 2, 1032)])
def test_more_large_groups_than_a_grids_second_dimension(io, L, width):
    """Groups that take a block each, one value at a time and in vectors, forward and backward.  Groups of some
    2000 values: 1e-5 of the terms as in the group norm tests, and half a step of the type."""
    groups = 70001
    C = groups * width
    x, dy = (torch.randn(1, L, C, device="cuda").to(io) for _ in range(2))
    w = 1 + 0.2 * torch.randn(C, device="cuda")
    y, mean, rstd = kda.kda_group_norm_fwd(x, groups, w, None)
    step = torch.finfo(io).eps / 2
    ry, rm, rr = gn_reference(x, groups, w, None, 1e-5, "none")
    assert ((y.double() - ry).abs() <= 2e-5 * (1 + ry.abs()) + step * ry.abs()).all()
    assert (mean - rm).abs().max() <= 1e-5 and (rstd / rr - 1).abs().max() <= 1e-5
    del y, ry
    got = kda.kda_group_norm_bwd(x, dy, groups, w, None, mean, rstd)
    refs, terms = gn_bwd_reference(x, dy, groups, w, None, mean, rstd, "none")
    for g, r, t in zip(got, refs, terms):
        assert ((g.double() - r).abs() <= 1e-5 * t + (step * r.abs() if g.dtype == BF else 0) + 1e-30).all()


def test_step_of_as_many_sequences_as_an_int_counts():
    """2^31 - 1 sequences of one channel: the last rows, where the count of the launches passes 31 bits."""
    B = 2 ** 31 - 1
    x = torch.full((B, 1, 1), 0.5, dtype=BF, device="cuda")
    g = torch.full((B, 1, 1), -1.0, dtype=BF, device="cuda")
    state = torch.full((B, 1), 2.0, device="cuda")
    x[-70000:, 0, 0] = torch.randn(70000, device="cuda").to(BF)
    y = kda.kda_glr_step(x, g, state)
    for rows in (slice(0, 70000), slice(B // 2, B // 2 + 70000), slice(-70000, None)):
        want = 2.0 * torch.exp(torch.tensor(-1.0, dtype=torch.float64)).item() + x[rows, 0].double()
        assert ((state[rows].double() - want).abs() <= 1e-6 * (1 + want.abs())).all()
        assert ((y[rows, 0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6).all()
