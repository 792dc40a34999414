"""Group norm with an activation and its gradients on the GPU against the formulas in 64 bits.

Tolerances.  y and the statistics, 2-norm of the error over that of the reference: bf16 2.4e-3 (one
rounding, averaged; for under 1000 values a rounding's largest, 2^-8), fp32 1e-5: sums of n <= 2^20 terms go in chains of at most n / 256 = 4096 terms and trees
above them; rounding errors of a chain add up like a random walk, 2^-24 sqrt(4096) / sqrt(3) = 2.2e-6
of the sum, on the mean and the variance, and half of that on rstd; a few roundings an
element follow.  dx is held against the terms that cancel in it, dweight and dbias against
the sum of their terms' magnitudes: 1e-5 of them, and 2^-8 of a bf16 value."""
import pytest
import torch

import kimi_delta_attention_gb300 as kda
from layer_ops_testutil import gn_bwd_reference, gn_reference, half_step

pytestmark = pytest.mark.gpu
EPS = 1e-5
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.load_library()


def close(got, ref, what):
    tol = (2.4e-3 if got.numel() >= 1000 else 2.0 ** -8) if got.dtype == BF else 1e-5
    assert got.shape == ref.shape and torch.isfinite(got).all(), what
    off = (got.double() - ref).norm()
    assert off <= tol * ref.norm() + 1e-12, f"{what}: {(off / ref.norm()).item():.3e}"


def against(got, ref, terms, what):
    assert got.shape == ref.shape and torch.isfinite(got).all(), what
    off = (got.double() - ref).abs() - (half_step(BF) * ref.abs() if got.dtype == BF else 0)
    assert (off <= 1.01e-5 * terms + 1e-30).all(), f"{what}: {(off / (terms + 1e-30)).max().item():.3e} of its terms"


def make(N, L, C, io, affine, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, dy = (1.5 * rn(N, L, C) + 0.4).to(io), rn(N, L, C).to(io)
    return x, dy, 1 + 0.3 * rn(C) if "w" in affine else None, 0.2 * rn(C) if "b" in affine else None


def check(x, dy, groups, w, b, act):
    y, mean, rstd = kda.kda_group_norm_fwd(x, groups, w, b, EPS, act)
    ry, rm, rr = gn_reference(x, groups, w, b, EPS, act)
    n = x[0].numel() // groups
    if n > 1:
        close(y, ry, "y")
    else:
        against(y, ry, torch.ones_like(ry), "y")
    against(mean, rm, x.double().abs().reshape(len(x), -1, groups, x.shape[-1] // groups).mean((1, 3)), "mean")
    close(rstd, rr, "rstd")
    got = kda.kda_group_norm_bwd(x, dy, groups, w, b, mean, rstd, act)
    ref, terms = gn_bwd_reference(x, dy, groups, w, b, mean, rstd, act)
    for g, r, t, what in zip(got, ref, terms, ("dx", "dweight", "dbias")):
        against(g, r, t, what)
    return y, mean, rstd, got


SIZES = [(1, 1, 1, 1), (5, 1, 64, 4), (300, 1, 4096, 32), (3, 77, 1001, 7), (2, 4099, 320, 32), (4, 1, 8192, 1), (7, 33, 96, 96),
         (2, 1000, 40, 5), (1, 5000, 2048, 16), (1, 1, 70000, 2), (2000, 1, 24, 3), (1, 1, 9, 3), (3, 5, 2056, 257), (1, 20000, 8, 2),
         (33, 1, 4096, 16), (9, 2, 1024, 8), (700, 1, 512, 64), (5, 64, 24, 1), (129, 1, 2048, 4), (2, 3, 30000, 6)]


@pytest.mark.parametrize("affine", ["wb", "w", ""])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("N,L,C,groups", SIZES)
def test_forward_and_backward(N, L, C, groups, io, act, affine):
    check(*make(N, L, C, io, affine, N + L + C)[:2], groups, *make(N, L, C, io, affine, N + L + C)[2:], act)


@pytest.mark.parametrize("io", [BF, F32])
def test_many_rows(io):
    """More rows than are in flight at once, one position a sample and several."""
    for N, L, C, groups in ((20011, 1, 256, 4), (3, 6007, 512, 8), (41, 503, 264, 3), (9000, 1, 1536, 12)):
        x, dy, w, b = make(N, L, C, io, "wb", N)
        check(x, dy, groups, w, b, "silu")


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("L,width", [(1, 2), (1, 7), (1, 9), (4, 2), (2, 4), (1, 33), (3, 11), (5, 13), (1, 127), (1, 129), (43, 3), (8, 32),
                                     (1, 257), (511, 1), (2, 256), (19, 27), (1, 515), (1, 1030), (683, 3), (1, 2047), (1, 2051)])
def test_groups_of_few_values(L, width, io):
    """Around the sizes at which a group takes more lanes, a whole warp, or chunks."""
    x, dy, w, b = make(37, L, 3 * width, io, "wb", width)
    check(x, dy, 3, w, b, "silu")


def test_one_group_a_row_is_layer_norm():
    x, dy, w, b = make(50, 1, 640, F32, "wb", 1)
    y, mean, rstd = kda.kda_group_norm_fwd(x, 1, w, b, EPS)
    y2, mean2, rstd2 = kda.kda_layer_norm_fwd(x, w, b, EPS)
    assert (y - y2).abs().max() <= 1e-5 and (mean - mean2).abs().max() <= 1e-6


@pytest.mark.parametrize("L", [1, 50])
def test_large_mean(L):
    """The variance is taken around the mean: a mean of 1000 and a deviation of 1."""
    x = torch.randn(4, L, 1024, device="cuda") + 1000
    y, mean, rstd = kda.kda_group_norm_fwd(x, 4, eps=EPS)
    ry, rm, rr = gn_reference(x, 4, None, None, EPS, "none")
    # x itself carries 2^-24 of 1000 a value (6e-5 of the deviation), the mean 3e-7 of 1000
    assert (y.double() - ry).abs().max() <= 1e-3
    assert ((rstd.double() - rr).abs() <= 2e-5 * rr).all()


@pytest.mark.parametrize("L", [1, 70])
def test_constant_groups(L):
    x = torch.full((3, L, 96), 2.5, device="cuda", dtype=BF)
    b = torch.randn(96, device="cuda")
    y, mean, rstd = kda.kda_group_norm_fwd(x, 8, None, b, EPS)
    assert torch.equal(y, b.bfloat16().expand(3, L, 96)) and (mean == 2.5).all()


@pytest.mark.parametrize("L", [1, 60])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_values_stay_in_their_group(L, bad):
    x, dy, w, b = make(4, L, 256, BF, "wb", 3)
    y, mean, rstd = kda.kda_group_norm_fwd(x, 8, w, b, EPS, "silu")
    dx, _, _ = kda.kda_group_norm_bwd(x, dy, 8, w, b, mean, rstd, "silu")
    x2 = x.clone()
    x2[1, L - 1, 70] = bad                      # group 2 of sample 1
    y2, mean2, rstd2 = kda.kda_group_norm_fwd(x2, 8, w, b, EPS, "silu")
    dx2, _, _ = kda.kda_group_norm_bwd(x2, dy, 8, w, b, mean2, rstd2, "silu")
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit[1, :, 64:96] = True
    assert torch.equal(y2[~hit], y[~hit]) and torch.isnan(y2[1, L - 1, 70])
    assert torch.equal(dx2[~hit], dx[~hit]) and torch.isnan(dx2[hit]).all()


def test_far_activations():
    """silu and its slope where e^-z overflows and where it vanishes."""
    x = torch.randn(8, 1, 64, device="cuda")
    b = torch.linspace(-300, 300, 64, device="cuda")
    y, mean, rstd = kda.kda_group_norm_fwd(x, 2, None, b, EPS, "silu")
    ry, _, _ = gn_reference(x, 2, None, b, EPS, "silu")
    assert ((y.double() - ry).abs() <= 1e-5 * ry.abs() + 1e-30).all()
    dx, dw, db = kda.kda_group_norm_bwd(x, torch.ones_like(x), 2, None, b, mean, rstd, "silu")
    assert torch.isfinite(dx).all() and abs(db[0].item()) <= 1e-30 and abs(db[-1].item() - 8) <= 1e-4


def test_gradients_against_differences():
    x, dy, w, b = make(2, 3, 12, F32, "wb", 4)
    _, mean, rstd = kda.kda_group_norm_fwd(x, 3, w, b, EPS, "silu")
    grads = kda.kda_group_norm_bwd(x, dy, 3, w, b, mean, rstd, "silu")
    f = lambda *a: (gn_reference(a[0], 3, a[1], a[2], EPS, "silu")[0] * dy.double()).sum().item()
    at = [t.double() for t in (x, w, b)]
    for k, grad in enumerate(grads):
        for i in range(0, grad.numel(), 3):
            e = torch.zeros_like(at[k])
            e.view(-1)[i] = 1e-5
            up, down = ([t + s * e if j == k else t for j, t in enumerate(at)] for s in (1, -1))
            num = (f(*up) - f(*down)) / 2e-5
            assert abs(num - grad.view(-1)[i].item()) <= 1e-4 * max(1, abs(num))


@pytest.mark.parametrize("L", [1, 9])
@pytest.mark.parametrize("io", [BF, F32])
def test_alignment(io, L):
    x, dy, w, b = make(20, L, 512, io, "wb", 5)

    def shift(t):
        s = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        s.copy_(t)
        return s

    y, mean, rstd, got = check(shift(x), shift(dy), 8, shift(w), shift(b), "silu")
    out = torch.empty(x.numel() + 1, dtype=io, device="cuda")[1:].view(x.shape)
    y2, _, _ = kda.kda_group_norm_fwd(x, 8, w, b, EPS, "silu", out=out)
    close(y2, gn_reference(x, 8, w, b, EPS, "silu")[0], "y")
    assert y2 is out


@pytest.mark.parametrize("N,L,C,groups", [(5000, 1, 513, 3), (3, 2000, 264, 8), (2, 9, 30000, 5)])
def test_repeats_bit_for_bit(N, L, C, groups):
    x, dy, w, b = make(N, L, C, F32, "wb", 6)
    runs = []
    for _ in range(3):
        y, mean, rstd = kda.kda_group_norm_fwd(x, groups, w, b, EPS, "silu")
        runs.append((y, mean, rstd, *kda.kda_group_norm_bwd(x, dy, groups, w, b, mean, rstd, "silu")))
    assert all(torch.equal(s, t) for r in runs[1:] for s, t in zip(runs[0], r))


def test_leading_dims_and_outputs_left_out():
    x, dy, w, b = make(6, 12, 64, F32, "wb", 7)
    x4, dy4 = x.view(6, 3, 4, 64), dy.view(6, 3, 4, 64)
    y, mean, rstd = kda.kda_group_norm_fwd(x, 4, w, b)
    y4, m4, r4 = kda.kda_group_norm_fwd(x4, 4, w, b)
    assert torch.equal(y4.view_as(y), y) and m4.shape == (6, 4)
    assert kda.kda_group_norm_fwd(x, 4, output_stats=False)[1:] == (None, None)
    dx, dw, db = kda.kda_group_norm_bwd(x4, dy4, 4, w, b, mean, rstd)
    for k, kw in enumerate(("output_dx", "output_dweight", "output_dbias")):
        only = kda.kda_group_norm_bwd(x, dy, 4, w, b, mean, rstd, **{n: n == kw for n in ("output_dx", "output_dweight", "output_dbias")})
        assert [t is None for t in only] == [n != k for n in range(3)] and torch.equal(only[k].view(-1), (dx, dw, db)[k].view(-1))


def test_no_samples():
    x = torch.empty(0, 5, 64, device="cuda")
    y, mean, rstd = kda.kda_group_norm_fwd(x, 4)
    dx, dw, db = kda.kda_group_norm_bwd(x, x, 4, None, None, mean, rstd)
    assert y.shape == x.shape and mean.shape == (0, 4) and (dw == 0).all() and (db == 0).all()


def test_no_samples_of_large_groups():
    x = torch.empty(0, 4096, 512, device="cuda")
    y, mean, rstd = kda.kda_group_norm_fwd(x, 4)
    dx, dw, db = kda.kda_group_norm_bwd(x, x, 4, None, None, mean, rstd)
    assert y.shape == dx.shape == x.shape and (dw == 0).all() and (db == 0).all()
