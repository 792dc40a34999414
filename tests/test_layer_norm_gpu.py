"""Layer norm and its gradients on the GPU against the formulas in 64 bits.

Tolerances (2-norm of the error over that of the reference): bf16 results 2.4e-3 (one
rounding); fp32 results 3e-6: the sums of n <= 20000 terms are trees of depth under 40
after chains of at most 16 terms (or n / 1024 in the wide kernels), each step 2^-24 of the
running sum, so below 60 * 2^-24 = 3.6e-6 at worst and a third of it in the mean."""
import pytest
import torch

import kimi_delta_attention_gb300 as kda

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.load_library()


def close(got, ref, what):
    tol = 2.4e-3 if got.dtype == torch.bfloat16 else 3e-6
    got = got.double()
    assert got.shape == ref.shape and torch.isfinite(got).all(), what
    assert (got - ref).norm() <= tol * ref.norm() + 1e-12, f"{what}: {((got - ref).norm() / ref.norm()).item():.3e}"


def ref_fwd(x, w, b):
    x = x.double()
    mean, var = x.mean(-1), x.var(-1, unbiased=False)
    rstd = (var + EPS) ** -0.5
    y = (x - mean[..., None]) * rstd[..., None]
    if w is not None:
        y = y * w.double()
    if b is not None:
        y = y + b.double()
    return y, mean, rstd


CASES = [(1, 1), (3, 7), (5, 64), (17, 128), (4, 1000), (2, 1001), (300, 512), (33, 4096), (9, 5120), (4, 16384),
         (3, 16383), (2, 20001), (700, 96), (5, 2050)]


@pytest.mark.parametrize("affine", ["wb", "w", ""])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", CASES)
def test_forward_and_backward(rows, D, io, affine):
    gen = torch.Generator(device="cuda").manual_seed(rows * 31 + D)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x, dy = (2 * rn(rows, D) + 1).to(io), rn(rows, D).to(io)
    w = 1 + 0.3 * rn(D) if "w" in affine else None
    b = 0.2 * rn(D) if "b" in affine else None
    y, mean, rstd = kda.kda_layer_norm_fwd(x, w, b, EPS)
    y_ref, m_ref, r_ref = ref_fwd(x, w, b)
    close(y, y_ref, "y")
    close(mean, m_ref, "mean")
    close(rstd, r_ref, "rstd")
    dx, dw, db = kda.kda_layer_norm_bwd(x, dy, w, mean, rstd)
    xd = x.double().requires_grad_()
    wd = (torch.ones(D, dtype=torch.float64, device="cuda") if w is None else w.double()).requires_grad_()
    bd = torch.zeros(D, dtype=torch.float64, device="cuda", requires_grad=True)
    xh = (xd - xd.mean(-1, keepdim=True)) * (xd.var(-1, unbiased=False, keepdim=True) + EPS) ** -0.5
    gx, gw, gb = torch.autograd.grad((dy.double() * (xh * wd + bd)).sum(), [xd, wd, bd])
    if D > 1:          # one value a row: dx is 0 but for rounding
        close(dx, gx, "dx") if D > 7 else None
        close(dw, gw, "dweight")
    close(db, gb, "dbias")


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", [(9001, 256), (4003, 1024), (2501, 4096), (1201, 8192), (907, 16384)])
def test_gradients_of_many_rows(rows, D, io):
    """Several rows a block, and more than are in flight at once; each sum over the rows is a chain
    of at most 10 rows, 32 groups and 10 parts, then a tree of 5: below the bound above."""
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, D, generator=gen, device="cuda").to(io)
    dy = torch.randn(rows, D, generator=gen, device="cuda").to(io)
    w = 1 + 0.3 * torch.randn(D, generator=gen, device="cuda")
    _, mean, rstd = kda.kda_layer_norm_fwd(x, w, None, EPS)
    dx, dw, db = kda.kda_layer_norm_bwd(x, dy, w, mean, rstd)
    _, m_ref, r_ref = ref_fwd(x, None, None)
    xh, d = (x.double() - m_ref[:, None]) * r_ref[:, None], dy.double()
    a = d * w.double()
    close(dx, r_ref[:, None] * (a - a.mean(-1, keepdim=True) - xh * (a * xh).mean(-1, keepdim=True)), "dx")
    close(dw, (d * xh).sum(0), "dweight")
    close(db, d.sum(0), "dbias")


def test_large_mean():
    """The variance is taken around the mean: a mean of 1000 and a deviation of 1."""
    x = torch.randn(8, 2048, device="cuda") + 1000
    y, mean, rstd = kda.kda_layer_norm_fwd(x, eps=EPS)
    y_ref, m_ref, r_ref = ref_fwd(x, None, None)
    # x itself carries 2^-24 of 1000 a value (6e-5 of the deviation), the mean 3e-7 of 1000
    assert (y.double() - y_ref).abs().max() <= 1e-3
    assert ((rstd.double() - r_ref).abs() <= 1e-5 * r_ref).all()


def test_constant_rows():
    x = torch.full((3, 300), 2.5, device="cuda", dtype=torch.bfloat16)
    b = torch.randn(300, device="cuda")
    y, mean, rstd = kda.kda_layer_norm_fwd(x, None, b, EPS)
    assert torch.equal(y, b.bfloat16().expand(3, 300)) and (mean == 2.5).all()


def test_gradient_against_differences():
    x = torch.randn(2, 37, device="cuda")
    dy, w = torch.randn(2, 37, device="cuda"), torch.randn(37, device="cuda")
    _, mean, rstd = kda.kda_layer_norm_fwd(x, w, None, EPS)
    dx, dw, _ = kda.kda_layer_norm_bwd(x, dy, w, mean, rstd)
    f = lambda xx, ww: (ref_fwd(xx, ww, None)[0] * dy.double()).sum().item()
    h = 1e-4
    for r, c in ((0, 0), (1, 17), (1, 36)):
        e = torch.zeros(2, 37, dtype=torch.float64, device="cuda")
        e[r, c] = h
        num = (f(x.double() + e, w) - f(x.double() - e, w)) / (2 * h)
        assert abs(num - dx[r, c].item()) <= 1e-4 * max(1, abs(num))
        e1 = e[r]
        num = (f(x, w.double() + e1) - f(x, w.double() - e1)) / (2 * h)
        assert abs(num - dw[c].item()) <= 1e-4 * max(1, abs(num))


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 8), (0, 3), (3, 5)])
def test_row_strides_and_alignment(io, offset, pad):
    D = 200
    big = torch.randn(40, D + offset + pad, device="cuda").to(io)
    x, dy = big[:20, offset:offset + D], big[20:, offset:offset + D]
    y, mean, rstd = kda.kda_layer_norm_fwd(x)
    y2, mean2, rstd2 = kda.kda_layer_norm_fwd(x.contiguous())
    # the vector and element kernels sum in another order: equal to a rounding
    assert (y.double() - y2.double()).abs().max() <= (0.04 if io == torch.bfloat16 else 1e-5)
    close(y, ref_fwd(x, None, None)[0], "y")
    dx, dw, db = kda.kda_layer_norm_bwd(x, dy, None, mean, rstd)
    dx2, dw2, db2 = kda.kda_layer_norm_bwd(x.contiguous(), dy.contiguous(), None, mean2, rstd2)
    close(dw, dw2.double(), "dweight")
    close(db, db2.double(), "dbias")
    close(dx, dx2.double(), "dx")


def test_nan_stays_in_its_row_and_leading_dims():
    x = torch.randn(2, 5, 256, device="cuda").bfloat16()
    x[1, 2, 3] = float("nan")
    y, mean, rstd = kda.kda_layer_norm_fwd(x)
    assert mean.shape == (2, 5)
    bad = torch.isnan(y).any(-1)
    assert bad.sum() == 1 and bad[1, 2]


def test_repeats_bit_for_bit():
    x, dy = torch.randn(5000, 513, device="cuda"), torch.randn(5000, 513, device="cuda")
    _, mean, rstd = kda.kda_layer_norm_fwd(x)
    a = kda.kda_layer_norm_bwd(x, dy, None, mean, rstd)
    b = kda.kda_layer_norm_bwd(x, dy, None, mean, rstd)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_no_rows():
    x = torch.empty(0, 64, device="cuda")
    y, mean, rstd = kda.kda_layer_norm_fwd(x)
    dx, dw, db = kda.kda_layer_norm_bwd(x, x, None, mean, rstd)
    assert y.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


def test_refusals():
    x = torch.randn(4, 32, device="cuda")

    def refused(fn, code=1):
        with pytest.raises(kda.KdaError) as e:
            fn()
        assert e.value.code == code

    refused(lambda: kda.kda_layer_norm_fwd(x.cpu()))
    refused(lambda: kda.kda_layer_norm_fwd(x.double()))
    refused(lambda: kda.kda_layer_norm_fwd(x.t()))
    refused(lambda: kda.kda_layer_norm_fwd(x, torch.ones(31, device="cuda")))
    refused(lambda: kda.kda_layer_norm_fwd(x, torch.ones(32, device="cuda", dtype=torch.bfloat16)))
    refused(lambda: kda.kda_layer_norm_fwd(x, eps=-1.0))
    refused(lambda: kda.kda_layer_norm_fwd(x, out=x))
    _, mean, rstd = kda.kda_layer_norm_fwd(x)
    refused(lambda: kda.kda_layer_norm_bwd(x, x[:2], None, mean, rstd))
    refused(lambda: kda.kda_layer_norm_bwd(x, x, None, mean[:2], rstd))
    refused(lambda: kda.kda_layer_norm_bwd(x, x, None, mean, rstd, output_dx=False, output_dweight=False,
                                           output_dbias=False))
    refused(lambda: kda.kda_layer_norm_bwd(x, x, None, mean, rstd,
                                           workspace=torch.empty(8, dtype=torch.uint8, device="cuda")), 6)


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [1, 2, 3, 4, 5, 7])
def test_gradients_of_narrow_rows(D, io):
    """A narrow row's dx cancels almost to nothing (D = 1: to nothing), so it is held against the
    terms that cancel: each is good to some roundings of 2^-24, 16 in all.  The reference takes the
    mean and rstd that the call is given."""
    gen = torch.Generator(device="cuda").manual_seed(D)
    x, dy = (2 * torch.randn(400, D, generator=gen, device="cuda") + 1).to(io), torch.randn(400, D, generator=gen, device="cuda").to(io)
    w = 1 + 0.3 * torch.randn(D, generator=gen, device="cuda")
    _, mean, rstd = kda.kda_layer_norm_fwd(x, w, None, EPS)
    dx, dw, db = kda.kda_layer_norm_bwd(x, dy, w, mean, rstd)
    r = rstd.double()[:, None]
    xh, a = (x.double() - mean.double()[:, None]) * r, dy.double() * w.double()
    c0, c1 = a.mean(-1, keepdim=True), (a * xh).mean(-1, keepdim=True)
    ref = r * (a - c0 - xh * c1)
    terms = r * (a.abs() + a.abs().mean(-1, keepdim=True) + xh.abs() * (a * xh).abs().mean(-1, keepdim=True))
    bound = 16 * 2.0 ** -24 * terms + (2.0 ** -8 * ref.abs() if io == torch.bfloat16 else 0)
    assert dx.dtype == io and ((dx.double() - ref).abs() <= bound).all()
    if D == 1:
        assert (dx == 0).all() and (dw == 0).all()
    close(dw, (dy.double() * xh).sum(0), "dweight")
    close(db, dy.double().sum(0), "dbias")
