"""The AdamW step on the GPU.

fp32 values against the formula in 64 bits: m and v take three roundings (3 * 2^-24 of their terms),
the update some eight (its error 16 * 2^-24 of it), p two more (2^-23 of it), and half a step of its type.
8-bit states: scales to three roundings of the block's largest magnitude / 448; a code is one of the
two around the exact value, the one that the value's random number picks unless it lies within
the roundings of the border between them."""
import math

import pytest
import torch

import kimi_delta_attention_gb300 as kda
from layer_ops_testutil import U, half_step

pytestmark = pytest.mark.gpu
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
LR, B1, B2, EPS, WD = 1e-2, 0.9, 0.95, 1e-8, 0.1


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.load_library()


def make(sizes, param=F32, grad=F32, bits=32, master=False, seed=0, fresh=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda n: torch.randn(n, generator=gen, device="cuda")
    d = dict(params=[rn(n).to(param) for n in sizes], grads=[(0.1 * rn(n)).to(grad) for n in sizes])
    d["masters"] = [p.float() + 1e-4 * rn(n) for p, n in zip(d["params"], sizes)] if master else None
    m = [torch.zeros(n, device="cuda") if fresh else 0.05 * rn(n) for n in sizes]
    v = [torch.zeros(n, device="cuda") if fresh else 0.01 * rn(n).square() for n in sizes]
    if bits == 8:
        blocks = [-(-n // 256) for n in sizes]
        d["exp_avg_scales"] = [torch.zeros(k, device="cuda") if fresh else 1e-4 * (1 + torch.rand(k, generator=gen, device="cuda")) for k in blocks]
        d["exp_avg_sq_scales"] = [s * 1e-2 for s in d["exp_avg_scales"]]
        wide = lambda s, n: s.repeat_interleave(256)[:n].clamp_min(1e-30)
        m = [(t / wide(s, len(t))).clamp(-448, 448).to(E4M3) for t, s in zip(m, d["exp_avg_scales"])]
        v = [(t / wide(s, len(t))).clamp(0, 448).to(E4M3) for t, s in zip(v, d["exp_avg_sq_scales"])]
    d["exp_avgs"], d["exp_avg_sqs"] = m, v
    return d


def values(d, name, scales):
    """The states a dict holds, in fp64."""
    if d.get(scales) is None:
        return [t.double() for t in d[name]]
    return [t.double() * s.double().repeat_interleave(256)[:len(t)] for t, s in zip(d[name], d[scales])]


def copy(d):
    return {n: None if x is None else [t.clone() for t in x] for n, x in d.items()}


def step(d, t, seed=5, **kw):
    a = dict(lr=LR, betas=(B1, B2), eps=EPS, weight_decay=WD, seed=seed)
    a.update(kw)
    more = {n: d[n] for n in ("masters", "exp_avg_scales", "exp_avg_sq_scales") if d.get(n) is not None}
    kda.kda_adamw_step(d["params"], d["grads"], d["exp_avgs"], d["exp_avg_sqs"], t, **a, **more)


M = 0xFFFFFFFF


def mix(x):
    x = ((x ^ (x >> 16)) * 0x71C61315) & M
    x = ((x ^ (x >> 15)) * 0x189C32BF) & M
    return x ^ (x >> 16)


def random_numbers(number, n, t, seed):
    """The two numbers in [0, 1) of every value of tensor `number`."""
    key = mix((seed & M) ^ mix((seed >> 32 & M) ^ mix(t)))
    key = mix((key + number * 0x9E3779B1) & M)
    h = mix((torch.arange(n, dtype=torch.int64, device="cuda") * 0x9E3779B1 & M) ^ key)
    return (h & 0xFFFF).double() / 65536, (h >> 16).double() / 65536


def check_codes(codes, scales, ref, err, u, keep, what):
    """ref: the exact values, err: how far an fp32 evaluation may be from them."""
    n = len(ref)
    if n == 0:
        return
    pad = torch.nn.functional.pad(ref.abs(), (0, -n % 256)).view(-1, 256)
    top = pad.amax(1)
    perr = torch.nn.functional.pad(err, (0, -n % 256)).view(-1, 256).amax(1)
    assert ((scales.double() - top / 448).abs() <= (perr + 3 * U * top) / 448 + 1e-45).all(), what
    wide = lambda t: t.repeat_interleave(256)[:n]
    y = torch.where(wide(top) > 0, ref.abs() / wide(top).clamp_min(1e-300) * 448, 0.0)
    ey = torch.where(wide(top) > 0, (err + wide(perr)) / wide(top).clamp_min(1e-300) * 448, 0.0) + 6 * U * y
    e = torch.floor(torch.log2(y.clamp_min(1e-300))).clamp(-6, 8)
    s = ((e.long() + 1020) << 52).view(torch.float64)               # 2^(e - 3) (a power of floats is not exact)
    lo = torch.floor(y / s) * s
    up = (y - lo) / s + u >= 1
    want = torch.where(up, lo + s, lo).clamp(max=448)
    if keep:
        want = torch.where((ref > 0) & (want == 0), 2.0 ** -9, want)
    got = codes.double()
    assert torch.isfinite(got).all() and ((got == 0) | (torch.sign(got) == torch.sign(ref))).all(), what
    near = ((y / s + u) - torch.round(y / s + u)).abs() <= (ey + 2.0 ** -20) / s      # (at a border: either code)
    bad = (got.abs() != want) & ~near
    assert not bad.any(), f"{what}: {int(bad.sum())} codes"
    assert ((got.abs() - want).abs() <= 2 * s).all(), what


def check(d, t, seed=5, scale=1.0):
    b = copy(d)
    m0, v0 = values(b, "exp_avgs", "exp_avg_scales"), values(b, "exp_avg_sqs", "exp_avg_sq_scales")
    kw = {} if scale == 1.0 else {"grad_scale": torch.tensor([scale], device="cuda")}
    step(d, t, seed, **kw)
    for i, g in enumerate(b["grads"]):
        g = g.double() * scale
        m, v = B1 * m0[i] + (1 - B1) * g, B2 * v0[i] + (1 - B2) * g * g
        em = 4 * U * (B1 * m0[i].abs() + (1 - B1) * g.abs())
        ev = 6 * U * v
        old = (b["masters"] or b["params"])[i].double()
        bc1, bc2 = 1 - B1 ** t, 1 - B2 ** t
        den = (v / bc2).sqrt() + EPS
        upd = LR / bc1 * m / den
        p = old * (1 - LR * WD) - upd
        ep = 4 * U * old.abs() + LR / bc1 * em / den + 16 * U * upd.abs()
        got = d["params"][i]
        assert ((got.double() - p).abs() <= ep + half_step(got.dtype) * (p.abs() + ep) + 1e-37).all(), f"params {i}"
        if d["masters"]:
            x = d["masters"][i]
            assert ((x.double() - p).abs() <= ep + U * p.abs()).all(), f"masters {i}"
            assert torch.equal(got, x.to(got.dtype))
        if d.get("exp_avg_scales") is None:
            assert ((d["exp_avgs"][i].double() - m).abs() <= em + 1e-37).all(), f"m {i}"
            assert ((d["exp_avg_sqs"][i].double() - v).abs() <= ev + 1e-37).all(), f"v {i}"
        else:
            um, uv = random_numbers(i, len(g), t, seed)
            check_codes(d["exp_avgs"][i], d["exp_avg_scales"][i], m, em, um, False, f"m {i}")
            check_codes(d["exp_avg_sqs"][i], d["exp_avg_sq_scales"][i], v, ev, uv, True, f"v {i}")


SIZES = [[1], [255, 256, 257], [5000], [0, 7, 0, 3], [1, 2, 3, 4, 5, 2048, 2049, 100001], [64] * 100]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,master", [(F32, F32, False), (BF, BF, False), (BF, F32, True), (BF, BF, True), (F32, BF, False)])
@pytest.mark.parametrize("n", range(len(SIZES)))
def test_step(n, param, grad, master, bits):
    for t, fresh in ((1, True), (50, False)):
        check(make(SIZES[n], param, grad, bits, master, seed=n, fresh=fresh), t)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(bits):
    """More than a launch takes; the numbers of the rounding go by a tensor's place in the whole list."""
    check(make([3 + i % 300 for i in range(1003)], BF, BF, bits, seed=20), 9, seed=-123456789012345)


@pytest.mark.parametrize("bits", [32, 8])
def test_mixed_types_and_alignment(bits):
    """Types tensor by tensor, and views that start anywhere."""
    d = make([700, 513, 2100, 64], BF, BF, bits, False, seed=21)
    d["params"][1], d["grads"][2] = d["params"][1].float(), d["grads"][2].float()

    def shift(t):
        s = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:]
        s.copy_(t)
        return s

    for name in ("params", "grads", "exp_avgs", "exp_avg_sqs"):
        d[name][2] = shift(d[name][2])
    check(d, 3)


def copy_some(d):
    return {n: None if x is None else [None if t is None else t.clone() for t in x] for n, x in d.items()}


def test_masters_for_some():
    d = make([700, 513], BF, BF, 32, False, seed=22)
    d["masters"] = [d["params"][0].float(), None]
    alone = [{n: None if x is None else [x[i]] for n, x in copy_some(d).items()} for i in (0, 1)]
    alone[1]["masters"] = None
    step(d, 3)
    for i in (0, 1):
        step(alone[i], 3)
        assert torch.equal(alone[i]["params"][0], d["params"][i])
    assert torch.equal(alone[0]["masters"][0], d["masters"][0])


def test_grad_scale_and_skip():
    check(make([3000, 17], F32, F32, 32, seed=23), 4, scale=0.25)
    check(make([3000, 17], BF, BF, 8, seed=23), 4, scale=0.25)
    for bits in (8, 32):
        for word in (1.0, float("nan")):
            d = make([3000, 17], BF, BF, bits, seed=24)
            b = copy(d)
            step(d, 4, skip=torch.tensor([word], device="cuda"))
            assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for n in d if d[n] for x, y in zip(d[n], b[n]))
        step(d, 4, skip=torch.zeros(1, device="cuda"))
        assert not torch.equal(d["params"][0], b["params"][0])


def test_device_step_and_rate():
    for bits in (8, 32):
        d = make([3000, 17], F32, F32, bits, seed=25)
        b = copy(d)
        step(d, 37)
        kda.kda_adamw_step(b["params"], b["grads"], b["exp_avgs"], b["exp_avg_sqs"], torch.tensor([37], dtype=torch.int32, device="cuda"),
                           lr=torch.tensor(LR, device="cuda"), betas=(B1, B2), eps=EPS, weight_decay=WD, seed=5,
                           **{n: b[n] for n in ("exp_avg_scales", "exp_avg_sq_scales") if n in b})
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for n in d if d[n] for x, y in zip(d[n], b[n]))


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_bad_gradients_stay_with_their_value(bad, bits):
    d = make([1000], F32, F32, bits, seed=26)
    b = copy(d)
    b["grads"][0][300] = bad
    step(d, 5)
    step(b, 5)
    rest = torch.arange(1000, device="cuda") != 300
    same = rest if bits == 32 else rest & ((torch.arange(1000, device="cuda") // 256) != 1)
    for n in ("params", "exp_avgs", "exp_avg_sqs"):
        x, y = d[n][0].float(), b[n][0].float()
        assert torch.equal(x[same], y[same]) and torch.isfinite(y[rest]).all() and not torch.isfinite(y[300])
    if bits == 8:
        assert torch.isfinite(b["exp_avg_scales"][0]).all() and torch.isfinite(b["exp_avg_sq_scales"][0]).all()


def test_zero_gradients_and_tiny_ones():
    d = make([600], F32, F32, 8, seed=27, fresh=True)
    d["grads"][0].zero_()
    p = d["params"][0].clone()
    step(d, 1, weight_decay=0.0)
    assert torch.equal(d["params"][0], p) and (d["exp_avgs"][0].float() == 0).all() and (d["exp_avg_scales"][0] == 0).all()
    d["grads"][0].fill_(1e-25)                          # squares below the smallest scale
    step(d, 2)
    assert torch.isfinite(d["params"][0]).all() and (d["exp_avg_sqs"][0].float() == 0).all()


def test_a_small_second_moment_is_not_lost():
    """Beside a value a million times larger, v keeps a code above 0 (or its step would be m / eps)."""
    d = make([256], F32, F32, 8, seed=28, fresh=True)
    d["grads"][0].fill_(1e-4)
    d["grads"][0][0] = 100.0
    step(d, 1)
    assert (d["exp_avg_sqs"][0].float() > 0).all()


def test_rounding_is_even_handed():
    """Over many seeds the states' mean is the exact value: each code is off by at most a step s with a
    variance of at most s^2 / 4, so the mean of n = 4000 by 5 s / (2 sqrt(n)) = 0.04 s at five deviations
    (and the numbers are multiples of 2^-16)."""
    n, runs = 512, 4000
    d = make([n], F32, F32, 8, seed=29)
    m0, v0 = values(d, "exp_avgs", "exp_avg_scales")[0], values(d, "exp_avg_sqs", "exp_avg_sq_scales")[0]
    g = d["grads"][0].double()
    sums = [torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(2)]
    for seed in range(runs):
        c = copy(d)
        step(c, 5, seed=seed)
        for s, name, sc in zip(sums, ("exp_avgs", "exp_avg_sqs"), ("exp_avg_scales", "exp_avg_sq_scales")):
            s += values(c, name, sc)[0]
    for s, ref in zip(sums, (B1 * m0 + (1 - B1) * g, B2 * v0 + (1 - B2) * g * g)):
        top = ref.abs().view(-1, 256).amax(1).repeat_interleave(256)
        y = ref.abs() / top * 448
        one = 2.0 ** (torch.floor(torch.log2(y.clamp_min(1e-9))).clamp(-6, 8) - 3) * top / 448
        ok = y > 2.0 ** -9                                        # (below, v is rounded up)
        assert ((s / runs - ref).abs() <= (0.04 + 2.0 ** -15) * one + 1e-6 * ref.abs())[ok].all()


def test_repeats_and_seeds():
    d = make([5000, 300], BF, BF, 8, seed=30)
    a, b, c = copy(d), copy(d), copy(d)
    step(a, 7, seed=1)
    step(b, 7, seed=1)
    step(c, 7, seed=2)
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for n in a if a[n] for x, y in zip(a[n], b[n]))
    assert not torch.equal(a["exp_avgs"][0].view(torch.uint8), c["exp_avgs"][0].view(torch.uint8))


def test_follows_torch_over_steps():
    """Ten steps beside torch's own optimizer in fp64: errors of a step stay, decayed, and add up."""
    d = make([300, 41], F32, F32, 32, seed=31, fresh=True)
    ref = [p.double().requires_grad_() for p in d["params"]]
    opt = torch.optim.AdamW(ref, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=WD)
    for t in range(1, 11):
        for g, p in zip(d["grads"], ref):
            g.copy_(torch.randn_like(g) * 0.1)
            p.grad = g.double()
        opt.step()
        step(d, t)
    for p, r in zip(d["params"], ref):
        assert (p.double() - r.detach()).abs().max() <= 10 * 20 * U * 4


def test_versions_rise():
    d = make([100], BF, BF, 8, master=True, seed=32)
    names = ("params", "exp_avgs", "exp_avg_sqs", "exp_avg_scales", "exp_avg_sq_scales", "masters")
    before, grads = [d[n][0]._version for n in names], d["grads"][0]._version
    step(d, 1)
    assert all(d[n][0]._version > b for n, b in zip(names, before)) and d["grads"][0]._version == grads


def test_how_far_codes_of_v_wander():
    """Under normal gradients, at the default beta2: without a bias (rounding is fair), and by some 23 % of the fp32 value.
    In units of v, a step takes it r (1 - beta2) off its code with E|r| = 0.97; rounding adds a variance of that times a code's
    step (0.068 to 0.125, 0.09 in the mean) and as much again because the block's largest, and with it the grid, moves alike; the
    average forgets at 2 (1 - beta2): sqrt(2 * 0.97 * 0.09 / 2) = 0.30 at most, 0.21 from the value's own steps alone.  Both are
    estimates to a quarter.  The mean of 51200 such values: 6 * 0.30 / sqrt(51200) = 0.008."""
    n, beta2 = 200 * 256, 0.999
    size = 10.0 ** (-2 * torch.rand(n, device="cuda"))
    kw = dict(lr=0.0, betas=(0.9, beta2), weight_decay=0.0)
    p = torch.zeros(n, device="cuda")
    v = size.square()
    scale = v.view(-1, 256).amax(1) / 448
    code = (v / scale.repeat_interleave(256)).to(E4M3)
    zero = lambda *s: torch.zeros(*s, device="cuda")
    m, m8, ms = zero(n), zero(n).to(E4M3), zero(200)
    for t in range(1, 4001):
        g = [size * torch.randn(n, device="cuda")]
        kda.kda_adamw_step([p], g, [m], [v], t, **kw)
        kda.kda_adamw_step([p], g, [m8], [code], t, exp_avg_scales=[ms], exp_avg_sq_scales=[scale], seed=3, **kw)
    ratio = code.double() * scale.double().repeat_interleave(256) / v.double()
    assert abs(ratio.mean().item() - 1) <= 0.008
    assert 0.75 * 0.21 <= ratio.std().item() <= 1.25 * 0.30
