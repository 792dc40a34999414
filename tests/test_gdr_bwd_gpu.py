"""The gated delta rule's gradients on the GPU against the recurrence's in 64 bits (by
autograd through the token recurrence) and against differences of the loss."""
import pytest
import torch

import kimi_delta_attention_gb300 as kda
from gdr_testutil import check, cuda, make, reference

pytestmark = pytest.mark.gpu
NAMES = ("q", "k", "v", "g", "beta", "s0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.load_library()


def backward(x):
    d = cuda(x)
    ws = torch.full((kda.kda_gdr_bwd_workspace_size(kda.make_shape(d["q"], d["v"], d["cu"])),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    got = kda.kda_gdr_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["do"], d["scale"], initial_state=d["s0"],
                          cu_seqlens=d["cu"], d_final_state=d["ds"], workspace=ws)
    assert kda.kda_read_device_status(ws) == 0
    return got


def compare(x):
    got = backward(x)
    if x["s0"] is None:
        ns = x["q"].shape[0] if x["cu"] is None else len(x["cu"]) - 1
        x = dict(x, s0=torch.zeros(ns, x["v"].shape[2], x["q"].shape[3], x["v"].shape[3]))
    for name, a, ref in zip(NAMES, got, reference(x, NAMES)):
        check(a, ref, "d" + name)


SHAPES = [
    dict(seqs=(1, 1), H=1, HV=1, K=128, V=128),
    dict(seqs=(2, 64), H=1, HV=1, K=128, V=128),
    dict(seqs=(1, 65), H=2, HV=2, K=128, V=64),
    dict(seqs=(1, 100), H=1, HV=3, K=64, V=128),
    dict(seqs=(2, 191), H=2, HV=4, K=64, V=64),
    dict(seqs=(1, 400), H=2, HV=4, K=128, V=128),
    dict(seqs=[1, 0, 64, 130, 2, 0, 63, 100], H=1, HV=2, K=128, V=128),
]


@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s['seqs']}-{s['H']}-{s['HV']}-{s['K']}-{s['V']}")
def test_gradients(shape, state):
    compare(make(state=state, seed=41, grads=True, **shape))


@pytest.mark.parametrize("K,V", [(128, 128), (64, 128), (128, 64)])
def test_gradients_of_many_sequences(K, V):
    compare(make([i * 7 % 5 if i % 50 else 90 for i in range(200)], 1, 2, K, V, state=True, seed=51, grads=True))


@pytest.mark.parametrize("gate", ["none", "strong", "cliff"])
def test_gradients_gates(gate):
    compare(make((1, 200), 1, 2, 128, 128, gate=gate, seed=42, grads=True))


def test_zero_beta():
    x = make((1, 150), 1, 2, 128, 128, seed=43, grads=True)
    x["beta"][0, 40:90] = 0.0
    compare(x)


def test_neighbours_do_not_meet():
    seqs = [70, 33, 100]
    x = make(seqs, 1, 2, 128, 128, seed=44, grads=True)
    a = backward(x)
    y = {n: t.clone() if torch.is_tensor(t) else t for n, t in x.items()}
    for n in ("q", "k", "v", "do", "g"):
        y[n][0, 70:103] = float("nan")
    y["v"][0, 80] = float("inf")
    y["s0"][1], y["ds"][1] = float("nan"), float("nan")
    b = backward(y)
    for s, t in zip(a[:5], b[:5]):
        assert torch.equal(s[0, :70], t[0, :70]) and torch.equal(s[0, 103:], t[0, 103:])
    assert torch.equal(a[5][[0, 2]], b[5][[0, 2]])


def test_repeats_bit_for_bit():
    x = make((2, 150), 2, 6, 128, 128, seed=45, grads=True)
    assert all(torch.equal(s, t) for s, t in zip(backward(x), backward(x)))


def test_against_differences():
    """Central differences of the loss through kda_gdr_fwd's own operation in 64 bits, along a
    random direction of each input."""
    x = make((1, 90), 1, 2, 64, 64, seed=46, grads=True)
    got = backward(x)
    gen = torch.Generator().manual_seed(1)

    def loss(y):
        o, S = reference(y)
        return ((o * x["do"].double()).sum() + (S * x["ds"].double()).sum()).item()

    for name, gr in zip(NAMES, got):
        u = torch.randn(x[name].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        moved = [loss(dict(x, **{name: x[name].double() + s * h * u})) for s in (1, -1)]
        num = (moved[0] - moved[1]) / (2 * h)
        ana = (gr.cpu().double() * u).sum().item()
        # a bf16 gradient's roundings, 2^-9 of each value, add up like a random walk along u
        slack = (3e-3 if gr.dtype == torch.bfloat16 else 1e-4) * (gr.cpu().double() * u).norm().item() * 4 + 1e-6
        assert abs(num - ana) <= slack + 1e-4 * abs(num), name


def test_on_another_stream():
    x = make((1, 300), 1, 2, 128, 128, seed=47, grads=True)
    ref = backward(x)
    d = cuda(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = kda.kda_gdr_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["do"], d["scale"], initial_state=d["s0"],
                          d_final_state=d["ds"], stream=side.cuda_stream)
    junk = [torch.randn(1 << 22, device="cuda") for _ in range(4)]
    side.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(ref, got)) and junk


def test_no_tokens():
    x = cuda(make([0, 0], 1, 2, 128, 128, seed=48, grads=True))
    got = kda.kda_gdr_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], initial_state=x["s0"],
                          cu_seqlens=x["cu"], d_final_state=x["ds"])
    assert torch.equal(got[5], x["ds"])


def test_refusals():
    x = cuda(make((1, 8), 2, 4, 128, 128, seed=1, grads=True))
    args = [x[n] for n in ("q", "k", "v", "g", "beta", "do")]

    def refused(fn, code=1):
        with pytest.raises(kda.KdaError) as e:
            fn()
        assert e.value.code == code

    refused(lambda: kda.kda_gdr_bwd(*[t.float() for t in args]), 2)
    refused(lambda: kda.kda_gdr_bwd(*args[:5], args[5].float()))
    refused(lambda: kda.kda_gdr_bwd(*args[:5], args[5][:, :4].contiguous()))
    refused(lambda: kda.kda_gdr_bwd(*args, d_final_state=x["ds"].bfloat16()))
    refused(lambda: kda.kda_gdr_bwd(*args, scale=0.0))
    refused(lambda: kda.kda_gdr_bwd(*args, workspace=torch.empty(256, dtype=torch.uint8, device="cuda")), 6)


@pytest.mark.parametrize("limit", ["1", "1000"])
def test_wait_limit(limit, monkeypatch):
    """A wait limit too short for the kernels' copies: the calls complete, with their result or
    a reported timeout, and the next calls are right."""
    x = make((2, 400), 2, 4, 128, 128, seed=49, grads=True)
    d = cuda(x)
    args = [d[n] for n in ("q", "k", "v", "g", "beta")]
    fws = torch.empty(kda.kda_gdr_fwd_workspace_size(kda.make_shape(d["q"], d["v"])), dtype=torch.uint8, device="cuda")
    bws = torch.empty(kda.kda_gdr_bwd_workspace_size(kda.make_shape(d["q"], d["v"])), dtype=torch.uint8, device="cuda")
    fwd = lambda: kda.kda_gdr_fwd(*args, d["scale"], initial_state=d["s0"], workspace=fws)
    bwd = lambda: kda.kda_gdr_bwd(*args, d["do"], d["scale"], initial_state=d["s0"], d_final_state=d["ds"], workspace=bws)
    ref_f, ref_b = fwd(), bwd()
    torch.cuda.synchronize()
    monkeypatch.setenv("KDA_WAIT_LIMIT_NS", limit)
    got = fwd()
    status = kda.kda_read_device_status(fws)
    assert status in (0, 5) and (status == 5 or all(torch.equal(s, t) for s, t in zip(ref_f, got)))
    got = bwd()
    status = kda.kda_read_device_status(bws)
    assert status in (0, 5) and (status == 5 or all(torch.equal(s, t) for s, t in zip(ref_b, got)))
    monkeypatch.delenv("KDA_WAIT_LIMIT_NS")
    assert all(torch.equal(s, t) for s, t in zip(ref_f, fwd())) and kda.kda_read_device_status(fws) == 0
    assert all(torch.equal(s, t) for s, t in zip(ref_b, bwd())) and kda.kda_read_device_status(bws) == 0


@pytest.mark.parametrize("K,V", [(128, 128), (64, 64), (128, 64)])
@pytest.mark.parametrize("H,HV", [(4, 8), (8, 8)])
def test_gradients_unit_after_unit(K, V, H, HV):
    """More (chunk, value head) pairs than processors, most chunks partial: a CTA's buffers pass from one
    pair to the next.  Against 64 bits, and each sequence's bits are those of a call of its own,
    where no CTA meets a second pair."""
    seqs = [70, 1, 64, 33] * 8
    x = make(seqs, H, HV, K, V, state=True, seed=52, grads=True)
    got = backward(x)
    for name, a, ref in zip(NAMES, got, reference(x, NAMES)):
        check(a, ref, "d" + name)
    at = 0
    for i, n in enumerate(seqs[:8]):
        one = {m: t[:, at:at + n].contiguous() if m in ("q", "k", "v", "g", "beta", "do") else t for m, t in x.items()}
        one.update(cu=None, s0=x["s0"][i:i + 1], ds=x["ds"][i:i + 1])
        alone = backward(one)
        assert all(torch.equal(s[:, at:at + n], t) for s, t in zip(got[:5], alone[:5])) and torch.equal(got[5][i:i + 1], alone[5])
        at += n


def test_no_sound_sequence():
    """Bounds that leave no chunk at all: the state's gradient passes through and the status, read by
    the next work on the stream, is there."""
    x = cuda(make([100], 1, 2, 128, 128, seed=53, grads=True))
    cu, status = torch.tensor([5, 100], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(20):
        status.zero_()
        got = kda.kda_gdr_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["do"], initial_state=x["s0"], cu_seqlens=cu,
                              d_final_state=x["ds"], status=status)
        seen = status.clone(), got[5].clone()
        assert seen[0].item() == 2 and torch.equal(seen[1], x["ds"])
