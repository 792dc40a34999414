"""The gated delta rule with a scalar gate on the GPU against the recurrence in 64 bits:
forward and serving step."""
import pytest
import torch

import kimi_delta_attention_gb300 as kda
from gdr_testutil import check, cuda, make, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.load_library()


def forward(x, **kw):
    d = cuda(x)
    ws = torch.full((kda.kda_gdr_fwd_workspace_size(kda.make_shape(d["q"], d["v"], d["cu"])),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    o, S = kda.kda_gdr_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["scale"], initial_state=d["s0"],
                           cu_seqlens=d["cu"], workspace=ws, **kw)
    assert kda.kda_read_device_status(ws) == 0
    return o, S


SHAPES = [
    dict(seqs=(1, 1), H=1, HV=1, K=128, V=128),
    dict(seqs=(2, 63), H=2, HV=2, K=128, V=128),
    dict(seqs=(1, 64), H=1, HV=3, K=128, V=64),
    dict(seqs=(3, 65), H=2, HV=4, K=64, V=128),
    dict(seqs=(2, 257), H=1, HV=2, K=64, V=64),
    dict(seqs=(1, 700), H=4, HV=8, K=128, V=128),
    dict(seqs=[1, 0, 64, 130, 2, 0, 63, 200], H=2, HV=6, K=128, V=128),
    dict(seqs=[0, 0], H=1, HV=2, K=128, V=128),
    dict(seqs=[5, 128, 333], H=3, HV=3, K=64, V=128),
]


@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s['seqs']}-{s['H']}-{s['HV']}-{s['K']}-{s['V']}")
def test_forward(shape, io, state):
    x = make(io=io, state=state, seed=11, **shape)
    o, S = forward(x)
    o_ref, S_ref = reference(x)
    check(o, o_ref, "o")
    check(S, S_ref, "state")


@pytest.mark.parametrize("K,V", [(128, 128), (64, 128), (128, 64), (64, 64)])
@pytest.mark.parametrize("state", [False, True])
def test_forward_more_chains_than_processors(K, V, state):
    x = make([70, 0, 193, 1, 64], 8, 32, K, V, state=state, seed=21)
    o, S = forward(x)
    o_ref, S_ref = reference(x)
    check(o, o_ref, "o")
    check(S, S_ref, "state")


@pytest.mark.parametrize("count", [200, 300])
def test_forward_hundreds_of_sequences(count):
    """Sequences start the longest first, up to a count; every one is done once either way."""
    x = make([i * 7 % 5 if i % 50 else 90 for i in range(count)], 1, 1, 128, 128, state=True, seed=22)
    o, S = forward(x)
    o_ref, S_ref = reference(x)
    check(o, o_ref, "o")
    check(S, S_ref, "state")


@pytest.mark.parametrize("gate", ["none", "strong", "cliff"])
def test_forward_gates(gate):
    x = make((1, 300), 2, 4, 128, 128, gate=gate, seed=5)
    o, S = forward(x)
    o_ref, S_ref = reference(x)
    check(o, o_ref, "o")
    check(S, S_ref, "state")


def test_forward_closed_gate_and_zero_beta():
    """g = -inf forgets everything before its token; beta = 0 writes nothing."""
    x = make((1, 200), 1, 2, 128, 128, seed=6)
    x["g"][0, 70] = float("-inf")
    x["beta"][0, 100:140] = 0.0
    o, S = forward(x)
    o_ref, S_ref = reference(x)
    check(o, o_ref, "o")
    check(S, S_ref, "state")


def test_forward_neighbours_do_not_meet():
    """A packed sequence full of NaN and infinities leaves the others' bits alone."""
    seqs = [70, 33, 100]
    x = make(seqs, 2, 2, 128, 128, seed=7)
    o, S = forward(x)
    y = {n: t.clone() if torch.is_tensor(t) else t for n, t in x.items()}
    for n in ("q", "k", "v"):
        y[n][0, 70:103] = float("nan")
        y[n][0, 80] = float("inf")
    y["g"][0, 70:103] = float("nan")
    y["s0"][1] = float("nan")
    o2, S2 = forward(y)
    for a, b in ((0, 70), (103, 203)):
        assert torch.equal(o[0, a:b], o2[0, a:b])
    assert torch.equal(S[0], S2[0]) and torch.equal(S[2], S2[2])


def test_forward_repeats_and_state_in_place():
    x = make((2, 150), 2, 4, 128, 128, seed=8)
    o, S = forward(x)
    o2, S2 = forward(x)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    d = cuda(x)
    o3, S3 = kda.kda_gdr_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["scale"], initial_state=d["s0"],
                             final_state=d["s0"])
    assert S3.data_ptr() == d["s0"].data_ptr()
    assert torch.equal(o, o3) and torch.equal(S, S3)


def test_forward_continues():
    """Two calls over the halves of a sequence give the state of one call over it."""
    x = make((1, 230), 1, 2, 128, 128, seed=9)
    d = cuda(x)
    part = lambda a, b, s: kda.kda_gdr_fwd(*(d[n][:, a:b].contiguous() for n in ("q", "k", "v", "g", "beta")),
                                           d["scale"], initial_state=s)
    o1, S1 = part(0, 101, d["s0"])
    o2, S2 = part(101, 230, S1)
    o_ref, S_ref = reference(x)
    check(torch.cat([o1, o2], 1), o_ref, "o")
    check(S2, S_ref, "state")


def test_forward_on_another_stream():
    x = make((1, 500), 2, 2, 128, 128, seed=10)
    d = cuda(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o, S = kda.kda_gdr_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["scale"], initial_state=d["s0"],
                           stream=side.cuda_stream)
    junk = [torch.randn(1 << 20, device="cuda") for _ in range(4)]   # would take a freed workspace
    side.synchronize()
    o_ref, S_ref = reference(x)
    check(o, o_ref, "o")
    check(S, S_ref, "state")
    assert junk


def test_forward_reports_bad_cu_seqlens():
    x = make([40, 60], 1, 1, 128, 128, seed=3)
    d = cuda(x)
    d["cu"] = torch.tensor([0, 140, 100], dtype=torch.int32, device="cuda")
    ws = torch.empty(kda.kda_gdr_fwd_workspace_size(kda.make_shape(d["q"], d["v"], d["cu"])), dtype=torch.uint8,
                     device="cuda")
    kda.kda_gdr_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["scale"], cu_seqlens=d["cu"], workspace=ws)
    assert kda.kda_read_device_status(ws) == 7


@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,HV,K,V", [(1, 1, 1, 128, 128), (5, 2, 6, 128, 64), (33, 1, 2, 64, 128), (3, 16, 32, 64, 64)])
def test_step(B, H, HV, K, V, T, io):
    x = make((B, T), H, HV, K, V, io=io, seed=20 + T)
    d = cuda(x)
    state = d["s0"].clone()
    o = kda.kda_gdr_step(d["q"], d["k"], d["v"], d["g"], d["beta"], state, d["scale"])
    o_ref, S_ref = reference(x)
    check(o, o_ref, "o")
    check(state, S_ref, "state")


@pytest.mark.parametrize("T", [1, 3])
def test_step_pool(T):
    """Slots in any order, empty rows, a slot out of range; the rest of the pool keeps its bits."""
    B, HV = 6, 4
    x = make((B, T), 2, HV, 128, 128, seed=30)
    d = cuda(x)
    pool = torch.randn(9, HV, 128, 128, device="cuda")
    slots = torch.tensor([7, -1, 0, 4, 9, -2147483648], dtype=torch.int32, device="cuda")
    live = [(0, 7), (2, 0), (3, 4)]
    for b, s in live:
        pool[s] = d["s0"][b]
    before = pool.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = kda.kda_gdr_step(d["q"], d["k"], d["v"], d["g"], d["beta"], pool, d["scale"], slots=slots, status=status)
    o_ref, S_ref = reference(x)
    for b, s in live:
        check(o[b], o_ref[b], "o")
        check(pool[s], S_ref[b], "state")
    assert o[[1, 4, 5]].abs().max().item() == 0
    kept = [i for i in range(9) if i not in (7, 0, 4)]
    assert torch.equal(pool[kept], before[kept])
    assert status.item() == 2 and kda.kda_read_device_status(status) == 7


def test_step_empty_row_with_nan_inputs():
    x = make((2, 1), 1, 1, 128, 128, seed=31)
    x["v"][1] = float("nan")
    x["k"][1] = float("inf")
    d = cuda(x)
    pool = d["s0"].clone()
    slots = torch.tensor([1, -1], dtype=torch.int32, device="cuda")
    o = kda.kda_gdr_step(d["q"], d["k"], d["v"], d["g"], d["beta"], pool, d["scale"], slots=slots)
    assert torch.isfinite(o).all() and torch.equal(pool[0], d["s0"][0])


def test_prefill_then_steps():
    """A chunked prefill followed by single steps is the recurrence over all tokens."""
    x = make((2, 75), 2, 4, 128, 128, seed=32)
    d = cuda(x)
    at = lambda a, b: [d[n][:, a:b].contiguous() for n in ("q", "k", "v", "g", "beta")]
    o, S = kda.kda_gdr_fwd(*at(0, 70), d["scale"], initial_state=d["s0"])
    outs = [o] + [kda.kda_gdr_step(*at(t, t + 1), S, d["scale"]) for t in range(70, 75)]
    o_ref, S_ref = reference(x)
    check(torch.cat(outs, 1), o_ref, "o")
    check(S, S_ref, "state")


def test_refusals():
    x = cuda(make((1, 8), 2, 4, 128, 128, seed=1))
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]

    def refused(fn, code=1):
        with pytest.raises(kda.KdaError) as e:
            fn()
        assert e.value.code == code

    refused(lambda: kda.kda_gdr_fwd(*[t.cpu() for t in args]))
    refused(lambda: kda.kda_gdr_fwd(args[0].half(), *args[1:]))
    refused(lambda: kda.kda_gdr_fwd(args[0].transpose(1, 2), *args[1:]))
    refused(lambda: kda.kda_gdr_fwd(*args[:3], args[3][..., None].expand(1, 8, 4, 128), args[4]))   # a gate per dim
    refused(lambda: kda.kda_gdr_fwd(*args, scale=-1.0))
    refused(lambda: kda.kda_gdr_fwd(*args, initial_state=x["s0"][:, :2].contiguous()))
    refused(lambda: kda.kda_gdr_fwd(*args, cu_seqlens=torch.tensor([0, 8], device="cuda")))         # int64
    refused(lambda: kda.kda_gdr_fwd(*args, out=args[2]))
    refused(lambda: kda.kda_gdr_fwd(*args, workspace=torch.empty(8, dtype=torch.uint8, device="cuda")), 6)
    cut = [t[..., :96].contiguous() for t in args[:3]]
    refused(lambda: kda.kda_gdr_fwd(*cut, *args[3:]), 2)
    refused(lambda: kda.kda_gdr_step(*args, x["s0"].bfloat16()))
    refused(lambda: kda.kda_gdr_step(*args, torch.cat([x["s0"]] * 2)))
    refused(lambda: kda.kda_gdr_step(*args, x["s0"], slots=torch.zeros(1, dtype=torch.int64, device="cuda")))


@pytest.mark.parametrize("B,T", [(0, 1), (0, 0), (3, 0)])
def test_step_without_requests(B, T):
    """A serving loop without a live request: the pool keeps its bits."""
    q = torch.empty(B, T, 2, 128, device="cuda", dtype=torch.bfloat16)
    v, g = torch.empty(B, T, 4, 128, device="cuda", dtype=torch.bfloat16), torch.empty(B, T, 4, device="cuda")
    pool = torch.randn(5, 4, 128, 128, device="cuda")
    before, slots = pool.clone(), torch.arange(B, dtype=torch.int32, device="cuda")
    o = kda.kda_gdr_step(q, q, v, g, g, pool, slots=slots)
    assert o.shape == (B, T, 4, 128) and torch.equal(pool, before)
