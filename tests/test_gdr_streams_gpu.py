"""Calls of the scalar-gate rule and of layer norm on another stream than the current one, and
captured in graphs."""
import pytest
import torch

import kimi_delta_attention_gb300 as kda
from gdr_testutil import cuda, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.load_library()


def pool_of(t):
    """The raw stream whose pool a tensor's block belongs to."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no segment")


def calls(d, rows, dy, mean, rstd):
    rule = [d[n] for n in ("q", "k", "v", "g", "beta")]
    return {
        "fwd": lambda **kw: kda.kda_gdr_fwd(*rule, d["scale"], initial_state=d["s0"], **kw),
        "bwd": lambda **kw: kda.kda_gdr_bwd(*rule, d["do"], d["scale"], initial_state=d["s0"], d_final_state=d["ds"], **kw),
        "step": lambda **kw: (kda.kda_gdr_step(*(t[:, :1].contiguous() for t in rule), d["s0"].clone(), d["scale"], **kw),),
        "norm": lambda **kw: kda.kda_layer_norm_fwd(rows, **kw),
        "norm_bwd": lambda **kw: kda.kda_layer_norm_bwd(rows, dy, None, mean, rstd, **kw),
    }


@pytest.fixture(scope="module")
def problem():
    d = cuda(make((2, 100), 2, 4, 128, 128, seed=61, grads=True))
    rows, dy = torch.randn(300, 512, device="cuda"), torch.randn(300, 512, device="cuda")
    _, mean, rstd = kda.kda_layer_norm_fwd(rows)
    return calls(d, rows, dy, mean, rstd)


@pytest.mark.parametrize("name", ["fwd", "bwd", "step", "norm", "norm_bwd"])
def test_blocks_come_from_the_stream_that_writes_them(problem, name):
    """Results written on a side stream never lie in a block that the current stream has freed
    but may still be reading."""
    call = problem[name]
    ref = [t for t in call() if t is not None]
    side = torch.cuda.Stream()
    freed = [torch.empty_like(t) for t in ref]
    freed = {t.data_ptr() for t in freed}          # (given back to the current stream's pool)
    torch.cuda.synchronize()
    got = [t for t in call(stream=side.cuda_stream) if t is not None]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    assert not freed & {t.data_ptr() for t in got}
    assert all(pool_of(t) == side.cuda_stream for t in got)
    again = [t for t in call(stream=torch.cuda.current_stream().cuda_stream) if t is not None]
    assert all(pool_of(t) == torch.cuda.current_stream().cuda_stream for t in again)
    assert all(torch.equal(a, b) for a, b in zip(ref, again))


def captured(call, inputs, others):
    """A call captured in a graph and replayed after its inputs took the values of `others`."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()                                     # (first call: set-up of the kernels)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for a, b in zip(inputs, others):
        a.copy_(b)
    graph.replay()
    got = [t.clone() for t in out if t is not None]
    for a, b in zip(inputs, others):
        a.copy_(b)                                 # (what the call updates in place)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, (t for t in out if t is not None)))
    for a, b in zip(inputs, others):
        a.copy_(b)
    ref = [t for t in call() if t is not None]
    assert len(ref) == len(got) and all(torch.equal(a, b) for a, b in zip(ref, got))


RULE = ("q", "k", "v", "g", "beta", "s0", "do", "ds")
SHAPES = {"prompt": dict(seqs=(1, 37), H=4, HV=8, K=128, V=128), "thin": dict(seqs=(1, 300), H=2, HV=4, K=128, V=128),
          "wide": dict(seqs=[70, 1, 200], H=8, HV=32, K=128, V=128), "small": dict(seqs=[300, 1, 100], H=16, HV=32, K=64, V=64)}


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rule_in_a_graph(shape):
    x, y = (cuda(make(seed=s, grads=True, **SHAPES[shape])) for s in (65, 66))
    names = [n for n in RULE if x[n] is not None]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]
    fwd = lambda: kda.kda_gdr_fwd(*args, x["scale"], initial_state=x["s0"], cu_seqlens=x["cu"], status=status)
    bwd = lambda: kda.kda_gdr_bwd(*args, x["do"], x["scale"], initial_state=x["s0"], cu_seqlens=x["cu"], d_final_state=x["ds"],
                                  status=status)
    for call in (fwd, bwd):
        keep = [x[n].clone() for n in names]
        captured(call, [x[n] for n in names], [y[n] for n in names])
        for n, t in zip(names, keep):
            x[n].copy_(t)
    assert status.item() == 0


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_step_in_a_graph(io):
    x, y = (cuda(make((6, 1), 2, 4, 128, 128, io=io, seed=s)) for s in (67, 68))
    names = ["q", "k", "v", "g", "beta", "s0"]
    slots = torch.tensor([3, -1, 0, 5, 4, 1], dtype=torch.int32, device="cuda")
    args = [x[n] for n in names[:5]]
    captured(lambda: (kda.kda_gdr_step(*args, x["s0"], x["scale"], slots=slots), x["s0"]),
             [x[n] for n in names] + [slots], [y[n] for n in names] + [slots.flip(0)])


@pytest.mark.parametrize("rows,D,io", [(24, 4096, torch.bfloat16), (3000, 1001, torch.float32), (9, 20000, torch.bfloat16)])
def test_norm_in_a_graph(rows, D, io):
    rn = lambda *s: torch.randn(*s, device="cuda")
    x, dy, w, b = rn(rows, D).to(io), rn(rows, D).to(io), rn(D), rn(D)

    def call():
        y, mean, rstd = kda.kda_layer_norm_fwd(x, w, b)
        return (y, mean, rstd, *kda.kda_layer_norm_bwd(x, dy, w, mean, rstd))

    captured(call, [x, dy, w, b], [rn(rows, D).to(io), rn(rows, D).to(io), rn(D), rn(D)])


def test_inputs_are_kept_for_the_stream():
    """Inputs given up after a call on a busy side stream are not handed out again before it is done."""
    side = torch.cuda.Stream()
    x = cuda(make((2, 100), 2, 4, 128, 128, seed=69, grads=True))
    rule = [x[n] for n in ("q", "k", "v", "g", "beta")]
    rows = torch.randn(300, 512, device="cuda")
    _, mean, rstd = kda.kda_layer_norm_fwd(rows)
    calls = [(lambda *a, **kw: kda.kda_gdr_fwd(*a[:5], initial_state=a[5], **kw), rule + [x["s0"]]),
             (lambda *a, **kw: kda.kda_gdr_bwd(*a[:6], initial_state=a[6], d_final_state=a[7], **kw), rule + [x["do"], x["s0"], x["ds"]]),
             (lambda *a, **kw: (kda.kda_gdr_step(*a, **kw),), [t[:, :1].contiguous() for t in rule] + [x["s0"]]),
             (lambda *a, **kw: kda.kda_layer_norm_fwd(*a, **kw), [rows]),
             (lambda *a, **kw: kda.kda_layer_norm_bwd(*a[:2], None, *a[2:], **kw), [rows, rows + 1, mean, rstd])]
    for call, tensors in calls:
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(int(2e7))            # some 10 ms
        given = [t.clone() for t in tensors]
        torch.cuda.current_stream().synchronize()
        kept = {t.data_ptr() for t in given}
        out = call(*given, stream=side.cuda_stream)
        sizes = [(t.shape, t.dtype) for t in given]
        del given
        again = [torch.empty(s, dtype=d, device="cuda") for s, d in sizes]
        assert not kept & {t.data_ptr() for t in again}
        side.synchronize()
        ref = call(*[t.clone() for t in tensors])
        assert all(torch.equal(a, b) for a, b in zip(out, ref) if a is not None)


@pytest.mark.parametrize("name", ["fwd", "bwd", "step", "norm", "norm_bwd"])
def test_default_stream_by_its_raw_number(problem, name):
    """stream=0 is the legacy default stream, for allocations too, whichever stream is current."""
    call = problem[name]
    ref = [t for t in call() if t is not None]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = [t for t in call(stream=0) if t is not None]
        torch.cuda.synchronize()
        assert all(pool_of(t) == 0 for t in got)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_status_on_the_default_stream():
    x = cuda(make([100], 1, 2, 128, 128, seed=70))
    cu, status = torch.tensor([0, 90], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        kda.kda_gdr_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], cu_seqlens=cu, stream=0, status=status)
        torch.cuda.synchronize()
    assert status.item() == 2
