"""Calls of the recurrence, group norm and the AdamW step on another stream than the current one, captured
in graphs, and two at once."""
import pytest
import torch

import kimi_delta_attention_gb300 as kda
from layer_ops_testutil import make_glr
from test_gdr_streams_gpu import captured, pool_of

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.load_library()


def adamw_problem(seed=0, bits=8):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda n: torch.randn(n, generator=gen, device="cuda")
    sizes = [3000, 17, 513]
    d = [[rn(n).to(BF) for n in sizes], [rn(n).to(BF) for n in sizes]]
    if bits == 32:
        return d + [[rn(n) for n in sizes], [rn(n).square() for n in sizes]]
    return d + [[rn(n).to(torch.float8_e4m3fn) for n in sizes], [rn(n).abs().to(torch.float8_e4m3fn) for n in sizes],
                [rn(-(-n // 256)).abs() for n in sizes], [rn(-(-n // 256)).abs() for n in sizes]]


def adamw(d, **kw):
    more = dict(exp_avg_scales=d[4], exp_avg_sq_scales=d[5]) if len(d) == 6 else {}
    kda.kda_adamw_step(*d[:4], 3, **more, **kw)
    return [t for i, x in enumerate(d) if i != 1 for t in x]


def copies(d):
    return [[t.clone() for t in x] for x in d]


def bytes_of(t):
    return t.contiguous().view(torch.uint8)


@pytest.fixture(scope="module")
def problem():
    d = make_glr([100, 300], 264, BF, F32, seed=61)
    y, _ = kda.kda_glr_fwd(d["x"], d["g"], initial_state=d["s0"], cu_seqlens=d["cu"])
    x, dy, w = (torch.randn(*s, device="cuda") for s in ((3, 500, 96), (3, 500, 96), (96,)))
    _, mean, rstd = kda.kda_group_norm_fwd(x, 4, w)
    rows, step = torch.randn(40, 512, device="cuda"), [t[:, :2].contiguous() for t in (d["x"], d["g"])]
    return {
        "glr": lambda **kw: kda.kda_glr_fwd(d["x"], d["g"], initial_state=d["s0"], cu_seqlens=d["cu"], **kw),
        "glr_bwd": lambda **kw: kda.kda_glr_bwd(d["g"], y, d["dy"], initial_state=d["s0"], cu_seqlens=d["cu"], d_final_state=d["ds"], **kw),
        "glr_step": lambda **kw: (kda.kda_glr_step(*step, d["s0"][:1].clone(), **kw),),
        "gn": lambda **kw: kda.kda_group_norm_fwd(x, 4, w, activation="silu", **kw),
        "gn_rows": lambda **kw: kda.kda_group_norm_fwd(rows, 4, **kw),
        "gn_bwd": lambda **kw: kda.kda_group_norm_bwd(x, dy, 4, w, None, mean, rstd, **kw),
    }


NAMES = ["glr", "glr_bwd", "glr_step", "gn", "gn_rows", "gn_bwd"]


@pytest.mark.parametrize("name", NAMES)
def test_blocks_come_from_the_stream_that_writes_them(problem, name):
    call = problem[name]
    ref = [t for t in call() if t is not None]
    side = torch.cuda.Stream()
    freed = {t.data_ptr() for t in [torch.empty_like(t) for t in ref]}
    torch.cuda.synchronize()
    got = [t for t in call(stream=side.cuda_stream) if t is not None]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    assert not freed & {t.data_ptr() for t in got} and all(pool_of(t) == side.cuda_stream for t in got)
    again = [t for t in call(stream=torch.cuda.current_stream().cuda_stream) if t is not None]
    assert all(torch.equal(a, b) for a, b in zip(ref, again))


@pytest.mark.parametrize("name", NAMES)
def test_default_stream_by_its_raw_number(problem, name):
    call = problem[name]
    ref = [t for t in call() if t is not None]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = [t for t in call(stream=0) if t is not None]
        torch.cuda.synchronize()
        assert all(pool_of(t) == 0 for t in got)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_on_another_stream(bits):
    d = adamw_problem(bits=bits)
    ref = adamw(copies(d))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = adamw(copies(d), stream=side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(bytes_of(a), bytes_of(b)) for a, b in zip(ref, got))


def test_inputs_are_kept_for_the_stream():
    side = torch.cuda.Stream()
    d = make_glr([200], 256, BF, F32, packed=False, seed=62)
    y, _ = kda.kda_glr_fwd(d["x"], d["g"])
    x = torch.randn(60, 512, device="cuda")
    _, mean, rstd = kda.kda_group_norm_fwd(x, 4)
    calls = [(lambda *a, **kw: kda.kda_glr_fwd(*a, **kw), [d["x"], d["g"], d["s0"]]),
             (lambda *a, **kw: kda.kda_glr_bwd(*a, **kw), [d["g"], y, d["dy"], d["s0"]]),
             (lambda *a, **kw: (kda.kda_glr_step(*a, **kw),), [d["x"][:, :1].contiguous(), d["g"][:, :1].contiguous(), d["s0"]]),
             (lambda *a, **kw: kda.kda_group_norm_fwd(a[0], 4, **kw), [x]),
             (lambda *a, **kw: kda.kda_group_norm_bwd(*a[:2], 4, None, None, *a[2:], **kw), [x, x + 1, mean, rstd])]
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
        again = [torch.empty(s, dtype=t, device="cuda") for s, t in sizes]
        assert not kept & {t.data_ptr() for t in again}
        side.synchronize()
        ref = call(*[t.clone() for t in tensors])
        assert all(torch.equal(a, b) for a, b in zip(out, ref) if a is not None)


# ------------------------------------------------------------------ graphs --
@pytest.mark.parametrize("lengths,D,io", [([37], 1024, BF), ([300, 1, 0, 2000], 264, BF), ([700, 90], 129, F32)])
def test_recurrence_in_a_graph(lengths, D, io):
    x, y = (make_glr(lengths, D, io, F32, seed=s) for s in (65, 66))
    names = ["x", "g", "s0", "dy", "ds"]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        out, state = kda.kda_glr_fwd(x["x"], x["g"], initial_state=x["s0"], cu_seqlens=x["cu"], status=status)
        return (out, state, *kda.kda_glr_bwd(x["g"], out, x["dy"], initial_state=x["s0"], cu_seqlens=x["cu"], d_final_state=x["ds"],
                                             status=status))

    captured(call, [x[n] for n in names], [y[n] for n in names])
    assert status.item() == 0


def test_step_in_a_graph():
    x, y = (make_glr([2] * 6, 200, BF, F32, packed=False, seed=s) for s in (67, 68))
    slots = torch.tensor([3, -1, 0, 5, 4, 1], dtype=torch.int32, device="cuda")
    captured(lambda: (kda.kda_glr_step(x["x"], x["g"], x["s0"], slots=slots), x["s0"]), [x["x"], x["g"], x["s0"], slots],
             [y["x"], y["g"], y["s0"], slots.flip(0)])


@pytest.mark.parametrize("shape,groups,io", [((24, 4096), 32, BF), ((3, 500, 96), 4, F32), ((2, 3000, 512), 8, BF), ((5, 7, 33), 3, BF)])
def test_group_norm_in_a_graph(shape, groups, io):
    rn = lambda *s: torch.randn(*s, device="cuda")
    x, dy, w, b = rn(*shape).to(io), rn(*shape).to(io), rn(shape[-1]), rn(shape[-1])

    def call():
        y, mean, rstd = kda.kda_group_norm_fwd(x, groups, w, b, activation="silu")
        return (y, mean, rstd, *kda.kda_group_norm_bwd(x, dy, groups, w, b, mean, rstd, "silu"))

    captured(call, [x, dy, w, b], [rn(*shape).to(io), rn(*shape).to(io), rn(shape[-1]), rn(shape[-1])])


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_in_a_graph(bits):
    d, e = adamw_problem(1, bits), adamw_problem(2, bits)
    flat = lambda x: [t for c in x for t in c]
    start = copies(d)
    ref = adamw(copies(d))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        adamw(d)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = adamw(d)
    for values, want in ((start, ref), (e, adamw(copies(e)))):
        for a, b in zip(flat(d), flat(values)):
            a.copy_(b)
        graph.replay()
        assert all(torch.equal(bytes_of(a), bytes_of(b)) for a, b in zip(out, want))


def test_two_at_once():
    """Calls that overlap on two streams, each with a workspace of its own."""
    a, b = (make_glr([3000, 100], 512, BF, F32, seed=s) for s in (71, 72))
    x = torch.randn(2, 3000, 512, device="cuda")
    calls = [lambda: kda.kda_glr_fwd(a["x"], a["g"], cu_seqlens=a["cu"]), lambda: kda.kda_glr_fwd(b["x"], b["g"], cu_seqlens=b["cu"]),
             lambda: kda.kda_group_norm_fwd(x, 8)]
    refs = [call() for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        outs = []
        for call, s in zip(calls, streams):
            with torch.cuda.stream(s):
                outs.append(call())
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for o, r in zip(outs, refs) for p, q in zip(o, r))
