"""What a call on another stream than the current one allocates comes from that stream's pool."""
import pytest
import torch

import kimi_delta_attention_gb300 as kda
from kimi_delta_attention_gb300 import workloads as W

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


@pytest.fixture(scope="module")
def problem():
    x = W.make_inputs(2, 128, 2, 4, 128, 128, "bf16", seed=71, init_state=True).to("cuda")
    do = torch.randn(x.v.shape, device="cuda").bfloat16()
    gate = (torch.randn(x.g.shape, device="cuda").bfloat16(), torch.randn(4, device="cuda"), torch.zeros(4, 128, device="cuda"))
    args = (x.q, x.k, x.v, x.g, x.beta)
    first = [t[:, :1].contiguous() for t in args]
    h, _ = kda.kda_chunk_states(*args, initial_state=x.initial_state)
    s = dict(initial_state=x.initial_state)
    return {
        "forward": lambda **kw: kda.kda_chunk_fwd(*args, x.scale, **s, **kw),
        "recurrent": lambda **kw: kda.kda_recurrent_fwd(*args, x.scale, **s, **kw),
        "gated": lambda **kw: kda.kda_chunk_fwd_gated(x.q, x.k, x.v, gate[0], x.beta, gate[1], gate[2], **s, **kw),
        "states": lambda **kw: kda.kda_chunk_states(*args, **s, **kw),
        "output": lambda **kw: (kda.kda_chunk_output(*args, h, x.scale, **kw),),
        "decode": lambda **kw: (kda.kda_decode(*first, x.initial_state.clone(), x.scale, **kw),),
        "backward": lambda **kw: kda.kda_backward(*args, do, x.scale, **s, **kw),
    }


@pytest.mark.parametrize("name", ["forward", "recurrent", "gated", "states", "output", "decode", "backward"])
def test_blocks_come_from_the_stream_that_writes_them(problem, name):
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


def test_inputs_are_kept_for_the_stream():
    """Inputs given up after a call on a busy side stream are not handed out again before it is done."""
    side = torch.cuda.Stream()
    x = W.make_inputs(2, 128, 2, 4, 128, 128, "bf16", seed=73, init_state=True).to("cuda")
    args = [x.q, x.k, x.v, x.g, x.beta]
    h, _ = kda.kda_chunk_states(*args)
    calls = [(lambda *a, **kw: kda.kda_chunk_fwd(*a[:5], initial_state=a[5], **kw), args + [x.initial_state]),
             (lambda *a, **kw: kda.kda_decode(*a, **kw), [t[:, :1].contiguous() for t in args] + [x.initial_state]),
             (lambda *a, **kw: kda.kda_chunk_states(*a, **kw), args),
             (lambda *a, **kw: kda.kda_chunk_output(*a, **kw), args + [h]),
             (lambda *a, **kw: kda.kda_backward(*a, **kw), args + [x.v])]
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
