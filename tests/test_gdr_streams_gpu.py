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
