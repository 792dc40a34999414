"""The linear recurrence's bounded waits, made to run out on the host's word: a limit of 1 ns, below what
the device's timer resolves, is over at once.  The calls end and report it, nothing of theirs is left under way, and the
next calls on the same workspace are right."""
import pytest
import torch

import kimi_delta_attention_gb300 as kda
from layer_ops_testutil import make_glr

pytestmark = pytest.mark.gpu
TIMEOUT = 5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.load_library()


# a tile alone; CTAs by themselves; clusters of as many as 16; packed; odd widths, which wait for the exchange alone
SHAPES = [([100], 64, False), ([600, 600], 16384, False), ([20000], 256, False), ([5000, 0, 3, 9000], 512, True), ([20000], 130, False)]


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lengths,D,packed", SHAPES, ids=lambda v: str(v).replace(" ", ""))
def test_runs_out(lengths, D, packed, io, monkeypatch):
    d = make_glr(lengths, D, io, torch.float32, packed=packed, seed=30)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    kw = dict(initial_state=d["s0"], cu_seqlens=d["cu"], workspace=ws)
    y, _ = ref = kda.kda_glr_fwd(d["x"], d["g"], **kw)
    calls = [(lambda: kda.kda_glr_fwd(d["x"], d["g"], **kw), ref)]
    back = lambda: kda.kda_glr_bwd(d["g"], y, d["dy"], d_final_state=d["ds"], **kw)
    calls.append((back, back()))
    for call, want in calls:
        for _ in range(3):
            with monkeypatch.context() as m:
                m.setenv("KDA_WAIT_LIMIT_NS", "1")
                call()
            assert kda.kda_read_device_status(ws) == TIMEOUT
        got = call()
        assert kda.kda_read_device_status(ws) == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want))
