"""The scalar-gate rule's bounded waits, made to run out on the host's word: a limit of 1 ns is
over before any copy can arrive.  The calls end, report it, leave work undone where a chain gave
up, and the next calls on the same workspace are right."""
import pytest
import torch

import kimi_delta_attention_gb300 as kda
from gdr_testutil import cuda, make

pytestmark = pytest.mark.gpu
TIMEOUT = 5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.load_library()


# thin chains, wide chains, chains of V = 64, each of 16 chunks and more
FORWARDS = [dict(seqs=(1, 1100), H=2, HV=2, K=128, V=128), dict(seqs=(2, 1050), H=8, HV=32, K=128, V=128),
            dict(seqs=(4, 1024), H=32, HV=32, K=64, V=64)]


@pytest.mark.parametrize("shape", FORWARDS, ids=lambda s: f"{s['seqs']}-{s['HV']}-{s['V']}")
def test_forward_runs_out(shape, monkeypatch):
    x = cuda(make(seed=62, **shape))
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]
    ws = torch.empty(kda.kda_gdr_fwd_workspace_size(kda.make_shape(x["q"], x["v"])), dtype=torch.uint8, device="cuda")
    fwd = lambda **kw: kda.kda_gdr_fwd(*args, x["scale"], initial_state=x["s0"], workspace=ws, **kw)
    ref = fwd()
    assert kda.kda_read_device_status(ws) == 0
    out, state = torch.full_like(x["v"], 77.0), torch.full_like(x["s0"], 77.0)
    with monkeypatch.context() as m:
        m.setenv("KDA_WAIT_LIMIT_NS", "1")
        fwd(out=out, final_state=state)
    assert kda.kda_read_device_status(ws) == TIMEOUT
    assert (out[:, -60:] == 77).all() and (state == 77).all()      # every chain gave up before its end
    assert all(torch.equal(s, t) for s, t in zip(ref, fwd())) and kda.kda_read_device_status(ws) == 0


@pytest.mark.parametrize("V", [128, 64])
def test_backward_runs_out(V, monkeypatch):
    x = cuda(make((2, 1030), 2, 4, 128, V, seed=63, grads=True))
    args = [x[n] for n in ("q", "k", "v", "g", "beta", "do")]
    ws = torch.empty(kda.kda_gdr_bwd_workspace_size(kda.make_shape(x["q"], x["v"])), dtype=torch.uint8, device="cuda")
    bwd = lambda: kda.kda_gdr_bwd(*args, x["scale"], initial_state=x["s0"], d_final_state=x["ds"], workspace=ws)
    ref = bwd()
    assert kda.kda_read_device_status(ws) == 0
    with monkeypatch.context() as m:
        m.setenv("KDA_WAIT_LIMIT_NS", "1")
        bwd()
    assert kda.kda_read_device_status(ws) == TIMEOUT
    assert all(torch.equal(s, t) for s, t in zip(ref, bwd())) and kda.kda_read_device_status(ws) == 0


def test_short_sequences_run_out_in_the_preparation(monkeypatch):
    """One chunk a sequence: no chain waits for a buffer; the preparation's own failure comes out
    through its record."""
    x = cuda(make((3, 40), 2, 2, 128, 128, seed=64))
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    with monkeypatch.context() as m:
        m.setenv("KDA_WAIT_LIMIT_NS", "1")
        kda.kda_gdr_fwd(*args, x["scale"], status=status)
    assert kda.kda_read_device_status(status) == TIMEOUT
    status.zero_()
    kda.kda_gdr_fwd(*args, x["scale"], status=status)
    assert kda.kda_read_device_status(status) == 0
