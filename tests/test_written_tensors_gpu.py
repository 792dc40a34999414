"""Tensors of the caller that a call writes change their version: a graph that has saved one
refuses its backward pass instead of using the new values."""
import pytest
import torch

import kimi_delta_attention_gb300 as kda
from kimi_delta_attention_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def x():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.load_library()
    return W.make_inputs(2, 65, 2, 4, 128, 128, "bf16", seed=72, init_state=True).to("cuda")


def saved(t):
    """A result whose backward pass needs t's present values."""
    w = torch.ones((), device="cuda", requires_grad=True)
    return (t.float() * w if t.dtype != torch.float32 else t * w).sum()


def check(t, call):
    y = saved(t)
    y.backward(retain_graph=True)
    before = t._version
    call()
    assert t._version > before
    if t.dtype == torch.float32:         # (saved itself, not a copy)
        with pytest.raises(RuntimeError, match="inplace operation"):
            y.backward()


def test_scalar_gate(x):
    g = x.g[..., 0].contiguous()
    rule = (x.q, x.k, x.v, g, x.beta)
    first = [t[:, :1].contiguous() for t in rule]
    state, out = x.initial_state.clone(), torch.empty_like(x.v)
    check(state, lambda: kda.kda_gdr_fwd(*rule, initial_state=state, final_state=state))
    check(out, lambda: kda.kda_gdr_fwd(*rule, out=out))
    check(state, lambda: kda.kda_gdr_step(*first, state))
    pool, slots = torch.zeros(3, *state.shape[1:], device="cuda"), torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    o1 = torch.empty_like(first[2])
    check(pool, lambda: kda.kda_gdr_step(*first, pool, slots=slots))
    check(o1, lambda: kda.kda_gdr_step(*first, pool, slots=slots, out=o1))
    rows = torch.randn(4, 64, device="cuda")
    y = torch.empty_like(rows)
    check(y, lambda: kda.kda_layer_norm_fwd(rows, out=y))


def test_gate_per_dimension(x):
    args = (x.q, x.k, x.v, x.g, x.beta)
    first = [t[:, :1].contiguous() for t in args]
    state, out = x.initial_state.clone(), torch.empty_like(x.v)
    for fn in (kda.kda_chunk_fwd, kda.kda_recurrent_fwd):
        check(state, lambda: fn(*args, initial_state=state, final_state=state))
        check(out, lambda: fn(*args, out=out))
    check(state, lambda: kda.kda_decode(*first, state))
    check(state, lambda: kda.kda_chunk_fwd_static_scratch(*args, initial_state=x.initial_state, final_state=state))
    check(state, lambda: kda.kda_chunk_states(*args, initial_state=x.initial_state, final_state=state))
    h, _ = kda.kda_chunk_states(*args)
    check(h, lambda: kda.kda_chunk_states(*args, h=h))
    check(out, lambda: kda.kda_chunk_output(*args, h, out=out))


def test_under_inference_mode(x):
    with torch.inference_mode():
        first = [t[:, :1].contiguous() for t in (x.q, x.k, x.v, x.g[..., 0].contiguous(), x.beta)]
        a, b = x.initial_state.clone(), x.initial_state.clone()
        assert torch.equal(kda.kda_gdr_step(*first, a), kda.kda_gdr_step(*first, b)) and torch.equal(a, b)
