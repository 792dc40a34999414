"""The gated linear recurrence on the GPU against its definition in 64 bits (bounds: layer_ops_testutil)."""
import pytest
import torch

import kimi_delta_attention_gb300 as kda
from layer_ops_testutil import glr_bwd_reference, glr_reference, make_glr, within

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kda.build()
    kda.load_library()


def check(d, lengths):
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(initial_state=d["s0"], cu_seqlens=d["cu"], status=word)
    y, state = kda.kda_glr_fwd(d["x"], d["g"], **kw)
    ry, ey, rs, es = glr_reference(d["x"], d["g"], d["s0"], lengths)
    within(y, ry, ey, "y")
    within(state, rs, es, "final state")
    dx, dg, ds0 = kda.kda_glr_bwd(d["g"], y, d["dy"], d_final_state=d["ds"], **kw)
    rx, ex, rg, eg, r0, e0 = glr_bwd_reference(d["g"], y, d["dy"], d["s0"], d["ds"], lengths)
    within(dx, rx, ex, "dx")
    within(dg, rg, eg, "dg")
    within(ds0, r0, e0, "d_initial_state")
    assert y.dtype == dx.dtype == d["x"].dtype and dg.dtype == d["g"].dtype
    assert word.item() == 0
    return y, state, dx, dg, ds0


TYPES = [(BF, F32), (BF, BF), (F32, F32), (F32, BF)]
SHAPES = [(1, 1, 1), (1, 2, 5), (3, 7, 64), (2, 63, 130), (1, 64, 128), (2, 65, 127), (1, 129, 4), (5, 100, 33), (1, 1000, 260),
          (2, 2500, 96), (64, 3, 512), (300, 1, 12), (1, 4097, 132)]


@pytest.mark.parametrize("io,gate", TYPES)
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_batched(B, T, D, io, gate):
    check(make_glr([T] * B, D, io, gate, state=B % 2 == 1, packed=False, seed=B * 1000 + T + D), [T] * B)


PACKED = [[5], [1, 1, 1], [64, 64], [63, 2, 1, 190], [0, 5, 0, 0, 70, 0], [300, 1, 511, 188], [1] * 200, [1000, 3, 2000, 64],
          [17, 0, 0, 0, 0, 47, 128, 0], [7] * 300 + [0] * 40 + [900]]


@pytest.mark.parametrize("io,gate", TYPES)
@pytest.mark.parametrize("D", [1, 67, 256])
@pytest.mark.parametrize("n", range(len(PACKED)))
def test_packed(n, D, io, gate):
    check(make_glr(PACKED[n], D, io, gate, state=(n + D) % 3 != 0, seed=100 * n + D), PACKED[n])


@pytest.mark.parametrize("B,T,D", [(1, 70000, 8), (1, 30000, 200), (2, 16384, 1024), (7, 1111, 4100)])
def test_long_and_wide(B, T, D):
    check(make_glr([T] * B, D, F32, F32, packed=False, seed=T), [T] * B)


@pytest.mark.parametrize("rates", [(1e-6, 1e-5), (5.0, 60.0)], ids=["hardly", "at once"])
def test_decays(rates):
    """States that hardly fade over the sequence, and ones that are gone with the next token."""
    check(make_glr([3000], 96, F32, F32, packed=False, seed=9, rates=rates), [3000])


def test_dropped_states():
    """g = -inf drops the state, in the gradients too; g = 0 keeps it."""
    d = make_glr([200, 150], 40, F32, F32, seed=10)
    d["g"][0, 5::17] = float("-inf")
    d["g"][0, :, 3] = 0
    d["g"][0, :, 4] = float("-inf")
    y, _, dx, dg, ds0 = check(d, [200, 150])
    assert torch.equal(y[..., 4], d["x"][..., 4]) and (dg[..., 4] == 0).all() and (ds0[:, 4] == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_bad_values_stay_in_their_sequence_and_channel(bad):
    lengths, D = [100, 60, 130, 1, 70], 36
    d = make_glr(lengths, D, F32, F32, seed=11)
    y, s = kda.kda_glr_fwd(d["x"], d["g"], initial_state=d["s0"], cu_seqlens=d["cu"])
    dx, dg, ds0 = kda.kda_glr_bwd(d["g"], y, d["dy"], initial_state=d["s0"], cu_seqlens=d["cu"], d_final_state=d["ds"])
    x, dy = d["x"].clone(), d["dy"].clone()
    x[0, 150, 7] = bad                                  # in the second sequence
    dy[0, 200, 7] = bad                                 # in the third
    y2, s2 = kda.kda_glr_fwd(x, d["g"], initial_state=d["s0"], cu_seqlens=d["cu"])
    dx2, dg2, ds2 = kda.kda_glr_bwd(d["g"], y, dy, initial_state=d["s0"], cu_seqlens=d["cu"], d_final_state=d["ds"])
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[0, 150:160, 7] = True
    assert torch.equal(y2[~hit], y[~hit]) and not torch.isfinite(y2[hit]).any()
    assert torch.equal(torch.cat([s2[:1], s2[2:]]), torch.cat([s[:1], s[2:]])) and not torch.isfinite(s2[1, 7])
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[0, 160:201, 7] = True
    assert torch.equal(dx2[~hit], dx[~hit]) and not torch.isfinite(dx2[hit]).any()
    assert torch.equal(dg2[~hit], dg[~hit]) and not torch.isfinite(ds2[2, 7])
    others = [0, 1, 3, 4]
    assert torch.equal(ds2[others], ds0[others])


def test_state_in_place_and_in_pieces():
    """A sequence taken in two calls, the state in one array, is the sequence in one (to rounding)."""
    d = make_glr([500], 100, F32, F32, packed=False, seed=12)
    y, s = kda.kda_glr_fwd(d["x"], d["g"], initial_state=d["s0"])
    state, parts = d["s0"].clone(), []
    for a, b in ((0, 123), (123, 500)):
        parts.append(kda.kda_glr_fwd(d["x"][:, a:b].contiguous(), d["g"][:, a:b].contiguous(), initial_state=state,
                                     final_state=state)[0])
    ry, ey, rs, es = glr_reference(d["x"], d["g"], d["s0"], [500])
    within(torch.cat(parts, 1), ry, ey, "y")
    within(state, rs, es, "state")


@pytest.mark.parametrize("lengths", [[2000, 3, 0, 900], [64] * 40, [5, 1000] * 9])
def test_final_states_over_initial_ones(lengths):
    """final_state may be initial_state, and d_initial_state would be d_final_state's: a sequence's end is
    written after its start was read, tiles apart or in one tile."""
    d = make_glr(lengths, 384, BF, F32, seed=20)
    y, s = kda.kda_glr_fwd(d["x"], d["g"], initial_state=d["s0"], cu_seqlens=d["cu"])
    for _ in range(10):
        state = d["s0"].clone()
        y2, s2 = kda.kda_glr_fwd(d["x"], d["g"], initial_state=state, cu_seqlens=d["cu"], final_state=state)
        assert s2 is state and torch.equal(y, y2) and torch.equal(s, s2)


@pytest.mark.parametrize("lengths", [[2000, 3, 0, 900], [64] * 40, [5, 1000] * 9])
def test_initial_gradients_over_final_ones(lengths):
    """At the C entry d_initial_state may be the array of d_final_state."""
    D = 384
    d = make_glr(lengths, D, BF, F32, seed=21)
    lib = kda.load_library()
    y, _ = kda.kda_glr_fwd(d["x"], d["g"], initial_state=d["s0"], cu_seqlens=d["cu"])
    ref = kda.kda_glr_bwd(d["g"], y, d["dy"], initial_state=d["s0"], cu_seqlens=d["cu"], d_final_state=d["ds"])
    shape = kda.KdaGlrShape(1, sum(lengths), D, len(lengths), 1, 0)
    ws = torch.empty(kda.kda_glr_bwd_workspace_size(shape), dtype=torch.uint8, device="cuda")
    for _ in range(5):
        state, dx, dg = d["ds"].clone(), torch.empty_like(y), torch.empty_like(d["g"])
        code = lib.kda_glr_bwd(shape, *(t.data_ptr() for t in (d["g"], y, d["dy"], d["s0"], d["cu"], state, dx, dg, state, ws)), ws.numel(),
                               torch.cuda.current_stream().cuda_stream)
        assert code == 0 and kda.kda_read_device_status(ws) == 0
        assert all(torch.equal(a, b) for a, b in zip((dx, dg, state), ref))


def test_gradients_against_differences():
    d = make_glr([9, 6], 3, F32, F32, seed=13)
    y, _ = kda.kda_glr_fwd(d["x"], d["g"], initial_state=d["s0"], cu_seqlens=d["cu"])
    grads = kda.kda_glr_bwd(d["g"], y, d["dy"], initial_state=d["s0"], cu_seqlens=d["cu"], d_final_state=d["ds"])

    def loss(x, g, s0):
        r, _, s, _ = glr_reference(x, g, s0, [9, 6])
        return ((r * d["dy"].double()).sum() + (s * d["ds"].double()).sum()).item()

    at = [d["x"].double(), d["g"].double(), d["s0"].double()]
    for k, grad in enumerate(grads):
        for i in range(0, grad.numel(), 5):
            e = torch.zeros_like(at[k])
            e.view(-1)[i] = 1e-5
            up, down = ([t + s * e if j == k else t for j, t in enumerate(at)] for s in (1, -1))
            num = (loss(*up) - loss(*down)) / 2e-5
            assert abs(num - grad.view(-1)[i].item()) <= 1e-4 * max(1, abs(num))


@pytest.mark.parametrize("T,D", [(300, 130), (5000, 64), (2000, 516)])
def test_repeats_bit_for_bit(T, D):
    d = make_glr([T] * 3, D, BF, F32, packed=False, seed=14)
    runs = []
    for _ in range(5):
        y, s = kda.kda_glr_fwd(d["x"], d["g"], initial_state=d["s0"])
        runs.append((y, s, *kda.kda_glr_bwd(d["g"], y, d["dy"], initial_state=d["s0"], d_final_state=d["ds"])))
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(runs[0], r))


@pytest.mark.parametrize("io", [BF, F32])
def test_alignment(io):
    """Views that start anywhere give what aligned copies give."""
    lengths, D = [70, 200], 128
    d = make_glr(lengths, D, io, F32, seed=15)
    shifted = {}
    for n, t in d.items():
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        shifted[n] = buf[1:].view(t.shape)
        shifted[n].copy_(t)
    check(shifted, lengths)
    out = torch.empty(d["x"].numel() + 3, dtype=io, device="cuda")[3:].view(d["x"].shape)
    y, _ = kda.kda_glr_fwd(d["x"], d["g"], initial_state=d["s0"], cu_seqlens=d["cu"], out=out)
    ry, ey, _, _ = glr_reference(d["x"], d["g"], d["s0"], lengths)
    within(y, ry, ey, "y")
    assert y is out


def test_no_tokens_and_no_sequences():
    s0 = torch.randn(3, 8, device="cuda")
    e = torch.empty(3, 0, 8, device="cuda")
    y, s = kda.kda_glr_fwd(e, e, initial_state=s0)
    assert y.shape == e.shape and torch.equal(s, s0)
    assert (kda.kda_glr_fwd(e, e)[1] == 0).all()
    assert torch.equal(kda.kda_glr_bwd(e, e, e, d_final_state=s0)[2], s0)
    z = torch.empty(0, 5, 8, device="cuda")
    assert kda.kda_glr_fwd(z, z)[0].shape == z.shape
    p = torch.empty(1, 0, 8, device="cuda")
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert torch.equal(kda.kda_glr_fwd(p, p, initial_state=s0, cu_seqlens=cu, status=status)[1], s0) and status.item() == 0


@pytest.mark.parametrize("cu", [[0, 50, 40, 100], [1, 50, 60, 100], [0, 50, 60, 90], [0, 50, 60, 300], [0, -5, 60, 100],
                                [0, 2000000000, 60, 100], [-2000000000, 50, 60, 100], [0, 0, 0, 0]])
def test_bad_cu_seqlens_are_reported(cu):
    d = make_glr([50, 10, 40], 70, F32, F32, seed=16)
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    for back in (False, True):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        if back:
            kda.kda_glr_bwd(d["g"], d["x"], d["dy"], initial_state=d["s0"], cu_seqlens=cu, d_final_state=d["ds"], status=status)
        else:
            kda.kda_glr_fwd(d["x"], d["g"], initial_state=d["s0"], cu_seqlens=cu, status=status)
        assert status.item() == 2 and kda.kda_read_device_status(status) == 7


def test_tokens_behind_the_last_sequence_stay():
    d = make_glr([50, 10, 40], 70, F32, F32, seed=17)
    cu = torch.tensor([0, 50, 60, 90], dtype=torch.int32, device="cuda")
    out = torch.full_like(d["x"], 7.0)
    kda.kda_glr_fwd(d["x"], d["g"], cu_seqlens=cu, out=out)
    assert (out[0, 90:] == 7).all()


# ------------------------------------------------------------------- step --
@pytest.mark.parametrize("io,gate", TYPES)
@pytest.mark.parametrize("B,T,D,pool", [(1, 1, 1, 0), (3, 1, 130, 0), (5, 3, 64, 11), (128, 1, 1024, 300), (2, 5, 8192, 0)])
def test_step(B, T, D, pool, io, gate):
    d = make_glr([T] * B, D, io, gate, packed=False, seed=B + T + D)
    state = torch.randn(pool or B, D, device="cuda")
    before = state.clone()
    slots = None
    live = list(range(B))
    at = live
    if pool:
        slots = torch.randperm(pool, device="cuda")[:B].to(torch.int32)
        slots[B // 2] = -1
        live = [b for b in range(B) if b != B // 2]
        at = slots[live].long().tolist()
    y = kda.kda_glr_step(d["x"], d["g"], state, slots=slots)
    ry, ey, rs, es = glr_reference(d["x"][live], d["g"][live], before[at], [T] * len(live))
    within(y[live], ry, ey, "y")
    within(state[at], rs, es, "state")
    rest = torch.ones(len(before), dtype=torch.bool)
    rest[at] = False
    assert torch.equal(state[rest], before[rest])
    if pool:
        assert (y[B // 2] == 0).all()


def test_step_is_the_forward_token_by_token():
    d = make_glr([20] * 3, 100, BF, F32, packed=False, seed=18)
    y, s = kda.kda_glr_fwd(d["x"], d["g"], initial_state=d["s0"])
    state, served = d["s0"].clone(), []
    for t in range(20):
        served.append(kda.kda_glr_step(d["x"][:, t:t + 1].contiguous(), d["g"][:, t:t + 1].contiguous(), state))
    _, _, rs, es = glr_reference(d["x"], d["g"], d["s0"], [20] * 3)
    within(state, rs, es, "state")
    ry, ey, _, _ = glr_reference(d["x"], d["g"], d["s0"], [20] * 3)
    within(torch.cat(served, 1), ry, ey, "y")


def test_step_slot_out_of_range():
    d = make_glr([1] * 3, 20, F32, F32, packed=False, seed=19)
    state = torch.randn(4, 20, device="cuda")
    before = state.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = kda.kda_glr_step(d["x"], d["g"], state, slots=torch.tensor([4, 1, -7], dtype=torch.int32, device="cuda"), status=status)
    assert status.item() == 2 and (y[0] == 0).all() and (y[2] == 0).all()
    assert torch.equal(state[[0, 2, 3]], before[[0, 2, 3]]) and not torch.equal(state[1], before[1])


@pytest.mark.parametrize("g_range,T", [((-0.01, -0.001), 400), ((-0.3, -0.01), 60)])
def test_decays_multiply_without_a_bias(g_range, T):
    """A state that only decays is e^(g T): each e^g has an error of its own channel's, 0.55 of 2^-24 as a deviation,
    which T tokens add up; over 4096 channels such errors average to 0.55 / 64 = 0.009 of T 2^-24 (6 deviations:
    0.05), so a mean above 0.1 is a bias of the exponential.  The same for the gradients' way back."""
    D = 4096
    lo, hi = g_range
    g = (lo + (hi - lo) * torch.rand(D, device="cuda")).expand(1, T, D).contiguous()
    zero, one = torch.zeros(1, T, D, device="cuda"), torch.ones(1, D, device="cuda")
    want = torch.exp(g[0, 0].double() * T)
    y, state = kda.kda_glr_fwd(zero, g, initial_state=one)
    ds0 = kda.kda_glr_bwd(g, y, zero, initial_state=one, d_final_state=one)[2]
    for got in (state, ds0):
        assert abs((got[0].double() / want - 1).mean().item()) <= 0.1 * T * 2.0 ** -24
