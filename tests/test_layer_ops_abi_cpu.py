"""Host-side checks of the C entries of the gated linear recurrence, group norm and the AdamW step (no
GPU: every call fails its checks, or has nothing to do, before anything is enqueued)."""
import ctypes
import struct

import pytest
import torch

import kimi_delta_attention_gb300 as kda
from kimi_delta_attention_gb300 import KdaError, _lib
from kimi_delta_attention_gb300.builder import build

STEP = 0x10000000
BF, F32 = _lib.KDA_BF16, _lib.KDA_F32


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load_library()


def at(i):
    return STEP * (i + 1)


# ------------------------------------------------------- linear recurrence --
def S(B=2, T=64, D=128, ns=0, io=BF, gate=F32):
    return _lib.KdaGlrShape(B, T, D, ns, io, gate)


def fwd(lib, s, ws_bytes=None, **kw):
    a = dict(x=at(0), g=at(1), s0=None, cu=None, y=at(2), fin=None, ws=at(4))
    a.update(kw)
    n = lib.kda_glr_fwd_workspace_size(s) if ws_bytes is None else ws_bytes
    return lib.kda_glr_fwd(s, a["x"], a["g"], a["s0"], a["cu"], a["y"], a["fin"], a["ws"], n or 256, None)


def bwd(lib, s, ws_bytes=None, **kw):
    a = dict(g=at(0), y=at(1), do=at(2), s0=None, cu=None, dfin=None, dx=at(3), dg=at(4), ds0=at(5), ws=at(6))
    a.update(kw)
    n = lib.kda_glr_bwd_workspace_size(s) if ws_bytes is None else ws_bytes
    return lib.kda_glr_bwd(s, a["g"], a["y"], a["do"], a["s0"], a["cu"], a["dfin"], a["dx"], a["dg"], a["ds0"], a["ws"], n or 256, None)


def step(lib, s, **kw):
    a = dict(x=at(0), g=at(1), state=at(2), slots=None, n=0, y=at(3), status=None)
    a.update(kw)
    return lib.kda_glr_step(s, a["x"], a["g"], a["state"], a["slots"], a["n"], a["y"], a["status"], None)


@pytest.mark.parametrize("entry", [fwd, bwd, step])
def test_recurrence_shapes(lib, entry):
    for s, code in ((S(D=0), 1), (S(T=-1), 1), (S(B=-1), 1), (S(io=7), 1), (S(gate=-1), 1), (S(ns=2), 1), (S(ns=-1), 1),
                    (S(B=1 << 16, T=1 << 16), 2)):
        assert entry(lib, s) == code
    assert lib.kda_glr_fwd_workspace_size(S(D=0)) == 0 and lib.kda_glr_bwd_workspace_size(None) == 0


def test_recurrence_forward_arguments(lib):
    s = S()
    assert fwd(lib, s, ws_bytes=255) == 6 and fwd(lib, s, ws=None) == 6
    for n in ("x", "g", "y"):
        assert fwd(lib, s, **{n: None}) == 1, n
    assert fwd(lib, s, x=at(0) + 1) == 3 and fwd(lib, s, g=at(1) + 2) == 3 and fwd(lib, s, fin=at(9) + 2) == 3
    assert fwd(lib, s, ws=at(4) + 8) == 3
    assert fwd(lib, s, y=at(0)) == 1 and fwd(lib, s, y=at(1) + 64) == 1 and fwd(lib, s, fin=at(2)) == 1
    assert fwd(lib, s, ws=at(0)) == 1 and fwd(lib, s, ws=at(2)) == 1
    assert fwd(lib, s, s0=at(9), fin=at(9) + 4) == 1                  # overlapping, not the same
    assert fwd(lib, S(ns=1), cu=at(9)) == 1 and fwd(lib, S(B=1), cu=at(9)) == 1
    assert fwd(lib, S(B=0)) == 0


def test_recurrence_backward_arguments(lib):
    s = S()
    assert bwd(lib, s, ws_bytes=16) == 6 and bwd(lib, s, ws=None) == 6
    for n in ("g", "y", "do", "dx", "dg"):
        assert bwd(lib, s, **{n: None}) == 1, n
    assert bwd(lib, s, y=at(1) + 1) == 3 and bwd(lib, s, dg=at(4) + 2) == 3 and bwd(lib, s, dfin=at(9) + 1) == 3
    assert bwd(lib, s, dx=at(2)) == 1 and bwd(lib, s, dg=at(3)) == 1 and bwd(lib, s, ds0=at(1)) == 1
    assert bwd(lib, s, s0=at(5)) == 1                                 # d_initial_state over initial_state
    assert bwd(lib, s, dfin=at(5) + 4) == 1
    assert bwd(lib, S(B=0)) == 0


def test_recurrence_step_arguments(lib):
    s = S(T=1)
    for n in ("x", "g", "state", "y"):
        assert step(lib, s, **{n: None}) == 1, n
    assert step(lib, s, slots=at(9) + 2, n=4) == 3 and step(lib, s, status=at(9) + 1) == 3 and step(lib, s, state=at(2) + 2) == 3
    assert step(lib, s, slots=at(9), n=-1) == 1 and step(lib, s, n=3) == 1
    assert step(lib, s, y=at(2)) == 1 and step(lib, s, y=at(0)) == 1 and step(lib, s, slots=at(2) + 64, n=4) == 1
    for e in (S(B=0, T=1), S(T=0)):
        assert step(lib, e) == 0 and step(lib, e, x=None, g=None, y=None, n=3) == 0


# -------------------------------------------------------------- group norm --
def norm(lib, N=4, L=3, C=64, groups=4, io=BF, act=1, eps=1e-5, ws_bytes=None, **kw):
    a = dict(x=at(0), w=at(1), b=at(2), y=at(3), mean=at(4), rstd=at(5), ws=at(6))
    a.update(kw)
    n = lib.kda_group_norm_fwd_workspace_size(N, L, C, groups) if ws_bytes is None else ws_bytes
    return lib.kda_group_norm_fwd(N, L, C, groups, io, act, a["x"], a["w"], a["b"], eps, a["y"], a["mean"], a["rstd"], a["ws"], n, None)


def norm_bwd(lib, N=4, L=3, C=64, groups=4, io=BF, act=1, ws_bytes=None, **kw):
    a = dict(x=at(0), dy=at(1), w=at(2), b=at(3), mean=at(4), rstd=at(5), dx=at(6), dw=at(7), db=at(8), ws=at(9))
    a.update(kw)
    n = lib.kda_group_norm_bwd_workspace_size(N, L, C, groups) if ws_bytes is None else ws_bytes
    return lib.kda_group_norm_bwd(N, L, C, groups, io, act, a["x"], a["dy"], a["w"], a["b"], a["mean"], a["rstd"], a["dx"], a["dw"],
                                  a["db"], a["ws"], n, None)


@pytest.mark.parametrize("entry", [norm, norm_bwd])
def test_group_norm_shapes(lib, entry):
    for kw, code in ((dict(N=-1), 1), (dict(L=0), 1), (dict(C=0), 1), (dict(groups=0), 1), (dict(groups=5), 1), (dict(io=4), 1),
                     (dict(act=2), 1), (dict(act=-1), 1), (dict(N=1 << 31), 2), (dict(N=1 << 20, L=1 << 20), 2)):
        assert entry(lib, ws_bytes=1 << 20, **kw) == code, kw
    assert lib.kda_group_norm_fwd_workspace_size(1, 1, 10, 3) == 0 and lib.kda_group_norm_bwd_workspace_size(1, 0, 10, 2) == 0


def test_group_norm_arguments(lib):
    for eps in (-1.0, float("nan"), float("inf")):
        assert norm(lib, eps=eps) == 1
    assert norm(lib, x=None) == 1 and norm(lib, y=None) == 1 and norm(lib, ws=None) == 6 and norm(lib, ws_bytes=8) == 6
    assert norm(lib, x=at(0) + 1) == 3 and norm(lib, io=F32, y=at(3) + 2) == 3 and norm(lib, w=at(1) + 2) == 3 and norm(lib, ws=at(6) + 4) == 3
    assert norm(lib, y=at(0)) == 1 and norm(lib, y=at(1)) == 1 and norm(lib, rstd=at(4)) == 1 and norm(lib, ws=at(0)) == 1
    assert norm(lib, N=0) == 0


def test_group_norm_backward_arguments(lib):
    for n in ("x", "dy", "mean", "rstd"):
        assert norm_bwd(lib, **{n: None}) == 1, n
    assert norm_bwd(lib, dx=None, dw=None, db=None) == 1
    assert norm_bwd(lib, ws=None) == 6 and norm_bwd(lib, ws_bytes=16) == 6
    assert norm_bwd(lib, ws=at(9) + 8) == 3 and norm_bwd(lib, dw=at(7) + 2) == 3
    assert norm_bwd(lib, dx=at(0)) == 1 and norm_bwd(lib, dw=at(8)) == 1 and norm_bwd(lib, ws=at(1)) == 1 and norm_bwd(lib, db=at(3)) == 1


def test_more_channels_than_32_bits_count_on_the_device(lib):
    for D in ((1 << 30) + 1, (1 << 31) - 8):
        for entry in (fwd, bwd, step):
            assert entry(lib, S(B=1, T=1, D=D)) == 2
        for entry in (norm, norm_bwd):
            assert entry(lib, ws_bytes=1 << 20, N=1, L=1, C=D, groups=1) == 2
            assert entry(lib, ws_bytes=1 << 20, N=1, L=3000, C=D, groups=D) == 2


def test_group_norm_of_no_samples(lib):
    """Groups of every way of the kernels: nothing to do, and no layout to work out."""
    for kw in (dict(L=3, C=64), dict(L=4096, C=512), dict(L=1, C=1024), dict(L=1, C=1 << 16), dict(L=77, C=1004)):
        size = dict(N=0, groups=4, **kw)
        assert lib.kda_group_norm_fwd_workspace_size(*(size[n] for n in ("N", "L", "C", "groups"))) == 256
        assert lib.kda_group_norm_bwd_workspace_size(*(size[n] for n in ("N", "L", "C", "groups"))) == 256
        assert norm(lib, **size) == 0 and norm(lib, x=None, y=None, **size) == 0


# ------------------------------------------------------------------- AdamW --
def tensor(i=0, n=1000, bits=8, param_type=BF, grad_type=BF, **kw):
    base = 10 * i
    a = dict(param=at(base), grad=at(base + 1), m=at(base + 2), v=at(base + 3), ms=at(base + 4) if bits == 8 else 0,
             vs=at(base + 5) if bits == 8 else 0, master=0)
    a.update(kw)
    return struct.pack("=10q", a["param"], a["grad"], a["m"], a["v"], a["ms"], a["vs"], a["master"], n, param_type, grad_type)


def adamw(lib, tensors, bits=8, count=None, **kw):
    c = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1, seed=0, state_bits=bits)
    c.update(kw)
    data = b"".join(tensors)
    return lib.kda_adamw_step(data, len(tensors) if count is None else count, _lib.KdaAdamwConfig(**c), None)


def test_adamw_settings(lib):
    t = [tensor()]
    for kw in (dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0), dict(beta2=-0.1), dict(beta2=float("nan")), dict(eps=-1e-9),
               dict(eps=float("inf")), dict(weight_decay=-0.1), dict(step=0), dict(step=1 << 31), dict(state_bits=16)):
        assert adamw(lib, t, **kw) == 1, kw
    for word in ("step_device", "lr_device", "grad_scale", "skip"):
        assert adamw(lib, t, **{word: at(50) + 2}) == 3
        assert adamw(lib, t, **{word: at(0) + 4}) == 1                # a word inside what the step writes
    assert adamw(lib, t, count=-1) == 1 and lib.kda_adamw_step(None, 1, _lib.KdaAdamwConfig(state_bits=32, step=1), None) == 1
    assert lib.kda_adamw_step(b"", 0, None, None) == 1
    assert adamw(lib, []) == 0
    assert adamw(lib, [tensor(n=0, m=0, v=0)]) == 0                   # nothing in it: no address needed


def test_adamw_settings_that_fp32_does_not_hold(lib):
    for kw in (dict(lr=1e39), dict(weight_decay=1e39), dict(eps=1e39), dict(eps=1e-38), dict(eps=1e-50), dict(eps=5e-324)):
        assert adamw(lib, [tensor()], **kw) == 1, kw
    t = tensor(n=0, m=0, v=0)
    assert adamw(lib, [t], eps=0.0) == 0 and adamw(lib, [t], eps=2.0 ** -126) == 0


def test_adamw_tensors(lib):
    for n in ("param", "grad", "m", "v", "ms", "vs"):
        assert adamw(lib, [tensor(**{n: 0})]) == 1, n
    assert adamw(lib, [tensor(bits=8)], bits=32) == 1                 # scales of 32-bit states
    assert adamw(lib, [tensor(n=-1)]) == 1 and adamw(lib, [tensor(n=1 << 41)]) == 1
    assert adamw(lib, [tensor(param=at(0) + 1)]) == 3 and adamw(lib, [tensor(grad=at(1) + 1)]) == 3
    assert adamw(lib, [tensor(ms=at(4) + 2)]) == 3 and adamw(lib, [tensor(bits=32, m=at(2) + 2)], bits=32) == 3
    assert adamw(lib, [tensor(master=at(6) + 2)]) == 3


def test_adamw_overlaps(lib):
    assert adamw(lib, [tensor(), tensor()]) == 1                      # the same tensor twice
    assert adamw(lib, [tensor(grad=at(0))]) == 1 and adamw(lib, [tensor(m=at(3))]) == 1
    assert adamw(lib, [tensor(0), tensor(1, grad=at(0) + 500)]) == 1
    assert adamw(lib, [tensor(0), tensor(1, param=at(2))]) == 1
    assert adamw(lib, [tensor(0), tensor(1, grad=at(11) - 600, m=at(11) + 1300)]) == 1
    assert adamw(lib, [tensor(0, master=at(6)), tensor(1, vs=at(6) + 3996)]) == 1


# ----------------------------------------------------------------- binding --
def test_binding_refuses_host_tensors(lib):
    x, s = torch.zeros(1, 4, 8), torch.zeros(1, 8)
    calls = [lambda: kda.kda_glr_fwd(x, x), lambda: kda.kda_glr_bwd(x, x, x), lambda: kda.kda_glr_step(x, x, s),
             lambda: kda.kda_group_norm_fwd(x, 2), lambda: kda.kda_group_norm_bwd(x, x, 2, None, None, s, s),
             lambda: kda.kda_adamw_step([s], [s], [s], [s], 1), lambda: kda.kda_group_norm_fwd(x, 2, activation="tanh")]
    for call in calls:
        with pytest.raises(KdaError) as e:
            call()
        assert e.value.code == 1
    assert kda.kda_adamw_step([], [], [], [], 1) is None


def test_struct_layouts():
    assert ctypes.sizeof(_lib.KdaGlrShape) == 24 and ctypes.sizeof(_lib.KdaAdamwConfig) == 96
