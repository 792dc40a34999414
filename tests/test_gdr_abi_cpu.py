"""Host-side checks of the gated delta rule's and layer norm's C entries (no GPU: every call
fails its checks, or has nothing to do, before anything is enqueued)."""
import ctypes

import pytest

from kimi_delta_attention_gb300 import _lib
from kimi_delta_attention_gb300.builder import build

P, F, Z = ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
STEP = 0x10000000
BF, F32 = _lib.KDA_BF16, _lib.KDA_F32


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load_library()


def at(i):
    return STEP * (i + 1)


def S(B=1, T=64, H=2, HV=4, K=128, V=128, ns=0, io=BF):
    return _lib.KdaShape(B, T, H, HV, K, V, ns, io)


def fwd(lib, s, scale=0.1, ws_bytes=None, **kw):
    a = dict(q=at(0), k=at(1), v=at(2), g=at(3), beta=at(4), s0=None, cu=None, out=at(5), sfin=None, ws=at(7))
    a.update(kw)
    n = lib.kda_gdr_fwd_workspace_size(s) if ws_bytes is None else ws_bytes
    return lib.kda_gdr_fwd(s, a["q"], a["k"], a["v"], a["g"], a["beta"], scale, a["s0"], a["cu"], a["out"], a["sfin"],
                           a["ws"], n or 256, None)


def bwd(lib, s, scale=0.1, ws_bytes=None, **kw):
    a = dict(q=at(0), k=at(1), v=at(2), g=at(3), beta=at(4), s0=None, cu=None, do=at(5), dfin=None, dq=at(6), dk=at(7),
             dv=at(8), dg=at(9), dbeta=at(10), ds0=at(11), ws=at(12))
    a.update(kw)
    n = lib.kda_gdr_bwd_workspace_size(s) if ws_bytes is None else ws_bytes
    return lib.kda_gdr_bwd(s, a["q"], a["k"], a["v"], a["g"], a["beta"], scale, a["s0"], a["cu"], a["do"], a["dfin"], a["dq"],
                           a["dk"], a["dv"], a["dg"], a["dbeta"], a["ds0"], a["ws"], n or 256, None)


def step(lib, s, scale=0.1, **kw):
    a = dict(q=at(0), k=at(1), v=at(2), g=at(3), beta=at(4), state=at(5), slots=None, n=0, out=at(6), status=None)
    a.update(kw)
    return lib.kda_gdr_step(s, a["q"], a["k"], a["v"], a["g"], a["beta"], scale, a["state"], a["slots"], a["n"], a["out"],
                            a["status"], None)


BAD_SHAPES = [(S(HV=3), 1), (S(H=0), 1), (S(T=-1), 1), (S(B=-1), 1), (S(io=7), 1), (S(K=96), 2), (S(V=32), 2), (S(ns=2), 1)]


@pytest.mark.parametrize("entry", [fwd, bwd, step])
def test_shapes(lib, entry):
    for s, code in BAD_SHAPES:
        assert entry(lib, s) == code
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert entry(lib, S(), scale=scale) == 1
    assert entry(lib, S(B=1 << 15, HV=1 << 14, H=1)) == 2       # more (sequence, head) pairs than are counted


def test_forward_arguments(lib):
    s = S()
    need = lib.kda_gdr_fwd_workspace_size(s)
    assert need > 256 and lib.kda_gdr_fwd_workspace_size(S(io=F32)) == 256
    assert lib.kda_gdr_fwd_workspace_size(S(T=0)) == 256 and lib.kda_gdr_fwd_workspace_size(None) == 0
    assert fwd(lib, s, ws_bytes=need - 1) == 6 and fwd(lib, s, ws=None) == 6
    for n in ("q", "k", "v", "g", "beta", "out"):
        assert fwd(lib, s, **{n: None}) == 1, n
    for n in ("q", "k", "v", "out", "ws"):
        assert fwd(lib, s, **{n: at(20) + 8}) == 3, n
    assert fwd(lib, s, g=at(3) + 2) == 3 and fwd(lib, s, sfin=at(9) + 4) == 3
    assert fwd(lib, s, out=at(2)) == 1 and fwd(lib, s, sfin=at(3)) == 1 and fwd(lib, s, ws=at(0)) == 1
    assert fwd(lib, s, s0=at(9), sfin=at(9) + 16) == 1          # overlapping, not the same
    assert fwd(lib, S(ns=1, B=2), cu=at(9)) == 1 and fwd(lib, S(), cu=at(9)) == 1
    assert fwd(lib, S(B=0)) == 0                                # no sequences: nothing to do


def test_backward_arguments(lib):
    s = S()
    need = lib.kda_gdr_bwd_workspace_size(s)
    # a record, S and dS', vn and z a chunk and value head; grouped heads' shares of dq and dk
    assert need == 256 + 128 + 4 * (33792 + 2 * 65536 + 2 * 32768) + 2 * 64 * 4 * 128 * 4
    assert lib.kda_gdr_bwd_workspace_size(S(io=F32)) == 0
    assert bwd(lib, S(io=F32)) == 2                             # bf16 only
    assert bwd(lib, s, ws_bytes=need - 1) == 6 and bwd(lib, s, ws=None) == 6
    for n in ("q", "k", "v", "g", "beta", "do", "dq", "dk", "dv", "dg", "dbeta"):
        assert bwd(lib, s, **{n: None}) == 1, n
    for n in ("do", "dfin", "dq", "dk", "dv", "ds0", "ws"):
        assert bwd(lib, s, **{n: at(20) + 8}) == 3, n
    assert bwd(lib, s, dq=at(0)) == 1 and bwd(lib, s, dk=at(6)) == 1 and bwd(lib, s, ds0=at(5)) == 1
    assert bwd(lib, s, ws=at(2)) == 1 and bwd(lib, s, dg=at(10)) == 1
    assert bwd(lib, S(B=0)) == 0


def test_step_arguments(lib):
    s = S(T=1)
    for n in ("q", "k", "v", "g", "beta", "state", "out"):
        assert step(lib, s, **{n: None}) == 1, n
    for n in ("q", "state", "out"):
        assert step(lib, s, **{n: at(20) + 8}) == 3, n
    assert step(lib, s, slots=at(9) + 2, n=4) == 3 and step(lib, s, status=at(9) + 1) == 3
    assert step(lib, s, slots=at(9), n=-1) == 1 and step(lib, s, n=3) == 1        # a pool's size without slots
    assert step(lib, s, out=at(5)) == 1 and step(lib, s, out=at(2)) == 1
    assert step(lib, s, slots=at(5) + 64, n=4) == 1                               # the slots inside the pool
    assert step(lib, S(B=0)) == 0 and step(lib, S(T=0)) == 0


def norm(lib, rows=4, D=64, io=BF, ld=None, eps=1e-5, **kw):
    a = dict(x=at(0), w=at(1), b=at(2), y=at(3), mean=at(4), rstd=at(5))
    a.update(kw)
    return lib.kda_layer_norm_fwd(rows, D, io, a["x"], D if ld is None else ld, a["w"], a["b"], eps, a["y"], a["mean"],
                                  a["rstd"], None)


def norm_bwd(lib, rows=4, D=64, io=BF, ldx=None, ldy=None, ws_bytes=None, **kw):
    a = dict(x=at(0), dy=at(1), w=at(2), mean=at(3), rstd=at(4), dx=at(5), dw=at(6), db=at(7), ws=at(8))
    a.update(kw)
    n = lib.kda_layer_norm_bwd_workspace_size(rows, D) if ws_bytes is None else ws_bytes
    return lib.kda_layer_norm_bwd(rows, D, io, a["x"], D if ldx is None else ldx, a["dy"], D if ldy is None else ldy, a["w"],
                                  a["mean"], a["rstd"], a["dx"], a["dw"], a["db"], a["ws"], n, None)


def test_layer_norm_arguments(lib):
    assert norm(lib, rows=-1) == 1 and norm(lib, D=0) == 1 and norm(lib, ld=63) == 1 and norm(lib, io=3) == 1
    assert norm(lib, rows=1 << 31) == 1
    for eps in (-1.0, float("nan"), float("inf")):
        assert norm(lib, eps=eps) == 1
    assert norm(lib, x=None) == 1 and norm(lib, y=None) == 1
    assert norm(lib, x=at(0) + 1) == 3 and norm(lib, io=F32, y=at(3) + 2) == 3 and norm(lib, w=at(1) + 2) == 3
    assert norm(lib, y=at(0)) == 1 and norm(lib, y=at(1)) == 1 and norm(lib, rstd=at(4)) == 1
    assert norm(lib, rows=0) == 0


def test_layer_norm_backward_arguments(lib):
    assert norm_bwd(lib, rows=-1, ws_bytes=1 << 20) == 1 and norm_bwd(lib, ldy=1) == 1 and norm_bwd(lib, ldx=1) == 1
    for n in ("x", "dy", "mean", "rstd"):
        assert norm_bwd(lib, **{n: None}) == 1, n
    assert norm_bwd(lib, dx=None, dw=None, db=None) == 1        # nothing asked for
    assert norm_bwd(lib, ws=None) == 6 and norm_bwd(lib, ws_bytes=16) == 6
    assert norm_bwd(lib, ws=at(8) + 8) == 3 and norm_bwd(lib, dw=at(6) + 2) == 3
    assert norm_bwd(lib, dx=at(0)) == 1 and norm_bwd(lib, dw=at(7)) == 1 and norm_bwd(lib, ws=at(1)) == 1
    assert lib.kda_layer_norm_bwd_workspace_size(-1, 4) == 0


def test_step_without_requests(lib):
    """No sequences, or no tokens: nothing to do, with a pool too (an empty slots array may have
    no address); a pool's size is checked all the same."""
    for s in (S(B=0, T=1), S(T=0)):
        assert step(lib, s, n=3) == 0 and step(lib, s, slots=at(9), n=3) == 0
        assert step(lib, s, q=None, k=None, v=None, out=None, n=3) == 0
        assert step(lib, s, n=-1) == 1
