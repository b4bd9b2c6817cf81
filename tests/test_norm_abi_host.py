"""Host-side refusals of the norm entry points: fake addresses, nothing is enqueued."""
import ctypes
import os

import pytest

import state_space_model_04_b200 as ssd
from state_space_model_04_b200 import ssd as binding

OK, INVALID, UNSUP, CUDA, TIMEOUT, WS, INTERNAL = range(7)

pytestmark = pytest.mark.skipif(not os.path.exists(binding.LIB_PATH), reason="library not built")


def p(i):
    return ctypes.c_void_p(0x10000000 + 0x4000000 * i)


def fwd(rows=4, D=64, io=1, res=0, x=p(0), lx=64, r=p(1), lr=64, scale=1.0, w=p(2), eps=1e-5, out=p(3), lo=64,
        ro=p(4), lro=64):
    return ssd.lib().ssd_residual_norm(rows, D, io, res, x, lx, r, lr, scale, w, eps, out, lo, ro, lro, None)


def bwd(rows=4, D=64, io=1, res=0, dout=p(0), r=p(1), w=p(2), dro=p(3), dx=p(4), dres=p(5), dw=p(6), ws=p(7),
        ws_bytes=1 << 25, ld=64, scale=1.0, eps=1e-5):
    return ssd.lib().ssd_residual_norm_backward(rows, D, io, res, dout, ld, r, ld, w, dro, ld, scale, eps, dx, ld, dres,
                                                ld, dw, ws, ws_bytes, None)


def gate(rows=4, D=64, groups=1, io=1, first=0, y=p(0), ly=64, z=p(1), lz=64, w=p(2), eps=1e-5, out=p(3), lo=64):
    return ssd.lib().ssd_gated_norm(rows, D, groups, io, first, y, ly, z, lz, w, eps, out, lo, None)


def gate_bwd(rows=4, D=64, groups=1, io=1, first=0, dout=p(0), y=p(1), z=p(2), w=p(3), dy=p(4), dz=p(5), dw=p(6),
             ws=p(7), ws_bytes=1 << 25, ld=64):
    return ssd.lib().ssd_gated_norm_backward(rows, D, groups, io, first, dout, ld, y, ld, z, ld, w, 1e-5, dy, ld, dz, ld,
                                             dw, ws, ws_bytes, None)


@pytest.mark.parametrize("call,kw,status", [
    (fwd, dict(rows=-1), INVALID), (fwd, dict(D=0), INVALID), (fwd, dict(io=5), INVALID), (fwd, dict(res=9), INVALID),
    (fwd, dict(io=0, res=1), UNSUP), (fwd, dict(D=16385, lx=20000, lr=20000, lo=20000, lro=20000), UNSUP),
    (fwd, dict(eps=-1e-5), INVALID), (fwd, dict(eps=float("nan")), INVALID), (fwd, dict(eps=float("inf")), INVALID),
    (fwd, dict(scale=float("inf")), INVALID), (fwd, dict(x=None), INVALID), (fwd, dict(w=None), INVALID),
    (fwd, dict(out=None), INVALID), (fwd, dict(lx=63), INVALID), (fwd, dict(lo=-64), INVALID),
    (fwd, dict(x=ctypes.c_void_p(0x10000001)), INVALID), (fwd, dict(r=ctypes.c_void_p(0x14000002)), INVALID),
    (fwd, dict(w=ctypes.c_void_p(0x18000004)), INVALID),
    (fwd, dict(out=p(0)), INVALID), (fwd, dict(out=p(2)), INVALID), (fwd, dict(ro=p(3)), INVALID),
    (fwd, dict(ro=p(1), lro=128), INVALID), (fwd, dict(ro=ctypes.c_void_p(0x14000040)), INVALID),
    (bwd, dict(dout=None), INVALID), (bwd, dict(r=None), INVALID), (bwd, dict(ws=None), WS), (bwd, dict(ws_bytes=64), WS),
    (bwd, dict(dx=p(0)), INVALID), (bwd, dict(dw=p(2)), INVALID), (bwd, dict(dw=p(1)), INVALID),
    (bwd, dict(ws=p(4)), INVALID), (bwd, dict(dres=p(1)), INVALID), (bwd, dict(scale=float("nan")), INVALID),
    (gate, dict(groups=0), INVALID), (gate, dict(groups=3), INVALID), (gate, dict(first=2), INVALID),
    (gate, dict(out=p(0)), INVALID), (gate, dict(z=None), INVALID), (gate, dict(lz=1), INVALID),
    (gate, dict(D=70000, groups=70000, ly=70000, lz=70000, lo=70000), UNSUP),
    (gate_bwd, dict(dy=p(1)), INVALID), (gate_bwd, dict(dz=p(4)), INVALID), (gate_bwd, dict(ws_bytes=0), WS),
    (gate_bwd, dict(ws=p(2)), INVALID), (gate_bwd, dict(io=-1), INVALID), (gate_bwd, dict(dz=None), INVALID),
])
def test_norm_refusals(call, kw, status):
    assert call(**kw) == status, ssd.last_error()
    assert ssd.last_error() != ""


def test_norm_refuses_rows_beyond_the_address_space():
    for call in (lambda: fwd(rows=1 << 40, lx=1 << 40), lambda: fwd(rows=1 << 62, lx=64),
                 lambda: gate(rows=1 << 33, lo=1 << 33), lambda: bwd(rows=1 << 31, ld=1 << 31)):
        assert call() == INVALID
        assert "address space" in ssd.last_error()


def test_norm_overlap_of_column_slices():
    """Slices of one buffer that share a row's columns are refused, whichever starts first."""
    a, b = ctypes.c_void_p(0x10000000 + 96), ctypes.c_void_p(0x10000000)
    for y, out in ((a, b), (b, a)):
        assert gate(y=y, ly=128, out=out, lo=128) == INVALID  # 64 columns of 2 bytes, 48 apart
        assert "overlaps" in ssd.last_error()
    assert gate(y=b, ly=256, out=ctypes.c_void_p(0x10000000 + 128), lo=128) == INVALID  # other strides


def test_norm_no_rows_needs_no_matrices():
    assert fwd(rows=0, x=None, out=None, ro=None, r=None) == OK
    assert gate(rows=0, y=None, z=None, out=None) == OK


def test_norm_workspace_size():
    size = ssd.norm_backward_workspace_size
    assert size(1, 64) >= 64 * 4 and size(32768, 2560) >= 2560 * 4
    assert size(0, 64) == 0 and size(4, 64, 3) == 0 and size(4, 16385) == 0 and size(-1, 64) == 0
    # a bounded number of parts: it does not grow with the rows for ever
    assert size(1 << 40, 2560) == size(1 << 30, 2560)
