"""Host-side refusals of the prefill's backward entry points: fake addresses, nothing is enqueued."""
import ctypes
import os

import pytest

import state_space_model_04_b200 as ssd
from state_space_model_04_b200 import ssd as binding

OK, INVALID, UNSUP, CUDA, TIMEOUT, WS, INTERNAL = range(7)

pytestmark = pytest.mark.skipif(not os.path.exists(binding.LIB_PATH), reason="library not built")

INS = ("dy", "x", "dt", "A", "B", "C", "D", "h0", "dh_final")
OUTS = ("dx", "ddt", "dA", "dB", "dC", "dD", "dh0")


def p(i):
    return ctypes.c_void_p(0x10000000 + 0x4000000 * i)


PTRS = dict({n: p(i) for i, n in enumerate(INS + OUTS)}, workspace=p(40), dt_bias=p(30), ddt_bias=p(31))


def plain(b=2, T=100, H=4, P=64, N=128, G=2, io=1, ws_bytes=1 << 30, **kw):
    a = dict(PTRS, **kw)
    return ssd.lib().ssd_prefill_backward(b, T, H, P, N, G, io, *(a[n] for n in INS), *(a[n] for n in OUTS),
                                          a["workspace"], ws_bytes, None)


def raw(b=2, T=100, H=4, P=64, N=128, G=2, io=1, lo=0.0, hi=float("inf"), ws_bytes=1 << 30, **kw):
    a = dict(PTRS, **kw)
    return ssd.lib().ssd_prefill_backward_dt_raw(b, T, H, P, N, G, io, a["dy"], a["x"], a["dt"], a["dt_bias"], lo, hi,
                                                 a["A"], a["B"], a["C"], a["D"], a["h0"], a["dh_final"], a["dx"],
                                                 a["ddt"], a["ddt_bias"], a["dA"], a["dB"], a["dC"], a["dD"], a["dh0"],
                                                 a["workspace"], ws_bytes, None)


@pytest.mark.parametrize("call", [plain, raw])
@pytest.mark.parametrize("kw,status", [
    (dict(b=-1), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(G=3), INVALID), (dict(G=0), INVALID),
    (dict(P=32), UNSUP), (dict(N=96), UNSUP), (dict(io=7), INVALID),
    (dict(ws_bytes=255), WS), (dict(workspace=None), WS), (dict(workspace=ctypes.c_void_p(0x50000008)), INVALID),
] + [({n: None}, INVALID) for n in INS[:7] + OUTS[:6]]
    + [({n: ctypes.c_void_p(PTRS[n].value + 4)}, INVALID) for n in INS + OUTS]
    + [({n: PTRS["x"]}, INVALID) for n in OUTS] + [({"dx": PTRS["dy"]}, INVALID), ({"dh0": PTRS["h0"]}, INVALID),
       ({"dh0": PTRS["dh_final"]}, INVALID), ({"dA": PTRS["dD"]}, INVALID), ({"dB": PTRS["dC"]}, INVALID),
       ({"workspace": PTRS["B"]}, INVALID), ({"workspace": PTRS["dh0"]}, INVALID)])
def test_refusals(call, kw, status):
    assert call(**kw) == status, ssd.last_error()
    assert ssd.last_error() != ""


@pytest.mark.parametrize("io,N", [(0, 64), (0, 128), (1, 64), (1, 128)])
def test_workspace_one_byte_short(io, N):
    need = ssd.prefill_backward_workspace_size(2, 100, 4, 64, N, 2, io)
    assert need > 256
    assert plain(N=N, io=io, ws_bytes=need - 1) == WS


@pytest.mark.parametrize("lo,hi", [(-1.0, 1.0), (float("nan"), 1.0), (0.0, float("nan")), (0.5, 0.5), (1.0, 0.5)])
def test_raw_step_clamp_refusals(lo, hi):
    assert raw(lo=lo, hi=hi) == INVALID


def test_raw_step_bias_refusals():
    assert raw(ddt_bias=PTRS["dA"]) == INVALID and "ddt_bias" in ssd.last_error()
    assert raw(ddt_bias=PTRS["dt_bias"]) == INVALID
    assert raw(dt_bias=PTRS["dD"]) == INVALID
    assert raw(dt_bias=ctypes.c_void_p(PTRS["dt_bias"].value + 4)) == INVALID


def test_workspace_size():
    size = ssd.prefill_backward_workspace_size
    assert size(0, 10, 4, 64, 64, 1, 0) == 0 and size(1, 0, 4, 64, 64, 1, 0) == 0
    assert size(1, 10, 4, 32, 64, 1, 0) == 0 and size(1, 10, 4, 64, 64, 3, 0) == 0
    assert size(1, 1, 1, 64, 64, 1, 0) >= 256 and size(2, 4096, 8, 64, 128, 1, 1) > size(1, 4096, 8, 64, 128, 1, 1)


def test_too_many_chunks_for_one_launch():
    assert ssd.prefill_backward_workspace_size(1 << 20, 1 << 20, 64, 64, 64, 1, 0) == 0
    assert plain(b=1 << 20, T=1 << 20, H=64, G=1, N=64, io=0, h0=None, dh_final=None, dh0=None) in (INVALID, UNSUP)


@pytest.mark.parametrize("ns", [0, 999999, 10**10 + 1])
def test_starve_limit_refusals(ns):
    assert ssd.lib().ssd_debug_starve_next_prefill_backward(ns) == INVALID


@pytest.mark.parametrize("role", [-1, 7])
def test_lag_role_refusals(role):
    assert ssd.lib().ssd_debug_lag_next_prefill_backward(role) == INVALID
    assert ssd.last_error() != ""
