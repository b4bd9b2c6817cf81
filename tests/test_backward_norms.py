"""The limits of test_backward_norms_gpu are tight: mistakes planted in the 64-bit reference pass them."""
import numpy as np
import pytest
import torch

from ssd_inputs import make_prefill
from tests.backward_ref import step_gradients
from tests.backward_spread import limits, spread

NAMES = ("dx", "ddt", "dA", "dB", "dC", "dD", "dh0")


def setup(b, T, H, G, N, **kw):
    c = make_prefill(b, T, H, 64, N, G, 64, dtype="bf16", seed=b + T + H + G, **dict(dict(h0_std=0.3), **kw))
    x, dt, A, B, C, D = (torch.from_numpy(np.ascontiguousarray(v)).double() for v in (c.x, c.dt, c.A, c.B, c.C, c.D))
    h0 = torch.zeros(b, H, 64, N, dtype=torch.float64) if c.h0 is None else torch.from_numpy(c.h0).double()
    g = torch.Generator().manual_seed(3)
    rnd = lambda t, s=1.0: torch.randn(t.shape, generator=g, dtype=torch.float64) * s  # noqa: E731
    return rnd(x), x, dt, A, B, C, D, h0, rnd(h0, 0.5)


@pytest.mark.parametrize("kw", [dict(), dict(dt_scale=1e-3), dict(dt_scale=30.0), dict(dt_scale=20.0, h0_std=0.0)])
@pytest.mark.parametrize("shape", [(1, 128, 1, 1), (2, 150, 4, 2), (1, 129, 16, 8)])
def test_zeros_fail(shape, kw):
    b, T, H, G = shape
    args = setup(b, T, H, G, 128, **kw)
    ref, sp = step_gradients(*args), spread(*args)
    for io, tc in ((torch.bfloat16, True), (torch.bfloat16, False), (torch.float32, False)):
        lim = limits(sp, ref, T, io, tc)
        for k in NAMES:
            assert lim[k] < 0.05 * ref[k].norm().item(), (k, lim[k] / ref[k].norm().item())


@pytest.mark.parametrize("H", [37, 80])
def test_a_head_left_out_fails(H):
    args = setup(1, 40, H, 1, 128)
    ref = step_gradients(*args)
    lim = limits(spread(*args), ref, 40, torch.bfloat16, True)
    dy, x, dt, A, B, C, D, h0, d = args
    s = slice(H - 1)
    less = step_gradients(dy[:, :, s], x[:, :, s], dt[:, :, s], A[s], B, C, D[s], h0[:, s], d[:, s])
    for k in ("dB", "dC"):
        assert (less[k] - ref[k]).norm().item() > 2 * lim[k], k


@pytest.mark.parametrize("seed", [1, 2])
def test_the_spread_is_the_size_of_the_gradients(seed):
    """For operands of random sign the root of the terms' squares is what the sums come to."""
    args = setup(1, 60 + seed, 8, 2, 64)
    ref, sp = step_gradients(*args), spread(*args)
    for k in ("dx", "ddt", "dB", "dC", "dD", "dh0"):
        assert 0.4 < sp[k].norm().item() / ref[k].norm().item() < 2.5, k
