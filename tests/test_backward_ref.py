"""The 64-bit reference of the prefill's gradients, pinned on the CPU: its forward half is the
oracle's recurrence, and its gradients are the oracle's central differences."""
import numpy as np
import pytest
import torch

import oracle
from ssd_inputs import make_prefill
from tests.backward_ref import step_gradients


def _tensors(c):
    return [torch.from_numpy(np.ascontiguousarray(v)).double() for v in (c.x, c.dt, c.A, c.B, c.C, c.D, c.h0)]


@pytest.mark.parametrize("shape", [(1, 9, 2, 1), (2, 5, 4, 2), (1, 1, 1, 1)])
def test_reference_matches_oracle_differences(shape):
    b, T, H, G = shape
    c = make_prefill(b, T, H, 64, 64, G, 64, dtype="f32", h0_std=0.5, seed=sum(shape), dt_scale=4.0)
    x, dt, A, B, C, D, h0 = _tensors(c)
    g = torch.Generator().manual_seed(1)
    rnd = lambda t: torch.randn(t.shape, generator=g, dtype=torch.float64)  # noqa: E731
    cy, ch = rnd(x), rnd(h0)
    out = step_gradients(cy, x, dt, A, B, C, D, h0, ch)
    y, hf = oracle.ssd_recurrence(*(t.numpy() for t in (x, dt, A, B, C, D, h0)))
    np.testing.assert_allclose(out["y"].numpy(), y, rtol=1e-6, atol=1e-6)  # the oracle reads fp32 inputs

    def loss(v):  # in torch, in 64 bits: the recurrence as the oracle states it
        x, dt, A, B, C, D, h = v
        tot = 0.0
        rep = lambda t: t.repeat_interleave(H // G, 2)  # noqa: E731
        for t in range(T):
            h = torch.exp(dt[:, t] * A)[..., None, None] * h + (dt[:, t, :, None] * x[:, t])[..., None] * rep(B)[:, t, :, None, :]
            tot = tot + ((h * rep(C)[:, t, :, None, :]).sum(-1) + D[:, None] * x[:, t]).mul(cy[:, t]).sum()
        return (tot + (h * ch).sum()).item()

    base = [x, dt, A, B, C, D, h0]
    for i, name in enumerate(["dx", "ddt", "dA", "dB", "dC", "dD", "dh0"]):
        d, s = rnd(base[i]), 1e-5
        f = [loss([t + (e * s * d if k == i else 0) for k, t in enumerate(base)]) for e in (1, -1)]
        num, ana = (f[0] - f[1]) / (2 * s), (out[name] * d).sum().item()
        assert abs(num - ana) <= 1e-6 * max(1.0, abs(ana)), name


def test_magnitudes_bound_the_gradients():
    c = make_prefill(1, 20, 2, 64, 64, 1, 64, dtype="f32", h0_std=0.5, seed=3)
    t = _tensors(c)
    dy = torch.randn(t[0].shape, dtype=torch.float64)
    a, m = step_gradients(dy, *t), step_gradients(dy, *t, absolute=True)
    for k in a:
        assert (a[k].abs() <= m[k] * (1 + 1e-12) + 1e-300).all(), k
