"""The gate of the gated norm over the whole range of z, closed gates among it, on fp32: each result
relative to its own size.  u = 2^-24.  With y of one magnitude in a group of D <= 8192 elements:
  k             the mean's sum 5 + 16 + 32 u, half of it in the root, 4 u for the root's own: 31 u
  sigmoid       the exponential 2 u, 1 + e one, the quotient 4 u: 7 u (where e is below 2^-126 its step of 2^-149
                besides)
  products      at most 5 roundings: 5 u
so 43 u; silu'(z) = s + z s (1 - s) besides takes 8 u of s and of 1 - s: 48 u of s (1 + |z|), and dy's difference
two terms of 43 u and their mean."""
import pytest
import torch

from tests.test_norm_gpu import gated_backward_ref

pytestmark = pytest.mark.gpu

ssd = pytest.importorskip("state_space_model_04_b200")

U = 2.0 ** -24


def gates(rows, D):
    g = torch.Generator(device="cuda").manual_seed(D)
    z = torch.linspace(-103.0, 95.0, rows * D, dtype=torch.float64, device="cuda").float()
    return z[torch.randperm(rows * D, generator=g, device="cuda")].view(rows, D), g


@pytest.mark.parametrize("rows,D,groups", [(7, 63, 1), (5, 96, 3), (9, 2560, 4), (3, 2560, 1), (2, 8192, 1), (4, 4096, 4),
                                           (2, 3001, 1)])
def test_forward(rows, D, groups):
    z, g = gates(rows, D)
    y = torch.where(torch.rand(rows, D, generator=g, device="cuda") < 0.5, -1.5, 1.5)
    w = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    out = ssd.gated_norm(y, z, w, groups=groups, norm_before_gate=True)
    zd = z.double()
    k = (2.25 + 1e-5) ** -0.5
    s = torch.exp(torch.where(zd < 0, zd, 0)) / (1 + torch.exp(-zd.abs()))
    ref = y.double() * k * w.double() * zd * s
    floor = 2.0 ** -149 * (1 + zd.abs()) * 2
    bad = (out.double() - ref).abs() / (43 * U * ref.abs() + floor)
    assert bad.max().item() <= 1, (bad.max().item(), z.flatten()[bad.argmax()].item())


@pytest.mark.parametrize("rows,D,groups", [(7, 63, 1), (5, 96, 3), (9, 2560, 4), (3, 2560, 1), (2, 8192, 1), (4, 4096, 4),
                                           (2, 3001, 1)])
def test_backward(rows, D, groups):
    z, g = gates(rows, D)
    y = torch.where(torch.rand(rows, D, generator=g, device="cuda") < 0.5, -1.5, 1.5)
    dout = torch.randn(rows, D, generator=g, device="cuda")
    w = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    dy, dz, dw = ssd.gated_norm_backward(dout, y, z, w, groups=groups, norm_before_gate=True)
    ry, my, rz, mz, rw, mw = gated_backward_ref(dout, y, z, w, groups, 1e-5, True)
    floor = 2.0 ** -149 * (1 + z.double().abs()) * 16 * dout.double().abs().clamp_min(1)
    assert ((dz.double() - rz).abs() <= 48 * U * mz + floor).all()
    assert ((dy.double() - ry).abs() <= 3 * 43 * U * my + floor).all()
    assert ((dw.double() - rw).abs() <= (48 + rows) * U * mw + floor.sum(0)).all()
