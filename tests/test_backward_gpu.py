"""prefill_backward against the token-by-token gradients in 64 bits.

Tolerances, per element, as a multiple of the magnitude behind the element (the same sums of
absolute values, tests/backward_ref.py), u = 2^-24 and v = 2^-8 (half a step of bf16):
  fp32 path     at most 128 terms a product in a chunk, three products in a row, one scan step a
                chunk and the decay factors: (512 + 2 chunks) u; half a step of the output's type
  tensor cores  V and Y from states of 16 bits (two halves), the states from weighted rows of 16
                bits: 4 v^2 for the fp32 gradients; the pair terms, weighted rows and states that
                feed only bf16 gradients round to bf16 once each: 2 v (a product of two of them),
                dx 1 v for M and 4 v^2
  da            as a suffix sum inside a chunk it also carries u of the chunk's sum of pair terms,
                at most 2 sum of the magnitudes of da over the chunk (each pair (i, j) counts in
                some da_t between them), so ddt gets 512 u |A| times that
  dA, ddt_bias  sums of those bounds over tokens
"""
import numpy as np
import pytest
import torch

from ssd_inputs import make_prefill
from tests.backward_ref import step_gradients
from tests.helpers import prefill_inputs

pytestmark = pytest.mark.gpu

ssd = pytest.importorskip("state_space_model_04_b200")

U, V = 2.0 ** -24, 2.0 ** -8
NAMES = ("dx", "ddt", "dA", "dB", "dC", "dD", "dh0")


def inputs(case, seed=0, dhf=True):
    t = prefill_inputs(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dy = torch.randn(t["x"].shape, generator=g, device="cuda").to(t["x"].dtype)
    d = torch.randn(case.b, case.H, 64, case.N, generator=g, device="cuda") * 0.5 if dhf else None
    return t, dy, d


def bounds(t, dy, dhf, ref, tc):
    """Error bounds by name.  tc: the tensor-core path's intermediate roundings."""
    mag = step_gradients(dy, t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"], t["h0"], dhf, absolute=True)
    T = t["dt"].shape[1]
    nc = -(-T // 64)
    f = (512 + 2 * nc) * U + (4 * V * V if tc else 0)
    damag = mag["da"]
    chunk = torch.zeros_like(damag)
    for c in range(0, T, 128):
        chunk[:, c:c + 128] = damag[:, c:c + 128].sum(1, keepdim=True)
    daerr = f * (damag + 2 * chunk)
    A = t["A"].double().abs()
    out = {k: f * mag[k] for k in ("dx", "dB", "dC", "dD", "dh0")}
    if tc:
        for k, c in (("dx", 1), ("dB", 2), ("dC", 2)):
            out[k] = out[k] + c * V * (1 + V) * mag[k]
    out["ddt"] = f * mag["ddt"] + A * daerr
    out["dA"] = (t["dt"].double() * daerr).sum((0, 1)) + f * mag["dA"]
    half = torch.finfo(t["x"].dtype).eps / 2 if t["x"].dtype != torch.float32 else 0.0
    for k in ("dx", "dB", "dC"):
        out[k] = out[k] + half * (ref[k].abs() + out[k])
    return out


def check_grads(got, ref, bnd, names=NAMES):
    for k in names:
        g = getattr(got, k)
        assert torch.isfinite(g).all(), k
        r = ((g.double() - ref[k]).abs() / (bnd[k] + 1e-30)).max().item() if g.numel() else 0.0
        assert r <= 1.0, "%s: %.3f of its bound" % (k, r)


def run_case(case, seed=0, dhf=True, tc=False):
    t, dy, d = inputs(case, seed, dhf)
    got = ssd.prefill_backward(dy, t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"], h0=t["h0"], dh_final=d, check=True)
    ref = step_gradients(dy, t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"], t["h0"], d)
    check_grads(got, ref, bounds(t, dy, d, ref, tc))
    return got, ref, t, dy, d


# b, T, H, N, G
SHAPES = [(1, 1, 1, 64, 1), (1, 63, 2, 64, 1), (1, 64, 2, 128, 2), (2, 65, 4, 64, 2), (1, 200, 6, 128, 3),
          (3, 129, 2, 128, 1), (1, 512, 4, 64, 1), (2, 321, 8, 128, 8)]


@pytest.mark.parametrize("shape", SHAPES)
def test_fp32(shape):
    b, T, H, N, G = shape
    run_case(make_prefill(b, T, H, 64, N, G, 64, dtype="f32", h0_std=0.3, seed=sum(shape)))


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[3] == 64])
def test_bf16_small_state(shape):
    b, T, H, N, G = shape
    run_case(make_prefill(b, T, H, 64, N, G, 64, dtype="bf16", h0_std=0.3, seed=sum(shape)))


# b, T, H, N, G: one token, less and more than a chunk, several chunks, groups, more items than SMs
TC_SHAPES = [(1, 1, 1, 128, 1), (1, 128, 1, 128, 1), (1, 127, 3, 128, 1), (1, 129, 2, 128, 2), (2, 300, 4, 128, 2),
             (1, 700, 6, 128, 1), (3, 257, 16, 128, 4), (2, 1100, 24, 128, 3)]


@pytest.mark.parametrize("shape", TC_SHAPES)
def test_bf16_tensor_cores(shape):
    b, T, H, N, G = shape
    run_case(make_prefill(b, T, H, 64, N, G, 64, dtype="bf16", h0_std=0.3, seed=sum(shape)), tc=True)
