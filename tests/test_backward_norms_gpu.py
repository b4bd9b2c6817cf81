"""The 2-norm of every gradient's error, beside the element bounds of test_backward_gpu: close enough to
the kernels' own roundings that a gradient of zeros or a head left out of a group's sum fails
(tests/test_backward_norms.py shows that the limits are that tight)."""
import pytest
import torch

from ssd_inputs import make_prefill
from tests.backward_ref import step_gradients
from tests.backward_spread import limits, spread
from tests.test_backward_gpu import NAMES, inputs

pytestmark = pytest.mark.gpu

ssd = pytest.importorskip("state_space_model_04_b200")

PATHS = [("f32", 64), ("f32", 128), ("bf16", 64), ("bf16", 128)]


def check(t, dy, d):
    args = (dy, t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"], t["h0"], d)
    got = ssd.prefill_backward(*args[:7], h0=t["h0"], dh_final=d, check=True)
    ref = step_gradients(*args)
    io = t["x"].dtype
    lim = limits(spread(*args), ref, t["dt"].shape[1], io, io == torch.bfloat16 and t["B"].shape[-1] == 128)
    bad = []
    for k in NAMES:
        off = (getattr(got, k).double() - ref[k]).norm().item()
        if not off <= lim[k]:
            bad.append("%s: %.3g off, %.3g of its norm, limit %.3g" % (k, off, off / ref[k].norm().item(), lim[k]))
    assert not bad, bad


def case(b, T, H, G, io, N, seed=0, **kw):
    c = make_prefill(b, T, H, 64, N, G, 64, dtype=io, seed=seed or b + T + H + G, **dict(dict(h0_std=0.3), **kw))
    return inputs(c, seed)


@pytest.mark.parametrize("io,N", PATHS)
@pytest.mark.parametrize("shape", [(1, 1, 1, 1), (1, 127, 3, 1), (1, 128, 4, 1), (1, 129, 2, 2), (2, 300, 4, 2),
                                   (3, 257, 16, 4), (2, 1100, 24, 3), (1, 3000, 2, 1), (2, 2049, 2, 1)])
def test_shapes(shape, io, N):
    b, T, H, G = shape
    check(*case(b, T, H, G, io, N))


@pytest.mark.parametrize("io,N", PATHS)
@pytest.mark.parametrize("shape", [(1, 1500, 37, 1), (1, 300, 80, 1), (2, 1300, 64, 8), (1, 2500, 76, 2)])
def test_heads_over_many_blocks(shape, io, N):
    b, T, H, G = shape
    check(*case(b, T, H, G, io, N))


@pytest.mark.parametrize("io,N", PATHS)
@pytest.mark.parametrize("scale", [1e-3, 30.0])
def test_weak_and_strong_decay(io, N, scale):
    check(*case(2, 300, 4, 2, io, N, 41, dt_scale=scale))


@pytest.mark.parametrize("io,N", PATHS)
@pytest.mark.parametrize("T", [66, 129])
def test_dA_behind_strong_steps(io, N, T):
    """As in test_backward_edges_gpu: with no state entering and steps that erase it, dA is many orders
    below its neighbours."""
    for seed in (236, 391):
        check(*case(1, T, 16, 8, io, N, seed, h0_std=0.0, dt_scale=20.0))


@pytest.mark.parametrize("io,N", PATHS)
@pytest.mark.parametrize("step", [6.0, 30.0, 100.0, 2000.0, 1e5])
def test_steps_that_reset_the_state(io, N, step):
    """Ordinary steps with some that erase the state between them: the decay between two tokens behind
    such a step is as exact as any other, however much the prefix sums of both hold, and the decay of the
    step itself gets no gradient (dA, times the step, would show it).  The operands x of those tokens are
    small, as their products with the step are to be like the others'."""
    t, dy, d = case(2, 400, 4, 2, io, N, 43)
    at = torch.tensor([0, 3, 37, 38, 70, 127, 128, 200, 230, 255, 301, 390])
    t["dt"][:, at] = step
    t["x"][:, at] = (t["x"][:, at].double() * 0.05 / step).to(t["x"].dtype)
    check(t, dy, d)


@pytest.mark.parametrize("io,N,b,T,H,part", [("bf16", 128, 110, 4096, 80, 10), ("f32", 64, 28, 16384, 80, 4)])
def test_every_sequence_beyond_32_bits(io, N, b, T, H, part):
    """More than 2^31 elements of x: every sequence and head gets what calls of a few sequences give it,
    and dA and dD are the sums of theirs.  The calls differ in how they cut sequences and heads, so an fp32
    state may round the other way: a step of 2^-16 of a state's halves on the tensor cores, two of them in a
    term, u times the sums' lengths on the fp32 pipes.  Results in bf16, and the factors rounded to bf16,
    then land a step (2^-7) away in one of 2^7 cases: an rms of 2^-10.5 each, three of them.  dS^T is
    rounded to bf16 as the sum over the heads a block holds, so in dB and dC that rounding, v / sqrt(3) in
    the mean square at most, is another one in each call: sqrt(2 / 3) v, and a quarter more."""
    dtype = torch.bfloat16 if io == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(52)
    x = torch.empty(b, T, H, 64, dtype=dtype, device="cuda").normal_(generator=g)
    assert x.numel() > 2 ** 31
    dy = torch.empty_like(x).normal_(generator=g)
    B, C = (torch.empty(b, T, 1, N, dtype=dtype, device="cuda").normal_(generator=g) for _ in range(2))
    dt = torch.empty(b, T, H, device="cuda").uniform_(0.001, 0.1, generator=g)
    A, D = -torch.empty(H, device="cuda").uniform_(1, 16, generator=g), torch.ones(H, device="cuda")
    got = ssd.prefill_backward(dy, x, dt, A, B, C, D, check=True)
    fine = 2.0 ** -15 if io == "bf16" else 4e-6
    coarse = 2.0 ** -9 if io == "bf16" else fine
    shares = 1.25 * (2 / 3) ** 0.5 * 2.0 ** -8 if io == "bf16" else fine
    sums = dict(dA=0.0, dD=0.0)
    for i in range(0, b, part):
        s = slice(i, min(b, i + part))
        ref = ssd.prefill_backward(dy[s], x[s], dt[s], A, B[s], C[s], D, check=True)
        for k, dims, tol in (("dx", (1, 3), coarse), ("ddt", 1, fine), ("dB", 1, shares), ("dC", 1, shares),
                             ("dh0", (2, 3), fine)):
            r = getattr(ref, k)
            off = torch.linalg.vector_norm(getattr(got, k)[s].float() - r.float(), dim=dims, dtype=torch.float64)
            norm = torch.linalg.vector_norm(r, dim=dims, dtype=torch.float64)
            assert (off <= tol * norm).all(), (k, i, (off / norm).max().item())
        for k in sums:
            sums[k] = sums[k] + getattr(ref, k).double()
    for k, r in sums.items():
        assert (getattr(got, k).double() - r).norm() <= fine * r.norm(), k
    del x, dy, B, C, dt, got, ref, r, off, norm
    torch.cuda.empty_cache()
