"""Residual and gated norms, forward and backward, against their formulas in 64 bits.

Tolerances, per element, from the arithmetic (u = 2^-24, half a step of fp32):
  stored results : half a step of the output's type on the result, finfo.eps / 2
  fp32 sums      : a reduction over a row adds at most 32 terms in a thread, 5 + 16 across
                   threads; with the operand roundings and the exponential (2 + 1.2 |z| ulp,
                   |z| < 16 here) every factor stays below 80 u of the sum of magnitudes
  dweight        : besides, a sum over rows: rows / 64 + 64 additions at most in a chain
Each bound is that count times u times the magnitude (the formula with absolute values).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ssd = pytest.importorskip("state_space_model_04_b200")

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def rand(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def close(got, ref, mag, what, count=80):
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != F32 else 0.0
    err = count * U * mag
    bound = half * (ref.abs() + err) + err + 1e-37
    bad = ((got.double() - ref).abs() / bound).max().item() if ref.numel() else 0.0
    assert torch.isfinite(got).all() and bad <= 1.0, "%s: %.3f of its bound" % (what, bad)


def residual_ref(x, res, w, scale, eps):
    r = scale * x.double() + (0 if res is None else res.double())
    rmag = (scale * x.double()).abs() + (0 if res is None else res.double().abs())
    k = (r.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    # r itself may cancel: its error is u of its terms, in the mean too
    kmag = 1 + (rmag.pow(2).mean(-1, keepdim=True)) * k * k
    return r, r * k * w.double(), rmag, (rmag * k + (r * k).abs() * kmag) * w.double().abs()


def residual_backward_ref(dout, r, w, dro, scale, eps):
    g, r, w = dout.double(), r.double(), w.double()
    k = (r.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    n = r * k
    dr = k * (g * w - n * (g * w * n).mean(-1, keepdim=True))
    mag = k * ((g * w).abs() + n.abs() * (g * w * n).abs().mean(-1, keepdim=True))
    if dro is not None:
        dr, mag = dr + dro.double(), mag + dro.double().abs()
    D = dout.shape[-1]
    return dr, mag, (g * n).reshape(-1, D).sum(0), (g * n).abs().reshape(-1, D).sum(0)


def gated_ref(y, z, w, groups, eps, first):
    D = y.shape[-1]
    y, z, w = y.double(), z.double(), w.double()
    gate = z * torch.sigmoid(z)
    v = (y if first else y * gate).reshape(-1, groups, D // groups)
    k = (v.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    out = (v * k).reshape(y.shape) * w * (gate if first else 1)
    return out, out.abs()


def gated_backward_ref(dout, y, z, w, groups, eps, first):
    shape, D = y.shape, y.shape[-1]
    go, y, z, w = dout.double(), y.double(), z.double(), w.double()
    sg = torch.sigmoid(z)
    gate, dgate = z * sg, sg * (1 + z * (1 - sg))
    dmag = sg * (1 + z.abs())
    v = (y if first else y * gate).reshape(-1, groups, D // groups)
    k = (v.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    n = v * k
    t = go * gate if first else go
    gw = (t * w).reshape(v.shape)
    dv = (k * (gw - n * (gw * n).mean(-1, keepdim=True))).reshape(shape)
    mv = (k * (gw.abs() + n.abs() * (gw * n).abs().mean(-1, keepdim=True))).reshape(shape)
    dw, mw = (t * n.reshape(shape)).reshape(-1, D).sum(0), (t * n.reshape(shape)).abs().reshape(-1, D).sum(0)
    if first:
        u = go * n.reshape(shape) * w
        return dv, mv, u * dgate, u.abs() * dmag, dw, mw
    return dv * gate, mv * gate.abs(), dv * y * dgate, mv * y.abs() * dmag, dw, mw


SHAPES = [(1, 1), (1, 64), (3, 7), (1, 2560), (2, 2049), (5, 8), (257, 96), (33, 2560), (4, 16384), (7, 5001),
          (3, 16383), (1000, 320), (130, 6152)]


@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("io,res", [(BF, F32), (BF, BF), (F32, F32)])
def test_residual_norm(rows, D, io, res):
    g = gen(rows * 7 + D)
    x, w = rand(g, rows, D, dtype=io), 1 + 0.1 * rand(g, D)
    residual = rand(g, rows, D, std=2.0, dtype=res)
    for rsd, scale in ((residual, 0.5), (None, 1.0)):
        ro = torch.empty(rows, D, dtype=res, device="cuda") if rsd is None else None
        out, r = ssd.residual_norm(x, w, rsd, scale=scale, eps=1e-5, residual_out=ro)
        rr, oo, rmag, omag = residual_ref(x, rsd, w, scale, 1e-5)
        close(r, rr, rmag, "r")
        close(out, oo, omag, "out")


@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("io,res", [(BF, F32), (BF, BF), (F32, F32)])
def test_residual_norm_backward(rows, D, io, res):
    g = gen(rows * 11 + D)
    dout, w = rand(g, rows, D, dtype=io), 1 + 0.1 * rand(g, D)
    r, dro = rand(g, rows, D, std=2.0, dtype=res), rand(g, rows, D, dtype=res)
    for d in (dro, None):
        dx, dres, dw = ssd.residual_norm_backward(dout, r, w, d, scale=0.25, eps=1e-5)
        dr, mag, dwr, dwm = residual_backward_ref(dout, r, w, d, 0.25, 1e-5)
        close(dres, dr, mag, "dresidual")
        close(dx, 0.25 * dr, 0.25 * mag, "dx")
        close(dw, dwr, dwm, "dweight", 144 + rows / 64)
    dx, none, _ = ssd.residual_norm_backward(dout, r, w, dro, scale=0.25, want_dresidual=False)
    assert none is None
    dr, mag, _, _ = residual_backward_ref(dout, r, w, dro, 0.25, 1e-5)
    close(dx, 0.25 * dr, 0.25 * mag, "dx alone")


GATED = [(1, 1, 1), (1, 5120, 1), (3, 96, 3), (32, 5120, 8), (5, 1000, 8), (9, 777, 7), (2, 16384, 1), (3, 16384, 2),
         (515, 256, 4), (64, 40, 5), (2, 10001, 1)]


@pytest.mark.parametrize("rows,D,groups", GATED)
@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("first", [False, True])
def test_gated_norm(rows, D, groups, io, first):
    g = gen(rows + D * 3 + groups)
    y, z, dout = rand(g, rows, D, dtype=io), rand(g, rows, D, std=2.0, dtype=io), rand(g, rows, D, dtype=io)
    w = 1 + 0.1 * rand(g, D)
    out = ssd.gated_norm(y, z, w, groups=groups, norm_before_gate=first)
    ref, mag = gated_ref(y, z, w, groups, 1e-5, first)
    close(out, ref, mag, "out")
    dy, dz, dw = ssd.gated_norm_backward(dout, y, z, w, groups=groups, norm_before_gate=first)
    ry, my, rz, mz, rw, mw = gated_backward_ref(dout, y, z, w, groups, 1e-5, first)
    close(dy, ry, my, "dy")
    close(dz, rz, mz, "dz")
    close(dw, rw, mw, "dweight", 144 + rows / 64)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("offset", [0, 8, 3])
def test_strided_operands(io, offset):
    """Slices of wider rows at aligned and odd offsets, in and out; what lies beside an output
    slice stays as it was."""
    g = gen(5 + offset)
    rows, D, W = 37, 512, 1240
    wide = [rand(g, 2, rows, W, dtype=io) for _ in range(4)]
    y, z, dout = (t[..., offset:offset + D] for t in wide[:3])
    w = 1 + 0.1 * rand(g, D)
    keep = wide[3].clone()
    dz = wide[3][..., offset:offset + D]
    out = ssd.gated_norm(y, z, w, groups=2)
    ref, mag = gated_ref(y, z, w, 2, 1e-5, False)
    close(out, ref, mag, "out")
    dy, dz2, dw = ssd.gated_norm_backward(dout, y, z, w, groups=2, dz=dz)
    assert dz2.data_ptr() == dz.data_ptr()
    ry, my, rz, mz, rw, mw = gated_backward_ref(dout, y, z, w, 2, 1e-5, False)
    close(dy, ry, my, "dy")
    close(dz, rz, mz, "dz")
    close(dw, rw, mw, "dweight", 146)
    assert torch.equal(wide[3][..., :offset], keep[..., :offset])
    assert torch.equal(wide[3][..., offset + D:], keep[..., offset + D:])
    out, r = ssd.residual_norm(y, w, z, scale=2.0)
    rr, oo, rmag, omag = residual_ref(y, z, w, 2.0, 1e-5)
    close(r, rr, rmag, "r")
    close(out, oo, omag, "out")


def test_side_by_side_in_one_buffer():
    """Both gradients as column slices of one buffer, and a result beside its operand."""
    g = gen(21)
    rows, D = 45, 320
    y, z, dout = (rand(g, rows, D, dtype=BF) for _ in range(3))
    w = 1 + 0.1 * rand(g, D)
    want = ssd.gated_norm_backward(dout, y, z, w)
    buf = torch.zeros(rows, 2 * D + 16, dtype=BF, device="cuda")
    dy, dz, dw = ssd.gated_norm_backward(dout, y, z, w, dy=buf[:, :D], dz=buf[:, D + 8:2 * D + 8])
    assert torch.equal(dy, want[0]) and torch.equal(dz, want[1]) and torch.equal(dw, want[2])
    assert (buf[:, D:D + 8] == 0).all() and (buf[:, 2 * D + 8:] == 0).all()
    pair = torch.cat([y, y], 1)
    ssd.gated_norm(pair[:, :D], z, w, out=pair[:, D:])
    assert torch.equal(pair[:, D:], ssd.gated_norm(y, z, w)) and torch.equal(pair[:, :D], y)


@pytest.mark.parametrize("D,offset", [(32, 0), (31, 1)])
def test_rows_beyond_32_bit_offsets(D, offset):
    """Short rows so far apart that those side by side in a block pass 2^32 bytes; the same values
    packed give the same bits (the sums of a row do not depend on its place)."""
    g = gen(22)
    rows, ld = 11, (1 << 29) + 8  # bf16: 1 GiB and 16 bytes apart
    store = torch.empty((rows - 1) * ld + 64, dtype=BF, device="cuda")
    far = store.as_strided((rows, D), (ld, 1), offset)
    x, res, dout, w = rand(g, rows, D, dtype=BF), rand(g, rows, D), rand(g, rows, D, dtype=BF), 1 + 0.1 * rand(g, D)
    far.copy_(x)
    for a, b in zip(ssd.residual_norm(x, w, res), ssd.residual_norm(far, w, res)):
        assert torch.equal(a, b)
    assert torch.equal(ssd.gated_norm(dout, x, w), ssd.gated_norm(dout, far, w))
    ref = ssd.gated_norm_backward(dout, x, x, w)
    got = ssd.gated_norm_backward(dout, far, far, w)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    mag = gated_backward_ref(dout, x, x, w, 1, 1e-5, False)[5]  # the same 11 terms, added in two orders
    assert ((ref[2] - got[2]).double().abs() <= 2 * 10 * U * mag).all()
    r = res.to(BF)
    ref = ssd.residual_norm_backward(x, r, w)
    got = ssd.residual_norm_backward(far, r, w)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])


def test_in_place_residual_and_gradient():
    g = gen(3)
    x, res, w = rand(g, 65, 2560, dtype=BF), rand(g, 65, 2560), 1 + 0.1 * rand(g, 2560)
    out, r = ssd.residual_norm(x, w, res.clone(), scale=0.5)
    buf = res.clone()
    out2, r2 = ssd.residual_norm(x, w, buf, scale=0.5, residual_out=buf)
    assert r2.data_ptr() == buf.data_ptr() and torch.equal(r, buf) and torch.equal(out, out2)
    dout, dro = rand(g, 65, 2560, dtype=BF), rand(g, 65, 2560)
    want = ssd.residual_norm_backward(dout, r, w, dro.clone(), scale=0.5)
    got = ssd.residual_norm_backward(dout, r, w, dro, scale=0.5, dresidual=dro)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_no_rows():
    w = torch.ones(64, device="cuda")
    e = torch.empty(0, 64, dtype=BF, device="cuda")
    out, r = ssd.residual_norm(e, w, torch.empty(0, 64, device="cuda"))
    assert out.shape == (0, 64) and r.shape == (0, 64)
    dw = torch.full((64,), 7.0, device="cuda")
    ssd.residual_norm_backward(e, torch.empty(0, 64, device="cuda"), w, dweight=dw)
    assert (dw == 0).all()
    dw.fill_(7.0)
    ssd.gated_norm_backward(e, e, e, w, dweight=dw)
    assert (dw == 0).all() and ssd.gated_norm(e, e, w).shape == (0, 64)


def test_extreme_gates_and_zero_rows():
    """Saturated gates give 0 and y, a zero row gives zeros and finite gradients."""
    y = torch.ones(3, 64, device="cuda")
    z = torch.tensor([[-200.0], [200.0], [0.0]], device="cuda").expand(3, 64).contiguous()
    w = torch.ones(64, device="cuda")
    out = ssd.gated_norm(y, z, w, norm_before_gate=True)
    assert (out[0] == 0).all() and (out[2] == 0).all()
    torch.testing.assert_close(out[1], torch.full((64,), 200.0, device="cuda"), rtol=2e-5, atol=0)
    for first in (False, True):
        for t in ssd.gated_norm_backward(y, torch.zeros_like(y), z, w, norm_before_gate=first):
            assert torch.isfinite(t).all()
    out, _ = ssd.residual_norm(torch.zeros(2, 64, device="cuda"), w)
    assert (out == 0).all()


def test_nan_and_inf_stay_in_their_row():
    g = gen(9)
    x, w = rand(g, 6, 256, dtype=BF), torch.ones(256, device="cuda")
    x[2, 5] = float("nan")
    x[4, 7] = float("inf")
    out, _ = ssd.residual_norm(x, w)
    clean = torch.isfinite(out).all(-1)
    assert clean.tolist() == [True, True, False, True, False, True]


def test_other_stream_graph_and_repeat():
    """A captured backward pass replays on new contents; the same call gives the same bits; a
    call on a side stream is ordered there."""
    g = gen(21)
    rows, D = 3000, 2560
    mk = lambda: (rand(g, rows, D, dtype=BF), rand(g, rows, D, dtype=BF), rand(g, rows, D, dtype=BF))  # noqa: E731
    dout, y, z = mk()
    w = 1 + 0.1 * rand(g, D)
    dy, dz, dw = torch.empty_like(y), torch.empty_like(y), torch.empty(D, device="cuda")
    ws = torch.empty(ssd.norm_backward_workspace_size(rows, D), dtype=torch.uint8, device="cuda")
    kw = dict(dy=dy, dz=dz, dweight=dw, workspace=ws)
    ssd.gated_norm_backward(dout, y, z, w, **kw)
    first = [t.clone() for t in (dy, dz, dw)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in (dy, dz, dw):
            t.zero_()
        ssd.gated_norm_backward(dout, y, z, w, stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, (dy, dz, dw)):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssd.gated_norm_backward(dout, y, z, w, **kw)
    for t, n in zip((dout, y, z), mk()):
        t.copy_(n)
    graph.replay()
    got = [t.clone() for t in (dy, dz, dw)]
    want = ssd.gated_norm_backward(dout, y, z, w)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_temporary_workspace_on_another_stream():
    """Memory taken on the current stream right behind a call on another is not the call's workspace."""
    g = gen(31)
    x, r, w = rand(g, 20000, 2560, dtype=BF), rand(g, 20000, 2560), 1 + 0.1 * rand(g, 2560)
    want = ssd.residual_norm_backward(x, r, w)[2], ssd.gated_norm_backward(x, x, x, w)[2]
    need = ssd.norm_backward_workspace_size(20000, 2560)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        a = ssd.residual_norm_backward(x, r, w, stream=s)[2]
        torch.empty(need, dtype=torch.uint8, device="cuda").fill_(255)
        b = ssd.gated_norm_backward(x, x, x, w, stream=s)[2]
        torch.empty(need, dtype=torch.uint8, device="cuda").fill_(255)
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_gradients_against_differences():
    """Central differences of sum(out * c) along random directions, fp32."""
    g = gen(31)
    rows, D = 4, 96
    y, z, w = rand(g, rows, D), rand(g, rows, D), 1 + 0.1 * rand(g, D)
    c = rand(g, rows, D)
    for first in (False, True):
        dy, dz, dw = ssd.gated_norm_backward(c, y, z, w, groups=3, norm_before_gate=first)
        for t, grad in ((y, dy), (z, dz), (w, dw)):
            d = rand(g, *t.shape)
            h = 2.0 ** -7

            def f(s):
                a = [v.double() + (s * d.double() if v is t else 0) for v in (y, z, w)]
                return (gated_ref(*a, 3, 1e-5, first)[0] * c.double()).sum().item()

            num = (f(h) - f(-h)) / (2 * h)
            # the difference's own error is h^2 / 6 of the third derivative; the directions are O(1)
            assert abs(num - (grad.double() * d.double()).sum().item()) <= 2e-3 * np.sqrt(rows * D)


def test_binding_refusals():
    w = torch.ones(64, device="cuda")
    x = torch.ones(4, 64, device="cuda")
    with pytest.raises(ValueError):
        ssd.residual_norm(x.cpu(), w)
    with pytest.raises(TypeError):
        ssd.residual_norm(x.half(), w)
    with pytest.raises(TypeError):
        ssd.residual_norm(x, w.bfloat16())
    with pytest.raises(ValueError):
        ssd.residual_norm(x, torch.ones(32, device="cuda"))
    with pytest.raises(ValueError):
        ssd.residual_norm(x, w, torch.ones(3, 64, device="cuda"))
    with pytest.raises(ValueError):
        ssd.residual_norm(x.t().contiguous().t(), w)  # rows not contiguous
    with pytest.raises(ValueError):
        ssd.residual_norm(x[:1].expand(4, 64), w)  # rows overlap
    with pytest.raises(TypeError):
        ssd.gated_norm(x, x.bfloat16(), w)
    with pytest.raises(ssd.SSDError):
        ssd.gated_norm(x, x, w, groups=5)
    with pytest.raises(ssd.SSDError):
        ssd.gated_norm(x, x, w, out=x)
    with pytest.raises(ssd.SSDError):
        ssd.residual_norm(x, w, eps=-1.0)
    with pytest.raises(ssd.SSDError):
        ssd.residual_norm(x, w, scale=float("nan"))
    with pytest.raises(ssd.SSDError):
        ssd.gated_norm_backward(x, x, x, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
