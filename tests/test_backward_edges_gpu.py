"""prefill_backward at its edges: empty calls, the raw step, extreme decays, a lone non-finite
sequence, long calls, given outputs, streams and graphs, a wait that runs out, and together with
the norms around it.  Bounds as in test_backward_gpu."""
import numpy as np
import pytest
import torch

from ssd_inputs import make_prefill
from tests.backward_ref import step_gradients
from tests.test_backward_gpu import NAMES, U, bounds, check_grads, inputs, run_case

pytestmark = pytest.mark.gpu

ssd = pytest.importorskip("state_space_model_04_b200")

# io, N: the fp32 pipes and the tensor cores
PATHS = [("f32", 64), ("f32", 128), ("bf16", 64), ("bf16", 128)]


def on_tc(io, N):
    return io == "bf16" and N == 128


def draw(b, T, H, N, G, io, seed, **kw):
    return inputs(make_prefill(b, T, H, 64, N, G, 64, dtype=io, h0_std=0.3, seed=seed, **kw), seed)


def call(t, dy, d, **kw):
    return ssd.prefill_backward(dy, t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"], h0=t["h0"], dh_final=d, **kw)


def same(a, b, names=NAMES):
    for k in names:
        assert torch.equal(getattr(a, k), getattr(b, k)), k


@pytest.mark.parametrize("io,N", PATHS)
@pytest.mark.parametrize("b,T", [(2, 0), (0, 5)])
def test_no_tokens(io, N, b, T):
    dt_io = torch.float32 if io == "f32" else torch.bfloat16
    H = 3
    x, B = torch.empty(b, T, H, 64, dtype=dt_io, device="cuda"), torch.empty(b, T, 1, N, dtype=dt_io, device="cuda")
    dt, A = torch.empty(b, T, H, device="cuda"), -torch.ones(H, device="cuda")
    d = torch.randn(b, H, 64, N, device="cuda")
    for dhf in (d, None):
        grads = ssd.PrefillGrads(x.clone(), dt.clone(), torch.full_like(A, 7.0), B.clone(), B.clone(),
                                 torch.full_like(A, 7.0), torch.full_like(d, 7.0), torch.full_like(A, 7.0))
        ssd.prefill_backward(x, x.clone(), dt, A, B, B, torch.ones_like(A), dh_final=dhf, grads=grads, dt_raw=True,
                             check=True)
        assert (grads.dA == 0).all() and (grads.dD == 0).all() and (grads.ddt_bias == 0).all()
        assert torch.equal(grads.dh0, torch.zeros_like(d) if dhf is None else d)


@pytest.mark.parametrize("io,N", PATHS)
@pytest.mark.parametrize("bias", [True, False])
def test_raw_step(io, N, bias):
    """The chain rule through clamp(softplus(raw + bias)), with steps below, inside and above the
    clamp.  The kernel forms dt in fp32, a few u off: a term that decays by exp(-S) moves by 8 u S of
    itself, at most 8 u of the undecayed term, and the bounds get 64 u of the magnitudes for it."""
    b, T, H, G = 2, 200, 6, 2
    t, dy, d = draw(b, T, H, N, G, io, 31)
    rng = np.random.default_rng(32)
    raw = torch.from_numpy((rng.standard_normal((b, T, H)) * 1.5 - 3.0).astype(np.float32)).cuda()
    bv = torch.from_numpy((rng.standard_normal(H) * 0.5).astype(np.float32)).cuda() if bias else None
    lo, hi = 0.01, 0.2
    z = raw + (0 if bv is None else bv)  # one rounding, as the kernel adds
    sp = torch.nn.functional.softplus(z.double(), threshold=1e9)
    for lim in (lo, hi):  # no draw so near a limit that rounding could decide
        assert ((sp / lim - 1).abs() > 1e-5).all()
    assert (sp < lo).any() and (sp > hi).any() and ((sp > lo) & (sp < hi)).any()
    dt = sp.clamp(lo, hi)
    slope = torch.where((sp >= lo) & (sp <= hi), torch.sigmoid(z.double()), torch.zeros_like(sp))
    got = ssd.prefill_backward(dy, t["x"], raw, t["A"], t["B"], t["C"], t["D"], h0=t["h0"], dh_final=d, dt_raw=True,
                               dt_bias=bv, dt_min=lo, dt_max=hi, check=True)
    t["dt"] = dt
    ref = step_gradients(dy, t["x"], dt, t["A"], t["B"], t["C"], t["D"], t["h0"], d)
    mag = step_gradients(dy, t["x"], dt, t["A"], t["B"], t["C"], t["D"], t["h0"], d, absolute=True)
    bnd = bounds(t, dy, d, ref, on_tc(io, N))
    for k in NAMES:
        bnd[k] = bnd[k] + 64 * U * mag[k]
    check_grads(got, ref, bnd, ("dx", "dA", "dB", "dC", "dD", "dh0"))
    err = slope * (bnd["ddt"] + 8 * U * ref["ddt"].abs())
    assert ((got.ddt.double() - slope * ref["ddt"]).abs() <= err + 1e-30).all()
    assert (got.ddt[slope == 0] == 0).all()
    if bias:
        assert ((got.ddt_bias.double() - (slope * ref["ddt"]).sum((0, 1))).abs() <= err.sum((0, 1))).all()
    else:
        assert got.ddt_bias is None


def test_raw_step_extremes():
    """Steps at which softplus underflows, is linear, or overflows an exponential: finite gradients,
    none where the slope is zero."""
    for io, N in PATHS:
        t, dy, d = draw(1, 130, 2, N, 1, io, 33)
        raw = torch.full((1, 130, 2), -4.0, device="cuda")
        raw[:, 3], raw[:, 70], raw[:, 100], raw[:, 129] = -200.0, 30.0, 95.0, -95.0
        got = ssd.prefill_backward(dy, t["x"], raw, t["A"], t["B"], t["C"], t["D"], h0=t["h0"], dh_final=d, dt_raw=True,
                                   dt_max=100.0, check=True)
        for k in NAMES:
            assert torch.isfinite(getattr(got, k)).all(), (io, N, k)
        assert (got.ddt[:, 3] == 0).all() and (got.ddt[:, 70] != 0).any()


@pytest.mark.parametrize("io,N", PATHS)
@pytest.mark.parametrize("scale", [1e-3, 30.0, 3000.0])
def test_weak_and_strong_decay(io, N, scale):
    """From almost none (the sums run over the whole sequence) to a state that one step erases."""
    run_case(make_prefill(2, 300, 4, 64, N, 2, 64, dtype=io, h0_std=0.3, seed=41, dt_scale=scale), tc=on_tc(io, N))


@pytest.mark.parametrize("io,N", PATHS)
@pytest.mark.parametrize("T", [2, 66, 129])
def test_dA_behind_strong_steps(io, N, T):
    """With no state entering and steps that erase it, dA is what the last adjoint sends back through
    one step's decay, many orders below x, dy and the adjoint: what a token adds to the adjoint itself
    must leave no rounding in it."""
    for seed in (236, 391):
        run_case(make_prefill(1, T, 16, 64, N, 8, 64, dtype=io, h0_std=0.0, seed=seed, dt_scale=20.0), seed,
                 tc=on_tc(io, N))


@pytest.mark.parametrize("io,N", PATHS)
def test_no_decay_and_zero_steps(io, N):
    """A = 0 (a plain running sum) and steps of zero length, which leave the state alone."""
    t, dy, d = draw(1, 150, 2, N, 1, io, 42)
    t["A"] = torch.tensor([0.0, -4.0], device="cuda")
    t["dt"][:, 20:90] = 0.0
    t["dt"][:, 149] = 0.0
    got = call(t, dy, d, check=True)
    ref = step_gradients(dy, t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"], t["h0"], d)
    check_grads(got, ref, bounds(t, dy, d, ref, on_tc(io, N)))


@pytest.mark.parametrize("io,N", PATHS)
@pytest.mark.parametrize("h0,dhf", [(False, False), (True, False), (False, True)])
def test_absent_states(io, N, h0, dhf):
    t, dy, d = draw(1, 140, 2, N, 1, io, 43)
    if not h0:
        t["h0"] = None
    d = d if dhf else None
    got = call(t, dy, d, check=True)
    ref = step_gradients(dy, t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"], t["h0"], d)
    check_grads(got, ref, bounds(t, dy, d, ref, on_tc(io, N)))


@pytest.mark.parametrize("shape", [(1, 3000, 1, 128, 1), (1, 5000, 3, 128, 3), (2, 2049, 2, 128, 1), (1, 2500, 76, 128, 2)])
def test_long_sequences(shape):
    """The pass over the states splits sequences into segments: all of them with few heads, and those
    that would begin another wave of blocks with just too many."""
    b, T, H, N, G = shape
    run_case(make_prefill(b, T, H, 64, N, G, 64, dtype="bf16", h0_std=0.3, seed=sum(shape)), tc=True)


@pytest.mark.parametrize("shape", [(1, 1500, 37, 128, 1), (1, 300, 80, 128, 1), (2, 1300, 64, 128, 8)])
def test_heads_over_many_blocks(shape):
    """A group's heads over several blocks in uneven parts; one head a block; more groups than SMs."""
    b, T, H, N, G = shape
    run_case(make_prefill(b, T, H, 64, N, G, 64, dtype="bf16", h0_std=0.3, seed=sum(shape)), tc=True)


@pytest.mark.parametrize("shape", [(1, 700, 37, 64, 1), (1, 60, 80, 128, 1), (2, 640, 64, 64, 8)])
def test_heads_over_many_blocks_fp32(shape):
    b, T, H, N, G = shape
    run_case(make_prefill(b, T, H, 64, N, G, 64, dtype="f32", h0_std=0.3, seed=sum(shape)))


def test_bf16_on_the_fp32_pipes():
    """The hook that routes the prefill to the fp32 pipes routes its gradients too."""
    ssd.debug_force_fma_prefill(True)
    try:
        run_case(make_prefill(2, 200, 4, 64, 128, 2, 64, dtype="bf16", h0_std=0.3, seed=44), tc=False)
    finally:
        ssd.debug_force_fma_prefill(False)


@pytest.mark.parametrize("io,N", PATHS)
@pytest.mark.parametrize("T", [77, 128, 300])
def test_sequences_do_not_touch(io, N, T):
    """What one sequence of a batch holds does not reach the others, whole chunks or not: the
    neighbours of a sequence of NaN and infinities get the bits they get beside an ordinary one."""
    t, dy, d = draw(3, T, 2, N, 1, io, 45)
    clean = call(t, dy, d, check=True)
    bad = {k: v.clone() for k, v in t.items() if isinstance(v, torch.Tensor)}
    bad_dy, bad_d = dy.clone(), d.clone()
    for v, fill in ((bad["x"], float("nan")), (bad["B"], float("inf")), (bad["C"], float("nan")),
                    (bad["h0"], float("nan")), (bad_dy, float("-inf")), (bad_d, float("nan"))):
        v[1] = fill
    bad["dt"][1] = float("nan")
    got = call(bad, bad_dy, bad_d, check=True)
    for k in ("dx", "ddt", "dB", "dC", "dh0"):
        for i in (0, 2):
            assert torch.equal(getattr(got, k)[i], getattr(clean, k)[i]), (k, i)
    assert torch.isnan(got.dx[1]).any()


@pytest.mark.parametrize("io,N", PATHS)
def test_given_outputs_and_repeats(io, N):
    """Outputs and a workspace full of NaN take the same bits, again and again, and nothing behind them
    is written; without dh0 the rest is the same."""
    t, dy, d = draw(2, 333, 6, N, 3, io, 46)
    want = call(t, dy, d)
    need = ssd.prefill_backward_workspace_size(2, 333, 6, 64, N, 3, ssd.SSD_F32 if io == "f32" else ssd.SSD_BF16)
    guard = 64
    for rep in range(3):
        def fill(v):
            flat = torch.full((v.numel() + guard,), float("nan"), dtype=v.dtype, device="cuda")
            return flat, flat[:v.numel()].view(v.shape)
        flats, views = zip(*(fill(getattr(want, k)) for k in NAMES))
        ws = torch.full((need + guard,), 255, dtype=torch.uint8, device="cuda")
        out = call(t, dy, d, grads=ssd.PrefillGrads(**dict(zip(NAMES, views)), ddt_bias=None), workspace=ws, check=True)
        same(out, want)
        assert all(torch.isnan(f[-guard:]).all() for f in flats) and (ws[need:] == 255).all()
    out = call(t, dy, d, want_dh0=False)
    assert out.dh0 is None
    same(out, want, NAMES[:-1])


@pytest.mark.parametrize("io,N", PATHS)
def test_streams_and_graphs(io, N):
    """On a stream of its own; captured, and replayed on new contents; two graphs over one workspace
    replayed in turn."""
    t, dy, d = draw(2, 260, 4, N, 2, io, 47)
    t2, dy2, d2 = draw(2, 260, 4, N, 2, io, 48)
    want, want2 = call(t, dy, d), call(t2, dy2, d2)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = call(t, dy, d)
    s.synchronize()
    same(got, want)
    got = call(t, dy, d, stream=s)
    s.synchronize()
    same(got, want)
    need = ssd.prefill_backward_workspace_size(2, 260, 4, 64, N, 2, ssd.SSD_F32 if io == "f32" else ssd.SSD_BF16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for src in ((t, dy, d), (t2, dy2, d2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(*src, workspace=ws))
        graphs.append(g)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    same(outs[0], want)
    same(outs[1], want2)
    for k in ("x", "dt", "A", "B", "C", "D", "h0"):
        t[k].copy_(t2[k])
    dy.copy_(dy2)
    d.copy_(d2)
    graphs[0].replay()
    torch.cuda.synchronize()
    same(outs[0], want2)


def test_two_calls_at_once():
    """Calls of both paths and a prefill side by side on streams of their own."""
    cases = [draw(2, 1500, 12, N, 1, io, 55) for io, N in PATHS]
    want = [call(*c) for c in cases]
    t = cases[3][0]
    y = ssd.prefill(t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"], h0=t["h0"])[0]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(5)]
    for _ in range(6):
        outs = []
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                outs.append(call(*c))
        with torch.cuda.stream(streams[4]):
            y2 = ssd.prefill(t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"], h0=t["h0"])[0]
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            same(o, w)
        assert torch.equal(y, y2)


def test_temporary_workspace_on_another_stream():
    """A call on a stream of its own without a workspace given: memory taken on the current stream right
    behind the call is not the call's workspace, still in use."""
    s = torch.cuda.Stream()
    for io, N in (("bf16", 128), ("f32", 64)):
        t, dy, d = draw(2, 2048, 8, N, 1, io, 54)
        want = call(t, dy, d, check=True)
        need = ssd.prefill_backward_workspace_size(2, 2048, 8, 64, N, 1, ssd.SSD_F32 if io == "f32" else ssd.SSD_BF16)
        torch.cuda.synchronize()
        for stream in (s, s.cuda_stream):
            outs = []
            for _ in range(4):
                outs.append(call(t, dy, d, stream=stream))
                torch.empty(need, dtype=torch.uint8, device="cuda").fill_(255)
            torch.cuda.synchronize()
            for o in outs:
                same(o, want)


def test_wait_that_runs_out():
    """The starved call gives up after its limit and says so; the next call is right."""
    t, dy, d = draw(1, 300, 2, 128, 1, "bf16", 49)
    want = call(t, dy, d, check=True)
    ws = torch.empty(ssd.prefill_backward_workspace_size(1, 300, 2, 64, 128, 1, ssd.SSD_BF16), dtype=torch.uint8,
                     device="cuda")
    ssd.debug_starve_next_prefill_backward(0.1)
    call(t, dy, d, workspace=ws)
    with pytest.raises(ssd.SSDError) as e:
        ssd.prefill_check(ws)
    assert e.value.status == 4 and "wait site" in str(e.value)  # SSD_ERR_TIMEOUT
    same(call(t, dy, d, workspace=ws, check=True), want)


def test_against_differences():
    """fp32 gradients along a direction in each input against a central difference of the forward
    recurrence in 64 bits.  The difference's own error is of the order step^2 (1e-8 of the third
    derivative) and 1e-16 / step of rounding; the gradients carry the bounds of the fp32 path, a few
    hundred u of sums whose signs differ: 1e-3 of the directional derivative's own terms holds both."""
    b, T, H, N, G = 1, 70, 2, 64, 1
    t, dy, d = draw(b, T, H, N, G, "f32", 50)
    got = call(t, dy, d, check=True)
    names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", D="dD", h0="dh0")
    base = {k: t[k].double() for k in names}
    g = torch.Generator(device="cuda").manual_seed(51)

    def loss(v):
        h, tot = v["h0"], 0.0
        for i in range(T):
            h = torch.exp(v["dt"][:, i] * v["A"])[..., None, None] * h + \
                (v["dt"][:, i, :, None] * v["x"][:, i])[..., None] * v["B"][:, i, :, None, :]
            y = (h * v["C"][:, i, :, None, :]).sum(-1) + v["D"][:, None] * v["x"][:, i]
            tot = tot + (y * dy[:, i].double()).sum()
        return (tot + (h * d.double()).sum()).item()

    for k, gk in names.items():
        u = torch.randn(base[k].shape, generator=g, device="cuda", dtype=torch.float64)
        if k == "dt":
            u = u * base[k]
        step = 1e-4
        diff = (loss(dict(base, **{k: base[k] + step * u})) - loss(dict(base, **{k: base[k] - step * u}))) / (2 * step)
        terms = getattr(got, gk).double() * u
        assert abs(terms.sum().item() - diff) <= 1e-3 * terms.norm().item() + 1e-6 * abs(diff), k


def test_offsets_beyond_32_bits():
    """More than 2^31 elements of x: the last sequences get what they get in a call of their own."""
    for io, N, b, T, H in ((torch.bfloat16, 128, 110, 4096, 80), (torch.float32, 64, 28, 16384, 80)):
        g = torch.Generator(device="cuda").manual_seed(52)
        x = torch.empty(b, T, H, 64, dtype=io, device="cuda").normal_(generator=g)
        assert x.numel() > 2 ** 31
        dy = torch.empty_like(x).normal_(generator=g)
        B, C = (torch.empty(b, T, 1, N, dtype=io, device="cuda").normal_(generator=g) for _ in range(2))
        dt = torch.empty(b, T, H, device="cuda").uniform_(0.001, 0.1, generator=g)
        A, D = -torch.empty(H, device="cuda").uniform_(1, 16, generator=g), torch.ones(H, device="cuda")
        got = ssd.prefill_backward(dy, x, dt, A, B, C, D, check=True)
        n = 2
        ref = ssd.prefill_backward(dy[-n:], x[-n:], dt[-n:], A, B[-n:], C[-n:], D, check=True)
        for k in ("dx", "ddt", "dB", "dC", "dh0"):
            a, r = getattr(got, k)[-n:].double(), getattr(ref, k).double()
            # two runs within the path's bound of each other: 16-bit results by a step of bf16
            assert (a - r).norm() <= (2.0 ** -7 if io == torch.bfloat16 else 1e-5) * r.norm(), k
        del x, dy, B, C, dt, got, ref, a, r
        torch.cuda.empty_cache()


def test_block_forward_and_backward():
    """The operators as a block uses them: residual norm, the SSD with the raw step, gated norm, and
    back; against the composition differentiated in 64 bits.  Each stage's error is its bound, at most
    600 u of sums of magnitudes; those are within 16 times the results' norms (sums of 64 to 128 terms
    of random sign), and three stages of them stay below 3e-3 of each gradient's norm."""
    b, T, H, N, G = 2, 190, 4, 64, 2
    Dm, di = 256, H * 64
    g = torch.Generator(device="cuda").manual_seed(60)
    r = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std
    leaf = dict(u=r(b, T, Dm), res=r(b, T, Dm), w1=1 + 0.1 * r(Dm), z=r(b, T, di), w2=1 + 0.1 * r(di),
                raw=r(b, T, H, std=0.5) - 3, bias=r(H, std=0.3), A=-(0.5 + r(H).abs()), D=r(H), B=r(b, T, G, N),
                C=r(b, T, G, N), h0=r(b, H, 64, N, std=0.3))
    dout, dres_out, dhf = r(b, T, di), r(b, T, Dm), r(b, H, 64, N)
    assert Dm == di
    # forward
    a, r1 = ssd.residual_norm(leaf["u"], leaf["w1"], leaf["res"], scale=0.5)
    x = a.view(b, T, H, 64)
    y, hT = ssd.prefill(x, leaf["raw"], leaf["A"], leaf["B"], leaf["C"], leaf["D"], chunk=64, h0=leaf["h0"], dt_raw=True,
                        dt_bias=leaf["bias"])
    y = y.reshape(b, T, di)
    out = ssd.gated_norm(y, leaf["z"], leaf["w2"], groups=G)
    # backward
    dy, dz, dw2 = ssd.gated_norm_backward(dout, y, leaf["z"], leaf["w2"], groups=G)
    gr = ssd.prefill_backward(dy.view(b, T, H, 64), x, leaf["raw"], leaf["A"], leaf["B"], leaf["C"], leaf["D"],
                              h0=leaf["h0"], dh_final=dhf, dt_raw=True, dt_bias=leaf["bias"])
    du, dres, dw1 = ssd.residual_norm_backward(gr.dx.view(b, T, Dm), r1, leaf["w1"], dres_out, scale=0.5)
    got = dict(u=du, res=dres, w1=dw1, z=dz, w2=dw2, raw=gr.ddt, bias=gr.ddt_bias, A=gr.dA, D=gr.dD, B=gr.dB, C=gr.dC,
               h0=gr.dh0)
    # the same in 64 bits
    v = {k: t.double().cpu().requires_grad_() for k, t in leaf.items()}

    def norm(t, w, groups=1):
        s = t.reshape(b, T, groups, -1)
        return (s * (s.pow(2).mean(-1, keepdim=True) + 1e-5).rsqrt()).reshape(t.shape) * w

    rr = v["res"] + 0.5 * v["u"]
    xr = norm(rr, v["w1"]).view(b, T, H, 64)
    dt = torch.nn.functional.softplus(v["raw"] + v["bias"])
    h, ys = v["h0"], []
    Bh, Ch = (v[k].repeat_interleave(H // G, 2) for k in "BC")
    for i in range(T):
        h = torch.exp(dt[:, i] * v["A"])[..., None, None] * h + (dt[:, i, :, None] * xr[:, i])[..., None] * Bh[:, i, :, None, :]
        ys.append((h * Ch[:, i, :, None, :]).sum(-1) + v["D"][:, None] * xr[:, i])
    yr = torch.stack(ys, 1).reshape(b, T, di)
    orf = norm(yr * torch.nn.functional.silu(v["z"]), v["w2"], G)
    loss = (orf * dout.double().cpu()).sum() + (rr * dres_out.double().cpu()).sum() + (h * dhf.double().cpu()).sum()
    loss.backward()

    def near(a, ref, k):
        assert (a.double().cpu() - ref).norm() <= 3e-3 * ref.norm(), k

    near(out, orf.detach(), "out")
    near(hT, h.detach(), "h_final")
    for k in leaf:
        near(got[k], v[k].grad, k)


def test_binding_refusals():
    t, dy, d = draw(1, 40, 2, 64, 1, "f32", 53)
    ok = lambda **kw: call(t, dy, d, **kw)
    good = ok()
    with pytest.raises((ValueError, TypeError)):
        call(t, dy.bfloat16(), d)
    with pytest.raises((ValueError, TypeError)):
        call(t, dy[:, :39], d)
    with pytest.raises((ValueError, TypeError)):
        call(t, dy.transpose(1, 2).contiguous().transpose(1, 2), d)
    with pytest.raises((ValueError, TypeError)):
        call(t, dy, d.bfloat16())
    with pytest.raises((ValueError, TypeError)):
        call(t, dy.cpu(), d)
    with pytest.raises(ValueError):
        ok(dt_bias=torch.zeros(2, device="cuda"))
    with pytest.raises((ValueError, TypeError)):
        ok(grads=good._replace(dx=good.dx.bfloat16()))
    with pytest.raises(ValueError):
        ok(grads=good._replace(ddt_bias=torch.zeros(2, device="cuda")))
    with pytest.raises(ssd.SSDError):
        ok(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ssd.SSDError):
        ok(grads=good._replace(dx=t["x"]))
    with pytest.raises(ssd.SSDError):
        ok(dt_raw=True, dt_min=1.0, dt_max=0.5)
