"""Calls on a stream given by name: neither the temporary workspace nor the results may be memory that
work queued on the current stream still uses, before the call or behind it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ssd = pytest.importorskip("state_space_model_04_b200")

BF = torch.bfloat16
WAIT = 40_000_000  # clock ticks, about 20 ms: longer than it takes to queue all that follows


def rnd(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def operators():
    """name, call(stream), the bytes of the workspace it allocates."""
    g = torch.Generator(device="cuda").manual_seed(5)
    b, T, H, N = 2, 1024, 8, 128
    calls = []
    for io, n in ((BF, N), (torch.float32, 64)):
        x, dy = rnd(g, b, T, H, 64, dtype=io), rnd(g, b, T, H, 64, dtype=io)
        B, C = rnd(g, b, T, 1, n, dtype=io), rnd(g, b, T, 1, n, dtype=io)
        dt, A, D = 0.01 + 0.05 * torch.rand(b, T, H, generator=g, device="cuda"), -torch.ones(H, device="cuda"), rnd(g, H)
        code = ssd.SSD_BF16 if io == BF else ssd.SSD_F32
        calls.append(("prefill", lambda s, a=(x, dt, A, B, C, D): ssd.prefill(*a, stream=s),
                      ssd.prefill_workspace_size(b, T, H, 64, n, 1, 256, code)))
        calls.append(("prefill_backward", lambda s, a=(dy, x, dt, A, B, C, D): ssd.prefill_backward(*a, stream=s),
                      ssd.prefill_backward_workspace_size(b, T, H, 64, n, 1, code)))
        if io == BF:
            calls.append(("prefill_local_state", lambda s, a=(x, dt, A, B): ssd.prefill_local_state(*a, stream=s),
                          int(ssd.lib().ssd_prefill_local_state_workspace_size(b, T, H, 64, n, 1, code))))
    rows, W = 12000, 2560
    m, r, w = rnd(g, rows, W, dtype=BF), rnd(g, rows, W), 1 + 0.1 * rnd(g, W)
    ws = ssd.norm_backward_workspace_size(rows, W)
    calls.append(("residual_norm", lambda s: ssd.residual_norm(m, w, r, stream=s), 0))
    calls.append(("residual_norm_backward", lambda s: ssd.residual_norm_backward(m, r, w, stream=s), ws))
    calls.append(("gated_norm", lambda s: (ssd.gated_norm(m, m, w, stream=s),), 0))
    calls.append(("gated_norm_backward", lambda s: ssd.gated_norm_backward(m, m, m, w, stream=s), ws))
    return calls


def same(got, want):
    for a, b in zip(got, want):
        assert (a is None and b is None) or torch.equal(a, b)


def handles(s):
    return s, s.cuda_stream


@pytest.mark.parametrize("which", range(9))
def test_memory_just_freed_on_the_current_stream(which):
    """Blocks of the sizes the call needs, freed with work on them still queued: that work and the call
    keep their values."""
    name, call, ws = operators()[which]
    want = call(None)
    torch.cuda.synchronize()
    sizes = [n for n in [ws] + [t.numel() * t.element_size() for t in want if t is not None] if n]
    for s in handles(torch.cuda.Stream()):
        blocks = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda._sleep(WAIT)
        kept = [b.clone() for b in blocks]
        for b in blocks:
            b.fill_(255)
        del blocks, b
        got = call(s)
        torch.cuda.synchronize()
        same(got, want)
        assert all((k == 7).all() for k in kept), name
        del got, kept


@pytest.mark.parametrize("which", range(9))
def test_results_dropped_while_the_call_runs(which):
    """Results that nobody keeps are written by the call long after their blocks were freed: what the
    current stream takes then is not theirs."""
    name, call, ws = operators()[which]
    want = call(None)
    sizes = [t.numel() * t.element_size() for t in want if t is not None] + ([ws] if ws else [])
    del want
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in handles(s):
        with torch.cuda.stream(s):
            torch.cuda._sleep(WAIT)
        call(stream)
        mine = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda.synchronize()
        assert all((m == 7).all() for m in mine), name


@pytest.mark.parametrize("which", range(9))
def test_results_read_and_dropped_on_the_current_stream(which):
    """Results read by work queued on the current stream and dropped: a call that follows on the given
    stream does not get their memory before that work is done."""
    name, call, _ = operators()[which]
    want = call(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = call(s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(WAIT)
    kept = [None if t is None else t.clone() for t in got]
    sizes = [t.numel() * t.element_size() for t in want if t is not None]
    del got
    with torch.cuda.stream(s):
        for n in sizes:
            torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    same(kept, want)


def test_default_stream_by_its_handle():
    """Handle 0 is the default stream, wherever the call is made from."""
    for name, call, _ in operators():
        want = call(None)
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.Stream()):
            got = call(0)
        torch.cuda.synchronize()
        same(got, want)


def test_captured_on_a_stream_that_joins():
    """A call on a second stream of a capture, replayed."""
    for name, call, _ in operators():
        want = call(None)
        torch.cuda.synchronize()
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            side.wait_stream(torch.cuda.current_stream())
            got = call(side)
            torch.cuda.current_stream().wait_stream(side)
        for t in got:
            if t is not None:
                t.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        same(got, want)
        del graph


def test_the_current_stream_stays():
    """Through a call on another stream, one that is refused among them."""
    x, w = torch.ones(4, 64, device="cuda"), torch.ones(64, device="cuda")
    for here in (torch.cuda.default_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(here):
            for s in handles(torch.cuda.Stream()):
                ssd.residual_norm(x, w, stream=s)
                assert torch.cuda.current_stream() == here
                with pytest.raises(ssd.SSDError):
                    ssd.residual_norm(x, w, eps=-1.0, stream=s)
                assert torch.cuda.current_stream() == here
