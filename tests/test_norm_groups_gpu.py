"""Groups on both sides of every length where the gated norm takes another kernel: a warp a group with two
to four vectors a thread, or a block.  Bounds as in test_norm_gpu."""
import pytest
import torch

from tests.test_norm_gpu import BF, F32, close, gated_backward_ref, gated_ref, gen, rand

pytestmark = pytest.mark.gpu

ssd = pytest.importorskip("state_space_model_04_b200")


@pytest.mark.parametrize("L", [256, 264, 512, 520, 768, 776, 1024, 1032])
@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("rows,groups", [(3, 2), (411, 5)])
def test_group_lengths(L, io, first, rows, groups):
    g, D = gen(L + rows), L * groups
    y, z, dout = rand(g, rows, D, dtype=io), rand(g, rows, D, std=2.0, dtype=io), rand(g, rows, D, dtype=io)
    w = 1 + 0.1 * rand(g, D)
    out = ssd.gated_norm(y, z, w, groups=groups, norm_before_gate=first)
    ref, mag = gated_ref(y, z, w, groups, 1e-5, first)
    close(out, ref, mag, "out")
    ws = torch.full((ssd.norm_backward_workspace_size(rows, D, groups) + 64,), 255, dtype=torch.uint8, device="cuda")
    dy, dz, dw = ssd.gated_norm_backward(dout, y, z, w, groups=groups, norm_before_gate=first, workspace=ws)
    assert (ws[-64:] == 255).all()
    ry, my, rz, mz, rw, mw = gated_backward_ref(dout, y, z, w, groups, 1e-5, first)
    close(dy, ry, my, "dy")
    close(dz, rz, mz, "dz")
    close(dw, rw, mw, "dweight", 144 + rows / 64)


def test_sizes_beyond_an_int_are_refused():
    """2^32 + 1 groups are not one group, nor rows of 2^32 + 64 elements rows of 64."""
    x, w = torch.ones(4, 64, device="cuda"), torch.ones(64, device="cuda")
    for groups in (2**32 + 1, 2**31, 0, -1):
        with pytest.raises((ValueError, ssd.SSDError)):
            ssd.gated_norm(x, x, w, groups=groups)
        with pytest.raises((ValueError, ssd.SSDError)):
            ssd.gated_norm_backward(x, x, x, w, groups=groups)
    wide = torch.empty(0, 2**32 + 64, device="cuda")
    with pytest.raises(ValueError):
        ssd.residual_norm(wide, w)
    with pytest.raises(ValueError):
        ssd.gated_norm(wide, wide, w)
