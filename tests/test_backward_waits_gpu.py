"""The tensor-core gradients with one role of the main pass's warps held back at every item: each of
the others has to wait for it wherever it needs it, so the results are the same bits.  A role that
goes by a barrier's parity without knowing the phase before complete runs into one that lags."""
import pytest
import torch

from tests.test_backward_edges_gpu import call, draw, same

pytestmark = pytest.mark.gpu

ssd = pytest.importorskip("state_space_model_04_b200")

ROLES = ["pair", "row", "issue", "ddt", "store", "load", "dot"]


# several items a group in one CTA; groups cut between CTAs, several groups a CTA; one item a group
@pytest.mark.parametrize("shape", [(2, 1100, 24, 3), (2, 1300, 64, 8), (1, 1500, 37, 1), (1, 900, 12, 12)])
@pytest.mark.parametrize("role", range(len(ROLES)), ids=ROLES)
def test_a_role_that_lags(shape, role):
    b, T, H, G = shape
    t, dy, d = draw(b, T, H, 128, G, "bf16", 71)
    want = call(t, dy, d, check=True)
    for _ in range(2):
        ssd.debug_lag_next_prefill_backward(role)
        same(call(t, dy, d, check=True), want)
    same(call(t, dy, d, check=True), want)  # the hook is for one call
