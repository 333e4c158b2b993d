"""Host-side checks of the training losses' limits that no single argument shows: nothing is launched."""
import ctypes

import pytest

from precision_moe_expert_amd import binding

FAKE, BIG = 1 << 20, 1 << 60


def _calls(hd):
    L, h = binding.lib(), ctypes.byref(hd)
    return dict(loss=L.moe_lm_head_loss(h, *[FAKE] * 6, 0, None),
                distill=L.moe_lm_head_distill(h, 4, 1.0, *[FAKE] * 8, 0, None),
                loss_bwd=L.moe_lm_head_loss_backward(h, *[FAKE] * 9, 0, None),
                distill_bwd=L.moe_lm_head_distill_backward(h, 4, 1.0, *[FAKE] * 10, 0, None))


@pytest.mark.parametrize("T,V", [(1 << 20, 1 << 20), (1 << 20, 1 << 19), ((1 << 20) - 3, (1 << 19) - 1),
                                 (1 << 19, 1 << 20)])
def test_more_tiles_than_a_launch_holds(T, V):
    """The forward is refused before anything is enqueued; the gradient goes by pieces of the vocabulary."""
    hd = binding.MoeLmHead(T, 64, V, 1e-6, 1.0, 0, 0)
    got = _calls(hd)
    assert got["loss"] == got["distill"] == binding.MOE_ERR_UNSUPPORTED
    assert got["loss_bwd"] == got["distill_bwd"] == binding.MOE_ERR_WORKSPACE_TOO_SMALL
    size = binding.lib().moe_lm_head_loss_workspace_bytes
    assert size(ctypes.byref(hd), 0, 0) == 0 and size(ctypes.byref(hd), 4, 0) == 0
    assert size(ctypes.byref(hd), 0, 1) > 0


@pytest.mark.parametrize("T,H,V", [(1 << 20, 8, 1 << 18), (1 << 18, 64, 1 << 20), (1 << 20, 32768, 100),
                                   (1, 32768, 1 << 20), (1 << 20, 4096, 1 << 18)])
def test_largest_calls_that_are_taken(T, H, V):
    hd = binding.MoeLmHead(T, H, V, 1e-6, 1.0, 0, 0)
    assert set(_calls(hd).values()) == {binding.MOE_ERR_WORKSPACE_TOO_SMALL}
