"""Calls of the training losses at the ends of what their documentation allows."""
import math

import pytest
import torch

import precision_moe_expert_amd as moe
from tests import loss_ref as lr

pytestmark = pytest.mark.gpu

F32 = lr.F32


@pytest.mark.parametrize("T,E,k", [(70, 48, 3), (70, 45, 3), (1100, 200, 2), (90, 1000, 4)])
def test_balance_far_logits(torch_gpu, T, E, k):
    """Whole rows at a mask's value (1e9 and beyond, either sign): equal probabilities where they are equal, the
    largest alone where they differ by their own spacing."""
    torch.manual_seed(T + E)
    logits = torch.randn(T, E)
    for i, far in enumerate((-1e9, -1e10, -1e30, 1e10, 3e9, -65537.0, 1e38, -2.5e9)):
        logits[i] = far
        logits[8 + i] = far * (1 + torch.rand(E) * 1e-3)
        logits[16 + i, E // 2:] = far  # the others stand beside it
    ids = torch.topk(logits, k, 1).indices.int()
    layer = moe.make_layer(T, 256, 128, E, k, moe.FMT_INT4)
    g = torch.tensor([0.7])
    ref = lr.balance_ref(logits, ids, k, d_loss=g)
    assert torch.isfinite(ref["probs"]).all() and abs(float(ref["probs"].sum()) - 1) < 1e-9
    loss, counts, tokens, probs = moe.balance_loss(layer, logits.cuda(), ids.cuda())
    assert torch.equal(counts.cpu().long(), ref["counts"])
    # a row's p are off by its sum's E/16 + 16 steps; a difference of logits below 128 in magnitude by 2^-17, one step
    # of exp's argument there, above that p is 0
    step = 128 * F32
    assert torch.allclose(probs.cpu().double(), ref["probs"], rtol=(T + E + 64) * F32 + step, atol=0)
    assert torch.allclose(loss.cpu().double(), ref["loss"], rtol=(T + E + 64) * F32 + step, atol=0)
    d = moe.balance_loss_backward(layer, logits.cuda(), counts, tokens, g.cuda())
    a = 0.7 * E / (k * T * T) * ref["counts"][0].double()
    assert ((d.cpu().double() - ref["d_logits"]).abs() <= a.max() * ((E + 64) * F32 + 2 * step)).all()
