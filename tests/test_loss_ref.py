"""The 64-bit loss references: their gradients against central differences of
their losses, and the cases whose value is known."""
import math

import pytest
import torch

from tests import loss_ref as lr


def _diff(f, x, step=1e-5):
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        d = torch.zeros(x.numel(), dtype=x.dtype)
        d[i] = step
        d = d.view_as(x)
        g.view(-1)[i] = (f(x + d) - f(x - d)) / (2 * step)
    return g


@pytest.mark.parametrize("eps,scale", [(1e-6, 1.0), (0.0, 0.5), (0.3, 2.0)])
@pytest.mark.parametrize("kind", ["ce", "distill"])
def test_head_gradients_match_differences(kind, eps, scale):
    torch.manual_seed(5)
    T, H, V = 4, 8, 11
    h, w = torch.randn(T, H, dtype=torch.float64), torch.randn(V, H, dtype=torch.float64)
    g = torch.randn(T, dtype=torch.float64)
    if kind == "ce":
        y = torch.tensor([3, -1, 10, 0])
        loss = lambda a, b: lr.ce_ref(a, b, y, eps, scale).loss()[1]  # noqa: E731
        ref = lr.ce_ref(h, w, y, eps, scale)
    else:
        ids = torch.tensor([[1, 1, 4], [-1, -1, -1], [0, 10, -1], [7, 2, 7]])
        tl = torch.randn(T, 3, dtype=torch.float64)
        tl[3, 1] = -math.inf

        def loss(a, b):
            r, have, q = lr.distill_ref(a, b, ids, tl, 0.7, eps, scale)
            return lr.distill_loss(r, ids, have, q)[1]
        ref = lr.distill_ref(h, w, ids, tl, 0.7, eps, scale)[0]
    d_h, _, d_w, _ = ref.grads(g, True)
    assert torch.allclose(d_h, _diff(lambda a: (loss(a, w) * g).sum(), h), atol=1e-7)
    assert torch.allclose(d_w, _diff(lambda b: (loss(h, b) * g).sum(), w), atol=1e-7)


def test_balance_gradient_matches_differences():
    torch.manual_seed(6)
    T, E, k = 9, 5, 2
    x = torch.randn(T, E, dtype=torch.float64)
    ids = torch.topk(x, k, 1).indices.int()
    mask = torch.tensor([1, 1, 0, 1, 1, 1, 0, 1, 1], dtype=torch.uint8)
    off, g = [1, 4, 4, 8], torch.randn(3, dtype=torch.float64)
    got = lr.balance_ref(x, ids, k, mask, off, g)["d_logits"]
    f = lambda v: (lr.balance_ref(v, ids, k, mask, off)["loss"] * g).sum()  # noqa: E731
    assert torch.allclose(got, _diff(f, x), atol=1e-8)


def test_known_values():
    # a head of equal rows: every id has probability 1/V
    h, w = torch.randn(3, 8), torch.ones(7, 8)
    lse, loss, _, _ = lr.ce_ref(h, w, torch.tensor([0, 6, 3])).loss()
    assert torch.allclose(loss, torch.full((3,), math.log(7.0), dtype=torch.float64))
    # a teacher equal to the student over the whole vocabulary: no divergence, no gradient
    ids = torch.arange(7).expand(3, 7).int()
    w = torch.randn(7, 8)
    r, have, q = lr.distill_ref(h, w, ids, (lr.ce_ref(h, w, torch.zeros(3)).logits).float())
    assert lr.distill_loss(r, ids, have, q)[1].abs().max() < 1e-6
    assert r.grads(torch.ones(3), False)[0].abs().max() < 1e-5
    # uniform routing: loss 1
    ids = torch.tensor([[0, 1], [2, 3]]).int()
    assert abs(lr.balance_ref(torch.zeros(2, 4), ids, 2)["loss"].item() - 1.0) < 1e-12
