"""Norms of the gradients' errors, against 64 bits, where a head that fits its
data makes large parts cancel: targets drawn from the head's own probabilities,
rows of h with a common direction, one frequent id.

Bound: what is rounded to bf16 is the result (its rounding is known, 1.25 times
it allows for fp32 sums) and G's entries other than the target's, each off by at
most 2^-8 of itself, evenly spread, so by 2^-8 / sqrt(3) in the mean square: the
norm they leave in d_w is that times sqrt(sum G^2 |h|^2), in d_h times
sqrt(sum G^2 |W|^2).  The norm over a whole gradient is close to that mean; that
over one row of d_w has most of it in one direction and may be a few times it."""
import math

import pytest
import torch

import precision_moe_expert_amd as moe
from tests import loss_ref as lr

pytestmark = pytest.mark.gpu

STEP = lr.BF16 / math.sqrt(3.0)


def _fitted(T, H, V, seed, ignored=0.1):
    """(h, w, y, d_loss): id V // 3 takes about a fifth of the targets."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    way = torch.randn(H, generator=g, device="cuda")
    h = (torch.randn(T, H, generator=g, device="cuda") + 1.5 * way).bfloat16()
    w = torch.randn(V, H, generator=g, device="cuda") / math.sqrt(H)
    z = h.double() / torch.sqrt((h.double() ** 2).mean(1, keepdim=True) + 1e-6)
    w[V // 3] = 0.0
    lse = torch.logsumexp(z @ w.double().t(), 1).mean()
    w[V // 3] = way * ((lse + math.log(0.25)) / (z @ way.double()).mean()).float()
    w = w.bfloat16()
    p = torch.softmax(z @ w.double().t(), 1)
    y = torch.multinomial(p, 1, generator=g)[:, 0].int()
    y = torch.where(torch.rand(T, generator=g, device="cuda") < ignored, -1, y).int()
    return h, w, y, torch.full((T,), 1.0 / T, device="cuda"), g


def _rounding(x):
    return torch.linalg.norm(x.bfloat16().double() - x)


@pytest.mark.parametrize("T,H,V", [(4096, 256, 512), (200, 256, 700), (900, 520, 257), (3000, 512, 5003),
                                   (8200, 512, 2000), (1200, 1024, 70001)])
def test_fitted_head(torch_gpu, T, H, V):
    h, w, y, dl, _ = _fitted(T, H, V, T + V)
    ref = lr.ce_ref(h, w, y)
    loss, lse = moe.lm_head_loss(h, w, y)
    gh, gw = moe.lm_head_loss_backward(h, w, y, loss, lse, dl, weight_grad=True)
    d_h, _, d_w, _ = ref.grads(dl, True)
    G = (ref.r * dl[ref.rows].double())[:, None] * torch.where(ref.q > 0, 0.0, ref.p)
    size_h = (G ** 2).sum(0) @ (ref.w ** 2).sum(1)
    size_w = (G ** 2).t() @ (ref.x ** 2).sum(1)  # of each row
    norm = torch.linalg.norm
    assert norm(gh.double() - d_h) <= 1.25 * _rounding(d_h) + STEP * size_h.sqrt()
    assert norm(gw.double() - d_w) <= 1.25 * _rounding(d_w) + STEP * size_w.sum().sqrt()
    f = V // 3
    assert norm(gw[f].double() - d_w[f]) <= 1.25 * _rounding(d_w[f]) + 3 * STEP * size_w[f].sqrt()


# (T, H, V, K) where the entries at the slots' ids are few for the vocabulary, and where they are many and stay rounded
SLOTS = [(1500, 512, 32000, 33), (200, 1024, 32000, 64), (2500, 256, 4500, 5), (30, 264, 1000, 16), (70, 512, 20001, 128),
         (1500, 512, 8000, 33), (600, 256, 1000, 64)]


@pytest.mark.parametrize("T,H,V,K", SLOTS)
def test_fitted_student(torch_gpu, T, H, V, K):
    """A teacher close to the student: its ids are the student's best ones, so that their entries of G are most of it,
    and p and q cancel in part."""
    h, w, _, dl, g = _fitted(T, H, V, T + K)
    z = h.double() / torch.sqrt((h.double() ** 2).mean(1, keepdim=True) + 1e-6)
    top = (2.0 * (z @ w.double().t())).float()
    top = (top + torch.randn(top.shape, generator=g, device="cuda")).topk(K, 1)
    ids, tl = top.indices.int(), top.values
    ids[::9] = -1
    ref, have, q = lr.distill_ref(h, w, ids, tl, 0.5)
    loss, lse, logp = moe.lm_head_distill(h, w, ids, tl, teacher_scale=0.5)
    gh, gw = moe.lm_head_distill_backward(h, w, ids, tl, lse, logp, dl, weight_grad=True, teacher_scale=0.5)
    d_h, _, d_w, _ = ref.grads(dl, True)
    G = (ref.r * dl[ref.rows].double())[:, None] * (ref.p - ref.q)
    if K * 900 <= V or T * K <= max(V // 2, 1024):
        G = torch.where(ref.q > 0, 0.0, G)
    size_h = (G ** 2).sum(0) @ (ref.w ** 2).sum(1)
    size_w = (G ** 2).sum(1) @ (ref.x ** 2).sum(1)
    norm = torch.linalg.norm
    assert norm(gh.double() - d_h) <= 1.25 * _rounding(d_h) + STEP * size_h.sqrt()
    assert norm(gw.double() - d_w) <= 1.25 * _rounding(d_w) + STEP * size_w.sqrt()
