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


@pytest.mark.parametrize("scale,eps", [(1e9, 1e-6), (3e12, 1e-6), (1e25, 1e-6), (2.0 ** 31, 0.0)])
@pytest.mark.parametrize("T,H,V", [(3, 64, 5000), (70, 136, 301), (300, 64, 500), (1100, 64, 9001), (9, 4096, 300)])
def test_head_far_logits(torch_gpu, T, H, V, scale, eps):
    """A temperature near 0: logits of 1e9 and beyond.  The losses are within the rounding of such logits; what the
    gradients weigh, p - [target], stays within -1 and 1 and the gradients finite."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T + V)
    h = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w = (torch.randn(V, H, generator=g, device="cuda") / math.sqrt(H)).bfloat16()
    y = torch.randint(0, V, (T,), generator=g, device="cuda").int()
    y[::3] = (lr.ce_ref(h, w, y, eps, 1.0).logits[::3]).argmax(1).int()  # p = 1 there
    ids = torch.stack([y, (y + 7) % V], 1).int().contiguous()
    tl = torch.randn(T, 2, generator=g, device="cuda")
    ref = lr.ce_ref(h, w, y, eps, scale)
    lse, want, b_lse, b_loss = ref.loss()
    loss, got_lse = moe.lm_head_loss(h, w, y, norm_eps=eps, logit_scale=scale)
    assert ((got_lse.double() - lse).abs() <= b_lse).all() and ((loss.double() - want).abs() <= b_loss).all()
    assert (loss >= 0).all()
    kl, klse, logp = moe.lm_head_distill(h, w, ids, tl, norm_eps=eps, logit_scale=scale)
    assert ((klse.double() - lse).abs() <= b_lse).all() and kl.isfinite().all() and (logp <= 0).all()
    dl = torch.randn(T, generator=g, device="cuda")
    grads = moe.lm_head_loss_backward(h, w, y, loss, lse.float(), dl, weight_grad=True, norm_eps=eps,
                                      logit_scale=scale)
    grads += moe.lm_head_distill_backward(h, w, ids, tl, klse, logp, dl, weight_grad=True, norm_eps=eps,
                                          logit_scale=scale)
    size = (scale * ref.r * dl.double().abs()).max()
    for d, rows in zip(grads, (ref.w, ref.x, ref.w, ref.x)):
        # at most every |entry| 1 of G's row or column, u and its part along h
        assert d.isfinite().all() and d.double().abs().max() <= 4 * size * rows.abs().sum(0).max() + 4 * size * rows.abs().sum()


@pytest.mark.parametrize("T,H,V", [(4, 64, 40), (300, 64, 500), (9, 4096, 300)])
def test_confident_losses_are_not_negative(torch_gpu, T, H, V):
    """Rows that are their target's row of W many times over: lse and the target's logit are equal but for rounding."""
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    w = torch.randn(V, H, generator=g, device="cuda").bfloat16()
    y = torch.randint(0, V, (T,), generator=g, device="cuda").int()
    h = w[y.long()].contiguous()
    loss, lse = moe.lm_head_loss(h, w, y, norm_eps=0.0, logit_scale=7.3)
    assert (loss >= 0).all() and (loss <= lse.abs() * 8 * F32).all()
    logp = moe.lm_head_distill(h, w, y[:, None].contiguous(), torch.zeros(T, 1, device="cuda"), norm_eps=0.0,
                               logit_scale=7.3)[2]
    assert (logp <= 0).all()


def test_unaligned_views_are_named(torch_gpu):
    """The labels of a shifted sequence start between 16-byte addresses: the refusal says which argument, and a clone
    is taken."""
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    h = torch.randn(9, 64, generator=g, device="cuda").bfloat16()
    w = torch.randn(100, 64, generator=g, device="cuda").bfloat16()
    ids = torch.randint(0, 100, (9,), generator=g, device="cuda").int()
    with pytest.raises(ValueError, match="targets.*aligned"):
        moe.lm_head_loss(h[:-1], w, ids[1:])
    loss, lse = moe.lm_head_loss(h[:-1], w, ids[1:].clone())
    ref = lr.ce_ref(h[:-1], w, ids[1:])
    assert ((loss.double() - ref.loss()[1]).abs() <= ref.loss()[3]).all()
    dl = torch.ones(9, device="cuda")
    with pytest.raises(ValueError, match="d_loss.*aligned"):
        moe.lm_head_loss_backward(h[:-1], w, ids[1:].clone(), loss, lse, dl[1:])
    with pytest.raises(ValueError, match="^h: .*aligned"):
        moe.lm_head_loss(torch.empty(9 * 64 + 4, device="cuda").bfloat16()[4:].view(9, 64), w, ids)
    layer = moe.make_layer(8, 256, 128, 16, 2, moe.FMT_INT4)
    lg, top = torch.randn(8, 16, device="cuda"), torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    mask = torch.ones(9, dtype=torch.bool, device="cuda")
    with pytest.raises(ValueError, match="token_mask.*aligned"):
        moe.balance_loss(layer, lg, top, token_mask=mask[1:])


@pytest.mark.parametrize("T,H,V", [(3, 64, 5000), (70, 136, 301), (300, 64, 500), (1100, 64, 901), (9, 4096, 300)])
def test_lowest_ids(torch_gpu, T, H, V):
    """The type's lowest and highest ids mark tokens and slots that are not there."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    h = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w = (torch.randn(V, H, generator=g, device="cuda") / math.sqrt(H)).bfloat16()
    y = torch.randint(0, V, (T,), generator=g, device="cuda").int()
    y[1::2] = -2 ** 31
    ids = torch.stack([y, torch.full_like(y, -2 ** 31), torch.full_like(y, 2 ** 31 - 1), y], 1).contiguous()
    tl = torch.randn(T, 4, generator=g, device="cuda")
    dl = torch.randn(T, generator=g, device="cuda")
    loss, lse = moe.lm_head_loss(h, w, y)
    kl, klse, logp = moe.lm_head_distill(h, w, ids, tl)
    ref = lr.ce_ref(h, w, y)
    assert ((lse.double() - ref.loss()[0]).abs() <= ref.loss()[2]).all()
    assert ((loss.double() - ref.loss()[1]).abs() <= ref.loss()[3]).all()
    assert ((klse.double() - ref.loss()[0]).abs() <= ref.loss()[2]).all() and (logp[:, 1:3] == 0).all()
    d_h, b_h, d_w, b_w = ref.grads(dl, True)  # a teacher whose slots are all the one id is that id
    for gh, gw in (moe.lm_head_loss_backward(h, w, y, loss, lse, dl, weight_grad=True),
                   moe.lm_head_distill_backward(h, w, ids, tl, klse, logp, dl, weight_grad=True)):
        assert ((gh.double() - d_h).abs() <= b_h * 1.01 + 1e-30).all()
        assert ((gw.double() - d_w).abs() <= b_w * 1.01 + 1e-30).all()


@pytest.mark.parametrize("T,H", [(1, 64), (300, 72), (5, 4096)])
def test_one_id_costs_nothing(torch_gpu, T, H):
    """A vocabulary of one id: loss +0 (not -0) and no gradient."""
    h = torch.randn(T, H, device="cuda").bfloat16()
    w = torch.randn(1, H, device="cuda").bfloat16()
    y = torch.zeros(T, dtype=torch.int32, device="cuda")
    loss, lse = moe.lm_head_loss(h, w, y)
    # lse is l itself but for the rounding of l log2 e and back
    assert not torch.signbit(loss).any() and (loss <= 8 * F32 * lse.abs()).all()
    d_h, d_w = moe.lm_head_loss_backward(h, w, y, torch.zeros_like(loss), lse, torch.ones_like(loss), weight_grad=True)
    assert (d_h == 0).all() and (d_w == 0).all()
