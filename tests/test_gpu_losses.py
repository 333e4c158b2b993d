"""GPU parity of the training losses (LM-head cross entropy, distillation,
balance loss) and of their gradients against the 64-bit references, element by
element within the references' rounding bounds."""
import math

import pytest
import torch

import precision_moe_expert_amd as moe
from precision_moe_expert_amd import binding, synth
from tests import gpu_util as gu
from tests import loss_ref as lr

pytestmark = pytest.mark.gpu

# (T, H, V): one row and column, ids on block edges, one more and one less than tiles of 16 to 256, odd vocabularies
SHAPES = [(1, 8, 1), (1, 64, 1000), (3, 72, 129), (16, 128, 128), (17, 40, 255), (63, 256, 257), (65, 200, 1024),
          (127, 136, 300), (129, 520, 1301), (255, 64, 513), (300, 256, 5003), (513, 192, 2050), (64, 1024, 8001)]


def _close(got, want, bound, label):
    err = (got.double() - want).abs()
    bad = ~((err <= bound + 1e-30) | (got.isnan() & want.isnan()))
    assert not bad.any(), (label, int(bad.sum()), float((err / (bound + 1e-30)).max()),
                           [int(i) for i in torch.nonzero(bad)[0]])


def _inputs(T, H, V, seed=0, ignored=0.3):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1000 * T + V)
    h = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w = (torch.randn(V, H, generator=g, device="cuda") * 2.5 / math.sqrt(H)).bfloat16()
    y = torch.randint(0, V, (T,), generator=g, device="cuda").int()
    if T > 1:
        y[0], y[-1] = 0, V - 1
    drop = torch.rand(T, generator=g, device="cuda") < ignored
    drop[: 1] = False
    y = torch.where(drop, -100, y).int()
    dl = torch.randn(T, generator=g, device="cuda")
    return h, w, y, dl, g


def _teacher(T, K, V, g, y=None):
    """Slots with absent ids, ids out of range, -infinity logits, repeated ids and empty rows."""
    ids = torch.randint(0, V, (T, K), generator=g, device="cuda").int()
    tl = torch.randn(T, K, generator=g, device="cuda") * 2
    u = torch.rand(T, K, generator=g, device="cuda")
    ids = torch.where(u < 0.1, -1, torch.where(u < 0.15, V, ids)).int()
    tl = torch.where((u > 0.15) & (u < 0.2), -math.inf, tl)
    tl = torch.where(u < 0.15, math.nan, tl)  # whatever absent slots hold
    if K > 2:
        ids[:, K - 1] = ids[:, 0]
    if T > 2:
        ids[1] = -5
    return ids.contiguous(), tl.contiguous()


@pytest.mark.parametrize("eps,scale", [(1e-6, 1.0), (0.0, 0.7)])
@pytest.mark.parametrize("T,H,V", SHAPES)
def test_cross_entropy(torch_gpu, T, H, V, eps, scale):
    h, w, y, dl, _ = _inputs(T, H, V)
    keep = y >= 0
    hn = torch.where(keep[:, None], h, math.nan).bfloat16()  # rows that do not count are never used
    ref = lr.ce_ref(h, w, y, eps, scale)
    lse, loss, b_lse, b_loss = ref.loss()
    got, got_lse = moe.lm_head_loss(hn, w, y, norm_eps=eps, logit_scale=scale)
    _close(got_lse, lse, b_lse, "lse")
    _close(got, loss, b_loss, "loss")
    d_h, b_h, d_w, b_w = ref.grads(dl, True)
    dln = torch.where(keep, dl, math.nan)
    gh, gw = moe.lm_head_loss_backward(hn, w, y, got, got_lse, dln, weight_grad=True, norm_eps=eps,
                                       logit_scale=scale)
    _close(gh, d_h, b_h, "d_h")
    _close(gw, d_w, b_w, "d_w")
    gh2, gw2 = moe.lm_head_loss_backward(hn, w, y, got, got_lse, dln, norm_eps=eps, logit_scale=scale)
    assert gw2 is None
    _close(gh2, d_h, b_h, "d_h of a frozen head")


# wide rows with few columns: the sum over H is split between workgroups (each on
# both sides of 256 rows, of whole tiles and of a multiple of 64 columns of h)
WIDE = [(1, 4096, 3), (2, 6488, 1118), (3, 2048, 700), (64, 7168, 2049), (137, 6872, 4001), (256, 4096, 300),
        (257, 4096, 501), (300, 1032, 257), (900, 2048, 130), (1500, 5000, 66)]


@pytest.mark.parametrize("T,H,V", WIDE)
def test_cross_entropy_wide_rows(torch_gpu, T, H, V):
    test_cross_entropy(torch_gpu, T, H, V, 1e-6, 0.9)


@pytest.mark.parametrize("T,H,V", WIDE)
def test_distillation_wide_rows(torch_gpu, T, H, V):
    test_distillation(torch_gpu, T, H, V, 5, True)


@pytest.mark.parametrize("nans", [True, False])
@pytest.mark.parametrize("K", [1, 2, 7, 64, 65, 256])
@pytest.mark.parametrize("T,H,V", [(1, 64, 100), (5, 72, 129), (130, 136, 3001), (300, 256, 513)])
def test_distillation(torch_gpu, T, H, V, K, nans):
    """nans: some of the slots that are there hold a NaN too, which spoils their row and its ids and nothing else."""
    h, w, _, dl, g = _inputs(T, H, V, seed=K)
    ids, tl = _teacher(T, K, V, g)
    if not nans:
        tl = torch.where(tl.isnan() & (ids >= 0) & (ids < V), 0.5, tl)
    ref, have, q = lr.distill_ref(h, w, ids, tl, 0.8, 1e-6, 0.9)
    hn = torch.where(ref.counts[:, None], h, math.nan).bfloat16()
    lse, loss, logp, b_lse, b_loss, b_logp = lr.distill_loss(ref, ids, have, q)
    got, got_lse, got_logp = moe.lm_head_distill(hn, w, ids, tl, teacher_scale=0.8, logit_scale=0.9)
    _close(got_lse, lse, b_lse, "lse")
    _close(got_logp, logp, b_logp, "logp")
    _close(got, loss, b_loss, "loss")
    d_h, b_h, d_w, b_w = ref.grads(dl, True)
    gh, gw = moe.lm_head_distill_backward(hn, w, ids, tl, got_lse, got_logp, dl, weight_grad=True, teacher_scale=0.8,
                                          logit_scale=0.9)
    _close(gh, d_h, b_h, "d_h")
    _close(gw, d_w, b_w, "d_w")


@pytest.mark.parametrize("T,H,V", [(66, 1024, 50001), (100, 1024, 32000), (128, 1536, 30001), (65, 512, 24001)])
def test_forward_of_one_tile_row(torch_gpu, T, H, V):
    """65 to 128 rows, read where they are, strided ones too."""
    h, w, y, _, g = _inputs(T, H, V)
    wide = torch.full((T, H + 16), math.nan, device="cuda").bfloat16()
    wide[:, :H] = torch.where((y >= 0)[:, None], h, math.nan)
    ref = lr.ce_ref(h, w, y, 1e-6, 0.8)
    lse, loss, b_lse, b_loss = ref.loss()
    got, got_lse = moe.lm_head_loss(wide[:, :H], w, y, logit_scale=0.8)
    _close(got_lse, lse, b_lse, "lse")
    _close(got, loss, b_loss, "loss")
    ids, tl = _teacher(T, 33, V, g)
    tl = torch.where(tl.isnan() & (ids >= 0) & (ids < V), 0.5, tl)
    ref, have, q = lr.distill_ref(h, w, ids, tl, 0.7)
    lse, loss, logp, b_lse, b_loss, b_logp = lr.distill_loss(ref, ids, have, q)
    got, got_lse, got_logp = moe.lm_head_distill(h, w, ids, tl, teacher_scale=0.7)
    _close(got_lse, lse, b_lse, "lse")
    _close(got_logp, logp, b_logp, "logp")
    _close(got, loss, b_loss, "loss")


@pytest.mark.parametrize("T,H,V", [(130, 256, 24001), (192, 520, 24001), (193, 512, 24001), (370, 520, 16001), (560, 256, 9001)])
def test_cross_entropy_between_tiles(torch_gpu, T, H, V):
    test_cross_entropy(torch_gpu, T, H, V, 1e-6, 0.9)


@pytest.mark.parametrize("T,H,V", [(150, 256, 24001), (192, 520, 24001), (370, 256, 16001)])
def test_distillation_between_tiles(torch_gpu, T, H, V):
    test_distillation(torch_gpu, T, H, V, 7, False)


@pytest.mark.parametrize("kind", ["ce", "distill"])
@pytest.mark.parametrize("T,H,V,ignored", [(2100, 520, 9000, 0.0), (2100, 520, 9000, 0.9), (2100, 520, 9000, 0.96),
                                           (2900, 256, 7001, 0.1)])
def test_head_last_round(torch_gpu, T, H, V, ignored, kind):
    """Large tiles whose last round is done in halves, some of them without rows."""
    h, w, y, dl, g = _inputs(T, H, V, ignored=ignored)
    if kind == "ce":
        ref = lr.ce_ref(h, w, y)
        lse, loss, b_lse, b_loss = ref.loss()
        got, got_lse = moe.lm_head_loss(h, w, y)
        gh, gw = moe.lm_head_loss_backward(h, w, y, got, got_lse, dl, weight_grad=True)
    else:
        ids, tl = _teacher(T, 5, V, g)
        tl = torch.where(tl.isnan() & (ids >= 0) & (ids < V), 0.5, tl)
        ids = torch.where((y < 0)[:, None], -1, ids).int()
        ref, have, q = lr.distill_ref(h, w, ids, tl)
        lse, loss, logp, b_lse, b_loss, b_logp = lr.distill_loss(ref, ids, have, q)
        got, got_lse, got_logp = moe.lm_head_distill(h, w, ids, tl)
        _close(got_logp, logp, b_logp, "logp")
        gh, gw = moe.lm_head_distill_backward(h, w, ids, tl, got_lse, got_logp, dl, weight_grad=True)
    _close(got_lse, lse, b_lse, "lse")
    _close(got, loss, b_loss, "loss")
    d_h, b_h, d_w, b_w = ref.grads(dl, True)
    _close(gh, d_h, b_h, "d_h")
    _close(gw, d_w, b_w, "d_w")


@pytest.mark.parametrize("T,H,V", [(5, 64, 300), (70, 136, 301), (300, 64, 500), (1100, 64, 129), (9, 4096, 300)])
def test_distillation_lowest_logits(torch_gpu, T, H, V):
    """Teacher logits of the type's lowest value are slots that are there: probability 0 beside others, equal where
    a token has no others, whatever the scale."""
    K = 6
    h, w, _, dl, g = _inputs(T, H, V)
    ids = torch.stack([torch.randperm(V, generator=g, device="cuda")[:K] for _ in range(T)]).int()
    tl = torch.randn(T, K, generator=g, device="cuda")
    low = torch.finfo(torch.float32).min
    tl[:, 2] = low
    tl[::3] = low
    tl[1, 0] = 2e38
    ref, have, q = lr.distill_ref(h, w, ids, tl, 2.0, 1e-6, 1.0)
    assert have.all() and (q[0] == q[0, 0]).all()
    lse, loss, logp, b_lse, b_loss, b_logp = lr.distill_loss(ref, ids, have, q)
    got, got_lse, got_logp = moe.lm_head_distill(h, w, ids, tl, teacher_scale=2.0)
    _close(got_logp, logp, b_logp, "logp")
    _close(got, loss, b_loss, "loss")
    d_h, b_h, d_w, b_w = ref.grads(dl, True)
    gh, gw = moe.lm_head_distill_backward(h, w, ids, tl, got_lse, got_logp, dl, weight_grad=True, teacher_scale=2.0)
    _close(gh, d_h, b_h, "d_h")
    _close(gw, d_w, b_w, "d_w")


def test_cross_entropy_masks(torch_gpu):
    """No token counts; all do; ids past the vocabulary; confident rows."""
    T, H, V = 70, 128, 500
    h, w, y, dl, _ = _inputs(T, H, V, ignored=0.0)
    none = torch.full_like(y, -1)
    bad = torch.full_like(h, math.inf)
    loss, lse = moe.lm_head_loss(bad, w, none)
    gh, gw = moe.lm_head_loss_backward(bad, w, none, loss, lse, dl, weight_grad=True)
    for t in (loss, lse, gh, gw):
        assert (t == 0).all()
    past = y.clone()
    past[::2], past[3] = V, 2 ** 31 - 1
    out = past >= V
    loss, lse = moe.lm_head_loss(h, w, past)
    ref = lr.ce_ref(h, w, past)
    assert loss[out].isnan().all() and (lse[out] == 0).all()
    _close(torch.where(out, 0.0, loss), ref.loss()[1], ref.loss()[3], "loss")
    gh, gw = moe.lm_head_loss_backward(h, w, past, loss, lse, dl, weight_grad=True)
    d_h, b_h, d_w, b_w = ref.grads(dl, True)
    _close(gh, d_h, b_h, "d_h")
    _close(gw, d_w, b_w, "d_w")
    # rows that are their target's row of W, far from the others
    h = (w[y.long()].float() * 8).bfloat16()
    ref = lr.ce_ref(h, w, y, 0.0, 1.0)
    loss, lse = moe.lm_head_loss(h, w, y, norm_eps=0.0)
    _close(loss, ref.loss()[1], ref.loss()[3], "confident loss")
    gh, _ = moe.lm_head_loss_backward(h, w, y, loss, lse, dl, norm_eps=0.0)
    d_h, b_h, _, _ = ref.grads(dl, False)
    _close(gh, d_h, b_h, "confident d_h")


@pytest.mark.parametrize("T,V,spread", [(40, 300, 3), (600, 129, 129), (2500, 700, 2), (2500, 3000, 3000), (5000, 90, 1)])
def test_repeated_targets(torch_gpu, T, V, spread):
    """Many tokens of one target: the rows of d_w that the fp32 entries go to, alone, in pairs and in thousands, the
    same each time."""
    H = 72
    h, w, y, dl, g = _inputs(T, H, V, ignored=0.2)
    y = torch.where(y >= 0, torch.randint(0, spread, (T,), generator=g, device="cuda").int() * (V // spread), y).int()
    ref = lr.ce_ref(h, w, y)
    loss, lse = moe.lm_head_loss(h, w, y)
    d_h, b_h, d_w, b_w = ref.grads(dl, True)
    got = moe.lm_head_loss_backward(h, w, y, loss, lse, dl, weight_grad=True)
    _close(got[0], d_h, b_h, "d_h")
    _close(got[1], d_w, b_w, "d_w")
    again = moe.lm_head_loss_backward(h, w, y, loss, lse, dl, weight_grad=True)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("T,K,V", [(20, 5, 1000), (20, 5, 300), (300, 9, 12000), (300, 9, 9000)])
def test_entry_precision(torch_gpu, T, K, V):
    """Where the entries at the target's ids are kept in fp32 (few of them for the vocabulary; cross entropy always),
    the gradients of peaked rows are within 1.25 of the rounding of the results themselves; bf16 entries alone would
    add as much again."""
    H = 256
    h, w, y, dl, g = _inputs(T, H, V, ignored=0.0)
    ids = torch.randint(0, V, (T, K), generator=g, device="cuda").int()
    tl = torch.randn(T, K, generator=g, device="cuda")
    ref = lr.ce_ref(h, w, y)
    loss, lse = moe.lm_head_loss(h, w, y)
    pairs = [(ref, moe.lm_head_loss_backward(h, w, y, loss, lse, dl, weight_grad=True))]
    if T * K <= V // 4:
        loss, lse, logp = moe.lm_head_distill(h, w, ids, tl)
        pairs.append((lr.distill_ref(h, w, ids, tl)[0],
                      moe.lm_head_distill_backward(h, w, ids, tl, lse, logp, dl, weight_grad=True)))
    for ref, got in pairs:
        want = ref.grads(dl, True)
        for a, b in zip(got, (want[0], want[2])):
            rounding = torch.linalg.norm(b.bfloat16().double() - b)
            # G's other entries are rounded too: their share of G's norm, in quadrature
            rest = torch.linalg.norm(torch.where(ref.q > 0, 0.0, ref.p)) / torch.linalg.norm(ref.p - ref.q)
            assert torch.linalg.norm(a.double() - b) <= rounding * (1.25 + rest)


def test_head_rows_strided(torch_gpu):
    T, H, V = 90, 200, 700
    h, w, y, dl, _ = _inputs(T, H, V)
    hw = torch.full((T, H + 24), math.nan, device="cuda").bfloat16()
    ww = torch.full((V, H + 8), math.nan, device="cuda").bfloat16()
    hw[:, 8:8 + H], ww[:, :H] = h, w
    hs, ws = hw[:, 8:8 + H], ww[:, :H]
    loss, lse = moe.lm_head_loss(h, w, y)
    loss2, lse2 = moe.lm_head_loss(hs, ws, y)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    for a, b in zip(moe.lm_head_loss_backward(h, w, y, loss, lse, dl, weight_grad=True),
                    moe.lm_head_loss_backward(hs, ws, y, loss, lse, dl, weight_grad=True)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["ce", "distill"])
def test_head_pieces(torch_gpu, kind):
    """Enough tokens that the backward takes the vocabulary in several pieces."""
    T, H, V, K = 4100, 64, 70001, 5
    h, w, y, dl, g = _inputs(T, H, V)
    ids, tl = _teacher(T, K, V, g)
    if kind == "ce":
        ref = lr.ce_ref(h, w, y)
        loss, lse = moe.lm_head_loss(h, w, y)
        _close(loss, ref.loss()[1], ref.loss()[3], "loss")
        gh, gw = moe.lm_head_loss_backward(h, w, y, loss, lse, dl, weight_grad=True)
    else:
        ref, have, q = lr.distill_ref(h, w, ids, tl)
        loss, lse, logp = moe.lm_head_distill(h, w, ids, tl)
        _close(loss, *[lr.distill_loss(ref, ids, have, q)[i] for i in (1, 4)], "loss")
        gh, gw = moe.lm_head_distill_backward(h, w, ids, tl, lse, logp, dl, weight_grad=True)
    d_h, b_h, d_w, b_w = ref.grads(dl, True)
    _close(gh, d_h, b_h, "d_h")
    _close(gw, d_w, b_w, "d_w")


def test_head_without_tokens(torch_gpu):
    h, w = torch.empty(0, 64, device="cuda").bfloat16(), torch.randn(50, 64, device="cuda").bfloat16()
    y, f = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda")
    loss, lse = moe.lm_head_loss(h, w, y)
    assert loss.shape == (0,)
    gh, gw = moe.lm_head_loss_backward(h, w, y, loss, lse, f, weight_grad=True)
    assert gh.shape == (0, 64) and (gw == 0).all()
    ids, tl = y.view(0, 1).expand(0, 3).contiguous(), f.view(0, 1).expand(0, 3).contiguous()
    loss, lse, logp = moe.lm_head_distill(h, w, ids, tl)
    assert moe.lm_head_distill_backward(h, w, ids, tl, lse, logp, f)[0].shape == (0, 64)


BALANCE = [(1, 1, 1), (1, 8, 2), (15, 5, 2), (16, 64, 4), (17, 65, 3), (33, 130, 8), (300, 128, 8), (1000, 256, 8),
           (700, 384, 6), (130, 385, 1), (90, 1000, 16), (70, 1024, 16), (20000, 60, 4), (1024, 33, 2), (1025, 64, 2),
           (2100, 1024, 8), (1500, 390, 7)]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T,E,k", BALANCE)
def test_balance(torch_gpu, T, E, k, packed):
    torch.manual_seed(T + E)
    logits = torch.randn(T, E) + torch.randn(E)
    if E > 3:
        logits[::3, E // 2] = -math.inf  # masked experts
    if T > 4:
        logits[4] = -math.inf
    ids = torch.topk(logits, k, 1).indices.int()
    if T > 2:
        ids[2, 0] = -1
        ids[T - 1, k - 1] = E
    layer = moe.make_layer(T, 256, 128, E, k, moe.FMT_INT4)
    mask = off = None
    if packed:
        mask = (torch.rand(T) < 0.7).to(torch.uint8)
        logits[mask == 0] = math.nan
        off = [min(T, 1), min(T, 2), min(T, 2), T // 2, T // 2, T - T // 5, T - T // 5]
        off = torch.tensor(sorted(off)).int()
    S = 1 if off is None else len(off) - 1
    g = torch.randn(S)
    ref = lr.balance_ref(logits, ids, k, mask, None if off is None else off.tolist(), g)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    lg, msk, offd = logits.cuda(), dev(mask), dev(off)
    loss, counts, tokens, probs = moe.balance_loss(layer, lg, ids.cuda(), token_mask=msk, seg_offsets=offd)
    assert torch.equal(counts.cpu().long(), ref["counts"]) and torch.equal(tokens.cpu().long(), ref["tokens"])
    _close(probs.cpu(), ref["probs"], ref["b_probs"], "probs")
    _close(loss.cpu(), ref["loss"], ref["b_loss"], "loss")
    d = moe.balance_loss_backward(layer, lg, counts, tokens, g.cuda(), token_mask=msk, seg_offsets=offd)
    _close(d.cpu(), ref["d_logits"], ref["b_grad"], "d_logits")
    base = torch.randn(T, E, device="cuda")
    both = moe.balance_loss_backward(layer, lg, counts, tokens, g.cuda(), token_mask=msk, seg_offsets=offd,
                                     d_logits=base.clone())
    assert torch.equal(both, base + d)
    # the same sums in the same order each time
    again = moe.balance_loss(layer, lg, ids.cuda(), token_mask=None if msk is None else msk.bool(), seg_offsets=offd)
    assert all(torch.equal(a, b) for a, b in zip((loss, counts, tokens, probs), again))


@pytest.mark.parametrize("T,E,k", [(70, 48, 3), (70, 45, 3), (1100, 200, 2)])
def test_balance_lowest_logits(torch_gpu, T, E, k):
    """Masks of the type's lowest value: probability 0 beside others, equal where a row has no others; so at the
    other end of the range."""
    torch.manual_seed(T)
    logits = torch.randn(T, E)
    low = torch.finfo(torch.float32).min
    logits[:, E // 2] = low
    logits[::3] = low
    logits[1] = -low
    logits[2, 3] = 3e38
    ids = torch.topk(logits, k, 1).indices.int()
    layer = moe.make_layer(T, 256, 128, E, k, moe.FMT_INT4)
    g = torch.tensor([0.7])
    ref = lr.balance_ref(logits, ids, k, d_loss=g)
    loss, counts, tokens, probs = moe.balance_loss(layer, logits.cuda(), ids.cuda())
    # |m - x| of a lowest value enters the reference's bound where p is 0: such rows count with their sum of p, 1
    assert torch.allclose(probs.cpu().double(), ref["probs"], rtol=(T + 64) * 2.0 ** -24, atol=16 * 2.0 ** -24)
    assert torch.allclose(loss.cpu().double(), ref["loss"], rtol=(T + E + 64) * 2.0 ** -24, atol=0)
    d = moe.balance_loss_backward(layer, logits.cuda(), counts, tokens, g.cuda())
    a = 0.7 * E / (k * T * T) * ref["counts"][0].double()
    assert ((d.cpu().double() - ref["d_logits"]).abs() <= a.max() * (E + 64) * 2.0 ** -24).all()


@pytest.mark.parametrize("T,E,k,most", [(900, 48, 3, 4), (1100, 385, 2, 4), (3000, 48, 3, 3), (5000, 130, 4, 40)])
def test_balance_many_segments(torch_gpu, T, E, k, most):
    """More segments than slabs, up to `most` - 1 tokens each, empty ones among them (3000 tokens: more than 1024
    segments)."""
    torch.manual_seed(1)
    off = [0]
    while off[-1] < T:
        off.append(min(T, off[-1] + int(torch.randint(0, most, (1,)))))
    off = torch.tensor(off + [T]).int()
    logits = torch.randn(T, E)
    ids = torch.topk(logits, k, 1).indices.int()
    layer = moe.make_layer(T, 256, 128, E, k, moe.FMT_INT4)
    g = torch.randn(len(off) - 1)
    ref = lr.balance_ref(logits, ids, k, None, off.tolist(), g)
    loss, counts, tokens, probs = moe.balance_loss(layer, logits.cuda(), ids.cuda(), seg_offsets=off.cuda())
    assert torch.equal(counts.cpu().long(), ref["counts"]) and torch.equal(tokens.cpu().long(), ref["tokens"])
    _close(loss.cpu(), ref["loss"], ref["b_loss"], "loss")
    d = moe.balance_loss_backward(layer, logits.cuda(), counts, tokens, g.cuda(), seg_offsets=off.cuda())
    _close(d.cpu(), ref["d_logits"], ref["b_grad"], "d_logits")


def test_balance_without_tokens(torch_gpu):
    layer = moe.make_layer(0, 256, 128, 8, 2, moe.FMT_INT4)
    out = moe.balance_loss(layer, torch.empty(0, 8, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert all((t == 0).all() for t in out) and out[1].shape == (1, 8)


def _step(d, cfg, w_lm, y, ids, tl, off):
    """One adapter training step's losses and gradients: the layer, both head losses, the balance loss."""
    route = moe.route_permute(d.logits, d.layer)
    out = moe.expert_forward(d.layer, d.x, d.logits, d.w13, d.w2, d.s13, d.s2, adapter=d.oft, chunk_experts=cfg.chunk)
    loss, lse = moe.lm_head_loss(out, w_lm, y)
    kl, klse, logp = moe.lm_head_distill(out, w_lm, ids, tl)
    bal, counts, tokens, probs = moe.balance_loss(d.layer, d.logits, route["topk_ids"], seg_offsets=off)
    g = torch.full((cfg.T,), 1.0 / cfg.T, device="cuda")
    d_h, _ = moe.lm_head_loss_backward(out, w_lm, y, loss, lse, g)
    d_k, _ = moe.lm_head_distill_backward(out, w_lm, ids, tl, klse, logp, g)
    bwd = moe.prepare_backward_weights(d.layer, d.w13, d.w2, d.s13, d.s2)
    d_x, d_logits, d_r = moe.expert_backward(d.layer, d.x, d.logits, d.w13, d.w2, d.s13, d.s2, bwd, d_h + d_k,
                                             adapter=d.oft, chunk_experts=cfg.chunk)
    routed = d_logits.clone()
    moe.balance_loss_backward(d.layer, d.logits, counts, tokens, torch.full((len(off) - 1,), 0.01, device="cuda"),
                              seg_offsets=off, d_logits=d_logits)
    return dict(out=out, loss=loss, kl=kl, bal=bal, d_h=d_h, d_k=d_k, d_x=d_x, d_logits=d_logits, d_r=d_r,
                routed=routed, counts=counts)


def _step_inputs():
    cfg = synth.LayerConfig("losses", 77, T=200, H=512, E=12, k=3, I=256, fmt=binding.FMT_INT4, chunk=5, oft=True)
    d = gu.DevInputs(synth.make_inputs(cfg))
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    w_lm = (torch.randn(1003, cfg.H, generator=g, device="cuda") / 8).bfloat16()
    y = torch.randint(-200, 1003, (cfg.T,), generator=g, device="cuda").int()
    ids, tl = _teacher(cfg.T, 9, 1003, g)
    tl = torch.where(tl.isnan() & (ids >= 0) & (ids < 1003), 0.5, tl)  # a NaN in a slot that is there is the caller's
    return cfg, d, w_lm, y, ids, tl, torch.tensor([0, 50, 51, 200], device="cuda").int()


def test_training_step(torch_gpu):
    cfg, d, w_lm, y, ids, tl, off = _step_inputs()
    s = _step(d, cfg, w_lm, y, ids, tl, off)
    ref = lr.ce_ref(s["out"], w_lm, y)
    _close(s["loss"], ref.loss()[1], ref.loss()[3], "loss")
    g = torch.full((cfg.T,), 1.0 / cfg.T, device="cuda")
    d_h, b_h, _, _ = ref.grads(g, False)
    _close(s["d_h"], d_h, b_h, "d_h")
    kr, have, q = lr.distill_ref(s["out"], w_lm, ids, tl)
    d_k, b_k, _, _ = kr.grads(g, False)
    _close(s["d_k"], d_k, b_k, "d_k")
    # the loss is the negative of the head's log-prob of the same targets (either within the forward's bound)
    lp = moe.lm_head_logprob(s["out"], w_lm, y.clamp(min=0))
    _close(torch.where(y >= 0, -lp, 0.0), ref.loss()[1], ref.loss()[3], "log-prob")
    br = lr.balance_ref(d.logits.cpu(), torch.topk(d.logits, cfg.k, 1).indices.cpu(), cfg.k, None, off.tolist(),
                        torch.full((3,), 0.01))
    _close(s["bal"].cpu(), br["loss"], br["b_loss"], "balance")
    add = s["d_logits"].double() - s["routed"].double()
    _close(add.cpu(), br["d_logits"], br["b_grad"] + 2 * lr.F32 * (s["d_logits"].abs() + s["routed"].abs()).cpu(),
           "balance d_logits")
    assert s["d_x"].isfinite().all() and s["d_r"].abs().max() > 0


def test_captured_step_replays(torch_gpu):
    """The step captured into a graph on a side stream and replayed between eager work gives the eager results."""
    cfg, d, w_lm, y, ids, tl, off = _step_inputs()
    eager = _step(d, cfg, w_lm, y, ids, tl, off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(d, cfg, w_lm, y, ids, tl, off)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = _step(d, cfg, w_lm, y, ids, tl, off)
    for i in range(4):
        for t in held.values():
            t.fill_(float(i) if t.is_floating_point() else i)
        graph.replay()
        junk = torch.randn(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        assert junk.isfinite()
        for k, t in held.items():
            assert torch.equal(t, eager[k]), (i, k)
        other = moe.lm_head_loss(eager["out"], w_lm, y)[0]
        assert torch.equal(other, eager["loss"])


def test_two_streams(torch_gpu):
    """Calls on two streams at once, each with its own workspace."""
    a, b = _inputs(200, 256, 3000, 1), _inputs(130, 512, 4000, 2)
    want = [moe.lm_head_loss(*x[:3]) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, x in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                loss, lse = moe.lm_head_loss(*x[:3])
                got[i].append((loss, lse, moe.lm_head_loss_backward(*x[:3], loss, lse, x[3])[0]))
    torch.cuda.synchronize()
    for i in range(2):
        for loss, lse, dh in got[i]:
            assert torch.equal(loss, want[i][0]) and torch.equal(lse, want[i][1])
            assert torch.equal(dh, got[i][0][2])


def test_wrappers_refuse(torch_gpu):
    h, w, y, dl, _ = _inputs(8, 64, 100)
    lse = torch.zeros(8, device="cuda")
    bad = [lambda: moe.lm_head_loss(h.float(), w, y), lambda: moe.lm_head_loss(h, w.half(), y),
           lambda: moe.lm_head_loss(h, w, y.long()), lambda: moe.lm_head_loss(h, w, y[:7]),
           lambda: moe.lm_head_loss(h, w[:, :56].contiguous(), y), lambda: moe.lm_head_loss(h.cpu(), w, y),
           lambda: moe.lm_head_loss(h, w.t().contiguous().t(), y),
           lambda: moe.lm_head_loss(h[:1].expand(8, 64), w, y), lambda: moe.lm_head_loss(h, w, y.cpu()),
           lambda: moe.lm_head_loss_backward(h, w, y, lse, lse[:7], dl),
           lambda: moe.lm_head_loss_backward(h, w, y, lse, lse, dl.double()),
           lambda: moe.lm_head_distill(h, w, y, dl),
           lambda: moe.lm_head_distill(h, w, y[:, None].expand(8, 2), dl[:, None].expand(8, 2))]
    layer = moe.make_layer(8, 256, 128, 16, 2, moe.FMT_INT4)
    lg, ids = torch.zeros(8, 16, device="cuda"), torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    off = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad += [lambda: moe.balance_loss(layer, lg[:7], ids), lambda: moe.balance_loss(layer, lg, ids.long()),
            lambda: moe.balance_loss(layer, lg, ids, seg_offsets=off),
            lambda: moe.balance_loss(layer, lg, ids, token_mask=lg[:, 0])]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    for f in (lambda: moe.lm_head_loss(h, w, y, norm_eps=-1.0), lambda: moe.lm_head_loss(h, w, y, logit_scale=0.0),
              lambda: moe.lm_head_loss(h, w, y, ws=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(moe.MoeError):
            f()
