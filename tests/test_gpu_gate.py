"""GPU parity of the gate and of the expert layer behind it."""
import math

import pytest
import torch

import precision_moe_expert_amd as moe
from precision_moe_expert_amd import binding
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu
INF = math.inf


def _case(T, E, seed, out=0.0, bias=0.1):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) * 2 + torch.randn(E, generator=g)
    b = torch.randn(E, generator=g) * bias
    b[torch.randperm(E, generator=g)[:int(E * out)]] = -INF
    return logits, b, g


def _layer(T, E, k):
    return moe.make_layer(T, 256, 128, E, k, moe.FMT_FP8)


def _gate(sigmoid, groups, top, top2, renorm, scale):
    return moe.make_gate(moe.GATE_SIGMOID if sigmoid else moe.GATE_SOFTMAX, groups, top,
                         moe.GROUP_TOP2 if top2 else moe.GROUP_MAX, renorm, scale)


def _check_forward(logits, bias, k, sigmoid=True, groups=1, top=1, top2=True, renorm=True, scale=2.5, permute=False):
    T, E = logits.shape
    want, w = ref.gate(logits, bias, k, sigmoid, groups, top, top2, renorm, scale)
    r = moe.route_gated(_layer(T, E, k), _gate(sigmoid, groups, top, top2, renorm, scale), logits.cuda(),
                        None if bias is None else bias.cuda(), permute=permute)
    assert torch.equal(r["topk_ids"].cpu(), want)
    got = r["topk_w"].cpu().double()
    # formed in 64 bits, rounded once; softmax's sum over all experts may be one of fp32 terms: the difference and the
    # exponential of each (5 half steps), at most E / 16 + 4 additions in a row
    steps = 1 if sigmoid or renorm else E // 16 + 12
    assert bool(((got - w).abs() <= w.abs() * ref.F32 * (steps + 1e-6) + 1e-44).all())
    return r


@pytest.mark.parametrize("T", [1, 5, 1024, 1031])
@pytest.mark.parametrize("E,k,groups,top", [(256, 8, 8, 4), (256, 8, 1, 1), (384, 6, 1, 1), (72, 4, 8, 3), (8, 8, 2, 2),
                                            (60, 5, 4, 2), (1, 1, 1, 1), (1024, 16, 64, 20), (700, 3, 7, 2),
                                            (9, 2, 9, 2), (512, 1, 2, 1), (1024, 8, 16, 4), (1000, 16, 1, 1),
                                            (528, 6, 2, 2), (33, 16, 1, 1), (17, 9, 1, 1)])
def test_choice_and_weights(T, E, k, groups, top):
    if T > 1000 and E > 400:
        T = 40 if T == 1024 else 1030
    logits, bias, _ = _case(T, E, T * 31 + E)
    for sigmoid, top2, renorm in ((True, True, True), (False, False, False), (False, True, True), (True, False, False)):
        _check_forward(logits, bias if sigmoid or E < 300 else None, k, sigmoid, groups, top, top2, renorm)


@pytest.mark.parametrize("T", [3, 1500])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_experts_out(T, sigmoid):
    logits, bias, _ = _case(T, 64, 7, out=0.4)
    logits[::3, 5:20] = -INF
    logits[1, 30:40] = math.nan
    bias[50] = math.nan
    logits[0, 50] = math.nan
    logits[2, :] = -INF                     # nobody is in
    logits[1, :60] = -INF                   # fewer are in than chosen
    for groups, top, top2 in ((1, 1, True), (8, 2, True), (8, 3, False), (16, 4, True)):
        for renorm in (True, False):
            r = _check_forward(logits, bias, 6, sigmoid, groups, top, top2, renorm)
    assert bool((r["topk_w"][2] == 0).all()) and r["topk_ids"][2].unique().numel() == 6


@pytest.mark.parametrize("T", [4, 1200])
def test_ties_go_to_the_lowest(T):
    logits = torch.zeros(T, 48)
    logits[:, 30] = 1.0
    logits[:, 7] = 1.0
    bias = torch.zeros(48)
    r = _check_forward(logits, bias, 4)
    assert r["topk_ids"][0].tolist() == [7, 30, 0, 1]
    _check_forward(logits, bias, 4, groups=6, top=2)
    _check_forward(logits, None, 4, sigmoid=False, groups=6, top=3, top2=False)
    logits[1, 3] = -0.0
    _check_forward(logits, bias, 4)


@pytest.mark.parametrize("T", [3, 1100])
def test_far_logits(T):
    logits = torch.randn(T, 32, generator=torch.Generator().manual_seed(2))
    logits[0, :] *= 1e30                    # beyond exp's range on both sides
    logits[1, 3] = INF
    logits[1, 9] = INF
    logits[2, :] = torch.finfo(torch.float32).min
    logits[2, 4] = -1000.0
    for sigmoid in (True, False):
        for renorm in (True, False):
            _check_forward(logits, None, 5, sigmoid, renorm=renorm)
    big = torch.zeros(32)
    big[11] = 1e30
    big[12] = INF
    big[13] = -1e30
    _check_forward(logits, big, 5, True, groups=4, top=2)


@pytest.mark.parametrize("k", [1, 2, 3])
def test_infinite_logits(k):
    """One, two and three experts with all of a token's softmax, as many as are chosen or fewer."""
    for E, groups in ((32, 1), (256, 4), (30, 3)):
        logits = torch.randn(9, E, generator=torch.Generator().manual_seed(E + k))
        for t, at in ((1, [3]), (2, [3, 9]), (4, [0, 1, E - 1])):
            logits[t, at] = INF
        for sigmoid in (True, False):
            for renorm in (True, False):
                _check_forward(logits, None, k, sigmoid, groups, groups, True, renorm)


@pytest.mark.parametrize("T", [3, 260])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2), (3, 2)])
def test_values_closer_than_fp32(T, groups, top):
    """Biases that put neighbours within a few 1e-9 of each other, inside a group and between groups."""
    g = torch.Generator().manual_seed(T)
    logits = torch.randn(T, 48, generator=g)
    bias = (0.5 - torch.sigmoid(logits[1].double())).float()            # row 1: every c is 0.5 to a rounding
    _check_forward(logits, bias, 6, True, groups, top)
    _check_forward(logits, bias, 6, True, groups, top, top2=False)
    p = torch.softmax(logits.double(), 1)
    _check_forward(logits, (0.01 - p[2]).float(), 6, False, groups, top, renorm=False)


def test_a_chosen_score_of_zero():
    logits = torch.zeros(5, 32)
    logits[:, 9] = -1e4
    bias = torch.zeros(32)
    bias[9] = 5.0
    _check_forward(logits, bias, 1)
    _check_forward(logits, bias, 3)
    _check_forward(logits, bias, 2, sigmoid=False)


def test_close_values_are_told_apart():
    # sigmoids that round to the same fp32 number
    logits = torch.tensor([[20.0, 20.5, 21.0, 3.0] + [0.0] * 12] * 3)
    bias = torch.zeros(16)
    bias[3] = 0.05
    r = _check_forward(logits, bias, 3)
    assert r["topk_ids"][0].tolist() == [2, 1, 0] or r["topk_ids"][0].tolist()[0] == 3


@pytest.mark.parametrize("T,E,k", [(1, 16, 4), (64, 128, 8), (65, 128, 8), (700, 40, 3)])
def test_permutation_is_that_of_the_ids(T, E, k):
    logits, bias, _ = _case(T, E, 3)
    r = _check_forward(logits, bias, k, groups=4, top=2, permute=True)
    ids = r["topk_ids"].flatten().long().cpu()
    order = torch.sort(ids, stable=True).indices
    assert torch.equal(r["sorted_rows"].cpu().long(), order)
    assert torch.equal(r["row_of"].cpu().long()[order], torch.arange(T * k))
    counts = torch.bincount(ids, minlength=E)
    assert torch.equal(r["expert_offsets"].cpu().long(), torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]))
    n = int(r["num_active"][0])
    assert torch.equal(r["active_experts"][:n].cpu().long(), torch.nonzero(counts)[:, 0])


def test_softmax_gate_agrees_with_the_layers_own_routing():
    logits, _, _ = _case(300, 64, 9)
    layer = _layer(300, 64, 6)
    own = moe.route_permute(logits.cuda(), layer)
    r = moe.route_gated(layer, moe.make_gate(moe.GATE_SOFTMAX), logits.cuda())
    for name in ("topk_ids", "expert_offsets", "sorted_rows", "row_of"):
        assert torch.equal(own[name], r[name]), name
    torch.testing.assert_close(own["topk_w"], r["topk_w"], rtol=1e-5, atol=0)


def _check_backward(logits, bias, ids, dw, sigmoid, renorm, scale=2.5, start=None):
    T, E = logits.shape
    want, bound = ref.gate_grad(logits, bias, ids, dw, sigmoid, renorm, scale)
    d = None if start is None else start.clone().cuda()
    got = moe.route_gated_backward(_layer(T, E, ids.shape[1]), _gate(sigmoid, 1, 1, True, renorm, scale), logits.cuda(),
                                   ids.cuda(), dw.cuda(), None if bias is None else bias.cuda(), d_logits=d)
    got = got.cpu().double()
    if start is not None:
        want = want + start.double()
        bound = bound + ref.F32 * want.abs()
    assert bool(((got - want).abs() <= bound).all()), float(((got - want).abs() / bound).max())
    return got


@pytest.mark.parametrize("T", [1, 6, 64, 1027])
@pytest.mark.parametrize("E,k", [(256, 8), (384, 8), (60, 5), (1, 1), (1024, 16), (67, 3), (516, 2), (640, 8)])
def test_gradient(T, E, k):
    logits, bias, g = _case(T, E, T + E, out=0.1)
    for sigmoid in (True, False):
        ids, _ = ref.gate(logits, bias, k, sigmoid)
        dw = torch.randn(T, k, generator=g)
        for renorm in (True, False):
            _check_backward(logits, bias, ids, dw, sigmoid, renorm)
            _check_backward(logits, None, ids, dw, sigmoid, renorm, start=torch.randn(T, E, generator=g))


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_odd_rows(sigmoid, renorm):
    logits, bias, g = _case(8, 24, 4, out=0.2)
    ids, _ = ref.gate(logits, bias, 4, sigmoid)
    dw = torch.randn(8, 4, generator=g)
    logits[1] = -INF
    logits[2, :20] = math.nan
    logits[3, int(ids[3, 1])] = -INF        # a chosen one is out
    ids[4, 0], ids[4, 2] = -1, 24           # absent slots
    ids[5, 3] = ids[5, 0]                   # an id twice
    ids[6, :] = ids[6, 1]
    logits[7] *= 20
    got = _check_backward(logits, bias, ids, dw, sigmoid, renorm)
    assert bool((got[1] == 0).all())
    _check_backward(logits, bias, ids, dw, sigmoid, renorm, start=torch.ones(8, 24))


@pytest.mark.parametrize("E", [24, 26])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
def test_nan_in_absent_places(sigmoid, renorm, E):
    """Gradients and logits that belong to no slot or to an expert that is out."""
    logits, bias, g = _case(6, E, 11)
    ids, _ = ref.gate(logits, bias, 4, sigmoid)
    dw = torch.randn(6, 4, generator=g)
    ids[0, 1], dw[0, 1] = -1, math.nan
    ids[1, 3], dw[1, 3] = 1 << 30, INF
    bias[int(ids[2, 0])] = -INF
    clean = dw.clone()
    clean[(ids < 0) | (ids >= E)] = 0.0
    out = torch.where((ids >= 0) & (ids < E), bias[ids.long().clamp(0, E - 1)] == -INF, False)
    dw[out] = math.nan
    clean[out] = 0.0
    logits[:, bias == -INF] = math.nan
    layer, gate = _layer(6, E, 4), _gate(sigmoid, 1, 1, True, renorm, 1.0)
    got = moe.route_gated_backward(layer, gate, logits.cuda(), ids.cuda(), dw.cuda(), bias.cuda()).cpu().double()
    want, bound = ref.gate_grad(logits, bias, ids, clean, sigmoid, renorm, 1.0)
    assert bool(((got - want).abs() <= bound).all())


def test_gradient_against_differences():
    logits, bias, g = _case(12, 20, 8)
    for sigmoid in (True, False):
        for renorm in (True, False):
            ids, _ = ref.gate(logits, bias, 3, sigmoid)
            dw = torch.randn(12, 3, generator=g)
            got = _check_backward(logits, bias, ids, dw, sigmoid, renorm, 1.0)
            way = torch.randn(12, 20, generator=g).double()
            h = 1e-5
            f = [(ref.gate_weights(logits.double() + s * h * way, bias, ids, sigmoid, renorm, 1.0) * dw.double()).sum()
                 for s in (1, -1)]
            d = float((f[0] - f[1]) / (2 * h))
            assert abs(d - float((got * way).sum())) <= 1e-4 * float((got * way).abs().sum()) + 1e-9


@pytest.mark.parametrize("E,k", [(24, 4), (26, 4), (64, 8), (67, 16), (16, 1), (18, 1)])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_chosen_scores_near_zero(E, k, renorm):
    """All chosen logits far below 0 (a bias chooses such experts): below fp32's smallest sigmoids the weights that sum
    to `scale` are still those of the forward, and so is their gradient; from -745 on the forward's are 0."""
    levels = [-60.0, -86.0, -90.0, -95.0, -101.0, -110.0, -690.0, -800.0]
    g = torch.Generator().manual_seed(E + k)
    T = 3 * len(levels)
    logits = torch.randn(T, E, generator=g)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    far = torch.tensor(levels * 3)[:, None] - 1.5 * torch.rand(T, k, generator=g)
    far[2 * len(levels):, 0] = 2.0                       # all but one
    logits.scatter_(1, ids.long(), far)
    dw = torch.randn(T, k, generator=g)
    dw[:len(levels)] *= 0.01
    dw[len(levels):2 * len(levels)] *= 200.0
    got = _check_backward(logits, None, ids, dw, True, renorm)
    _check_backward(logits, torch.zeros(E), ids, dw, True, renorm, start=torch.randn(T, E, generator=g))
    if renorm and k > 1:                                 # not lost: of the size of d_w
        part = got.abs().amax(1)[:len(levels) - 1]
        assert bool((part > 1e-4).all()) and bool((part < 1.0).all())
    assert bool((got[len(levels) - 1] == 0).all())


def test_gradient_of_far_scores_against_differences():
    l = torch.randn(6, 20, generator=torch.Generator().manual_seed(1)) - 95.0
    ids = torch.arange(20).repeat(6, 1)[:, 3:8].int()
    dw = torch.randn(6, 5, generator=torch.Generator().manual_seed(2))
    got = _check_backward(l, None, ids, dw, True, True, 1.0)
    h = 1e-5
    for e in (3, 6):
        d = torch.zeros(6, 20, dtype=torch.float64)
        d[:, e] = h
        up, dn = (ref.gate_weights(l.double() + s * d, None, ids, True, True, 1.0) for s in (1, -1))
        # cubic term of the difference h^2, rounding of 64 bits 1e-16 / h
        assert bool((((up - dn) * dw.double()).sum(1) / (2 * h) - got[:, e]).abs().max() < 1e-6)


@pytest.mark.parametrize("T,E,k,groups", [(37, 384, 6, 1), (300, 256, 8, 8), (130, 1000, 16, 1), (40, 17, 5, 1),
                                          (9, 1024, 4, 16), (33, 60, 5, 4), (21, 64, 16, 1)])
def test_softmax_weights_are_rounded_once(T, E, k, groups):
    """Weights that are not renormalised, in 64 bits up to their one rounding, whichever way a token's choice was made."""
    logits, bias, g = _case(T, E, T + 3 * E, out=0.1)
    logits *= 1.0 + 3.0 * torch.rand(T, 1, generator=g)
    logits[1] = 0.25                        # equal terms: a sum of E
    logits[3, ::2] = logits[3, 0]           # ties: the choice is made in 64 bits
    logits[4] = -INF
    logits[4, 5] = 1e30
    for b in (None, bias * 0.5 / E):
        want, w = ref.gate(logits, b, k, False, groups, max(1, groups // 2), False, False, 1.5)
        r = moe.route_gated(_layer(T, E, k), _gate(False, groups, max(1, groups // 2), False, False, 1.5), logits.cuda(),
                            None if b is None else b.cuda(), permute=False)
        assert torch.equal(r["topk_ids"].cpu(), want)
        off = (r["topk_w"].cpu().double() - w).abs()
        # one rounding; of fp32's subnormal numbers half of the smallest
        worst = float((off / (w.abs() * ref.F32 * (1 + 1e-6) + 2.0 ** -150 * (1 + 1e-6))).max())
        assert worst <= 1.0


def test_softmax_weights_of_large_logits():
    """Far from 0 and far from each other: steps of fp32 between the logits from 2^-20 to more than exp's range."""
    g = torch.Generator().manual_seed(7)
    rows = [torch.randn(40, generator=g) * a + b for a in (1.0, 30.0, 300.0)
            for b in (1e3, -5e5, 2.0 ** 24, -2.0 ** 29, 2.0 ** 30, 2.0 ** 31, -1e30, 3e38)]
    rows += [torch.randn(40, generator=g) * 1e30, torch.randn(40, generator=g) * 3e9, torch.full((40,), 3.4e38)]
    logits = torch.stack(rows)
    for E in (40, 32, 16):
        l = logits[:, :E].contiguous()
        want, w = ref.gate(l, None, 6, False, 1, 1, True, False, 1.0)
        r = moe.route_gated(_layer(len(rows), E, 6), _gate(False, 1, 1, True, False, 1.0), l.cuda(), permute=False)
        assert torch.equal(r["topk_ids"].cpu(), want)
        worst = float(((r["topk_w"].cpu().double() - w).abs() / (w * ref.F32 * (1 + 1e-6) + 2.0 ** -150 * (1 + 1e-6))).max())
        assert worst <= 1.0


def _expert_inputs(T=96, H=256, I=256, E=16, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).bfloat16()
    logits = torch.randn(T, E, generator=g)
    w13, s13 = zip(*(ref.make_weights(2 * I, H, False, g) for _ in range(E)))
    w2, s2 = zip(*(ref.make_weights(H, I, False, g) for _ in range(E)))
    to = lambda t: torch.stack(t).cuda()  # noqa: E731
    scale = 0.05                          # keeps h in range
    return x.cuda(), logits.cuda(), to(w13), to(w2), to(s13) * scale, to(s2) * scale, g


def test_expert_forward_through_the_gate():
    """With a softmax gate without groups the layer's own result; with any gate, the
    combination of the experts' outputs by the gate's ids and weights."""
    T, H, I, E, k = 96, 256, 256, 16, 4
    x, logits, w13, w2, s13, s2, g = _expert_inputs(T, H, I, E)
    layer = moe.make_layer(T, H, I, E, k, moe.FMT_FP8)
    plain = moe.expert_forward(layer, x, logits, w13, w2, s13, s2, chunk_experts=4)
    same = moe.expert_forward_gated(layer, moe.make_gate(moe.GATE_SOFTMAX), x, logits, w13, w2, s13, s2,
                                    chunk_experts=4)
    # the weights agree to a few fp32 steps, the results' roundings may fall apart by one bf16 step
    torch.testing.assert_close(same.float(), plain.float(), rtol=2 ** -7, atol=1e-4 * float(plain.abs().max()))
    gate = moe.make_gate(moe.GATE_SIGMOID, 4, 2, moe.GROUP_TOP2, True, 2.5)
    bias = (torch.randn(E, generator=g) * 0.2).cuda()
    out = moe.expert_forward_gated(layer, gate, x, logits, w13, w2, s13, s2, bias, chunk_experts=4)
    r = moe.route_gated(layer, gate, logits, bias)
    # each expert's output, one expert at a time through a layer that knows only it
    one = moe.make_layer(T, H, I, 1, 1, moe.FMT_FP8)
    zero = torch.zeros(T, 1, device="cuda")
    y = torch.stack([moe.expert_forward(one, x, zero, w13[e:e + 1], w2[e:e + 1], s13[e:e + 1], s2[e:e + 1])
                     for e in range(E)])
    rows = y[r["topk_ids"].long(), torch.arange(T, device="cuda")[:, None]]      # [T][k][H]
    perm = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda")
    perm[r["row_of"].long()] = rows.reshape(T * k, H)
    want = moe.combine(layer, perm, r["topk_w"], r["row_of"])
    # the same rows, weights and order of sums; tiles of other heights may add in another order
    torch.testing.assert_close(out.float(), want.float(), rtol=2 ** -6, atol=1e-3 * float(want.abs().max()))


@pytest.mark.parametrize("sigmoid,renorm", [(True, True), (False, False), (False, True)])
def test_expert_backward_through_the_gate(sigmoid, renorm):
    T, H, I, E, k = 96, 256, 256, 16, 4
    x, logits, w13, w2, s13, s2, g = _expert_inputs(T, H, I, E, 1)
    layer = moe.make_layer(T, H, I, E, k, moe.FMT_FP8)
    d_out = torch.randn(T, H, generator=g).bfloat16().cuda()
    bw = moe.prepare_backward_weights(layer, w13, w2, s13, s2)
    args = (x, logits, w13, w2, s13, s2, bw, d_out)
    gate = _gate(sigmoid, 4, 2, True, renorm, 1.5)
    bias = (torch.randn(E, generator=g) * 0.2).cuda()
    d_x, d_l, d_a = moe.expert_backward_gated(layer, gate, *args, bias=bias, chunk_experts=4)
    assert d_a is None
    r = moe.route_gated(layer, gate, logits, bias)
    # g_tj = <d_out_t, y_tj> with the forward's own expert outputs (rounded to bf16 here)
    one = moe.make_layer(T, H, I, 1, 1, moe.FMT_FP8)
    zero = torch.zeros(T, 1, device="cuda")
    y = torch.stack([moe.expert_forward(one, x, zero, w13[e:e + 1], w2[e:e + 1], s13[e:e + 1], s2[e:e + 1])
                     for e in range(E)]).double()
    rows = y[r["topk_ids"].long(), torch.arange(T, device="cuda")[:, None]]
    dw = (rows * d_out.double()[:, None, :]).sum(2)
    mag = (rows * d_out.double()[:, None, :]).abs().sum(2)
    want, _ = ref.gate_grad(logits.cpu(), bias.cpu(), r["topk_ids"].cpu(), dw.float().cpu(), sigmoid, renorm, 1.5)
    # y and the backward's fp16 operands are each off by up to 2^-8 and 2^-11 of their terms
    s, _ = ref.gate_scores(logits.cpu(), bias.cpu(), sigmoid)
    tot = s.gather(1, r["topk_ids"].cpu().long()).sum(1, keepdim=True) if renorm else torch.ones(T, 1)
    slack = 1.5 * mag.sum(1, keepdim=True).cpu() * 2 ** -7 / tot * s
    assert bool(((d_l.cpu().double() - want).abs() <= slack + 1e-9).all())
    # d_x is linear in the weights: against the layer's own backward where the gate is its routing
    own = moe.expert_backward(layer, *args, chunk_experts=4)
    same = moe.expert_backward_gated(layer, moe.make_gate(moe.GATE_SOFTMAX), *args, chunk_experts=4)
    torch.testing.assert_close(same[0].float(), own[0].float(), rtol=2 ** -7, atol=1e-4 * float(own[0].abs().max()))
    torch.testing.assert_close(same[1], own[1], rtol=1e-3, atol=1e-4 * float(own[1].abs().max()))


def test_empty_and_refused():
    layer = _layer(0, 32, 4)
    r = moe.route_gated(layer, moe.make_gate(), torch.empty(0, 32, device="cuda"))
    assert r["topk_ids"].shape == (0, 4)
    d = moe.route_gated_backward(layer, moe.make_gate(), torch.empty(0, 32, device="cuda"), r["topk_ids"],
                                 r["topk_w"])
    assert d.shape == (0, 32)
    layer, l = _layer(4, 32, 4), torch.zeros(4, 32, device="cuda")
    with pytest.raises(ValueError):
        moe.route_gated(layer, moe.make_gate(), l.double())
    with pytest.raises(ValueError):
        moe.route_gated(layer, moe.make_gate(), l, torch.zeros(31, device="cuda"))
    with pytest.raises(ValueError):
        moe.route_gated(layer, moe.make_gate(), l[:, ::2])
    with pytest.raises(binding.MoeError):
        moe.route_gated(layer, moe.make_gate(groups=5), l)
