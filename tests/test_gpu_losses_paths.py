"""GPU parity of the training losses at sizes and in uses that take their less common paths: widths past 8192, token
lists past 8192, vocabularies in pieces, strided rows whose sum is split, calls at once and replayed."""
import math

import pytest
import torch

import precision_moe_expert_amd as moe
from tests import loss_ref as lr

pytestmark = pytest.mark.gpu


def _close(got, want, bound, label):
    err = (got.double() - want).abs()
    bad = ~(err <= bound + 1e-30)
    assert not bad.any(), (label, int(bad.sum()), float((err / (bound + 1e-30)).max()))


def _inputs(T, H, V, ignored=0.2, K=0, hot=0.0):
    """hot: share of the ids that are one of three."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T + H + V + K)
    h = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w = (torch.randn(V, H, generator=g, device="cuda") * 2.5 / math.sqrt(H)).bfloat16()
    shape = (T, K) if K else (T,)
    ids = torch.randint(0, V, shape, generator=g, device="cuda")
    near = torch.randint(0, 3, shape, generator=g, device="cuda") * (V // 3)
    ids = torch.where(torch.rand(shape, generator=g, device="cuda") < hot, near, ids)
    drop = torch.rand(T, generator=g, device="cuda") < ignored
    ids = torch.where(drop[:, None] if K else drop, -100, ids).int()
    return h, w, ids, torch.randn(T, K or 1, generator=g, device="cuda"), torch.randn(T, generator=g, device="cuda")


def _check_ce(T, H, V, ignored=0.2, hot=0.0):
    h, w, y, _, dl = _inputs(T, H, V, ignored, 0, hot)
    ref = lr.ce_ref(h, w, y)
    lse, want, b_lse, b_loss = ref.loss()
    loss, got_lse = moe.lm_head_loss(h, w, y)
    _close(got_lse, lse, b_lse, "lse")
    _close(loss, want, b_loss, "loss")
    got = moe.lm_head_loss_backward(h, w, y, loss, got_lse, dl, weight_grad=True)
    d_h, b_h, d_w, b_w = ref.grads(dl, True)
    _close(got[0], d_h, b_h, "d_h")
    _close(got[1], d_w, b_w, "d_w")
    again = moe.lm_head_loss_backward(h, w, y, loss, got_lse, dl, weight_grad=True)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert torch.equal(moe.lm_head_loss_backward(h, w, y, loss, got_lse, dl)[0].double().isfinite(),
                       torch.ones_like(got[0], dtype=torch.bool))


def _check_distill(T, H, V, K, ignored=0.2, hot=0.0):
    h, w, ids, tl, dl = _inputs(T, H, V, ignored, K, hot)
    ref, have, q = lr.distill_ref(h, w, ids, tl)
    lse, want, logp, b_lse, b_loss, b_logp = lr.distill_loss(ref, ids, have, q)
    loss, got_lse, got_logp = moe.lm_head_distill(h, w, ids, tl)
    _close(got_lse, lse, b_lse, "lse")
    _close(got_logp, logp, b_logp, "logp")
    _close(loss, want, b_loss, "loss")
    got = moe.lm_head_distill_backward(h, w, ids, tl, got_lse, got_logp, dl, weight_grad=True)
    d_h, b_h, d_w, b_w = ref.grads(dl, True)
    _close(got[0], d_h, b_h, "d_h")
    _close(got[1], d_w, b_w, "d_w")
    again = moe.lm_head_distill_backward(h, w, ids, tl, got_lse, got_logp, dl, weight_grad=True)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("T,H,V", [(5, 8200, 300), (70, 12288, 513), (3, 32768, 129), (600, 9000, 200)])
def test_wide_hidden(torch_gpu, T, H, V):
    _check_ce(T, H, V)
    _check_distill(T, H, V, 5)


@pytest.mark.parametrize("T,H,V,hot", [(8193, 64, 300, 0.0), (17001, 72, 500, 0.3), (66000, 64, 200, 0.05)])
def test_many_tokens(torch_gpu, T, H, V, hot):
    """Token lists of more than one round, more than 65536 targets."""
    _check_ce(T, H, V, 0.3, hot)
    _check_distill(T, H, V, 3, 0.3, hot)


@pytest.mark.parametrize("kind", ["ce", "distill"])
def test_pieces_of_a_trained_head(torch_gpu, kind):
    """Both products of a piece in one launch, for more than one piece, with ids that many tokens share."""
    T, H, V = 8192, 2048, 50257
    if kind == "ce":
        _check_ce(T, H, V, 0.05, 0.3)
    else:
        _check_distill(T, H, V, 33, 0.05, 0.3)


@pytest.mark.parametrize("T,H,V,K", [(1025, 64, 20000, 4), (1500, 136, 9000, 2), (2000, 72, 257, 1), (40, 520, 4000, 40),
                                     (1024, 64, 5000, 5)])
def test_shared_ids(torch_gpu, T, H, V, K):
    """Most slots on three ids, several of them in one token: few ids with hundreds of tokens each."""
    _check_distill(T, H, V, K, 0.1, 0.9)


@pytest.mark.parametrize("T,H,V", [(64, 7168, 2049), (2, 6488, 1118), (257, 4096, 501), (900, 2048, 130)])
def test_split_rows_strided(torch_gpu, T, H, V):
    """Sums over H that are split between workgroups, on rows of wider matrices."""
    h, w, y, _, dl = _inputs(T, H, V)
    hw = torch.full((T, H + 24), math.nan, device="cuda").bfloat16()
    ww = torch.full((V, H + 8), math.nan, device="cuda").bfloat16()
    hw[:, 8:8 + H], ww[:, :H] = h, w
    hs, ws = hw[:, 8:8 + H], ww[:, :H]
    loss, lse = moe.lm_head_loss(h, w, y)
    assert all(torch.equal(a, b) for a, b in zip((loss, lse), moe.lm_head_loss(hs, ws, y)))
    for a, b in zip(moe.lm_head_loss_backward(h, w, y, loss, lse, dl, weight_grad=True),
                    moe.lm_head_loss_backward(hs, ws, y, loss, lse, dl, weight_grad=True)):
        assert torch.equal(a, b)


def test_no_token_counts(torch_gpu):
    for T in (40, 1000, 1100, 9000):
        h, w, y, _, dl = _inputs(T, 64, 700, 2.0)
        h[:] = math.nan
        loss, lse = moe.lm_head_loss(h, w, y)
        for t in (loss, lse, *moe.lm_head_loss_backward(h, w, y, loss, lse, dl, weight_grad=True)):
            assert (t == 0).all()
        ids, tl = y[:, None].expand(T, 3).contiguous(), torch.randn(T, 3, device="cuda")
        kl, lse, logp = moe.lm_head_distill(h, w, ids, tl)
        for t in (kl, lse, logp, *moe.lm_head_distill_backward(h, w, ids, tl, lse, logp, dl, weight_grad=True)):
            assert (t == 0).all()


def _all(ce, kl, bal):
    """Losses and gradients of the three operators."""
    h, w, y, _, dl = ce
    loss, lse = moe.lm_head_loss(h, w, y)
    out = [loss, lse, *moe.lm_head_loss_backward(h, w, y, loss, lse, dl, weight_grad=True)]
    h, w, ids, tl, dl = kl
    k, klse, logp = moe.lm_head_distill(h, w, ids, tl)
    out += [k, klse, logp, *moe.lm_head_distill_backward(h, w, ids, tl, klse, logp, dl, weight_grad=True)]
    layer, logits, top, off, g = bal
    b, counts, tokens, probs = moe.balance_loss(layer, logits, top, seg_offsets=off)
    return out + [b, counts, tokens, probs, moe.balance_loss_backward(layer, logits, counts, tokens, g, seg_offsets=off)]


def _sets(T, seed):
    torch.manual_seed(seed)
    logits = torch.randn(T, 96, device="cuda")
    bal = (moe.make_layer(T, 256, 128, 96, 3, moe.FMT_INT4), logits, torch.topk(logits, 3, 1).indices.int(),
           torch.tensor([0, T // 3, T // 3, T], device="cuda").int(), torch.randn(3, device="cuda"))
    return _inputs(T, 256, 3000 + seed, 0.2, 0, 0.2), _inputs(T, 192, 9000 + seed, 0.2, 6, 0.2), bal


def test_streams_against_serial(torch_gpu):
    """All operators on two streams at once, each call with its own workspace, against the calls made alone."""
    sets = [_sets(1400, 1), _sets(300, 2)]
    want = []
    for s in sets:
        want.append(_all(*s))
        torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], [[], []]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for i, s in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                got[i].append(_all(*s))
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            for a, b in zip(out, want[i]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("T", [300, 1400])
def test_captured_gradients_replay_on_new_inputs(torch_gpu, T):
    a, b = _sets(T, 3), _sets(T, 4)
    b = tuple(tuple(x[:y.shape[0]] if torch.is_tensor(x) and x.shape != y.shape else x for x, y in zip(p, q))
              for p, q in zip(b, a))
    for p in b[:2]:  # ids of the smaller vocabulary
        p[2].clamp_(max=2999)
    want = []
    for s in (a, b):
        want.append([t.clone() for t in _all(*s)])
    hold = tuple(tuple(x.clone() if torch.is_tensor(x) else x for x in p) for p in a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _all(*hold)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _all(*hold)
    for i in (1, 0, 1, 1, 0):
        for p, q in zip(hold, (a, b)[i]):
            for x, y in zip(p, q):
                if torch.is_tensor(x):
                    x.copy_(y)
        graph.replay()
        junk = torch.randn(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        assert junk.isfinite()
        for x, y in zip(out, want[i]):
            assert torch.equal(x, y)
