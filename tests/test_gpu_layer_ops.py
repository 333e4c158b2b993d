"""The gate, the FP8 projection and the clip as a layer uses them: a training step
around frozen experts, decoding through a graph, streams side by side."""
import pytest
import torch

import precision_moe_expert_amd as moe
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu
T, H, I, E, K, S = 200, 512, 256, 16, 4, 384     # S: the shared expert's width


class Layer:
    """Frozen experts, a trained router and a trained shared expert in FP8."""

    def __init__(self, seed=0, pow2=False):
        g = torch.Generator().manual_seed(seed)
        fmt = moe.FMT_FP8_POW2 if pow2 else moe.FMT_FP8
        self.fmt = fmt
        many = lambda N, K: [torch.stack(v).cuda() for v in zip(*(ref.make_weights(N, K, pow2, g) for _ in range(E)))]  # noqa: E731
        (self.w13, s13), (self.w2, s2) = many(2 * I, H), many(H, I)
        self.s13, self.s2 = s13 / 16, s2 / 16
        self.u, us = ref.make_weights(2 * S, H, pow2, g, "cuda")
        self.d, ds = ref.make_weights(H, S, pow2, g, "cuda")
        self.us, self.ds = us / 16, ds / 16
        self.ut, self.dt = moe.fp8_linear_transpose(self.u, self.us), moe.fp8_linear_transpose(self.d, self.ds)
        self.router = (torch.randn(E, H, generator=g) / H ** 0.5).cuda()
        self.bias = (torch.randn(E, generator=g) * 0.1).cuda()
        self.gate = moe.make_gate(moe.GATE_SIGMOID, 4, 2, moe.GROUP_TOP2, True, 2.5)
        self.g = g

    def layer(self, n):
        return moe.make_layer(n, H, I, E, K, self.fmt)

    def experts(self):
        return self.w13, self.w2, self.s13, self.s2

    def inputs(self, n):
        x = torch.randn(n, H, generator=self.g).bfloat16().cuda()
        return x, x.float() @ self.router.t(), torch.randn(n, H, generator=self.g).bfloat16().cuda()

    def forward(self, x, logits):
        routed = moe.expert_forward_gated(self.layer(len(x)), self.gate, x, logits, *self.experts(), self.bias,
                                          chunk_experts=8)
        u = moe.fp8_linear(x, self.u, self.us, self.fmt)
        h = swiglu(u)
        return routed, u, h, moe.fp8_linear(h, self.d, self.ds, self.fmt)

    def backward(self, x, logits, u, h, d_out, bw, limit):
        layer = self.layer(len(x))
        d_x, d_logits, _ = moe.expert_backward_gated(layer, self.gate, x, logits, *self.experts(), bw, d_out,
                                                     self.bias, chunk_experts=8)
        r = moe.route_gated(layer, self.gate, logits, self.bias, permute=False)
        bal, counts, tokens, _ = moe.balance_loss(layer, logits, r["topk_ids"])
        moe.balance_loss_backward(layer, logits, counts, tokens, torch.full_like(bal, 0.01), d_logits=d_logits)
        d_h, d_wd = moe.fp8_linear_backward(d_out, *self.dt, self.fmt, x=h, weight_grad=True)
        d_u = swiglu_grad(u, d_h)
        d_xs, d_wu = moe.fp8_linear_backward(d_u, *self.ut, self.fmt, x=x, weight_grad=True)
        raw = (d_logits.clone(), d_wu.clone(), d_wd.clone())
        norm = moe.clip_grads([d_logits, d_wu, d_wd], limit)
        return dict(d_x=d_x, d_xs=d_xs, d_h=d_h, d_u=d_u, d_logits=d_logits, d_wu=d_wu, d_wd=d_wd, norm=norm,
                    raw=raw, ids=r["topk_ids"], counts=counts)


def swiglu(u):
    a, b = u.float().chunk(2, 1)
    return (a * torch.sigmoid(a) * b).bfloat16()


def swiglu_grad(u, d_h):
    a, b = u.float().chunk(2, 1)
    s, d = torch.sigmoid(a), d_h.float()
    return torch.cat([d * b * s * (1 + a * (1 - s)), d * a * s], 1).bfloat16()


def _near(got, want, bound):
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())


@pytest.mark.parametrize("pow2", [False, True])
def test_a_training_step(pow2):
    L = Layer(1, pow2)
    x, logits, d_out = L.inputs(T)
    bw = moe.prepare_backward_weights(L.layer(T), *L.experts())
    routed, u, h, shared = L.forward(x, logits)
    g = L.backward(x, logits, u, h, d_out, bw, 0.5)
    # the shared expert, product by product on what each was given
    wu, wd = ref.weights(L.u, L.us), ref.weights(L.d, L.ds)
    q = lambda v, axis: ref.quantized(v, axis, pow2)  # noqa: E731
    _near(u, *ref.product(q(x, 1), wu))
    _near(shared, *ref.product(q(h, 1), wd))
    _near(g["d_h"], *ref.product(q(d_out, 1), wd.T))
    _near(g["d_xs"], *ref.product(q(g["d_u"], 1), wu.T))
    raw_l, raw_u, raw_d = g["raw"]
    _near(raw_d, *ref.product(q(d_out, 0).T, q(h, 0).T))
    _near(raw_u, *ref.product(q(g["d_u"], 0).T, q(x, 0).T))
    # the routing, and its gradient with the balance loss's on top
    ids, _ = ref.gate(logits.cpu(), L.bias.cpu(), K, True, 4, 2, True, True, 2.5)
    assert torch.equal(g["ids"].cpu(), ids)
    assert torch.equal(g["counts"][0].cpu().long(), torch.bincount(ids.flatten().long(), minlength=E))
    alone = moe.expert_backward_gated(L.layer(T), L.gate, x, logits, *L.experts(), bw, d_out, L.bias,
                                      chunk_experts=8)[1]
    p = torch.softmax(logits.double(), 1)
    a = 0.01 * E / (K * T * T) * g["counts"].double()
    want = alone.double() + p * (a - (p * a).sum(1, keepdim=True))
    # two fp32 results added: a rounding of each and of the sum, and the balance gradient's own few
    assert bool(((raw_l.double() - want).abs() <= 40 * ref.F32 * (want.abs() + p * a.amax())).all())
    # the clip of all three
    total = sum(float(t.double().square().sum()) for t in g["raw"]) ** 0.5
    assert total > 0.5 and abs(float(g["norm"]) - total) <= 1.01 * ref.F32 * total
    for raw, name in zip(g["raw"], ("d_logits", "d_wu", "d_wd")):
        w = raw.double() * (0.5 / total)
        assert bool(((g[name].double() - w).abs() <= w.abs() * (ref.HALF[raw.dtype] + 2.01 * ref.F32) + 1e-44).all())
    assert routed.shape == shared.shape == (T, H)


def _flat(r):
    return [t for v in r.values() for t in (v if isinstance(v, tuple) else (v,))]


def test_a_training_step_in_a_graph():
    """Captured once, replayed on new inputs with eager steps in between."""
    L = Layer(2)
    x, logits, d_out = L.inputs(T)
    bw = moe.prepare_backward_weights(L.layer(T), *L.experts())

    def step():
        routed, u, h, shared = L.forward(x, logits)
        return dict(routed=routed, shared=shared, **L.backward(x, logits, u, h, d_out, bw, 0.5))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(4):
        for dst, src in zip((x, logits, d_out), L.inputs(T)):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in _flat(out)]
        for a, b in zip(got, _flat(step())):
            assert torch.equal(a, b)


@pytest.mark.parametrize("n", [1, 3, 20])
def test_decoding_in_a_graph(n):
    L = Layer(3)
    x, logits, _ = L.inputs(n)
    L.forward(x, logits)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = L.forward(x, logits)
    for _ in range(4):
        for dst, src in zip((x, logits), L.inputs(n)):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, L.forward(x, logits)):
            assert torch.equal(a, b)


def test_streams_side_by_side():
    """Calls on two streams, each with its own workspaces, give what they give one after the other."""
    L = Layer(4)
    bw = moe.prepare_backward_weights(L.layer(T), *L.experts())
    sets = [L.inputs(T) for _ in range(2)]

    def step(x, logits, d_out):
        routed, u, h, shared = L.forward(x, logits)
        return _flat(dict(routed=routed, shared=shared, **L.backward(x, logits, u, h, d_out, bw, 0.5)))

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None, None]
    for _ in range(3):
        for i, (stream, s) in enumerate(zip(streams, sets)):
            with torch.cuda.stream(stream):
                got[i] = step(*s)
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_given_workspaces():
    """One workspace handed from call to call, its contents left over from the last, gives the same results."""
    L = Layer(5)
    x, logits, d_out = L.inputs(T)
    big = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    layer = L.layer(T)
    r0 = moe.route_gated(layer, L.gate, logits, L.bias)
    r1 = moe.route_gated(layer, L.gate, logits, L.bias, ws=big)
    n = int(r0["num_active"][0])
    for name in r0:
        a, b = (v[name][:n] if name == "active_experts" else v[name][:1] if name == "num_active" else v[name]
                for v in (r0, r1))
        assert torch.equal(a, b), name
    y = moe.fp8_linear(x, L.u, L.us)
    assert torch.equal(moe.fp8_linear(x, L.u, L.us, ws=big), y)
    a = moe.fp8_linear_backward(y, *L.ut, x=x, weight_grad=True)
    b = moe.fp8_linear_backward(y, *L.ut, x=x, weight_grad=True, ws=big)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(moe.grad_norm([x, y]), moe.grad_norm([x, y], ws=big))
    f = moe.expert_forward_gated(layer, L.gate, x, logits, *L.experts(), L.bias, chunk_experts=3)
    assert torch.equal(moe.expert_forward_gated(layer, L.gate, x, logits, *L.experts(), L.bias, chunk_experts=16,
                                                ws=big), f)
