"""Timed cases of the layer around the experts: the gate (scores, balance bias,
groups, top-k) with its gradient, the dense FP8 projection with a scale per
block of 128 with its gradients, and the clip of a list of gradients by their
global norm.

`run` computes a case in plain torch operations, or, where `own` is set, with
the library's entry points.  `exact` gives the same outputs from the
definitions in 64 bits.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0


def listed():
    return [
        # one generated token through a sigmoid gate with groups: call latency
        dict(name="gate fwd 1 token", op="gate", dir="fwd", T=1, E=256, k=8, score="sigmoid", groups=8, top_groups=4,
             top2=True, renorm=True, bias=True, out=0.0),
        # the training batch through the same gate
        dict(name="gate fwd 16384 groups", op="gate", dir="fwd", T=16384, E=256, k=8, score="sigmoid", groups=8,
             top_groups=4, top2=True, renorm=True, bias=True, out=0.0),
        # a batch with odd counts, softmax scores, some experts out of service
        dict(name="gate fwd 5001 softmax", op="gate", dir="fwd", T=5001, E=384, k=6, score="softmax", groups=1,
             top_groups=1, top2=False, renorm=False, bias=True, out=0.05),
        # gradient of a small batch
        dict(name="gate bwd 64", op="gate", dir="bwd", T=64, E=384, k=8, score="sigmoid", groups=1, top_groups=1,
             top2=False, renorm=True, bias=True, out=0.0),
        # gradient of a training batch, softmax without renormalisation: every logit has one
        dict(name="gate bwd 32768 softmax", op="gate", dir="bwd", T=32768, E=256, k=6, score="softmax", groups=8,
             top_groups=3, top2=False, renorm=False, bias=False, out=0.0),
        # one generated token through the gate/up rows of a shared expert: the weight stream
        dict(name="fp8 fwd 1 token", op="fp8", dir="fwd", M=1, K=7168, N=4096, pow2=False, dw=False),
        # the decode batch through its down projection
        dict(name="fp8 fwd 64 tokens", op="fp8", dir="fwd", M=64, K=2048, N=7168, pow2=False, dw=False),
        # a training batch, power-of-two scales
        dict(name="fp8 fwd 4096 pow2", op="fp8", dir="fwd", M=4096, K=7168, N=4096, pow2=True, dw=False),
        # an odd batch through a frozen projection whose sizes end inside a block
        dict(name="fp8 bwd 3001 frozen", op="fp8", dir="bwd", M=3001, K=7168, N=4160, pow2=False, dw=False),
        # the training batch through a trained projection: the largest products
        dict(name="fp8 bwd 8192 trained", op="fp8", dir="bwd", M=8192, K=7168, N=4096, pow2=False, dw=True),
        # an adapter's and a router's gradients: call latency
        dict(name="clip adapter", op="clip", count=3, largest=256 * 7168, bf16=0.0, pick=1),
        # a head's, its router's and many adapters' gradients, two types
        dict(name="clip head and adapters", op="clip", count=48, largest=32000 * 7168, bf16=0.5, pick=2),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gate", "gate", "fp8", "fp8", "clip"])
    if op == "clip":
        return dict(op=op, count=_log_int(rng, 1, 60), largest=_log_int(rng, 1000, 1 << 26),
                    bf16=rng.choice([0.0, 0.3, 1.0]), pick=rng.randrange(1 << 30))
    d = rng.choice(["fwd", "bwd"])
    if op == "gate":
        T = _log_int(rng, 1, 32768)
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log_int(rng, max(1, 8 // groups), 384 // groups)
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(8, top_groups * (E // groups)))
        return dict(op=op, dir=d, T=T, E=E, k=k, score=rng.choice(["softmax", "sigmoid"]), groups=groups,
                    top_groups=top_groups, top2=rng.random() < 0.5, renorm=rng.random() < 0.6,
                    bias=rng.random() < 0.7, out=rng.choice([0.0, 0.0, 0.1]))
    while True:
        M, K, N = _log_int(rng, 1, 8192), 16 * _log_int(rng, 8, 1152), 16 * _log_int(rng, 8, 1152)
        if M * K * N <= 8192 * 7168 * 4096 and K * N <= 7168 * 18432:
            break
    return dict(op=op, dir=d, M=M, K=K, N=N, pow2=rng.random() < 0.4, dw=d == "bwd" and rng.random() < 0.5)


def _sizes(case):
    """(elements, whether bf16) of each tensor of a clip case: the largest first, the others far smaller."""
    rng = random.Random(case["pick"])
    n, top = case["count"], case["largest"]
    sizes = [top] + [_log_int(rng, 1, max(1, min(top, 1 << 20))) for _ in range(n - 1)]
    return [(m, (i + 0.5) / n < case["bf16"]) for i, m in enumerate(sizes)]


# ---- inputs -----------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "gate":
        return _prepare_gate(case, g)
    if case["op"] == "clip":
        grads = [torch.randn(n, generator=g, device="cuda") * 10 ** (-2 - i % 3) for i, (n, _) in
                 enumerate(_sizes(case))]
        grads = [t.bfloat16() if b else t for t, (_, b) in zip(grads, _sizes(case))]
        # a norm of a third to three times the limit, or about, as training has it
        norm = math.sqrt(sum(float(t.double().square().sum()) for t in grads))
        limit = norm * (0.3 + 0.6 * float(torch.rand(1, generator=g, device="cuda")))
        return dict(case=case, grads=grads, outs=[torch.empty_like(t) for t in grads], limit=limit)
    return _prepare_fp8(case, g)


def _prepare_gate(case, g):
    T, E, k = case["T"], case["E"], case["k"]
    # a skewed router: a per-expert preference on top of the token's logits
    logits = torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")
    bias = None
    if case["bias"] or case["out"] > 0:
        size = 0.1 if case["score"] == "sigmoid" else 0.5 / E
        bias = torch.randn(E, generator=g, device="cuda") * (size if case["bias"] else 0.0)
        # experts out of service
        bias[torch.randperm(E, generator=g, device="cuda")[:int(E * case["out"])]] = -math.inf
    s = dict(case=case, logits=logits, bias=bias, scale=2.5 if case["renorm"] else 1.0)
    if case["dir"] == "bwd":
        s["ids"] = _choose(case, logits, bias)[0].int()
        s["d_w"] = torch.randn(T, k, generator=g, device="cuda") * 0.01
    return s


def _prepare_fp8(case, g):
    M, K, N = case["M"], case["K"], case["N"]
    w = torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K)
    w *= torch.exp(0.5 * torch.randn(N, 1, generator=g, device="cuda"))     # rows of different sizes
    codes, scales = _quantize_weights(w, case["pow2"])
    # activations with a few loud channels, as a residual stream has them
    x = torch.randn(M, K, generator=g, device="cuda")
    x[:, torch.randperm(K, generator=g, device="cuda")[:max(1, K // 256)]] *= 20.0
    s = dict(case=case, w=codes, ws=scales, x=x.bfloat16())
    if case["dir"] == "bwd":
        d_y = torch.randn(M, N, generator=g, device="cuda") * 1e-3
        d_y *= torch.exp(torch.randn(M, 1, generator=g, device="cuda"))
        d_y[torch.rand(M, generator=g, device="cuda") < 0.05] = 0.0          # padded tokens
        s["d_y"] = d_y.bfloat16()
        s["wt"], s["wts"] = codes.view(torch.uint8).t().contiguous(), scales.t().contiguous()
    return s


def _blocks(v, axis):
    """v with `axis` cut into blocks of 128, zeros behind its end."""
    n = v.shape[axis]
    pad = -n % 128
    if pad:
        shape = list(v.shape)
        shape[axis] = pad
        v = torch.cat([v, v.new_zeros(shape)], axis)
    return v.unflatten(axis, (-1, 128))


def _scale_of(amax, pow2):
    """amax / 448 rounded once to 32 bits, or the power of two at or above it; 1 for a block of zeros."""
    s = (amax.double() / E4M3_MAX).float()
    if pow2:
        m, e = torch.frexp(s)
        s = torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))
    return torch.where(amax > 0, s, torch.ones_like(s))


def _codes(v, s):
    """Codes of v / s, the quotient rounded once to 32 bits, then to e4m3."""
    return (v.double() / s.double()).float().clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _quantize_weights(w, pow2):
    N, K = w.shape
    b = _blocks(_blocks(w, 1), 0)                                   # [N/128][128][K/128][128]
    s = _scale_of(b.abs().amax((1, 3)), pow2)
    codes = _codes(b, s[:, None, :, None]).view(torch.uint8).flatten(2, 3).flatten(0, 1)[:N, :K].contiguous()
    return codes, s


# ---- plain form -------------------------------------------------------------

def _out(logits, bias):
    """Where an expert takes no part."""
    o = torch.isnan(logits) | (logits == -math.inf)
    return o if bias is None else o | (torch.isnan(bias) | (bias == -math.inf))[None, :]


def _scores(case, l, bias):
    """Scores of l, in l's precision."""
    out = _out(l, bias)
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        v = torch.where(out, -math.inf, l)
        m = v.amax(1, keepdim=True)
        e = torch.where(v == m, 1.0, torch.exp(v - m))
        e = torch.where(out, 0.0, e)
        t = e.sum(1, keepdim=True)
        s = e / torch.where(t > 0, t, 1.0)
    return torch.where(out, 0.0, s)


def _top(v, k):
    """The k largest of each row, ties to the lowest index: a stable sort."""
    return torch.sort(v, dim=1, descending=True, stable=True).indices[:, :k]


def _choose(case, logits, bias):
    """(ids [T][k], scores at ids), in 64 bits: values next to each other decide whole numbers."""
    T, E, G = case["T"], case["E"], case["groups"]
    s, dead = _scores(case, logits.double(), bias), _out(logits, bias)
    c = torch.where(dead, -math.inf, s if bias is None else s + bias.double())
    if G > 1:
        v = c.view(T, G, E // G).sort(2, descending=True).values
        top = v[..., 0]
        if case["top2"] and E // G > 1:
            top = torch.where(v[..., 1] > -math.inf, top + v[..., 1], top)
        chosen = torch.zeros(T, G, dtype=torch.bool, device=s.device).scatter_(1, _top(top, case["top_groups"]), True)
        # experts of other groups come after those that are out
        c = torch.where(chosen.repeat_interleave(E // G, 1), torch.where(dead, -1e300, c), -math.inf)
    ids = _top(c, case["k"])
    return ids, s.gather(1, ids)


def _plain_gate(s):
    c, bias = s["case"], s["bias"]
    if c["dir"] == "fwd":
        ids, w = _choose(c, s["logits"], bias)
        if c["renorm"]:
            t = w.sum(1, keepdim=True)
            w = w / torch.where(t > 0, t, 1.0)
        return dict(ids=ids.int(), w=(w * s["scale"]).float())
    p = _scores(c, s["logits"], bias)
    ids = s["ids"].long()
    at = p.gather(1, ids)
    d = s["d_w"] * s["scale"]
    if c["renorm"]:
        t = at.sum(1, keepdim=True)
        t = torch.where(t > 0, t, 1.0)
        d = (d - (d * at).sum(1, keepdim=True) / t) / t
    ds = torch.zeros_like(p).scatter_(1, ids, d)
    if c["score"] == "sigmoid":
        e = torch.exp(-s["logits"].abs())
        return dict(d_logits=torch.where(_out(s["logits"], bias), 0.0, ds * e / ((1 + e) * (1 + e))))
    return dict(d_logits=p * (ds - (ds * p).sum(1, keepdim=True)))


def _rounded(v, axis, pow2):
    """v as its e4m3 codes stand for it, a scale per 128 along `axis`."""
    b = _blocks(v.float(), axis)
    s = _scale_of(b.abs().amax(axis + 1, keepdim=True), pow2)
    return (_codes(b, s).float() * s).flatten(axis, axis + 1).narrow(axis, 0, v.shape[axis])


def _weights(codes, scales):
    N, K = codes.shape
    full = scales.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return codes.view(torch.float8_e4m3fn).float() * full


def _plain_fp8(s):
    c = s["case"]
    if c["dir"] == "fwd":
        return dict(y=(_rounded(s["x"], 1, c["pow2"]) @ _weights(s["w"], s["ws"]).t()).bfloat16())
    d_x = (_rounded(s["d_y"], 1, c["pow2"]) @ _weights(s["w"], s["ws"])).bfloat16()
    d_w = None
    if c["dw"]:
        d_w = (_rounded(s["d_y"], 0, c["pow2"]).t() @ _rounded(s["x"], 0, c["pow2"])).bfloat16()
    return dict(d_x=d_x, d_w=d_w)


def _plain_clip(s):
    # squares in 64 bits: 32 overflow for large gradients and lose small ones in long sums
    norm = torch.sqrt(torch.stack([t.double().square().sum() for t in s["grads"]]).sum())
    c = torch.where((norm > s["limit"]) & torch.isfinite(norm), s["limit"] / norm, 1.0).float()
    return dict(norm=norm.float().reshape(1), outs=[(t.float() * c).to(t.dtype) for t in s["grads"]])


# ---- the library's calls ----------------------------------------------------

def _own(s):
    import precision_moe_expert_amd as moe
    c = s["case"]
    if c["op"] == "gate":
        layer = moe.make_layer(c["T"], 256, 128, c["E"], c["k"], moe.FMT_FP8)
        gate = moe.make_gate(moe.GATE_SIGMOID if c["score"] == "sigmoid" else moe.GATE_SOFTMAX, groups=c["groups"],
                             top_groups=c["top_groups"],
                             group_score=moe.GROUP_TOP2 if c["top2"] else moe.GROUP_MAX, renormalize=c["renorm"],
                             scale=s["scale"])
        if c["dir"] == "fwd":
            r = moe.route_gated(layer, gate, s["logits"], bias=s["bias"], permute=False)
            return dict(ids=r["topk_ids"], w=r["topk_w"])
        return dict(d_logits=moe.route_gated_backward(layer, gate, s["logits"], s["ids"], s["d_w"], bias=s["bias"]))
    if c["op"] == "fp8":
        fmt = moe.FMT_FP8_POW2 if c["pow2"] else moe.FMT_FP8
        if c["dir"] == "fwd":
            return dict(y=moe.fp8_linear(s["x"], s["w"], s["ws"], fmt))
        d_x, d_w = moe.fp8_linear_backward(s["d_y"], s["wt"], s["wts"], fmt, x=s["x"] if c["dw"] else None,
                                           weight_grad=c["dw"])
        return dict(d_x=d_x, d_w=d_w)
    norm = moe.clip_grads(s["grads"], s["limit"], out=s["outs"])
    return dict(norm=norm, outs=s["outs"])


def run(state):
    if own:
        return _own(state)
    return {"gate": _plain_gate, "fp8": _plain_fp8, "clip": _plain_clip}[state["case"]["op"]](state)


def work(case):
    if case["op"] == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        bias = E * 4 if case["bias"] or case["out"] > 0 else 0
        if case["dir"] == "fwd":
            return dict(bytes=T * E * 4 + T * k * 8 + bias, flops=6 * T * E)
        return dict(bytes=2 * T * E * 4 + T * k * 8 + bias, flops=9 * T * E)
    if case["op"] == "clip":
        total = sum(n * (2 if b else 4) for n, b in _sizes(case))
        return dict(bytes=2 * total + 4, flops=3 * sum(n for n, _ in _sizes(case)))
    M, K, N = case["M"], case["K"], case["N"]
    scales = -(-N // 128) * -(-K // 128) * 4
    nbytes = N * K + scales + M * K * 2 + M * N * 2
    if case["dw"]:
        nbytes += N * K * 2 + M * K * 2
    return dict(bytes=nbytes, flops=(4 if case["dw"] else 2) * M * K * N)


# ---- the definitions in 64 bits ---------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        flat = [t.double() for t in s["grads"]]
        norm = math.sqrt(math.fsum(float(t.dot(t)) for t in flat))
        c = s["limit"] / norm if norm > s["limit"] else 1.0
        return dict(norm=torch.tensor([norm], dtype=torch.float64, device="cuda"), outs=[t * c for t in flat])
    if case["op"] == "gate":
        return _exact_gate(case, s)
    return _exact_fp8(case, s)


def _exact_gate(case, s):
    T, E, G, k = case["T"], case["E"], case["groups"], case["k"]
    l = s["logits"].double()
    b = torch.zeros(E, dtype=torch.float64, device="cuda") if s["bias"] is None else s["bias"].double()
    lm = l.masked_fill((b == -math.inf)[None, :], -math.inf)
    p = torch.sigmoid(lm) if case["score"] == "sigmoid" else torch.softmax(lm, 1)
    if case["dir"] == "fwd":
        v = p + b
        if G > 1:
            per = v.reshape(T, G, E // G)
            n = min(2 if case["top2"] else 1, E // G)
            top = torch.topk(per, n, dim=2).values
            worth = torch.where(torch.isinf(top), 0.0, top).sum(2).masked_fill(torch.isinf(top[..., 0]), -math.inf)
            rank = torch.argsort(torch.argsort(-worth, dim=1, stable=True), dim=1, stable=True)
            # an expert out of a chosen group still comes before any of another group
            v = torch.where(torch.isinf(per), -1e6, per)
            v = v.masked_fill((rank >= case["top_groups"])[..., None], -1e9).reshape(T, E)
        ids = torch.argsort(-v, dim=1, stable=True)[:, :k]
        w = torch.take_along_dim(p, ids, 1) * s["scale"]
        if case["renorm"]:
            w = w / (w.sum(1, keepdim=True) / s["scale"]).clamp_min(1e-300)
        return dict(ids=None, w=w)
    hot = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_(1, s["ids"].long(), 1.0)
    d = torch.zeros_like(hot).scatter_(1, s["ids"].long(), s["d_w"].double() * s["scale"])
    if case["renorm"]:
        t = (p * hot).sum(1, keepdim=True).clamp_min(1e-300)
        d = hot * (d / t - (d * p).sum(1, keepdim=True) / t ** 2)
    if case["score"] == "sigmoid":
        return dict(d_logits=d * p * torch.sigmoid(-lm))
    return dict(d_logits=p * d - p * (p * d).sum(1, keepdim=True))


def _exact_codes(v, axis, pow2):
    """The values of v's codes in 64 bits, rounded to e4m3 by arithmetic."""
    v = v.double().transpose(axis, -1)
    n = v.shape[-1]
    res = torch.empty_like(v)
    for at in range(0, n, 128):
        part = v[..., at:at + 128]
        big = part.abs().amax(-1, keepdim=True)
        s = (big / E4M3_MAX).float().double()
        if pow2:
            s = torch.exp2(torch.ceil(torch.log2(s.clamp_min(1e-30))))
        s = torch.where(big > 0, s, 1.0)
        q = (part / s).float().double()
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
        res[..., at:at + 128] = (torch.round(q / step) * step).clamp(-E4M3_MAX, E4M3_MAX) * s
    return res.transpose(axis, -1)


def _exact_fp8(case, s):
    N, K = case["N"], case["K"]
    c = s["w"].to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    w = torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 7), m * 2.0 ** -9) * (1 - 2 * (c >> 7)).double()
    del c, e, m
    rows, cols = torch.arange(N, device="cuda") // 128, torch.arange(K, device="cuda") // 128
    w *= s["ws"].double()[rows][:, cols]
    if case["dir"] == "fwd":
        return dict(y=_exact_codes(s["x"], 1, case["pow2"]) @ w.T)
    d_x = _exact_codes(s["d_y"], 1, case["pow2"]) @ w
    del w
    d_w = None
    if case["dw"]:
        d_w = _exact_codes(s["d_y"], 0, case["pow2"]).T @ _exact_codes(s["x"], 0, case["pow2"])
    return dict(d_x=d_x, d_w=d_w)
