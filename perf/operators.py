"""Timed cases of the training-loss operators: LM-head cross entropy,
distillation from a teacher's top logits through the same head, and the
router's balance loss, each with its gradient.

`run` computes a case in plain torch operations in 32 bits, or, where `own` is
set, with the library's entry points.  `exact` gives the same outputs from the
definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6      # of the head's parameter-free RMSNorm


def listed():
    return [
        # one generated token scored against a small head: call latency
        dict(name="ce fwd 1 token", op="ce", dir="fwd", T=1, H=2048, V=32000, ignored=0.0, dw=False),
        # the decode batch on the 32000-row head: the weight stream bounds it
        dict(name="ce fwd 64 tokens", op="ce", dir="fwd", T=64, H=7168, V=32000, ignored=0.0, dw=False),
        # scoring a training batch, odd vocabulary, a third of it prompt
        dict(name="ce fwd 4096 odd V", op="ce", dir="fwd", T=4096, H=2048, V=50257, ignored=0.3, dw=False),
        # one short sequence into a frozen head: few rows, odd count
        dict(name="ce bwd 200 frozen", op="ce", dir="bwd", T=200, H=7168, V=32000, ignored=0.2, dw=False),
        # a training batch into a trained head: the largest products
        dict(name="ce bwd 8192 trained", op="ce", dir="bwd", T=8192, H=7168, V=32000, ignored=0.0, dw=True),
        # a small distillation batch
        dict(name="distill fwd 96", op="distill", dir="fwd", T=96, H=2048, V=32000, K=16, ignored=0.0, dw=False),
        # a full distillation batch, 64 teacher logits a token
        dict(name="distill fwd 4096", op="distill", dir="fwd", T=4096, H=7168, V=32000, K=64, ignored=0.1, dw=False),
        # adapter distillation through a frozen head, odd sizes, padded tail
        dict(name="distill bwd 3001 frozen", op="distill", dir="bwd", T=3001, H=2048, V=50257, K=33, ignored=0.5,
             dw=False),
        # the decode-sized router: launch latency
        dict(name="balance fwd 64", op="balance", dir="fwd", T=64, E=384, k=8, S=1, ignored=0.0),
        # a training batch, per-sequence losses over packed sequences
        dict(name="balance fwd 16384 packed", op="balance", dir="fwd", T=16384, E=256, k=8, S=13, ignored=0.1),
        # gradient of one whole-batch loss, and with a padded packed batch
        dict(name="balance bwd 4096", op="balance", dir="bwd", T=4096, E=128, k=8, S=1, ignored=0.0),
        dict(name="balance bwd 32768 packed", op="balance", dir="bwd", T=32768, E=384, k=8, S=40, ignored=0.2),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ce", "ce", "distill", "distill", "balance"])
    d = rng.choice(["fwd", "bwd"])
    ignored = rng.choice([0.0, round(rng.uniform(0.05, 0.8), 2)])
    if op == "balance":
        T = _log_int(rng, 1, 32768)
        E = _log_int(rng, 8, 384)
        return dict(op=op, dir=d, T=T, E=E, k=rng.randint(1, min(8, E // 2)), S=_log_int(rng, 1, min(T, 64)),
                    ignored=ignored)
    while True:
        T, H, V = _log_int(rng, 1, 8192), 8 * _log_int(rng, 16, 896), _log_int(rng, 1000, 131072)
        if T * H * V <= 8192 * 7168 * 32000 and H * V <= 7168 * 64000:
            break
    c = dict(op=op, dir=d, T=T, H=H, V=V, ignored=ignored, dw=d == "bwd" and rng.random() < 0.5)
    if op == "distill":
        c["K"] = _log_int(rng, 1, 128)
    return c


def _kept(T, ignored):
    """Tokens of a case that count."""
    return T - int(T * ignored)


def _log_sum_exp(h, w, rows=2048):
    """Per-token log of the sum of exponentials, by blocks of tokens: what the forward call of a step saved."""
    wf, out = w.float(), []
    for i in range(0, h.shape[0], rows):
        out.append(torch.logsumexp(_normed(h[i:i + rows].float()) @ wf.t(), 1))
    return torch.cat(out)


def _normed(hf):
    return hf * _inv_rms(hf)


def _inv_rms(hf):
    return 1.0 / torch.sqrt((hf * hf).mean(1, keepdim=True) + EPS)


def _row_dots(h, w, ids, rows=512):
    """logits at ids [T][K] (ids valid rows of w)."""
    return torch.cat([(_normed(h[i:i + rows].float())[:, None, :] * w[ids[i:i + rows]].float()).sum(2)
                      for i in range(0, h.shape[0], rows)])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T = case["T"]
    n = _kept(T, case["ignored"])
    keep = torch.zeros(T, dtype=torch.bool, device="cuda")
    keep[torch.randperm(T, generator=g, device="cuda")[:n]] = True
    if case["op"] == "balance":
        E, k, S = case["E"], case["k"], case["S"]
        # a skewed router: a per-expert preference on top of the token's logits
        logits = torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")
        ids = torch.topk(logits, k, dim=1).indices.int()
        off = None
        if S > 1:
            cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda").sort().values
            off = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)]).int()
        mask = keep.to(torch.uint8) if n < T else None
        s = dict(case=case, logits=logits, ids=ids, mask=mask, off=off)
        if case["dir"] == "bwd":
            s["counts"], s["tokens"] = _counts(s)
            s["d_loss"] = torch.rand(S, generator=g, device="cuda") * 0.01
        return s
    H, V = case["H"], case["V"]
    w = (torch.randn(V, H, generator=g, device="cuda") * (2.5 / math.sqrt(H))).bfloat16()
    h = torch.randn(T, H, generator=g, device="cuda")
    s = dict(case=case, w=w)
    if case["op"] == "ce":
        y = torch.randint(0, V, (T,), generator=g, device="cuda")
        # every other token leans towards its target, as a trained model's do
        lean = torch.arange(T, device="cuda")[:, None] % 2 * (torch.rand(T, 1, generator=g, device="cuda") * 4.0)
        h = (h + lean * w[y].float()).bfloat16()
        s.update(h=h, y=torch.where(keep, y, -100).int())
        if case["dir"] == "bwd":
            s["lse"] = torch.where(keep, _log_sum_exp(h, w), 0.0)
            s["loss"] = torch.where(keep, s["lse"] - _row_dots(h, w, y[:, None])[:, 0], 0.0)
    else:
        K = min(case["K"], V)
        h = h.bfloat16()
        base = torch.randint(0, V, (T, 1), generator=g, device="cuda")
        step = torch.randint(1, V // K + 1, (T, 1), generator=g, device="cuda")
        j = torch.arange(K, device="cuda")
        ids = (base + j * step) % V                                       # K different rows
        tl = (torch.randn(T, K, generator=g, device="cuda") * 2.0).sort(1, descending=True).values
        have = keep[:, None] & (j < torch.randint((K + 1) // 2, K + 1, (T, 1), generator=g, device="cuda"))
        s.update(h=h, ids=torch.where(have, ids, -1).int(), tl=tl)
        if case["dir"] == "bwd":
            s["lse"] = torch.where(keep, _log_sum_exp(h, w), 0.0)
            s["logp"] = torch.where(have, _row_dots(h, w, ids, 64) - s["lse"][:, None], 0.0)
    if case["dir"] == "bwd":
        s["d_loss"] = torch.randn(T, generator=g, device="cuda") / n if n else torch.zeros(T, device="cuda")
    return s


# ---- plain form -------------------------------------------------------------

def _head_backward(s, h, w, d_logits):
    hf = h.float()
    r = _inv_rms(hf)
    z = hf * r
    dz = d_logits @ w.float()
    d_h = r * (dz - z * (z * dz).mean(1, keepdim=True))
    d_w = (d_logits.t() @ z).bfloat16() if s["case"]["dw"] else None
    return d_h.bfloat16(), d_w


def _plain_ce(s):
    h, w, y = s["h"], s["w"], s["y"].long()
    keep = y >= 0
    at = y.clamp(min=0)[:, None]
    logits = _normed(h.float()) @ w.float().t()
    if s["case"]["dir"] == "fwd":
        m = logits.max(1, keepdim=True).values
        lse = (m + torch.log(torch.exp(logits - m).sum(1, keepdim=True)))[:, 0]
        loss = lse - logits.gather(1, at)[:, 0]
        return dict(loss=torch.where(keep, loss, 0.0), lse=torch.where(keep, lse, 0.0))
    p = torch.exp(logits - s["lse"][:, None])
    p.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
    p *= torch.where(keep, s["d_loss"], 0.0)[:, None]
    d_h, d_w = _head_backward(s, h, w, p)
    return dict(d_h=d_h, d_w=d_w)


def _teacher(ids, tl):
    """Teacher probabilities over the slots that are there, and their logarithms."""
    have = ids >= 0
    t = torch.where(have, tl, -math.inf)
    m = t.max(1, keepdim=True).values
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(t - m)
    tot = e.sum(1, keepdim=True)
    q = e / torch.where(tot > 0, tot, 1.0)
    return have, q, torch.where(have, t - m - torch.log(torch.where(tot > 0, tot, 1.0)), 0.0)


def _plain_distill(s):
    h, w, ids = s["h"], s["w"], s["ids"].long()
    have, q, logq = _teacher(ids, s["tl"])
    keep, at = have.any(1), ids.clamp(min=0)
    logits = _normed(h.float()) @ w.float().t()
    if s["case"]["dir"] == "fwd":
        m = logits.max(1, keepdim=True).values
        lse = m + torch.log(torch.exp(logits - m).sum(1, keepdim=True))
        logp = torch.where(have, logits.gather(1, at) - lse, 0.0)
        return dict(loss=(q * (logq - logp)).sum(1), lse=torch.where(keep, lse[:, 0], 0.0), logp=logp)
    p = torch.exp(logits - s["lse"][:, None])
    p.scatter_add_(1, at, -q)
    p *= torch.where(keep, s["d_loss"], 0.0)[:, None]
    d_h, d_w = _head_backward(s, h, w, p)
    return dict(d_h=d_h, d_w=d_w)


def _segment_of(s):
    """Segment of each token."""
    T, S = s["case"]["T"], s["case"]["S"]
    if s["off"] is None:
        return torch.zeros(T, dtype=torch.long, device="cuda")
    return torch.searchsorted(s["off"][1:S].contiguous(), torch.arange(T, dtype=torch.int32, device="cuda"),
                              right=True)


def _in_segment(s):
    """[S][T]: 1 where the token is in the segment and counts."""
    seg = _segment_of(s)
    on = (seg[None, :] == torch.arange(s["case"]["S"], device="cuda")[:, None])
    return on if s["mask"] is None else on & (s["mask"] != 0)[None, :]


def _counts(s):
    on = _in_segment(s).float()     # sums of ones: exact in 32 bits
    hot = torch.zeros(s["case"]["T"], s["case"]["E"], device="cuda").scatter_(1, s["ids"].long(), 1.0)
    return (on @ hot).int(), on.sum(1).int()


def _plain_balance(s):
    c = s["case"]
    E, k = c["E"], c["k"]
    e = torch.exp(s["logits"] - s["logits"].max(1, keepdim=True).values)
    p = e / e.sum(1, keepdim=True)
    if c["dir"] == "fwd":
        counts, tokens = _counts(s)
        n = tokens.clamp(min=1).float()[:, None]
        probs = _in_segment(s).float() @ p / n
        loss = (counts.float() * probs).sum(1) * (E / k) / n[:, 0]
        return dict(loss=loss, counts=counts, tokens=tokens, probs=probs)
    n = s["tokens"].clamp(min=1).float()
    a = s["counts"].float() * (s["d_loss"] * (E / k) / n / n)[:, None]
    a = (a - a.mean(1, keepdim=True))[_segment_of(s)]
    if s["mask"] is not None:
        p = p * (s["mask"] != 0).float()[:, None]
    return dict(d_logits=p * (a - (p * a).sum(1, keepdim=True)))


# ---- the library's calls ----------------------------------------------------

def _own(s):
    import precision_moe_expert_amd as moe
    c = s["case"]
    if c["op"] == "ce":
        if c["dir"] == "fwd":
            loss, lse = moe.lm_head_loss(s["h"], s["w"], s["y"])
            return dict(loss=loss, lse=lse)
        d_h, d_w = moe.lm_head_loss_backward(s["h"], s["w"], s["y"], s["loss"], s["lse"], s["d_loss"],
                                             weight_grad=c["dw"])
        return dict(d_h=d_h, d_w=d_w)
    if c["op"] == "distill":
        if c["dir"] == "fwd":
            loss, lse, logp = moe.lm_head_distill(s["h"], s["w"], s["ids"], s["tl"])
            return dict(loss=loss, lse=lse, logp=logp)
        d_h, d_w = moe.lm_head_distill_backward(s["h"], s["w"], s["ids"], s["tl"], s["lse"], s["logp"], s["d_loss"],
                                                weight_grad=c["dw"])
        return dict(d_h=d_h, d_w=d_w)
    layer = moe.make_layer(c["T"], 256, 128, c["E"], c["k"], moe.FMT_INT4)
    if c["dir"] == "fwd":
        loss, counts, tokens, probs = moe.balance_loss(layer, s["logits"], s["ids"], token_mask=s["mask"],
                                                       seg_offsets=s["off"])
        return dict(loss=loss, counts=counts, tokens=tokens, probs=probs)
    return dict(d_logits=moe.balance_loss_backward(layer, s["logits"], s["counts"], s["tokens"], s["d_loss"],
                                                   token_mask=s["mask"], seg_offsets=s["off"]))


def run(state):
    if own:
        return _own(state)
    return {"ce": _plain_ce, "distill": _plain_distill, "balance": _plain_balance}[state["case"]["op"]](state)


def work(case):
    T, n = case["T"], _kept(case["T"], case["ignored"])
    if case["op"] == "balance":
        E, k, S = case["E"], case["k"], case["S"]
        side = S * E * 8 + S * 12 + (T if n < T else 0)
        if case["dir"] == "fwd":
            return dict(bytes=n * E * 4 + n * k * 4 + side, flops=5 * n * E)
        return dict(bytes=n * E * 4 + T * E * 4 + side, flops=9 * n * E)
    H, V, K = case["H"], case["V"], case.get("K", 1)
    per_token = T * 8 + T * K * (8 if case["op"] == "distill" else 4)
    if case["dir"] == "fwd":
        return dict(bytes=n * H * 2 + V * H * 2 + per_token + T * K * 4, flops=2 * n * H * V)
    grads = T * H * 2 + (V * H * 2 if case["dw"] else 0)
    return dict(bytes=n * H * 2 + V * H * 2 + per_token + T * 4 + grads,
                flops=(6 if case["dw"] else 4) * n * H * V)


# ---- the definitions in 64 bits ---------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "balance":
        return _exact_balance(case, s)
    T = case["T"]
    if case["op"] == "ce":
        rows = torch.nonzero(s["y"] >= 0)[:, 0]
        target = torch.zeros(len(rows), case["V"], dtype=torch.float64, device="cuda")
        target[torch.arange(len(rows), device="cuda"), s["y"][rows].long()] = 1.0
    else:
        rows = torch.nonzero((s["ids"] >= 0).any(1))[:, 0]
        there = s["ids"][rows] >= 0
        q = torch.softmax(s["tl"][rows].double().masked_fill(~there, -math.inf), 1)
        target = torch.zeros(len(rows), case["V"], dtype=torch.float64, device="cuda")
        target.scatter_add_(1, s["ids"][rows].long().clamp(min=0), q * there)
    w = s["w"].double()
    x = s["h"][rows].double()
    rms = torch.sqrt(x.pow(2).mean(1) + EPS)
    logits = (x / rms[:, None]) @ w.T
    if case["dir"] == "fwd":
        logp = torch.log_softmax(logits, 1)
        lse = torch.zeros(T, dtype=torch.float64, device="cuda")
        loss = torch.zeros_like(lse)
        lse[rows] = torch.logsumexp(logits, 1)
        loss[rows] = (torch.xlogy(target, target) - target * logp).sum(1)
        if case["op"] == "ce":
            return dict(loss=loss, lse=lse)
        full = torch.zeros(T, s["ids"].shape[1], dtype=torch.float64, device="cuda")
        full[rows] = torch.take_along_dim(logp, s["ids"][rows].long().clamp(min=0), 1) * there
        return dict(loss=loss, lse=lse, logp=full)
    d = (torch.softmax(logits, 1) - target) * s["d_loss"][rows].double()[:, None]
    del target, logits
    d_w = (d.T @ (x / rms[:, None])) if case["dw"] else None
    dz = d @ w
    d_x = dz / rms[:, None] - x * ((dz * x).mean(1) / rms ** 3)[:, None]
    d_h = torch.zeros(T, case["H"], dtype=torch.float64, device="cuda")
    d_h[rows] = d_x
    return dict(d_h=d_h, d_w=d_w)


def _exact_balance(case, s):
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    off = [0, T] if s["off"] is None else s["off"].tolist()
    on = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"] != 0
    p = torch.softmax(s["logits"].double(), 1)
    loss, probs = [], []
    grad = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    for i in range(S):
        t = torch.nonzero(on[off[i]:off[i + 1]])[:, 0] + off[i]
        n = max(1, len(t))
        c = torch.bincount(s["ids"][t].reshape(-1).long(), minlength=E).double()
        probs.append(p[t].sum(0) / n)
        loss.append((c * probs[-1]).sum() * E / (k * n))
        if case["dir"] == "bwd":
            a = float(s["d_loss"][i].double()) * E * c / (k * n * n)
            grad[t] = p[t] * (a - (p[t] @ a)[:, None])
    if case["dir"] == "bwd":
        return dict(d_logits=grad)
    return dict(loss=torch.stack(loss), counts=None, tokens=None, probs=torch.stack(probs))
