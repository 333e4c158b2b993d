"""Plain 64-bit forms of the training losses and of their gradients, with
bounds for a device result: loops and elementary operations on CPU tensors,
written from the definitions in include/moe_lp.h.

Rounding counts used in the bounds: a bf16 result is off by at most 2^-8 of
its value, an fp32 operation by 2^-24; a sum of n fp32 terms by n 2^-24 of the
sum of their magnitudes, in any order."""
import math

import torch

BF16, F32 = 2.0 ** -8, 2.0 ** -24


class HeadRef:
    """Reference of one head loss.  target: dense [T][V] weights of the counted
    rows (one-hot, or the teacher's q), counts: [T] bool."""

    def __init__(self, h, w, counts, target, eps, scale):
        self.counts, self.eps, self.scale = counts, eps, scale
        self.rows = torch.nonzero(counts)[:, 0]
        self.T, self.H, self.V = h.shape[0], h.shape[1], w.shape[0]
        self.w = w.double()
        self.x = h[self.rows].double()
        n = self.rows.numel()
        ms = (self.x ** 2).sum(1) / self.H
        self.r = 1.0 / torch.sqrt(ms + eps) if eps > 0 else torch.ones(n, dtype=torch.float64, device=h.device)
        self.z = self.x * self.r[:, None]
        self.logits = scale * (self.z @ self.w.T)
        m = self.logits.max(1).values if n else self.logits.sum(1)
        self.lse_c = m + torch.log(torch.exp(self.logits - m[:, None]).sum(1))
        self.p = torch.exp(self.logits - self.lse_c[:, None])
        self.q = target[self.rows].double()
        # error of a logit: H products summed in fp32, 1/rms (its sum of H squares enters by half its relative
        # error, then a mean, an addition, a root, a quotient) and the two scalings
        mag = scale * (self.z.abs() @ self.w.abs().T)
        self.d_logit = mag.max(1).values * (1.5 * self.H + 16) * F32 if n else m
        # ... and of lse: the largest of them, exp (argument and 4 steps), V + 16 additions of the sum, log and sum
        span = (self.logits.max(1).values - self.logits.min(1).values) if n else m
        self.d_lse = self.d_logit + (span + 8 + min(self.V, 2048) + 16) * F32 + 8 * self.lse_c.abs() * F32

    def full(self, v):
        out = torch.zeros(self.T, *v.shape[1:], dtype=torch.float64, device=v.device)
        out[self.rows] = v
        return out

    def loss(self):
        """(lse, loss, bound of lse, bound of loss)."""
        logp = self.logits - self.lse_c[:, None]
        hq = torch.where(self.q > 0, self.q * torch.log(torch.where(self.q > 0, self.q, 1.0)), 0.0)
        loss = (hq - self.q * logp).sum(1)
        # q has a relative error of some 300 steps (a softmax of at most 256 teacher logits), and there are at most
        # 256 terms
        wsum = self.q.sum(1)
        size = (hq.abs() + (self.q * logp).abs()).sum(1)
        d_loss = wsum * (self.d_logit + self.d_lse) + size * 600 * F32 + 64 * F32 * wsum
        return self.full(self.lse_c), self.full(loss), self.full(self.d_lse), self.full(d_loss)

    def grads(self, g, weight_grad):
        """d_h, bound, d_w, bound for dL/dloss g [T]."""
        n = self.rows.numel()
        g = g[self.rows].double()
        cf = (self.scale * self.r * g)[:, None]
        G = cf * (self.p - self.q)
        # G: bf16 rounding, and p by its exponent's error and some 16 steps (q: as in loss)
        dl = (self.d_logit + self.d_lse)[:, None] if n else 0.0
        dG = G.abs() * (BF16 + 16 * F32) + cf.abs() * (self.p * (dl + 32 * F32) + self.q * 600 * F32)
        u = G @ self.w
        du = dG @ self.w.abs() + (G.abs() @ self.w.abs()) * (self.V + 16) * F32
        d_h, dd = u, du
        if self.eps > 0:
            c = (self.r ** 2)[:, None]
            d_h = u - c * self.x * (self.x * u).mean(1, keepdim=True)
            mean = (self.x.abs() * du).mean(1, keepdim=True)
            size = (self.x * u).abs().mean(1, keepdim=True)
            dd = du + c * self.x.abs() * (mean + size * (4 * self.H + 16) * F32)
        dd = dd + (d_h.abs() + dd) * BF16
        d_w = dw_b = None
        if weight_grad:
            d_w = G.T @ self.x
            dw_b = dG.T @ self.x.abs() + (G.abs().T @ self.x.abs()) * (n + 16) * F32
            dw_b = dw_b + (d_w.abs() + dw_b) * BF16
        return self.full(d_h), self.full(dd), d_w, dw_b


def ce_ref(h, w, targets, eps=1e-6, scale=1.0):
    T, V = h.shape[0], w.shape[0]
    counts = (targets >= 0) & (targets < V)
    target = torch.zeros(T, V, dtype=torch.float64, device=h.device)
    rows = torch.nonzero(counts)[:, 0]
    target[rows, targets[rows].long()] = 1.0
    return HeadRef(h, w, counts, target, eps, scale)


def teacher_probs(ids, tl, V, tscale=1.0):
    """(present [T][K], q [T][K]); a row without a present slot has q = 0."""
    have = (ids >= 0) & (ids < V) & (tl != -math.inf)
    x = torch.where(have, tl.double() * tscale, torch.full_like(tl.double(), -math.inf))
    m = x.max(1, keepdim=True).values
    e = torch.where(have, torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m)), 0.0)
    s = e.sum(1, keepdim=True)
    return have, e / torch.where(s > 0, s, 1.0)


def distill_ref(h, w, ids, tl, tscale=1.0, eps=1e-6, scale=1.0):
    """(reference, present, dense logp at the slots is ref.logits - lse).  The
    loss of repeated ids is that of the slots (see distill_loss)."""
    V = w.shape[0]
    have, q = teacher_probs(ids, tl, V, tscale)
    target = torch.zeros(h.shape[0], V, dtype=torch.float64, device=h.device)
    target.scatter_add_(1, torch.where(have, ids, 0).long(), q)
    return HeadRef(h, w, have.any(1), target, eps, scale), have, q


def distill_loss(ref, ids, have, q):
    """(lse, loss, logp [T][K], bounds of the three) from the slots."""
    at = torch.where(have, ids, 0).long()[ref.rows]
    hv, qr = have[ref.rows], q[ref.rows]
    logp = torch.where(hv, torch.gather(ref.logits, 1, at) - ref.lse_c[:, None], 0.0)
    logq = torch.where(qr > 0, torch.log(torch.where(qr > 0, qr, 1.0)), 0.0)
    loss = (qr * (logq - logp)).sum(1)
    d = ref.d_logit + ref.d_lse
    d_loss = d + (qr * (logq.abs() + logp.abs())).sum(1) * 600 * F32 + 64 * F32
    d_logp = torch.where(hv, d[:, None] + 2 * F32 * logp.abs(), 0.0)
    return (ref.full(ref.lse_c), ref.full(loss), ref.full(logp), ref.full(ref.d_lse), ref.full(d_loss),
            ref.full(d_logp))


def balance_ref(logits, ids, k, mask=None, off=None, d_loss=None):
    """Per segment, token by token: loss, counts, tokens, probs, d_logits (None
    without d_loss) and the bounds of loss, probs and d_logits."""
    T, E = logits.shape
    off = [0, T] if off is None else [int(v) for v in off]
    S = len(off) - 1
    on = torch.ones(T, dtype=torch.bool) if mask is None else mask.bool()
    x = torch.where(on[:, None], logits.double(), 0.0)  # whatever masked rows hold
    m = x.max(1, keepdim=True).values if T else x.sum(1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(x - m)
    s = e.sum(1, keepdim=True)
    p = e / torch.where(s > 0, s, 1.0)
    fin = torch.where(x == -math.inf, m, x)
    # p: the exponent's argument, exp (4 steps), a sum of E terms, a reciprocal and a product
    rel = ((m - fin).abs().max(1).values + E / 16 + 16) * F32 if T else x.sum(1)
    loss = torch.zeros(S, dtype=torch.float64)
    counts = torch.zeros(S, E, dtype=torch.int64)
    tokens = torch.zeros(S, dtype=torch.int64)
    probs, b_probs = torch.zeros(S, E, dtype=torch.float64), torch.zeros(S, E, dtype=torch.float64)
    b_loss = torch.zeros(S, dtype=torch.float64)
    grad = b_grad = None
    if d_loss is not None:
        grad, b_grad = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    for i in range(S):
        t = torch.arange(off[i], off[i + 1])
        t = t[on[t]]
        n = len(t)
        tokens[i] = n
        if n == 0:
            continue
        c = ids[t].reshape(-1).long()
        counts[i] = torch.bincount(c[(c >= 0) & (c < E)], minlength=E)
        probs[i] = p[t].sum(0) / n
        # at most n additions, then a reciprocal and a product
        b_probs[i] = (p[t] * rel[t][:, None]).sum(0) / n + probs[i] * (n + 4) * F32
        cf = counts[i].double()
        loss[i] = E / (k * n) * (cf * probs[i]).sum()
        b_loss[i] = E / (k * n) * (cf * b_probs[i]).sum() + loss[i] * (E / 64 + 32) * F32
        if d_loss is not None:
            f = d_loss[i].double() * E / (k * n * n)
            a = f * cf
            grad[t] = p[t] * (a - (p[t] @ a)[:, None])
            ca = (f * (cf - cf.mean())).abs() + f.abs() * cf.mean() * 4 * F32
            dot = (p[t] @ ca)[:, None]
            # a few steps in a and in the differences, p's error in front and in the sum; where a row has no p its
            # sum of p is not 1, but then p is 0
            b_grad[t] = p[t] * ((ca + dot) * (rel[t][:, None] * 2 + (E / 16 + 32) * F32))
    return dict(loss=loss, counts=counts, tokens=tokens, probs=probs, d_logits=grad, b_loss=b_loss, b_probs=b_probs,
                b_grad=b_grad)
