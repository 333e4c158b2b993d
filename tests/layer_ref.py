"""The gate, the dense FP8 projection and the clip by the global norm from their
definitions in 64 bits, with bounds for what the library rounds."""
import math

import torch

HALF = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}  # a rounding's most
F32 = HALF[torch.float32]


# ---- the gate ----

def gate_out(logits, bias):
    o = torch.isnan(logits) | (logits == -math.inf)
    return o if bias is None else o | (torch.isnan(bias) | (bias == -math.inf))


def gate_scores(logits, bias, sigmoid):
    out = gate_out(logits, bias)
    l = logits.double()
    if sigmoid:
        s = torch.sigmoid(l)
    else:
        v = l.masked_fill(out, -math.inf)
        m = v.amax(1, keepdim=True)
        e = torch.where(v == m, 1.0, torch.exp(v - m)).masked_fill(out, 0.0)
        z = e.sum(1, keepdim=True)
        s = e / torch.where(z > 0, z, 1.0)
    return s.masked_fill(out, 0.0), out


def gate(logits, bias, k, sigmoid=True, groups=1, top_groups=1, top2=True, renorm=True, scale=1.0):
    """(ids, w in 64 bits), token by token in plain Python."""
    s, out = gate_scores(logits, bias, sigmoid)
    T, E = s.shape
    b = [0.0] * E if bias is None else bias.double().tolist()
    ids, w = [], []
    for t in range(T):
        st, ot = s[t].tolist(), out[t].tolist()
        c = [-math.inf if ot[e] else st[e] + b[e] for e in range(E)]
        per = E // groups
        worth = []
        for g in range(groups):
            v = sorted((c[e] for e in range(g * per, g * per + per) if not ot[e]), reverse=True)
            worth.append(-math.inf if not v else v[0] + v[1] if top2 and len(v) > 1 else v[0])
        best = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
        pool = [e for e in range(E) if e // per in best]
        row = sorted(pool, key=lambda e: (ot[e], -c[e] if not ot[e] else 0.0, e))[:k]
        tot = sum(st[e] for e in row)
        ids.append(row)
        w.append([scale * st[e] / (tot if tot > 0 else 1.0) if renorm else scale * st[e] for e in row])
    return torch.tensor(ids, dtype=torch.int32), torch.tensor(w, dtype=torch.float64)


def gate_weights(l64, bias, ids, sigmoid, renorm, scale):
    """w [T][k] as a differentiable function of the logits in 64 bits."""
    out = gate_out(l64, bias)
    if sigmoid:
        s = torch.sigmoid(l64)
    else:
        s = torch.softmax(l64.masked_fill(out, -math.inf), 1)
    w = torch.where(out, torch.zeros_like(s), s).gather(1, ids.long())
    return scale * (w / w.sum(1, keepdim=True) if renorm else w)


def gate_grad(logits, bias, ids, dw, sigmoid, renorm, scale):
    """(d_logits, bound) in 64 bits by the formulas.

    The bound counts what fp32 arithmetic rounds, in units of half a step: exp
    (2) of an argument that was rounded itself (|l - m| more), sums of E terms,
    reciprocals and products (24 together), relative to the sums of magnitudes
    that the differences are taken of."""
    s, out = gate_scores(logits, bias, sigmoid)
    T, E = s.shape
    ids = ids.long()
    there = (ids >= 0) & (ids < E)
    at = ids.clamp(0, E - 1)
    sj = s.gather(1, at) * there
    g = dw.double() * scale
    mag = g.abs()
    if renorm:
        tot = sj.sum(1, keepdim=True)
        it = torch.where(tot > 0, 1.0 / tot, 0.0)
        dot = (g * sj).sum(1, keepdim=True) * it
        mag = (mag + (mag * sj).sum(1, keepdim=True) * it) * it
        g = (g - dot) * it
    live = there & ~out.gather(1, at)
    ds = torch.zeros_like(s).scatter_add_(1, at, torch.where(live, g, 0.0))
    dm = torch.zeros_like(s).scatter_add_(1, at, torch.where(live, mag, 0.0))
    l = logits.double().masked_fill(out, 0.0)
    if sigmoid:
        e = torch.exp(-l.abs())
        d = e / (1 + e) ** 2
        grad, big = ds * d, dm * d
        spread = torch.zeros_like(l)
    else:
        m = l.masked_fill(out, -math.inf).amax(1, keepdim=True)
        spread = (l - m).abs().masked_fill(out | ~torch.isfinite(l - m), 0.0)
        grad = s * (ds - (ds * s).sum(1, keepdim=True) * (0.0 if renorm else 1.0))
        big = s * (dm + (dm * s).sum(1, keepdim=True))
    spread = spread.amax(1, keepdim=True)
    return grad, big * F32 * (24 + math.log2(E) + 4 * spread) + 1e-37


# ---- the dense FP8 projection ----

def e4m3(codes):
    """Values of E4M3 codes in 64 bits."""
    c = codes.view(torch.uint8).long()
    e, m = (c >> 3) & 15, (c & 7).double()
    return torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 7), m * 2.0 ** -9) * (1 - 2 * (c >> 7))


def block_scale(amax, pow2):
    s = (amax.double() / 448).float()
    if pow2:
        s = torch.exp2(torch.ceil(torch.log2(s.double().clamp_min(2.0 ** -127)))).float()
    return torch.where(amax > 0, s, 1.0)


def quantized(v, axis, pow2):
    """What the codes of v [.., ..] stand for, in 64 bits: a scale per 128 along axis, the quotient rounded to fp32,
    then to e4m3 (nearest even)."""
    v = v.double().transpose(axis, -1)
    res = torch.empty_like(v)
    for at in range(0, v.shape[-1], 128):
        part = v[..., at:at + 128]
        s = block_scale(part.abs().amax(-1, keepdim=True).float(), pow2).double()
        q = (part / s).float().double()
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
        res[..., at:at + 128] = (torch.round(q / step) * step).clamp(-448, 448) * s
    return res.transpose(axis, -1)


def weights(codes, scale):
    N, K = codes.shape
    return e4m3(codes) * scale.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


def make_weights(N, K, pow2, gen, device="cpu"):
    """Random codes over the whole range of E4M3 (no NaN) and scales."""
    codes = torch.randint(0, 256, (N, K), generator=gen, dtype=torch.uint8)
    codes = torch.where((codes & 127) == 127, codes - 1, codes)
    s = torch.exp(torch.randn((N + 127) // 128, (K + 127) // 128, generator=gen)) * 2.0 ** -10
    if pow2:
        s = torch.exp2(torch.floor(torch.log2(s)))
    return codes.to(device), s.float().to(device)


def group_maxima(a, b):
    """Sum over groups of 8 consecutive k of the largest |a[m][k] b[n][k]|."""
    pad = -a.shape[1] % 8
    a, b = (torch.nn.functional.pad(v.abs(), (0, pad)).unflatten(1, (-1, 8)) for v in (a, b))
    rows = max(1, (1 << 26) // (b.shape[0] * a.shape[1]))
    res = []
    for i in range(0, a.shape[0], rows):
        part = a[i:i + rows]
        top = part[:, None, :, 0] * b[None, :, :, 0]
        for k in range(1, 8):
            torch.maximum(top, part[:, None, :, k] * b[None, :, :, k], out=top)
        res.append(top.sum(2))
    return torch.cat(res)


def product(a, b):
    """(a b^T, bound of the library's bf16 result).

    The matrix core takes E4M3 products 8 consecutive k at a time, aligned to the
    largest exponent among them with 13 bits kept below it (probed: beside 2^16
    and -2^16 a product of 2^3 is kept and one of 2^2 is lost in the same group of
    8, and kept in any other): each of the other 7 loses less than 2^-13 of the
    largest.  Then fp32 roundings, one per group of 8 and two per block, of sums
    no larger than the sum of the magnitudes, and the result's."""
    y, mag = a @ b.T, a.abs() @ b.abs().T
    steps = (a.shape[1] + 7) // 8 + 2 * ((a.shape[1] + 127) // 128)
    return y, HALF[torch.bfloat16] * y.abs() + 7 * 2.0 ** -13 * group_maxima(a, b) * (1 + 2 ** -8) \
        + mag * (steps + 2) * F32 + 1e-38
