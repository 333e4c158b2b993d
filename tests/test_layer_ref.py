"""The 64-bit references against differences and against each other."""
from fractions import Fraction

import torch

from tests import layer_ref as ref


def _logits(T, E, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, E, generator=g) * 2, torch.randn(E, generator=g) * 0.1, g


def test_gate_gradient_is_that_of_the_weights():
    for sigmoid in (True, False):
        for renorm in (True, False):
            l, b, g = _logits(5, 12, 3)
            b[4] = -float("inf")
            ids, w = ref.gate(l, b, 3, sigmoid=sigmoid, groups=4, top_groups=2, renorm=renorm, scale=1.5)
            dw = torch.randn(5, 3, generator=g)
            x = l.double().requires_grad_()
            f = ref.gate_weights(x, b, ids, sigmoid, renorm, 1.5)
            torch.testing.assert_close(f.detach(), w, rtol=1e-12, atol=0)
            (f * dw.double()).sum().backward()
            got, _ = ref.gate_grad(l, b, ids, dw, sigmoid, renorm, 1.5)
            torch.testing.assert_close(got, x.grad, rtol=1e-9, atol=1e-14)
            step = 1e-5
            for t, e in ((0, 0), (1, int(ids[1, 0])), (2, int(ids[2, 2])), (3, 4)):
                up, dn = x.detach().clone(), x.detach().clone()
                up[t, e] += step
                dn[t, e] -= step
                d = ((ref.gate_weights(up, b, ids, sigmoid, renorm, 1.5)
                      - ref.gate_weights(dn, b, ids, sigmoid, renorm, 1.5)) * dw.double()).sum() / (2 * step)
                assert abs(float(d - got[t, e])) < 1e-8


def test_gate_choice_without_groups_is_topk():
    l, b, _ = _logits(9, 16, 5)
    ids, _ = ref.gate(l, b, 4)
    want = torch.topk(torch.sigmoid(l.double()) + b.double(), 4, dim=1).indices
    assert torch.equal(ids.long(), want)


def test_quantizer_agrees_with_the_type():
    g = torch.Generator().manual_seed(1)
    v = torch.randn(6, 300, generator=g)
    for pow2 in (False, True):
        got = ref.quantized(v, 1, pow2)
        for at in (0, 128, 256):
            part = v[:, at:at + 128]
            s = ref.block_scale(part.abs().amax(1, keepdim=True), pow2)
            want = (part.double() / s.double()).float().to(torch.float8_e4m3fn)
            assert torch.equal(got[:, at:at + 128], ref.e4m3(want) * s.double())
            assert torch.equal(ref.e4m3(want).float(), want.float())
        assert torch.equal(ref.quantized(v.T.contiguous(), 0, pow2), got.T)


def test_power_of_two_scale_is_the_smallest_at_or_above():
    a = torch.tensor([0.0, 448.0, 448.5, 1.0, 3.5, 1e-30])
    s = ref.block_scale(a, True)
    assert s[0] == 1 and s[1] == 1 and s[2] == 2
    assert bool((s[1:].double() * 448 >= a[1:].double() * (1 - 1e-7)).all()) and bool((s[1:].double() * 224 < a[1:]).all())


def _fp32(v):
    """A positive fraction rounded to fp32 (nearest even)."""
    e = v.numerator.bit_length() - v.denominator.bit_length() - 24
    e += (v / Fraction(2) ** e >= 1 << 24) - (v / Fraction(2) ** e < 1 << 23)
    return round(v / Fraction(2) ** e) * Fraction(2) ** e      # 24 bits kept; round() takes ties to even


def test_a_product_and_a_correction_are_the_quotient():
    """q = x r, q + r (x - q s) with r = 1 / s is x / s rounded once, for every pair of bf16 mantissas of x and of the
    largest of its block (other exponents shift both alike)."""
    wrong = 0
    for top in range(128, 256):
        s = _fp32(Fraction(top, 448))
        r = _fp32(1 / s)
        for x in range(128, 256):
            q = _fp32(x * r)
            e = x - q * s
            e = _fp32(e) if e > 0 else -_fp32(-e) if e < 0 else 0     # one rounding, as of a fused operation
            assert _fp32(q + r * e) == _fp32(x / s)
            wrong += q != _fp32(x / s)
    assert wrong > 0                                                  # the product alone is not
