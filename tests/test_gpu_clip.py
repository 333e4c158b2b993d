"""GPU parity of the global norm and the clipping by it."""
import math

import pytest
import torch

import precision_moe_expert_amd as moe
from precision_moe_expert_amd import binding
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _grads(sizes, seed, types=TYPES):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * 10.0 ** (-(i % 3))).to(types[i % len(types)]).cuda()
            for i, n in enumerate(sizes)]


def _norm(ts):
    return math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in ts))


def _check(before, after, norm, limit):
    want = _norm(before)
    # sums in 64 bits, one rounding
    assert abs(float(norm) - want) <= want * ref.F32 * (1 + 1e-6) and norm.shape == (1,)
    c = limit / want if want > limit else 1.0
    for b, a in zip(before, after):
        assert a.dtype == b.dtype and a.shape == b.shape
        w = b.double() * c
        # c rounded to fp32, the product to fp32 and then to the type (fp16: down to its smallest step)
        tol = w.abs() * (ref.HALF[a.dtype] + 2.01 * ref.F32) + (2.0 ** -25 if a.dtype == torch.float16 else 1e-44)
        if c == 1.0:
            assert torch.equal(a, b)
        assert bool(((a.double() - w).abs() <= tol).all())


@pytest.mark.parametrize("sizes", [[1], [7, 1, 3], [1000, 0, 17], [8191, 8192, 8193, 16385], [1 << 20, 5, 40000],
                                   list(range(1, 200)), [3_000_001, 3, 12_345_678]])
@pytest.mark.parametrize("part", [0.3, 3.0])
def test_norm_and_clip(sizes, part):
    grads = _grads(sizes, len(sizes))
    before = [t.clone() for t in grads]
    limit = _norm(before) * part
    outs = [torch.full_like(t, 9.0) for t in grads]
    norm = moe.clip_grads(grads, limit, out=outs)
    _check(before, outs, norm, limit)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    assert torch.equal(moe.grad_norm(grads), norm)
    assert torch.equal(moe.clip_grads(grads, limit), norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, outs))
    again = [t.clone() for t in before]
    moe.scale_grads(again, norm, limit)
    if part > 1:
        assert all(torch.equal(a, b) for a, b in zip(again, outs))
    else:  # from the rounded norm: c may be one step off
        _check(before, again, norm, limit)


def test_views_at_any_address():
    flat = _grads([5000], 3, [torch.bfloat16])[0]
    for a, b in ((1, 4001), (3, 10), (8, 2000), (5, 5)):
        before = flat.clone()
        v = flat[a:b]
        limit = 0.5 * _norm([v]) if b > a else 1.0
        norm = moe.clip_grads([v], limit)
        _check([before[a:b]], [v], norm, limit)
        assert torch.equal(flat[:a], before[:a]) and torch.equal(flat[b:], before[b:])
    src, dst = _grads([999], 4, [torch.float32])[0], torch.zeros(1003, device="cuda")
    norm = moe.clip_grads([src], 1.0, out=[dst[1:1000]])   # aligned in, unaligned out
    _check([src], [dst[1:1000]], norm, 1.0)
    assert bool((dst[:1] == 0).all()) and bool((dst[1000:] == 0).all())


def test_many_launches_of_lists():
    grads = _grads([33] * 401, 5)
    before = [t.clone() for t in grads]
    _check(before, grads, moe.clip_grads(grads, 0.1), 0.1)


def test_large_and_small_values():
    big = [torch.full((4096,), 1e30, device="cuda"), torch.full((10,), -3e38, device="cuda")]
    # 9.5e38, past fp32's 3.4e38: a norm that is not finite, and nothing is clipped
    assert float(moe.clip_grads(big, 1.0)) == math.inf and float(big[0][0]) == float(torch.tensor(1e30))
    big = [torch.full((4096,), 1e30, device="cuda"), torch.full((1,), -3e38, device="cuda")]
    _check([t.clone() for t in big], big, moe.clip_grads(big, 1.0), 1.0)
    small = [torch.full((4096,), 1e-30, device="cuda")]
    _check([t.clone() for t in small], small, moe.clip_grads(small, 1e-31), 1e-31)
    zero = [torch.zeros(100, device="cuda")]
    assert float(moe.clip_grads(zero, 0.0)) == 0.0
    one = _grads([100], 1)
    assert bool((one[0] != 0).any())
    moe.clip_grads(one, 0.0)
    assert bool((one[0] == 0).all())
    keep = _grads([100], 1)
    moe.clip_grads(keep, math.inf)
    assert torch.equal(keep[0], _grads([100], 1)[0])


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_norm_that_is_not_finite_clips_nothing(bad):
    grads = _grads([300, 40, 8], 2)
    grads[1][7] = bad
    before = [t.clone() for t in grads]
    norm = moe.clip_grads(grads, 1.0)
    assert not math.isfinite(float(norm))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(grads, before))
    outs = [torch.zeros_like(t) for t in grads]
    moe.clip_grads(grads, 1.0, out=outs)
    assert torch.equal(outs[0], before[0]) and torch.equal(outs[2], before[2])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_copies_of_what_is_not_clipped(dtype):
    t = torch.randn(999, device="cuda").to(dtype)
    t[::7] = math.nan
    t[3], t[990] = math.inf, -math.inf
    out = torch.zeros_like(t)
    moe.clip_grads([t], 1.0, out=[out])
    assert bool((out.isnan() == t.isnan()).all()) and torch.equal(out[~t.isnan()], t[~t.isnan()])


def test_a_norm_among_the_tensors_is_refused():
    flat = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        moe.scale_grads([flat[:32]], flat[5:6], 1.0)
    with pytest.raises(ValueError):
        moe.scale_grads([flat[:32]], flat[40:41], 1.0, out=[flat[32:]])
    moe.scale_grads([flat[:32]], flat[40:41], 0.5)
    moe.scale_grads([], flat[40:41], 0.5)
    moe.scale_grads([flat[40:40]], flat[40:41], 0.5)
    assert bool((flat[:32] == 0.5).all()) and bool((flat[32:] == 1).all())


def test_same_norm_in_every_run():
    grads = _grads([1_000_003, 77, 250_000], 6)
    norms = {float(moe.grad_norm(grads)) for _ in range(5)}
    assert len(norms) == 1


def test_empty_and_refused():
    assert float(moe.grad_norm([])) == 0.0 and float(moe.clip_grads([], 1.0)) == 0.0
    e = torch.empty(0, device="cuda")
    assert float(moe.clip_grads([e, e], 1.0)) == 0.0
    a, b = torch.ones(8, device="cuda"), torch.ones(8, device="cuda")
    for bad in (lambda: moe.clip_grads([a, a], 1.0), lambda: moe.clip_grads([a, b], 1.0, out=[b, a]),
                lambda: moe.clip_grads([a, b], 1.0, out=[b, b]), lambda: moe.clip_grads([a.double()], 1.0),
                lambda: moe.clip_grads([a[::2]], 1.0), lambda: moe.clip_grads([a], 1.0, out=[b.half()]),
                lambda: moe.clip_grads([a], 1.0, out=[b[:4]]), lambda: moe.clip_grads([a], 1.0, out=[]),
                lambda: moe.scale_grads([a], torch.ones(2, device="cuda"), 1.0)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(binding.MoeError):
        moe.clip_grads([a], -1.0)
    assert float(moe.grad_norm([a, a])) == 4.0               # read twice is fine


def test_overlapping_tensors_are_refused():
    flat = torch.ones(100, device="cuda")
    for bad in (([flat[:50], flat[49:]], None), ([flat[10:20], flat], None), ([flat[:50]], [flat[1:51]]),
                ([flat[:10], flat[10:20]], [flat[20:30], flat[5:15]])):
        with pytest.raises(ValueError):
            moe.clip_grads(bad[0], 1.0, out=bad[1])
        with pytest.raises(ValueError):
            moe.scale_grads(bad[0], torch.ones(1, device="cuda"), 1.0, out=bad[1])
    assert bool((flat == 1).all())
    moe.clip_grads([flat[50:], flat[:50]], 5.0)
    assert abs(float(flat.norm()) - 5.0) < 1e-5
