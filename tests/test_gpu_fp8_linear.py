"""GPU parity of the dense FP8 projection and its gradients."""
import pytest
import torch

import precision_moe_expert_amd as moe
from precision_moe_expert_amd import binding
from tests import layer_ref as ref
from tests.linear_choices import CHOICES

pytestmark = pytest.mark.gpu
FMT = {False: moe.FMT_FP8, True: moe.FMT_FP8_POW2}


def _inputs(M, K, N, pow2, seed):
    g = torch.Generator().manual_seed(seed)
    codes, s = ref.make_weights(N, K, pow2, g, "cuda")
    x = torch.randn(M, K, generator=g)
    x[:, ::17] *= 30.0
    x[M // 2] = 0.0
    if M > 3:
        x[1] *= 1e-20
        x[2] *= 1e20
    d_y = torch.randn(M, N, generator=g) * torch.exp(3 * torch.randn(M, 1, generator=g))
    d_y[M // 3] = 0.0
    return x.bfloat16().cuda(), codes, s, d_y.bfloat16().cuda()


def _near(got, want, bound):
    off = (got.double() - want).abs()
    assert got.dtype == torch.bfloat16 and got.shape == want.shape
    assert bool((off <= bound).all()), (float((off / bound).max()), int((off > bound).sum()))
    # together: a rounding to bf16 is 2^-8 of its value at most, and what the matrix core cuts is far below that
    # where the values of a row are alike; rows of very different size are looked at one by one
    size = want.norm(dim=1)
    assert bool((off.norm(dim=1) <= 2.0 ** -8 * size + bound.norm(dim=1) / 8).all())


def _check(M, K, N, pow2, seed=0, dx=True, dw=True):
    x, codes, s, d_y = _inputs(M, K, N, pow2, seed)
    w = ref.weights(codes, s)
    _near(moe.fp8_linear(x, codes, s, FMT[pow2]), *ref.product(ref.quantized(x, 1, pow2), w))
    wt, st = moe.fp8_linear_transpose(codes, s)
    assert torch.equal(wt, codes.T) and torch.equal(st, s.T)
    got = moe.fp8_linear_backward(d_y, wt, st, FMT[pow2], x=x if dw else None, input_grad=dx, weight_grad=dw)
    assert (got[0] is not None) == dx and (got[1] is not None) == dw
    if dx:
        _near(got[0], *ref.product(ref.quantized(d_y, 1, pow2), w.T))
    if dw:
        # the gradient of rows that are 1e20 of others: by columns the codes of the small ones are 0
        _near(got[1], *ref.product(ref.quantized(d_y, 0, pow2).T, ref.quantized(x, 0, pow2).T))


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 128, 129, 300])
def test_rows(M, pow2):
    _check(M, 400, 272, pow2, M)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("K,N", [(16, 16), (16, 272), (128, 128), (144, 48), (256, 512), (1040, 16), (4112, 144),
                                 (112, 1040), (240, 4112)])
def test_widths(K, N, pow2):
    for M in (1, 9, 40, 200):
        _check(M, K, N, pow2, K + N)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,K,N", [(5000, 256, 2576), (2100, 2576, 3856), (1030, 4096, 512), (513, 7168, 256)])
def test_large(M, K, N, pow2):
    _check(M, K, N, pow2, 1)


@pytest.mark.parametrize("M,K,N", [(12, 4096, 48), (13, 4096, 48), (16, 1024, 32), (16, 1040, 32), (6, 7168, 16),
                                   (7, 7168, 16), (3, 14336, 16), (1, 47104, 16), (1, 131072, 16), (2, 16, 131072)])
def test_few_rows_of_any_length(M, K, N):
    """Both sides of what is quantized on the way, up to the longest rows and most columns."""
    for pow2 in (False, True):
        _check(M, K, N, pow2, K, dw=K * N < 1 << 20)


@pytest.mark.parametrize("M", [2, 3, 7, 11, 12, 16, 17, 32, 33])
@pytest.mark.parametrize("K,N", [(2048, 1040), (1040, 4112), (4352, 272), (144, 128), (7168, 80)])
@pytest.mark.parametrize("pow2", [False, True])
def test_batches_of_single_tokens(M, K, N, pow2):
    _check(M, K, N, pow2, M + K, dw=M == 17)


@pytest.mark.parametrize("M,K,N", [(40, 2064, 4096), (64, 144, 2048), (100, 272, 1040), (256, 4096, 2048), (33, 1152, 80),
                                   (200, 128, 512), (65, 656, 144)])
@pytest.mark.parametrize("pow2", [False, True])
def test_a_few_dozen_rows(M, K, N, pow2):
    """Odd numbers of blocks, one block, a last one that is not whole, columns that end inside a tile."""
    _check(M, K, N, pow2, M, dw=M == 33)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,K,N", [s for s, _ in CHOICES])
def test_every_choice_of_kernel(M, K, N, pow2):
    """Sizes of every tile, split, last round in halves and joined launch that a call may choose."""
    _check(M, K, N, pow2, M)


def test_one_gradient_alone():
    _check(70, 256, 144, False, 3, dx=True, dw=False)
    _check(70, 256, 144, False, 3, dx=False, dw=True)


def test_strided_rows_and_given_output():
    M, K, N = 77, 272, 144
    x, codes, s, d_y = _inputs(M, K, N, False, 5)
    wide = torch.full((M, K + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + K] = x
    wide_y = torch.full((M, N + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_y[:, :N] = d_y
    want = moe.fp8_linear(x, codes, s)
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    got = moe.fp8_linear(wide[:, 8:8 + K], codes, s, out=out)
    assert got is out and torch.equal(out, want)
    assert torch.equal(moe.fp8_linear(x, codes.view(torch.float8_e4m3fn), s), want)
    wt, st = moe.fp8_linear_transpose(codes, s)
    a = moe.fp8_linear_backward(d_y, wt, st, x=x, weight_grad=True)
    b = moe.fp8_linear_backward(wide_y[:, :N], wt, st, x=wide[:, 8:8 + K], weight_grad=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rows_behind_the_last_are_left():
    """A result that is the front of a larger buffer: nothing behind it is written."""
    M, K, N = 45, 256, 144
    x, codes, s, _ = _inputs(M, K, N, False, 6)
    buf = torch.full((M + 300, N), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.fp8_linear(x, codes, s, out=buf[:M])
    assert torch.equal(buf[:M], moe.fp8_linear(x, codes, s)) and bool((buf[M:] == 7).all())


def test_values_at_the_quantizers_borders():
    """Quotients that fall on e4m3's ties and below its smallest number."""
    K, N = 256, 128
    x = torch.zeros(6, K)
    x[0, :128] = torch.arange(128) * 2.0 ** -10          # down to half of the smallest code's step
    x[0, 0] = 448.0
    x[1] = torch.linspace(0, 448, K)
    x[2] = 448.0 / torch.arange(1, K + 1)
    x[3, 5] = 2.0 ** -133                                # a row of one fp32 subnormal
    x[4] = torch.finfo(torch.bfloat16).max
    x[5] = torch.randn(K, generator=torch.Generator().manual_seed(0)) * 2.0 ** -125
    g = torch.Generator().manual_seed(3)
    for pow2 in (False, True):
        codes, s = ref.make_weights(N, K, pow2, g, "cuda")
        s = s * 2.0 ** -8
        xb = x.bfloat16().cuda()
        # products below fp32's normal range may be flushed: 2^-126 per block
        y, bound = ref.product(ref.quantized(xb, 1, pow2), ref.weights(codes, s))
        _near(moe.fp8_linear(xb, codes, s, FMT[pow2]), y, bound + 4 * 2.0 ** -126)


@pytest.mark.parametrize("M,K", [(3, 400), (300, 400), (40, 272), (20, 656)])
@pytest.mark.parametrize("pow2", [False, True])
def test_values_that_are_not_finite(M, K, pow2):
    """A NaN or an infinity reaches its own row of the result (its own column's gradients) and no other."""
    N = 144
    x, codes, s, d_y = _inputs(M, K, N, pow2, 8)
    codes = codes.clamp_min(1)
    wt, st = moe.fp8_linear_transpose(codes, s)
    want = moe.fp8_linear(x, codes, s, FMT[pow2])
    d_x, d_w = moe.fp8_linear_backward(d_y, wt, st, FMT[pow2], x=x, weight_grad=True)
    x, d_y = x.clone(), d_y.clone()
    x[1, K - 1] = float("nan")
    x[2, 5] = float("inf")
    d_y[1, 7] = -float("inf")
    y = moe.fp8_linear(x, codes, s, FMT[pow2])
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[1:3] = True
    assert not bool(y[bad].isfinite().any()) and torch.equal(y[~bad], want[~bad])
    a, b = moe.fp8_linear_backward(d_y, wt, st, FMT[pow2], x=x, weight_grad=True)
    bad[2] = False
    assert not bool(a[bad].isfinite().any()) and torch.equal(a[~bad], d_x[~bad])
    rows, cols = torch.ones(N, dtype=torch.bool, device="cuda"), torch.ones(K, dtype=torch.bool, device="cuda")
    rows[7] = False
    cols[[5, K - 1]] = False
    assert torch.equal(b[rows][:, cols], d_w[rows][:, cols])
    assert not bool(b[7].isfinite().any()) and not bool(b[:, ~cols].isfinite().any())


def test_an_output_over_an_input_is_refused():
    x, codes, s, _ = _inputs(40, 256, 256, False, 4)
    flat = torch.empty(3 * 40 * 256, dtype=torch.bfloat16, device="cuda")
    y, part = flat[:40 * 256].view(40, 256), flat[256:].view(torch.bfloat16)[:40 * 256].view(40, 256)
    with pytest.raises(ValueError):
        moe.fp8_linear(x, codes, s, out=x)
    with pytest.raises(ValueError):
        moe.fp8_linear(y.copy_(x), codes, s, out=part)
    with pytest.raises(ValueError):
        moe.fp8_linear(x, codes, s, out=codes.view(torch.bfloat16).reshape(-1)[:40 * 256].view(40, 256))
    moe.fp8_linear(y, codes, s, out=flat[40 * 256:2 * 40 * 256].view(40, 256))      # side by side is fine


def test_gradient_against_differences():
    """Where the quantizers are exact (codes times one power of two) the projection is linear."""
    M, K, N = 40, 256, 128
    g = torch.Generator().manual_seed(9)
    codes, s = ref.make_weights(N, K, True, g, "cuda")
    pick = lambda *sh: (torch.randint(-8, 9, sh, generator=g).float()).bfloat16().cuda()  # noqa: E731
    x, d_y, way = pick(M, K), pick(M, N), pick(M, K)
    w = ref.weights(codes, s)
    wt, st = moe.fp8_linear_transpose(codes, s)
    d_x, d_w = moe.fp8_linear_backward(d_y, wt, st, moe.FMT_FP8_POW2, x=x, weight_grad=True)
    up, dn = ((moe.fp8_linear(x + sg * way, codes, s, moe.FMT_FP8_POW2).double() * d_y.double()).sum() for sg in (1, -1))
    size = float(((x.double().abs() + way.double().abs()) @ w.T.abs() * d_y.double().abs()).sum())
    assert abs(float((up - dn) / 2 - (d_x.double() * way.double()).sum())) <= 2 ** -7 * size
    _near(d_w, *ref.product(d_y.double().T, x.double().T))


def test_empty_and_refused():
    x, codes, s, d_y = _inputs(4, 256, 128, False, 1)
    assert moe.fp8_linear(x[:0], codes, s).shape == (0, 128)
    wt, st = moe.fp8_linear_transpose(codes, s)
    d_x, d_w = moe.fp8_linear_backward(d_y[:0], wt, st, x=x[:0], weight_grad=True)
    assert d_x.shape == (0, 256) and bool((d_w == 0).all())
    for bad in (lambda: moe.fp8_linear(x[:, :240], codes, s), lambda: moe.fp8_linear(x.float(), codes, s),
                lambda: moe.fp8_linear(x, codes, s.T), lambda: moe.fp8_linear(x, codes.view(torch.int8), s),
                lambda: moe.fp8_linear(x, codes.cpu(), s), lambda: moe.fp8_linear(x.T, codes, s),
                lambda: moe.fp8_linear_backward(d_y, wt, st, weight_grad=True),
                lambda: moe.fp8_linear_backward(d_y, wt, st, x=x[:2], weight_grad=True),
                lambda: moe.fp8_linear(x, codes, s, out=torch.empty(4, 128, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(binding.MoeError):
        moe.fp8_linear(x, codes, s, moe.FMT_MXFP4)
    tiny = torch.empty(64, dtype=torch.uint8, device="cuda")
    assert torch.equal(moe.fp8_linear(x, codes, s, ws=tiny), moe.fp8_linear(x, codes, s))   # 4 rows need none
    with pytest.raises(binding.MoeError):
        moe.fp8_linear(x.repeat(8, 1), codes, s, ws=tiny)
    with pytest.raises(binding.MoeError):
        moe.fp8_linear_backward(d_y, wt, st, input_grad=False)
