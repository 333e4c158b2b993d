"""Host-side checks of the training-loss entry points: every call here fails
validation (or has nothing to do), so no kernel is launched."""
import ctypes
import math

import pytest

from precision_moe_expert_amd import binding

FAKE = 1 << 20  # aligned non-null address; never dereferenced
BIG = 1 << 50
INV, UNS, SMALL, OK = (binding.MOE_ERR_INVALID_ARGUMENT, binding.MOE_ERR_UNSUPPORTED,
                       binding.MOE_ERR_WORKSPACE_TOO_SMALL, binding.MOE_OK)


def _head(T=64, H=256, V=1000, eps=1e-6, scale=1.0, hs=0, ws=0):
    return binding.MoeLmHead(T, H, V, eps, scale, hs, ws)


def _loss(hd, ptrs=None, nb=BIG):
    p = [FAKE] * 6
    for i, v in (ptrs or {}).items():
        p[i] = v
    return binding.lib().moe_lm_head_loss(ctypes.byref(hd), *p, nb, None)


def _loss_bwd(hd, ptrs=None, nb=BIG):
    p = [FAKE] * 9
    for i, v in (ptrs or {}).items():
        p[i] = v
    return binding.lib().moe_lm_head_loss_backward(ctypes.byref(hd), *p, nb, None)


def _distill(hd, top=4, ts=1.0, ptrs=None, nb=BIG):
    p = [FAKE] * 8
    for i, v in (ptrs or {}).items():
        p[i] = v
    return binding.lib().moe_lm_head_distill(ctypes.byref(hd), top, ts, *p, nb, None)


def _distill_bwd(hd, top=4, ts=1.0, ptrs=None, nb=BIG):
    p = [FAKE] * 10
    for i, v in (ptrs or {}).items():
        p[i] = v
    return binding.lib().moe_lm_head_distill_backward(ctypes.byref(hd), top, ts, *p, nb, None)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INV), (dict(H=0), INV), (dict(V=0), INV), (dict(eps=-1.0), INV), (dict(eps=math.nan), INV),
    (dict(eps=math.inf), INV), (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=math.nan), INV),
    (dict(scale=math.inf), INV), (dict(hs=-8), INV), (dict(hs=248), INV), (dict(ws=128), INV), (dict(H=252), UNS),
    (dict(hs=260), UNS), (dict(ws=257), UNS), (dict(ws=(1 << 22) + 8), UNS), (dict(H=1 << 16), UNS), (dict(V=(1 << 20) + 1), UNS),
    (dict(T=(1 << 20) + 1), UNS)])
def test_head_descriptor(change, status):
    hd = _head(**change)
    assert binding.lib().moe_lm_head_loss_workspace_bytes(ctypes.byref(hd), 0, 1) == 0
    for f in (_loss, _loss_bwd, _distill, _distill_bwd):
        assert f(hd) == status


def test_head_pointers_and_workspace():
    hd, lib = _head(), binding.lib()
    for f, n, optional in ((_loss, 6, ()), (_loss_bwd, 9, (7,)), (_distill, 8, ()), (_distill_bwd, 10, (8,))):
        for i in range(n):
            assert f(hd, ptrs={i: FAKE + 8}) == INV, (f, i)
            if i in optional:  # d_w: a frozen head
                assert f(hd, ptrs={i: None}, nb=0) == SMALL
            else:
                assert f(hd, ptrs={i: None}) == INV, (f, i)
        assert f(hd, nb=0) == SMALL
        assert f(_head(T=0), ptrs={i: None for i in range(n)}) == OK  # nothing to do
    size = lambda top, bwd: lib.moe_lm_head_loss_workspace_bytes(ctypes.byref(hd), top, bwd)  # noqa: E731
    assert 0 < size(0, 0) < size(8, 0) and 0 < size(0, 1) < size(8, 1)
    assert _loss(hd, nb=size(0, 0) - 1) == SMALL and _loss_bwd(hd, nb=size(0, 1) - 1) == SMALL
    assert _distill(hd, nb=size(4, 0) - 1) == SMALL and _distill_bwd(hd, nb=size(4, 1) - 1) == SMALL
    assert lib.moe_lm_head_loss(None, *[FAKE] * 6, BIG, None) == INV
    assert lib.moe_lm_head_loss_workspace_bytes(None, 0, 0) == 0


def test_head_workspace_is_bounded():
    """The gradient of the logits is held a piece at a time, whatever the vocabulary."""
    for T in (1, 64, 8192, 65536):
        for V in (1000, 32000, 1 << 20):
            nb = binding.lm_head_loss_workspace_bytes(T, 2048, V, backward=True)
            assert nb <= T * 2048 * 4 * 64 + max(512 << 20, (T + 256) * 512) + (T + 256) * 2048 * 2 + T * 64 + (1 << 20)


def test_teacher_arguments():
    hd = _head()
    for f in (_distill, _distill_bwd):
        assert f(hd, top=0) == INV and f(hd, top=-1) == INV and f(hd, top=257) == UNS
        assert f(hd, top=256, nb=0) == SMALL
        for ts in (0.0, -1.0, math.nan, math.inf):
            assert f(hd, ts=ts) == INV


def _balance(L, S=1, ptrs=None, nb=BIG, off=FAKE, mask=None):
    p = [FAKE] * 7
    for i, v in (ptrs or {}).items():
        p[i] = v
    return binding.lib().moe_balance_loss(ctypes.byref(L), p[0], p[1], mask, off, S, *p[2:], nb, None)


def _balance_bwd(L, S=1, ptrs=None, off=FAKE, mask=None):
    p = [FAKE] * 5
    for i, v in (ptrs or {}).items():
        p[i] = v
    return binding.lib().moe_balance_loss_backward(ctypes.byref(L), p[0], mask, off, S, p[1], p[2], p[3], 0, p[4],
                                                   None)


def test_balance_arguments():
    L = binding.make_layer(64, 256, 128, 16, 2, binding.FMT_INT4)
    ws = binding.lib().moe_balance_loss_workspace_bytes
    assert ws(ctypes.byref(L), 1) > 0 and ws(ctypes.byref(L), 0) == 0 and ws(ctypes.byref(L), 65537) == 0
    assert _balance(L, nb=ws(ctypes.byref(L), 1) - 1) == SMALL
    for i in range(7):
        assert _balance(L, ptrs={i: None}) == INV and _balance(L, ptrs={i: FAKE + 4}) == INV
    for i in range(5):
        assert _balance_bwd(L, ptrs={i: None}) == INV and _balance_bwd(L, ptrs={i: FAKE + 4}) == INV
    for kw in (dict(mask=FAKE + 1), dict(off=FAKE + 4), dict(S=0), dict(S=3, off=None)):
        assert _balance(L, **kw) == INV and _balance_bwd(L, **kw) == INV
    assert _balance(L, S=65537) == UNS and _balance_bwd(L, S=65537) == UNS
    bad = binding.make_layer(64, 256, 128, 2000, 2, binding.FMT_INT4)
    assert _balance(bad) == UNS and _balance_bwd(bad) == UNS
    none = binding.make_layer(0, 256, 128, 16, 2, binding.FMT_INT4)
    assert _balance_bwd(none, ptrs={i: None for i in range(5)}) == OK


def test_cpu_tensors_are_refused():
    import torch
    h, w, y = torch.zeros(4, 64).bfloat16(), torch.zeros(9, 64).bfloat16(), torch.zeros(4, dtype=torch.int32)
    f = torch.zeros(4)
    L = binding.make_layer(4, 256, 128, 8, 2, binding.FMT_INT4)
    lg, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: binding.lm_head_loss(h, w, y), lambda: binding.lm_head_loss_backward(h, w, y, f, f, f),
                 lambda: binding.lm_head_distill(h, w, ids, lg[:, :2].contiguous()),
                 lambda: binding.balance_loss(L, lg, ids),
                 lambda: binding.balance_loss_backward(L, lg, ids, y, f)):
        with pytest.raises(ValueError):
            call()
