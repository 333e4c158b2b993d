"""Host-side checks of the gate, FP8 projection and clip entry points: every call
here fails validation (or has nothing to do), so no kernel is launched."""
import ctypes
import math

import pytest
import torch

from precision_moe_expert_amd import binding

FAKE = 1 << 20  # aligned non-null address; never dereferenced
BIG = 1 << 50
INV, UNS, SMALL, OK = (binding.MOE_ERR_INVALID_ARGUMENT, binding.MOE_ERR_UNSUPPORTED,
                       binding.MOE_ERR_WORKSPACE_TOO_SMALL, binding.MOE_OK)
R = ctypes.byref


def _layer(T=64, E=64, k=8):
    return binding.make_layer(T, 256, 256, E, k, binding.FMT_FP8)


def _calls(layer, gate, ptrs=None, nb=BIG, bias=FAKE):
    """Status of each gate entry."""
    p = dict(logits=FAKE, ids=FAKE, w=FAKE, d=FAKE, ws=FAKE)
    p.update(ptrs or {})
    L = binding.lib()
    ro = binding.MoeRouteOut(p["ids"], p["w"], *[FAKE] * 5)
    qw, sc = binding.MoeQWeights(FAKE, FAKE), binding.MoeScales(FAKE, FAKE, None, None)
    return [L.moe_route_gated(R(layer), R(gate), p["logits"], bias, R(ro), p["ws"], nb, None),
            L.moe_route_gated_backward(R(layer), R(gate), p["logits"], bias, p["ids"], p["w"], 0, p["d"], None),
            L.moe_expert_forward_gated(R(layer), R(gate), FAKE, p["logits"], bias, R(qw), R(sc), None, 1, p["d"],
                                       p["ws"], nb, None),
            L.moe_expert_backward_gated(R(layer), R(gate), FAKE, p["logits"], bias, R(qw), R(sc), FAKE, None, FAKE, 1,
                                        FAKE, p["d"], None, p["ws"], nb, None)]


@pytest.mark.parametrize("change,status", [
    (dict(score=2), INV), (dict(score=-1), INV), (dict(groups=0), INV), (dict(groups=7), INV),
    (dict(groups=8, top_groups=0), INV), (dict(groups=8, top_groups=9), INV), (dict(group_score=2), INV),
    (dict(groups=16, top_groups=1), INV),  # 4 experts for 8 slots
    (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=math.nan), INV), (dict(scale=math.inf), INV)])
def test_gate_descriptor(change, status):
    assert _calls(_layer(), binding.make_gate(**change)) == [status] * 4


def test_gate_limits_and_pointers():
    g = binding.make_gate()
    bad = binding.make_gate()
    bad.renormalize = 2
    assert _calls(_layer(), bad) == [INV] * 4
    assert _calls(_layer(E=128, k=1), binding.make_gate(groups=128, top_groups=2)) == [UNS] * 4
    assert _calls(_layer(), g, bias=FAKE + 4) == [INV] * 4
    assert _calls(_layer(), g, dict(logits=None)) == [INV] * 4
    assert _calls(_layer(), g, dict(logits=FAKE + 8)) == [INV] * 4
    assert _calls(_layer(), g, dict(ids=None, w=None))[:2] == [INV] * 2
    assert _calls(_layer(), g, dict(d=None))[1:] == [INV] * 3
    assert _calls(_layer(), g, dict(ws=None))[0] == INV
    assert _calls(_layer(), g, nb=64)[0] == SMALL
    assert _calls(_layer(), g, nb=64)[2:] == [SMALL] * 2
    assert _calls(_layer(T=0), g, dict(logits=None, ids=None, w=None, d=None, ws=None)) == [OK] * 4
    L = binding.lib()
    layer = _layer()
    for missing in range(5):  # the permutation's arrays: all or none
        perm = [FAKE] * 5
        perm[missing] = None
        ro = binding.MoeRouteOut(FAKE, FAKE, *perm)
        assert L.moe_route_gated(R(layer), R(g), FAKE, None, R(ro), FAKE, BIG, None) == INV
    assert L.moe_route_gated(R(layer), None, FAKE, None, R(ro), FAKE, BIG, None) == INV
    assert L.moe_route_gated(R(layer), R(g), FAKE, None, None, FAKE, BIG, None) == INV


def test_gate_gradient_over_an_input_is_refused():
    """d_logits of 64 x 64 floats: over an input's first bytes, its last ones, all of it."""
    layer, gate, L = _layer(), binding.make_gate(), binding.lib()
    big, small, bias = 64 * 64 * 4, 64 * 8 * 4, 64 * 4
    at = dict(logits=1 << 24, bias=2 << 24, ids=3 << 24, w=4 << 24)
    qw, sc = binding.MoeQWeights(FAKE, FAKE), binding.MoeScales(FAKE, FAKE, None, None)
    for name, size in (("logits", big), ("bias", bias), ("ids", small), ("w", small)):
        for d in (at[name], at[name] - big + 16, at[name] + size - 16):
            for add in (0, 1):
                assert L.moe_route_gated_backward(R(layer), R(gate), at["logits"], at["bias"], at["ids"], at["w"], add, d,
                                                  None) == INV
            if name in ("logits", "bias"):
                assert L.moe_expert_backward_gated(R(layer), R(gate), FAKE, at["logits"], at["bias"], R(qw), R(sc), FAKE,
                                                   None, FAKE, 1, FAKE, d, None, FAKE, BIG, None) == INV


def _linear(M=64, K=256, N=512, fmt=binding.FMT_FP8, xs=0, ys=0):
    return binding.MoeLinear(M, K, N, fmt, xs, ys)


def _fwd(lin, ptrs=None, nb=BIG):
    p = [FAKE] * 5
    for i, v in (ptrs or {}).items():
        p[i] = v
    return binding.lib().moe_fp8_linear(R(lin), *p, nb, None)


def _bwd(lin, ptrs=None, nb=BIG):
    p = [FAKE] * 7
    for i, v in (ptrs or {}).items():
        p[i] = v
    return binding.lib().moe_fp8_linear_backward(R(lin), *p, nb, None)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), INV), (dict(K=0), INV), (dict(N=0), INV), (dict(fmt=9), INV), (dict(fmt=binding.FMT_INT4), UNS),
    (dict(fmt=binding.FMT_MXFP4), UNS), (dict(K=248), UNS), (dict(N=8), UNS), (dict(K=(1 << 17) + 16), UNS),
    (dict(N=(1 << 17) + 16), UNS), (dict(M=(1 << 20) + 1), UNS), (dict(xs=-8), INV), (dict(xs=248), INV),
    (dict(xs=260), UNS), (dict(ys=504), INV), (dict(ys=516), UNS), (dict(xs=(1 << 22) + 8), UNS)])
def test_linear_descriptor(change, status):
    lin = _linear(**change)
    assert binding.lib().moe_fp8_linear_workspace_bytes(R(lin), 0) == 0
    assert _fwd(lin) == status and _bwd(lin) == status
    assert binding.lib().moe_fp8_linear_transpose(R(lin), *[FAKE] * 4, None) == status


def test_linear_pointers_and_workspace():
    lin, L = _linear(), binding.lib()
    for i in range(5):
        assert _fwd(lin, {i: None}) == INV and _fwd(lin, {i: FAKE + 8}) == INV
    for i in (0, 1, 2, 3, 6):
        assert _bwd(lin, {i: None}) == INV and _bwd(lin, {i: FAKE + 8}) == INV
    for i in (4, 5):
        assert _bwd(lin, {i: FAKE + 8}) == INV
    assert _bwd(lin, {4: None, 5: None}) == INV
    for i in range(4):
        p = [FAKE] * 4
        p[i] = None
        assert L.moe_fp8_linear_transpose(R(lin), *p, None) == INV
    need = L.moe_fp8_linear_workspace_bytes(R(lin), 0)
    assert need >= 64 * 256 and _fwd(lin, nb=need - 1) == SMALL
    for grads, ptrs in ((1, {5: None}), (2, {4: None}), (3, {})):
        need = L.moe_fp8_linear_workspace_bytes(R(lin), grads)
        assert need > 0 and _bwd(lin, ptrs, need - 1) == SMALL
    assert L.moe_fp8_linear_workspace_bytes(R(lin), 4) == 0 and L.moe_fp8_linear_workspace_bytes(R(lin), -1) == 0
    few = _linear(M=4)  # quantized on the way: no workspace
    assert L.moe_fp8_linear_workspace_bytes(R(few), 0) == 0 and L.moe_fp8_linear_workspace_bytes(R(few), 1) == 0
    assert _fwd(few, {4: FAKE + 8}) == INV and L.moe_fp8_linear_workspace_bytes(R(few), 2) > 0
    assert _bwd(few, {4: None}, 0) == SMALL and _bwd(few, {4: None, 6: None}, 0) == INV
    none = _linear(M=0)
    assert [L.moe_fp8_linear_workspace_bytes(R(none), g) for g in range(4)] == [0] * 4
    assert _fwd(none, {i: None for i in range(5)}) == OK
    assert _bwd(none, {0: None, 1: None, 2: None, 3: None, 5: None, 6: None}) == OK


def _list(*items):
    arr = (binding.MoeTensor * max(1, len(items)))()
    for i, it in enumerate(items):
        arr[i] = binding.MoeTensor(*it)
    return arr


@pytest.mark.parametrize("item,status", [
    ((FAKE, FAKE, -1, 0), INV), ((FAKE, FAKE, 4, 3), INV), ((FAKE, FAKE, 4, -1), INV), ((None, FAKE, 4, 0), INV),
    ((FAKE + 2, FAKE, 4, 0), INV), ((FAKE + 1, FAKE, 4, 1), INV), ((FAKE, FAKE, (1 << 40) + 1, 0), UNS)])
def test_clip_tensors(item, status):
    L, a = binding.lib(), _list((FAKE, FAKE, 8, 0), item)
    assert L.moe_grad_norm(a, 2, FAKE, FAKE, BIG, None) == status
    assert L.moe_grad_clip(a, 2, 1.0, FAKE, FAKE, BIG, None) == status
    assert L.moe_grad_scale(a, 2, FAKE, 1.0, None) == status


def test_clip_pointers():
    L, a = binding.lib(), _list((FAKE, None, 8, 0))
    assert L.moe_grad_clip(a, 1, 1.0, FAKE, FAKE, BIG, None) == INV       # no place for the results
    a = _list((FAKE, FAKE + 2, 8, 0))
    assert L.moe_grad_clip(a, 1, 1.0, FAKE, FAKE, BIG, None) == INV
    a = _list((FAKE, FAKE, 8, 0))
    for norm, ws in ((None, FAKE), (FAKE + 2, FAKE), (FAKE, None), (FAKE, FAKE + 8)):
        assert L.moe_grad_clip(a, 1, 1.0, norm, ws, BIG, None) == INV
        assert L.moe_grad_norm(a, 1, norm, ws, BIG, None) == INV
    for limit in (-1.0, math.nan):
        assert L.moe_grad_clip(a, 1, limit, FAKE, FAKE, BIG, None) == INV
        assert L.moe_grad_scale(a, 1, FAKE, limit, None) == INV
    assert L.moe_grad_scale(a, 1, None, 1.0, None) == INV
    assert L.moe_grad_norm(a, -1, FAKE, FAKE, BIG, None) == INV
    assert L.moe_grad_norm(None, 1, FAKE, FAKE, BIG, None) == INV
    need = L.moe_grad_norm_workspace_bytes(1)
    assert need > 0 and L.moe_grad_norm(a, 1, FAKE, FAKE, need - 1, None) == SMALL
    assert L.moe_grad_norm_workspace_bytes(-1) == 0
    assert L.moe_grad_scale(None, 0, FAKE, 1.0, None) == OK


def test_wrappers_refuse_host_tensors():
    x, w = torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(16, 32, dtype=torch.uint8)
    with pytest.raises(ValueError):
        binding.fp8_linear(x, w, torch.zeros(1, 1))
    with pytest.raises(ValueError):
        binding.fp8_linear_transpose(w, torch.zeros(1, 1))
    with pytest.raises(ValueError):
        binding.fp8_linear_backward(torch.zeros(4, 16, dtype=torch.bfloat16), w.T.contiguous(), torch.zeros(1, 1))
    with pytest.raises(ValueError):
        binding.route_gated(_layer(T=2), binding.make_gate(), torch.zeros(2, 64))
    with pytest.raises(ValueError):
        binding.clip_grads([torch.zeros(4)], 1.0)
    with pytest.raises(ValueError):
        binding.clip_grads([torch.zeros(4)], 1.0, out=[])


@pytest.mark.parametrize("call", ["clip", "norm", "scale"])
def test_lists_that_can_be_read_once(monkeypatch, call):
    """Generators of tensors on a device that is not the current one: the call made again there has the same tensors."""
    class Done(Exception):
        pass

    seen, turns = [], iter([True])

    def tensors(grads, out, write=True):
        seen.append((list(grads), None if out is None else list(out)))
        return torch.device("cuda", 1), None, len(seen[-1][0])

    def elsewhere(device):
        if next(turns, False):
            return True
        raise Done

    class On:
        def __init__(self, device):
            pass

        def __enter__(self):
            pass

        def __exit__(self, *e):
            pass

    monkeypatch.setattr(binding, "_tensors", tensors)
    monkeypatch.setattr(binding, "_elsewhere", elsewhere)
    monkeypatch.setattr(torch.cuda, "device", On)
    a, b = [torch.zeros(4), torch.ones(3)], [torch.zeros(4), torch.ones(3)]
    with pytest.raises(Done):
        if call == "clip":
            binding.clip_grads((t for t in a), 1.0, out=(t for t in b))
        elif call == "norm":
            binding.grad_norm(t for t in a)
        else:
            binding.scale_grads((t for t in a), torch.ones(1), 1.0, out=(t for t in b))
    assert len(seen) == 2
    for grads, out in seen:
        assert len(grads) == 2 and all(x is y for x, y in zip(grads, a))
        assert call == "norm" or (len(out) == 2 and all(x is y for x, y in zip(out, b)))
