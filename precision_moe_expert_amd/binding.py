"""ctypes binding of libmoe_lp.so (include/moe_lp.h).

Argument marshalling only: torch supplies device memory and the current HIP
stream; every step of the MoE expert forward runs in the library's kernels.
If the library is missing the first call raises; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_lp.so")
_lib = None

MOE_OK, MOE_ERR_INVALID_ARGUMENT, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE_TOO_SMALL, MOE_ERR_DEVICE = range(5)
FMT_INT4, FMT_FP8, FMT_MXFP4, FMT_FP8_POW2, FMT_NVFP4 = 1, 2, 3, 4, 5
WL_ROWS, WL_KBLOCKED = 0, 1

EXPORTED = ("moe_abi_version", "moe_status_str", "moe_workspace_bytes", "moe_route_workspace_bytes", "moe_tile_rows",
            "moe_route_permute", "moe_expert_forward", "moe_expert_forward_timed", "moe_combine",
            "moe_lm_head_workspace_bytes", "moe_lm_head_logprob", "moe_materialized_workspace_bytes",
            "moe_expert_forward_materialized", "moe_backward_weights_bytes", "moe_prepare_backward_weights",
            "moe_backward_workspace_bytes", "moe_expert_backward", "moe_pack_weights_kblocked",
            "moe_quantize_activations", "moe_expert_forward_noalloc", "moe_lm_head_loss_workspace_bytes",
            "moe_lm_head_loss", "moe_lm_head_loss_backward", "moe_lm_head_distill", "moe_lm_head_distill_backward",
            "moe_balance_loss_workspace_bytes", "moe_balance_loss", "moe_balance_loss_backward", "moe_route_gated",
            "moe_route_gated_backward", "moe_expert_forward_gated", "moe_expert_backward_gated",
            "moe_fp8_linear_workspace_bytes", "moe_fp8_linear", "moe_fp8_linear_transpose", "moe_fp8_linear_backward",
            "moe_grad_norm_workspace_bytes", "moe_grad_norm", "moe_grad_clip", "moe_grad_scale")
NOALLOC_SCRATCH_BYTES = 64 << 20  # MOE_NOALLOC_SCRATCH_BYTES
GATE_SOFTMAX, GATE_SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1
LINEAR_FORWARD, LINEAR_D_X, LINEAR_D_W = 0, 1, 2
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}  # moe_dtype
STAGES = ("route", "permute", "act", "gemm1", "gemm2", "combine", "dequant")


class MoeLayer(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("wformat", ctypes.c_int32),
                ("oft_block", ctypes.c_int32), ("tile_rows", ctypes.c_int32),
                ("adapter_expert_stride", ctypes.c_int64), ("weight_layout", ctypes.c_int32)]


class MoeQWeights(ctypes.Structure):
    _fields_ = [("w13", ctypes.c_void_p), ("w2", ctypes.c_void_p)]


class MoeScales(ctypes.Structure):
    _fields_ = [("s13", ctypes.c_void_p), ("s2", ctypes.c_void_p), ("g13", ctypes.c_void_p), ("g2", ctypes.c_void_p)]


class MoeRouteOut(ctypes.Structure):
    _fields_ = [("topk_ids", ctypes.c_void_p), ("topk_w", ctypes.c_void_p), ("expert_offsets", ctypes.c_void_p),
                ("sorted_rows", ctypes.c_void_p), ("row_of", ctypes.c_void_p), ("active_experts", ctypes.c_void_p),
                ("num_active", ctypes.c_void_p)]


class MoeLmHead(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("norm_eps", ctypes.c_float), ("logit_scale", ctypes.c_float), ("h_stride", ctypes.c_int64),
                ("w_stride", ctypes.c_int64)]


class MoeGate(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("num_groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_score", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float)]


class MoeLinear(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32),
                ("wformat", ctypes.c_int32), ("x_stride", ctypes.c_int64), ("dy_stride", ctypes.c_int64)]


class MoeTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("out", ctypes.c_void_p), ("num", ctypes.c_int64),
                ("dtype", ctypes.c_int32)]


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_str(status)} (status {status})")
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(_LIB_PATH)
        L.moe_abi_version.restype = ctypes.c_int32
        L.moe_status_str.restype = ctypes.c_char_p
        L.moe_status_str.argtypes = [ctypes.c_int]
        L.moe_workspace_bytes.restype = ctypes.c_size_t
        L.moe_workspace_bytes.argtypes = [ctypes.POINTER(MoeLayer), ctypes.c_int32]
        L.moe_tile_rows.restype = ctypes.c_int32
        L.moe_tile_rows.argtypes = [ctypes.POINTER(MoeLayer)]
        L.moe_route_workspace_bytes.restype = ctypes.c_size_t
        L.moe_route_workspace_bytes.argtypes = [ctypes.POINTER(MoeLayer)]
        L.moe_lm_head_workspace_bytes.restype = ctypes.c_size_t
        L.moe_lm_head_workspace_bytes.argtypes = [ctypes.c_int32, ctypes.c_int32]
        L.moe_route_permute.restype = ctypes.c_int
        L.moe_route_permute.argtypes = [ctypes.POINTER(MoeLayer), ctypes.c_void_p, ctypes.POINTER(MoeRouteOut),
                                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        L.moe_expert_forward.restype = ctypes.c_int
        L.moe_expert_forward.argtypes = [ctypes.POINTER(MoeLayer), ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.POINTER(MoeQWeights), ctypes.POINTER(MoeScales), ctypes.c_void_p,
                                         ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                         ctypes.c_void_p]
        L.moe_expert_forward_noalloc.restype = ctypes.c_int
        L.moe_expert_forward_noalloc.argtypes = [ctypes.POINTER(MoeLayer), ctypes.c_void_p, ctypes.c_void_p,
                                                 ctypes.POINTER(MoeQWeights), ctypes.POINTER(MoeScales),
                                                 ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]
        L.moe_expert_forward_timed.restype = ctypes.c_int
        L.moe_expert_forward_timed.argtypes = L.moe_expert_forward.argtypes + [ctypes.POINTER(ctypes.c_float),
                                                                                ctypes.POINTER(ctypes.c_int32)]
        L.moe_materialized_workspace_bytes.restype = ctypes.c_size_t
        L.moe_materialized_workspace_bytes.argtypes = [ctypes.POINTER(MoeLayer), ctypes.c_int32]
        L.moe_expert_forward_materialized.restype = ctypes.c_int
        L.moe_expert_forward_materialized.argtypes = L.moe_expert_forward_timed.argtypes
        L.moe_backward_weights_bytes.restype = ctypes.c_size_t
        L.moe_backward_weights_bytes.argtypes = [ctypes.POINTER(MoeLayer)]
        L.moe_pack_weights_kblocked.restype = ctypes.c_int
        L.moe_pack_weights_kblocked.argtypes = [ctypes.POINTER(MoeLayer), ctypes.POINTER(MoeQWeights),
                                                ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
        L.moe_prepare_backward_weights.restype = ctypes.c_int
        L.moe_prepare_backward_weights.argtypes = [ctypes.POINTER(MoeLayer), ctypes.POINTER(MoeQWeights),
                                                   ctypes.POINTER(MoeScales), ctypes.c_void_p, ctypes.c_size_t,
                                                   ctypes.c_void_p]
        L.moe_backward_workspace_bytes.restype = ctypes.c_size_t
        L.moe_backward_workspace_bytes.argtypes = [ctypes.POINTER(MoeLayer), ctypes.c_int32]
        L.moe_expert_backward.restype = ctypes.c_int
        L.moe_expert_backward.argtypes = [ctypes.POINTER(MoeLayer), ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.POINTER(MoeQWeights), ctypes.POINTER(MoeScales), ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                          ctypes.c_void_p, ctypes.POINTER(ctypes.c_float),
                                          ctypes.POINTER(ctypes.c_int32)]
        L.moe_quantize_activations.restype = ctypes.c_int
        L.moe_quantize_activations.argtypes = [ctypes.POINTER(MoeLayer), ctypes.c_void_p, ctypes.c_void_p,
                                               ctypes.c_void_p, ctypes.c_void_p]
        L.moe_combine.restype = ctypes.c_int
        L.moe_combine.argtypes = [ctypes.POINTER(MoeLayer), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                  ctypes.c_void_p, ctypes.c_void_p]
        L.moe_lm_head_logprob.restype = ctypes.c_int
        L.moe_lm_head_logprob.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_size_t, ctypes.c_void_p]
        head, vp, i32, f32, sz = ctypes.POINTER(MoeLmHead), ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, \
            ctypes.c_size_t
        L.moe_lm_head_loss_workspace_bytes.restype = sz
        L.moe_lm_head_loss_workspace_bytes.argtypes = [head, i32, i32]
        L.moe_lm_head_loss.restype = ctypes.c_int
        L.moe_lm_head_loss.argtypes = [head] + [vp] * 6 + [sz, vp]
        L.moe_lm_head_loss_backward.restype = ctypes.c_int
        L.moe_lm_head_loss_backward.argtypes = [head] + [vp] * 9 + [sz, vp]
        L.moe_lm_head_distill.restype = ctypes.c_int
        L.moe_lm_head_distill.argtypes = [head, i32, f32] + [vp] * 8 + [sz, vp]
        L.moe_lm_head_distill_backward.restype = ctypes.c_int
        L.moe_lm_head_distill_backward.argtypes = [head, i32, f32] + [vp] * 10 + [sz, vp]
        L.moe_balance_loss_workspace_bytes.restype = sz
        L.moe_balance_loss_workspace_bytes.argtypes = [ctypes.POINTER(MoeLayer), i32]
        L.moe_balance_loss.restype = ctypes.c_int
        L.moe_balance_loss.argtypes = [ctypes.POINTER(MoeLayer)] + [vp] * 4 + [i32] + [vp] * 5 + [sz, vp]
        L.moe_balance_loss_backward.restype = ctypes.c_int
        L.moe_balance_loss_backward.argtypes = [ctypes.POINTER(MoeLayer)] + [vp] * 3 + [i32] + [vp] * 3 + [i32, vp,
                                                                                                          vp]
        layer, gate, lin = ctypes.POINTER(MoeLayer), ctypes.POINTER(MoeGate), ctypes.POINTER(MoeLinear)
        qw, sc = ctypes.POINTER(MoeQWeights), ctypes.POINTER(MoeScales)
        for name, args in (
                ("moe_route_gated", [layer, gate, vp, vp, ctypes.POINTER(MoeRouteOut), vp, sz, vp]),
                ("moe_route_gated_backward", [layer, gate] + [vp] * 4 + [i32, vp, vp]),
                ("moe_expert_forward_gated", [layer, gate, vp, vp, vp, qw, sc, vp, i32, vp, vp, sz, vp]),
                ("moe_expert_backward_gated", [layer, gate, vp, vp, vp, qw, sc, vp, vp, vp, i32] + [vp] * 4 + [sz, vp]),
                ("moe_fp8_linear", [lin] + [vp] * 5 + [sz, vp]),
                ("moe_fp8_linear_transpose", [lin] + [vp] * 5),
                ("moe_fp8_linear_backward", [lin] + [vp] * 7 + [sz, vp]),
                ("moe_grad_norm", [vp, i32, vp, vp, sz, vp]),        # first: an array of MoeTensor, or its words
                ("moe_grad_clip", [vp, i32, f32, vp, vp, sz, vp]),
                ("moe_grad_scale", [vp, i32, vp, f32, vp])):
            getattr(L, name).restype, getattr(L, name).argtypes = ctypes.c_int, args
        L.moe_fp8_linear_workspace_bytes.restype, L.moe_fp8_linear_workspace_bytes.argtypes = sz, [lin, i32]
        L.moe_grad_norm_workspace_bytes.restype, L.moe_grad_norm_workspace_bytes.argtypes = sz, [i32]
        _lib = L
    return _lib


def status_str(status: int) -> str:
    return lib().moe_status_str(int(status)).decode()


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("device tensor expected")
    return t.data_ptr()


def _need(t, name: str, nbytes: int, elem: int | None = None):
    """A device tensor, contiguous, of at least nbytes (and elem-byte elements
    when given): the library reads and writes exactly the sizes the layer
    implies, so a smaller or strided tensor would be accessed out of bounds."""
    if t is None:
        raise ValueError(f"{name}: tensor required")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous device tensor expected")
    if elem is not None and t.element_size() != elem:
        raise ValueError(f"{name}: {elem}-byte elements expected, got {t.dtype}")
    if t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name}: {t.numel() * t.element_size()} bytes, the layer needs {nbytes}")


def _weight_bytes(fmt: int, N: int, K: int, E: int):
    """(packed code bytes, scale bytes) of E expert matrices [N][K]."""
    codes = E * N * K if fmt in (FMT_FP8, FMT_FP8_POW2) else E * N * K // 2
    if fmt == FMT_INT4:
        sc = E * (K // 32) * N * 2
    elif fmt in (FMT_FP8, FMT_FP8_POW2):
        sc = E * (N // 128) * (K // 128) * 4
    elif fmt == FMT_NVFP4:
        sc = E * (K // 16) * N
    else:
        sc = E * (K // 32) * N
    return codes, sc


def _check_forward_args(layer: MoeLayer, x, logits, w13, w2, s13, s2, adapter, out, g13, g2):
    T, H, I, E = layer.num_tokens, layer.hidden, layer.inter, layer.num_experts
    if T == 0:
        return
    fmt = layer.wformat
    _need(x, "x", T * H * 2, 2)
    _need(logits, "logits", T * E * 4, 4)
    _need(out, "out", T * H * 2, 2)
    c13, sc13 = _weight_bytes(fmt, 2 * I, H, E)
    c2, sc2 = _weight_bytes(fmt, H, I, E)
    _need(w13, "w13", c13)
    _need(w2, "w2", c2)
    _need(s13, "s13", sc13)
    _need(s2, "s2", sc2)
    if fmt == FMT_NVFP4:
        _need(g13, "g13", E * 4, 4)
        _need(g2, "g2", E * 4, 4)
    if layer.oft_block:
        stride = layer.adapter_expert_stride
        _need(adapter, "adapter", ((E - 1) * stride + H * 32) * 2 if stride else H * 32 * 2, 2)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def make_layer(T, H, I, E, k, fmt, oft=False, adapter_expert_stride=None, tile_rows=0,
               weight_layout=0) -> MoeLayer:
    stride = (H // 32) * 1024 if adapter_expert_stride is None else adapter_expert_stride
    return MoeLayer(T, H, I, E, k, fmt, 32 if oft else 0, tile_rows, stride if oft else 0, weight_layout)


def workspace_bytes(layer: MoeLayer, chunk_experts: int = 1) -> int:
    return lib().moe_workspace_bytes(ctypes.byref(layer), int(chunk_experts))


def tile_rows(layer: MoeLayer) -> int:
    return lib().moe_tile_rows(ctypes.byref(layer))


def alloc_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def route_permute(logits: torch.Tensor, layer: MoeLayer, ws: torch.Tensor | None = None) -> dict:
    """Router top-k + permutation; returns a dict of device tensors."""
    T, E, k = layer.num_tokens, layer.num_experts, layer.top_k
    dev = logits.device
    i32 = dict(dtype=torch.int32, device=dev)
    out = dict(topk_ids=torch.empty((T, k), **i32), topk_w=torch.empty((T, k), dtype=torch.float32, device=dev),
               expert_offsets=torch.empty(E + 1, **i32), sorted_rows=torch.empty(T * k, **i32),
               row_of=torch.empty(T * k, **i32), active_experts=torch.empty(E, **i32),
               num_active=torch.zeros(4, **i32))
    ro = MoeRouteOut(*[_ptr(out[n]) for n in ("topk_ids", "topk_w", "expert_offsets", "sorted_rows", "row_of",
                                              "active_experts", "num_active")])
    if ws is None:
        ws = alloc_workspace(lib().moe_route_workspace_bytes(ctypes.byref(layer)), dev)
    _check(lib().moe_route_permute(ctypes.byref(layer), _ptr(logits), ctypes.byref(ro), _ptr(ws), ws.numel(),
                                   _stream()), "moe_route_permute")
    return out


def expert_forward(layer: MoeLayer, x: torch.Tensor, logits: torch.Tensor, w13, w2, s13, s2, adapter=None,
                   chunk_experts: int = 1, out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                   g13=None, g2=None):
    """moe_expert_forward: x [T][H] bf16, logits [T][E] fp32 -> out [T][H] bf16."""
    if out is None:
        out = torch.empty((layer.num_tokens, layer.hidden), dtype=torch.bfloat16, device=x.device)
    if ws is None:
        ws = alloc_workspace(workspace_bytes(layer, chunk_experts), x.device)
    _check_forward_args(layer, x, logits, w13, w2, s13, s2, adapter, out, g13, g2)
    qw = MoeQWeights(_ptr(w13), _ptr(w2))
    sc = MoeScales(_ptr(s13), _ptr(s2), _ptr(g13), _ptr(g2))
    _check(lib().moe_expert_forward(ctypes.byref(layer), _ptr(x), _ptr(logits), ctypes.byref(qw), ctypes.byref(sc),
                                    _ptr(adapter), int(chunk_experts), _ptr(out), _ptr(ws), ws.numel(), _stream()),
           "moe_expert_forward")
    return out


def expert_forward_noalloc(layer: MoeLayer, x, logits, w13, w2, s13, s2, adapter=None, chunk_experts: int = 1,
                           out: torch.Tensor | None = None, g13=None, g2=None):
    """moe_expert_forward_noalloc: as expert_forward, with the library's static
    per-GPU scratch in place of a workspace (layers whose workspace fits it)."""
    if out is None:
        out = torch.empty((layer.num_tokens, layer.hidden), dtype=torch.bfloat16, device=x.device)
    if workspace_bytes(layer, chunk_experts) <= NOALLOC_SCRATCH_BYTES:  # else the library refuses first
        _check_forward_args(layer, x, logits, w13, w2, s13, s2, adapter, out, g13, g2)
    qw = MoeQWeights(_ptr(w13), _ptr(w2))
    sc = MoeScales(_ptr(s13), _ptr(s2), _ptr(g13), _ptr(g2))
    _check(lib().moe_expert_forward_noalloc(ctypes.byref(layer), _ptr(x), _ptr(logits), ctypes.byref(qw),
                                            ctypes.byref(sc), _ptr(adapter), int(chunk_experts), _ptr(out),
                                            _stream()), "moe_expert_forward_noalloc")
    return out


def expert_forward_timed(layer: MoeLayer, x, logits, w13, w2, s13, s2, adapter=None, chunk_experts: int = 1,
                         out=None, ws=None, g13=None, g2=None):
    """moe_expert_forward_timed: same result, plus per-stage event times.
    Returns (out, {stage: (ms, launches)})."""
    if out is None:
        out = torch.empty((layer.num_tokens, layer.hidden), dtype=torch.bfloat16, device=x.device)
    if ws is None:
        ws = alloc_workspace(workspace_bytes(layer, chunk_experts), x.device)
    _check_forward_args(layer, x, logits, w13, w2, s13, s2, adapter, out, g13, g2)
    qw = MoeQWeights(_ptr(w13), _ptr(w2))
    sc = MoeScales(_ptr(s13), _ptr(s2), _ptr(g13), _ptr(g2))
    ms = (ctypes.c_float * len(STAGES))()
    n = (ctypes.c_int32 * len(STAGES))()
    _check(lib().moe_expert_forward_timed(ctypes.byref(layer), _ptr(x), _ptr(logits), ctypes.byref(qw),
                                          ctypes.byref(sc), _ptr(adapter), int(chunk_experts), _ptr(out), _ptr(ws),
                                          ws.numel(), _stream(), ms, n), "moe_expert_forward_timed")
    return out, {name: (float(ms[i]), int(n[i])) for i, name in enumerate(STAGES)}


def materialized_workspace_bytes(layer: MoeLayer, chunk_experts: int) -> int:
    return lib().moe_materialized_workspace_bytes(ctypes.byref(layer), int(chunk_experts))


def expert_forward_materialized(layer: MoeLayer, x, logits, w13, w2, s13, s2, adapter=None, chunk_experts: int = 1,
                                out=None, ws=None, timed: bool = False, g13=None, g2=None):
    """moe_expert_forward_materialized: per chunk, the experts' BF16 copy in ws,
    then BF16 GEMMs.  Returns out, or (out, {stage: (ms, launches)}) if timed."""
    if out is None:
        out = torch.empty((layer.num_tokens, layer.hidden), dtype=torch.bfloat16, device=x.device)
    if ws is None:
        ws = alloc_workspace(materialized_workspace_bytes(layer, chunk_experts), x.device)
    _check_forward_args(layer, x, logits, w13, w2, s13, s2, adapter, out, g13, g2)
    qw = MoeQWeights(_ptr(w13), _ptr(w2))
    sc = MoeScales(_ptr(s13), _ptr(s2), _ptr(g13), _ptr(g2))
    ms = (ctypes.c_float * len(STAGES))() if timed else None
    n = (ctypes.c_int32 * len(STAGES))() if timed else None
    _check(lib().moe_expert_forward_materialized(ctypes.byref(layer), _ptr(x), _ptr(logits), ctypes.byref(qw),
                                                 ctypes.byref(sc), _ptr(adapter), int(chunk_experts), _ptr(out),
                                                 _ptr(ws), ws.numel(), _stream(), ms, n),
           "moe_expert_forward_materialized")
    if timed:
        return out, {name: (float(ms[i]), int(n[i])) for i, name in enumerate(STAGES)}
    return out


def backward_weights_bytes(layer: MoeLayer) -> int:
    return lib().moe_backward_weights_bytes(ctypes.byref(layer))


def prepare_backward_weights(layer: MoeLayer, w13, w2, s13, s2, out: torch.Tensor | None = None) -> torch.Tensor:
    """moe_prepare_backward_weights: the transposed copy of the frozen weights."""
    n = backward_weights_bytes(layer)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_backward_weights_bytes")
    if out is None:
        out = torch.empty(n, dtype=torch.uint8, device=w13.device)
    qw = MoeQWeights(_ptr(w13), _ptr(w2))
    sc = MoeScales(_ptr(s13), _ptr(s2), None, None)
    _check(lib().moe_prepare_backward_weights(ctypes.byref(layer), ctypes.byref(qw), ctypes.byref(sc), _ptr(out),
                                              out.numel(), _stream()), "moe_prepare_backward_weights")
    return out


def pack_weights_kblocked(layer: MoeLayer, w13, w2):
    """moe_pack_weights_kblocked -> (w13, w2) in 16-row x 128-K tiles (same sizes)."""
    o13, o2 = torch.empty_like(w13), torch.empty_like(w2)
    qw = MoeQWeights(_ptr(w13), _ptr(w2))
    _check(lib().moe_pack_weights_kblocked(ctypes.byref(layer), ctypes.byref(qw), _ptr(o13), _ptr(o2), _stream()),
           "moe_pack_weights_kblocked")
    return o13, o2


def backward_workspace_bytes(layer: MoeLayer, chunk_experts: int = 1) -> int:
    return lib().moe_backward_workspace_bytes(ctypes.byref(layer), int(chunk_experts))


def expert_backward(layer: MoeLayer, x, logits, w13, w2, s13, s2, bwd_weights, d_out, adapter=None,
                    chunk_experts: int = 1, ws=None, d_x=None, d_logits=None, d_adapter=None, timed: bool = False,
                    g13=None, g2=None):
    """moe_expert_backward -> (d_x [T][H] bf16, d_logits [T][E] fp32, d_adapter fp32 or None)
    (+ {stage: (ms, launches)} if timed)."""
    T, H, E = layer.num_tokens, layer.hidden, layer.num_experts
    dev = x.device
    if d_x is None:
        d_x = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    if d_logits is None:
        d_logits = torch.empty((T, E), dtype=torch.float32, device=dev)
    if adapter is not None and d_adapter is None:
        d_adapter = torch.empty(adapter.shape, dtype=torch.float32, device=dev)
    if ws is None:
        ws = alloc_workspace(backward_workspace_bytes(layer, chunk_experts), dev)
    qw = MoeQWeights(_ptr(w13), _ptr(w2))
    sc = MoeScales(_ptr(s13), _ptr(s2), _ptr(g13), _ptr(g2))
    ms = (ctypes.c_float * len(STAGES))() if timed else None
    n = (ctypes.c_int32 * len(STAGES))() if timed else None
    _check(lib().moe_expert_backward(ctypes.byref(layer), _ptr(x), _ptr(logits), ctypes.byref(qw), ctypes.byref(sc),
                                     _ptr(bwd_weights), _ptr(adapter), _ptr(d_out), int(chunk_experts), _ptr(d_x),
                                     _ptr(d_logits), _ptr(d_adapter), _ptr(ws), ws.numel(), _stream(), ms, n),
           "moe_expert_backward")
    if timed:
        return d_x, d_logits, d_adapter, {name: (float(ms[i]), int(n[i])) for i, name in enumerate(STAGES)}
    return d_x, d_logits, d_adapter


def quantize_activations(layer: MoeLayer, x: torch.Tensor):
    """moe_quantize_activations -> (codes [T][H] uint8, scales): fp32 [T][H/128]
    for FP8 layers, E8M0 bytes [T][H/32] for MXFP4 layers."""
    T, H = layer.num_tokens, layer.hidden
    codes = torch.empty((T, H), dtype=torch.uint8, device=x.device)
    if layer.wformat in (FMT_FP8, FMT_FP8_POW2):
        scales = torch.empty((T, H // 128), dtype=torch.float32, device=x.device)
    else:
        scales = torch.empty((T, H // 32), dtype=torch.uint8, device=x.device)
    _check(lib().moe_quantize_activations(ctypes.byref(layer), _ptr(x), _ptr(codes), _ptr(scales), _stream()),
           "moe_quantize_activations")
    return codes, scales


def combine(layer: MoeLayer, y_perm: torch.Tensor, topk_w: torch.Tensor, row_of: torch.Tensor,
            out: torch.Tensor | None = None):
    if out is None:
        out = torch.empty((layer.num_tokens, layer.hidden), dtype=torch.bfloat16, device=y_perm.device)
    _check(lib().moe_combine(ctypes.byref(layer), _ptr(y_perm), _ptr(topk_w), _ptr(row_of), _ptr(out), _stream()),
           "moe_combine")
    return out


def lm_head_logprob(h: torch.Tensor, w_lm: torch.Tensor, targets: torch.Tensor, ws: torch.Tensor | None = None):
    T, H = h.shape
    V = w_lm.shape[0]
    lp = torch.empty(T, dtype=torch.float32, device=h.device)
    if ws is None:
        ws = alloc_workspace(lib().moe_lm_head_workspace_bytes(T, V), h.device)
    _check(lib().moe_lm_head_logprob(T, H, V, _ptr(h), _ptr(w_lm), _ptr(targets), _ptr(lp), _ptr(ws), ws.numel(),
                                     _stream()), "moe_lm_head_logprob")
    return lp


# ---- training losses ----

def _aligned(t, name: str) -> int:
    """The tensor's address, which the library wants on 16 bytes (a slice may start between them)."""
    p = t.data_ptr()
    if p % 16:
        raise ValueError(f"{name}: address not 16-byte aligned (a view that starts inside another tensor); "
                         "pass a clone()")
    return p


def _typed(t, name: str, dtype, shape, device):
    """The address of a contiguous tensor of this type and shape on the call's device."""
    if t is None or t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous {dtype} tensor of shape {tuple(shape)} on {device} expected, got "
                         + ("None" if t is None else f"{t.dtype} {tuple(t.shape)} on {t.device}"))
    return _aligned(t, name)


def _rows(t, name: str, device):
    """A bf16 matrix whose rows are contiguous; (pointer, row stride for the descriptor: 0 = contiguous)."""
    if t.dtype != torch.bfloat16 or t.dim() != 2 or t.device != device or not t.is_cuda:
        raise ValueError(f"{name}: bf16 device matrix expected, got {t.dtype} {tuple(t.shape)} on {t.device}")
    if t.is_contiguous():
        return _aligned(t, name), 0
    if t.stride(1) != 1 or t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}: rows must be contiguous and must not overlap, got strides {t.stride()}")
    return _aligned(t, name), t.stride(0)


def _raw_stream(device) -> int:
    """The current stream of the device as a handle (torch.cuda.current_stream builds an object first)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


class _On:
    """The device of the call's tensors, made current where it is not."""

    def __init__(self, device):
        if device.type != "cuda":
            raise ValueError("device tensors expected")
        self._d = None if device.index == torch.cuda.current_device() else torch.cuda.device(device)

    def __enter__(self):
        if self._d is not None:
            self._d.__enter__()

    def __exit__(self, *e):
        if self._d is not None:
            self._d.__exit__(*e)


def _head(h, w_lm, norm_eps, logit_scale):
    """(descriptor, pointer of h, pointer of W) of a call on h [T][H] and W [V][H]."""
    hp, hs = _rows(h, "h", h.device)
    wp, ws = _rows(w_lm, "w_lm", h.device)
    if h.shape[1] != w_lm.shape[1]:
        raise ValueError(f"h has {h.shape[1]} columns, w_lm {w_lm.shape[1]}")
    return MoeLmHead(h.shape[0], h.shape[1], w_lm.shape[0], norm_eps, logit_scale, hs, ws), hp, wp


def _head_ws(head, top: int, backward: bool, ws, device):
    if ws is None:
        ws = torch.empty(max(lib().moe_lm_head_loss_workspace_bytes(ctypes.byref(head), top, backward), 256),
                         dtype=torch.uint8, device=device)
    elif ws.device != device or not ws.is_contiguous():
        raise ValueError("ws: contiguous tensor on the call's device expected")
    return ws, ws.numel() * ws.element_size()


def lm_head_loss_workspace_bytes(T: int, H: int, V: int, top: int = 0, backward: bool = False) -> int:
    """Workspace of the head's losses: top = 0 for cross entropy, else the teacher logits per token."""
    return lib().moe_lm_head_loss_workspace_bytes(ctypes.byref(MoeLmHead(T, H, V, 0.0, 1.0, 0, 0)), top, backward)


def lm_head_loss(h: torch.Tensor, w_lm: torch.Tensor, targets: torch.Tensor, norm_eps: float = 1e-6,
                 logit_scale: float = 1.0, ws: torch.Tensor | None = None):
    """moe_lm_head_loss: cross entropy of targets [T] int32 (negative: the token
    does not count) under the head w_lm [V][H] on h [T][H]; rows of h and w_lm
    may be strided.  Returns (loss [T], lse [T]) fp32."""
    dev = h.device
    with _On(dev):
        head, hp, wp = _head(h, w_lm, norm_eps, logit_scale)
        T = head.num_tokens
        y = _typed(targets, "targets", torch.int32, (T,), dev)
        loss = torch.empty(T, dtype=torch.float32, device=dev)
        lse = torch.empty(T, dtype=torch.float32, device=dev)
        ws, nb = _head_ws(head, 0, False, ws, dev)
        _check(lib().moe_lm_head_loss(ctypes.byref(head), hp, wp, y, loss.data_ptr(), lse.data_ptr(), ws.data_ptr(),
                                      nb, _raw_stream(dev)), "moe_lm_head_loss")
    return loss, lse


def lm_head_loss_backward(h, w_lm, targets, loss, lse, d_loss, weight_grad: bool = False, norm_eps: float = 1e-6,
                          logit_scale: float = 1.0, ws: torch.Tensor | None = None):
    """moe_lm_head_loss_backward: (d_h [T][H] bf16, d_w [V][H] bf16 or None) for
    d_loss [T] fp32, with loss and lse from lm_head_loss on the same arguments."""
    dev = h.device
    with _On(dev):
        head, hp, wp = _head(h, w_lm, norm_eps, logit_scale)
        T = head.num_tokens
        y = _typed(targets, "targets", torch.int32, (T,), dev)
        lo = _typed(loss, "loss", torch.float32, (T,), dev)
        ls = _typed(lse, "lse", torch.float32, (T,), dev)
        dl = _typed(d_loss, "d_loss", torch.float32, (T,), dev)
        d_h = torch.empty((T, head.hidden), dtype=torch.bfloat16, device=dev)
        d_w = torch.empty((head.vocab, head.hidden), dtype=torch.bfloat16, device=dev) if weight_grad else None
        ws, nb = _head_ws(head, 0, True, ws, dev)
        _check(lib().moe_lm_head_loss_backward(ctypes.byref(head), hp, wp, y, lo, ls, dl, d_h.data_ptr(), _ptr(d_w),
                                               ws.data_ptr(), nb, _raw_stream(dev)), "moe_lm_head_loss_backward")
    return d_h, d_w


def lm_head_distill(h, w_lm, teacher_ids, teacher_logits, teacher_scale: float = 1.0, norm_eps: float = 1e-6,
                    logit_scale: float = 1.0, ws: torch.Tensor | None = None):
    """moe_lm_head_distill: KL divergence from the softmax over a teacher's top
    logits (teacher_ids [T][K] int32, absent where negative; teacher_logits
    [T][K] fp32) to the head's softmax.  Returns (loss [T], lse [T],
    logp [T][K]) fp32."""
    dev = h.device
    with _On(dev):
        head, hp, wp = _head(h, w_lm, norm_eps, logit_scale)
        T, K = head.num_tokens, teacher_ids.shape[-1]
        ip = _typed(teacher_ids, "teacher_ids", torch.int32, (T, K), dev)
        tp = _typed(teacher_logits, "teacher_logits", torch.float32, (T, K), dev)
        loss = torch.empty(T, dtype=torch.float32, device=dev)
        lse = torch.empty(T, dtype=torch.float32, device=dev)
        logp = torch.empty((T, K), dtype=torch.float32, device=dev)
        ws, nb = _head_ws(head, K, False, ws, dev)
        _check(lib().moe_lm_head_distill(ctypes.byref(head), K, teacher_scale, hp, wp, ip, tp, loss.data_ptr(),
                                         lse.data_ptr(), logp.data_ptr(), ws.data_ptr(), nb, _raw_stream(dev)),
               "moe_lm_head_distill")
    return loss, lse, logp


def lm_head_distill_backward(h, w_lm, teacher_ids, teacher_logits, lse, logp, d_loss, weight_grad: bool = False,
                             teacher_scale: float = 1.0, norm_eps: float = 1e-6, logit_scale: float = 1.0,
                             ws: torch.Tensor | None = None):
    """moe_lm_head_distill_backward: (d_h, d_w or None) as lm_head_loss_backward,
    with lse and logp from lm_head_distill on the same arguments."""
    dev = h.device
    with _On(dev):
        head, hp, wp = _head(h, w_lm, norm_eps, logit_scale)
        T, K = head.num_tokens, teacher_ids.shape[-1]
        ip = _typed(teacher_ids, "teacher_ids", torch.int32, (T, K), dev)
        tp = _typed(teacher_logits, "teacher_logits", torch.float32, (T, K), dev)
        ls = _typed(lse, "lse", torch.float32, (T,), dev)
        lp = _typed(logp, "logp", torch.float32, (T, K), dev)
        dl = _typed(d_loss, "d_loss", torch.float32, (T,), dev)
        d_h = torch.empty((T, head.hidden), dtype=torch.bfloat16, device=dev)
        d_w = torch.empty((head.vocab, head.hidden), dtype=torch.bfloat16, device=dev) if weight_grad else None
        ws, nb = _head_ws(head, K, True, ws, dev)
        _check(lib().moe_lm_head_distill_backward(ctypes.byref(head), K, teacher_scale, hp, wp, ip, tp, ls, lp, dl,
                                                  d_h.data_ptr(), _ptr(d_w), ws.data_ptr(), nb, _raw_stream(dev)),
               "moe_lm_head_distill_backward")
    return d_h, d_w


def _segments(layer, token_mask, seg_offsets, dev):
    """(segments, mask pointer, offsets pointer) of the balance calls."""
    S = 1 if seg_offsets is None else seg_offsets.numel() - 1
    if S < 1:
        raise ValueError("seg_offsets: at least two entries expected")
    if token_mask is not None and token_mask.dtype == torch.bool:
        token_mask = token_mask.view(torch.uint8)
    mp = None if token_mask is None else _typed(token_mask, "token_mask", torch.uint8, (layer.num_tokens,), dev)
    return S, mp, None if seg_offsets is None else _typed(seg_offsets, "seg_offsets", torch.int32, (S + 1,), dev)


def balance_loss(layer: MoeLayer, logits, topk_ids, token_mask=None, seg_offsets=None, ws=None):
    """moe_balance_loss on router logits [T][E] fp32 and topk_ids [T][k] int32
    (route_permute's), per segment of seg_offsets [S+1] int32 (None: one
    segment), over the tokens where token_mask [T] (bool or uint8) is set.
    Returns (loss [S], counts [S][E] int32, tokens [S] int32, probs [S][E])."""
    dev, T, E = logits.device, layer.num_tokens, layer.num_experts
    with _On(dev):
        S, mp, op = _segments(layer, token_mask, seg_offsets, dev)
        lp = _typed(logits, "logits", torch.float32, (T, E), dev)
        ip = _typed(topk_ids, "topk_ids", torch.int32, (T, layer.top_k), dev)
        loss = torch.empty(S, dtype=torch.float32, device=dev)
        counts = torch.empty((S, E), dtype=torch.int32, device=dev)
        tokens = torch.empty(S, dtype=torch.int32, device=dev)
        probs = torch.empty((S, E), dtype=torch.float32, device=dev)
        if ws is None:
            ws = torch.empty(max(lib().moe_balance_loss_workspace_bytes(ctypes.byref(layer), S), 256),
                             dtype=torch.uint8, device=dev)
        elif ws.device != dev or not ws.is_contiguous():
            raise ValueError("ws: contiguous tensor on the call's device expected")
        _check(lib().moe_balance_loss(ctypes.byref(layer), lp, ip, mp, op, S, loss.data_ptr(), counts.data_ptr(),
                                      tokens.data_ptr(), probs.data_ptr(), ws.data_ptr(),
                                      ws.numel() * ws.element_size(), _raw_stream(dev)), "moe_balance_loss")
    return loss, counts, tokens, probs


def balance_loss_backward(layer: MoeLayer, logits, counts, tokens, d_loss, token_mask=None, seg_offsets=None,
                          d_logits: torch.Tensor | None = None):
    """moe_balance_loss_backward: dL/dlogits [T][E] fp32 for d_loss [S] fp32, with
    counts and tokens from balance_loss.  Where d_logits is given (the one of
    expert_backward), the gradient is added to it."""
    dev, T, E = logits.device, layer.num_tokens, layer.num_experts
    with _On(dev):
        S, mp, op = _segments(layer, token_mask, seg_offsets, dev)
        lp = _typed(logits, "logits", torch.float32, (T, E), dev)
        cp = _typed(counts, "counts", torch.int32, (S, E), dev)
        np_ = _typed(tokens, "tokens", torch.int32, (S,), dev)
        dl = _typed(d_loss, "d_loss", torch.float32, (S,), dev)
        add = d_logits is not None
        if not add:
            d_logits = torch.empty((T, E), dtype=torch.float32, device=dev)
        dp = _typed(d_logits, "d_logits", torch.float32, (T, E), dev)
        _check(lib().moe_balance_loss_backward(ctypes.byref(layer), lp, mp, op, S, cp, np_, dl, add, dp, _raw_stream(dev)),
               "moe_balance_loss_backward")
    return d_logits


# ---- the gate ----

def make_gate(score: int = GATE_SIGMOID, groups: int = 1, top_groups: int = 1, group_score: int = GROUP_TOP2,
              renormalize: bool = True, scale: float = 1.0) -> MoeGate:
    """A gate's descriptor (moe_gate): score GATE_SOFTMAX or GATE_SIGMOID, the
    top_groups best of `groups` groups by GROUP_MAX or GROUP_TOP2."""
    return MoeGate(score, groups, top_groups, group_score, int(renormalize), scale)


def _elsewhere(device) -> bool:
    """Whether a call's device is not the current one (the caller then makes it current and calls itself again)."""
    if device.type != "cuda":
        raise ValueError("device tensors expected")
    return device.index != torch._C._cuda_getDevice()


def _workspace(nbytes: int, ws, like):
    """(workspace, its address, its bytes): the caller's, a new one, or none where none is needed."""
    if ws is None:
        if nbytes == 0:
            return None, None, 0
        ws = like.new_empty(nbytes, dtype=torch.uint8)
        return ws, ws.data_ptr(), nbytes
    if ws.device != like.device or not ws.is_contiguous():
        raise ValueError("ws: contiguous tensor on the call's device expected")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _gate_inputs(layer, logits, bias):
    """(device, pointer of logits, pointer of bias or None) of a gate's call."""
    dev, E = logits.device, layer.num_experts
    return (dev, _typed(logits, "logits", torch.float32, (layer.num_tokens, E), dev),
            None if bias is None else _typed(bias, "bias", torch.float32, (E,), dev))


def route_gated(layer: MoeLayer, gate: MoeGate, logits, bias=None, permute: bool = True, ws=None) -> dict:
    """moe_route_gated on router logits [T][E] fp32 with a balance bias [E] fp32:
    a dict as route_permute's; without `permute` only topk_ids and topk_w."""
    if _elsewhere(logits.device):
        with torch.cuda.device(logits.device):
            return route_gated(layer, gate, logits, bias, permute, ws)
    T, E, k = layer.num_tokens, layer.num_experts, layer.top_k
    dev, lp, bp = _gate_inputs(layer, logits, bias)
    ids, w = logits.new_empty((T, k), dtype=torch.int32), logits.new_empty((T, k))
    out = dict(topk_ids=ids, topk_w=w)
    ro, wp, nb = MoeRouteOut(ids.data_ptr(), w.data_ptr()), None, 0
    if permute:
        for name, n in (("expert_offsets", E + 1), ("sorted_rows", T * k), ("row_of", T * k), ("active_experts", E),
                        ("num_active", 4)):
            out[name] = (torch.empty if T else torch.zeros)(n, dtype=torch.int32, device=dev)
            setattr(ro, name, out[name].data_ptr())
        ws, wp, nb = _workspace(lib().moe_route_workspace_bytes(ctypes.byref(layer)), ws, logits)
    _check(lib().moe_route_gated(ctypes.byref(layer), ctypes.byref(gate), lp, bp, ctypes.byref(ro), wp, nb,
                                 _raw_stream(dev)), "moe_route_gated")
    return out


def route_gated_backward(layer: MoeLayer, gate: MoeGate, logits, topk_ids, d_topk_w, bias=None,
                         d_logits: torch.Tensor | None = None):
    """moe_route_gated_backward: dL/dlogits [T][E] fp32 for d_topk_w [T][k] fp32, with
    topk_ids from route_gated.  Where d_logits is given (balance_loss_backward's),
    the gradient is added to it."""
    if _elsewhere(logits.device):
        with torch.cuda.device(logits.device):
            return route_gated_backward(layer, gate, logits, topk_ids, d_topk_w, bias, d_logits)
    T, E, k = layer.num_tokens, layer.num_experts, layer.top_k
    dev, lp, bp = _gate_inputs(layer, logits, bias)
    ip = _typed(topk_ids, "topk_ids", torch.int32, (T, k), dev)
    wp = _typed(d_topk_w, "d_topk_w", torch.float32, (T, k), dev)
    add = d_logits is not None
    if not add:
        d_logits = torch.empty_like(logits)
    dp = _typed(d_logits, "d_logits", torch.float32, (T, E), dev)
    _check(lib().moe_route_gated_backward(ctypes.byref(layer), ctypes.byref(gate), lp, bp, ip, wp, add, dp,
                                          _raw_stream(dev)), "moe_route_gated_backward")
    return d_logits


def expert_forward_gated(layer: MoeLayer, gate: MoeGate, x, logits, w13, w2, s13, s2, bias=None, adapter=None,
                         chunk_experts: int = 1, out: torch.Tensor | None = None, ws=None, g13=None, g2=None):
    """moe_expert_forward_gated: expert_forward with its routing through a gate."""
    with _On(logits.device):
        dev, lp, bp = _gate_inputs(layer, logits, bias)
        if out is None:
            out = torch.empty((layer.num_tokens, layer.hidden), dtype=torch.bfloat16, device=dev)
        ws, wp, nb = _workspace(workspace_bytes(layer, chunk_experts), ws, logits)
        _check_forward_args(layer, x, logits, w13, w2, s13, s2, adapter, out, g13, g2)
        qw = MoeQWeights(_ptr(w13), _ptr(w2))
        sc = MoeScales(_ptr(s13), _ptr(s2), _ptr(g13), _ptr(g2))
        _check(lib().moe_expert_forward_gated(ctypes.byref(layer), ctypes.byref(gate), _ptr(x), lp, bp,
                                              ctypes.byref(qw), ctypes.byref(sc), _ptr(adapter), int(chunk_experts),
                                              _ptr(out), wp, nb, _raw_stream(dev)),
               "moe_expert_forward_gated")
    return out


def expert_backward_gated(layer: MoeLayer, gate: MoeGate, x, logits, w13, w2, s13, s2, bwd_weights, d_out, bias=None,
                          adapter=None, chunk_experts: int = 1, ws=None, g13=None, g2=None):
    """moe_expert_backward_gated -> (d_x [T][H] bf16, d_logits [T][E] fp32, d_adapter fp32 or None)."""
    T, H, E = layer.num_tokens, layer.hidden, layer.num_experts
    with _On(logits.device):
        dev, lp, bp = _gate_inputs(layer, logits, bias)
        d_x = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        d_logits = torch.empty((T, E), dtype=torch.float32, device=dev)
        d_adapter = None if adapter is None else torch.empty(adapter.shape, dtype=torch.float32, device=dev)
        ws, wp, nb = _workspace(backward_workspace_bytes(layer, chunk_experts), ws, logits)
        _check_forward_args(layer, x, logits, w13, w2, s13, s2, adapter, d_x, g13, g2)
        _need(d_out, "d_out", T * H * 2, 2)
        _need(bwd_weights, "bwd_weights", backward_weights_bytes(layer))
        qw = MoeQWeights(_ptr(w13), _ptr(w2))
        sc = MoeScales(_ptr(s13), _ptr(s2), _ptr(g13), _ptr(g2))
        _check(lib().moe_expert_backward_gated(ctypes.byref(layer), ctypes.byref(gate), _ptr(x), lp, bp,
                                               ctypes.byref(qw), ctypes.byref(sc), _ptr(bwd_weights), _ptr(adapter),
                                               _ptr(d_out), int(chunk_experts), d_x.data_ptr(), d_logits.data_ptr(),
                                               _ptr(d_adapter), wp, nb, _raw_stream(dev)),
               "moe_expert_backward_gated")
    return d_x, d_logits, d_adapter


# ---- the dense FP8 projection ----

def _codes(w, name: str, device):
    """The address of a matrix of E4M3 codes (uint8 or float8_e4m3fn)."""
    if w.dtype == torch.float8_e4m3fn:
        w = w.view(torch.uint8)
    return _typed(w, name, torch.uint8, w.shape if w.dim() == 2 else (0, 0), device)


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _apart(out, inputs):
    """Refuses a result that lies over an input: workgroups still read the input while others write."""
    first = out.data_ptr()
    end = first + out.numel() * out.element_size()
    for t in inputs:
        if t.numel() and out.numel():
            a = t.data_ptr()
            last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
            if first < a + (last + 1) * t.element_size() and a < end:
                raise ValueError("out: overlaps an input")


def fp8_linear_workspace_bytes(M: int, K: int, N: int, grads: int = LINEAR_FORWARD) -> int:
    """Workspace of fp8_linear, or of fp8_linear_backward for LINEAR_D_X, LINEAR_D_W or both or-ed."""
    return lib().moe_fp8_linear_workspace_bytes(ctypes.byref(MoeLinear(M, K, N, FMT_FP8, 0, 0)), grads)


def fp8_linear(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, fmt: int = FMT_FP8,
               out: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """moe_fp8_linear: x [M][K] bf16 (rows may be strided) through W [N][K] in E4M3
    codes with scales [ceil(N/128)][ceil(K/128)] fp32 -> [M][N] bf16."""
    dev = x.device
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return fp8_linear(x, w, w_scale, fmt, out, ws)
    xp, xs = _rows(x, "x", dev)
    wp = _codes(w, "w", dev)
    (M, K), N = x.shape, w.shape[0]
    if w.shape[1] != K:
        raise ValueError(f"x has {K} columns, w {w.shape[1]}")
    sp = _typed(w_scale, "w_scale", torch.float32, (_blocks(N), _blocks(K)), dev)
    lin = MoeLinear(M, K, N, fmt, xs, 0)
    if out is None:
        out = x.new_empty((M, N))
    else:
        _apart(out, (x, w, w_scale))
    op = _typed(out, "out", torch.bfloat16, (M, N), dev)
    need = lib().moe_fp8_linear_workspace_bytes(ctypes.byref(lin), LINEAR_FORWARD) if ws is None else 0
    ws, wsp, nb = _workspace(need, ws, x)
    _check(lib().moe_fp8_linear(ctypes.byref(lin), xp, wp, sp, op, wsp, nb, _raw_stream(dev)), "moe_fp8_linear")
    return out


def fp8_linear_transpose(w: torch.Tensor, w_scale: torch.Tensor):
    """moe_fp8_linear_transpose -> (w_t [K][N] uint8, w_t_scale): what fp8_linear_backward reads."""
    dev = w.device
    with _On(dev):
        wp = _codes(w, "w", dev)
        N, K = w.shape
        sp = _typed(w_scale, "w_scale", torch.float32, (_blocks(N), _blocks(K)), dev)
        wt = torch.empty((K, N), dtype=torch.uint8, device=dev)
        st = torch.empty((_blocks(K), _blocks(N)), dtype=torch.float32, device=dev)
        _check(lib().moe_fp8_linear_transpose(ctypes.byref(MoeLinear(0, K, N, FMT_FP8, 0, 0)), wp, sp, wt.data_ptr(),
                                              st.data_ptr(), _raw_stream(dev)), "moe_fp8_linear_transpose")
    return wt, st


def fp8_linear_backward(d_y: torch.Tensor, w_t: torch.Tensor, w_t_scale: torch.Tensor, fmt: int = FMT_FP8,
                        x: torch.Tensor | None = None, input_grad: bool = True, weight_grad: bool = False,
                        ws: torch.Tensor | None = None):
    """moe_fp8_linear_backward -> (d_x [M][K] bf16 or None, d_w [N][K] bf16 or None) for
    d_y [M][N] bf16, with fp8_linear_transpose's copy of W and, for d_w, the
    forward's x [M][K] bf16 (rows of d_y and x may be strided)."""
    dev = d_y.device
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return fp8_linear_backward(d_y, w_t, w_t_scale, fmt, x, input_grad, weight_grad, ws)
    yp, ys = _rows(d_y, "d_y", dev)
    wp = _codes(w_t, "w_t", dev)
    (M, N), K = d_y.shape, w_t.shape[0]
    if w_t.shape[1] != N:
        raise ValueError(f"d_y has {N} columns, w_t {w_t.shape[1]}")
    sp = _typed(w_t_scale, "w_t_scale", torch.float32, (_blocks(K), _blocks(N)), dev)
    xp, xs = None, 0
    if weight_grad:
        if x is None:
            raise ValueError("x: needed for the weight's gradient")
        xp, xs = _rows(x, "x", dev)
        if tuple(x.shape) != (M, K):
            raise ValueError(f"x: shape {(M, K)} expected, got {tuple(x.shape)}")
    lin = MoeLinear(M, K, N, fmt, xs, ys)
    d_x = d_y.new_empty((M, K)) if input_grad else None
    d_w = d_y.new_empty((N, K)) if weight_grad else None
    grads = (LINEAR_D_X if input_grad else 0) | (LINEAR_D_W if weight_grad else 0)
    need = lib().moe_fp8_linear_workspace_bytes(ctypes.byref(lin), grads) if ws is None else 0
    ws, wsp, nb = _workspace(need, ws, d_y)
    _check(lib().moe_fp8_linear_backward(ctypes.byref(lin), yp, wp, sp, xp, _ptr(d_x), _ptr(d_w), wsp, nb,
                                         _raw_stream(dev)), "moe_fp8_linear_backward")
    return d_x, d_w


# ---- clipping by the global norm ----

def _lists(grads, out):
    """What may be readable once only, as lists: a call on another device than the current one reads it twice."""
    return (grads if isinstance(grads, list) else list(grads),
            out if out is None or isinstance(out, list) else list(out))


def _tensors(grads, out, write: bool = True):
    """(device, moe_tensor array, count) of a list of gradients; out: None (in place), or where the results go."""
    dest = grads if out is None else out
    n = len(grads)
    if len(dest) != n:
        raise ValueError(f"out: {len(dest)} tensors for {n}")
    if n == 0:
        return torch.device("cuda", torch.cuda.current_device()), None, 0
    dev, spans, flat = grads[0].device, [], []
    if dev.type != "cuda":
        raise ValueError("device tensors expected")
    index = dev.index
    for i, (g, o) in enumerate(zip(grads, dest)):
        kind = _DTYPES.get(g.dtype)
        if kind is None or g.get_device() != index or not g.is_contiguous():
            raise ValueError(f"grads[{i}]: contiguous fp32, bf16 or fp16 tensor on {dev} expected, got {g.dtype} "
                             f"{tuple(g.shape)} on {g.device}")
        first, size = g.data_ptr(), g.numel()
        to = first
        if o is not g:
            if o.dtype != g.dtype or o.shape != g.shape or o.get_device() != index or not o.is_contiguous():
                raise ValueError(f"out[{i}]: contiguous {g.dtype} {tuple(g.shape)} on {dev} expected, got {o.dtype} "
                                 f"{tuple(o.shape)} on {o.device}")
            to = o.data_ptr()
        if write and size:
            nb = size * 4 if kind == 0 else size * 2
            spans.append((to, to + nb, True))
            if to != first:
                spans.append((first, first + nb, False))
        flat += (first, to, size, kind)
    spans.sort()
    written = read = 0  # ends of what lies before, in the order of addresses
    for first, end, writes in spans:
        if first < written or (writes and first < read):
            raise ValueError("grads, out: tensors overlap")
        if writes:
            written = end
        elif end > read:
            read = end
    # moe_tensor is four 8-byte words (the type in the lower half of the last)
    return dev, (ctypes.c_int64 * (4 * n))(*flat), n


def _norm_call(grads, out, ws, max_norm):
    grads, out = _lists(grads, out)
    dev, arr, n = _tensors(grads, out, write=max_norm is not None)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return _norm_call(grads, out, ws, max_norm)
    norm = torch.empty(1, dtype=torch.float32, device=dev)
    ws, wp, nb = _workspace(lib().moe_grad_norm_workspace_bytes(n) if ws is None else 0, ws, norm)
    if max_norm is None:
        _check(lib().moe_grad_norm(arr, n, norm.data_ptr(), wp, nb, _raw_stream(dev)), "moe_grad_norm")
    else:
        _check(lib().moe_grad_clip(arr, n, max_norm, norm.data_ptr(), wp, nb, _raw_stream(dev)), "moe_grad_clip")
    return norm


def grad_norm(grads, ws: torch.Tensor | None = None) -> torch.Tensor:
    """moe_grad_norm: the 2-norm over every element of every tensor (fp32, bf16 or
    fp16), as a device tensor [1] fp32."""
    return _norm_call(grads, None, ws, None)


def clip_grads(grads, max_norm: float, out=None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """moe_grad_clip: scales the tensors by max_norm / norm where their common norm
    is larger, in place or into the tensors `out`; returns the norm [1] fp32."""
    return _norm_call(grads, out, ws, float(max_norm))


def scale_grads(grads, norm: torch.Tensor, max_norm: float, out=None) -> None:
    """moe_grad_scale: the scaling of clip_grads for a norm [1] fp32 on the device (one joined over ranks)."""
    grads, out = _lists(grads, out)
    dev, arr, n = _tensors(grads, out)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return scale_grads(grads, norm, max_norm, out)
    if norm.dtype != torch.float32 or norm.numel() != 1 or norm.device != dev:
        raise ValueError(f"norm: one fp32 value on {dev} expected")
    at = norm.data_ptr()
    if n and any(size and to - 4 < at < to + size * (4 if kind == 0 else 2)
                 for to, size, kind in zip(arr[1::4], arr[2::4], arr[3::4])):
        raise ValueError("norm: lies in a tensor that is written")
    _check(lib().moe_grad_scale(arr, n, norm.data_ptr(), max_norm, _raw_stream(dev)), "moe_grad_scale")
