"""Python binding of libsi_moe: the decode-time MoE FFN stage on GB300.

Argument marshalling only. Every step of the computation runs in the CUDA
kernels of ``libsi_moe.so`` (built in-tree from ``csrc/``); PyTorch supplies
device memory and streams. There is no CPU fallback: if the library is not
built, or a tensor is not on a CUDA device, the calls raise.

Names follow the C ABI in ``include/si_moe.h``. Results carry no gradient, but for
those of ``si_moe_gather``, ``si_moe_combine``, ``si_moe_matmul``, ``si_swiglu``,
``si_moe_gateup`` and ``si_moe_experts``.
"""
from __future__ import annotations

import ctypes
import os

import torch
import torch.autograd.forward_ad as _forward_ad
from torch.autograd.function import once_differentiable

from ._build import LIB, build  # noqa: F401

SI_OK, SI_ERR_INVALID_ARG, SI_ERR_UNSUPPORTED, SI_ERR_WORKSPACE = 0, 1, 2, 3
SI_ERR_CUDA, SI_ERR_HANDSHAKE, SI_ERR_TIMEOUT = 4, 5, 6
SI_F32, SI_F16, SI_Q8_0, SI_Q8_1, SI_Q4_K, SI_Q5_K, SI_BF16 = 0, 1, 8, 9, 12, 13, 30
DTYPES = {"f32": SI_F32, "f16": SI_F16, "q8_0": SI_Q8_0, "q8_1": SI_Q8_1, "q4_k": SI_Q4_K,
          "q5_k": SI_Q5_K, "bf16": SI_BF16}

_vp = ctypes.c_void_p
_i32, _i64, _sz, _f32 = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


class SiError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


class SiMoeLayer(ctypes.Structure):
    """Mirror of ``si_moe_layer``."""
    _fields_ = [
        ("hidden", _i32), ("n_experts", _i32), ("top_k", _i32), ("inter", _i32),
        ("expert_type", _i32), ("w_gate", _vp), ("w_up", _vp), ("w_down", _vp),
        ("shared_inter", _i32), ("shared_type", _i32),
        ("ws_gate", _vp), ("ws_up", _vp), ("ws_down", _vp), ("w_shared_sigmoid", _vp),
        ("w_router", _vp), ("router_type", _i32), ("w_norm", _vp), ("eps", _f32),
        ("down_type", _i32),
    ]


class SiMxfp4Experts(ctypes.Structure):
    """Mirror of ``si_mxfp4_experts``."""
    _fields_ = [
        ("hidden", _i32), ("inter", _i32), ("n_experts", _i32),
        ("gate_codes", _vp), ("gate_scales", _vp), ("up_codes", _vp), ("up_scales", _vp),
        ("down_codes", _vp), ("down_scales", _vp),
    ]


class SiExperts(ctypes.Structure):
    """Mirror of ``si_experts``."""
    _fields_ = [
        ("type", _i32), ("hidden", _i32), ("inter", _i32), ("n_experts", _i32), ("gate_up", _vp), ("down", _vp),
    ]


# name -> (restype, argtypes), exactly the exports of include/si_moe.h
SIGNATURES = {
    "si_status_string": (ctypes.c_char_p, [_i32]),
    "si_version": (_i32, []),
    "si_row_bytes": (_sz, [_i32, _i64]),
    "si_quantize_q8_1": (_i32, [_vp, _i32, _i64, _vp, _vp]),
    "si_moe_router_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "si_moe_router_topk": (_i32, [_vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp,
                                  _vp, _sz, _vp]),
    "si_moe_router_topk_noalloc": (_i32, [_vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp,
                                          _vp, _vp]),
    "si_moe_router_noalloc_status": (_i32, [_vp, ctypes.POINTER(_i32)]),
    "si_moe_ffn_workspace_bytes": (_sz, [ctypes.POINTER(SiMoeLayer), _i32]),
    "si_moe_ffn_decode": (_i32, [ctypes.POINTER(SiMoeLayer), _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                 _vp, _sz, _vp]),
    "si_moe_ffn_decode_ep": (_i32, [ctypes.POINTER(SiMoeLayer), _i32, _i32, _vp, _vp, _vp, _vp, _vp,
                                    _vp, _sz, _vp]),
    "si_moe_combine_slots": (_i32, [_vp, _vp, _i32, _i32, _vp, _vp]),
    "si_moe_ffn_batched_workspace_bytes": (_sz, [ctypes.POINTER(SiMoeLayer), _i32]),
    "si_moe_ffn_batched": (_i32, [ctypes.POINTER(SiMoeLayer), _i32, _i32, _vp, _vp, _vp, _vp, _vp,
                                  _sz, _vp]),
    "si_add_rmsnorm3": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _f32, _vp, _vp, _vp, _vp]),
    "si_moe_layer_workspace_bytes": (_sz, [ctypes.POINTER(SiMoeLayer)]),
    "si_moe_layer_decode": (_i32, [ctypes.POINTER(SiMoeLayer), _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                   _vp, _vp, _sz, _vp]),
    "si_moe_stack_workspace_bytes": (_sz, [ctypes.POINTER(SiMoeLayer), _i32]),
    "si_moe_stack_graph_create": (_i32, [ctypes.POINTER(SiMoeLayer), _i32, _i32, _vp, _vp, _vp,
                                         _vp, _vp, _sz, _vp, ctypes.POINTER(_vp)]),
    "si_moe_stack_graph_create_mode": (_i32, [ctypes.POINTER(SiMoeLayer), _i32, _i32, _vp, _vp,
                                              _vp, _vp, _vp, _sz, _i32, _vp,
                                              ctypes.POINTER(_vp)]),
    "si_graph_is_persistent": (_i32, [_vp]),
    "si_moe_layer_batched_workspace_bytes": (_sz, [ctypes.POINTER(SiMoeLayer), _i32]),
    "si_moe_layer_decode_batched": (_i32, [ctypes.POINTER(SiMoeLayer), _i32, _i32, _vp, _vp, _vp, _vp,
                                           _vp, _vp, _vp, _vp, _sz, _vp]),
    "si_moe_stack_batched_workspace_bytes": (_sz, [ctypes.POINTER(SiMoeLayer), _i32, _i32]),
    "si_moe_stack_graph_create_batched": (_i32, [ctypes.POINTER(SiMoeLayer), _i32, _i32, _i32, _vp,
                                                 _vp, _vp, _vp, _vp, _sz, _vp, ctypes.POINTER(_vp)]),
    "si_requant_q4_k": (_i32, [_vp, _i32, _i64, _i64, _vp, _vp]),
    "si_mxfp4_scale_bytes": (_sz, [_i64, _i64]),
    "si_quantize_mxfp4": (_i32, [_vp, _i32, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _vp]),
    "si_dequantize_mxfp4": (_i32, [_vp, _vp, _i64, _i64, _i64, _vp, _i32, _i64, _i64, _vp]),
    "si_mxfp4_matmul_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "si_mxfp4_matmul": (_i32, [_vp, _vp, _i64, _vp, _vp, _i64, _i64, _vp, _i32, _i64, _vp, _sz, _vp]),
    "si_moe_sort_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "si_moe_sort": (_i32, [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "si_moe_gather": (_i32, [_vp, _i32, _i32, _i32, _i64, _vp, _vp, _vp, _vp]),
    "si_moe_gather_backward": (_i32, [_vp, _i32, _i32, _i32, _i64, _vp, _vp, _vp]),
    "si_moe_combine": (_i32, [_vp, _i32, _i32, _i32, _i64, _vp, _vp, _vp, _vp]),
    "si_moe_combine_f32": (_i32, [_vp, _i32, _i32, _i64, _vp, _vp, _vp, _i32, _vp]),
    "si_moe_combine_backward": (_i32, [_vp, _vp, _i32, _i32, _i32, _i64, _vp, _vp, _vp, _vp, _vp,
                                       _vp]),
    "si_moe_matmul_workspace_bytes": (_sz, []),
    "si_moe_matmul": (_i32, [_vp, _i32, _i64, _i64, _vp, _i32, _i64, _i64, _i64, _i64, _i32, _vp, _vp, _i32, _i64,
                             _vp, _sz, _vp]),
    "si_moe_matmul_grad_w": (_i32, [_vp, _i64, _vp, _i64, _i32, _i64, _i32, _i64, _i64, _vp, _vp, _i32, _vp, _sz,
                                    _vp]),
    "si_moe_gateup": (_i32, [_vp, _i32, _i64, _i64, _vp, _i32, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "si_moe_down_backward_workspace_bytes": (_sz, [_i64, _i32, _i64]),
    "si_moe_down_backward": (_i32, [_vp, _i32, _i64, _i64, _vp, _i32, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                    _vp, _vp, _sz, _vp]),
    "si_moe_experts_workspace_bytes": (_sz, [ctypes.POINTER(SiExperts), _i32, _i32]),
    "si_moe_experts_kept_bytes": (_sz, [ctypes.POINTER(SiExperts), _i32, _i32]),
    "si_moe_experts": (_i32, [ctypes.POINTER(SiExperts), _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "si_moe_experts_backward": (_i32, [ctypes.POINTER(SiExperts), _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                       _vp, _sz, _vp]),
    "si_quantize_mxint8": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _vp, _vp]),
    "si_dequantize_mxint8": (_i32, [_vp, _vp, _i64, _i64, _vp, _i32, _i64, _vp]),
    "si_swiglu": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _vp, _vp, _vp]),
    "si_swiglu_backward": (_i32, [_vp, _i32, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "si_moe_ffn_mxfp4_workspace_bytes": (_sz, [ctypes.POINTER(SiMxfp4Experts), _i32, _i32]),
    "si_moe_ffn_mxfp4": (_i32, [ctypes.POINTER(SiMxfp4Experts), _i32, _i32, _vp, _vp, _vp, _vp, _vp,
                                _sz, _vp]),
    "si_graph_launch": (_i32, [_vp, _vp]),
    "si_graph_destroy": (None, [_vp]),
    "si_workspace_status": (_i32, [_vp, _vp, ctypes.POINTER(_i32)]),
    "si_moe_ffn_gateup": (_i32, [ctypes.POINTER(SiMoeLayer), _i32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "si_test_q4k_block_dots": (_i32, [_vp, _i32, _i32, _vp, _vp, _vp]),
    "si_test_block_dots": (_i32, [_i32, _vp, _i32, _i32, _vp, _i32, _vp, _vp]),
    "si_test_wait_timeout": (_i32, [ctypes.c_uint64, _vp, _vp]),
    "si_test_poll_timeout": (_i32, [ctypes.c_uint64, _vp, _vp]),
    "si_test_umma_f16": (_i32, [_vp, _vp, _i32, _i32, _vp, _vp, _vp]),
    "si_test_unfused_add_rmsnorm": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _f32, _vp, _vp, _vp,
                                           _vp]),
}

_lib = None


def library() -> ctypes.CDLL:
    """The loaded libsi_moe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise RuntimeError(f"{LIB} is not built; run moe_decode_ffn_gb300.build() first")
        lib = ctypes.CDLL(LIB)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return library().si_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != SI_OK:
        raise SiError(status, where)


def _cuda(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _opt(t, name):
    return None if t is None else _cuda(t, name)


def _shaped(t, name: str, numel: int, dtypes) -> int:
    """Device pointer of ``t`` after checking that it holds exactly ``numel``
    elements of one of ``dtypes``: the C ABI takes raw pointers and cannot
    tell a short buffer from a long one."""
    p = _cuda(t, name)
    if t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    return p


_BF16 = (torch.bfloat16,)
_FLOATS = (torch.bfloat16, torch.float32)
_I32 = (torch.int32,)
_F32 = (torch.float32,)
_U8 = (torch.uint8,)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _xtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SI_BF16
    if t.dtype == torch.float32:
        return SI_F32
    raise ValueError(f"unsupported dtype {t.dtype}")


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """A zeroed, 256-byte aligned device workspace of ``nbytes`` bytes."""
    if nbytes <= 0:
        raise ValueError("workspace size query returned 0 (invalid shapes)")
    return torch.zeros(int(nbytes), dtype=torch.uint8, device=device or "cuda")


# ----------------------------------------------------------------------------
# calls
# ----------------------------------------------------------------------------

def si_quantize_q8_1(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    n = x.numel()
    if out is None:
        out = torch.empty(n // 32 * 36, dtype=torch.uint8, device=x.device)
    _check(library().si_quantize_q8_1(_cuda(x, "x"), _xtype(x), n,
                                      _shaped(out, "out", n // 32 * 36, _U8), _stream(stream)),
           "si_quantize_q8_1")
    return out


def router_workspace_bytes(n_experts: int, hidden: int, n_tokens: int) -> int:
    return int(library().si_moe_router_workspace_bytes(n_experts, hidden, n_tokens))


def si_moe_router_topk(x: torch.Tensor, w_router: torch.Tensor, top_k: int = 8,
                       want_logits: bool = False, ws: torch.Tensor | None = None, stream=None):
    """x [T, H], w_router [E, H] (bf16 or fp32) -> (ids int32 [T, k], w fp32 [T, k], logits|None)."""
    T, H = x.shape
    E = w_router.shape[0]
    if tuple(w_router.shape) != (E, H):
        raise ValueError(f"w_router has shape {tuple(w_router.shape)}, expected ({E}, {H})")
    dev = x.device
    ids = torch.empty(T, top_k, dtype=torch.int32, device=dev)
    wts = torch.empty(T, top_k, dtype=torch.float32, device=dev)
    logits = torch.empty(T, E, dtype=torch.float32, device=dev) if want_logits else None
    if ws is None:
        ws = workspace(router_workspace_bytes(E, H, T), dev)
    _check(library().si_moe_router_topk(
        _cuda(x, "x"), _xtype(x), _cuda(w_router, "w_router"), _xtype(w_router), H, E, top_k, T,
        _cuda(ids, "ids"), _cuda(wts, "w"), _opt(logits, "logits"), _cuda(ws, "ws"), ws.numel(),
        _stream(stream)), "si_moe_router_topk")
    return ids, wts, logits


def si_moe_router_topk_noalloc(x: torch.Tensor, w_router: torch.Tensor, top_k: int = 8,
                               want_logits: bool = False, stream=None):
    """Router + top-k through the entry point that allocates nothing on the
    device side (its scratch is built into the library). The output tensors
    here are the caller's; the call itself needs no workspace."""
    T, H = x.shape
    E = w_router.shape[0]
    if tuple(w_router.shape) != (E, H):
        raise ValueError(f"w_router has shape {tuple(w_router.shape)}, expected ({E}, {H})")
    dev = x.device
    ids = torch.empty(T, top_k, dtype=torch.int32, device=dev)
    wts = torch.empty(T, top_k, dtype=torch.float32, device=dev)
    logits = torch.empty(T, E, dtype=torch.float32, device=dev) if want_logits else None
    _check(library().si_moe_router_topk_noalloc(
        _cuda(x, "x"), _xtype(x), _cuda(w_router, "w_router"), _xtype(w_router), H, E, top_k, T,
        _cuda(ids, "ids"), _cuda(wts, "w"), _opt(logits, "logits"), _stream(stream)),
        "si_moe_router_topk_noalloc")
    return ids, wts, logits


def si_moe_router_noalloc_status(stream=None) -> int:
    """Reads and clears the device status of the no-alloc router's scratch."""
    v = _i32(0)
    _check(library().si_moe_router_noalloc_status(_stream(stream), ctypes.byref(v)),
           "si_moe_router_noalloc_status")
    return v.value


class Layer:
    """Device weights of one layer plus the ``si_moe_layer`` descriptor.

    ``t`` maps the generator's names (gate, up, down, sh_gate, sh_up, sh_down,
    w_sg, w_router, w_norm) to CUDA tensors; formats come from ``spec``.
    """

    def __init__(self, spec, t: dict):
        self.spec, self.t = spec, t
        s = SiMoeLayer()
        s.hidden, s.n_experts, s.top_k, s.inter = spec.hidden, spec.n_experts, spec.top_k, spec.inter
        s.expert_type = DTYPES[spec.expert_type]
        s.w_gate, s.w_up, s.w_down = (_cuda(t[k], k) for k in ("gate", "up", "down"))
        s.shared_inter = spec.shared_inter
        s.shared_type = DTYPES[spec.shared_type]
        if spec.shared_inter > 0:
            s.ws_gate, s.ws_up, s.ws_down, s.w_shared_sigmoid = (
                _cuda(t[k], k) for k in ("sh_gate", "sh_up", "sh_down", "w_sg"))
        if "w_router" in t:
            s.w_router = _cuda(t["w_router"], "w_router")
            s.router_type = _xtype(t["w_router"])
        if "w_norm" in t:
            s.w_norm = _cuda(t["w_norm"], "w_norm")
        s.eps = spec.eps
        s.down_type = DTYPES[spec.down_type] if getattr(spec, "down_type", "") else SI_F32
        self.c = s

    @property
    def ref(self):
        return ctypes.byref(self.c)


def ffn_workspace_bytes(layer: Layer, n_tokens: int = 1) -> int:
    return int(library().si_moe_ffn_workspace_bytes(layer.ref, n_tokens))


def si_moe_ffn_decode(layer: Layer, x: torch.Tensor, ids: torch.Tensor, w: torch.Tensor,
                      x_q8_1: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                      stream=None):
    """One token: x bf16 [H] -> (routed bf16 [H], shared bf16 [H] or None)."""
    H = layer.spec.hidden
    routed = torch.empty(H, dtype=torch.bfloat16, device=x.device)
    shared = torch.empty(H, dtype=torch.bfloat16, device=x.device) if layer.spec.shared_inter else None
    if ws is None:
        ws = workspace(ffn_workspace_bytes(layer), x.device)
    k = layer.spec.top_k
    _check(library().si_moe_ffn_decode(
        layer.ref, 1, _shaped(x, "x", H, _BF16),
        None if x_q8_1 is None else _shaped(x_q8_1, "x_q8_1", H // 32 * 36, _U8),
        _shaped(ids, "ids", k, _I32), _shaped(w, "w", k, _F32),
        _cuda(routed, "routed"), _opt(shared, "shared"), _cuda(ws, "ws"), ws.numel(),
        _stream(stream)), "si_moe_ffn_decode")
    return routed, shared


def si_moe_ffn_decode_ep(layer: Layer, e0: int, e1: int, x: torch.Tensor, ids: torch.Tensor,
                         ws: torch.Tensor | None = None, stream=None):
    """The slots of experts in [e0, e1) for one token: -> (slot_y fp32 [k, H]
    with zeros for the other slots, shared bf16 [H] or None)."""
    H, k = layer.spec.hidden, layer.spec.top_k
    slot_y = torch.empty(k, H, dtype=torch.float32, device=x.device)
    shared = torch.empty(H, dtype=torch.bfloat16, device=x.device) if layer.spec.shared_inter else None
    if ws is None:
        ws = workspace(ffn_workspace_bytes(layer), x.device)
    _check(library().si_moe_ffn_decode_ep(
        layer.ref, e0, e1, _shaped(x, "x", H, _BF16), None, _shaped(ids, "ids", k, _I32),
        _cuda(slot_y, "slot_y"), _opt(shared, "shared"), _cuda(ws, "ws"), ws.numel(), _stream(stream)),
        "si_moe_ffn_decode_ep")
    return slot_y, shared


def si_moe_combine_slots(slot_y: torch.Tensor, w: torch.Tensor, stream=None) -> torch.Tensor:
    """routed = bf16(sum_r w[r] * slot_y[r]) in rank order: slot_y fp32 [k, H], w fp32 [k]."""
    k, H = slot_y.shape
    routed = torch.empty(H, dtype=torch.bfloat16, device=slot_y.device)
    _check(library().si_moe_combine_slots(_shaped(slot_y, "slot_y", k * H, _F32), _shaped(w, "w", k, _F32),
                                          k, H, _cuda(routed, "routed"), _stream(stream)),
           "si_moe_combine_slots")
    return routed


SI_FFN_AUTO, SI_FFN_INT8, SI_FFN_TENSOR = 0, 1, 2


def ffn_batched_workspace_bytes(layer: Layer, n_tokens: int) -> int:
    return int(library().si_moe_ffn_batched_workspace_bytes(layer.ref, n_tokens))


def si_moe_ffn_batched(layer: Layer, x: torch.Tensor, ids: torch.Tensor, w: torch.Tensor,
                       mode: int = SI_FFN_AUTO, ws: torch.Tensor | None = None, stream=None):
    """T tokens with per-token routing: x bf16 [T, H], ids int32 [T, k], w fp32 [T, k]
    -> routed bf16 [T, H]."""
    T = x.shape[0]
    H, k = layer.spec.hidden, layer.spec.top_k
    routed = torch.empty(T, H, dtype=torch.bfloat16, device=x.device)
    if ws is None:
        ws = workspace(ffn_batched_workspace_bytes(layer, T), x.device)
    _check(library().si_moe_ffn_batched(
        layer.ref, T, mode, _shaped(x, "x", T * H, _BF16), _shaped(ids, "ids", T * k, _I32),
        _shaped(w, "w", T * k, _F32),
        _cuda(routed, "routed"), _cuda(ws, "ws"), ws.numel(), _stream(stream)),
        "si_moe_ffn_batched")
    return routed


def si_add_rmsnorm3(a, b, c, w_norm, eps: float = 1e-6, want_q8: bool = False, stream=None):
    """Rows [R, n] (or [n]) of bf16 -> (sum, norm, norm Q8_1 bytes | None)."""
    n = a.shape[-1]
    rows = a.numel() // n
    s = torch.empty_like(a)
    y = torch.empty_like(a)
    q8 = torch.empty(rows * (n // 32) * 36, dtype=torch.uint8, device=a.device) if want_q8 else None
    _check(library().si_add_rmsnorm3(_shaped(a, "a", rows * n, _BF16), _shaped(b, "b", rows * n, _BF16),
                                     None if c is None else _shaped(c, "c", rows * n, _BF16),
                                     _shaped(w_norm, "w_norm", n, _BF16), n, rows, eps, _cuda(s, "sum"),
                                     _cuda(y, "norm"), _opt(q8, "q8"), _stream(stream)),
           "si_add_rmsnorm3")
    return s, y, q8


def layer_workspace_bytes(layer: Layer) -> int:
    return int(library().si_moe_layer_workspace_bytes(layer.ref))


def si_moe_layer_decode(layer: Layer, x, residual=None, ws=None, stream=None) -> dict:
    H, k = layer.spec.hidden, layer.spec.top_k
    dev = x.device
    out = {n: torch.empty(H, dtype=torch.bfloat16, device=dev)
           for n in ("sum", "y", "routed", "shared")}
    out["ids"] = torch.empty(k, dtype=torch.int32, device=dev)
    out["w"] = torch.empty(k, dtype=torch.float32, device=dev)
    if ws is None:
        ws = workspace(layer_workspace_bytes(layer), dev)
    res = x if residual is None else residual
    _check(library().si_moe_layer_decode(
        layer.ref, _shaped(x, "x", H, _BF16), _shaped(res, "residual", H, _BF16),
        _cuda(out["sum"], "sum"),
        _cuda(out["y"], "y"), _cuda(out["ids"], "ids"), _cuda(out["w"], "w"),
        _cuda(out["routed"], "routed"), _cuda(out["shared"], "shared"), _cuda(ws, "ws"),
        ws.numel(), _stream(stream)), "si_moe_layer_decode")
    return out


SI_STACK_AUTO, SI_STACK_PER_LAYER, SI_STACK_PERSISTENT = 0, 1, 2


class StackGraph:
    """n_layers x n_tokens decode captured as one CUDA graph (buffers owned here).

    mode: SI_STACK_AUTO (the persistent kernel when it supports the layers),
    SI_STACK_PER_LAYER or SI_STACK_PERSISTENT."""

    def __init__(self, layers, x_in: torch.Tensor, want_ids: bool = True, stream=None,
                 mode: int = SI_STACK_AUTO):
        self.layers = list(layers)
        arr = (SiMoeLayer * len(self.layers))(*[l.c for l in self.layers])
        self._arr = arr
        T, H = x_in.shape
        if H != self.layers[0].spec.hidden or x_in.dtype != torch.bfloat16:
            raise ValueError(f"x_in must be bf16 [T, {self.layers[0].spec.hidden}], got "
                             f"{x_in.dtype} {tuple(x_in.shape)}")
        k = self.layers[0].spec.top_k
        dev = x_in.device
        self.x_in = x_in
        self.y = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        self.sum = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        self.ids = (torch.empty(T, len(self.layers), k, dtype=torch.int32, device=dev)
                    if want_ids else None)
        nb = int(library().si_moe_stack_workspace_bytes(arr, len(self.layers)))
        self.ws = workspace(nb, dev)
        h = _vp()
        cap = torch.cuda.Stream(device=dev)
        cap.wait_stream(torch.cuda.current_stream())
        _check(library().si_moe_stack_graph_create_mode(
            arr, len(self.layers), T, _cuda(x_in, "x_in"), _cuda(self.y, "y"),
            _cuda(self.sum, "sum"), _opt(self.ids, "ids"), _cuda(self.ws, "ws"), self.ws.numel(),
            mode, _stream(cap), ctypes.byref(h)), "si_moe_stack_graph_create_mode")
        self.handle = h
        self.stream = stream
        self.persistent = bool(library().si_graph_is_persistent(h))

    def launch(self, stream=None):
        _check(library().si_graph_launch(self.handle, _stream(stream)), "si_graph_launch")

    def close(self):
        if self.handle:
            library().si_graph_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def layer_batched_workspace_bytes(layer: Layer, n_tokens: int) -> int:
    return int(library().si_moe_layer_batched_workspace_bytes(layer.ref, n_tokens))


def si_moe_layer_decode_batched(layer: Layer, x: torch.Tensor, residual=None, mode: int = SI_FFN_AUTO,
                                ws=None, stream=None) -> dict:
    """T tokens through one layer, each routed on its own: x bf16 [T, H] ->
    {sum, y, routed: bf16 [T, H], ids: int32 [T, k], w: fp32 [T, k]}."""
    T, H = x.shape
    k = layer.spec.top_k
    dev = x.device
    out = {n: torch.empty(T, H, dtype=torch.bfloat16, device=dev) for n in ("sum", "y", "routed")}
    out["ids"] = torch.empty(T, k, dtype=torch.int32, device=dev)
    out["w"] = torch.empty(T, k, dtype=torch.float32, device=dev)
    if ws is None:
        ws = workspace(layer_batched_workspace_bytes(layer, T), dev)
    res = x if residual is None else residual
    _check(library().si_moe_layer_decode_batched(
        layer.ref, T, mode, _shaped(x, "x", T * H, _BF16), _shaped(res, "residual", T * H, _BF16),
        _cuda(out["sum"], "sum"), _cuda(out["y"], "y"), _cuda(out["ids"], "ids"), _cuda(out["w"], "w"),
        _cuda(out["routed"], "routed"), _cuda(ws, "ws"), ws.numel(), _stream(stream)),
        "si_moe_layer_decode_batched")
    return out


class BatchedStackGraph:
    """T tokens through n_layers layers together (per-token routing), captured
    as one CUDA graph; buffers owned here."""

    def __init__(self, layers, x_in: torch.Tensor, mode: int = SI_FFN_AUTO, want_ids: bool = True):
        self.layers = list(layers)
        arr = (SiMoeLayer * len(self.layers))(*[l.c for l in self.layers])
        self._arr = arr
        T, H = x_in.shape
        if H != self.layers[0].spec.hidden or x_in.dtype != torch.bfloat16:
            raise ValueError(f"x_in must be bf16 [T, {self.layers[0].spec.hidden}]")
        k = self.layers[0].spec.top_k
        dev = x_in.device
        self.x_in = x_in
        self.y = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        self.sum = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        self.ids = (torch.empty(len(self.layers), T, k, dtype=torch.int32, device=dev)
                    if want_ids else None)
        nb = int(library().si_moe_stack_batched_workspace_bytes(arr, len(self.layers), T))
        self.ws = workspace(nb, dev)
        h = _vp()
        cap = torch.cuda.Stream(device=dev)
        cap.wait_stream(torch.cuda.current_stream())
        _check(library().si_moe_stack_graph_create_batched(
            arr, len(self.layers), T, mode, _cuda(x_in, "x_in"), _cuda(self.y, "y"),
            _cuda(self.sum, "sum"), _opt(self.ids, "ids"), _cuda(self.ws, "ws"), self.ws.numel(),
            _stream(cap), ctypes.byref(h)), "si_moe_stack_graph_create_batched")
        self.handle = h
        # one token in the automatic mode: the persistent stack kernel when it takes the layers
        self.persistent = bool(library().si_graph_is_persistent(h))

    def launch(self, stream=None):
        _check(library().si_graph_launch(self.handle, _stream(stream)), "si_graph_launch")

    def close(self):
        if self.handle:
            library().si_graph_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def si_requant_q4_k(src: torch.Tensor, src_type: str, rows: int, cols: int,
                    out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Load-time requant: Q8_0 or Q5_K rows (uint8 [rows, row bytes]) -> Q4_K
    rows (uint8 [rows, cols / 256 * 144])."""
    if out is None:
        out = torch.empty(rows, cols // 256 * 144, dtype=torch.uint8, device=src.device)
    src_rb = int(library().si_row_bytes(DTYPES[src_type], cols))
    _check(library().si_requant_q4_k(_shaped(src, "src", rows * src_rb, _U8), DTYPES[src_type],
                                     rows, cols, _shaped(out, "out", rows * (cols // 256 * 144), _U8),
                                     _stream(stream)), "si_requant_q4_k")
    return out


# ----------------------------------------------------------------------------
# MXFP4 matrices and their products, tokens sorted by expert
# ----------------------------------------------------------------------------

_TYPES = {torch.float32: SI_F32, torch.float16: SI_F16, torch.bfloat16: SI_BF16}
_Tensor, _empty = torch.Tensor, torch.empty
_u8, _i32_t, _f32_t, _bf16_t = torch.uint8, torch.int32, torch.float32, torch.bfloat16

# A decode step makes these calls back to back, and the host time of one is longer
# than its kernels. So the usual case (the current stream of the current device)
# runs straight through; _elsewhere takes the others. A torch without CUDA has
# neither binding, and no tensor for which they are asked.
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _elsewhere(call, stream, first, *args, **kw):
    """``call`` with the device of ``first`` current and, if ``stream`` is given,
    on that stream: what the call allocates then belongs to the stream, so an
    output or a temporary workspace is not handed out again while the kernels
    run. Inputs are marked as used by it."""
    if not isinstance(first, _Tensor) or not first.is_cuda:
        raise ValueError("expected CUDA tensors")
    if stream is None:
        with torch.cuda.device(first.device):
            return call(first, *args, **kw)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=first.device)
    if stream.device != first.device:
        raise ValueError(f"tensors on {first.device}, stream on {stream.device}")
    for t in (first, *args, *kw.values()):
        if isinstance(t, _Tensor) and t.is_cuda:
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        return call(first, *args, **kw)


def _dual() -> bool:
    """Whether forward-mode differentiation is under way (one look at a number: the usual calls pay for no more)."""
    return getattr(_forward_ad, "_current_level", 0) >= 0


def _no_tangents(call: str, *tensors):
    """Refuses dual tensors: the gradients are reverse mode's, and a tangent would be lost without a word."""
    for t in tensors:
        if isinstance(t, _Tensor) and _forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError(f"{call} hands no forward-mode tangent on: its gradients are reverse mode's")


def _ptr(t, dev: int, numel: int, dtype, name: str) -> int:
    """Device pointer of ``t`` after checking its device, size, dtype and that it is contiguous."""
    if t.get_device() == dev and t.dtype is dtype and t.numel() == numel and t.is_contiguous():
        return t.data_ptr()
    _shaped(t, name, numel, (dtype,))
    raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")


def _too_many(T: int, k: int):
    """T * k has to be an int of the C ABI: ctypes would pass on the low 32 bits of a larger one."""
    raise ValueError(f"{T} tokens x {k} ranks, expected fewer than 2^31 pairs")


def _bad_type(t, name: str):
    raise ValueError(f"{name} has dtype {t.dtype}, expected float32, float16 or bfloat16")


def _scratch(nbytes: int, device) -> torch.Tensor:
    """A workspace for one call: only its status header has to be zero."""
    if nbytes <= 0:
        raise ValueError("workspace size query returned 0 (invalid shapes)")
    ws = _empty((int(nbytes),), dtype=_u8, device=device)
    ws[:256].zero_()
    return ws


def mxfp4_scale_shape(rows: int, cols: int) -> tuple:
    """Shape of the scale tiles of a [rows, cols] matrix: 128 rows x 4 blocks of 32 each."""
    return (-(-rows // 128), -(-cols // 128), 512)


def _scales(t, dev: int, n: int, rows: int, cols: int, many: bool, name: str) -> int:
    """Device pointer of the scale tiles of a matrix (or ``many``: n of them) after
    checking their shape; flat bytes are taken as tiles too. Scales that lie row by
    row can have the same number of bytes, so that alone does not do."""
    r, c = (rows + 127) // 128, (cols + 127) // 128
    if t.shape == ((n, r, c, 512) if many else (r, c, 512)) or t.dim() == 1:
        return _ptr(t, dev, n * r * c * 512, _u8, name)
    shape = (n, *mxfp4_scale_shape(rows, cols)) if many else mxfp4_scale_shape(rows, cols)
    raise ValueError(f"{name} have shape {tuple(t.shape)}, expected tiles {shape} or their bytes")


def _mxfp4(codes, scales, dev: int, name: str, dims: int):
    """(matrices, rows, cols, pointers) of an MXFP4 pair after checking that they belong together."""
    if not isinstance(codes, _Tensor) or codes.dim() != dims:
        raise ValueError(f"{name} codes must be uint8 [{'n, ' if dims == 3 else ''}rows, cols / 2]")
    if dims == 2:
        n, (rows, cols) = 1, codes.shape
    else:
        n, rows, cols = codes.shape
    cols *= 2
    if cols == 0 or cols % 32:
        raise ValueError(f"{name} has {cols} columns, expected a multiple of 32")
    return (n, rows, cols, _ptr(codes, dev, n * rows * cols // 2, _u8, name),
            _scales(scales, dev, n, rows, cols, dims == 3, f"{name} scales"))


def _strides(t: torch.Tensor, name: str):
    """(matrices, rows, cols, row stride, matrix stride) of a 2-D or 3-D tensor with contiguous columns."""
    if t.dim() == 2:
        n, (rows, cols), mat, (row, col) = 1, t.shape, 0, t.stride()
    elif t.dim() == 3:
        (n, rows, cols), (mat, row, col) = t.shape, t.stride()
    else:
        raise ValueError(f"{name} must be [rows, cols] or [n, rows, cols]")
    if col != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous columns")
    return n, rows, cols, row if rows > 1 else cols, mat if n > 1 else 0


def si_quantize_mxfp4(x: torch.Tensor, codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                      stream=None):
    """x [rows, cols] or [n, rows, cols] (fp32, fp16, bf16; rows and matrices at
    any stride without overlap) -> (codes uint8 [.., rows, cols / 2], scale tiles uint8
    [.., ceil(rows / 128), ceil(cols / 128), 512])."""
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(si_quantize_mxfp4, stream, x, codes, scales)
    n, rows, cols, row, mat = _strides(x, "x")
    if cols == 0 or cols % 32:
        raise ValueError(f"x has {cols} columns, expected a multiple of 32")
    tr, tc, many, d = (rows + 127) // 128, (cols + 127) // 128, x.dim() == 3, x.device
    if x.dtype not in _TYPES:
        _bad_type(x, "x")
    if codes is None:
        codes = _empty((n, rows, cols // 2) if many else (rows, cols // 2), dtype=_u8, device=d)
    else:
        _ptr(codes, dev, n * rows * cols // 2, _u8, "codes")
    if scales is None:
        scales = _empty((n, tr, tc, 512) if many else (tr, tc, 512), dtype=_u8, device=d)
    else:
        _scales(scales, dev, n, rows, cols, many, "scales")
    st = library().si_quantize_mxfp4(x.data_ptr(), _TYPES[x.dtype], n, rows, cols, row, mat, codes.data_ptr(),
                                     scales.data_ptr(), _raw_stream(dev))
    if st:
        _check(st, "si_quantize_mxfp4")
    return codes, scales


def si_dequantize_mxfp4(codes: torch.Tensor, scales: torch.Tensor, dtype=torch.bfloat16,
                        out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values of an MXFP4 matrix (or n of them) as ``dtype`` or into ``out``."""
    dev = codes.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(si_dequantize_mxfp4, stream, codes, scales, dtype, out)
    dims = 3 if codes.dim() == 3 else 2
    n, rows, cols, c, sc = _mxfp4(codes, scales, dev, "x", dims)
    shape = (n, rows, cols) if dims == 3 else (rows, cols)
    if out is None:
        out = _empty(shape, dtype=dtype, device=codes.device)
        row, mat = cols, rows * cols
    elif out.shape != shape or out.get_device() != dev:
        raise ValueError(f"out has shape {tuple(out.shape)} on {out.device}, expected {shape} on cuda:{dev}")
    else:
        _, _, _, row, mat = _strides(out, "out")
    if out.dtype not in _TYPES:
        _bad_type(out, "out")
    st = library().si_dequantize_mxfp4(c, sc, n, rows, cols, out.data_ptr(), _TYPES[out.dtype], row, mat,
                                       _raw_stream(dev))
    if st:
        _check(st, "si_dequantize_mxfp4")
    return out


def mxfp4_matmul_workspace_bytes(m: int, n: int, k: int) -> int:
    return int(library().si_mxfp4_matmul_workspace_bytes(m, n, k))


def si_mxfp4_matmul(a_codes: torch.Tensor, a_scales: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
                    dtype=torch.bfloat16, out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """a [m, k] and w [n, k] in MXFP4 -> a w^T [m, n] in ``dtype`` or into ``out``
    (any row stride); without rows (m or n 0) nothing is launched. ``ws`` receives the
    device status; without it a wait that ran out on the device, which leaves
    the result incomplete, is not reported."""
    dev = a_codes.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(si_mxfp4_matmul, stream, a_codes, a_scales, w_codes, w_scales, dtype, out, ws)
    _, m, k, ac, asc = _mxfp4(a_codes, a_scales, dev, "a", 2)
    _, n, k2, wc, wsc = _mxfp4(w_codes, w_scales, dev, "w", 2)
    if k != k2:
        raise ValueError(f"a has {k} columns, w has {k2}")
    if out is None:
        out, ld = _empty((m, n), dtype=dtype, device=a_codes.device), n
    elif out.shape != (m, n) or out.get_device() != dev:
        raise ValueError(f"out has shape {tuple(out.shape)} on {out.device}, expected {(m, n)} on cuda:{dev}")
    else:
        ld = _strides(out, "out")[3]
    if out.dtype not in _TYPES:
        _bad_type(out, "out")
    if m == 0 or n == 0:
        return out
    st = library().si_mxfp4_matmul(ac, asc, m, wc, wsc, n, k, out.data_ptr(), _TYPES[out.dtype], ld,
                                   None if ws is None else _ptr(ws, dev, ws.numel(), _u8, "ws"),
                                   0 if ws is None else ws.numel(), _raw_stream(dev))
    if st:
        _check(st, "si_mxfp4_matmul")
    return out


def si_moe_sort(ids: torch.Tensor, n_experts: int, stream=None):
    """ids int32 [T, k] -> (order int32 [T * k], position int32 [T, k], offsets
    int32 [n_experts + 1]); pairs whose id is outside [0, n_experts) are dropped
    (position -1)."""
    dev = ids.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(si_moe_sort, stream, ids, n_experts)
    (T, k), d, lib = ids.shape, ids.device, library()
    n = T * k
    if n >> 31:
        _too_many(T, k)
    if n_experts >> 31:
        raise ValueError(f"{n_experts} experts, expected 1..1024")
    order = _empty((n,), dtype=_i32_t, device=d)
    position = _empty((T, k), dtype=_i32_t, device=d)
    offsets = _empty((n_experts + 1 if n_experts > 0 else 1,), dtype=_i32_t, device=d)
    need = lib.si_moe_sort_workspace_bytes(T, k, n_experts)
    ws = _empty((need,), dtype=_u8, device=d) if need else None
    st = lib.si_moe_sort(_ptr(ids, dev, n, _i32_t, "ids"), T, k, n_experts, order.data_ptr(),
                         position.data_ptr(), offsets.data_ptr(), ws.data_ptr() if need else None, need,
                         _raw_stream(dev))
    if st:
        _check(st, "si_moe_sort")
    return order, position, offsets


def _kept(offsets: torch.Tensor, dev: int) -> int:
    """Address of the number of kept pairs, the last of the offsets."""
    n = offsets.numel()
    if offsets.dim() != 1 or n < 1:
        raise ValueError("offsets must be int32 [n_experts + 1]")
    return _ptr(offsets, dev, n, _i32_t, "offsets") + 4 * (n - 1)


def si_moe_gather(x: torch.Tensor, position: torch.Tensor, offsets: torch.Tensor, stream=None) -> torch.Tensor:
    """xs[position[t, r]] = x[t]: x [T, H] -> [T * k, H], zero rows behind the kept pairs.
    Differentiable in x (once)."""
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(si_moe_gather, stream, x, position, offsets)
    if _dual():
        _no_tangents("si_moe_gather", x)
    if x.requires_grad and torch.is_grad_enabled():
        return _Gather.apply(x, position, offsets)
    (T, H), k, dtype = x.shape, position.shape[-1], x.dtype
    n = T * k
    if n >> 31:
        _too_many(T, k)
    if dtype not in _TYPES:
        _bad_type(x, "x")
    xs = _empty((n, H), dtype=dtype, device=x.device)
    st = library().si_moe_gather(_ptr(x, dev, T * H, dtype, "x"), _TYPES[dtype], T, k, H,
                                 _ptr(position, dev, n, _i32_t, "position"), _kept(offsets, dev),
                                 xs.data_ptr(), _raw_stream(dev))
    if st:
        _check(st, "si_moe_gather")
    return xs


def si_moe_gather_backward(gxs: torch.Tensor, position: torch.Tensor, stream=None, dtype=None) -> torch.Tensor:
    """gx[t] = sum_r gxs[position[t, r]]: gxs [T * k, H] -> [T, H] in gxs' type, or fp32 rows in ``dtype``."""
    dev = gxs.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(si_moe_gather_backward, stream, gxs, position, None, dtype)
    if dtype is not None and dtype is not gxs.dtype:
        return _combine_f32(dev, gxs, position, None, dtype)
    (T, k), H, dtype = position.shape, gxs.shape[-1], gxs.dtype
    n = T * k
    if n >> 31:
        _too_many(T, k)
    if dtype not in _TYPES:
        _bad_type(gxs, "gxs")
    gx = _empty((T, H), dtype=dtype, device=gxs.device)
    st = library().si_moe_gather_backward(_ptr(gxs, dev, n * H, dtype, "gxs"), _TYPES[dtype], T, k, H,
                                          _ptr(position, dev, n, _i32_t, "position"), gx.data_ptr(),
                                          _raw_stream(dev))
    if st:
        _check(st, "si_moe_gather_backward")
    return gx


def si_moe_combine(ys: torch.Tensor, position: torch.Tensor, w: torch.Tensor, stream=None, dtype=None) -> torch.Tensor:
    """y[t] = sum_r w[t, r] ys[position[t, r]]: ys [T * k, H], w fp32 [T, k] -> [T, H] in ys'
    type, or fp32 rows in ``dtype``. Differentiable in ys and w (once)."""
    dev = ys.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(si_moe_combine, stream, ys, position, w, None, dtype)
    if _dual():
        _no_tangents("si_moe_combine", ys, w)
    if (ys.requires_grad or w.requires_grad) and torch.is_grad_enabled():
        return _Combine.apply(ys, position, w, dtype)
    if dtype is not None and dtype is not ys.dtype:
        return _combine_f32(dev, ys, position, w, dtype)
    (T, k), H, dtype = position.shape, ys.shape[-1], ys.dtype
    n = T * k
    if n >> 31:
        _too_many(T, k)
    if dtype not in _TYPES:
        _bad_type(ys, "ys")
    y = _empty((T, H), dtype=dtype, device=ys.device)
    st = library().si_moe_combine(_ptr(ys, dev, n * H, dtype, "ys"), _TYPES[dtype], T, k, H,
                                  _ptr(position, dev, n, _i32_t, "position"), _ptr(w, dev, n, _f32_t, "w"),
                                  y.data_ptr(), _raw_stream(dev))
    if st:
        _check(st, "si_moe_combine")
    return y


def _combine_f32(dev: int, ys, position, w, dtype):
    (T, k), H = position.shape, ys.shape[-1]
    n = T * k
    if n >> 31:
        _too_many(T, k)
    if dtype not in _TYPES:
        raise ValueError(f"dtype is {dtype}, expected float32, float16 or bfloat16")
    y = _empty((T, H), dtype=dtype, device=ys.device)
    st = library().si_moe_combine_f32(_ptr(ys, dev, n * H, _f32_t, "rows summed in another type"), T, k, H,
                                      _ptr(position, dev, n, _i32_t, "position"),
                                      None if w is None else _ptr(w, dev, n, _f32_t, "w"), y.data_ptr(), _TYPES[dtype],
                                      _raw_stream(dev))
    if st:
        _check(st, "si_moe_combine_f32")
    return y


def si_moe_combine_backward(gy: torch.Tensor, ys: torch.Tensor, position: torch.Tensor, offsets: torch.Tensor,
                            w: torch.Tensor, stream=None):
    """gy [T, H], ys [T * k, H] -> (gys [T * k, H], gw fp32 [T, k])."""
    dev = gy.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(si_moe_combine_backward, stream, gy, ys, position, offsets, w)
    return _combine_backward(dev, gy, ys, position, offsets, w)


def _combine_backward(dev: int, gy, ys, position, offsets, w, gys=None):
    (T, k), H, dtype, d = position.shape, gy.shape[-1], gy.dtype, gy.device
    n = T * k
    if n >> 31:
        _too_many(T, k)
    if dtype not in _TYPES:
        _bad_type(gy, "gy")
    if gys is None:
        gys = _empty((n, H), dtype=dtype, device=d)
    gw = _empty((T, k), dtype=_f32_t, device=d)
    st = library().si_moe_combine_backward(
        _ptr(gy, dev, T * H, dtype, "gy"), _ptr(ys, dev, n * H, dtype, "ys"), _TYPES[dtype], T, k, H,
        _ptr(position, dev, n, _i32_t, "position"), _kept(offsets, dev), _ptr(w, dev, n, _f32_t, "w"),
        gys.data_ptr(), gw.data_ptr(), _raw_stream(dev))
    if st:
        _check(st, "si_moe_combine_backward")
    return gys, gw


class _Gather(torch.autograd.Function):
    """si_moe_gather of an x that requires a gradient."""

    @staticmethod
    def forward(ctx, x, position, offsets):
        ctx.save_for_backward(position)
        return si_moe_gather(x, position, offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, gxs):
        position, = ctx.saved_tensors
        return si_moe_gather_backward(gxs.contiguous(), position), None, None


class _Combine(torch.autograd.Function):
    """si_moe_combine of rows or weights that require a gradient. Without the
    sort's offsets the places may have gaps, so the rows' gradient starts as zeros
    and the kernel, told that every row is kept, clears none."""

    @staticmethod
    def forward(ctx, ys, position, w, dtype):
        ctx.save_for_backward(ys, position, w)
        return si_moe_combine(ys, position, w, None, dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        ys, position, w = ctx.saved_tensors
        kept = torch.full((1,), position.numel(), dtype=_i32_t, device=ys.device)
        gys, gw = _combine_backward(ys.get_device(), gy.to(ys.dtype).contiguous(), ys, position, kept, w,
                                    torch.zeros_like(ys))
        return (gys if ctx.needs_input_grad[0] else None, None, gw.view(w.shape) if ctx.needs_input_grad[2] else None,
                None)


# ----------------------------------------------------------------------------
# Products of sorted rows in 16 bits, activations kept in 8, the experts' training
# ----------------------------------------------------------------------------

_HALVES = {torch.float16: SI_F16, torch.bfloat16: SI_BF16}
_i8 = torch.int8


def moe_matmul_workspace_bytes() -> int:
    return int(library().si_moe_matmul_workspace_bytes())


def _half(t, name: str) -> int:
    """Type code of a 16-bit tensor."""
    code = _HALVES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} has dtype {t.dtype}, expected bfloat16 or float16")
    return code


def _rows_of_gradient(gy, dtype):
    """A gradient that autograd hands on, as contiguous rows of ``dtype`` (an operand of the tensor cores)
    that start on 16-byte boundaries."""
    if gy.dtype is not dtype:
        gy = gy.to(dtype)
    gy = gy.contiguous()
    return gy.clone() if gy.data_ptr() & 15 else gy


def _same(t, like, name: str, dims: int):
    """Checks that ``t`` has the device, the type and ``dims`` dimensions beside ``like``."""
    if not isinstance(t, _Tensor) or t.dim() != dims:
        raise ValueError(f"{name} must be a tensor of {dims} dimensions")
    if t.get_device() != like.get_device() or t.dtype is not like.dtype:
        raise ValueError(f"{name} is {t.dtype} on {t.device}, expected {like.dtype} on {like.device}")


def _width(n: int, name: str, log: int = 20):
    if n < 8 or n % 8 or n > 1 << log:
        raise ValueError(f"{name} is {n} wide, expected a multiple of 8 up to 2^{log}")


def _rows(t, name: str):
    """(row stride, pointer) of rows whose values are contiguous and which start on 16-byte boundaries."""
    rows, cols = t.shape
    ld = t.stride(0) if rows > 1 else cols
    p = t.data_ptr()
    if (t.stride(1) != 1 and cols > 1) or ld < cols or (ld * t.element_size() | p) & 15:
        raise ValueError(f"{name} must have contiguous values in rows that start on 16-byte boundaries without overlap, "
                         f"got strides {t.stride()}")
    return ld, p


def _matrices(w, name: str):
    """(experts, rows, cols, row stride, matrix stride, by columns, pointer) of [E, n, k], or of a transposed view."""
    E, n, k = w.shape
    mat, row, col = w.stride()
    by = 0
    if col != 1 and row == 1:
        by, row = 1, col
    inner, outer = (n, k) if by else (k, n)
    if E == 1:
        mat = row * outer
    p = w.data_ptr()
    if (col != 1 and not by) or row < inner or mat < row * (outer - 1) + inner or (2 * row | 2 * mat | p) & 15:
        raise ValueError(f"{name} must be [E, n, k] with contiguous rows or columns that start on 16-byte boundaries "
                         f"without overlap, got strides {w.stride()}")
    return E, n, k, row, mat, by, p


def _offsets(offsets, dev: int, E: int) -> int:
    if offsets.dim() != 1:
        raise ValueError("offsets must be int32 [n_experts + 1]")
    return _ptr(offsets, dev, E + 1, _i32_t, "offsets")


def _status_word(ws, dev: int):
    return (None, 0) if ws is None else (_ptr(ws, dev, ws.numel(), _u8, "ws"), ws.numel())


def si_moe_matmul(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, dtype=None, out: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Sorted rows through their experts' matrices: x [R, k] and w [E, n, k] (bf16 or
    fp16; rows of x at any 16-byte aligned stride, matrices by rows or, as a
    transposed view, by columns), offsets int32 [E + 1] of ``si_moe_sort`` -> [R, n] in
    x's type, in ``dtype`` (that or fp32) or into ``out``; zero rows for rows of no expert.
    Differentiable in x and w (once), without ``out``: the gradient of the result enters the products
    as an operand and is rounded to x's type first, an fp32 result's too (in fp16 beyond 65504 to
    infinity, below 6e-8 to zero). ``ws`` (``moe_matmul_workspace_bytes``)
    receives the device status; without it a wait that ran out on the device, which
    leaves the result incomplete, is not reported."""
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(si_moe_matmul, stream, x, w, offsets, dtype, out, ws)
    if _dual():
        _no_tangents("si_moe_matmul", x, w)
    if (x.requires_grad or w.requires_grad) and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("out cannot be given where x or w requires a gradient")
        return _Matmul.apply(x, w, offsets, dtype, ws)
    return _matmul(dev, x, w, offsets, dtype, out, ws)


def _matmul(dev: int, x, w, offsets, dtype=None, out=None, ws=None, turned=False):
    """si_moe_matmul without a history; ``turned``: through w transposed."""
    t = _half(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [R, k]")
    _same(w, x, "w", 3)
    (R, k), (E, n, k2, ldw, mat, by, wp) = x.shape, _matrices(w, "w")
    if turned:
        n, k2, by = k2, n, 1 - by
    if k != k2:
        raise ValueError(f"x is {k} wide, w takes {k2}")
    _width(n, "out")
    _width(k, "x", 21)
    ldx, xp = _rows(x, "x")
    op = _offsets(offsets, dev, E)
    if out is None:
        out, ldo = _empty((R, n), dtype=dtype or x.dtype, device=x.device), n
        yp = out.data_ptr()
    else:
        if out.shape != (R, n) or out.get_device() != dev:
            raise ValueError(f"out has shape {tuple(out.shape)} on {out.device}, expected {(R, n)} on cuda:{dev}")
        ldo, yp = _rows(out, "out")
        if R and yp in (xp, wp):
            raise ValueError("out is x or w itself")
    if out.dtype is not x.dtype and out.dtype is not _f32_t:
        raise ValueError(f"the result is {out.dtype}, expected {x.dtype} or float32")
    st = library().si_moe_matmul(xp, t, R, ldx, wp, E, n, k, ldw, mat, by, op, yp, _TYPES[out.dtype], ldo,
                                 *_status_word(ws, dev), _raw_stream(dev))
    if st:
        _check(st, "si_moe_matmul")
    return out


def si_moe_matmul_grad_w(gy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, dtype=None,
                         ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The gradient of the matrices of ``si_moe_matmul``: gy [R, n] and x [R, k] -> gw [E, n, k],
    gw[e] the sum of gy[r] x[r]^T over expert e's rows, zeros without rows, in gy's type or fp32."""
    dev = gy.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(si_moe_matmul_grad_w, stream, gy, x, offsets, dtype, ws)
    return _grad_w(dev, gy, x, offsets, dtype, ws)


def _grad_w(dev: int, gy, x, offsets, dtype=None, ws=None):
    t = _half(gy, "gy")
    if gy.dim() != 2:
        raise ValueError("gy must be [R, n]")
    _same(x, gy, "x", 2)
    (R, n), (R2, k), E = gy.shape, x.shape, offsets.numel() - 1
    if R != R2:
        raise ValueError(f"gy has {R} rows, x has {R2}")
    if E < 1:
        raise ValueError("offsets must be int32 [n_experts + 1]")
    _width(n, "gy", 21)
    _width(k, "x")
    ldg, gp = _rows(gy, "gy")
    ldx, xp = _rows(x, "x")
    op = _offsets(offsets, dev, E)
    dtype = dtype or gy.dtype
    if dtype is not gy.dtype and dtype is not _f32_t:
        raise ValueError(f"the result is {dtype}, expected {gy.dtype} or float32")
    gw = _empty((E, n, k), dtype=dtype, device=gy.device)
    st = library().si_moe_matmul_grad_w(gp, ldg, xp, ldx, t, R, E, n, k, op, gw.data_ptr(), _TYPES[dtype],
                                        *_status_word(ws, dev), _raw_stream(dev))
    if st:
        _check(st, "si_moe_matmul_grad_w")
    return gw


def si_moe_matmul_backward(gy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                           ws: torch.Tensor | None = None, stream=None):
    """gy [R, n], and x [R, k], w [E, n, k] of the product -> (gx [R, k], gw [E, n, k])."""
    dev = gy.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(si_moe_matmul_backward, stream, gy, x, w, offsets, ws)
    gw = _grad_w(dev, gy, x, offsets, None, ws)
    if w.shape != gw.shape:
        raise ValueError(f"w has shape {tuple(w.shape)}, expected {tuple(gw.shape)}")
    return _matmul(dev, gy, w, offsets, None, None, ws, True), gw


class _Matmul(torch.autograd.Function):
    """si_moe_matmul of an x or a w that requires a gradient."""

    @staticmethod
    def forward(ctx, x, w, offsets, dtype, ws):
        if x.dim() == 2:
            _width(x.shape[1], "x, whose width is that of its gradient,")
        ctx.save_for_backward(x, w, offsets)
        ctx.ws = ws
        return si_moe_matmul(x, w, offsets, dtype, None, ws)

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        x, w, offsets = ctx.saved_tensors
        gy, dev, need = _rows_of_gradient(gy, x.dtype), x.get_device(), ctx.needs_input_grad
        gx = _matmul(dev, gy, w, offsets, None, None, ctx.ws, True) if need[0] else None
        gw = _grad_w(dev, gy, x, offsets, None, ctx.ws) if need[1] else None
        return gx, gw, None, None, None


def mxint8_scale_shape(rows: int, cols: int) -> tuple:
    """Shape of the scales of [rows, cols] values: one for 32 of a row."""
    return (rows, -(-cols // 32))


def _act_rows(t, name: str):
    """Row stride of [rows, cols] with contiguous values, rows without overlap."""
    rows, cols = t.shape
    ld = t.stride(0) if rows > 1 else cols
    if (t.stride(1) != 1 and cols > 1) or ld < cols:
        raise ValueError(f"{name} must have contiguous values in rows without overlap, got strides {t.stride()}")
    return ld


def si_quantize_mxint8(x: torch.Tensor, stream=None):
    """x [rows, cols] (fp32, fp16, bf16; rows at any stride without overlap) in 8 bits ->
    (codes int8 [rows, cols], scales uint8 [rows, ceil(cols / 32)])."""
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(si_quantize_mxint8, stream, x)
    if x.dim() != 2 or x.shape[1] == 0:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected [rows, cols]")
    if x.dtype not in _TYPES:
        _bad_type(x, "x")
    (rows, cols), d = x.shape, x.device
    ld = _act_rows(x, "x")
    codes = _empty((rows, cols), dtype=_i8, device=d)
    scales = _empty((rows, (cols + 31) // 32), dtype=_u8, device=d)
    st = library().si_quantize_mxint8(x.data_ptr(), _TYPES[x.dtype], rows, cols, ld, codes.data_ptr(),
                                      scales.data_ptr(), _raw_stream(dev))
    if st:
        _check(st, "si_quantize_mxint8")
    return codes, scales


def si_dequantize_mxint8(codes: torch.Tensor, scales: torch.Tensor, dtype=torch.bfloat16,
                         out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values of ``si_quantize_mxint8``'s codes as ``dtype`` or into ``out``."""
    dev = codes.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(si_dequantize_mxint8, stream, codes, scales, dtype, out)
    if codes.dim() != 2 or codes.shape[1] == 0:
        raise ValueError(f"codes have shape {tuple(codes.shape)}, expected [rows, cols]")
    rows, cols = codes.shape
    c = _ptr(codes, dev, rows * cols, _i8, "codes")
    if scales.shape != (rows, (cols + 31) // 32):
        raise ValueError(f"scales have shape {tuple(scales.shape)}, expected {mxint8_scale_shape(rows, cols)}")
    s = _ptr(scales, dev, scales.numel(), _u8, "scales")
    if out is None:
        out, ld = _empty((rows, cols), dtype=dtype, device=codes.device), cols
    elif out.shape != (rows, cols) or out.get_device() != dev:
        raise ValueError(f"out has shape {tuple(out.shape)} on {out.device}, expected {(rows, cols)} on cuda:{dev}")
    else:
        ld = _act_rows(out, "out")
    if out.dtype not in _TYPES:
        _bad_type(out, "out")
    st = library().si_dequantize_mxint8(c, s, rows, cols, out.data_ptr(), _TYPES[out.dtype], ld, _raw_stream(dev))
    if st:
        _check(st, "si_dequantize_mxint8")
    return out


def _kept_empty(rows: int, inter: int, device):
    """Room for g and u of ``rows`` rows in 8 bits, each with blocks of its own."""
    return (_empty((rows, 2 * inter), dtype=_i8, device=device),
            _empty((rows, 2 * ((inter + 31) // 32)), dtype=_u8, device=device))


def si_swiglu(gu: torch.Tensor, keep: bool = False, stream=None):
    """h = silu(g) * u: gu [R, 2 I] (g, then u; fp32, fp16, bf16, rows at any stride) -> h [R, I];
    with ``keep`` (h, kept), kept = (codes int8 [R, 2 I], scales uint8 [R, 2 ceil(I / 32)]) for
    ``si_swiglu_backward``. Differentiable (once): the history holds g and u in 8 bits."""
    dev = gu.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(si_swiglu, stream, gu, keep)
    if gu.dim() != 2 or gu.shape[1] == 0 or gu.shape[1] % 2:
        raise ValueError(f"gu has shape {tuple(gu.shape)}, expected [R, 2 I]")
    if gu.dtype not in _TYPES:
        _bad_type(gu, "gu")
    if _dual():
        _no_tangents("si_swiglu", gu)
    if gu.requires_grad and torch.is_grad_enabled():
        h, codes, scales = _Swiglu.apply(gu)
        return (h, (codes, scales)) if keep else h
    rows, inter, d = gu.shape[0], gu.shape[1] // 2, gu.device
    ld = _act_rows(gu, "gu")
    h = _empty((rows, inter), dtype=gu.dtype, device=d)
    kept = _kept_empty(rows, inter, d) if keep else None
    cp, sp = (kept[0].data_ptr(), kept[1].data_ptr()) if keep else (None, None)
    st = library().si_swiglu(gu.data_ptr(), _TYPES[gu.dtype], rows, inter, ld, h.data_ptr(), cp, sp, _raw_stream(dev))
    if st:
        _check(st, "si_swiglu")
    return (h, kept) if keep else h


def si_swiglu_backward(gh: torch.Tensor, kept, w: torch.Tensor | None = None, order: torch.Tensor | None = None,
                       stream=None):
    """The gradients of h = silu(g) u, from the kept g and u, in rows that enter a sum as
    w * h: gh [R, I] -> (ggu [R, 2 I], wh [R, I], gw). Without ``w`` every weight is 1 and gw
    None; w fp32 of R values is row r's, or with ``order`` int32 [R] (``si_moe_sort``'s, w the
    [T, k] weights) w[order[r]]. gw has w's shape; rows of no pair (order -1) give zero rows, pairs
    without a row gw 0."""
    return _swiglu_backward(gh, kept, w, order, True, stream)


def _swiglu_backward(gh, kept, w, order, want_wh, stream=None):
    codes, scales = kept
    dev = gh.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(lambda gh, c, s, w, o: _swiglu_backward(gh, (c, s), w, o, want_wh), stream, gh, codes, scales,
                          w, order)
    if gh.dim() != 2 or gh.shape[1] == 0:
        raise ValueError(f"gh has shape {tuple(gh.shape)}, expected [R, I]")
    (R, I), d, dtype = gh.shape, gh.device, gh.dtype
    if dtype not in _TYPES:
        _bad_type(gh, "gh")
    if codes.shape != (R, 2 * I) or scales.shape != (R, 2 * ((I + 31) // 32)):
        raise ValueError(f"kept codes and scales have shapes {tuple(codes.shape)} and {tuple(scales.shape)}, expected "
                         f"{(R, 2 * I)} and {(R, 2 * ((I + 31) // 32))}")
    if order is not None and w is None:
        raise ValueError("order needs w")
    gp, cp = _ptr(gh, dev, R * I, dtype, "gh"), _ptr(codes, dev, 2 * R * I, _i8, "codes")
    sp = _ptr(scales, dev, scales.numel(), _u8, "scales")
    wp = None if w is None else _ptr(w, dev, R, _f32_t, "w")
    op = None if order is None else _ptr(order, dev, R, _i32_t, "order")
    ggu = _empty((R, 2 * I), dtype=dtype, device=d)
    wh = _empty((R, I), dtype=dtype, device=d) if want_wh else None
    gw = None if w is None else _empty(w.shape, dtype=_f32_t, device=d)
    st = library().si_swiglu_backward(gp, _TYPES[dtype], R, I, cp, sp, wp, op, ggu.data_ptr(),
                                      wh.data_ptr() if want_wh else None, None if gw is None else gw.data_ptr(),
                                      _raw_stream(dev))
    if st:
        _check(st, "si_swiglu_backward")
    return ggu, wh, gw


class _Swiglu(torch.autograd.Function):
    """si_swiglu of a gu that requires a gradient."""

    @staticmethod
    def forward(ctx, gu):
        h, kept = si_swiglu(gu, True)
        ctx.save_for_backward(*kept)
        ctx.mark_non_differentiable(*kept)
        return h, *kept

    @staticmethod
    @once_differentiable
    def backward(ctx, gh, *_):
        return _swiglu_backward(gh.contiguous(), ctx.saved_tensors, None, None, False)[0]


def si_moe_gateup(x: torch.Tensor, gate_up: torch.Tensor, offsets: torch.Tensor, keep: bool = False,
                  ws: torch.Tensor | None = None, stream=None):
    """si_swiglu of si_moe_matmul's fp32 sums in one launch: sorted rows x [R, H] and gate_up
    [E, 2 I, H] contiguous (bf16 or fp16) -> h [R, I], with ``keep`` (h, kept) as ``si_swiglu``.
    Differentiable in x and gate_up (once): the history holds both, and g and u in 8 bits."""
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(si_moe_gateup, stream, x, gate_up, offsets, keep, ws)
    if _dual():
        _no_tangents("si_moe_gateup", x, gate_up)
    if (x.requires_grad or gate_up.requires_grad) and torch.is_grad_enabled():
        h, codes, scales = _Gateup.apply(x, gate_up, offsets, ws)
        return (h, (codes, scales)) if keep else h
    return _gateup(dev, x, gate_up, offsets, keep, ws)


def _gateup(dev: int, x, gate_up, offsets, keep, ws):
    """si_moe_gateup without a history."""
    t = _half(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [R, H]")
    _same(gate_up, x, "gate_up", 3)
    (R, H), (E, rows, cols), d = x.shape, gate_up.shape, x.device
    if cols != H or rows % 2:
        raise ValueError(f"gate_up has shape {tuple(gate_up.shape)}, expected [E, 2 I, {H}]")
    I = rows // 2
    _width(I, "h")
    _width(H, "x")
    ldx, xp = _rows(x, "x")
    wp, op = _ptr(gate_up, dev, E * rows * H, x.dtype, "gate_up"), _offsets(offsets, dev, E)
    h = _empty((R, I), dtype=x.dtype, device=d)
    kept = _kept_empty(R, I, d) if keep else None
    cp, sp = (kept[0].data_ptr(), kept[1].data_ptr()) if keep else (None, None)
    st = library().si_moe_gateup(xp, t, R, ldx, wp, E, I, H, op, h.data_ptr(), cp, sp, *_status_word(ws, dev),
                                 _raw_stream(dev))
    if st:
        _check(st, "si_moe_gateup")
    return (h, kept) if keep else h


class _Gateup(torch.autograd.Function):
    """si_moe_gateup of an x or a gate_up that requires a gradient."""

    @staticmethod
    def forward(ctx, x, gate_up, offsets, ws):
        h, kept = _gateup(x.get_device(), x, gate_up, offsets, True, ws)
        ctx.save_for_backward(x, gate_up, offsets, *kept)
        ctx.mark_non_differentiable(*kept)
        ctx.ws = ws
        return h, *kept

    @staticmethod
    @once_differentiable
    def backward(ctx, gh, *_):
        x, gate_up, offsets, codes, scales = ctx.saved_tensors
        dev, need = x.get_device(), ctx.needs_input_grad
        ggu = _swiglu_backward(gh.contiguous(), (codes, scales), None, None, False)[0]
        gx = _matmul(dev, ggu, gate_up, offsets, None, None, ctx.ws, True) if need[0] else None
        ggate_up = _grad_w(dev, ggu, x, offsets, None, ctx.ws) if need[1] else None
        return gx, ggate_up, None, None


def moe_down_backward_workspace_bytes(rows: int, n_experts: int, inter: int) -> int:
    return int(library().si_moe_down_backward_workspace_bytes(rows, n_experts, inter))


def si_moe_down_backward(gy: torch.Tensor, down: torch.Tensor, kept, offsets: torch.Tensor,
                         w: torch.Tensor | None = None, order: torch.Tensor | None = None,
                         ws: torch.Tensor | None = None, stream=None):
    """``si_swiglu_backward`` of gh = si_moe_matmul(gy, down^T) in one launch, gh in fp32 and not
    written: sorted rows gy [R, H], down [E, H, I] contiguous (bf16 or fp16), kept of
    ``si_moe_gateup`` -> (ggu [R, 2 I], wh [R, I], gw). ``ws``, if given, has at least
    ``moe_down_backward_workspace_bytes(R, E, I)`` bytes with w."""
    return _down_backward(gy, down, kept, offsets, w, order, ws, True, True, stream)


def _down_backward(gy, down, kept, offsets, w, order, ws, want_wh, want_gw, stream=None):
    codes, scales = kept
    dev = gy.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(lambda gy, down, c, s, *a: _down_backward(gy, down, (c, s), *a, want_wh, want_gw), stream, gy,
                          down, codes, scales, offsets, w, order, ws)
    t = _half(gy, "gy")
    if gy.dim() != 2:
        raise ValueError("gy must be [R, H]")
    _same(down, gy, "down", 3)
    (R, H), (E, H2, I), d = gy.shape, down.shape, gy.device
    if H != H2:
        raise ValueError(f"gy is {H} wide, down has {H2} rows")
    _width(I, "wh")
    _width(H, "gy")
    if codes.shape != (R, 2 * I) or scales.shape != (R, 2 * ((I + 31) // 32)):
        raise ValueError(f"kept codes and scales have shapes {tuple(codes.shape)} and {tuple(scales.shape)}, expected "
                         f"{(R, 2 * I)} and {(R, 2 * ((I + 31) // 32))}")
    if order is not None and w is None:
        raise ValueError("order needs w")
    ldg, gp = _rows(gy, "gy")
    dp, op = _ptr(down, dev, E * H * I, gy.dtype, "down"), _offsets(offsets, dev, E)
    cp, sp = _ptr(codes, dev, 2 * R * I, _i8, "codes"), _ptr(scales, dev, scales.numel(), _u8, "scales")
    wp = None if w is None else _ptr(w, dev, R, _f32_t, "w")
    rp = None if order is None else _ptr(order, dev, R, _i32_t, "order")
    ggu = _empty((R, 2 * I), dtype=gy.dtype, device=d)
    wh = _empty((R, I), dtype=gy.dtype, device=d) if want_wh else None
    gw = None
    if w is not None and want_gw:
        gw = _empty(w.shape, dtype=_f32_t, device=d)
        if ws is None and R:                     # for the partial sums alone: nobody reads its status word
            ws = _empty((moe_down_backward_workspace_bytes(R, E, I),), dtype=_u8, device=d)
    st = library().si_moe_down_backward(gp, t, R, ldg, dp, E, H, I, op, cp, sp, wp, rp, ggu.data_ptr(),
                                        wh.data_ptr() if want_wh else None, None if gw is None else gw.data_ptr(),
                                        *_status_word(ws, dev), _raw_stream(dev))
    if st:
        _check(st, "si_moe_down_backward")
    return ggu, wh, gw


def _experts_of(gate_up, down=None):
    """The ``si_experts`` of gate_up [E, 2 I, H] and down (without it the sizes alone)."""
    E, rows, H = gate_up.shape
    return SiExperts(_half(gate_up, "gate_up"), H, rows // 2, E, None if down is None else gate_up.data_ptr(),
                     None if down is None else down.data_ptr())


def moe_experts_workspace_bytes(n_tokens: int, top_k: int, gate_up: torch.Tensor) -> int:
    """Of ``si_moe_experts`` and its gradients."""
    if n_tokens * top_k >> 31:
        return 0
    return int(library().si_moe_experts_workspace_bytes(_experts_of(gate_up), n_tokens, top_k))


def si_moe_experts(x: torch.Tensor, ids: torch.Tensor, w: torch.Tensor, gate_up: torch.Tensor, down: torch.Tensor,
                   ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The routed experts in 16 bits, differentiable: x [T, H], ids int32 [T, k], w fp32 [T, k],
    gate_up [E, 2 I, H] (gate rows first) and down [E, H, I] contiguous, bf16 or fp16 as x -> [T, H]:
    y[t] = sum_r w[t, r] down[e] (silu(g) u), (g, u) = gate_up[e] x[t], e = ids[t, r]; ids outside
    [0, E) are dropped; without tokens nothing is launched, and the matrices' gradients are
    zeros. The gradients (once) reach x, w, gate_up and down; their history
    holds x and, of the experts' rows, g and u in 8 bits alone. ``ws`` is kept by the caller
    (``moe_experts_workspace_bytes``) and receives the device status; without it each call takes
    one of its own, and a wait that ran out on the device, which leaves the results incomplete,
    is not reported."""
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        return _elsewhere(si_moe_experts, stream, x, ids, w, gate_up, down, ws)
    if x.dim() != 2 or ids.dim() != 2 or ids.shape[0] != x.shape[0]:
        raise ValueError(f"x has shape {tuple(x.shape)}, ids {tuple(ids.shape)}, expected [T, H] and [T, k]")
    if _dual():
        _no_tangents("si_moe_experts", x, w, gate_up, down)
    if torch.is_grad_enabled() and (x.requires_grad or w.requires_grad or gate_up.requires_grad or down.requires_grad):
        return _Experts.apply(x, ids, w, gate_up, down, ws)
    return _experts_forward(dev, x, ids, w, gate_up, down, ws, False)[0]


def _experts_forward(dev: int, x, ids, w, gate_up, down, ws, keep: bool):
    _half(x, "x")
    _same(gate_up, x, "gate_up", 3)
    (T, H), k, (E, rows, cols), d, lib = x.shape, ids.shape[1], gate_up.shape, x.device, library()
    n, I = T * k, rows // 2
    if cols != H or rows % 2 or down.shape != (E, H, I):
        raise ValueError(f"gate_up has shape {tuple(gate_up.shape)} and down {tuple(down.shape)}, expected [E, 2 I, {H}] "
                         f"and [E, {H}, I]")
    _width(H, "x")
    _width(I, "down")
    if n >> 31:
        _too_many(T, k)
    if w.shape != ids.shape:
        raise ValueError(f"w has shape {tuple(w.shape)}, expected {tuple(ids.shape)}")
    _ptr(gate_up, dev, E * rows * H, x.dtype, "gate_up"), _ptr(down, dev, E * H * I, x.dtype, "down")
    L = _experts_of(gate_up, down)
    y, kept = _empty((T, H), dtype=x.dtype, device=d), None
    if T == 0 and lib.si_moe_experts_kept_bytes(L, 1, k):   # sizes that a token could have
        _ptr(x, dev, 0, x.dtype, "x"), _ptr(ids, dev, 0, _i32_t, "ids"), _ptr(w, dev, 0, _f32_t, "w")
        return y, None
    if keep:
        kept = _empty((lib.si_moe_experts_kept_bytes(L, T, k),), dtype=_u8, device=d)
    if ws is None:                               # nobody reads its status word
        ws = _empty((lib.si_moe_experts_workspace_bytes(L, T, k),), dtype=_u8, device=d)
    m = ws.numel()
    st = lib.si_moe_experts(L, T, k, _ptr(x, dev, T * H, x.dtype, "x"), _ptr(ids, dev, n, _i32_t, "ids"),
                            _ptr(w, dev, n, _f32_t, "w"), y.data_ptr(), kept.data_ptr() if keep else None,
                            _ptr(ws, dev, m, _u8, "ws"), m, _raw_stream(dev))
    if st:
        _check(st, "si_moe_experts")
    return y, kept


class _Experts(torch.autograd.Function):
    """si_moe_experts with a gradient. gh = down^T gy stays in the registers of the launch
    that forms it, and x's gradient in fp32 rows until the ranks are summed: so every
    gradient is rounded once as an operand of a product and once as a result."""

    @staticmethod
    def forward(ctx, x, ids, w, gate_up, down, ws):
        y, kept = _experts_forward(x.get_device(), x, ids, w, gate_up, down, ws, True)
        ctx.save_for_backward(x, w, gate_up, down, kept)
        ctx.ws, ctx.k = ws, ids.shape[1]
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        x, w, gate_up, down, kept = ctx.saved_tensors
        ws, k, need, lib, dev = ctx.ws, ctx.k, ctx.needs_input_grad, library(), x.get_device()
        T, H = x.shape
        if T == 0:
            return tuple(torch.zeros_like(t) if need[i] else None
                         for i, t in enumerate((x, None, w, gate_up, down, None)))
        L, gy = _experts_of(gate_up, down), _rows_of_gradient(gy, x.dtype)
        gx, gw, ggate_up, gdown = (_empty(t.shape, dtype=t.dtype, device=t.device) if need[i] else None
                                   for i, t in ((0, x), (2, w), (3, gate_up), (4, down)))
        if ws is None:
            ws = _empty((lib.si_moe_experts_workspace_bytes(L, T, k),), dtype=_u8, device=x.device)
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        m = ws.numel()
        st = lib.si_moe_experts_backward(L, T, k, _ptr(gy, dev, T * H, x.dtype, "gy"), x.data_ptr(), w.data_ptr(),
                                         kept.data_ptr(), p(gx), p(gw), p(ggate_up), p(gdown),
                                         _ptr(ws, dev, m, _u8, "ws"), m, _raw_stream(dev))
        if st:
            _check(st, "si_moe_experts_backward")
        return gx, None, gw, ggate_up, gdown, None


class Mxfp4Experts:
    """The routed experts of one layer in MXFP4 plus the ``si_mxfp4_experts``
    descriptor. ``gate``, ``up`` [E, I, H] and ``down`` [E, H, I] are (codes,
    scales) as ``si_quantize_mxfp4`` returns them: the scales in tiles
    (``mxfp4_scale_shape``), not row by row as checkpoints hold them."""

    def __init__(self, gate, up, down):
        self.gate, self.up, self.down = gate, up, down
        if not isinstance(gate[0], _Tensor) or not gate[0].is_cuda:
            raise ValueError("gate must be CUDA tensors")
        self.dev = gate[0].get_device()
        E, I, H, gc, gs = _mxfp4(*gate, self.dev, "gate", 3)
        n, rows, cols, uc, us = _mxfp4(*up, self.dev, "up", 3)
        if (n, rows, cols) != (E, I, H):
            raise ValueError(f"up must be {E} matrices [{I}, {H}], as gate")
        n, rows, cols, dc, ds = _mxfp4(*down, self.dev, "down", 3)
        if (n, rows, cols) != (E, H, I):
            raise ValueError(f"down must be {E} matrices [{H}, {I}]")
        if (H | I | E) >> 31:
            raise ValueError(f"{E} experts of width {H} x {I}, expected at most 1024 of 65536 x 65536")
        self.hidden, self.inter, self.n_experts = H, I, E
        self.c = SiMxfp4Experts(H, I, E, gc, gs, uc, us, dc, ds)
        self.ref = ctypes.byref(self.c)

    @classmethod
    def quantize(cls, gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor, stream=None):
        """From weights gate, up [E, I, H] and down [E, H, I] in fp32, fp16 or bf16."""
        return cls(*(si_quantize_mxfp4(t, stream=stream) for t in (gate, up, down)))


def ffn_mxfp4_workspace_bytes(experts: Mxfp4Experts, n_tokens: int, top_k: int) -> int:
    if (n_tokens | top_k) >> 31:
        return 0
    return int(library().si_moe_ffn_mxfp4_workspace_bytes(experts.ref, n_tokens, top_k))


def si_moe_ffn_mxfp4(experts: Mxfp4Experts, x: torch.Tensor, ids: torch.Tensor, w: torch.Tensor,
                     ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """T tokens with per-token routing: x bf16 [T, H], ids int32 [T, k], w fp32
    [T, k] -> routed bf16 [T, H]. ``ws`` is kept by the caller and receives the
    device status (``si_workspace_status``); without it each call takes one of its
    own, and a wait that ran out on the device, which leaves the result
    incomplete, is not reported."""
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _current_device():
        weights = (*experts.gate, *experts.up, *experts.down)
        return _elsewhere(lambda x, ids, w, ws, *_: si_moe_ffn_mxfp4(experts, x, ids, w, ws), stream, x, ids, w, ws,
                          *weights)
    (T, k), H = ids.shape, experts.hidden
    pairs = T * k
    if pairs >> 31:
        _too_many(T, k)
    if experts.dev != dev:
        raise ValueError(f"tensors on cuda:{dev}, experts on cuda:{experts.dev}")
    if ws is None:
        ws = _scratch(ffn_mxfp4_workspace_bytes(experts, T, k), x.device)
    routed = _empty((T, H), dtype=_bf16_t, device=x.device)
    n = ws.numel()
    st = library().si_moe_ffn_mxfp4(
        experts.ref, T, k, _ptr(x, dev, T * H, _bf16_t, "x"), _ptr(ids, dev, pairs, _i32_t, "ids"),
        _ptr(w, dev, pairs, _f32_t, "w"), routed.data_ptr(), _ptr(ws, dev, n, _u8, "ws"), n, _raw_stream(dev))
    if st:
        _check(st, "si_moe_ffn_mxfp4")
    return routed


def si_workspace_status(ws: torch.Tensor, stream=None) -> int:
    v = _i32(0)
    _check(library().si_workspace_status(_cuda(ws, "ws"), _stream(stream), ctypes.byref(v)),
           "si_workspace_status")
    return v.value


def si_test_q4k_block_dots(w: torch.Tensor, rows: int, k: int, a_q8_1: torch.Tensor, stream=None):
    out = torch.empty(rows, k // 32, dtype=torch.int32, device=w.device)
    _check(library().si_test_q4k_block_dots(_shaped(w, "w", rows * (k // 256 * 144), _U8), rows, k,
                                            _shaped(a_q8_1, "a", k // 32 * 36, _U8),
                                            _cuda(out, "out"), _stream(stream)),
           "si_test_q4k_block_dots")
    return out


SI_TEST_DOTS_Q4K_SB, SI_TEST_DOTS_Q4K_HALF, SI_TEST_DOTS_Q5K_HALF = 0, 1, 2
SI_TEST_DOTS_Q4K_SB_TOKENS, SI_TEST_DOTS_Q4K_HALF_TOKENS = 3, 4


def si_test_block_dots(kind: int, w: torch.Tensor, rows: int, k: int, a_q8_1: torch.Tensor,
                       n_vec: int = 1, stream=None):
    """Exact int32 block sums of the library's integer dot helper `kind` ->
    int32 [n_vec, rows, k / 32]."""
    sbb = 176 if kind == SI_TEST_DOTS_Q5K_HALF else 144
    out = torch.empty(n_vec, rows, k // 32, dtype=torch.int32, device=w.device)
    _check(library().si_test_block_dots(kind, _shaped(w, "w", rows * (k // 256 * sbb), _U8), rows, k,
                                        _shaped(a_q8_1, "a", n_vec * (k // 32 * 36), _U8), n_vec,
                                        _cuda(out, "out"), _stream(stream)),
           "si_test_block_dots")
    return out


def si_test_unfused_add_rmsnorm(a, b, c, w_norm, eps: float = 1e-6, stream=None):
    n = a.shape[-1]
    rows = a.numel() // n
    t, s, y = torch.empty_like(a), torch.empty_like(a), torch.empty_like(a)
    _check(library().si_test_unfused_add_rmsnorm(
        _cuda(a, "a"), _cuda(b, "b"), _cuda(c, "c"), _cuda(w_norm, "w_norm"), n, rows, eps,
        _cuda(t, "t"), _cuda(s, "sum"), _cuda(y, "norm"), _stream(stream)),
        "si_test_unfused_add_rmsnorm")
    return s, y


def device_layer(spec, seed: int, layer: int = 0, device="cuda") -> Layer:
    """Generate one layer's synthetic weights on the device and wrap them."""
    import gen
    L = gen.make_layer(spec, seed, layer, device=device)
    t = {k: v for k, v in L.items() if isinstance(v, torch.Tensor)}
    return Layer(spec, t)
