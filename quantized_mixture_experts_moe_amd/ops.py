"""Thin ctypes binding of libqmoe.so (include/qmoe.h), same call names.

This module only marshals arguments: torch tensors supply device memory and
the current HIP stream; every step of the layer runs in the library's HIP
kernels.  Loading fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from .shapes import SCHEME_CODE

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqmoe.so")

QMOE_OK, QMOE_ERR_INVALID_ARG, QMOE_ERR_UNSUPPORTED, QMOE_ERR_HIP = 0, 1, 2, 3
QMOE_DT_BF16, QMOE_DT_F32 = 0, 1
QMOE_FLAG_DUMP_ACC = 1
QMOE_FLAG_PREPACKED = 2
# QMOE_ABI_VERSION of the include/qmoe.h this binding follows; loading a
# library that reports another version fails.
ABI_VERSION = 4

# Every symbol include/qmoe.h declares.
EXPORTS = (
    "qmoe_abi_version", "qmoe_status_str", "qmoe_last_hip_error", "qmoe_route",
    "qmoe_align_capacity", "qmoe_align_workspace", "qmoe_align", "qmoe_check_flags",
    "qmoe_align_noalloc", "qmoe_route_align", "qmoe_default_block_m",
    "qmoe_grouped_ffn_workspace", "qmoe_grouped_ffn_debug_offsets", "qmoe_grouped_ffn",
    "qmoe_grouped_ffn_profiled", "qmoe_combine", "qmoe_prepack", "qmoe_decode_workspace",
    "qmoe_decode", "qmoe_fp8_quant", "qmoe_fp8_matmul_workspace", "qmoe_fp8_matmul",
    "qmoe_fp8_grouped_matmul", "qmoe_balance_workspace", "qmoe_balance", "qmoe_balance_backward",
    "qmoe_pre_norm", "qmoe_post_norm", "qmoe_norm_backward_workspace", "qmoe_pre_norm_backward",
    "qmoe_post_norm_backward",
)
# Forms in which pre_norm and post_norm write a norm (qmoe_form).
NORM_FORMS = {"bf16": 0, "f32": 1, "int8": 2, "e4m3": 3, "e4m3_128": 4}
# Largest batch qmoe_decode takes (QMOE_DECODE_MAX_TOKENS).
DECODE_MAX_TOKENS = 16
# Batches up to this size take the one-launch qmoe_decode in moe_forward's
# automatic choice: measured on one MI355X for the 512-expert top-10 a8w4
# block (both paths on the same box), the one launch is faster at 1, 2 and
# 4 tokens (42.3 against 47.1 us, 58.2 against 64.9 us, 85.6 against 87.1
# us), level at 3 (72.1 against 71.6 us), slower from 6 tokens on (114.2
# against 111.2 us; 8 tokens 140.5 against 132.2 us), where the grouped
# kernels stream the weights at a higher rate.
DECODE_PREFERRED_MAX_TOKENS = 4


class QmoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_lib().qmoe_status_str(status).decode()} (status {status})")


class FfnDesc(ctypes.Structure):
    _fields_ = [("scheme", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
                ("I", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("block_m", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class Weights(ctypes.Structure):
    _fields_ = [("w13", ctypes.c_void_p), ("w13_scale", ctypes.c_void_p),
                ("w2", ctypes.c_void_p), ("w2_scale", ctypes.c_void_p)]


_LIB: Optional[ctypes.CDLL] = None


def _lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; "
                           "g.build()'` or `python -m quantized_mixture_experts_moe_amd.build_lib`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    L.qmoe_abi_version.restype = ctypes.c_int
    if L.qmoe_abi_version() != ABI_VERSION:
        raise RuntimeError(f"{LIB_PATH} reports ABI version {L.qmoe_abi_version()}, this "
                           f"binding expects {ABI_VERSION}; rebuild the library")
    L.qmoe_status_str.restype = ctypes.c_char_p
    L.qmoe_status_str.argtypes = [ctypes.c_int]
    L.qmoe_last_hip_error.restype = ctypes.c_int
    L.qmoe_route.restype = ctypes.c_int
    L.qmoe_route.argtypes = [vp, i32, i32, i32, vp, vp, vp]
    L.qmoe_align_capacity.restype = sz
    L.qmoe_align_capacity.argtypes = [i32, i32, i32, i32]
    L.qmoe_align_workspace.restype = sz
    L.qmoe_align_workspace.argtypes = [i32, i32, i32]
    L.qmoe_align.restype = ctypes.c_int
    L.qmoe_align.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
    L.qmoe_default_block_m.restype = ctypes.c_int32
    L.qmoe_default_block_m.argtypes = [i32, i32, i32, i32, i32, i32]
    L.qmoe_route_align.restype = ctypes.c_int
    L.qmoe_route_align.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.qmoe_align_noalloc.restype = ctypes.c_int
    L.qmoe_align_noalloc.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp]
    L.qmoe_check_flags.restype = ctypes.c_int
    L.qmoe_check_flags.argtypes = [vp, ctypes.POINTER(ctypes.c_int32), vp]
    L.qmoe_grouped_ffn_workspace.restype = sz
    L.qmoe_grouped_ffn_workspace.argtypes = [ctypes.POINTER(FfnDesc)]
    L.qmoe_grouped_ffn_debug_offsets.restype = ctypes.c_int
    L.qmoe_grouped_ffn_debug_offsets.argtypes = [ctypes.POINTER(FfnDesc),
                                                 ctypes.POINTER(sz), ctypes.POINTER(sz)]
    L.qmoe_grouped_ffn.restype = ctypes.c_int
    L.qmoe_grouped_ffn.argtypes = [ctypes.POINTER(FfnDesc), vp, vp, ctypes.POINTER(Weights),
                                   vp, vp, vp, vp, vp, sz, vp]
    L.qmoe_grouped_ffn_profiled.restype = ctypes.c_int
    L.qmoe_grouped_ffn_profiled.argtypes = [ctypes.POINTER(FfnDesc), vp, vp,
                                            ctypes.POINTER(Weights), vp, vp, vp, vp, vp, sz,
                                            ctypes.POINTER(ctypes.c_void_p), vp]
    L.qmoe_combine.restype = ctypes.c_int
    L.qmoe_combine.argtypes = [vp, i32, vp, i32, i32, i32, vp, vp, vp]
    L.qmoe_prepack.restype = ctypes.c_int
    L.qmoe_prepack.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp]
    L.qmoe_decode_workspace.restype = sz
    L.qmoe_decode_workspace.argtypes = [ctypes.POINTER(FfnDesc)]
    L.qmoe_decode.restype = ctypes.c_int
    L.qmoe_decode.argtypes = [ctypes.POINTER(FfnDesc), vp, vp, vp, ctypes.POINTER(Weights), vp,
                              vp, vp, vp, vp, vp, sz, vp]
    f32 = ctypes.c_float
    for name, res, args in (
            ("qmoe_fp8_quant", ctypes.c_int, [vp] + [i32] * 6 + [vp] * 5),
            ("qmoe_fp8_matmul_workspace", sz, [i32] * 3),
            ("qmoe_fp8_matmul", ctypes.c_int, [vp] * 4 + [i32] * 4 + [vp, i32, vp, sz, vp]),
            ("qmoe_fp8_grouped_matmul", ctypes.c_int,
             [vp, vp, i32] + [vp] * 6 + [i32] * 6 + [vp, i32, vp]),
            ("qmoe_balance_workspace", sz, [i32] * 2),
            ("qmoe_balance", ctypes.c_int, [vp] * 3 + [i32] * 3 + [f32] + [vp] * 5 + [sz, vp]),
            ("qmoe_balance_backward", ctypes.c_int, [vp] * 5 + [i32] * 3 + [f32, vp, vp]),
            ("qmoe_pre_norm", ctypes.c_int, [vp, i32, vp, f32] + [i32] * 3 + [vp] * 3),
            ("qmoe_post_norm", ctypes.c_int,
             [vp, vp, i32, vp, vp, i32, f32, f32, i32, i32, vp, vp, i32, vp, vp, vp]),
            ("qmoe_norm_backward_workspace", sz, [i32]),
            ("qmoe_pre_norm_backward", ctypes.c_int,
             [vp, vp, i32, vp, f32, vp, i32, i32, vp, vp, vp, sz, vp]),
            ("qmoe_post_norm_backward", ctypes.c_int,
             [vp, vp, i32, vp, vp, i32, f32, f32, i32, i32, vp, vp, vp, vp, vp, sz, vp])):
        getattr(L, name).restype, getattr(L, name).argtypes = res, args
    _LIB = L
    return L


def lib() -> ctypes.CDLL:
    return _lib()


def _check(status: int, what: str):
    if status != QMOE_OK:
        raise QmoeError(status, what)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to libqmoe must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libqmoe must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _ws(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------- routing

def route(logits: torch.Tensor, k: int, ids: Optional[torch.Tensor] = None,
          w: Optional[torch.Tensor] = None):
    """qmoe_route: (topk_ids int32 [T,k], topk_w fp32 [T,k])."""
    T, E = logits.shape
    assert logits.dtype == torch.float32
    if ids is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    if w is None:
        w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    _check(_lib().qmoe_route(_ptr(logits), T, E, k, _ptr(ids), _ptr(w), _stream(logits.device)),
           "qmoe_route")
    return ids, w


# ---------------------------------------------------------------- align

def align_capacity(T: int, k: int, E: int, block_m: int) -> int:
    return int(_lib().qmoe_align_capacity(T, k, E, block_m))


def align_workspace(T: int, k: int, E: int) -> int:
    return int(_lib().qmoe_align_workspace(T, k, E))


def align(topk_ids: torch.Tensor, E: int, block_m: int, ws: Optional[torch.Tensor] = None,
          out: Optional[dict] = None) -> dict:
    """qmoe_align: expert-sorted, block_m-padded pair slots (``out`` reuses a
    previous result's buffers)."""
    T, k = topk_ids.shape
    dev = topk_ids.device
    cap = align_capacity(T, k, E, block_m)
    if out is None:
        out = {
            "sorted_pair_ids": torch.empty(cap, dtype=torch.int32, device=dev),
            "tile_expert": torch.empty(cap // block_m, dtype=torch.int32, device=dev),
            "expert_offsets": torch.empty(E + 1, dtype=torch.int32, device=dev),
            "num_padded": torch.empty(1, dtype=torch.int32, device=dev),
            "block_m": block_m,
        }
        ws = out.get("ws", ws)
    else:
        ws = out["ws"]
    need = align_workspace(T, k, E)
    if ws is None or ws.numel() < need:
        ws = _ws(need, dev)
    out["ws"] = ws
    _check(_lib().qmoe_align(_ptr(topk_ids), T, k, E, block_m, _ptr(out["sorted_pair_ids"]),
                             _ptr(out["tile_expert"]), _ptr(out["expert_offsets"]),
                             _ptr(out["num_padded"]), _ptr(ws), ws.numel(), _stream(dev)),
           "qmoe_align")
    return out


def route_align(logits: torch.Tensor, k: int, block_m: int, ids=None, w=None,
                out: Optional[dict] = None):
    """qmoe_route_align: (topk_ids, topk_w, grouping dict) in one call (one
    launch up to 16 tokens); ``out`` reuses a previous grouping's buffers."""
    T, E = logits.shape
    assert logits.dtype == torch.float32
    dev = logits.device
    if ids is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    if w is None:
        w = torch.empty((T, k), dtype=torch.float32, device=dev)
    cap = align_capacity(T, k, E, block_m)
    if out is None:
        out = {
            "sorted_pair_ids": torch.empty(cap, dtype=torch.int32, device=dev),
            "tile_expert": torch.empty(cap // block_m, dtype=torch.int32, device=dev),
            "expert_offsets": torch.empty(E + 1, dtype=torch.int32, device=dev),
            "num_padded": torch.empty(1, dtype=torch.int32, device=dev),
            "block_m": block_m,
        }
    need = align_workspace(T, k, E)
    ws = out.get("ws")
    if ws is None or ws.numel() < need:
        ws = _ws(need, dev)
    out["ws"] = ws
    _check(_lib().qmoe_route_align(_ptr(logits), T, E, k, block_m, _ptr(ids), _ptr(w),
                                   _ptr(out["sorted_pair_ids"]), _ptr(out["tile_expert"]),
                                   _ptr(out["expert_offsets"]), _ptr(out["num_padded"]),
                                   _ptr(ws), ws.numel(), _stream(dev)), "qmoe_route_align")
    return ids, w, out


def align_noalloc(topk_ids: torch.Tensor, E: int, block_m: int, out: Optional[dict] = None,
                  flags: Optional[torch.Tensor] = None) -> dict:
    """qmoe_align_noalloc: the outputs of qmoe_align with the workspace held
    inside the library (``out`` reuses a previous result's buffers; ``flags``
    is an optional int32 device tensor of one element for the flag word)."""
    T, k = topk_ids.shape
    dev = topk_ids.device
    cap = align_capacity(T, k, E, block_m)
    if out is None:
        out = {
            "sorted_pair_ids": torch.empty(cap, dtype=torch.int32, device=dev),
            "tile_expert": torch.empty(cap // block_m, dtype=torch.int32, device=dev),
            "expert_offsets": torch.empty(E + 1, dtype=torch.int32, device=dev),
            "num_padded": torch.empty(1, dtype=torch.int32, device=dev),
            "block_m": block_m,
        }
    _check(_lib().qmoe_align_noalloc(_ptr(topk_ids), T, k, E, block_m,
                                     _ptr(out["sorted_pair_ids"]), _ptr(out["tile_expert"]),
                                     _ptr(out["expert_offsets"]), _ptr(out["num_padded"]),
                                     _ptr(flags), _stream(dev)), "qmoe_align_noalloc")
    return out


def check_flags(align_ws: torch.Tensor) -> int:
    v = ctypes.c_int32(0)
    _check(_lib().qmoe_check_flags(_ptr(align_ws), ctypes.byref(v), _stream(align_ws.device)),
           "qmoe_check_flags")
    return int(v.value)


# ---------------------------------------------------------------- grouped FFN

def make_desc(scheme: str, T: int, H: int, I: int, E: int, k: int, block_m: int,
              flags: int = 0) -> FfnDesc:
    return FfnDesc(SCHEME_CODE[scheme], T, H, I, E, k, block_m, flags)


def grouped_ffn_workspace(desc: FfnDesc) -> int:
    return int(_lib().qmoe_grouped_ffn_workspace(ctypes.byref(desc)))


def grouped_ffn_debug_offsets(desc: FfnDesc):
    a1, a2 = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(_lib().qmoe_grouped_ffn_debug_offsets(ctypes.byref(desc), ctypes.byref(a1),
                                                 ctypes.byref(a2)), "debug offsets")
    return int(a1.value), int(a2.value)


def prepack(scheme: str, codes: torch.Tensor, scales: torch.Tensor):
    """qmoe_prepack of one stacked weight tensor (codes [E, N, K bytes]);
    returns (codes, scales) in the streaming layout, same shapes and dtypes.
    W8A8 scales are per-channel and stay as they are (returned as given)."""
    E, N = codes.shape[0], codes.shape[1]
    K = codes.shape[2] * (1 if scheme == "w8a8" else 2)
    c_out = torch.empty_like(codes)
    s_out = scales if scheme == "w8a8" else torch.empty_like(scales)
    _check(_lib().qmoe_prepack(SCHEME_CODE[scheme], E, N, K, _ptr(codes), _ptr(scales),
                               _ptr(c_out), None if scheme == "w8a8" else _ptr(s_out),
                               _stream(codes.device)), "qmoe_prepack")
    return c_out, s_out


def prepack_weights(scheme: str, weights: dict) -> dict:
    """Both projections of a weight dict in the streaming layout; the
    returned dict carries prepacked=True, which grouped_ffn turns into
    QMOE_FLAG_PREPACKED."""
    w13, w13s = prepack(scheme, weights["w13"], weights["w13_scale"])
    w2, w2s = prepack(scheme, weights["w2"], weights["w2_scale"])
    return {"w13": w13, "w13_scale": w13s, "w2": w2, "w2_scale": w2s, "prepacked": True}


def grouped_ffn(scheme: str, x: torch.Tensor, x_scale: Optional[torch.Tensor], weights: dict,
                al: dict, E: int, k: int, flags: int = 0, ws: Optional[torch.Tensor] = None,
                y_pairs: Optional[torch.Tensor] = None, stage_events=None):
    """qmoe_grouped_ffn (qmoe_grouped_ffn_profiled when four recorded
    torch.cuda.Event objects are given); returns (y_pairs [T*k, H], ws)."""
    T, H = x.shape
    I = weights["w13"].shape[1] // 2
    dev = x.device
    if weights.get("prepacked", False):
        flags |= QMOE_FLAG_PREPACKED
    desc = make_desc(scheme, T, H, I, E, k, al["block_m"], flags)
    need = grouped_ffn_workspace(desc)
    if need == 0:
        raise QmoeError(QMOE_ERR_INVALID_ARG, "qmoe_grouped_ffn_workspace")
    if ws is None or ws.numel() < need:
        ws = _ws(need, dev)
    if y_pairs is None:
        ydt = torch.float32 if scheme == "w8a8" else torch.bfloat16
        y_pairs = torch.empty((T * k, H), dtype=ydt, device=dev)
    w = Weights(_ptr(weights["w13"]), _ptr(weights["w13_scale"]), _ptr(weights["w2"]),
                _ptr(weights["w2_scale"]))
    args = (ctypes.byref(desc), _ptr(x), _ptr(x_scale), ctypes.byref(w),
            _ptr(al["sorted_pair_ids"]), _ptr(al["tile_expert"]), _ptr(al["num_padded"]),
            _ptr(y_pairs), _ptr(ws), ws.numel())
    if stage_events is None:
        _check(_lib().qmoe_grouped_ffn(*args, _stream(dev)), "qmoe_grouped_ffn")
    else:
        ev = (ctypes.c_void_p * 4)(*[e.cuda_event for e in stage_events])
        _check(_lib().qmoe_grouped_ffn_profiled(*args, ev, _stream(dev)),
               "qmoe_grouped_ffn_profiled")
    return y_pairs, ws


# ---------------------------------------------------------------- combine

def combine(y_pairs: torch.Tensor, topk_w: torch.Tensor, want_bf16: bool = True,
            want_f32: bool = False, out_bf16=None, out_f32=None):
    """qmoe_combine; returns (out_bf16 or None, out_f32 or None)."""
    T, k = topk_w.shape
    H = y_pairs.shape[1]
    dev = y_pairs.device
    ydt = QMOE_DT_F32 if y_pairs.dtype == torch.float32 else QMOE_DT_BF16
    if want_bf16 and out_bf16 is None:
        out_bf16 = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    if want_f32 and out_f32 is None:
        out_f32 = torch.empty((T, H), dtype=torch.float32, device=dev)
    _check(_lib().qmoe_combine(_ptr(y_pairs), ydt, _ptr(topk_w), T, k, H, _ptr(out_bf16),
                               _ptr(out_f32), _stream(dev)), "qmoe_combine")
    return out_bf16, out_f32


# ---------------------------------------------------------------- whole layer

def moe_forward(scheme: str, logits: torch.Tensor, x: torch.Tensor,
                x_scale: Optional[torch.Tensor], weights: dict, k: int, block_m: int,
                flags: int = 0, want_f32: bool = False, fused_routing: bool = False,
                path: str = "grouped") -> dict:
    """route -> align -> grouped_ffn -> combine, all on the current stream
    (``fused_routing``: route and align through qmoe_route_align).
    ``path="auto"`` sends batches of up to DECODE_PREFERRED_MAX_TOKENS tokens
    (without debug flags) to the one-launch qmoe_decode instead; its outputs
    are the same bits."""
    if path not in ("grouped", "auto"):
        raise ValueError(f"path must be 'grouped' or 'auto', not {path!r}")
    if path == "auto" and flags == 0 and 0 < x.shape[0] <= DECODE_PREFERRED_MAX_TOKENS:
        return decode_forward(scheme, logits, x, x_scale, weights, k, want_f32=want_f32)
    E = logits.shape[1]
    if fused_routing:
        ids, w, al = route_align(logits, k, block_m)
    else:
        ids, w = route(logits, k)
        al = align(ids, E, block_m)
    y, ws = grouped_ffn(scheme, x, x_scale, weights, al, E, k, flags=flags)
    out_bf16, out_f32 = combine(y, w, want_bf16=True, want_f32=want_f32)
    return {"topk_ids": ids, "topk_w": w, "align": al, "y_pairs": y, "ws": ws,
            "out": out_bf16, "out_f32": out_f32}


# ---------------------------------------------------------------- one-launch decode

def decode_workspace(scheme: str, H: int, I: int, E: int, k: int, flags: int = 0) -> int:
    """qmoe_decode_workspace (bytes; sized for every T up to DECODE_MAX_TOKENS)."""
    return int(_lib().qmoe_decode_workspace(ctypes.byref(make_desc(scheme, 1, H, I, E, k, 16,
                                                                   flags))))


def decode_forward(scheme: str, logits: torch.Tensor, x: torch.Tensor,
                   x_scale: Optional[torch.Tensor], weights: dict, k: int,
                   want_f32: bool = False, ws: Optional[torch.Tensor] = None,
                   y_pairs: Optional[torch.Tensor] = None, want_y: bool = True,
                   out: Optional[dict] = None) -> dict:
    """qmoe_decode: the whole layer in one launch for T <= DECODE_MAX_TOKENS.
    ``ws`` must come from a previous call (or be zero-filled): the library
    keeps arrival counters in it that each call leaves at zero."""
    T, H = x.shape
    E = logits.shape[1]
    I = weights["w13"].shape[1] // 2
    dev = x.device
    flags = QMOE_FLAG_PREPACKED if weights.get("prepacked", False) else 0
    desc = make_desc(scheme, T, H, I, E, k, 16, flags)
    need = int(_lib().qmoe_decode_workspace(ctypes.byref(desc)))
    if need == 0:
        raise QmoeError(QMOE_ERR_INVALID_ARG if T <= DECODE_MAX_TOKENS else QMOE_ERR_UNSUPPORTED,
                        "qmoe_decode_workspace")
    if ws is None or ws.numel() < need:
        ws = torch.zeros(need, dtype=torch.uint8, device=dev)
    out = {} if out is None else out
    ids = out.get("topk_ids")
    if ids is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = out.get("topk_w")
    if w is None:
        w = torch.empty((T, k), dtype=torch.float32, device=dev)
    if want_y and y_pairs is None:
        ydt = torch.float32 if scheme == "w8a8" else torch.bfloat16
        y_pairs = torch.empty((T * k, H), dtype=ydt, device=dev)
    ob = out.get("out")
    if ob is None:
        ob = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    of = out.get("out_f32")
    if want_f32 and of is None:
        of = torch.empty((T, H), dtype=torch.float32, device=dev)
    wts = Weights(_ptr(weights["w13"]), _ptr(weights["w13_scale"]), _ptr(weights["w2"]),
                  _ptr(weights["w2_scale"]))
    _check(_lib().qmoe_decode(ctypes.byref(desc), _ptr(logits), _ptr(x), _ptr(x_scale),
                              ctypes.byref(wts), _ptr(ids), _ptr(w), _ptr(y_pairs), _ptr(ob),
                              _ptr(of) if want_f32 else None, _ptr(ws), ws.numel(),
                              _stream(dev)), "qmoe_decode")
    return {"topk_ids": ids, "topk_w": w, "y_pairs": y_pairs, "ws": ws, "out": ob,
            "out_f32": of if want_f32 else None}



# ---------------------------------------------------------------- around the experts
# Block-128 fp8 quantizer and products, balance loss, norms.  These check
# shapes, types and devices here (ValueError), since the C ABI sees pointers
# only, and run on the current stream of the tensors' device.  None of them
# records itself for autograd, whatever its arguments require: gradients are calls
# of their own.

# These checks and look-ups stand in front of calls whose kernels take a few
# microseconds, so messages are formed only when they are raised.

def _need(ok, what: str, *values):
    if not ok:
        raise ValueError(what % values if values else what)


def _tensor(t, name: str, shape: tuple, *dtypes):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))}, not {t.dtype}")


def _one_device(first, *others):
    """The device of the tensors given (None for one left out)."""
    dev = first.device
    if dev.type != "cuda":
        raise ValueError(f"tensors passed to libqmoe must live on the GPU, not on {dev}")
    for t in others:
        if t is not None and t.device != dev:
            raise ValueError(f"all tensors must live on one GPU, not on {dev} and {t.device}")
    return dev


def _addr(t):
    """A tensor's address (None for one left out)."""
    if t is None:
        return None
    if t.is_contiguous():
        return t.data_ptr()
    raise ValueError("tensors passed to libqmoe must be contiguous")


def _raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# The current device and its stream without Python objects in between (0.1
# against 1.9 us), where this torch has the calls.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(dev, name: str, *args):
    """The library call `name` with the device current (a launch goes to the
    current device's context) and its current stream as the last argument."""
    index = dev.index
    if _current_device() == index:
        status = getattr(_LIB or _lib(), name)(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            status = getattr(_LIB or _lib(), name)(*args, _raw_stream(index))
    if status != QMOE_OK:
        raise QmoeError(status, name)


def _float_kind(t, name: str) -> int:
    if t.dtype == torch.bfloat16:
        return QMOE_DT_BF16
    if t.dtype == torch.float32:
        return QMOE_DT_F32
    raise ValueError(f"{name} must be bfloat16 or float32, not {t.dtype}")


def _blocks(n: int) -> int:
    return (n + 127) // 128


def fp8_quant(x: torch.Tensor, block: bool = False, act: Optional[str] = None, rows: bool = True,
              cols: bool = False) -> dict:
    """qmoe_fp8_quant.  x [M, K] (weights with block=True: [N, K] or the stack
    [E, N, K]; act="silu_mul": [M, 2K] = gate | up).  Returns "codes" (uint8
    e4m3) and "scale" with `rows`, "codes_t" and "scale_t" (the transpose,
    groups along the columns of x) with `cols`."""
    _need(act in (None, "silu_mul"), "act must be None or 'silu_mul', not %r", act)
    _need(rows or cols, "rows or cols (or both)")
    _need(not (block and act), "block scales are for weights: act does not go with them")
    _need(x.dim() == 2 or (block and x.dim() == 3), "x must be [M, K] (or [E, N, K] with block)")
    dt, dev = _float_kind(x, "x"), _one_device(x)
    B = x.shape[0] if x.dim() == 3 else 1
    M, K = x.shape[-2:]
    if act:
        _need(K % 2 == 0, "act='silu_mul' takes [M, 2K]")
        K //= 2
    _need(K >= 1, "x has no columns")
    lead = (B,) if x.dim() == 3 else ()
    out = {}

    def new(shape, dtype):
        return torch.empty(shape, dtype=dtype, device=dev)

    if rows:
        out["codes"] = new(lead + (M, 128 * _blocks(K)), torch.uint8)
        out["scale"] = new(lead + ((_blocks(M), _blocks(K)) if block else (_blocks(K), M)),
                           torch.float32)
    if cols:
        out["codes_t"] = new(lead + (K, 128 * _blocks(M)), torch.uint8)
        out["scale_t"] = new(lead + ((_blocks(K), _blocks(M)) if block else (_blocks(M), K)),
                             torch.float32)
    _call(dev, "qmoe_fp8_quant", _addr(x), dt, B, M, K, int(block), int(act is not None),
          _addr(out.get("codes")), _addr(out.get("scale")), _addr(out.get("codes_t")),
          _addr(out.get("scale_t")))
    return out


def _operand(codes, scale, name: str, block: bool, lead=()):
    """Checks codes [.., rows, K] with their scales; returns (rows, K)."""
    shape = codes.shape
    _need(len(shape) == 2 + len(lead), "%s must have %d axes", name, 2 + len(lead))
    n, k = shape[-2], shape[-1]
    _need(k >= 128 and k % 128 == 0, "%s's row length %d is not a multiple of 128", name, k)
    kb = k // 128
    want = lead + (((n + 127) // 128, kb) if block else (kb, n))
    if (scale.shape != want or codes.dtype != torch.uint8 or scale.dtype != torch.float32
            or shape[:-2] != lead):
        _tensor(codes, name, lead + (n, k), torch.uint8)
        _tensor(scale, f"{name}_scale", want, torch.float32)
    return n, k


def _out(out, shape, dtype, dev):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _tensor(out, "out", shape, dtype)
    return out


def fp8_matmul_workspace(M: int, N: int, K: int) -> int:
    return int(_lib().qmoe_fp8_matmul_workspace(M, N, K))


def fp8_matmul(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
               b_block: bool = True, out_dtype: torch.dtype = torch.bfloat16,
               ws: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """qmoe_fp8_matmul: a [M, K] . b [N, K]^T -> [M, N] of e4m3 codes (uint8);
    b_block says that b's scales are per 128 x 128 block, not per row."""
    M, K = _operand(a, a_scale, "a", False)
    N, K2 = _operand(b, b_scale, "b", b_block)
    _need(K == K2, "a's rows have %d values, b's %d", K, K2)
    _need(out_dtype in (torch.bfloat16, torch.float32), "out_dtype must be bfloat16 or float32")
    dev = _one_device(a, a_scale, b, b_scale, ws, out)
    out = _out(out, (M, N), out_dtype, dev)
    need = fp8_matmul_workspace(M, N, K)
    if ws is None or ws.numel() * ws.element_size() < need:
        ws = _ws(need, dev) if need else None
    _call(dev, "qmoe_fp8_matmul", _addr(a), _addr(a_scale), _addr(b), _addr(b_scale),
          int(b_block), M, N, K, _addr(out), _float_kind(out, "out"), _addr(ws),
          0 if ws is None else ws.numel() * ws.element_size())
    return out


def fp8_grouped_matmul(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor,
                       b_scale: torch.Tensor, al: dict, k: int, pair_rows: bool = False,
                       out_dtype: torch.dtype = torch.bfloat16,
                       out: Optional[torch.Tensor] = None):
    """qmoe_fp8_grouped_matmul: row p of the result is a[row(p)] . b[expert of
    pair p]^T, row(p) = p // k (a [T, K]) or p (pair_rows, a [T*k, K]);
    `al` is align's (or route_align's) result."""
    _need(b.dim() == 3, "b must be [E, N, K]")
    E = b.shape[0]
    rows, K = _operand(a, a_scale, "a", False)
    N, K2 = _operand(b, b_scale, "b", True, (E,))
    _need(K == K2, "a's rows have %d values, b's %d", K, K2)
    _need(k >= 1 and (not pair_rows or rows % k == 0),
          "%d pair rows are not a multiple of k = %d", rows, k)
    _need(out_dtype in (torch.bfloat16, torch.float32), "out_dtype must be bfloat16 or float32")
    T, bm = rows // k if pair_rows else rows, al["block_m"]
    cap = align_capacity(T, k, E, bm)
    _need(cap > 0, "bad sizes: T %d, k %d, E %d, block_m %d", T, k, E, bm)
    _tensor(al["sorted_pair_ids"], "sorted_pair_ids", (cap,), torch.int32)
    _tensor(al["tile_expert"], "tile_expert", (cap // bm,), torch.int32)
    _tensor(al["expert_offsets"], "expert_offsets", (E + 1,), torch.int32)
    _tensor(al["num_padded"], "num_padded", (1,), torch.int32)
    dev = _one_device(a, a_scale, b, b_scale, al["sorted_pair_ids"], al["tile_expert"],
                      al["expert_offsets"], al["num_padded"], out)
    out = _out(out, (T * k, N), out_dtype, dev)
    _call(dev, "qmoe_fp8_grouped_matmul", _addr(a), _addr(a_scale), int(pair_rows), _addr(b),
          _addr(b_scale), _addr(al["sorted_pair_ids"]), _addr(al["tile_expert"]),
          _addr(al["expert_offsets"]), _addr(al["num_padded"]), T, k, E, bm, N, K, _addr(out),
          _float_kind(out, "out"))
    return out


# Tile height (align's block_m) for the block-128 fp8 expert products: they
# take an expert's rows whatever the height, so the least padding is best.
FP8_BLOCK_M = 16


def fp8_moe_forward(logits: torch.Tensor, x: torch.Tensor, x_scale: torch.Tensor, weights: dict,
                    k: int) -> dict:
    """The layer with block-128 fp8 experts: route -> align -> gate/up product
    -> SiLU*mul and quantization -> down product -> combine.  x [T, H] codes
    with x_scale [H/128, T] (fp8_quant or a norm's "e4m3_128" form); weights:
    w13 [E, 2I, H], w2 [E, H, I] codes and their 128 x 128 block scales
    (fp8_quant(w, block=True)), H % 128 == 0, I % 128 == 0.  Between the calls
    values are rounded as they would be between calls of a user's own: gate/up
    and the pairs' outputs to bf16, SiLU*mul to e4m3."""
    T, E = logits.shape
    _need(x.shape[0] == T, "x has %d rows, logits %d", x.shape[0], T)
    with torch.cuda.device(_one_device(logits, x)):
        ids, w, al = route_align(logits, k, FP8_BLOCK_M)
        gu = fp8_grouped_matmul(x, x_scale, weights["w13"], weights["w13_scale"], al, k)
        h = fp8_quant(gu, act="silu_mul")
        y = fp8_grouped_matmul(h["codes"], h["scale"], weights["w2"], weights["w2_scale"], al, k,
                               pair_rows=True)
        out, _ = combine(y, w)
    return {"topk_ids": ids, "topk_w": w, "align": al, "y_pairs": y, "out": out}


def _mask_ptr(mask, T: int):
    if mask is None:
        return None
    _tensor(mask, "mask", (T,), torch.uint8, torch.bool)
    return _addr(mask)


def balance_loss(logits: torch.Tensor, topk_ids: torch.Tensor,
                 mask: Optional[torch.Tensor] = None, coef: float = 1.0,
                 ws: Optional[torch.Tensor] = None) -> dict:
    """qmoe_balance: {"loss" fp32 [1], "counts" int32 [E], "probs" fp32 [E],
    "tokens" int32 [1]} of router logits [T, E] and their picks [T, k]; mask
    [T] (uint8 or bool): 0 drops a token."""
    _need(logits.dim() == 2 and topk_ids.dim() == 2, "logits must be [T, E] and topk_ids [T, k]")
    T, E = logits.shape
    k = topk_ids.shape[1]
    _tensor(logits, "logits", (T, E), torch.float32)
    _tensor(topk_ids, "topk_ids", (T, k), torch.int32)
    dev = _one_device(logits, topk_ids, mask, ws)
    need = _lib().qmoe_balance_workspace(T, E)
    if need and (ws is None or ws.numel() * ws.element_size() < need):
        ws = _ws(need, dev)
    r = {"loss": torch.empty(1, dtype=torch.float32, device=dev),
         "counts": torch.empty(E, dtype=torch.int32, device=dev),
         "probs": torch.empty(E, dtype=torch.float32, device=dev),
         "tokens": torch.empty(1, dtype=torch.int32, device=dev)}
    _call(dev, "qmoe_balance", _addr(logits), _addr(topk_ids), _mask_ptr(mask, T), T, E, k, coef,
          r["loss"].data_ptr(), r["counts"].data_ptr(), r["probs"].data_ptr(),
          r["tokens"].data_ptr(), _addr(ws), 0 if ws is None else ws.numel() * ws.element_size())
    return r


def balance_loss_backward(logits: torch.Tensor, counts: torch.Tensor, tokens: torch.Tensor,
                          k: int, dloss: torch.Tensor, mask: Optional[torch.Tensor] = None,
                          coef: float = 1.0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """qmoe_balance_backward: the gradient of balance_loss (same logits, mask
    and coef, its counts and tokens) to the logits; dloss fp32 [1]."""
    _need(logits.dim() == 2, "logits must be [T, E]")
    T, E = logits.shape
    _tensor(logits, "logits", (T, E), torch.float32)
    _tensor(counts, "counts", (E,), torch.int32)
    _tensor(tokens, "tokens", (1,), torch.int32)
    _tensor(dloss, "dloss", (1,), torch.float32)
    dev = _one_device(logits, counts, tokens, dloss, mask, out)
    out = _out(out, (T, E), torch.float32, dev)
    _call(dev, "qmoe_balance_backward", _addr(logits), _mask_ptr(mask, T), _addr(counts),
          _addr(tokens), _addr(dloss), T, E, k, coef, _addr(out))
    return out


def _new_form(form: str, T: int, H: int, dev):
    """Code of a form and its new (n, scale)."""
    _need(form in NORM_FORMS,
          "a norm is written as one of %s, not %r", list(NORM_FORMS), form)
    if form in ("bf16", "f32"):
        dt = torch.bfloat16 if form == "bf16" else torch.float32
        return NORM_FORMS[form], torch.empty((T, H), dtype=dt, device=dev), None
    if form == "e4m3_128":
        n = torch.empty((T, 128 * _blocks(H)), dtype=torch.uint8, device=dev)
        return NORM_FORMS[form], n, torch.empty((_blocks(H), T), dtype=torch.float32, device=dev)
    n = torch.empty((T, H), dtype=torch.int8 if form == "int8" else torch.uint8, device=dev)
    return NORM_FORMS[form], n, torch.empty(T, dtype=torch.float32, device=dev)


def _gate_kind(gate, T: int, H: int, dtype):
    """(qmoe_gate, its pointer) of a gate that broadcasts to [T, H] as torch
    tensors do: None, fp32 [H] per column, fp32 [T, 1] per token, or [T, H] in
    the activations' type."""
    if gate is None:
        return 0, None
    if gate.dim() == 1:
        _tensor(gate, "a gate per column", (H,), torch.float32)
        return 1, _addr(gate)
    if tuple(gate.shape) == (T, 1) and (H > 1 or gate.dtype != dtype):
        _tensor(gate, "a gate per token", (T, 1), torch.float32)
        return 2, _addr(gate)
    _tensor(gate, "gate", (T, H), dtype)
    return 3, _addr(gate)


def pre_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, out: str = "bf16"):
    """qmoe_pre_norm: (n, scale) with n = x / rms(x) * weight in the form
    `out`: "bf16", "f32" (scale None), "int8" or "e4m3" (scale [T]: the
    grouped FFN's x and x_scale), "e4m3_128" (scale [H/128, T])."""
    _need(x.dim() == 2, "x must be [T, H]")
    T, H = x.shape
    dt = _float_kind(x, "x")
    _tensor(weight, "weight", (H,), torch.float32)
    dev = _one_device(x, weight)
    form, n, scale = _new_form(out, T, H, dev)
    _call(dev, "qmoe_pre_norm", _addr(x), dt, _addr(weight), eps, T, H, form, n.data_ptr(),
          _addr(scale))
    return n, scale


def post_norm(y: torch.Tensor, weight: torch.Tensor, x: torch.Tensor,
              gate: Optional[torch.Tensor] = None, alpha: float = 1.0, eps: float = 1e-6,
              next_weight: Optional[torch.Tensor] = None, next_out: str = "bf16",
              out: Optional[torch.Tensor] = None):
    """qmoe_post_norm: (out, n, scale) with out = alpha * x + gate * (y /
    rms(y) * weight) and, with next_weight, the next block's norm of out in
    the form next_out (as pre_norm gives; else n and scale are None).
    ``out`` may be x."""
    _need(y.dim() == 2, "y must be [T, H]")
    T, H = y.shape
    dt = _float_kind(y, "y")
    _tensor(x, "x", (T, H), y.dtype)
    _tensor(weight, "weight", (H,), torch.float32)
    dev = _one_device(y, x, weight, gate, next_weight, out)
    kind, gp = _gate_kind(gate, T, H, y.dtype)
    out = _out(out, (T, H), y.dtype, dev)
    form, n, scale = 0, None, None
    if next_weight is not None:
        _tensor(next_weight, "next_weight", (H,), torch.float32)
        form, n, scale = _new_form(next_out, T, H, dev)
    _call(dev, "qmoe_post_norm", _addr(y), _addr(x), dt, _addr(weight), gp, kind, alpha, eps, T, H,
          _addr(out), _addr(next_weight), form, _addr(n), _addr(scale))
    return out, n, scale


def _norm_ws(ws, H: int, dev):
    need = int(_lib().qmoe_norm_backward_workspace(H))
    if ws is None or ws.numel() * ws.element_size() < need:
        ws = _ws(need, dev)
    return ws, ws.numel() * ws.element_size()


def pre_norm_backward(dn: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                      dres: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """qmoe_pre_norm_backward: (dx, dweight) for the gradient dn of pre_norm's
    n; dres, the gradient that reaches x along the residual stream, is added
    to dx."""
    _need(x.dim() == 2, "x must be [T, H]")
    T, H = x.shape
    dt = _float_kind(x, "x")
    _tensor(dn, "dn", (T, H), x.dtype)
    _tensor(weight, "weight", (H,), torch.float32)
    if dres is not None:
        _tensor(dres, "dres", (T, H), x.dtype)
    dev = _one_device(dn, x, weight, dres, ws)
    dx = torch.empty_like(x)
    dw = torch.empty(H, dtype=torch.float32, device=dev)
    ws, nbytes = _norm_ws(ws, H, dev)
    _call(dev, "qmoe_pre_norm_backward", _addr(dn), _addr(x), dt, _addr(weight), eps,
          _addr(dres), T, H, dx.data_ptr(), dw.data_ptr(), _addr(ws), nbytes)
    return dx, dw


def post_norm_backward(dout: torch.Tensor, y: torch.Tensor, weight: torch.Tensor,
                       gate: Optional[torch.Tensor] = None, alpha: float = 1.0,
                       eps: float = 1e-6, ws: Optional[torch.Tensor] = None) -> dict:
    """qmoe_post_norm_backward: {"dy", "dres" (x's gradient, alpha * dout),
    "dw", "dgate" (None without a gate)} for the gradient dout of post_norm's
    out."""
    _need(y.dim() == 2, "y must be [T, H]")
    T, H = y.shape
    dt = _float_kind(y, "y")
    _tensor(dout, "dout", (T, H), y.dtype)
    _tensor(weight, "weight", (H,), torch.float32)
    dev = _one_device(dout, y, weight, gate, ws)
    kind, gp = _gate_kind(gate, T, H, y.dtype)
    r = {"dy": torch.empty_like(y), "dres": torch.empty_like(y),
         "dw": torch.empty(H, dtype=torch.float32, device=dev),
         "dgate": None if gate is None else torch.empty_like(gate)}
    ws, nbytes = _norm_ws(ws, H, dev)
    _call(dev, "qmoe_post_norm_backward", _addr(dout), _addr(y), dt, _addr(weight), gp, kind, alpha,
          eps, T, H, r["dy"].data_ptr(), r["dres"].data_ptr(), r["dw"].data_ptr(),
          _addr(r["dgate"]), _addr(ws), nbytes)
    return r
