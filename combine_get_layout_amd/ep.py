"""Thin Python binding of libep.so (include/ep.h): argument marshalling only.

Every function has the name of the C entry point it calls and takes torch
tensors that already live on the GPU; it passes their data pointers, the shape
and the current HIP stream through ctypes and turns a negative status into a
RuntimeError. No step of the computation happens here. The allocation helpers
at the bottom only create empty tensors of the sizes the C ABI documents.

If libep.so has not been built the first call raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libep.so")

EP_OK, EP_ERR_ARG, EP_ERR_UNSUPPORTED, EP_ERR_HIP, EP_ERR_DEVICE, EP_ERR_SCRATCH = 0, -1, -2, -3, -4, -5
EP_LAYOUT_SCRATCH_BYTES = 4 << 20
EP_DEVERR_EXPERT_ID, EP_DEVERR_CAPACITY, EP_DEVERR_FLAG, EP_DEVERR_TIMEOUT = 1, 2, 4, 8
EP_DEVERR_LOGIT = 16
EP_FUSED_WITHHOLD = 1
EP_SEG_BF16, EP_SEG_FP8, EP_SEG_SCALES = 1, 2, 4
EP_FMT_PLAIN, EP_FMT_CHUNKED = 0, 1
EP_HIER_SCALEOUT, EP_HIER_FORWARD = 1, 2
EP_WEIGHT_NK, EP_WEIGHT_KN = 0, 1
EP_GRAD_BF16, EP_GRAD_F32 = 0, 1
EP_FEW_MAX_TOKENS = 128
EP_STREAM_BF16, EP_STREAM_F32 = 0, 1
EP_SCORE_SOFTMAX, EP_SCORE_SIGMOID = 0, 1
EP_W4_INT, EP_W4_E2M1 = 0, 1

_P = ctypes.c_void_p
_byref = ctypes.byref


class ep_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "K", "E", "R", "G")]


LAYOUT_FIELDS = ("tokens_per_expert", "tokens_per_rank", "tokens_per_group", "expert_offsets",
                 "rank_offsets", "group_offsets", "is_token_in_rank", "is_token_in_group",
                 "slot", "group_slot", "expert_slot")


class ep_layout(ctypes.Structure):
    _fields_ = [(n, _P) for n in LAYOUT_FIELDS]


class ep_tokens(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("x", "x_fp8", "x_scales", "topk_idx", "topk_weights")]


class ep_recv(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("x", "x_fp8", "x_scales", "src_idx", "topk_idx",
                                  "topk_weights")] + [("capacity", ctypes.c_int64)]


class ep_fused_opts(ctypes.Structure):
    _fields_ = [("tile_tokens", ctypes.c_int32), ("timeout_us", ctypes.c_uint32),
                ("test_flags", ctypes.c_uint32), ("withhold_batch", ctypes.c_int32),
                ("ring_batches", ctypes.c_int32)]


class ep_sources(ctypes.Structure):
    _fields_ = [("S", ctypes.c_int32), ("capacity", ctypes.c_int64), ("counts", _P),
                ("recv_offsets", _P), ("src_slot", _P)]


class ep_rows(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("x", "x_fp8", "x_scales")]


class ep_experts(ctypes.Structure):
    _fields_ = [("F", ctypes.c_int32)] + [(n, _P) for n in ("w13", "w2", "w13_fp8", "w13_scales",
                                                            "w2_fp8", "w2_scales")]


class ep_norm_out(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("h", "y", "y_fp8", "y_scales", "rstd")]


class ep_router(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("score", "top_groups", "group_top", "normalize")] + \
               [("scale", ctypes.c_float), ("bias", _P)]


class ep_experts_w4(ctypes.Structure):
    _fields_ = [("F", ctypes.c_int32), ("form", ctypes.c_int32)] + \
               [(n, _P) for n in ("w13", "w13_scales", "w2", "w2_scales")]


EXPORTS = ("ep_workspace_bytes", "ep_record_bytes", "ep_chunked_record_bytes", "ep_get_layout",
           "ep_get_layout_noalloc",
           "ep_dispatch", "ep_dispatch_expand", "ep_hierarchical_dispatch",
           "ep_hierarchical_dispatch_fused", "ep_combine",
           "ep_combine_expand", "ep_partial_row_bytes", "ep_combine_two_level",
           "ep_source_workspace_bytes", "ep_source_layout", "ep_source_dispatch",
           "ep_copy_epilogue", "ep_source_dispatch_fused", "ep_expert_matmul", "ep_expert_swiglu",
           "ep_swiglu_grad", "ep_expert_wgrad", "ep_few_workspace_bytes", "ep_moe_few",
           "ep_rms_norm", "ep_norm_workspace_bytes", "ep_rms_norm_grad", "ep_route", "ep_route_grad",
           "ep_few_w4_workspace_bytes", "ep_moe_few_w4",
           "ep_clear_errors", "ep_check_errors", "ep_check_sticky_errors",
           "ep_status_string")

_lib = None


def lib() -> ctypes.CDLL:
    """Load libep.so (raises if it is missing: build it first)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -m combine_get_layout_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    sp = ctypes.POINTER(ep_shape)
    lp = ctypes.POINTER(ep_layout)
    i64, u32, sz = ctypes.c_int64, ctypes.c_uint32, ctypes.c_size_t
    L.ep_workspace_bytes.argtypes = [sp]
    L.ep_workspace_bytes.restype = sz
    L.ep_record_bytes.argtypes = [sp, ctypes.c_int]
    L.ep_record_bytes.restype = i64
    L.ep_chunked_record_bytes.argtypes = [sp, ctypes.c_int]
    L.ep_chunked_record_bytes.restype = i64
    L.ep_get_layout.argtypes = [sp, _P, lp, _P, sz, _P]
    L.ep_get_layout_noalloc.argtypes = [sp, _P, lp, _P, _P]
    L.ep_dispatch.argtypes = [sp, lp, ctypes.POINTER(ep_tokens), ctypes.POINTER(ep_recv), _P, sz, _P]
    L.ep_dispatch_expand.argtypes = L.ep_dispatch.argtypes
    L.ep_hierarchical_dispatch.argtypes = [sp, lp, ctypes.POINTER(ep_tokens), u32, ctypes.c_int,
                                           _P, i64, _P, i64, _P, sz, _P]
    L.ep_hierarchical_dispatch_fused.argtypes = [sp, lp, ctypes.POINTER(ep_tokens), u32, _P, i64, _P,
                                                 i64, ctypes.POINTER(ep_fused_opts), _P, sz, _P]
    L.ep_combine.argtypes = [sp, lp, _P, i64, i64, ctypes.c_int, u32, _P, _P, _P, sz, _P]
    L.ep_combine_expand.argtypes = L.ep_combine.argtypes
    L.ep_partial_row_bytes.argtypes = [sp]
    L.ep_partial_row_bytes.restype = i64
    L.ep_combine_two_level.argtypes = [sp, lp, _P, _P, i64, i64, ctypes.c_int, u32, _P, _P, i64,
                                       ctypes.c_int, _P, _P, sz, _P]
    xp = ctypes.POINTER(ep_sources)
    L.ep_source_workspace_bytes.argtypes = [sp, ctypes.c_int32]
    L.ep_source_workspace_bytes.restype = sz
    L.ep_source_layout.argtypes = [sp, _P, xp, _P, sz, _P]
    L.ep_source_dispatch.argtypes = [sp, xp, ctypes.POINTER(ep_tokens), u32, _P, _P, sz, _P]
    L.ep_copy_epilogue.argtypes = [sp, xp, _P, u32, ctypes.c_int, ctypes.POINTER(ep_recv), _P, sz,
                                   _P]
    L.ep_source_dispatch_fused.argtypes = [sp, xp, ctypes.POINTER(ep_tokens), u32, _P,
                                           ctypes.POINTER(ep_recv), _P, sz, _P]
    i32, ci = ctypes.c_int32, ctypes.c_int
    L.ep_expert_matmul.argtypes = [sp, lp, _P, i64, i32, _P, i32, ci, _P, _P, sz, _P]
    L.ep_expert_swiglu.argtypes = [sp, lp, _P, i64, _P, i32, _P, _P, _P, _P, sz, _P]
    L.ep_swiglu_grad.argtypes = [sp, lp, i32, _P, _P, _P, i64, _P, _P, _P, _P, _P, sz, _P]
    L.ep_expert_wgrad.argtypes = [sp, lp, _P, i64, i32, ctypes.POINTER(ep_rows), i32, _P, ci, _P, sz, _P]
    L.ep_few_workspace_bytes.argtypes = [sp, i32]
    L.ep_few_workspace_bytes.restype = sz
    L.ep_moe_few.argtypes = [sp, ctypes.POINTER(ep_tokens), ctypes.POINTER(ep_experts), _P, _P, sz, _P]
    f32, rp = ctypes.c_float, ctypes.POINTER(ep_router)
    L.ep_rms_norm.argtypes = [sp, _P, _P, ci, _P, f32, ctypes.POINTER(ep_norm_out), _P]
    L.ep_norm_workspace_bytes.argtypes = [sp]
    L.ep_norm_workspace_bytes.restype = sz
    L.ep_rms_norm_grad.argtypes = [sp, _P, ci, _P, _P, _P, _P, _P, _P, _P, _P, sz, _P]
    L.ep_route.argtypes = [sp, _P, rp, _P, _P, _P, sz, _P]
    L.ep_route_grad.argtypes = [sp, _P, rp, _P, _P, _P, ci, _P, sz, _P]
    L.ep_few_w4_workspace_bytes.argtypes = [sp, i32]
    L.ep_few_w4_workspace_bytes.restype = sz
    L.ep_moe_few_w4.argtypes = [sp, ctypes.POINTER(ep_tokens), ctypes.POINTER(ep_experts_w4), _P, _P, sz, _P]
    L.ep_clear_errors.argtypes = [_P, _P]
    L.ep_check_errors.argtypes = [_P, _P, ctypes.POINTER(u32)]
    L.ep_check_sticky_errors.argtypes = [_P, _P, ctypes.POINTER(u32)]
    L.ep_status_string.argtypes = [ctypes.c_int]
    L.ep_status_string.restype = ctypes.c_char_p
    for f in ("ep_get_layout", "ep_get_layout_noalloc", "ep_dispatch", "ep_dispatch_expand",
              "ep_hierarchical_dispatch", "ep_hierarchical_dispatch_fused",
              "ep_combine", "ep_combine_expand", "ep_combine_two_level", "ep_source_layout",
              "ep_source_dispatch", "ep_copy_epilogue", "ep_source_dispatch_fused",
              "ep_expert_matmul", "ep_expert_swiglu", "ep_swiglu_grad", "ep_expert_wgrad",
              "ep_moe_few", "ep_rms_norm", "ep_rms_norm_grad", "ep_route", "ep_route_grad",
              "ep_moe_few_w4", "ep_clear_errors",
              "ep_check_errors",
              "ep_check_sticky_errors"):
        getattr(L, f).restype = ctypes.c_int
    _lib = L
    return L


def _ptr(t, name="tensor", nbytes=0, device=None):
    """Device address of a tensor argument (None passes through as NULL).

    A tensor must live on the GPU (on `device` where one is given), be contiguous
    and hold at least `nbytes` bytes (the size the C ABI reads or writes for the
    given shape); anything else raises before a kernel can touch memory it does
    not own. A plain int is taken as a device address the caller vouches for."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if device is None:
        if not t.is_cuda:
            raise ValueError(f"{name}: must be a GPU tensor")
    else:
        on = t.get_device()
        if on < 0:
            raise ValueError(f"{name}: must be a GPU tensor")
        if on != device:
            raise ValueError(f"{name}: on device {on}, the workspace on device {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{name}: {have} bytes, the call needs {nbytes}")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        # The handle of torch.cuda.current_stream(), without making its object (2.4 us of the
        # 16 of a small call); _cuda_getDevice runs torch's own initialisation and its checks.
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _stream_on(stream, device):
    """The handle of a stream that runs on `device`, where the call's tensors are: a
    kernel would fault on another device's memory. No stream or the NULL stream
    run on the current device; a stream given as a bare handle is the caller's to
    match."""
    if stream is None:
        runs = torch._C._cuda_getDevice()  # runs torch's own initialisation and its checks
        handle = torch._C._cuda_getCurrentRawStream(runs)
    else:
        handle = _stream(stream)
        if handle and isinstance(stream, int):
            return handle
        runs = stream.device_index if handle else torch._C._cuda_getDevice()
    if runs != device:
        raise ValueError(f"workspace: on device {device}, the call's stream on device {runs}")
    return handle


def _check(rc: int, what: str):
    if rc != EP_OK:
        raise RuntimeError(f"{what}: {lib().ep_status_string(rc).decode()} (status {rc})")


def make_shape(T, H, K, E, R, G=1) -> ep_shape:
    return ep_shape(int(T), int(H), int(K), int(E), int(R), int(G))


def _ws(ws):
    return _ptr(ws, "workspace"), ws.numel() * ws.element_size()


_LAYOUT_BYTES = dict(
    tokens_per_expert=lambda s: 4 * s.E, tokens_per_rank=lambda s: 4 * s.R,
    tokens_per_group=lambda s: 4 * s.G, expert_offsets=lambda s: 4 * (s.E + 1),
    rank_offsets=lambda s: 4 * (s.R + 1), group_offsets=lambda s: 4 * (s.G + 1),
    is_token_in_rank=lambda s: s.T * s.R, is_token_in_group=lambda s: s.T * s.G,
    slot=lambda s: 4 * s.T * s.K, group_slot=lambda s: 4 * s.T * s.K,
    expert_slot=lambda s: 4 * s.T * s.K)


def _layout_struct(shape: ep_shape, layout: dict, device=None) -> ep_layout:
    L = ep_layout()
    for n in LAYOUT_FIELDS:
        t = layout.get(n)
        if t is not None:
            setattr(L, n, _ptr(t, n, _LAYOUT_BYTES[n](shape), device))
    return L


def _seg_of(tokens: dict) -> int:
    return ((EP_SEG_BF16 if tokens.get("x") is not None else 0) |
            (EP_SEG_FP8 if tokens.get("x_fp8") is not None else 0) |
            (EP_SEG_SCALES if tokens.get("x_scales") is not None else 0))


def _tokens_struct(shape: ep_shape, tokens: dict, device=None) -> ep_tokens:
    T, H, K = shape.T, shape.H, shape.K
    need = dict(x=2 * T * H, x_fp8=T * H, x_scales=4 * T * (H // 128), topk_idx=8 * T * K,
                topk_weights=4 * T * K)
    return ep_tokens(*[_ptr(tokens.get(n), n, need[n], device) for n in ("x", "x_fp8", "x_scales",
                                                                          "topk_idx", "topk_weights")])


def _recv_struct(shape: ep_shape, recv: dict, capacity: int) -> ep_recv:
    H, K, cap = shape.H, shape.K, max(int(capacity), 0)
    need = dict(x=2 * cap * H, x_fp8=cap * H, x_scales=4 * cap * (H // 128), src_idx=4 * cap,
                topk_idx=4 * cap * K, topk_weights=4 * cap * K)
    return ep_recv(*[_ptr(recv.get(n), "recv " + n, need[n]) for n in ("x", "x_fp8", "x_scales",
                                                                        "src_idx", "topk_idx",
                                                                        "topk_weights")],
                   int(capacity))


def ep_workspace_bytes(shape: ep_shape) -> int:
    return int(lib().ep_workspace_bytes(ctypes.byref(shape)))


def ep_record_bytes(shape: ep_shape, seg_flags: int) -> int:
    return int(lib().ep_record_bytes(ctypes.byref(shape), int(seg_flags)))


def ep_chunked_record_bytes(shape: ep_shape, seg_flags: int) -> int:
    return int(lib().ep_chunked_record_bytes(ctypes.byref(shape), int(seg_flags)))


def ep_get_layout(shape, topk_idx, layout: dict, ws, stream=None):
    L = _layout_struct(shape, layout)
    _check(lib().ep_get_layout(ctypes.byref(shape), _ptr(topk_idx, "topk_idx", 8 * shape.T * shape.K),
                               ctypes.byref(L), *_ws(ws), _stream(stream)), "ep_get_layout")


def ep_get_layout_noalloc(shape, topk_idx, layout: dict, errors, stream=None):
    """errors: a GPU tensor of at least 8 bytes (two u32 error words), e.g. a
    workspace."""
    L = _layout_struct(shape, layout)
    _check(lib().ep_get_layout_noalloc(ctypes.byref(shape),
                                       _ptr(topk_idx, "topk_idx", 8 * shape.T * shape.K),
                                       ctypes.byref(L), _ptr(errors, "errors", 8), _stream(stream)),
           "ep_get_layout_noalloc")


def ep_dispatch(shape, layout: dict, tokens: dict, recv: dict, capacity: int, ws, stream=None):
    L = _layout_struct(shape, layout)
    tk = _tokens_struct(shape, tokens)
    rv = _recv_struct(shape, recv, capacity)
    _check(lib().ep_dispatch(ctypes.byref(shape), ctypes.byref(L), ctypes.byref(tk),
                             ctypes.byref(rv), *_ws(ws), _stream(stream)), "ep_dispatch")


def ep_dispatch_expand(shape, layout: dict, tokens: dict, recv: dict, capacity: int, ws, stream=None):
    L = _layout_struct(shape, layout)
    tk = _tokens_struct(shape, tokens)
    rv = _recv_struct(shape, recv, capacity)
    _check(lib().ep_dispatch_expand(ctypes.byref(shape), ctypes.byref(L), ctypes.byref(tk),
                                    ctypes.byref(rv), *_ws(ws), _stream(stream)), "ep_dispatch_expand")


def ep_hierarchical_dispatch(shape, layout: dict, tokens: dict, epoch: int, steps: int, group_buf,
                             group_cap: int, peer_buf, peer_cap: int, ws, stream=None):
    L = _layout_struct(shape, layout)
    tk = _tokens_struct(shape, tokens)
    stride = max(ep_chunked_record_bytes(shape, _seg_of(tokens) or EP_SEG_BF16), 0)
    _check(lib().ep_hierarchical_dispatch(ctypes.byref(shape), ctypes.byref(L), ctypes.byref(tk),
                                          int(epoch), int(steps),
                                          _ptr(group_buf, "group_buf", max(int(group_cap), 0) * stride),
                                          int(group_cap),
                                          _ptr(peer_buf, "peer_buf", max(int(peer_cap), 0) * stride),
                                          int(peer_cap), *_ws(ws), _stream(stream)),
           "ep_hierarchical_dispatch")


def ep_hierarchical_dispatch_fused(shape, layout: dict, tokens: dict, epoch: int, group_buf,
                                   group_cap: int, peer_buf, peer_cap: int, ws, tile: int = 0,
                                   timeout_us: int = 0, withhold: int | None = None, ring: int = 0,
                                   stream=None):
    L = _layout_struct(shape, layout)
    tk = _tokens_struct(shape, tokens)
    stride = max(ep_chunked_record_bytes(shape, _seg_of(tokens) or EP_SEG_BF16), 0)
    opts = ep_fused_opts(int(tile), int(timeout_us), EP_FUSED_WITHHOLD if withhold is not None else 0,
                         int(withhold) if withhold is not None else 0, int(ring))
    _check(lib().ep_hierarchical_dispatch_fused(
        ctypes.byref(shape), ctypes.byref(L), ctypes.byref(tk), int(epoch),
        _ptr(group_buf, "group_buf", max(int(group_cap), 0) * stride), int(group_cap),
        _ptr(peer_buf, "peer_buf", max(int(peer_cap), 0) * stride), int(peer_cap),
        ctypes.byref(opts), *_ws(ws), _stream(stream)), "ep_hierarchical_dispatch_fused")


def _combine_args(shape, y, y_rows, y_row_stride, topk_weights, out):
    T, H, K = shape.T, shape.H, shape.K
    return (_ptr(y, "y", max(int(y_rows), 0) * max(int(y_row_stride), 0)), int(y_rows),
            int(y_row_stride), _ptr(topk_weights, "topk_weights", 4 * T * K),
            _ptr(out, "out", 2 * T * H))


def ep_combine(shape, layout: dict, y, y_rows: int, y_row_stride: int, y_format: int, epoch: int,
               topk_weights, out, ws, stream=None):
    L = _layout_struct(shape, layout)
    yp, yr, ys, wp, op = _combine_args(shape, y, y_rows, y_row_stride, topk_weights, out)
    _check(lib().ep_combine(ctypes.byref(shape), ctypes.byref(L), yp, yr, ys, int(y_format),
                            int(epoch), wp, op, *_ws(ws), _stream(stream)), "ep_combine")


def ep_combine_expand(shape, layout: dict, y, y_rows: int, y_row_stride: int, y_format: int,
                      epoch: int, topk_weights, out, ws, stream=None):
    L = _layout_struct(shape, layout)
    yp, yr, ys, wp, op = _combine_args(shape, y, y_rows, y_row_stride, topk_weights, out)
    _check(lib().ep_combine_expand(ctypes.byref(shape), ctypes.byref(L), yp, yr, ys, int(y_format),
                                   int(epoch), wp, op, *_ws(ws), _stream(stream)), "ep_combine_expand")


def ep_partial_row_bytes(shape: ep_shape) -> int:
    return int(lib().ep_partial_row_bytes(ctypes.byref(shape)))


def ep_combine_two_level(shape, layout: dict, topk_idx, y, y_rows: int, y_row_stride: int,
                         y_format: int, epoch: int, topk_weights, group_buf, group_cap: int,
                         steps: int, out, ws, stream=None):
    L = _layout_struct(shape, layout)
    yp, yr, ys, wp, op = _combine_args(shape, y, y_rows, y_row_stride, topk_weights, out)
    pstride = max(ep_partial_row_bytes(shape), 0)
    _check(lib().ep_combine_two_level(ctypes.byref(shape), ctypes.byref(L),
                                      _ptr(topk_idx, "topk_idx", 8 * shape.T * shape.K), yp, yr, ys,
                                      int(y_format), int(epoch), wp,
                                      _ptr(group_buf, "group_buf", max(int(group_cap), 0) * pstride),
                                      int(group_cap), int(steps), op, *_ws(ws), _stream(stream)),
           "ep_combine_two_level")


def _sources_struct(shape: ep_shape, sources: dict) -> ep_sources:
    S, R = int(sources["S"]), shape.R
    return ep_sources(S, int(sources["capacity"]),
                      _ptr(sources.get("counts"), "counts", 4 * S * R),
                      _ptr(sources.get("recv_offsets"), "recv_offsets", 4 * (R * S + 1)),
                      _ptr(sources.get("src_slot"), "src_slot", 4 * shape.T * shape.K))


def ep_source_workspace_bytes(shape: ep_shape, S: int) -> int:
    return int(lib().ep_source_workspace_bytes(ctypes.byref(shape), int(S)))


def _staging_bytes(shape: ep_shape, sources: dict, seg: int) -> int:
    rows = shape.R * int(sources["S"]) * max(int(sources["capacity"]), 0)
    return rows * max(ep_chunked_record_bytes(shape, seg or EP_SEG_BF16), 0)


def ep_source_layout(shape, topk_idx, sources: dict, ws, stream=None):
    X = _sources_struct(shape, sources)
    _check(lib().ep_source_layout(ctypes.byref(shape), _ptr(topk_idx, "topk_idx", 8 * shape.T * shape.K),
                                  ctypes.byref(X), *_ws(ws), _stream(stream)), "ep_source_layout")


def ep_source_dispatch(shape, sources: dict, tokens: dict, epoch: int, staging, ws, stream=None):
    X = _sources_struct(shape, sources)
    tk = _tokens_struct(shape, tokens)
    _check(lib().ep_source_dispatch(ctypes.byref(shape), ctypes.byref(X), ctypes.byref(tk),
                                    int(epoch),
                                    _ptr(staging, "staging", _staging_bytes(shape, sources, _seg_of(tokens))),
                                    *_ws(ws), _stream(stream)), "ep_source_dispatch")


def ep_copy_epilogue(shape, sources: dict, staging, epoch: int, seg_flags: int, recv: dict,
                     capacity: int, ws, stream=None):
    X = _sources_struct(shape, sources)
    rv = _recv_struct(shape, recv, capacity)
    _check(lib().ep_copy_epilogue(ctypes.byref(shape), ctypes.byref(X),
                                  _ptr(staging, "staging", _staging_bytes(shape, sources, int(seg_flags))),
                                  int(epoch), int(seg_flags), ctypes.byref(rv), *_ws(ws),
                                  _stream(stream)), "ep_copy_epilogue")


def ep_source_dispatch_fused(shape, sources: dict, tokens: dict, epoch: int, staging, recv: dict,
                             capacity: int, ws, stream=None):
    """ep_source_dispatch and ep_copy_epilogue in one launch (the record's
    pieces are those of `tokens`)."""
    X = _sources_struct(shape, sources)
    tk = _tokens_struct(shape, tokens)
    rv = _recv_struct(shape, recv, capacity)
    _check(lib().ep_source_dispatch_fused(
        ctypes.byref(shape), ctypes.byref(X), ctypes.byref(tk), int(epoch),
        _ptr(staging, "staging", _staging_bytes(shape, sources, _seg_of(tokens))), ctypes.byref(rv),
        *_ws(ws), _stream(stream)), "ep_source_dispatch_fused")


def ep_expert_matmul(shape, layout: dict, x, rows: int, k_dim: int, w, n_dim: int, w_order: int, y, ws,
                     stream=None):
    dev = ws.get_device()
    L = _layout_struct(shape, layout, dev)
    n = max(int(rows), 0)
    _check(lib().ep_expert_matmul(ctypes.byref(shape), ctypes.byref(L), _ptr(x, "x", 2 * n * k_dim, dev),
                                  int(rows), int(k_dim), _ptr(w, "w", 2 * shape.E * n_dim * k_dim, dev),
                                  int(n_dim), int(w_order), _ptr(y, "y", 2 * n * n_dim, dev), *_ws(ws),
                                  _stream_on(stream, dev)), "ep_expert_matmul")


def ep_expert_swiglu(shape, layout: dict, x, rows: int, w13, F: int, act, gu_fp8, gu_scales, ws,
                     stream=None):
    dev = ws.get_device()
    L = _layout_struct(shape, layout, dev)
    n = max(int(rows), 0)
    _check(lib().ep_expert_swiglu(ctypes.byref(shape), ctypes.byref(L), _ptr(x, "x", 2 * n * shape.H, dev),
                                  int(rows), _ptr(w13, "w13", 4 * shape.E * F * shape.H, dev), int(F),
                                  _ptr(act, "act", 2 * n * F, dev), _ptr(gu_fp8, "gu_fp8", 2 * n * F, dev),
                                  _ptr(gu_scales, "gu_scales", 8 * n * (F // 128), dev), *_ws(ws),
                                  _stream_on(stream, dev)), "ep_expert_swiglu")


def ep_swiglu_grad(shape, layout: dict, F: int, gu_fp8, gu_scales, d_act, rows: int, topk_weights, d_gu,
                   act_w, d_topk_weights, ws, stream=None):
    dev = ws.get_device()
    L = _layout_struct(shape, layout, dev)
    n, lanes = max(int(rows), 0), shape.T * shape.K
    _check(lib().ep_swiglu_grad(ctypes.byref(shape), ctypes.byref(L), int(F),
                                _ptr(gu_fp8, "gu_fp8", 2 * n * F, dev),
                                _ptr(gu_scales, "gu_scales", 8 * n * (F // 128), dev),
                                _ptr(d_act, "d_act", 2 * n * F, dev), int(rows),
                                _ptr(topk_weights, "topk_weights", 4 * lanes, dev),
                                _ptr(d_gu, "d_gu", 4 * n * F, dev), _ptr(act_w, "act_w", 2 * n * F, dev),
                                _ptr(d_topk_weights, "d_topk_weights", 4 * lanes, dev), *_ws(ws),
                                _stream_on(stream, dev)), "ep_swiglu_grad")


def ep_expert_wgrad(shape, layout: dict, dy, rows: int, n_dim: int, x: dict, k_dim: int, dw, dtype: int,
                    ws, stream=None):
    """x: {"x": bf16 rows} or {"x_fp8": e4m3 rows, "x_scales": scales}."""
    dev = ws.get_device()
    L = _layout_struct(shape, layout, dev)
    n = max(int(rows), 0)
    X = ep_rows(_ptr(x.get("x"), "x", 2 * n * k_dim, dev), _ptr(x.get("x_fp8"), "x_fp8", n * k_dim, dev),
                _ptr(x.get("x_scales"), "x_scales", 4 * n * (k_dim // 128), dev))
    size = 4 if int(dtype) == EP_GRAD_F32 else 2
    _check(lib().ep_expert_wgrad(ctypes.byref(shape), ctypes.byref(L), _ptr(dy, "dy", 2 * n * n_dim, dev),
                                 int(rows), int(n_dim), ctypes.byref(X), int(k_dim),
                                 _ptr(dw, "dw", size * shape.E * n_dim * k_dim, dev), int(dtype), *_ws(ws),
                                 _stream_on(stream, dev)), "ep_expert_wgrad")


def ep_few_workspace_bytes(shape: ep_shape, F: int) -> int:
    return int(lib().ep_few_workspace_bytes(ctypes.byref(shape), int(F)))


def ep_moe_few(shape, tokens: dict, experts: dict, out, ws, stream=None):
    """experts: {"F", "w13", "w2"} (bf16) or {"F", "w13_fp8", "w13_scales",
    "w2_fp8", "w2_scales"}."""
    dev = ws.get_device()
    tk = _tokens_struct(shape, tokens, dev)
    E, H, F = shape.E, shape.H, int(experts["F"])
    need = dict(w13=4 * E * F * H, w2=2 * E * H * F, w13_fp8=2 * E * F * H,
                w13_scales=8 * E * F * (H // 128), w2_fp8=E * H * F, w2_scales=4 * E * H * (F // 128))
    X = ep_experts(F, *[_ptr(experts.get(n), n, need[n], dev) for n in need])
    _check(lib().ep_moe_few(ctypes.byref(shape), ctypes.byref(tk), ctypes.byref(X),
                            _ptr(out, "out", 2 * shape.T * H, dev), *_ws(ws), _stream_on(stream, dev)), "ep_moe_few")


def ep_rms_norm(shape, x, residual, stream_type: int, gain, eps: float, out: dict, stream=None):
    """out: any of "h", "y", "y_fp8" with "y_scales", "rstd" (h may be residual)."""
    T, H = shape.T, shape.H
    # No workspace: the call runs where x is.
    dev = x.get_device() if isinstance(x, torch.Tensor) else None
    if dev is not None and dev < 0:
        raise ValueError("x: must be a GPU tensor")
    n = T * H
    wide = 4 * n if int(stream_type) == EP_STREAM_F32 else 2 * n
    get = out.get
    O = ep_norm_out(_ptr(get("h"), "h", wide, dev), _ptr(get("y"), "y", 2 * n, dev), _ptr(get("y_fp8"), "y_fp8", n, dev),
                    _ptr(get("y_scales"), "y_scales", 4 * T * (H // 128), dev), _ptr(get("rstd"), "rstd", 4 * T, dev))
    _check(lib().ep_rms_norm(_byref(shape), _ptr(x, "x", 2 * n, dev), _ptr(residual, "residual", wide, dev),
                             int(stream_type), _ptr(gain, "gain", 2 * H, dev), eps, _byref(O),
                             _stream(stream) if dev is None else _stream_on(stream, dev)), "ep_rms_norm")


def ep_norm_workspace_bytes(shape: ep_shape) -> int:
    return int(lib().ep_norm_workspace_bytes(ctypes.byref(shape)))


def ep_rms_norm_grad(shape, h, stream_type: int, gain, rstd, dy, d_stream, d_h, d_x, d_gain, ws, stream=None):
    dev = ws.get_device()
    T, H = shape.T, shape.H
    n = T * H
    wide = 4 * n if int(stream_type) == EP_STREAM_F32 else 2 * n
    _check(lib().ep_rms_norm_grad(_byref(shape), _ptr(h, "h", wide, dev), int(stream_type),
                                  _ptr(gain, "gain", 2 * H, dev), _ptr(rstd, "rstd", 4 * T, dev),
                                  _ptr(dy, "dy", 2 * n, dev), _ptr(d_stream, "d_stream", wide, dev),
                                  _ptr(d_h, "d_h", wide, dev), _ptr(d_x, "d_x", 2 * n, dev),
                                  _ptr(d_gain, "d_gain", 4 * H, dev), *_ws(ws), _stream_on(stream, dev)),
           "ep_rms_norm_grad")


def _router_struct(shape: ep_shape, router: dict, device) -> ep_router:
    get = router.get
    return ep_router(router["score"], get("top_groups", shape.G), get("group_top", 1), get("normalize", 1),
                     get("scale", 1.0), _ptr(get("bias"), "bias", 4 * shape.E, device))


def ep_route(shape, logits, router: dict, topk_idx, topk_weights, ws, stream=None):
    """router: {"score"} and, where they differ from the defaults, "top_groups" (all), "group_top" (1),
    "normalize" (True), "scale" (1.0), "bias" (None)."""
    dev = ws.get_device()
    R = _router_struct(shape, router, dev)
    T, lanes = shape.T, shape.T * shape.K
    _check(lib().ep_route(_byref(shape), _ptr(logits, "logits", 4 * T * shape.E, dev), _byref(R),
                          _ptr(topk_idx, "topk_idx", 8 * lanes, dev), _ptr(topk_weights, "topk_weights", 4 * lanes, dev),
                          *_ws(ws), _stream_on(stream, dev)), "ep_route")


def ep_route_grad(shape, logits, router: dict, topk_idx, d_topk_weights, d_logits, dtype: int, ws, stream=None):
    """router: as for ep_route."""
    dev = ws.get_device()
    R = _router_struct(shape, router, dev)
    n, lanes = shape.T * shape.E, shape.T * shape.K
    _check(lib().ep_route_grad(_byref(shape), _ptr(logits, "logits", 4 * n, dev), _byref(R),
                               _ptr(topk_idx, "topk_idx", 8 * lanes, dev),
                               _ptr(d_topk_weights, "d_topk_weights", 4 * lanes, dev),
                               _ptr(d_logits, "d_logits", (4 if int(dtype) == EP_GRAD_F32 else 2) * n, dev), int(dtype),
                               *_ws(ws), _stream_on(stream, dev)), "ep_route_grad")


def ep_few_w4_workspace_bytes(shape: ep_shape, F: int) -> int:
    return int(lib().ep_few_w4_workspace_bytes(ctypes.byref(shape), int(F)))


def ep_moe_few_w4(shape, tokens: dict, experts: dict, out, ws, stream=None):
    """experts: {"F", "form" (EP_W4_*), "w13", "w13_scales", "w2", "w2_scales"}."""
    dev = ws.get_device()
    T, H, lanes, F, form = shape.T, shape.H, shape.T * shape.K, int(experts["F"]), int(experts["form"])
    get = tokens.get
    tk = ep_tokens(_ptr(get("x"), "x", 2 * T * H, dev), None, None, _ptr(get("topk_idx"), "topk_idx", 8 * lanes, dev),
                   _ptr(get("topk_weights"), "topk_weights", 4 * lanes, dev))
    n = shape.E * F * H
    scales = n // 64 if form == EP_W4_INT else n // 32  # bytes: two for 128 values, one for 32
    get = experts.get
    X = ep_experts_w4(F, form, _ptr(get("w13"), "w13", n, dev), _ptr(get("w13_scales"), "w13_scales", 2 * scales, dev),
                      _ptr(get("w2"), "w2", n // 2, dev), _ptr(get("w2_scales"), "w2_scales", scales, dev))
    _check(lib().ep_moe_few_w4(_byref(shape), _byref(tk), _byref(X), _ptr(out, "out", 2 * T * H, dev), *_ws(ws),
                               _stream_on(stream, dev)), "ep_moe_few_w4")


def ep_clear_errors(ws, stream=None):
    _check(lib().ep_clear_errors(_ptr(ws, "workspace"), _stream(stream)), "ep_clear_errors")


def _error_bits(fn, name, ws, stream) -> int:
    bits = ctypes.c_uint32(0)
    rc = fn(_ptr(ws, "workspace"), _stream(stream), ctypes.byref(bits))
    if rc != EP_ERR_DEVICE:  # EP_ERR_DEVICE: bits are set, and returned
        _check(rc, name)
    return int(bits.value)


def ep_check_errors(ws, stream=None) -> int:
    """Error bits of the current pass (0 when none; EP_ERR_DEVICE is not
    raised: the bits are the answer)."""
    return _error_bits(lib().ep_check_errors, "ep_check_errors", ws, stream)


def ep_check_sticky_errors(ws, stream=None) -> int:
    """Error bits of every call since the last ep_clear_errors."""
    return _error_bits(lib().ep_check_sticky_errors, "ep_check_sticky_errors", ws, stream)


def ep_status_string(status: int) -> str:
    return lib().ep_status_string(int(status)).decode()


# --------------------------------------------------------------------------
# Allocation helpers (empty tensors of the documented sizes; no compute)
# --------------------------------------------------------------------------

def alloc_workspace(shape: ep_shape, device="cuda") -> torch.Tensor:
    """A zero-filled workspace (both error words start clear)."""
    n = ep_workspace_bytes(shape)
    if n == 0:
        raise RuntimeError("ep_workspace_bytes: unsupported shape")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def alloc_source_workspace(shape: ep_shape, S: int, device="cuda") -> torch.Tensor:
    """A zero-filled several-source workspace."""
    n = ep_source_workspace_bytes(shape, S)
    if n == 0:
        raise RuntimeError("ep_source_workspace_bytes: unsupported shape or source count")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def alloc_few_workspace(shape: ep_shape, F: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace of ep_moe_few."""
    n = ep_few_workspace_bytes(shape, F)
    if n == 0:
        raise RuntimeError("ep_few_workspace_bytes: unsupported shape or inner size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def alloc_norm_workspace(shape: ep_shape, device="cuda") -> torch.Tensor:
    """A zero-filled workspace of ep_rms_norm_grad."""
    n = ep_norm_workspace_bytes(shape)
    if n == 0:
        raise RuntimeError("ep_norm_workspace_bytes: unsupported shape")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def alloc_few_w4_workspace(shape: ep_shape, F: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace of ep_moe_few_w4."""
    n = ep_few_w4_workspace_bytes(shape, F)
    if n == 0:
        raise RuntimeError("ep_few_w4_workspace_bytes: unsupported shape or inner size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def alloc_sources(shape: ep_shape, S: int, capacity: int, device="cuda") -> dict:
    i32 = dict(dtype=torch.int32, device=device)
    return dict(S=int(S), capacity=int(capacity),
                counts=torch.empty((S, shape.R), **i32),
                recv_offsets=torch.empty(shape.R * S + 1, **i32),
                src_slot=torch.empty((shape.T, shape.K), **i32))


def alloc_layout(shape: ep_shape, device="cuda", masks=True, groups=True, expand=False) -> dict:
    i32 = dict(dtype=torch.int32, device=device)
    T, K, E, R, G = shape.T, shape.K, shape.E, shape.R, shape.G
    out = dict(
        tokens_per_expert=torch.empty(E, **i32),
        tokens_per_rank=torch.empty(R, **i32),
        expert_offsets=torch.empty(E + 1, **i32),
        rank_offsets=torch.empty(R + 1, **i32),
        slot=torch.empty((T, K), **i32),
    )
    if masks:
        out["is_token_in_rank"] = torch.empty((T, R), dtype=torch.uint8, device=device)
    if groups:
        out["tokens_per_group"] = torch.empty(G, **i32)
        out["group_offsets"] = torch.empty(G + 1, **i32)
        out["group_slot"] = torch.empty((T, K), **i32)
        if masks:
            out["is_token_in_group"] = torch.empty((T, G), dtype=torch.uint8, device=device)
    if expand:
        out["expert_slot"] = torch.empty((T, K), **i32)
    return out


def alloc_recv(shape: ep_shape, capacity: int, device="cuda", x=True, fp8=False, scales=False,
               meta=True) -> dict:
    H, K = shape.H, shape.K
    out = {}
    if x:
        out["x"] = torch.empty((capacity, H), dtype=torch.uint16, device=device)
    if fp8:
        out["x_fp8"] = torch.empty((capacity, H), dtype=torch.uint8, device=device)
    if scales:
        out["x_scales"] = torch.empty((capacity, H // 128), dtype=torch.float32, device=device)
    if meta:
        out["src_idx"] = torch.empty(capacity, dtype=torch.int32, device=device)
        out["topk_idx"] = torch.empty((capacity, K), dtype=torch.int32, device=device)
        out["topk_weights"] = torch.empty((capacity, K), dtype=torch.float32, device=device)
    return out
