"""ctypes binding of libmoe.so (include/moe.h). Argument marshalling only.

Every step of the layer runs in the HIP library. The functions here take torch tensors (or raw
integer addresses) and hand their device pointers to the C entry points of the same names. If
the library is missing, loading it raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import re

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "moe.h")

MODES = {"fp32": 0, "bf16": 1, "mxfp8": 2, "fp8_bwd": 3, "fp8": 4}
TYPES = {"fp32": 0, "bf16": 1, "int8": 2}
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED_SHAPE",
          3: "MOE_ERR_UNSUPPORTED_MODE", 4: "MOE_ERR_WORKSPACE_TOO_SMALL", 5: "MOE_ERR_HIP"}


class Desc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("F", ctypes.c_int32),
                ("E_total", ctypes.c_int32), ("E_local", ctypes.c_int32),
                ("expert_offset", ctypes.c_int32), ("topk", ctypes.c_int32), ("mode", ctypes.c_int32),
                ("recompute", ctypes.c_int32)]

    @classmethod
    def make(cls, T, H, F, E_total, topk, mode="bf16", E_local=None, expert_offset=0, recompute=False):
        m = MODES[mode] if isinstance(mode, str) else int(mode)
        return cls(T, H, F, E_total, E_total - expert_offset if E_local is None else E_local,
                   expert_offset, topk, m, int(recompute))


class SavedOffsets(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("idx", "weight", "counts", "offsets", "perm", "pair_pos", "qoff", "qcols",
                                               "hwt", "hwt_scales", "wdt", "wdt_scales", "wgut", "wgut_scales")]


class Tensor(ctypes.Structure):
    """moe_tensor: one of the tensors of a gradient norm."""
    _fields_ = [("data", ctypes.c_void_p), ("n", ctypes.c_int64), ("type", ctypes.c_int32)]


class MoEError(RuntimeError):
    def __init__(self, status, detail):
        self.status = status
        self.code = STATUS.get(status, str(status))
        super().__init__(f"{self.code}: {detail}")


_lib = None
_P = ctypes.c_void_p
_D = ctypes.POINTER(Desc)


def header_functions():
    """Names of the functions declared in include/moe.h."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\**\s*(moe_\w+)\s*\(", text, re.M)))


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m mixture_experts_layer_32_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        st = ctypes.c_int
        L.moe_query_sizes.argtypes = [_D, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t),
                                      ctypes.POINTER(ctypes.c_size_t)]
        L.moe_route.argtypes = [_D, _P, _P, _P, ctypes.c_size_t, _P]
        L.moe_route_static.argtypes = [_D, _P, _P, _P]
        L.moe_fwd.argtypes = [_D, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.moe_fwd_router.argtypes = [_D, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.moe_bwd.argtypes = [_D, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.moe_saved_layout.argtypes = [_D, ctypes.POINTER(SavedOffsets)]
        L.moe_status_string.argtypes = [st]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_last_error.argtypes = []
        L.moe_last_error.restype = ctypes.c_char_p
        L.moe_version.restype = ctypes.c_char_p
        L.moe_mx_quantize.argtypes = [_P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, _P, _P, _P]
        L.moe_fp8_block_quantize.argtypes = [_P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, _P, _P, _P, _P, _P]
        L.moe_query_router_sizes.argtypes = [_D, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]
        L.moe_router_fwd.argtypes = [_D, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.moe_router_bwd.argtypes = [_D, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.moe_query_few_sizes.argtypes = [_D, ctypes.POINTER(ctypes.c_size_t)]
        L.moe_fwd_few.argtypes = [_D, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        i64 = ctypes.c_int64
        L.moe_int8_quantize.argtypes = [_P, ctypes.c_int, i64, i64, _P, _P, _P]
        L.moe_int8_matmul.argtypes = [_P, _P, _P, _P, i64, i64, i64, ctypes.c_int, _P, _P, ctypes.c_int, _P]
        L.moe_query_int8_sizes.argtypes = [_D, ctypes.POINTER(ctypes.c_size_t)]
        L.moe_fwd_int8.argtypes = [_D, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        size, ci = ctypes.POINTER(ctypes.c_size_t), ctypes.c_int
        L.moe_query_sort_sizes.argtypes = [i64, ci, size]
        L.moe_sort_pairs.argtypes = [_P, i64, ci, ci, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.moe_dispatch.argtypes = [_P, ci, i64, ci, i64, _P, _P, i64, _P]
        L.moe_combine.argtypes = [_P, ci, i64, _P, _P, i64, ci, i64, _P, ci, _P]
        L.moe_combine_bwd.argtypes = [_P, ci, _P, ci, i64, _P, _P, _P, i64, ci, i64, ci, _P, _P, _P, _P]
        L.moe_query_int4_sizes.argtypes = [ci, i64, i64, ci, size, size]
        L.moe_int4_quantize.argtypes = [_P, ci, ci, i64, i64, ci, _P, _P, _P]
        L.moe_int4_pack.argtypes = [_P, _P, ci, i64, i64, ci, _P, _P, _P]
        L.moe_int4_matmul.argtypes = [_P, _P, _P, i64, i64, i64, ci, ci, _P, _P, ci, _P]
        tensors = ctypes.POINTER(Tensor)
        L.moe_query_norm_sizes.argtypes = [tensors, ci, size]
        L.moe_grad_norm.argtypes = [tensors, ci, _P, _P, ctypes.c_size_t, _P]
        L.moe_grad_clip.argtypes = [tensors, tensors, ci, _P, ctypes.c_float, _P]
        L.moe_clip_grad_norm.argtypes = [tensors, tensors, ci, ctypes.c_float, _P, _P, ctypes.c_size_t, _P]
        L.moe_profile_enable.argtypes = [ctypes.c_int]
        L.moe_profile_kernel.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_char_p),
                                         ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_double)]
        for n in ("moe_query_sizes", "moe_route", "moe_route_static", "moe_fwd", "moe_fwd_router", "moe_bwd", "moe_saved_layout", "moe_mx_quantize",
                  "moe_fp8_block_quantize", "moe_query_few_sizes", "moe_fwd_few", "moe_int8_quantize",
                  "moe_int8_matmul", "moe_query_int8_sizes", "moe_fwd_int8",
                  "moe_query_sort_sizes", "moe_sort_pairs", "moe_dispatch", "moe_combine", "moe_combine_bwd",
                  "moe_query_int4_sizes", "moe_int4_quantize", "moe_int4_pack", "moe_int4_matmul",
                  "moe_query_norm_sizes", "moe_grad_norm", "moe_grad_clip", "moe_clip_grad_norm",
                  "moe_query_router_sizes", "moe_router_fwd", "moe_router_bwd", "moe_profile_enable",
                  "moe_profile_disable", "moe_profile_collect", "moe_profile_kernel"):
            getattr(L, n).restype = st
        _lib = L
    return _lib


def _check(status):
    if status:
        raise MoEError(status, lib().moe_last_error().decode())


def ptr(t):
    """Device (or host) address of a tensor, an int address, or None (NULL)."""
    return t if t is None or isinstance(t, int) else t.data_ptr()


def _stream(stream):
    if type(stream) is int:
        return stream
    if stream is None:
        import torch
        # the current stream's handle without the Stream object, whose making takes 2.7 us a call
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


def version():
    return lib().moe_version().decode()


def query_sizes(desc: Desc):
    f, b, s = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().moe_query_sizes(ctypes.byref(desc), ctypes.byref(f), ctypes.byref(b), ctypes.byref(s)))
    return f.value, b.value, s.value


def saved_layout(desc: Desc) -> dict:
    o = SavedOffsets()
    _check(lib().moe_saved_layout(ctypes.byref(desc), ctypes.byref(o)))
    return {n: getattr(o, n) for n, _ in SavedOffsets._fields_}


def moe_route(desc, logits, saved, ws, ws_bytes, stream=None):
    _check(lib().moe_route(ctypes.byref(desc), ptr(logits), ptr(saved), ptr(ws), ws_bytes, _stream(stream)))


def moe_route_static(desc, logits, saved, stream=None):
    _check(lib().moe_route_static(ctypes.byref(desc), ptr(logits), ptr(saved), _stream(stream)))


def moe_fwd(desc, x, logits, w_gate, w_up, w_down, y, saved, ws, ws_bytes, stream=None):
    _check(lib().moe_fwd(ctypes.byref(desc), ptr(x), ptr(logits), ptr(w_gate), ptr(w_up), ptr(w_down), ptr(y),
                         ptr(saved), ptr(ws), ws_bytes, _stream(stream)))


def moe_fwd_router(desc, x, w_router, logits, w_gate, w_up, w_down, y, saved, ws, ws_bytes, stream=None):
    _check(lib().moe_fwd_router(ctypes.byref(desc), ptr(x), ptr(w_router), ptr(logits), ptr(w_gate), ptr(w_up),
                                ptr(w_down), ptr(y), ptr(saved), ptr(ws), ws_bytes, _stream(stream)))


def moe_bwd(desc, dy, x, w_gate, w_up, w_down, saved, dx, dlogits, dw_gate, dw_up, dw_down, ws, ws_bytes,
            stream=None):
    _check(lib().moe_bwd(ctypes.byref(desc), ptr(dy), ptr(x), ptr(w_gate), ptr(w_up), ptr(w_down), ptr(saved),
                         ptr(dx), ptr(dlogits), ptr(dw_gate), ptr(dw_up), ptr(dw_down), ptr(ws), ws_bytes,
                         _stream(stream)))


def query_router_sizes(desc: Desc):
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().moe_query_router_sizes(ctypes.byref(desc), ctypes.byref(f), ctypes.byref(b)))
    return f.value, b.value


def moe_router_fwd(desc, x, w_router, logits, ws, ws_bytes, stream=None):
    _check(lib().moe_router_fwd(ctypes.byref(desc), ptr(x), ptr(w_router), ptr(logits), ptr(ws), ws_bytes,
                                _stream(stream)))


def moe_router_bwd(desc, x, w_router, dlogits, dx, dw_router, ws, ws_bytes, stream=None):
    _check(lib().moe_router_bwd(ctypes.byref(desc), ptr(x), ptr(w_router), ptr(dlogits), ptr(dx), ptr(dw_router),
                                ptr(ws), ws_bytes, _stream(stream)))


def query_few_sizes(desc: Desc):
    n = ctypes.c_size_t()
    _check(lib().moe_query_few_sizes(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def moe_fwd_few(desc, x, w_router, logits, w_gate, w_up, w_down, y, ws, ws_bytes, stream=None):
    _check(lib().moe_fwd_few(ctypes.byref(desc), ptr(x), ptr(w_router), ptr(logits), ptr(w_gate), ptr(w_up),
                             ptr(w_down), ptr(y), ptr(ws), ws_bytes, _stream(stream)))


def moe_int8_quantize(x, type, rows, cols, q, scales, stream=None):
    _check(lib().moe_int8_quantize(ptr(x), type, rows, cols, ptr(q), ptr(scales), _stream(stream)))


def moe_int8_matmul(x, x_scales, w, w_scales, M, N, K, G, offsets, y, type, stream=None):
    _check(lib().moe_int8_matmul(ptr(x), ptr(x_scales), ptr(w), ptr(w_scales), M, N, K, G, ptr(offsets), ptr(y), type,
                                 _stream(stream)))


def query_int8_sizes(desc: Desc):
    n = ctypes.c_size_t()
    _check(lib().moe_query_int8_sizes(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def moe_fwd_int8(desc, x, w_router, logits, w_gate, s_gate, w_up, s_up, w_down, s_down, y, ws, ws_bytes, stream=None):
    _check(lib().moe_fwd_int8(ctypes.byref(desc), ptr(x), ptr(w_router), ptr(logits), ptr(w_gate), ptr(s_gate),
                              ptr(w_up), ptr(s_up), ptr(w_down), ptr(s_down), ptr(y), ptr(ws), ws_bytes,
                              _stream(stream)))


def query_sort_sizes(pairs, E_local):
    n = ctypes.c_size_t()
    _check(lib().moe_query_sort_sizes(pairs, E_local, ctypes.byref(n)))
    return n.value


def moe_sort_pairs(idx, pairs, E_local, expert_offset, offsets, perm, pair_pos, ws, ws_bytes, stream=None):
    _check(lib().moe_sort_pairs(ptr(idx), pairs, E_local, expert_offset, ptr(offsets), ptr(perm), ptr(pair_pos), ptr(ws),
                                ws_bytes, _stream(stream)))


def moe_dispatch(x, type, T, topk, H, pair_pos, rows, nrows, stream=None):
    _check(lib().moe_dispatch(ptr(x), type, T, topk, H, ptr(pair_pos), ptr(rows), nrows, _stream(stream)))


def moe_combine(rows, rows_type, nrows, pair_pos, weight, T, topk, H, y, type, stream=None):
    _check(lib().moe_combine(ptr(rows), rows_type, nrows, ptr(pair_pos), ptr(weight), T, topk, H, ptr(y), type,
                             _stream(stream)))


def moe_combine_bwd(dy, type, rows, rows_type, nrows, pair_pos, weight, idx, T, topk, H, E_total, drows, dweight,
                    dlogits, stream=None):
    _check(lib().moe_combine_bwd(ptr(dy), type, ptr(rows), rows_type, nrows, ptr(pair_pos), ptr(weight), ptr(idx), T,
                                 topk, H, E_total, ptr(drows), ptr(dweight), ptr(dlogits), _stream(stream)))


def query_int4_sizes(G, N, K, group):
    q, s = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().moe_query_int4_sizes(G, N, K, group, ctypes.byref(q), ctypes.byref(s)))
    return q.value, s.value


def moe_int4_quantize(x, type, G, N, K, group, q, scales, stream=None):
    _check(lib().moe_int4_quantize(ptr(x), type, G, N, K, group, ptr(q), ptr(scales), _stream(stream)))


def moe_int4_pack(values, in_scales, G, N, K, group, q, scales, stream=None):
    _check(lib().moe_int4_pack(ptr(values), ptr(in_scales), G, N, K, group, ptr(q), ptr(scales), _stream(stream)))


def moe_int4_matmul(x, q, scales, M, N, K, group, G, offsets, y, type, stream=None):
    _check(lib().moe_int4_matmul(ptr(x), ptr(q), ptr(scales), M, N, K, group, G, ptr(offsets), ptr(y), type,
                                 _stream(stream)))


def query_norm_sizes(tensors, count):
    n = ctypes.c_size_t()
    _check(lib().moe_query_norm_sizes(tensors, count, ctypes.byref(n)))
    return n.value


def moe_grad_norm(tensors, count, norm, ws, ws_bytes, stream=None):
    _check(lib().moe_grad_norm(tensors, count, ptr(norm), ptr(ws), ws_bytes, _stream(stream)))


def moe_grad_clip(tensors, out, count, norm, max_norm, stream=None):
    _check(lib().moe_grad_clip(tensors, out, count, ptr(norm), max_norm, _stream(stream)))


def moe_clip_grad_norm(tensors, out, count, max_norm, norm, ws, ws_bytes, stream=None):
    _check(lib().moe_clip_grad_norm(tensors, out, count, max_norm, ptr(norm), ptr(ws), ws_bytes, _stream(stream)))


def moe_mx_quantize(x, rows, cols, axis, q, scales, stream=None):
    _check(lib().moe_mx_quantize(ptr(x), rows, cols, axis, ptr(q), ptr(scales), _stream(stream)))


def moe_fp8_block_quantize(x, rows, cols, weight, q, scales, qt=None, scales_t=None, stream=None):
    _check(lib().moe_fp8_block_quantize(ptr(x), rows, cols, int(weight), ptr(q), ptr(scales), ptr(qt), ptr(scales_t),
                                        _stream(stream)))


def profile_enable(max_launches=4096):
    _check(lib().moe_profile_enable(max_launches))


def profile_disable():
    _check(lib().moe_profile_disable())


def profile_collect() -> dict:
    """{kernel name: (launches, total ms)} of the launches recorded since profile_enable()."""
    L = lib()
    _check(L.moe_profile_collect())
    out = {}
    i = 0
    while True:
        name, n, ms = ctypes.c_char_p(), ctypes.c_int(), ctypes.c_double()
        if L.moe_profile_kernel(i, ctypes.byref(name), ctypes.byref(n), ctypes.byref(ms)) != 0:
            break
        out[name.value.decode()] = (n.value, ms.value)
        i += 1
    return out
