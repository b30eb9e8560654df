"""ctypes binding of libmok (include/mok.h), entry point by entry point.

Argument marshalling only: every step of the layer runs in the HIP kernels of
libmok.so.  Tensor arguments may be torch tensors (their data_ptr() is passed)
or raw integer device addresses.  A non-OK status raises MokError.  If the
library is not built the first call raises; there is no other code path.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmok.so")

MOK_OK, MOK_ERR_INVALID_ARG, MOK_ERR_UNSUPPORTED, MOK_ERR_WORKSPACE, MOK_ERR_HIP, MOK_ERR_DEVICE = range(6)
MOK_PREC_F32, MOK_PREC_BF16, MOK_PREC_MXFP8, MOK_PREC_MXFP4 = range(4)
MOK_DTYPE_F32, MOK_DTYPE_BF16, MOK_DTYPE_F16 = range(3)
MOK_FLAG_SAVE_FOR_BACKWARD = 0x1
MOK_FLAG_SIGMOID_GATES = 0x2
MOK_FLAG_RENORM_GATES = 0x4
MOK_FLAG_SEPARATE_ROUTE_SORT = 0x8
MOK_FLAG_TILED_GEMMS = 0x10
MOK_FLAG_STREAM_GEMMS = 0x20
MOK_FLAG_MXFP8_WGRAD = 0x40
STAGES = ["router", "sort", "dispatch", "gemm_up", "gemm_down", "combine", "bwd_gate", "gemm_dh", "gemm_dx",
          "reduce_dx", "gemm_dw2", "regather", "gemm_dw13"]
MOK_NUM_STAGES = len(STAGES)
PRECISIONS = {"f32": MOK_PREC_F32, "bf16": MOK_PREC_BF16, "mxfp8": MOK_PREC_MXFP8, "mxfp4": MOK_PREC_MXFP4}


class mok_moe_config(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32), ("ffn", ctypes.c_int32),
                ("expert_begin", ctypes.c_int32), ("expert_end", ctypes.c_int32),
                ("precision", ctypes.c_int32), ("minibatch_rows", ctypes.c_int32),
                ("ring_bytes", ctypes.c_int64), ("flags", ctypes.c_uint32), ("mover_cus", ctypes.c_int32),
                ("stage_events", ctypes.c_void_p)]


class mok_saved_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("lse", "topk_idx", "topk_gate", "offsets", "row_of_pair", "pair_of_row", "A", "B", "H", "Y",
                 "total")]


class mok_workspace_layout(ctypes.Structure):
    _fields_ = [("status", ctypes.c_size_t), ("xp", ctypes.c_size_t), ("xp_scale", ctypes.c_size_t),
                ("xp_rows", ctypes.c_int64), ("hq", ctypes.c_size_t), ("hq_scale", ctypes.c_size_t),
                ("dy", ctypes.c_size_t), ("dab", ctypes.c_size_t),
                ("dxp", ctypes.c_size_t), ("wq", ctypes.c_size_t), ("wq_scale", ctypes.c_size_t),
                ("k_pad", ctypes.c_int64), ("total", ctypes.c_size_t)]


class mok_int4_weights(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p)]


class mok_int4_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("rows", "x_rows", "k", "E", "expert_begin", "expert_end", "N", "K", "group", "dtype")]


MOK_CHECK_LOGITS, MOK_CHECK_INDEX = 0x1, 0x2


class MokError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {mok_status_string(status)}")


_lib = None
_P = ctypes.c_void_p


def lib() -> ctypes.CDLL:
    """The loaded libmok.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with mixture_experts_layer_34_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        L.mok_status_string.restype = ctypes.c_char_p
        L.mok_status_string.argtypes = [ctypes.c_int]
        L.mok_version.restype = ctypes.c_int32
        L.mok_moe_workspace_query.restype = ctypes.c_int
        L.mok_moe_workspace_query.argtypes = [ctypes.POINTER(mok_moe_config), ctypes.c_int32,
                                              ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]
        L.mok_moe_saved_layout.restype = ctypes.c_int
        L.mok_moe_saved_layout.argtypes = [ctypes.POINTER(mok_moe_config), ctypes.c_int32,
                                           ctypes.POINTER(mok_saved_layout)]
        L.mok_moe_workspace_layout.restype = ctypes.c_int
        L.mok_moe_workspace_layout.argtypes = [ctypes.POINTER(mok_moe_config), ctypes.c_int32,
                                               ctypes.POINTER(mok_workspace_layout)]
        L.mok_moe_forward.restype = ctypes.c_int
        L.mok_moe_forward.argtypes = [_P, _P, _P, _P, _P, ctypes.c_int32, ctypes.POINTER(mok_moe_config), _P,
                                      _P, _P, _P, _P, _P, _P, _P, _P]
        L.mok_moe_forward_router.restype = ctypes.c_int
        L.mok_moe_forward_router.argtypes = [_P, _P, _P, _P, _P, ctypes.c_int32, ctypes.POINTER(mok_moe_config), _P,
                                             _P, _P, _P, _P, _P, _P, _P, _P, _P]
        L.mok_moe_forward_noalloc.restype = ctypes.c_int
        L.mok_moe_forward_noalloc.argtypes = [_P, _P, _P, _P, _P, ctypes.c_int32, ctypes.POINTER(mok_moe_config), _P,
                                              _P, _P, _P, _P, _P, _P]
        L.mok_moe_backward.restype = ctypes.c_int
        L.mok_moe_backward.argtypes = [_P, _P, _P, _P, _P, _P, ctypes.c_int32, ctypes.POINTER(mok_moe_config), _P,
                                       _P, _P, _P, _P, _P, _P, _P, _P]
        L.mok_quantize_mxfp8.restype = ctypes.c_int
        L.mok_quantize_mxfp8.argtypes = [_P, ctypes.c_int64, ctypes.c_int64, _P, _P, _P]
        L.mok_quantize_mxfp4.restype = ctypes.c_int
        L.mok_quantize_mxfp4.argtypes = [_P, ctypes.c_int64, ctypes.c_int64, _P, _P, _P]
        L.mok_moe_backward_mxfp8.restype = ctypes.c_int
        L.mok_moe_backward_mxfp8.argtypes = [_P, _P, _P, ctypes.c_int32, ctypes.POINTER(mok_moe_config), _P, _P, _P,
                                             _P, _P, _P, _P, _P, _P, _P, _P]
        L.mok_quantize_mxfp8_backward_weights.restype = ctypes.c_int
        L.mok_quantize_mxfp8_backward_weights.argtypes = [_P, _P, _P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                                          _P, _P, _P]
        L.mok_router_logits.restype = ctypes.c_int
        L.mok_router_logits.argtypes = [_P, _P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P, _P]
        L.mok_router_logits_backward.restype = ctypes.c_int
        L.mok_router_logits_backward.argtypes = [_P, _P, _P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P, _P,
                                                 _P]
        i32, i64 = ctypes.c_int32, ctypes.c_int64
        L.mok_sort_pairs_workspace_query.restype = ctypes.c_int
        L.mok_sort_pairs_workspace_query.argtypes = [i32, i32, i32, ctypes.POINTER(ctypes.c_size_t)]
        L.mok_sort_pairs.restype = ctypes.c_int
        L.mok_sort_pairs.argtypes = [_P, i32, i32, i32, i32, i32, _P, _P, _P, _P, _P, _P]
        for f in (L.mok_permute_rows, L.mok_unpermute_rows):
            f.restype = ctypes.c_int
            f.argtypes = [_P, _P, _P, i32, i32, i32, ctypes.c_int, i64, _P, _P]
        for f in (L.mok_permute_rows_backward, L.mok_unpermute_rows_backward):
            f.restype = ctypes.c_int
            f.argtypes = [_P, _P, _P, _P, i32, i32, i32, ctypes.c_int, i64, _P, _P, _P]
        L.mok_expert_matvec_int4.restype = ctypes.c_int
        L.mok_expert_matvec_int4.argtypes = [_P, _P, _P, ctypes.POINTER(mok_int4_weights),
                                             ctypes.POINTER(mok_int4_weights), ctypes.POINTER(mok_int4_config), _P,
                                             _P]
        L.mok_quantize_int4.restype = ctypes.c_int
        L.mok_quantize_int4.argtypes = [_P, i64, i64, i32, ctypes.c_int, _P, _P, _P, _P]
        _lib = L
    return _lib


def _ptr(v):
    if v is None:
        return None
    if isinstance(v, int):
        return v
    return v.data_ptr()


def _int32(where: str, sizes: int):
    """Refuses sizes (or-ed together) of which one is negative or past an int32:
    ctypes would cut it to its low 32 bits, and the library check what is left."""
    if sizes >> 31:
        raise MokError(MOK_ERR_INVALID_ARG, where)


def _check(status: int, where: str):
    if status != MOK_OK:
        raise MokError(status, where)


def make_config(T, d, E, ffn, expert_begin=0, expert_end=None, precision="bf16", minibatch_rows=0,
                ring_bytes=0, flags=0, mover_cus=0) -> mok_moe_config:
    prec = PRECISIONS[precision] if isinstance(precision, str) else int(precision)
    return mok_moe_config(T, d, E, ffn, expert_begin, E if expert_end is None else expert_end, prec,
                          minibatch_rows, ring_bytes, flags, mover_cus)


def mok_status_string(status: int) -> str:
    return lib().mok_status_string(int(status)).decode()


def mok_version() -> int:
    return int(lib().mok_version())


def mok_moe_workspace_query(cfg: mok_moe_config, k: int):
    ws, sv = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().mok_moe_workspace_query(ctypes.byref(cfg), k, ctypes.byref(ws), ctypes.byref(sv)),
           "mok_moe_workspace_query")
    return ws.value, sv.value


def mok_moe_saved_layout(cfg: mok_moe_config, k: int) -> dict:
    out = mok_saved_layout()
    _check(lib().mok_moe_saved_layout(ctypes.byref(cfg), k, ctypes.byref(out)), "mok_moe_saved_layout")
    return {n: getattr(out, n) for n, _ in mok_saved_layout._fields_}


def mok_moe_workspace_layout(cfg: mok_moe_config, k: int) -> dict:
    out = mok_workspace_layout()
    _check(lib().mok_moe_workspace_layout(ctypes.byref(cfg), k, ctypes.byref(out)), "mok_moe_workspace_layout")
    return {n: getattr(out, n) for n, _ in mok_workspace_layout._fields_}


def mok_moe_forward(x, router_logits, W1, W3, W2, k, cfg, w_scales, out, topk_idx, topk_gate, expert_counts,
                    expert_offsets, saved, workspace, stream=0):
    _check(lib().mok_moe_forward(_ptr(x), _ptr(router_logits), _ptr(W1), _ptr(W3), _ptr(W2), k, ctypes.byref(cfg),
                                 _ptr(w_scales), _ptr(out), _ptr(topk_idx), _ptr(topk_gate), _ptr(expert_counts),
                                 _ptr(expert_offsets), _ptr(saved), _ptr(workspace), stream or None),
           "mok_moe_forward")


def mok_moe_forward_router(x, Wr, W1, W3, W2, k, cfg, w_scales, router_logits, out, topk_idx, topk_gate,
                           expert_counts, expert_offsets, saved, workspace, stream=0):
    _check(lib().mok_moe_forward_router(_ptr(x), _ptr(Wr), _ptr(W1), _ptr(W3), _ptr(W2), k, ctypes.byref(cfg),
                                        _ptr(w_scales), _ptr(router_logits), _ptr(out), _ptr(topk_idx),
                                        _ptr(topk_gate), _ptr(expert_counts), _ptr(expert_offsets), _ptr(saved),
                                        _ptr(workspace), stream or None), "mok_moe_forward_router")


def mok_moe_forward_noalloc(x, router_logits, W1, W3, W2, k, cfg, out, topk_idx, topk_gate, expert_counts,
                            expert_offsets, saved, stream=0):
    _check(lib().mok_moe_forward_noalloc(_ptr(x), _ptr(router_logits), _ptr(W1), _ptr(W3), _ptr(W2), k,
                                         ctypes.byref(cfg), _ptr(out), _ptr(topk_idx), _ptr(topk_gate),
                                         _ptr(expert_counts), _ptr(expert_offsets), _ptr(saved), stream or None),
           "mok_moe_forward_noalloc")


def mok_moe_backward(dout, x, router_logits, W1, W3, W2, k, cfg, saved, dx, dW1, dW3, dW2, dgate, drouter_logits,
                     workspace, stream=0):
    _check(lib().mok_moe_backward(_ptr(dout), _ptr(x), _ptr(router_logits), _ptr(W1), _ptr(W3), _ptr(W2), k,
                                  ctypes.byref(cfg), _ptr(saved), _ptr(dx), _ptr(dW1), _ptr(dW3), _ptr(dW2),
                                  _ptr(dgate), _ptr(drouter_logits), _ptr(workspace), stream or None),
           "mok_moe_backward")


def mok_quantize_mxfp8(src_bf16, rows, K, dst_e4m3, dst_e8m0, stream=0):
    _check(lib().mok_quantize_mxfp8(_ptr(src_bf16), rows, K, _ptr(dst_e4m3), _ptr(dst_e8m0), stream or None),
           "mok_quantize_mxfp8")


def mok_quantize_mxfp4(src_bf16, rows, K, dst_e2m1, dst_e8m0, stream=0):
    _check(lib().mok_quantize_mxfp4(_ptr(src_bf16), rows, K, _ptr(dst_e2m1), _ptr(dst_e8m0), stream or None),
           "mok_quantize_mxfp4")


def mok_moe_backward_mxfp8(dout, x, router_logits, k, cfg, wt_e4m3, wt_e8m0, saved, dx, dW1, dW3, dW2, dgate,
                           drouter_logits, workspace, stream=0):
    _check(lib().mok_moe_backward_mxfp8(_ptr(dout), _ptr(x), _ptr(router_logits), k, ctypes.byref(cfg),
                                        _ptr(wt_e4m3), _ptr(wt_e8m0), _ptr(saved), _ptr(dx), _ptr(dW1), _ptr(dW3),
                                        _ptr(dW2), _ptr(dgate), _ptr(drouter_logits), _ptr(workspace),
                                        stream or None), "mok_moe_backward_mxfp8")


def mok_quantize_mxfp8_backward_weights(W1, W3, W2, E_loc, d, F, wt_e4m3, wt_e8m0, stream=0):
    _check(lib().mok_quantize_mxfp8_backward_weights(_ptr(W1), _ptr(W3), _ptr(W2), E_loc, d, F, _ptr(wt_e4m3),
                                                     _ptr(wt_e8m0), stream or None),
           "mok_quantize_mxfp8_backward_weights")


def mok_router_logits(x, Wr, T, d, E, logits, stream=0):
    _check(lib().mok_router_logits(_ptr(x), _ptr(Wr), T, d, E, _ptr(logits), stream or None), "mok_router_logits")


def mok_router_logits_backward(x, Wr, dlogits, T, d, E, dx, dWr, stream=0):
    _check(lib().mok_router_logits_backward(_ptr(x), _ptr(Wr), _ptr(dlogits), T, d, E, _ptr(dx), _ptr(dWr),
                                            stream or None), "mok_router_logits_backward")


def mok_sort_pairs_workspace_query(T, k, E) -> int:
    _int32("mok_sort_pairs_workspace_query", T | k | E)
    n = ctypes.c_size_t()
    _check(lib().mok_sort_pairs_workspace_query(T, k, E, ctypes.byref(n)), "mok_sort_pairs_workspace_query")
    return n.value


def mok_sort_pairs(topk_idx, T, k, E, expert_begin, expert_end, expert_counts, expert_offsets, row_of_pair,
                   pair_of_row, workspace, stream=0):
    _int32("mok_sort_pairs", T | k | E | expert_begin | expert_end)
    _check(lib().mok_sort_pairs(_ptr(topk_idx), T, k, E, expert_begin, expert_end, _ptr(expert_counts),
                                _ptr(expert_offsets), _ptr(row_of_pair), _ptr(pair_of_row), _ptr(workspace),
                                stream or None), "mok_sort_pairs")


def mok_permute_rows(x, gate, row_of_pair, T, k, d, dtype, rows, xp, stream=0):
    _int32("mok_permute_rows", T | k | d)
    _check(lib().mok_permute_rows(_ptr(x), _ptr(gate), _ptr(row_of_pair), T, k, d, dtype, rows, _ptr(xp),
                                  stream or None), "mok_permute_rows")


def mok_permute_rows_backward(dxp, x, gate, row_of_pair, T, k, d, dtype, rows, dx, dgate, stream=0):
    _int32("mok_permute_rows_backward", T | k | d)
    _check(lib().mok_permute_rows_backward(_ptr(dxp), _ptr(x), _ptr(gate), _ptr(row_of_pair), T, k, d, dtype, rows,
                                           _ptr(dx), _ptr(dgate), stream or None), "mok_permute_rows_backward")


def mok_unpermute_rows(y, gate, row_of_pair, T, k, d, dtype, rows, out, stream=0):
    _int32("mok_unpermute_rows", T | k | d)
    _check(lib().mok_unpermute_rows(_ptr(y), _ptr(gate), _ptr(row_of_pair), T, k, d, dtype, rows, _ptr(out),
                                    stream or None), "mok_unpermute_rows")


def mok_unpermute_rows_backward(dout, y, gate, row_of_pair, T, k, d, dtype, rows, dy, dgate, stream=0):
    _int32("mok_unpermute_rows_backward", T | k | d)
    _check(lib().mok_unpermute_rows_backward(_ptr(dout), _ptr(y), _ptr(gate), _ptr(row_of_pair), T, k, d, dtype, rows,
                                             _ptr(dy), _ptr(dgate), stream or None), "mok_unpermute_rows_backward")


def int4_weights(codes, scales, zeros) -> mok_int4_weights:
    return mok_int4_weights(_ptr(codes), _ptr(scales), _ptr(zeros))


def int4_config(rows, x_rows, k, E, expert_begin, expert_end, N, K, group, dtype) -> mok_int4_config:
    _int32("mok_int4_config", rows | x_rows | k | E | expert_begin | expert_end | N | K | group | dtype)
    return mok_int4_config(rows, x_rows, k, E, expert_begin, expert_end, N, K, group, dtype)


def mok_expert_matvec_int4(x, pair_of_row, expert_offsets, w: mok_int4_weights, w_up: mok_int4_weights | None,
                           cfg: mok_int4_config, out, stream=0):
    _check(lib().mok_expert_matvec_int4(_ptr(x), _ptr(pair_of_row), _ptr(expert_offsets), ctypes.byref(w),
                                        None if w_up is None else ctypes.byref(w_up), ctypes.byref(cfg), _ptr(out),
                                        stream or None), "mok_expert_matvec_int4")


def mok_quantize_int4(src, rows, K, group, dtype, codes, scales, zeros, stream=0):
    _int32("mok_quantize_int4", group)
    _check(lib().mok_quantize_int4(_ptr(src), rows, K, group, dtype, _ptr(codes), _ptr(scales), _ptr(zeros),
                                   stream or None), "mok_quantize_int4")
