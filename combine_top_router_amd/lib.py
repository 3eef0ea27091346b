"""ctypes binding of libmoe.so: the C ABI of include/moe.h, same names, argument
marshalling only.  Pointers are passed as Python ints (device addresses), streams as
ints (a hipStream_t, 0 = the null stream).  A failing call raises MoeError."""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "MOE_OK", "MOE_EINVAL", "MOE_EUNSUPPORTED", "MOE_EWORKSPACE", "MOE_EHIP",
    "MOE_F32", "MOE_BF16", "MOE_BWD_SAME", "MOE_BWD_MXFP8", "MOE_FWD_SAME", "MOE_FWD_MXFP8",
    "MOE_NORM_LAYER", "MOE_NORM_RMS",
    "MOE_SCORE_SOFTMAX", "MOE_SCORE_SIGMOID", "MOE_ACT_NONE", "MOE_ACT_RELU", "MOE_ACT_SILU", "MOE_ACT_GELU",
    "MOE_STATE_F32", "MOE_STATE_8BIT", "MOE_ADAMW_CLOCK_BYTES",
    "MoeShape", "MoeNormShape", "MoeOrthShape", "MoeGateShape", "MoeLinearShape", "MoeAdamwTensor", "MoeAdamwParams",
    "MoeError", "load", "lib_path", "EXPORTS",
    "moe_abi_version", "moe_last_error", "moe_workspace_bytes", "moe_route_topk",
    "moe_dispatch", "moe_dispatch_noscratch", "moe_fwd", "moe_combine", "moe_bwd", "moe_route_topk_bwd",
    "moe_mx_quantize", "moe_mx_quantize_cols", "moe_timing_enable", "moe_timing_read",
    "moe_router_fwd", "moe_router_bwd",
    "moe_balance_scratch_bytes", "moe_balance_fwd", "moe_balance_bwd",
    "moe_norm_scratch_bytes", "moe_norm_fwd", "moe_norm_bwd",
    "moe_orth_scratch_bytes", "moe_orthogonalize",
    "moe_gate_scratch_bytes", "moe_gate_fwd", "moe_gate_bwd", "moe_gate_update_bias",
    "moe_linear_scratch_bytes", "moe_linear_fwd_scratch_bytes", "moe_linear_fwd", "moe_linear_bwd", "moe_adamw",
]

MOE_OK, MOE_EINVAL, MOE_EUNSUPPORTED, MOE_EWORKSPACE, MOE_EHIP = 0, -1, -2, -3, -4
MOE_F32, MOE_BF16 = 0, 1
MOE_BWD_SAME, MOE_BWD_MXFP8 = 0, 1
MOE_FWD_SAME, MOE_FWD_MXFP8 = 0, 1
MOE_NORM_LAYER, MOE_NORM_RMS = 0, 1
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_ACT_NONE, MOE_ACT_RELU, MOE_ACT_SILU, MOE_ACT_GELU = 0, 1, 2, 3
MOE_STATE_F32, MOE_STATE_8BIT = 0, 1
MOE_ADAMW_CLOCK_BYTES = 32

_HERE = os.path.dirname(os.path.abspath(__file__))


def lib_path() -> str:
    return os.path.join(_HERE, "libmoe.so")


class MoeShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "H", "I", "E", "k", "e_begin", "e_local", "dtype", "bwd", "renorm", "fwd", "recompute",
                 "row_tile")]

    def __repr__(self):
        return "MoeShape(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class MoeNormShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "dtype", "kind")] + [("eps", ctypes.c_float)]


class MoeOrthShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n", "rows", "cols", "dtype", "steps")]


class MoeGateShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "E", "k", "score", "groups", "topk_groups", "group_top", "renorm")] + [("scale", ctypes.c_float)]


class MoeLinearShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "K", "N", "dtype", "act")]


class MoeAdamwTensor(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("p", "g", "master", "m", "v", "m_scale", "v_scale")]
                + [(n, ctypes.c_int64) for n in ("n", "at")] + [(n, ctypes.c_int32) for n in ("p_dtype", "g_dtype")])


class MoeAdamwParams(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")]
                + [("step", ctypes.c_int64), ("seed", ctypes.c_uint64), ("state", ctypes.c_int32),
                   ("stochastic", ctypes.c_int32)])


class MoeError(RuntimeError):
    def __init__(self, code: int, func: str, msg: str):
        super().__init__(f"{func} failed with status {code}: {msg}")
        self.code = code


_P = ctypes.c_void_p
_S = ctypes.POINTER(MoeShape)
_NS = ctypes.POINTER(MoeNormShape)
_OS = ctypes.POINTER(MoeOrthShape)
_GS = ctypes.POINTER(MoeGateShape)
_LS = ctypes.POINTER(MoeLinearShape)
_SZ = ctypes.POINTER(ctypes.c_size_t)
_F = ctypes.c_float
_SIG = {
    "moe_abi_version": (ctypes.c_int, []),
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_workspace_bytes": (ctypes.c_int, [_S, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]),
    "moe_route_topk": (ctypes.c_int, [_S, _P, _P, _P, _P]),
    "moe_dispatch": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_dispatch_noscratch": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_fwd": (ctypes.c_int, [_S] + [_P] * 12),
    "moe_combine": (ctypes.c_int, [_S, _P, _P, _P, _P]),
    "moe_bwd": (ctypes.c_int, [_S] + [_P] * 18),
    "moe_route_topk_bwd": (ctypes.c_int, [_S, _P, _P, _P, _P, _P, _P]),
    "moe_mx_quantize": (ctypes.c_int, [_P, ctypes.c_int64, ctypes.c_int32, _P, _P, _P]),
    "moe_mx_quantize_cols": (ctypes.c_int, [_P, ctypes.c_int32, _P, ctypes.c_int32, ctypes.c_int64, _P, _P, _P, _P,
                                            _P, _P]),
    "moe_router_fwd": (ctypes.c_int, [_S] + [_P] * 7),
    "moe_router_bwd": (ctypes.c_int, [_S] + [_P] * 8),
    "moe_balance_scratch_bytes": (ctypes.c_int, [_S, _SZ]),
    "moe_balance_fwd": (ctypes.c_int, [_S, _P, _P, _P, _F] + [_P] * 5),
    "moe_balance_bwd": (ctypes.c_int, [_S, _P, _P, _P, _F] + [_P] * 4),
    "moe_norm_scratch_bytes": (ctypes.c_int, [_NS, _SZ]),
    "moe_norm_fwd": (ctypes.c_int, [_NS] + [_P] * 9),
    "moe_norm_bwd": (ctypes.c_int, [_NS] + [_P] * 12),
    "moe_orth_scratch_bytes": (ctypes.c_int, [_OS, _SZ]),
    "moe_orthogonalize": (ctypes.c_int, [_OS, _P, _P, _F, _P, _P]),
    "moe_gate_scratch_bytes": (ctypes.c_int, [_GS, _SZ]),
    "moe_gate_fwd": (ctypes.c_int, [_GS] + [_P] * 8),
    "moe_gate_bwd": (ctypes.c_int, [_GS] + [_P] * 5),
    "moe_gate_update_bias": (ctypes.c_int, [_GS, _P, _P, _F, _P, _P]),
    "moe_linear_scratch_bytes": (ctypes.c_int, [_LS, _SZ]),
    "moe_linear_fwd_scratch_bytes": (ctypes.c_int, [_LS, _SZ]),
    "moe_linear_fwd": (ctypes.c_int, [_LS] + [_P] * 8),
    "moe_linear_bwd": (ctypes.c_int, [_LS] + [_P] * 10),
    "moe_adamw": (ctypes.c_int, [ctypes.POINTER(MoeAdamwParams), ctypes.POINTER(MoeAdamwTensor), ctypes.c_int32]
                  + [_P] * 4),
    "moe_timing_enable": (ctypes.c_int, [ctypes.c_int]),
    "moe_timing_read": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(ctypes.c_char_p),
                                       ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int)]),
}
EXPORTS = tuple(_SIG)

_lib = None


def load():
    """Load libmoe.so from the package directory; raise if it has not been built."""
    global _lib
    if _lib is None:
        path = lib_path()
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it with `python -m combine_top_router_amd.build`")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIG.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(rc: int, func: str):
    if rc != MOE_OK:
        raise MoeError(rc, func, moe_last_error())


def moe_abi_version() -> int:
    return load().moe_abi_version()


def moe_last_error() -> str:
    return load().moe_last_error().decode()


def moe_workspace_bytes(shape: MoeShape):
    saved = ctypes.c_size_t(0)
    scratch = ctypes.c_size_t(0)
    _check(load().moe_workspace_bytes(ctypes.byref(shape), ctypes.byref(saved), ctypes.byref(scratch)),
           "moe_workspace_bytes")
    return saved.value, scratch.value


def moe_route_topk(shape, logits, topk_idx, topk_w, stream=0):
    _check(load().moe_route_topk(ctypes.byref(shape), logits, topk_idx, topk_w, stream), "moe_route_topk")


def moe_dispatch(shape, topk_idx, x, counts, offsets, row_src, row_of, xp, scratch, stream=0):
    _check(load().moe_dispatch(ctypes.byref(shape), topk_idx, x, counts, offsets, row_src, row_of, xp,
                               scratch, stream), "moe_dispatch")


def moe_dispatch_noscratch(shape, topk_idx, x, counts, offsets, row_src, row_of, xp, stream=0):
    _check(load().moe_dispatch_noscratch(ctypes.byref(shape), topk_idx, x, counts, offsets, row_src, row_of, xp,
                                         stream), "moe_dispatch_noscratch")


def moe_fwd(shape, x, xp, offsets, row_src, topk_w, w_gate, w_up, w_down, yp, saved, scratch, stream=0):
    _check(load().moe_fwd(ctypes.byref(shape), x, xp, offsets, row_src, topk_w, w_gate, w_up, w_down, yp,
                          saved, scratch, stream), "moe_fwd")


def moe_combine(shape, yp, row_of, y, stream=0):
    _check(load().moe_combine(ctypes.byref(shape), yp, row_of, y, stream), "moe_combine")


def moe_bwd(shape, dy, x, xp, offsets, row_src, row_of, topk_w, w_gate, w_up, w_down, saved, dx,
            dw_gate, dw_up, dw_down, d_topk_w, scratch, stream=0):
    _check(load().moe_bwd(ctypes.byref(shape), dy, x, xp, offsets, row_src, row_of, topk_w, w_gate, w_up,
                          w_down, saved, dx, dw_gate, dw_up, dw_down, d_topk_w, scratch, stream), "moe_bwd")


def moe_route_topk_bwd(shape, logits, topk_idx, topk_w, d_topk_w, d_logits, stream=0):
    _check(load().moe_route_topk_bwd(ctypes.byref(shape), logits, topk_idx, topk_w, d_topk_w, d_logits, stream),
           "moe_route_topk_bwd")


def moe_mx_quantize(x, rows, K, codes, scales, stream=0):
    _check(load().moe_mx_quantize(x, rows, K, codes, scales, stream), "moe_mx_quantize")


def moe_mx_quantize_cols(x, N, offsets, groups, Rp, poff, codes, scales, row_codes=0, row_scales=0, stream=0):
    _check(load().moe_mx_quantize_cols(x, N, offsets, groups, Rp, poff, codes, scales, row_codes, row_scales,
                                       stream), "moe_mx_quantize_cols")


def moe_router_fwd(shape, x, w_r, logits, topk_idx, topk_w, scratch, stream=0):
    _check(load().moe_router_fwd(ctypes.byref(shape), x, w_r, logits, topk_idx, topk_w, scratch, stream),
           "moe_router_fwd")


def moe_router_bwd(shape, x, w_r, d_logits, dx_in, dx, dw_r, scratch, stream=0):
    _check(load().moe_router_bwd(ctypes.byref(shape), x, w_r, d_logits, dx_in, dx, dw_r, scratch, stream),
           "moe_router_bwd")


def _scratch_bytes(func, shape):
    n = ctypes.c_size_t(0)
    _check(getattr(load(), func)(ctypes.byref(shape), ctypes.byref(n)), func)
    return n.value


def moe_balance_scratch_bytes(shape: MoeShape) -> int:
    return _scratch_bytes("moe_balance_scratch_bytes", shape)


def moe_balance_fwd(shape, logits, topk_idx, mask, coef, loss, counts, prob, scratch, stream=0):
    _check(load().moe_balance_fwd(ctypes.byref(shape), logits, topk_idx, mask, coef, loss, counts, prob, scratch,
                                  stream), "moe_balance_fwd")


def moe_balance_bwd(shape, logits, counts, mask, coef, d_loss, d_logits_in, d_logits, stream=0):
    _check(load().moe_balance_bwd(ctypes.byref(shape), logits, counts, mask, coef, d_loss, d_logits_in, d_logits,
                                  stream), "moe_balance_bwd")


def moe_norm_scratch_bytes(shape: MoeNormShape) -> int:
    return _scratch_bytes("moe_norm_scratch_bytes", shape)


def moe_norm_fwd(shape, x, res, w, b, sum, y, mean, rstd, stream=0):
    _check(load().moe_norm_fwd(ctypes.byref(shape), x, res, w, b, sum, y, mean, rstd, stream), "moe_norm_fwd")


def moe_norm_bwd(shape, dy, s, res, w, mean, rstd, ds_in, dx, dw, db, scratch, stream=0):
    _check(load().moe_norm_bwd(ctypes.byref(shape), dy, s, res, w, mean, rstd, ds_in, dx, dw, db, scratch, stream),
           "moe_norm_bwd")


def moe_orth_scratch_bytes(shape: MoeOrthShape) -> int:
    return _scratch_bytes("moe_orth_scratch_bytes", shape)


def moe_orthogonalize(shape, g, o, scale, scratch, stream=0):
    _check(load().moe_orthogonalize(ctypes.byref(shape), g, o, scale, scratch, stream), "moe_orthogonalize")


def moe_gate_scratch_bytes(shape: MoeGateShape) -> int:
    return _scratch_bytes("moe_gate_scratch_bytes", shape)


def moe_gate_fwd(shape, logits, bias, mask, topk_idx, topk_w, counts, scratch, stream=0):
    _check(load().moe_gate_fwd(ctypes.byref(shape), logits, bias, mask, topk_idx, topk_w, counts, scratch, stream),
           "moe_gate_fwd")


def moe_gate_bwd(shape, logits, topk_idx, d_topk_w, d_logits, stream=0):
    _check(load().moe_gate_bwd(ctypes.byref(shape), logits, topk_idx, d_topk_w, d_logits, stream), "moe_gate_bwd")


def moe_gate_update_bias(shape, counts, bias, rate, bias_out, stream=0):
    _check(load().moe_gate_update_bias(ctypes.byref(shape), counts, bias, rate, bias_out, stream),
           "moe_gate_update_bias")


def moe_linear_scratch_bytes(shape: MoeLinearShape) -> int:
    return _scratch_bytes("moe_linear_scratch_bytes", shape)


def moe_linear_fwd_scratch_bytes(shape: MoeLinearShape) -> int:
    return _scratch_bytes("moe_linear_fwd_scratch_bytes", shape)


def moe_linear_fwd(shape, x, w, b, res, z, y, scratch, stream=0):
    _check(load().moe_linear_fwd(ctypes.byref(shape), x, w, b, res, z, y, scratch, stream), "moe_linear_fwd")


def moe_linear_bwd(shape, dy, x, w, z, dx_in, dx, dw, db, scratch, stream=0):
    _check(load().moe_linear_bwd(ctypes.byref(shape), dy, x, w, z, dx_in, dx, dw, db, scratch, stream),
           "moe_linear_bwd")


def moe_adamw(params, tensors, count, lr, grad_scale, clock, stream=0):
    """`tensors`: a ctypes array of MoeAdamwTensor, of which the first `count` are taken."""
    _check(load().moe_adamw(ctypes.byref(params), tensors, count, lr, grad_scale, clock, stream), "moe_adamw")


def moe_timing_enable(on: bool = True):
    _check(load().moe_timing_enable(1 if on else 0), "moe_timing_enable")


def moe_timing_read(capacity: int = 256):
    """[(kernel name, milliseconds)] of the kernels launched since the last read."""
    names = (ctypes.c_char_p * capacity)()
    ms = (ctypes.c_float * capacity)()
    n = ctypes.c_int(0)
    _check(load().moe_timing_read(capacity, names, ms, ctypes.byref(n)), "moe_timing_read")
    return [(names[i].decode(), float(ms[i])) for i in range(min(n.value, capacity))]
