"""ctypes view of libmok.so (include/mok.h).  Argument marshalling only."""
from __future__ import annotations

import ctypes
import importlib.util
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libmok.so")

c_void_p = ctypes.c_void_p
c_size_t = ctypes.c_size_t
c_int64 = ctypes.c_int64
c_int32 = ctypes.c_int32


class MoeDesc(ctypes.Structure):
    _fields_ = [("T", c_int64), ("d", c_int64), ("E", c_int64), ("I", c_int64),
                ("k", c_int32), ("dtype", c_int32), ("mb_tokens", c_int32),
                ("ring_slots", c_int32), ("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class SavedLayout(ctypes.Structure):
    _fields_ = [(n, c_size_t) for n in (
        "status", "topk_idx", "topk_w", "counts", "offsets", "pos", "token_of_row",
        "padded_offsets", "padded_pos", "padded_token", "row_weight", "x_perm", "gate_up",
        "nv_weight_scales", "w_gate_up_t", "w_down_col", "rows_max", "mb_count", "mb_stride", "ring_slots", "ring_slot_bytes", "total")]


class KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", c_int32), ("total_ms", ctypes.c_double)]


class RmsnormDesc(ctypes.Structure):
    _fields_ = [("rows", c_int64), ("d", c_int64), ("ld_x", c_int64), ("ld_res", c_int64),
                ("ld_s", c_int64), ("ld_y", c_int64), ("eps", ctypes.c_float),
                ("x_elem", c_int32), ("s_elem", c_int32), ("weight_elem", c_int32),
                ("accumulate", c_int32), ("reserved", ctypes.c_uint32)]


class BalanceDesc(ctypes.Structure):
    _fields_ = [("T", c_int64), ("ld_logits", c_int64), ("E", c_int32), ("k", c_int32),
                ("balance_coef", ctypes.c_float), ("z_coef", ctypes.c_float)]


class LinearDesc(ctypes.Structure):
    _fields_ = [("M", c_int64), ("N", c_int64), ("K", c_int64), ("ld_x", c_int64),
                ("act", c_int32), ("y_elem", c_int32), ("dx_elem", c_int32),
                ("accumulate", c_int32)]


class DropoutDesc(ctypes.Structure):
    _fields_ = [("rows", c_int64), ("d", c_int64), ("ld_x", c_int64), ("ld_res", c_int64),
                ("ld_y", c_int64), ("p", ctypes.c_double), ("x_elem", c_int32),
                ("y_elem", c_int32), ("site", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class PostPreDesc(ctypes.Structure):
    _fields_ = [("rows", c_int64), ("d", c_int64), ("ld_x", c_int64), ("ld_res", c_int64),
                ("ld_s", c_int64), ("ld_y", c_int64), ("ld_dx", c_int64), ("ld_dr", c_int64),
                ("eps", ctypes.c_float), ("residual_scale", ctypes.c_float),
                ("x_elem", c_int32), ("s_elem", c_int32), ("weight_elem", c_int32),
                ("gate_elem", c_int32), ("gate", c_int32), ("y_elem", c_int32),
                ("dx_elem", c_int32), ("accumulate", c_int32)]


class GroupedDesc(ctypes.Structure):
    _fields_ = [("rows", c_int64), ("N", c_int64), ("K", c_int64), ("E", c_int32),
                ("y_elem", c_int32), ("dx_elem", c_int32), ("accumulate", c_int32),
                ("ld_x", c_int64), ("ld_y", c_int64), ("ld_dx", c_int64)]


# name -> (restype, argtypes)
_SIGS = {
    "mok_moe_workspace_size": (c_int32, [ctypes.POINTER(MoeDesc), ctypes.POINTER(c_size_t),
                                         ctypes.POINTER(c_size_t), ctypes.POINTER(c_size_t)]),
    "mok_moe_saved_layout": (c_int32, [ctypes.POINTER(MoeDesc), ctypes.POINTER(SavedLayout)]),
    "mok_moe_forward": (c_int32, [ctypes.POINTER(MoeDesc), c_void_p, c_void_p, c_void_p, c_void_p,
                                  c_void_p, c_void_p, c_void_p, c_size_t, c_void_p, c_size_t,
                                  c_void_p]),
    "mok_moe_backward": (c_int32, [ctypes.POINTER(MoeDesc), c_void_p, c_void_p, c_void_p, c_void_p,
                                   c_void_p, c_void_p, c_void_p, c_size_t, c_void_p, c_void_p,
                                   c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "mok_moe_stage_workspace_size": (c_int32, [ctypes.POINTER(MoeDesc), ctypes.POINTER(c_size_t)]),
    "mok_moe_route": (c_int32, [ctypes.POINTER(MoeDesc), c_void_p, c_void_p, c_void_p, c_void_p,
                                c_void_p, c_void_p, c_size_t, c_void_p]),
    "mok_moe_dispatch_plan": (c_int32, [ctypes.POINTER(MoeDesc), c_void_p, c_void_p, c_void_p,
                                        c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "mok_moe_dispatch_plan_noalloc": (c_int32, [ctypes.POINTER(MoeDesc), c_void_p, c_void_p,
                                                c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "mok_mx_quantize": (c_int32, [c_void_p, c_int64, c_int64, c_int32, c_void_p, c_void_p,
                                  c_void_p, c_void_p]),
    "mok_gemm_bf16": (c_int32, [c_int64, c_int64, c_int64, c_void_p, c_int32, c_void_p, c_int32,
                                c_void_p, c_void_p, c_size_t, c_void_p]),
    "mok_gemm_mxfp8": (c_int32, [c_int64, c_int64, c_int64, c_void_p, c_void_p, c_void_p,
                                 c_void_p, c_void_p, c_int32, c_void_p, c_size_t, c_void_p]),
    "mok_nvfp4_tensor_scale": (c_int32, [c_void_p, c_int64, c_void_p, c_void_p]),
    "mok_nvfp4_quantize": (c_int32, [c_void_p, c_int64, c_int64, c_void_p, c_void_p, c_void_p,
                                     c_void_p]),
    "mok_nvfp4_quantize_cols": (c_int32, [c_void_p, c_int64, c_int64, c_int64, c_void_p,
                                          c_void_p, c_void_p, c_void_p]),
    "mok_gemm_nvfp4": (c_int32, [c_int64, c_int64, c_int64, c_void_p, c_void_p, c_void_p,
                                 c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                 c_void_p]),
    "mok_add_rmsnorm_forward": (c_int32, [ctypes.POINTER(RmsnormDesc)] + [c_void_p] * 9),
    "mok_add_rmsnorm_backward": (c_int32, [ctypes.POINTER(RmsnormDesc)] + [c_void_p] * 7
                                 + [c_size_t, c_void_p, c_void_p]),
    "mok_add_rmsnorm_workspace_size": (c_int32, [ctypes.POINTER(RmsnormDesc),
                                                 ctypes.POINTER(c_size_t)]),
    "mok_router_balance_forward": (c_int32, [ctypes.POINTER(BalanceDesc)] + [c_void_p] * 9
                                   + [c_size_t, c_void_p, c_void_p]),
    "mok_router_balance_workspace_size": (c_int32, [ctypes.POINTER(BalanceDesc),
                                                    ctypes.POINTER(c_size_t)]),
    "mok_router_balance_backward": (c_int32, [ctypes.POINTER(BalanceDesc)] + [c_void_p] * 8),
    "mok_linear_forward": (c_int32, [ctypes.POINTER(LinearDesc)] + [c_void_p] * 7
                           + [c_size_t, c_void_p, c_void_p]),
    "mok_linear_backward": (c_int32, [ctypes.POINTER(LinearDesc)] + [c_void_p] * 8
                            + [c_size_t, c_void_p, c_void_p]),
    "mok_linear_workspace_size": (c_int32, [ctypes.POINTER(LinearDesc), c_int32,
                                            ctypes.POINTER(c_size_t)]),
    "mok_dropout_forward": (c_int32, [ctypes.POINTER(DropoutDesc)] + [c_void_p] * 5),
    "mok_dropout_backward": (c_int32, [ctypes.POINTER(DropoutDesc)] + [c_void_p] * 4),
    "mok_post_pre_rmsnorm_forward": (c_int32, [ctypes.POINTER(PostPreDesc)] + [c_void_p] * 9),
    "mok_post_pre_rmsnorm_backward": (c_int32, [ctypes.POINTER(PostPreDesc)] + [c_void_p] * 13
                                      + [c_size_t, c_void_p, c_void_p]),
    "mok_post_pre_rmsnorm_workspace_size": (c_int32, [ctypes.POINTER(PostPreDesc),
                                                      ctypes.POINTER(c_size_t)]),
    "mok_grouped_linear_forward": (c_int32, [ctypes.POINTER(GroupedDesc)] + [c_void_p] * 6),
    "mok_grouped_linear_backward": (c_int32, [ctypes.POINTER(GroupedDesc)] + [c_void_p] * 7
                                    + [c_size_t, c_void_p, c_void_p]),
    "mok_grouped_linear_workspace_size": (c_int32, [ctypes.POINTER(GroupedDesc),
                                                    ctypes.POINTER(c_size_t)]),
    "mok_selftest_bounded_wait": (c_int32, [c_void_p, c_size_t, c_void_p]),
    "mok_fill_zero": (c_int32, [c_void_p, c_size_t, c_void_p]),
    "mok_get_device_status": (c_int32, [c_void_p, c_void_p, ctypes.POINTER(c_int32)]),
    "mok_status_string": (ctypes.c_char_p, [c_int32]),
    "mok_last_launch_count": (c_int32, []),
    "mok_profile_enable": (c_int32, [c_int32]),
    "mok_profile_reset": (c_int32, []),
    "mok_profile_collect": (c_int32, [ctypes.POINTER(KernelTime), c_int32, ctypes.POINTER(c_int32)]),
}

_lib = None


def load(path: str | None = None):
    """Loads libmok.so once.  Raises when it has not been built: there is no
    other implementation to fall back to."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with "
                           "`python -m routing_dispatch_grouped_router_gb300.build`")
    lib = ctypes.CDLL(p)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


_block = None


def block():
    """The module of block_binding.cpp (built beside libmok.so, which it calls)."""
    global _block
    if _block is None:
        load()
        from . import build
        path = build.BINDING
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -m routing_dispatch_grouped_router_gb300.build`")
        spec = importlib.util.spec_from_file_location("_block", path)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        _block = m
    return _block


def exported_names():
    return list(_SIGS)


class MokError(RuntimeError):
    def __init__(self, code: int, where: str):
        lib = load()
        super().__init__(f"{where}: {lib.mok_status_string(code).decode()} (code {code})")
        self.code = code


def check(code: int, where: str):
    if code != 0:
        raise MokError(code, where)
