"""ctypes loader of libmoe_b200.so (the C ABI declared in include/moe.h).

There is no fallback: if the shared library is missing or cannot be loaded this module
raises, so a product call can never silently run anything but the CUDA kernels.
"""
from __future__ import annotations

import ctypes
import os
import sys
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libmoe_b200.so")
BINDING_PATH = os.path.join(_PKG, "_lib", "moe_binding.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "moe.h")

MOE_OK = 0
MOE_ERR_ARG = -1
MOE_ERR_SHAPE = -2
MOE_ERR_WORKSPACE = -3
MOE_ERR_CUDA = -4
MOE_ERR_UNIMPLEMENTED = -5
MOE_ERR_DEVICE = -6

MOE_SOFTMAX = 0
MOE_SIGMOID = 1
MOE_SQRTSOFTPLUS = 2

MOE_ST_NAN_TOKENS = 0
MOE_ST_ZERO_DENOM = 1
MOE_ST_BAD_EXPERT_ID = 2
MOE_ST_PIPE_TIMEOUT = 3
MOE_ST_BAD_ROWS = 4
MOE_STATUS_WORDS = 8

MOE_STAGE_ROUTE = 0
MOE_STAGE_PERMUTE = 1
MOE_STAGE_FFN = 2
MOE_STAGE_COMBINE = 3
MOE_STAGE_FORWARD = 4
MOE_STAGE_STATS = 5
MOE_STAGE_BACKWARD = 6
MOE_STAGE_MX_FFN = 7
MOE_STAGE_MX_FORWARD = 8
MOE_NUM_STAGE_EVENTS = 8

MOE_BF16 = 0
MOE_F16 = 1
MOE_F32 = 2

MOE_GATE_NONE = 0
MOE_GATE_CHANNEL = 1
MOE_GATE_TOKEN = 2
MOE_GATE_FULL = 3


class MoeCfg(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("K", ctypes.c_int32), ("I", ctypes.c_int32), ("I_shared", ctypes.c_int32),
                ("score_fn", ctypes.c_int32), ("renorm", ctypes.c_int32),
                ("route_scale", ctypes.c_float), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32)]


class MoeNormCfg(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("first_row", ctypes.c_int64), ("p", ctypes.c_double),
                ("H", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("param_dtype", ctypes.c_int32), ("gate", ctypes.c_int32),
                ("eps", ctypes.c_float), ("residual_scale", ctypes.c_float),
                ("branch_scale", ctypes.c_float)]


_P = ctypes.c_void_p
_SZ = ctypes.c_size_t
_CFG = ctypes.POINTER(MoeCfg)
_I = ctypes.c_int
_NCFG = ctypes.POINTER(MoeNormCfg)
_I64 = ctypes.c_int64

SIGNATURES = {
    "moe_workspace_bytes": (_SZ, [_CFG, _I]),
    "moe_route": (_I, [_CFG, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_permute": (_I, [_CFG, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_permute_noalloc": (_I, [_CFG, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_grouped_ffn": (_I, [_CFG, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_combine": (_I, [_CFG, _P, _P, _P, _P, _P, _P, _P]),
    "moe_combine_invariant": (_I, [_CFG, _P, _P, _P, _P, _P, _P, _P]),
    "moe_forward": (_I, [_CFG, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                         _SZ, _P, _P]),
    "moe_router_stats": (_I, [_CFG, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_backward": (_I, [_CFG] + [_P] * 19 + [_I, _P, _P, _SZ, _P]),
    "moe_forward_train": (_I, [_CFG] + [_P] * 15 + [_SZ, _P]),
    "moe_forward_host_workspace_bytes": (_SZ, [_CFG, _I]),
    "moe_forward_host": (_I, [_CFG, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _SZ, _P]),
    "moe_residual_norm": (_I, [_NCFG] + [_P] * 10),
    "moe_residual_norm_workspace_bytes": (_SZ, [_NCFG]),
    "moe_residual_norm_backward": (_I, [_NCFG] + [_P] * 15 + [_SZ, _P]),
    "moe_dropout": (_I, [_I64, ctypes.c_int32, ctypes.c_int32, ctypes.c_double, _P, _P, _I64, _P,
                         _P, _P]),
    "moe_mx_quantize": (_I, [_I64] + [ctypes.c_int32] * 3 + [_P] * 4),
    "moe_mx_dequantize": (_I, [_I64] + [ctypes.c_int32] * 3 + [_P] * 4),
    "moe_mx_grouped_gemm": (_I, [_I64] + [ctypes.c_int32] * 4 + [_P] * 8),
    "moe_mx_grouped_ffn": (_I, [_CFG] + [_P] * 15 + [_SZ, _P]),
    "moe_mx_forward": (_I, [_CFG] + [_P] * 20 + [_SZ, _P]),
    "moe_status_string": (ctypes.c_char_p, [_I]),
    "moe_abi_version": (_I, []),
    "moe_pipeline_wait_selftest": (_I, [_P, ctypes.c_longlong, _P]),
}

_lock = threading.Lock()
_lib = None


def load():
    """The loaded library (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"libmoe_b200.so is not built ({LIB_PATH}); run "
                    "`python -m deterministic_invariant_routing_b200.build` (needs nvcc)")
            lib = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(lib, name)
                f.restype = res
                f.argtypes = args
            _lib = lib
    return _lib


_binding = None


def binding_target() -> str:
    """What the native part of the binding is compiled against, besides its sources."""
    import torch
    return f"torch {torch.__version__}, Python {sys.version_info[0]}.{sys.version_info[1]}"


def binding_built_for() -> str:
    """binding_target() of the native part's build, which it carries as text ("" if it does not)."""
    with open(BINDING_PATH, "rb") as f:
        _, mark, rest = f.read().partition(b"moe_binding built for ")
    return rest.partition(b"\0")[0].decode() if mark else ""


def load_binding(error):
    """The native part of the binding (csrc/binding.cpp), raising `error` for what it refuses."""
    global _binding
    load()
    with _lock:
        if _binding is None:
            if not os.path.exists(BINDING_PATH):
                raise RuntimeError(
                    f"moe_binding.so is not built ({BINDING_PATH}); run "
                    "`python -m deterministic_invariant_routing_b200.build` (needs nvcc and g++)")
            if binding_built_for() != binding_target():
                raise RuntimeError(
                    f"moe_binding.so was built for {binding_built_for() or 'an unknown torch'}, "
                    f"this is {binding_target()}; run "
                    "`python -m deterministic_invariant_routing_b200.build`")
            import importlib.machinery
            import importlib.util
            loader = importlib.machinery.ExtensionFileLoader("moe_binding", BINDING_PATH)
            spec = importlib.util.spec_from_file_location("moe_binding", BINDING_PATH,
                                                          loader=loader)
            m = importlib.util.module_from_spec(spec)
            loader.exec_module(m)
            m.init(error)
            _binding = m
    return _binding


def status_string(code: int) -> str:
    return load().moe_status_string(code).decode()
