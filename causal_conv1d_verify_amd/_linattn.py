"""ctypes view of liblinattn.so (the C ABI declared in include/linear_attention.h)."""

from __future__ import annotations

import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblinattn.so")

LA_SILU = 0
LA_SIGMOID = 1
LA_CALL_PREFILL, LA_CALL_UPDATE, LA_CALL_VERIFY, LA_CALL_COMMIT = range(4)
LA_KERNEL_TOKENS, LA_KERNEL_FEW, LA_KERNEL_CHUNKED, LA_KERNEL_CHUNKED_F32 = range(4)

EXPORTS = (
    "linattn_prefill",
    "linattn_prefill_workspace",
    "linattn_update",
    "linattn_verify",
    "linattn_commit",
    "linattn_describe",
    "norm_gated",
    "norm_residual",
    "linattn_strerror",
    "linattn_last_error",
    "linattn_abi_version",
)


class LaShape(ctypes.Structure):
    _fields_ = [
        ("n_seq", ctypes.c_int32), ("T", ctypes.c_int32),
        ("q_heads", ctypes.c_int32), ("v_heads", ctypes.c_int32),
        ("dk", ctypes.c_int32), ("dv", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("x_dtype", ctypes.c_int32), ("state_dtype", ctypes.c_int32),
        ("n_slots", ctypes.c_int32),
        ("q_seq_stride", ctypes.c_int64), ("q_tok_stride", ctypes.c_int64),
        ("q_head_stride", ctypes.c_int64),
        ("k_seq_stride", ctypes.c_int64), ("k_tok_stride", ctypes.c_int64),
        ("k_head_stride", ctypes.c_int64),
        ("v_seq_stride", ctypes.c_int64), ("v_tok_stride", ctypes.c_int64),
        ("v_head_stride", ctypes.c_int64),
        ("out_seq_stride", ctypes.c_int64), ("out_tok_stride", ctypes.c_int64),
        ("out_head_stride", ctypes.c_int64),
        ("g_seq_stride", ctypes.c_int64), ("g_tok_stride", ctypes.c_int64),
        ("state_slot_stride", ctypes.c_int64), ("tokens", ctypes.c_int64),
    ]


class LaNormShape(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32),
        ("eps", ctypes.c_float), ("scale", ctypes.c_float),
        ("x_dtype", ctypes.c_int32), ("res_dtype", ctypes.c_int32),
        ("activation", ctypes.c_int32), ("gate_first", ctypes.c_int32),
        ("y_row_stride", ctypes.c_int64), ("y_head_stride", ctypes.c_int64),
        ("gate_row_stride", ctypes.c_int64), ("gate_head_stride", ctypes.c_int64),
        ("out_row_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
        ("res_row_stride", ctypes.c_int64), ("res_out_row_stride", ctypes.c_int64),
    ]


class LaLaunchInfo(ctypes.Structure):
    _fields_ = [
        ("workgroups", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
        ("kernel", ctypes.c_int32), ("threads", ctypes.c_int32),
        ("state_cols", ctypes.c_int32), ("segment_tokens", ctypes.c_int32),
        ("launches", ctypes.c_int32), ("streaming", ctypes.c_int32),
    ]


_lib = None


def load() -> ctypes.CDLL:
    """Load the HIP library.  Raises if it has not been built: there is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m causal_conv1d_verify_amd.build` "
            "(or __graft_entry__.build()); linear attention has no non-HIP implementation")
    lib = ctypes.CDLL(LIB_PATH)
    S, N, V = ctypes.POINTER(LaShape), ctypes.POINTER(LaNormShape), ctypes.c_void_p
    for name, args in (("linattn_prefill", [S] + [V] * 10 + [ctypes.c_int64, V]),
                       ("linattn_update", [S] + [V] * 8), ("linattn_verify", [S] + [V] * 8),
                       ("linattn_commit", [S] + [V] * 7), ("norm_gated", [N] + [V] * 5),
                       ("norm_residual", [N] + [V] * 8)):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ctypes.c_int, args
    lib.linattn_prefill_workspace.restype = ctypes.c_int64
    lib.linattn_prefill_workspace.argtypes = [S]
    lib.linattn_describe.restype = ctypes.c_int
    lib.linattn_describe.argtypes = [ctypes.c_int, S, ctypes.POINTER(LaLaunchInfo)]
    lib.linattn_strerror.restype = ctypes.c_char_p
    lib.linattn_strerror.argtypes = [ctypes.c_int]
    lib.linattn_last_error.restype = ctypes.c_char_p
    lib.linattn_last_error.argtypes = []
    lib.linattn_abi_version.restype = ctypes.c_int
    lib.linattn_abi_version.argtypes = []
    _lib = lib
    return _lib


def error_message(lib, code: int) -> str:
    return f"{lib.linattn_strerror(code).decode()} ({code}): {lib.linattn_last_error().decode()}"
