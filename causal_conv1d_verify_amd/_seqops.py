"""ctypes view of libseqops.so (the C ABI declared in include/sequence_ops.h)."""

from __future__ import annotations

import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libseqops.so")

SQ_SCAN_PREFILL, SQ_SCAN_UPDATE, SQ_SCAN_VERIFY, SQ_SCAN_COMMIT = range(4)

EXPORTS = (
    "selscan_prefill",
    "selscan_prefill_workspace",
    "selscan_update",
    "selscan_verify",
    "selscan_commit",
    "selscan_describe",
    "norm_rotary",
    "accept_drafts",
    "accept_drafts_workspace",
    "seqops_strerror",
    "seqops_last_error",
    "seqops_abi_version",
)


def _fields(ctype, names):
    return [(name, ctype) for name in names.split()]


class SqScanShape(ctypes.Structure):
    _fields_ = [*_fields(ctypes.c_int32, "n_seq T d d_state x_dtype state_dtype n_slots softplus"),
                *_fields(ctypes.c_int64, "x_seq_stride x_tok_stride dt_seq_stride dt_tok_stride "
                         "z_seq_stride z_tok_stride b_seq_stride b_tok_stride c_seq_stride "
                         "c_tok_stride out_seq_stride out_tok_stride state_slot_stride tokens")]


class SqScanData(ctypes.Structure):
    _fields_ = _fields(ctypes.c_void_p, "x dt z B C A D dt_bias")


class SqScanInfo(ctypes.Structure):
    _fields_ = [*_fields(ctypes.c_int64, "workgroups workspace_bytes"),
                *_fields(ctypes.c_int32, "threads channels segment_tokens launches")]


class SqRotaryShape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), *_fields(ctypes.c_int32, "q_heads k_heads dim rot"),
                ("eps", ctypes.c_float), *_fields(ctypes.c_int32, "x_dtype interleaved wide_positions"),
                *_fields(ctypes.c_int64, "q_tok_stride q_head_stride k_tok_stride k_head_stride "
                         "q_out_tok_stride q_out_head_stride k_out_tok_stride k_out_head_stride")]


class SqAcceptShape(ctypes.Structure):
    _fields_ = [*_fields(ctypes.c_int32, "n_seq T vocab p_dtype"),
                *_fields(ctypes.c_int64, "tokens_stride parent_stride uniform_stride path_stride "
                         "target_seq_stride target_tok_stride draft_seq_stride draft_tok_stride")]


_lib = None


def load() -> ctypes.CDLL:
    """Load the HIP library.  Raises if it has not been built: there is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m causal_conv1d_verify_amd.build` "
            "(or __graft_entry__.build()); the scan, the rotation and the verdict on drafts have "
            "no non-HIP implementation")
    lib = ctypes.CDLL(LIB_PATH)
    V, I64 = ctypes.c_void_p, ctypes.c_int64
    S, D = ctypes.POINTER(SqScanShape), ctypes.POINTER(SqScanData)
    R, A = ctypes.POINTER(SqRotaryShape), ctypes.POINTER(SqAcceptShape)
    for name, restype, args in (
            ("selscan_prefill", ctypes.c_int, [S, D] + [V] * 6 + [I64, V]),
            ("selscan_prefill_workspace", I64, [S]),
            ("selscan_update", ctypes.c_int, [S, D] + [V] * 4),
            ("selscan_verify", ctypes.c_int, [S, D] + [V] * 4),
            ("selscan_commit", ctypes.c_int, [S, D] + [V] * 4),
            ("selscan_describe", ctypes.c_int, [ctypes.c_int, S, ctypes.POINTER(SqScanInfo)]),
            ("norm_rotary", ctypes.c_int, [R] + [V] * 9),
            ("accept_drafts", ctypes.c_int, [A] + [V] * 11 + [I64, V]),
            ("accept_drafts_workspace", I64, [A]),
            ("seqops_strerror", ctypes.c_char_p, [ctypes.c_int]),
            ("seqops_last_error", ctypes.c_char_p, []),
            ("seqops_abi_version", ctypes.c_int, [])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = restype, args
    _lib = lib
    return _lib


def error_message(lib, code: int) -> str:
    return f"{lib.seqops_strerror(code).decode()} ({code}): {lib.seqops_last_error().decode()}"
