"""ctypes loader for the HIP library and the C structs of include/ep_mi355x.h,
include/ep_mi355x_layer.h and include/ep_mi355x_expert.h.

There is no fallback: if the library is not built, loading raises.
"""
from __future__ import annotations

import ctypes
import os

import torch  # noqa: F401  (load torch's HIP runtime first so the library binds to it)

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libep_mi355x.so")

EP_OK = 0
EP_EINVAL = 1
EP_ENOTSUP = 2
EP_EHIP = 3
EP_EWORKSPACE = 4
EP_ESCRATCH = 5

EP_MAX_TOPK = 32
EP_MAX_KEYS = 1024
EP_LAYOUT_SCRATCH_BYTES = 9 << 18

EP_STATUS_INVALID_IDS = 0
EP_STATUS_ROWS_EXPERT = 1
EP_STATUS_ROWS_GROUP = 2
EP_STATUS_LIST_OVERFLOW = 3
EP_STATUS_COMBINE_OOB = 4
EP_STATUS_EXPERT_LIST_OVERFLOW = 5
EP_STATUS_SELECTIONS = 6
EP_STATUS_DISPATCH_OVERFLOW = 7
EP_STATUS_GENERATION = 8
EP_STATUS_STALE = 9
EP_STATUS_WORDS = 16

EP_FLAG_ZERO_PADDING = 1
EP_FLAG_GATHER_ROWS = 2
EP_FLAG_PACKED_WEIGHTS = 4

EP_FORMAT_BF16 = 0
EP_FORMAT_FP8_PACKED = 1
EP_ROWS_EXPERT = 0
EP_ROWS_GROUP = 1
EP_COMBINE_FLAT = 0
EP_COMBINE_GROUPED = 1

EP_MAX_ROUTE_GROUPS = 64
EP_MAX_LORA_RANK = 128
EP_SCORE_SOFTMAX = 0
EP_SCORE_SIGMOID = 1
EP_LOGITS_FP32 = 0
EP_LOGITS_BF16 = 1
EP_LORA_SCATTER_ROWS = 1
EP_ACT_NONE = 0
EP_ACT_RELU = 1
EP_ACT_SILU = 2
EP_ACT_GELU = 3
EP_ACT_GELU_TANH = 4

EXPORTS = (
    "ep_fp8_row_bytes",
    "ep_layout_workspace_bytes",
    "ep_layout",
    "ep_layout_noalloc",
    "ep_dispatch",
    "ep_combine",
    "ep_expert_gemm",
    "ep_expert_weights_packed_bytes",
    "ep_pack_expert_weights",
    "ep_strerror",
    "ep_route",
    "ep_route_backward",
    "ep_combine_backward",
    "ep_lora_workspace_bytes",
    "ep_lora",
    "ep_lora_backward",
    "ep_expert_linear",
    "ep_expert_linear_workspace_bytes",
    "ep_expert_linear_backward",
    "ep_balance_workspace_bytes",
    "ep_balance_loss",
    "ep_balance_loss_backward",
)


class Problem(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("hidden", ctypes.c_int32),
        ("topk", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("num_groups", ctypes.c_int32),
        ("expert_alignment", ctypes.c_int32),
        ("flags", ctypes.c_int32),
    ]


class LayoutStruct(ctypes.Structure):
    _fields_ = [
        ("counts", ctypes.c_void_p),
        ("offsets", ctypes.c_void_p),
        ("slot", ctypes.c_void_p),
        ("status", ctypes.c_void_p),
        ("group_counts", ctypes.c_void_p),
        ("group_offsets", ctypes.c_void_p),
        ("grow", ctypes.c_void_p),
        ("row_src", ctypes.c_void_p),
        ("row_topk_idx", ctypes.c_void_p),
        ("row_topk_weights", ctypes.c_void_p),
        ("row_capacity", ctypes.c_int64),
        ("expert_row_src", ctypes.c_void_p),
        ("expert_row_capacity", ctypes.c_int64),
        ("recv_stats", ctypes.c_void_p),
        ("generation", ctypes.c_uint32),
    ]


class Router(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("num_experts", ctypes.c_int32),
        ("topk", ctypes.c_int32),
        ("score", ctypes.c_int32),
        ("logits", ctypes.c_int32),
        ("num_groups", ctypes.c_int32),
        ("topk_groups", ctypes.c_int32),
        ("group_top", ctypes.c_int32),
        ("renormalize", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


class LoraWeights(ctypes.Structure):
    _fields_ = [
        ("a", ctypes.c_void_p),
        ("b", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("rank", ctypes.c_int32),
        ("n_out", ctypes.c_int32),
        ("flags", ctypes.c_int32),
    ]


class Linear(ctypes.Structure):
    _fields_ = [
        ("w", ctypes.c_void_p),
        ("bias", ctypes.c_void_p),
        ("n_out", ctypes.c_int32),
        ("activation", ctypes.c_int32),
        ("gated", ctypes.c_int32),
    ]


class Balance(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("num_experts", ctypes.c_int32),
        ("topk", ctypes.c_int32),
        ("score", ctypes.c_int32),
        ("logits", ctypes.c_int32),
        ("num_seqs", ctypes.c_int32),
        ("coef", ctypes.c_float),
    ]


class EPError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed with code {code}: {msg}")
        self.code = code


_LIB = None


def lib(path: str | None = None) -> ctypes.CDLL:
    """Load (once) and type the library's exports.  Raises if it is missing."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            f"HIP library {p} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`"
        )
    L = ctypes.CDLL(p)
    P = ctypes.POINTER(Problem)
    LS = ctypes.POINTER(LayoutStruct)
    vp = ctypes.c_void_p
    L.ep_fp8_row_bytes.argtypes = [ctypes.c_int32]
    L.ep_fp8_row_bytes.restype = ctypes.c_int64
    L.ep_layout_workspace_bytes.argtypes = [P]
    L.ep_layout_workspace_bytes.restype = ctypes.c_size_t
    L.ep_layout.argtypes = [P, vp, vp, LS, vp, ctypes.c_size_t, vp]
    L.ep_layout.restype = ctypes.c_int
    L.ep_layout_noalloc.argtypes = [P, vp, vp, LS, vp]
    L.ep_layout_noalloc.restype = ctypes.c_int
    L.ep_dispatch.argtypes = [P, LS, vp, vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, vp]
    L.ep_dispatch.restype = ctypes.c_int
    L.ep_combine.argtypes = [P, LS, vp, vp, vp, ctypes.c_int64, vp, vp, vp, ctypes.c_int32, vp]
    L.ep_combine.restype = ctypes.c_int
    L.ep_expert_gemm.argtypes = [P, LS, vp, ctypes.c_int64, vp, ctypes.c_int32, vp, ctypes.c_int64, vp]
    L.ep_expert_gemm.restype = ctypes.c_int
    L.ep_expert_weights_packed_bytes.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
    L.ep_expert_weights_packed_bytes.restype = ctypes.c_int64
    L.ep_pack_expert_weights.argtypes = [vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, vp, vp]
    L.ep_pack_expert_weights.restype = ctypes.c_int
    RT = ctypes.POINTER(Router)
    LW = ctypes.POINTER(LoraWeights)
    i64 = ctypes.c_int64
    L.ep_route.argtypes = [RT, vp, vp, vp, vp, vp, vp]
    L.ep_route.restype = ctypes.c_int
    L.ep_route_backward.argtypes = [RT, vp, vp, vp, vp, vp]
    L.ep_route_backward.restype = ctypes.c_int
    L.ep_combine_backward.argtypes = [P, LS, vp, vp, vp, i64, vp, vp, vp]
    L.ep_combine_backward.restype = ctypes.c_int
    L.ep_lora_workspace_bytes.argtypes = [P, LW, ctypes.c_int32]
    L.ep_lora_workspace_bytes.restype = ctypes.c_size_t
    L.ep_lora.argtypes = [P, LS, LW, vp, i64, vp, i64, vp, i64, vp, ctypes.c_size_t, vp]
    L.ep_lora.restype = ctypes.c_int
    L.ep_lora_backward.argtypes = [P, LS, LW, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, vp, ctypes.c_size_t, vp]
    L.ep_lora_backward.restype = ctypes.c_int
    LN = ctypes.POINTER(Linear)
    BL = ctypes.POINTER(Balance)
    L.ep_expert_linear.argtypes = [P, LS, LN, vp, i64, vp, i64, vp, i64, vp, i64, vp]
    L.ep_expert_linear.restype = ctypes.c_int
    L.ep_expert_linear_workspace_bytes.argtypes = [P, LN]
    L.ep_expert_linear_workspace_bytes.restype = ctypes.c_size_t
    L.ep_expert_linear_backward.argtypes = [P, LS, LN, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, vp,
                                            ctypes.c_size_t, vp]
    L.ep_expert_linear_backward.restype = ctypes.c_int
    L.ep_balance_workspace_bytes.argtypes = [BL]
    L.ep_balance_workspace_bytes.restype = ctypes.c_size_t
    L.ep_balance_loss.argtypes = [BL, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    L.ep_balance_loss.restype = ctypes.c_int
    L.ep_balance_loss_backward.argtypes = [BL, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.ep_balance_loss_backward.restype = ctypes.c_int
    L.ep_strerror.argtypes = [ctypes.c_int]
    L.ep_strerror.restype = ctypes.c_char_p
    if path is None:
        _LIB = L
    return L


def check(fn: str, code: int) -> None:
    if code != EP_OK:
        raise EPError(fn, code, lib().ep_strerror(code).decode())
