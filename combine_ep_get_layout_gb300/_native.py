"""ctypes view of ``libep_gb300.so`` (the C ABI in ``include/ep_gb300.h``).

Loading fails loudly when the library has not been built: there is no
fallback of any kind.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libep_gb300.so")

EP_OK = 0
EP_ERR_INVALID_ARG = 1
EP_ERR_UNSUPPORTED = 2
EP_ERR_CUDA = 3

EP_DTYPE_BF16 = 0
EP_DTYPE_FP8_E4M3 = 1
EP_DTYPE_FP8_E4M3_PACKED = 2

EP_ERRBIT_BAD_INDEX = 0x1
EP_ERRBIT_CAPACITY = 0x2
EP_ERRBIT_TIMEOUT = 0x4
EP_ERRBIT_STALE_LAYOUT = 0x8
EP_ERRBIT_DUP_EXPERT = 0x10

EP_MAX_RANKS = 64
EP_MAX_TOPK = 32
EP_MAX_EXPERTS = 4096
EP_MAX_HIDDEN = 16384
EP_FP8_GROUP = 128
EP_NOALLOC_SCRATCH_BYTES = 256 * 1024
EP_WORK_COUNTER_WORDS = 4

EP_SCORE_SOFTMAX = 0
EP_SCORE_SIGMOID = 1
EP_LOGITS_FP32 = 0
EP_LOGITS_BF16 = 1
EP_ACT_NONE = 0
EP_ACT_SWIGLU = 1
EP_ACT_RELU = 2
EP_ACT_SILU = 3
EP_ACT_GELU = 4
EP_ACT_GELU_TANH = 5
EP_TYPE_FP32 = 0
EP_TYPE_BF16 = 1
EP_MAX_SEQUENCES = 65536
EP_MAX_RANK = 128

ABI_VERSION = 2  # EP_ABI_VERSION of the header these bindings mirror


class ep_layout_t(C.Structure):
    _fields_ = [
        ("num_tokens_per_expert", C.c_void_p),
        ("num_tokens_per_rank", C.c_void_p),
        ("rank_prefix", C.c_void_p),
        ("is_token_in_rank", C.c_void_p),
        ("token_slot", C.c_void_p),
        ("error_word", C.c_void_p),
        ("work_counters", C.c_void_p),
    ]


class ep_dispatch_args_t(C.Structure):
    _fields_ = [
        ("x", C.c_void_p), ("num_tokens", C.c_int), ("hidden", C.c_int),
        ("topk_idx", C.c_void_p), ("topk_weights", C.c_void_p), ("num_topk", C.c_int),
        ("num_experts", C.c_int), ("num_ranks", C.c_int),
        ("layout", C.POINTER(ep_layout_t)), ("dtype", C.c_int),
        ("recv_x", C.c_void_p), ("recv_x_scales", C.c_void_p), ("recv_src_idx", C.c_void_p),
        ("recv_topk_idx", C.c_void_p), ("recv_topk_weights", C.c_void_p),
        ("recv_capacity", C.c_int), ("cumulative_recv_stats", C.c_void_p),
    ]


class ep_combine_args_t(C.Structure):
    _fields_ = [
        ("y", C.c_void_p), ("recv_capacity", C.c_int), ("hidden", C.c_int),
        ("layout", C.POINTER(ep_layout_t)), ("num_tokens", C.c_int), ("num_ranks", C.c_int),
        ("topk_idx", C.c_void_p), ("topk_weights", C.c_void_p), ("num_topk", C.c_int),
        ("num_experts", C.c_int), ("bias0", C.c_void_p), ("bias1", C.c_void_p),
        ("out", C.c_void_p),
    ]


class ep_expanded_layout_t(C.Structure):
    _fields_ = [
        ("num_rows_per_expert", C.c_void_p),
        ("expert_offset", C.c_void_p),
        ("token_slot", C.c_void_p),
        ("error_word", C.c_void_p),
        ("work_counters", C.c_void_p),
    ]


class ep_dispatch_expanded_args_t(C.Structure):
    _fields_ = [
        ("x", C.c_void_p), ("num_tokens", C.c_int), ("hidden", C.c_int),
        ("topk_idx", C.c_void_p), ("topk_weights", C.c_void_p), ("num_topk", C.c_int),
        ("num_experts", C.c_int), ("num_ranks", C.c_int),
        ("layout", C.POINTER(ep_expanded_layout_t)), ("dtype", C.c_int),
        ("recv_x", C.c_void_p), ("recv_x_scales", C.c_void_p), ("recv_src_idx", C.c_void_p),
        ("recv_topk_idx", C.c_void_p), ("recv_topk_weights", C.c_void_p),
        ("recv_capacity", C.c_int), ("zero_padding", C.c_int),
        ("cumulative_recv_stats", C.c_void_p),
    ]


class ep_combine_expanded_args_t(C.Structure):
    _fields_ = [
        ("y", C.c_void_p), ("recv_capacity", C.c_int), ("hidden", C.c_int),
        ("layout", C.POINTER(ep_expanded_layout_t)), ("num_tokens", C.c_int),
        ("num_topk", C.c_int), ("topk_idx", C.c_void_p), ("topk_weights", C.c_void_p),
        ("num_experts", C.c_int), ("bias0", C.c_void_p), ("bias1", C.c_void_p),
        ("out", C.c_void_p),
    ]


class ep_route_args_t(C.Structure):
    _fields_ = [
        ("logits", C.c_void_p), ("logits_type", C.c_int), ("row_stride", C.c_int64),
        ("num_tokens", C.c_int), ("num_experts", C.c_int), ("num_topk", C.c_int),
        ("score", C.c_int), ("bias", C.c_void_p), ("num_groups", C.c_int),
        ("topk_groups", C.c_int), ("group_top", C.c_int), ("renormalize", C.c_int),
        ("weight_scale", C.c_float), ("topk_idx", C.c_void_p), ("topk_weights", C.c_void_p),
    ]


class ep_route_backward_args_t(C.Structure):
    _fields_ = [
        ("grad_weights", C.c_void_p), ("logits", C.c_void_p), ("logits_type", C.c_int),
        ("row_stride", C.c_int64), ("topk_idx", C.c_void_p), ("num_tokens", C.c_int),
        ("num_experts", C.c_int), ("num_topk", C.c_int), ("score", C.c_int),
        ("renormalize", C.c_int), ("weight_scale", C.c_float), ("grad_logits", C.c_void_p),
    ]


class ep_expert_product_args_t(C.Structure):
    _fields_ = [
        ("x", C.c_void_p), ("recv_capacity", C.c_int), ("num_tokens", C.c_int),
        ("hidden", C.c_int), ("num_experts", C.c_int),
        ("layout", C.POINTER(ep_expanded_layout_t)), ("w", C.c_void_p), ("width", C.c_int),
        ("activation", C.c_int), ("out", C.c_void_p), ("preact", C.c_void_p),
    ]


class ep_expert_product_backward_args_t(C.Structure):
    _fields_ = [
        ("grad", C.c_void_p), ("x", C.c_void_p), ("w", C.c_void_p), ("recv_capacity", C.c_int),
        ("num_tokens", C.c_int), ("hidden", C.c_int), ("num_experts", C.c_int),
        ("layout", C.POINTER(ep_expanded_layout_t)), ("width", C.c_int), ("activation", C.c_int),
        ("preact", C.c_void_p), ("grad_preact", C.c_void_p), ("grad_x", C.c_void_p),
        ("grad_w", C.c_void_p),
    ]


class ep_adapter_product_args_t(C.Structure):
    _fields_ = [
        ("x", C.c_void_p), ("num_rows", C.c_int), ("hidden", C.c_int), ("w", C.c_void_p),
        ("width", C.c_int), ("lora_a", C.c_void_p), ("lora_b", C.c_void_p),
        ("num_adapters", C.c_int), ("rank", C.c_int), ("adapter_idx", C.c_void_p),
        ("adapter_scale", C.c_void_p), ("out", C.c_void_p), ("workspace", C.c_void_p),
        ("workspace_bytes", C.c_size_t), ("error_word", C.c_void_p),
    ]


class ep_balance_loss_args_t(C.Structure):
    _fields_ = [
        ("logits", C.c_void_p), ("logits_type", C.c_int), ("row_stride", C.c_int64),
        ("topk_idx", C.c_void_p), ("num_tokens", C.c_int), ("num_experts", C.c_int),
        ("num_topk", C.c_int), ("score", C.c_int), ("seq_offsets", C.c_void_p),
        ("num_sequences", C.c_int), ("losses", C.c_void_p), ("counts", C.c_void_p),
        ("probs", C.c_void_p), ("slopes", C.c_void_p), ("workspace", C.c_void_p),
        ("workspace_bytes", C.c_size_t),
    ]


class ep_balance_loss_backward_args_t(C.Structure):
    _fields_ = [
        ("grad_losses", C.c_void_p), ("logits", C.c_void_p), ("logits_type", C.c_int),
        ("row_stride", C.c_int64), ("num_tokens", C.c_int), ("num_experts", C.c_int),
        ("score", C.c_int), ("seq_offsets", C.c_void_p), ("num_sequences", C.c_int),
        ("slopes", C.c_void_p), ("add", C.c_void_p), ("grad_logits", C.c_void_p),
    ]


class ep_layer_norm_args_t(C.Structure):
    _fields_ = [
        ("x", C.c_void_p), ("type", C.c_int), ("row_stride", C.c_int64), ("num_rows", C.c_int),
        ("hidden", C.c_int), ("weight", C.c_void_p), ("bias", C.c_void_p), ("param_type", C.c_int),
        ("eps", C.c_float), ("out", C.c_void_p), ("mean", C.c_void_p), ("rstd", C.c_void_p),
    ]


class ep_layer_norm_backward_args_t(C.Structure):
    _fields_ = [
        ("grad", C.c_void_p), ("x", C.c_void_p), ("type", C.c_int), ("row_stride", C.c_int64),
        ("num_rows", C.c_int), ("hidden", C.c_int), ("mean", C.c_void_p), ("rstd", C.c_void_p),
        ("weight", C.c_void_p), ("param_type", C.c_int), ("add", C.c_void_p), ("grad_x", C.c_void_p),
        ("grad_weight", C.c_void_p), ("grad_bias", C.c_void_p), ("workspace", C.c_void_p),
        ("workspace_bytes", C.c_size_t),
    ]


class ep_dense_product_args_t(C.Structure):
    _fields_ = [
        ("x", C.c_void_p), ("row_stride", C.c_int64), ("num_rows", C.c_int), ("hidden", C.c_int),
        ("w", C.c_void_p), ("width", C.c_int), ("bias", C.c_void_p), ("bias_type", C.c_int),
        ("activation", C.c_int), ("residual", C.c_void_p), ("out", C.c_void_p), ("out_type", C.c_int),
        ("preact", C.c_void_p), ("error_word", C.c_void_p),
    ]


class ep_dense_product_backward_args_t(C.Structure):
    _fields_ = [
        ("grad", C.c_void_p), ("grad_type", C.c_int), ("x", C.c_void_p), ("row_stride", C.c_int64),
        ("num_rows", C.c_int), ("hidden", C.c_int), ("w", C.c_void_p), ("width", C.c_int),
        ("activation", C.c_int), ("preact", C.c_void_p), ("grad_preact", C.c_void_p),
        ("grad_x", C.c_void_p), ("grad_w", C.c_void_p), ("grad_bias", C.c_void_p),
        ("bias_type", C.c_int), ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t),
        ("error_word", C.c_void_p),
    ]


# name -> (restype, argtypes); mirrors include/ep_gb300.h
_p, _i, _sz = C.c_void_p, C.c_int, C.c_size_t
_LP = C.POINTER(ep_layout_t)
SIGNATURES = {
    "ep_layout_workspace_bytes": (_sz, [_i, _i, _i]),
    "ep_get_layout": (_i, [_p, _i, _i, _i, _i, _LP, _p, _sz, _p]),
    "ep_get_layout_noalloc": (_i, [_p, _i, _i, _i, _i, _LP, _p]),
    "ep_dispatch": (_i, [_p, _i, _i, _p, _p, _i, _i, _i, _LP, _i, _p, _p, _p, _p, _p, _i, _p]),
    "ep_combine": (_i, [_p, _i, _i, _LP, _i, _i, _p, _p, _i, _i, _p, _p]),
    "ep_fp8_packed_row_bytes": (_sz, [_i]),
    "ep_dispatch_ex": (_i, [C.POINTER(ep_dispatch_args_t), _p]),
    "ep_get_layout_and_dispatch": (_i, [C.POINTER(ep_dispatch_args_t), _p, _sz, _p]),
    "ep_combine_ex": (_i, [C.POINTER(ep_combine_args_t), _p]),
    "ep_expanded_layout_workspace_bytes": (_sz, [_i, _i]),
    "ep_get_layout_expanded": (_i, [_p, _i, _i, _i, _i, C.POINTER(ep_expanded_layout_t), _p, _sz, _p]),
    "ep_dispatch_expanded": (_i, [C.POINTER(ep_dispatch_expanded_args_t), _p]),
    "ep_combine_expanded": (_i, [C.POINTER(ep_combine_expanded_args_t), _p]),
    "ep_route": (_i, [C.POINTER(ep_route_args_t), _p]),
    "ep_route_backward": (_i, [C.POINTER(ep_route_backward_args_t), _p]),
    "ep_expert_product": (_i, [C.POINTER(ep_expert_product_args_t), _p]),
    "ep_expert_product_backward": (_i, [C.POINTER(ep_expert_product_backward_args_t), _p]),
    "ep_adapter_workspace_bytes": (_sz, [_i, _i, _i]),
    "ep_adapter_product": (_i, [C.POINTER(ep_adapter_product_args_t), _p]),
    "ep_balance_workspace_bytes": (_sz, [_i, _i, _i]),
    "ep_balance_loss": (_i, [C.POINTER(ep_balance_loss_args_t), _p]),
    "ep_balance_loss_backward": (_i, [C.POINTER(ep_balance_loss_backward_args_t), _p]),
    "ep_layer_norm": (_i, [C.POINTER(ep_layer_norm_args_t), _p]),
    "ep_layer_norm_workspace_bytes": (_sz, [_i, _i]),
    "ep_layer_norm_backward": (_i, [C.POINTER(ep_layer_norm_backward_args_t), _p]),
    "ep_dense_product": (_i, [C.POINTER(ep_dense_product_args_t), _p]),
    "ep_dense_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "ep_dense_product_backward": (_i, [C.POINTER(ep_dense_product_backward_args_t), _p]),
    "ep_selftest_bounded_waits": (_i, [_p, _p, _p, _p]),
    "ep_status_str": (C.c_char_p, [_i]),
    "ep_last_error": (C.c_char_p, []),
    "ep_abi_version": (_i, []),
}

_CODES = {C.c_void_p: "P", C.c_int: "i", C.c_int64: "q", C.c_float: "f", C.c_size_t: "N"}


def packer(cls):
    """A function from a structure's fields, in order and pointers as
    integers, to its bytes: building the structure takes three times as
    long, which short calls would notice."""
    s = struct.Struct("@" + "".join("P" if issubclass(t, C._Pointer) else _CODES[t] for _, t in cls._fields_) + "0P")
    assert s.size == C.sizeof(cls)
    return s.pack


_lock = threading.Lock()
_lib = None


def load():
    """The loaded library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m combine_ep_get_layout_gb300.build` "
                    "(or __graft_entry__.build()); there is no fallback path")
            lib = C.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(lib, name)
                f.restype = res
                f.argtypes = args
            if lib.ep_abi_version() != ABI_VERSION:
                raise RuntimeError("libep_gb300.so ABI version mismatch")
            _lib = lib
    return _lib
