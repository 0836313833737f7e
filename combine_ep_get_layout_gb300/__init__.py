"""MoE expert-parallel layout / dispatch / combine on one GB300 GPU.

A thin binding over the C ABI of ``libep_gb300.so`` (``include/ep_gb300.h``):
it only checks tensor dtypes/devices, allocates outputs the caller did not
pass, and marshals pointers and the current CUDA stream.  Every step of the
path runs in the library's CUDA kernels; there is no CPU fallback.

    lay = ep_get_layout(topk_idx, num_experts, num_ranks)
    d = ep_dispatch(x, topk_idx, topk_weights, lay, dtype="fp8")
    out = ep_combine(y, lay, topk_idx, topk_weights)

Expert ``e`` lives on logical rank ``e // (num_experts // num_ranks)``;
``topk_idx == -1`` means "no selection".
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass
from functools import lru_cache
from typing import Optional

import torch

from . import _native as N
from ._native import (EP_ERRBIT_BAD_INDEX, EP_ERRBIT_CAPACITY,  # noqa: F401
                      EP_ERRBIT_DUP_EXPERT, EP_ERRBIT_STALE_LAYOUT, EP_ERRBIT_TIMEOUT,
                      EP_FP8_GROUP)

__all__ = ["EPError", "Layout", "Dispatched", "ep_layout_workspace_bytes",
           "ep_get_layout", "ep_get_layout_noalloc", "ep_dispatch", "ep_dispatch_ex",
           "ep_get_layout_and_dispatch",
           "ep_combine", "ep_combine_ex", "ep_fp8_packed_row_bytes", "ExpandedLayout",
           "ep_expanded_layout_workspace_bytes", "ep_get_layout_expanded",
           "ep_dispatch_expanded", "ep_combine_expanded", "Routing", "ep_route",
           "ep_route_backward", "ep_expert_product", "ep_expert_product_backward",
           "ep_adapter_workspace_bytes", "ep_adapter_product", "Balance", "ep_balance_workspace_bytes",
           "ep_balance_loss", "ep_balance_loss_backward", "ep_layer_norm", "ep_layer_norm_workspace_bytes",
           "ep_layer_norm_backward", "ep_dense_product", "ep_dense_workspace_bytes",
           "ep_dense_product_backward", "ep_selftest_bounded_waits", "library_path"]


class EPError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        super().__init__(message)


def library_path() -> str:
    N.load()
    return N.LIB_PATH


def _check(status: int, fn: str):
    if status != N.EP_OK:
        lib = N.load()
        name = lib.ep_status_str(status).decode()
        detail = lib.ep_last_error().decode()
        raise EPError(status, f"{fn}: {name}: {detail}")


def _call(dev: torch.device, fn: str, *args):
    """Calls the library function ``fn`` with ``dev`` as the current CUDA
    device: the library launches on the calling thread's current device,
    which must be the one holding the tensors and owning the stream."""
    with torch.cuda.device(dev):
        _check(getattr(N.load(), fn)(*args), fn)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream, device) -> C.c_void_p:
    """The handle of ``stream`` (default: the device's current stream), which
    must belong to the tensors' device."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return C.c_void_p(stream.cuda_stream)


def _want(t: torch.Tensor, name: str, dtype, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def ep_fp8_packed_row_bytes(hidden: int) -> int:
    """Bytes of one packed fp8 row (codes, scales, zero padding)."""
    return int(N.load().ep_fp8_packed_row_bytes(hidden))


def ep_layout_workspace_bytes(num_tokens: int, num_experts: int, num_ranks: int) -> int:
    return int(N.load().ep_layout_workspace_bytes(num_tokens, num_experts, num_ranks))


@dataclass
class Layout:
    """Device tensors of one routing's layout (see ``ep_layout_t``)."""
    num_tokens_per_expert: torch.Tensor  # int32 [E]
    num_tokens_per_rank: torch.Tensor    # int32 [R]
    rank_prefix: torch.Tensor            # int32 [R+1]
    is_token_in_rank: torch.Tensor       # uint8 [T, R]
    token_slot: torch.Tensor             # int32 [T, R]
    error_word: torch.Tensor             # int32 [1] (bit flags)
    workspace: torch.Tensor              # uint8, zero-filled once
    num_tokens: int
    num_experts: int
    num_ranks: int
    work_counters: Optional[torch.Tensor] = None  # int32 [4]: blocks draw tokens from a counter

    @staticmethod
    def empty(num_tokens: int, num_experts: int, num_ranks: int, device,
              work_counters: bool = True) -> "Layout":
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        ws = ep_layout_workspace_bytes(num_tokens, num_experts, num_ranks)
        return Layout(
            torch.empty(num_experts, **i32), torch.empty(num_ranks, **i32),
            torch.empty(num_ranks + 1, **i32),
            torch.empty((num_tokens, num_ranks), dtype=torch.uint8, device=dev),
            torch.empty((num_tokens, num_ranks), **i32),
            torch.zeros(1, **i32),
            torch.zeros(max(ws, 16), dtype=torch.uint8, device=dev),
            num_tokens, num_experts, num_ranks,
            torch.zeros(N.EP_WORK_COUNTER_WORDS, **i32) if work_counters else None)

    def c_struct(self) -> N.ep_layout_t:
        return N.ep_layout_t(
            self.num_tokens_per_expert.data_ptr(), self.num_tokens_per_rank.data_ptr(),
            self.rank_prefix.data_ptr(), self.is_token_in_rank.data_ptr(),
            self.token_slot.data_ptr(), self.error_word.data_ptr(),
            None if self.work_counters is None else self.work_counters.data_ptr())

    def num_recv(self) -> int:
        """N, read back to the host (synchronises)."""
        return int(self.rank_prefix[self.num_ranks].item())

    def errors(self) -> int:
        """The device error word, read back to the host (synchronises)."""
        return int(self.error_word.item()) & 0xffffffff


def ep_get_layout(topk_idx: torch.Tensor, num_experts: int, num_ranks: int,
                  layout: Optional[Layout] = None, stream=None,
                  work_counters: bool = True) -> Layout:
    """The layout of one routing.  A new layout carries work counters
    unless ``work_counters`` is false (then dispatch and combine give each
    thread block a fixed stripe of tokens)."""
    _want(topk_idx, "topk_idx", torch.int64)
    T, K = topk_idx.shape
    dev = topk_idx.device
    if layout is None:
        layout = Layout.empty(T, num_experts, num_ranks, dev, work_counters)
    elif (layout.num_tokens, layout.num_experts, layout.num_ranks) != (T, num_experts, num_ranks):
        raise ValueError("layout was allocated for other sizes")
    st = layout.c_struct()
    _call(dev, "ep_get_layout",
          _ptr(topk_idx), T, K, num_experts, num_ranks, C.byref(st),
          _ptr(layout.workspace), layout.workspace.numel(), _stream(stream, dev))
    return layout


def ep_get_layout_noalloc(topk_idx: torch.Tensor, num_experts: int, num_ranks: int,
                          layout: Layout, stream=None) -> Layout:
    """ep_get_layout without a workspace: for callers that cannot allocate
    device memory when they call it.  The library's static scratch is used
    instead (``layout.workspace`` is ignored); the first call on a device
    should come before any stream capture, and calls must not overlap on
    the GPU."""
    _want(topk_idx, "topk_idx", torch.int64)
    T, K = topk_idx.shape
    if (layout.num_tokens, layout.num_experts, layout.num_ranks) != (T, num_experts, num_ranks):
        raise ValueError("layout was allocated for other sizes")
    st = layout.c_struct()
    _call(topk_idx.device, "ep_get_layout_noalloc",
          _ptr(topk_idx), T, K, num_experts, num_ranks, C.byref(st),
          _stream(stream, topk_idx.device))
    return layout


@dataclass
class Dispatched:
    recv_x: torch.Tensor                      # bf16 or float8_e4m3fn [cap, H]
    recv_x_scales: Optional[torch.Tensor]     # fp32 [cap, H/128] (fp8 only)
    recv_src_idx: Optional[torch.Tensor]      # int32 [cap]
    recv_topk_idx: Optional[torch.Tensor]     # int32 [cap, K]
    recv_topk_weights: Optional[torch.Tensor]  # fp32 [cap, K]


_DTYPES = {"bf16": N.EP_DTYPE_BF16, "fp8": N.EP_DTYPE_FP8_E4M3,
           "fp8_packed": N.EP_DTYPE_FP8_E4M3_PACKED}


def _dispatch_outputs(x, topk_idx, topk_weights, E, R, code, recv_capacity, out, metadata,
                      cumulative_recv_stats):
    """Checks the dispatch arguments and allocates the outputs not given."""
    _want(x, "x", torch.bfloat16)
    dev = x.device
    _want(topk_idx, "topk_idx", torch.int64, dev)
    T, H = x.shape
    K = topk_idx.shape[1]
    fp8 = code != N.EP_DTYPE_BF16
    packed = code == N.EP_DTYPE_FP8_E4M3_PACKED
    if recv_capacity is None:
        recv_capacity = out.recv_x.shape[0] if out is not None else T * min(K, R)
    if out is None:
        if packed:
            rx = torch.empty((recv_capacity, ep_fp8_packed_row_bytes(H)), dtype=torch.uint8, device=dev)
        else:
            rx = torch.empty((recv_capacity, H), dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16,
                             device=dev)
        out = Dispatched(
            rx,
            torch.empty((recv_capacity, H // EP_FP8_GROUP), dtype=torch.float32, device=dev)
            if fp8 and not packed else None,
            torch.empty(recv_capacity, dtype=torch.int32, device=dev) if metadata else None,
            torch.empty((recv_capacity, K), dtype=torch.int32, device=dev) if metadata else None,
            torch.empty((recv_capacity, K), dtype=torch.float32, device=dev)
            if metadata and topk_weights is not None else None)
    if topk_weights is not None:
        _want(topk_weights, "topk_weights", torch.float32, dev)
    _want(out.recv_x, "recv_x",
          torch.uint8 if packed else torch.float8_e4m3fn if fp8 else torch.bfloat16, dev)
    if out.recv_x.shape[0] < recv_capacity:
        raise ValueError("recv_x has fewer rows than recv_capacity")
    if cumulative_recv_stats is not None:
        if cumulative_recv_stats.dtype not in (torch.int32, torch.uint32) or \
                cumulative_recv_stats.numel() != E or not cumulative_recv_stats.is_cuda:
            raise ValueError("cumulative_recv_stats must be a 32-bit CUDA tensor of num_experts entries")
    return out, recv_capacity


def _dispatch_args(x, topk_idx, topk_weights, E, R, st, code, out, recv_capacity, stats):
    T, H = x.shape
    return N.ep_dispatch_args_t(
        x.data_ptr(), T, H, topk_idx.data_ptr(),
        None if topk_weights is None else topk_weights.data_ptr(), topk_idx.shape[1], E, R,
        C.pointer(st), code, out.recv_x.data_ptr(),
        None if out.recv_x_scales is None else out.recv_x_scales.data_ptr(),
        None if out.recv_src_idx is None else out.recv_src_idx.data_ptr(),
        None if out.recv_topk_idx is None else out.recv_topk_idx.data_ptr(),
        None if out.recv_topk_weights is None else out.recv_topk_weights.data_ptr(),
        recv_capacity, None if stats is None else stats.data_ptr())


def ep_dispatch(x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: Optional[torch.Tensor],
                layout: Layout, dtype: str = "bf16", recv_capacity: Optional[int] = None,
                out: Optional[Dispatched] = None, metadata: bool = True,
                cumulative_recv_stats: Optional[torch.Tensor] = None,
                stream=None) -> Dispatched:
    """Scatter rows of ``x`` (bf16 [T, H]) to their received slots.

    ``dtype`` is "bf16", "fp8" (e4m3 rows + a separate scale array) or
    "fp8_packed" (codes, scales and padding in one uint8 row of
    ``ep_fp8_packed_row_bytes(H)`` bytes).  Without ``recv_capacity`` the
    buffers are sized T * min(K, R), which needs no read-back of the layout.
    ``cumulative_recv_stats`` (uint32 [E]) is accumulated in place.  The
    plain C entry point ep_dispatch serves the options it has; the others go
    through ep_dispatch_ex.
    """
    E, R = layout.num_experts, layout.num_ranks
    code = _DTYPES[dtype]
    out, recv_capacity = _dispatch_outputs(x, topk_idx, topk_weights, E, R, code, recv_capacity, out,
                                           metadata, cumulative_recv_stats)
    dev = x.device
    T, H = x.shape
    K = topk_idx.shape[1]
    st = layout.c_struct()
    if code == N.EP_DTYPE_FP8_E4M3_PACKED or cumulative_recv_stats is not None:
        args = _dispatch_args(x, topk_idx, topk_weights, E, R, st, code, out, recv_capacity,
                              cumulative_recv_stats)
        _call(dev, "ep_dispatch_ex", C.byref(args), _stream(stream, dev))
    else:
        _call(dev, "ep_dispatch",
              _ptr(x), T, H, _ptr(topk_idx), _ptr(topk_weights), K, E, R, C.byref(st), code,
              _ptr(out.recv_x), _ptr(out.recv_x_scales), _ptr(out.recv_src_idx),
              _ptr(out.recv_topk_idx), _ptr(out.recv_topk_weights), recv_capacity,
              _stream(stream, dev))
    return out


def ep_get_layout_and_dispatch(x: torch.Tensor, topk_idx: torch.Tensor,
                               topk_weights: Optional[torch.Tensor], num_experts: int, num_ranks: int,
                               layout: Optional[Layout] = None, dtype: str = "fp8",
                               recv_capacity: Optional[int] = None, out: Optional[Dispatched] = None,
                               metadata: bool = True,
                               cumulative_recv_stats: Optional[torch.Tensor] = None,
                               stream=None, work_counters: bool = True):
    """ep_get_layout then ep_dispatch as one call: with fp8 rows the
    dispatch loads and casts its first rows while the layout kernel still
    runs.  Returns (layout, dispatched), both as the two calls give them."""
    T = topk_idx.shape[0]
    dev = x.device
    if layout is None:
        layout = Layout.empty(T, num_experts, num_ranks, dev, work_counters)
    elif (layout.num_tokens, layout.num_experts, layout.num_ranks) != (T, num_experts, num_ranks):
        raise ValueError("layout was allocated for other sizes")
    code = _DTYPES[dtype]
    out, recv_capacity = _dispatch_outputs(x, topk_idx, topk_weights, num_experts, num_ranks, code,
                                           recv_capacity, out, metadata, cumulative_recv_stats)
    st = layout.c_struct()
    args = _dispatch_args(x, topk_idx, topk_weights, num_experts, num_ranks, st, code, out,
                          recv_capacity, cumulative_recv_stats)
    _call(dev, "ep_get_layout_and_dispatch",
          C.byref(args), _ptr(layout.workspace), layout.workspace.numel(), _stream(stream, dev))
    return layout, out


ep_dispatch_ex = ep_dispatch


def ep_combine(y: torch.Tensor, layout: Layout, topk_idx: Optional[torch.Tensor] = None,
               topk_weights: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               bias0: Optional[torch.Tensor] = None, bias1: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """out[t] = bf16(bias0 + bias1 + sum over ranks r ascending of
    c[t,r] * y[token_slot[t,r]]), accumulated in fp32 in that order.

    Without weights c = 1; with ``topk_idx``/``topk_weights`` c[t,r] is the
    sum of t's gate weights on rank r.  The biases (bf16 [T, H]) are
    optional and go through ep_combine_ex.
    """
    _want(y, "y", torch.bfloat16)
    dev = y.device
    cap, H = y.shape
    T, R = layout.num_tokens, layout.num_ranks
    if (topk_idx is None) != (topk_weights is None):
        raise ValueError("pass both topk_idx and topk_weights, or neither")
    K = 0
    if topk_idx is not None:
        _want(topk_idx, "topk_idx", torch.int64, dev)
        _want(topk_weights, "topk_weights", torch.float32, dev)
        K = topk_idx.shape[1]
    for name, b in (("bias0", bias0), ("bias1", bias1)):
        if b is not None:
            _want(b, name, torch.bfloat16, dev)
            if tuple(b.shape) != (T, H):
                raise ValueError(f"{name} must be [num_tokens, hidden]")
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    _want(out, "out", torch.bfloat16, dev)
    st = layout.c_struct()
    if bias0 is not None or bias1 is not None:
        args = N.ep_combine_args_t(
            y.data_ptr(), cap, H, C.pointer(st), T, R,
            None if topk_idx is None else topk_idx.data_ptr(),
            None if topk_weights is None else topk_weights.data_ptr(), K, layout.num_experts,
            None if bias0 is None else bias0.data_ptr(),
            None if bias1 is None else bias1.data_ptr(), out.data_ptr())
        _call(dev, "ep_combine_ex", C.byref(args), _stream(stream, dev))
    else:
        _call(dev, "ep_combine",
              _ptr(y), cap, H, C.byref(st), T, R, _ptr(topk_idx), _ptr(topk_weights), K,
              layout.num_experts, _ptr(out), _stream(stream, dev))
    return out


ep_combine_ex = ep_combine


# ------------------------------------------------------------------ expanded

def ep_expanded_layout_workspace_bytes(num_tokens: int, num_experts: int) -> int:
    return int(N.load().ep_expanded_layout_workspace_bytes(num_tokens, num_experts))


@dataclass
class ExpandedLayout:
    """Device tensors of an expanded (one row per (token, expert)) layout."""
    num_rows_per_expert: torch.Tensor  # int32 [E]
    expert_offset: torch.Tensor        # int32 [E+1]
    token_slot: torch.Tensor           # int32 [T, K]
    error_word: torch.Tensor           # int32 [1]
    workspace: torch.Tensor            # uint8, zero-filled once
    num_tokens: int
    num_topk: int
    num_experts: int
    expert_alignment: int
    work_counters: Optional[torch.Tensor] = None  # int32 [4]: blocks draw tokens from a counter

    @staticmethod
    def empty(num_tokens: int, num_topk: int, num_experts: int, expert_alignment: int,
              device, work_counters: bool = True) -> "ExpandedLayout":
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        ws = ep_expanded_layout_workspace_bytes(num_tokens, num_experts)
        return ExpandedLayout(
            torch.empty(num_experts, **i32), torch.empty(num_experts + 1, **i32),
            torch.empty((num_tokens, num_topk), **i32), torch.zeros(1, **i32),
            torch.zeros(max(ws, 16), dtype=torch.uint8, device=dev),
            num_tokens, num_topk, num_experts, expert_alignment,
            torch.zeros(N.EP_WORK_COUNTER_WORDS, **i32) if work_counters else None)

    def c_struct(self) -> N.ep_expanded_layout_t:
        return N.ep_expanded_layout_t(
            self.num_rows_per_expert.data_ptr(), self.expert_offset.data_ptr(),
            self.token_slot.data_ptr(), self.error_word.data_ptr(),
            None if self.work_counters is None else self.work_counters.data_ptr())

    def num_rows(self) -> int:
        """Rows including padding, read back to the host (synchronises)."""
        return int(self.expert_offset[self.num_experts].item())

    def errors(self) -> int:
        return int(self.error_word.item()) & 0xffffffff

    def capacity_bound(self) -> int:
        """Rows that always suffice, without a read-back."""
        return self.num_tokens * self.num_topk + self.num_experts * (self.expert_alignment - 1)


def ep_get_layout_expanded(topk_idx: torch.Tensor, num_experts: int, expert_alignment: int = 1,
                           layout: Optional[ExpandedLayout] = None, stream=None,
                           work_counters: bool = True) -> ExpandedLayout:
    _want(topk_idx, "topk_idx", torch.int64)
    T, K = topk_idx.shape
    dev = topk_idx.device
    if layout is None:
        layout = ExpandedLayout.empty(T, K, num_experts, expert_alignment, dev, work_counters)
    elif (layout.num_tokens, layout.num_topk, layout.num_experts) != (T, K, num_experts):
        raise ValueError("layout was allocated for other sizes")
    layout.expert_alignment = expert_alignment
    st = layout.c_struct()
    _call(dev, "ep_get_layout_expanded",
          _ptr(topk_idx), T, K, num_experts, expert_alignment, C.byref(st), _ptr(layout.workspace),
          layout.workspace.numel(), _stream(stream, dev))
    return layout


def ep_dispatch_expanded(x: torch.Tensor, topk_idx: torch.Tensor,
                         topk_weights: Optional[torch.Tensor], layout: ExpandedLayout,
                         num_ranks: int, dtype: str = "bf16", recv_capacity: Optional[int] = None,
                         zero_padding: bool = True, out: Optional[Dispatched] = None,
                         metadata: bool = True,
                         cumulative_recv_stats: Optional[torch.Tensor] = None,
                         stream=None) -> Dispatched:
    """One row per (token, expert), grouped by expert (see ExpandedLayout)."""
    _want(x, "x", torch.bfloat16)
    dev = x.device
    _want(topk_idx, "topk_idx", torch.int64, dev)
    T, H = x.shape
    K = topk_idx.shape[1]
    E = layout.num_experts
    code = _DTYPES[dtype]
    fp8 = code != N.EP_DTYPE_BF16
    packed = code == N.EP_DTYPE_FP8_E4M3_PACKED
    if recv_capacity is None:
        recv_capacity = out.recv_x.shape[0] if out is not None else layout.capacity_bound()
    if out is None:
        if packed:
            rx = torch.empty((recv_capacity, ep_fp8_packed_row_bytes(H)), dtype=torch.uint8, device=dev)
        else:
            rx = torch.empty((recv_capacity, H), dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16,
                             device=dev)
        out = Dispatched(
            rx,
            torch.empty((recv_capacity, H // EP_FP8_GROUP), dtype=torch.float32, device=dev)
            if fp8 and not packed else None,
            torch.empty(recv_capacity, dtype=torch.int32, device=dev) if metadata else None,
            torch.empty((recv_capacity, K), dtype=torch.int32, device=dev) if metadata else None,
            torch.empty((recv_capacity, K), dtype=torch.float32, device=dev)
            if metadata and topk_weights is not None else None)
    if topk_weights is not None:
        _want(topk_weights, "topk_weights", torch.float32, dev)
    st = layout.c_struct()
    args = N.ep_dispatch_expanded_args_t(
        x.data_ptr(), T, H, topk_idx.data_ptr(),
        None if topk_weights is None else topk_weights.data_ptr(), K, E, num_ranks,
        C.pointer(st), code, out.recv_x.data_ptr(),
        None if out.recv_x_scales is None else out.recv_x_scales.data_ptr(),
        None if out.recv_src_idx is None else out.recv_src_idx.data_ptr(),
        None if out.recv_topk_idx is None else out.recv_topk_idx.data_ptr(),
        None if out.recv_topk_weights is None else out.recv_topk_weights.data_ptr(),
        recv_capacity, 1 if zero_padding else 0,
        None if cumulative_recv_stats is None else cumulative_recv_stats.data_ptr())
    _call(dev, "ep_dispatch_expanded", C.byref(args), _stream(stream, dev))
    return out


def ep_combine_expanded(y: torch.Tensor, layout: ExpandedLayout,
                        topk_idx: Optional[torch.Tensor] = None,
                        topk_weights: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, bias0: Optional[torch.Tensor] = None,
                        bias1: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[t] = bf16(bias0 + bias1 + sum over t's rows, ascending, of c * y[row])."""
    _want(y, "y", torch.bfloat16)
    dev = y.device
    cap, H = y.shape
    T, K = layout.num_tokens, layout.num_topk
    if (topk_idx is None) != (topk_weights is None):
        raise ValueError("pass both topk_idx and topk_weights, or neither")
    if topk_idx is not None:
        _want(topk_idx, "topk_idx", torch.int64, dev)
        _want(topk_weights, "topk_weights", torch.float32, dev)
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    st = layout.c_struct()
    args = N.ep_combine_expanded_args_t(
        y.data_ptr(), cap, H, C.pointer(st), T, K,
        None if topk_idx is None else topk_idx.data_ptr(),
        None if topk_weights is None else topk_weights.data_ptr(), layout.num_experts,
        None if bias0 is None else bias0.data_ptr(), None if bias1 is None else bias1.data_ptr(),
        out.data_ptr())
    _call(dev, "ep_combine_expanded", C.byref(args), _stream(stream, dev))
    return out


# ---------------------------------------- router, experts' products, adapters

@dataclass
class Routing:
    """A batch's experts and weights, as the layouts and dispatches take them."""
    topk_idx: torch.Tensor      # int64 [T, K], -1 = no selection
    topk_weights: torch.Tensor  # fp32 [T, K]


_SCORES = {"softmax": N.EP_SCORE_SOFTMAX, "sigmoid": N.EP_SCORE_SIGMOID}
_LOGITS = {torch.float32: N.EP_LOGITS_FP32, torch.bfloat16: N.EP_LOGITS_BF16}
_ACTIVATIONS = {None: N.EP_ACT_NONE, "swiglu": N.EP_ACT_SWIGLU}


def _want_shape(t: torch.Tensor, name: str, shape: tuple):
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_functions = {}
_route_args = N.packer(N.ep_route_args_t)
_route_backward_args = N.packer(N.ep_route_backward_args_t)
_product_args = N.packer(N.ep_expert_product_args_t)
_product_backward_args = N.packer(N.ep_expert_product_backward_args_t)
_adapter_args = N.packer(N.ep_adapter_product_args_t)

# These calls can be shorter than their set-up in Python, so each wrapper
# looks at its tensors in one expression and lets a second function say what
# is wrong.  Tensors are on device `i` (get_device() is -1 off the GPU).


def _empty(shape, dtype, dev, stream):
    """A new tensor for work on ``stream``: its memory comes from that
    stream's, so neither what held it before nor what holds it next overlaps
    the work."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _launch(index: int, fn: str, args: bytes, stream):
    """``_call`` for functions of one argument block, packed, and a stream."""
    if stream is None:
        handle = _raw_stream(index)
    elif stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
    else:
        handle = stream.cuda_stream
    f = _functions.get(fn)
    if f is None:
        f = N.load()[fn]
        f.restype, f.argtypes = C.c_int, [C.c_char_p, C.c_void_p]
        _functions[fn] = f
    if _current() == index:
        status = f(args, handle)
    else:
        with torch.cuda.device(index):
            status = f(args, handle)
    if status:
        _check(status, fn)


def _logits_sizes(logits: torch.Tensor) -> tuple:
    """T, E and the row stride of logits [T, E] (rows may be apart, a row's
    entries may not)."""
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if logits.dtype not in _LOGITS:
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError("logits must be [num_tokens, num_experts]")
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    T, E = logits.shape
    apart, step = logits.stride()
    if (E > 1 and step != 1) or (T > 1 and apart < E):
        raise ValueError("a row of logits must be contiguous, and rows must not overlap")
    return T, E, apart if T > 1 else max(E, 1)


def ep_route(logits: torch.Tensor, num_topk: int, score: str = "softmax",
             bias: Optional[torch.Tensor] = None, num_groups: int = 1, topk_groups: int = 1,
             group_top: int = 1, renormalize: bool = True, weight_scale: float = 1.0,
             out: Optional[Routing] = None, stream=None) -> Routing:
    """Each token's experts and weights from the gate's logits (fp32 or bf16
    [T, E]; rows may be a slice of wider ones).

    ``score`` is "softmax" or "sigmoid".  ``bias`` (fp32 [E]) is added to the
    scores for the choice only.  With ``num_groups`` > 1 only the experts of
    the ``topk_groups`` best groups are offered, a group's score being the sum
    of its ``group_top`` (1 or 2) largest keys.  ``renormalize`` divides a
    token's weights by their sum; ``weight_scale`` multiplies them.  Experts
    with a logit of -infinity or NaN are never chosen; missing choices are -1
    with weight 0.  Ties go to the lowest index.
    """
    T, E, apart = _logits_sizes(logits)
    dev = logits.device
    if bias is not None and not (bias.dtype is torch.float32 and bias.device == dev
                                 and bias.is_contiguous() and bias.shape == (E,)):
        _want(bias, "bias", torch.float32, dev)
        _want_shape(bias, "bias", (E,))
    if out is None:
        idx = _empty((T, num_topk), torch.int64, dev, stream)
        out = Routing(idx, _empty((T, num_topk), torch.float32, dev, stream))
    else:
        for name, t, dtype in (("topk_idx", out.topk_idx, torch.int64),
                               ("topk_weights", out.topk_weights, torch.float32)):
            _want(t, name, dtype, dev)
            _want_shape(t, name, (T, num_topk))
    _launch(dev.index, "ep_route", _route_args(
        logits.data_ptr(), _LOGITS[logits.dtype], apart, T, E, num_topk, _SCORES[score],
        0 if bias is None else bias.data_ptr(), num_groups, topk_groups, group_top,
        1 if renormalize else 0, weight_scale, out.topk_idx.data_ptr(), out.topk_weights.data_ptr()),
        stream)
    return out


def ep_route_backward(grad_weights: torch.Tensor, logits: torch.Tensor, topk_idx: torch.Tensor,
                      score: str = "softmax", renormalize: bool = True, weight_scale: float = 1.0,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gradient of ``ep_route``'s weights for the logits ([T, E], the
    logits' dtype), given the weights' gradient (fp32 [T, K]) and the choice.
    The choice itself, and so the bias, has no gradient."""
    T, E, apart = _logits_sizes(logits)
    dev, i = logits.device, logits.get_device()
    K = topk_idx.shape[-1]
    if not (topk_idx.dtype is torch.int64 and grad_weights.dtype is torch.float32
            and topk_idx.get_device() == i and grad_weights.get_device() == i
            and topk_idx.is_contiguous() and grad_weights.is_contiguous()
            and topk_idx.shape == (T, K) and grad_weights.shape == (T, K)):
        _refuse_tensors((topk_idx, "topk_idx", torch.int64, dev, (T, K)),
                        (grad_weights, "grad_weights", torch.float32, dev, (T, K)))
    if out is None:
        out = _empty((T, E), logits.dtype, dev, stream)
    else:
        _want(out, "out", logits.dtype, dev)
        _want_shape(out, "out", (T, E))
    _launch(i, "ep_route_backward", _route_backward_args(
        grad_weights.data_ptr(), logits.data_ptr(), _LOGITS[logits.dtype], apart,
        topk_idx.data_ptr(), T, E, K, _SCORES[score], 1 if renormalize else 0, weight_scale,
        out.data_ptr()), stream)
    return out


def _refuse_tensors(*wanted):
    """Raises for the first of (tensor, name, dtype, device, shape) that is
    not so (None tensors pass)."""
    for t, name, dtype, dev, shape in wanted:
        if t is not None:
            _want(t, name, dtype, dev)
            _want_shape(t, name, shape)


def _product_sizes(x, w, layout, activation):
    """(capacity, hidden, width, wide) of rows and weights, checked, and the
    layout's tensors where they are."""
    bf = torch.bfloat16
    if not (x.dtype is bf and w.dtype is bf and x.is_cuda and x.get_device() == w.get_device()
            and x.is_contiguous() and w.is_contiguous()):
        _want(x, "x", bf)
        _want(w, "w", bf, x.device)
    i = x.get_device()
    if not (layout.num_rows_per_expert.get_device() == i and layout.expert_offset.get_device() == i
            and layout.error_word.get_device() == i):
        for name in ("num_rows_per_expert", "expert_offset", "error_word"):
            at = getattr(layout, name).device
            if at != x.device:
                raise ValueError(f"layout.{name} is on {at}, expected {x.device}")
    if x.dim() != 2 or w.dim() != 3:
        raise ValueError("x must be [recv_capacity, hidden] and w [num_experts, outputs, hidden]")
    cap, H = x.shape
    experts, wide, inner = w.shape
    if experts != layout.num_experts or inner != H:
        _want_shape(w, "w", (layout.num_experts, wide, H))
    if activation == "swiglu":
        if wide % 2:
            raise ValueError("w must have an even number of outputs with swiglu")
        return cap, H, wide // 2, wide
    return cap, H, wide, wide


def ep_expert_product(x: torch.Tensor, w: torch.Tensor, layout: ExpandedLayout,
                      activation: Optional[str] = None, out: Optional[torch.Tensor] = None,
                      preact: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Each expert's rows times its weights.

    ``x`` bf16 [cap, H] are rows grouped by expert (``ep_dispatch_expanded``
    with dtype "bf16"), ``w`` bf16 [E, N, H].  Returns bf16 [cap, N], or with
    ``activation="swiglu"`` [cap, N/2]: silu of the first half of the outputs
    times the second.  ``preact`` (bf16 [cap, N]) receives the outputs before
    the activation, which the backward pass needs.  Padding rows and rows past
    the last are not written.  Sums are fp32.
    """
    act = _ACTIVATIONS[activation]
    cap, H, width, wide = _product_sizes(x, w, layout, activation)
    bf, dev = torch.bfloat16, x.device
    if out is None:
        out = _empty((cap, width), bf, dev, stream)
    elif not (out.dtype is bf and out.device == dev and out.is_contiguous() and out.shape == (cap, width)):
        _refuse_tensors((out, "out", bf, dev, (cap, width)))
    if preact is not None:
        _refuse_tensors((preact, "preact", bf, dev, (cap, wide)))
    lay = layout.c_struct()
    _launch(dev.index, "ep_expert_product", _product_args(
        x.data_ptr(), cap, layout.num_tokens, H, layout.num_experts, C.addressof(lay),
        w.data_ptr(), width, act, out.data_ptr(), 0 if preact is None else preact.data_ptr()), stream)
    return out


def ep_expert_product_backward(grad: torch.Tensor, x: torch.Tensor, w: torch.Tensor,
                               layout: ExpandedLayout, activation: Optional[str] = None,
                               preact: Optional[torch.Tensor] = None,
                               grad_x: Optional[torch.Tensor] = None,
                               grad_w: Optional[torch.Tensor] = None, need_x: bool = True,
                               need_w: bool = True, grad_preact: Optional[torch.Tensor] = None,
                               stream=None):
    """(grad_x, grad_w) of ``ep_expert_product`` for the output's gradient
    ``grad`` (bf16 [cap, width]); either is None when not needed.  With swiglu
    ``preact`` is what the forward pass kept, and ``grad_preact`` (bf16 like
    it, allocated when not given) receives its gradient.  Rows of ``grad_x``
    outside the layout's are not written; ``grad_w`` of an expert without rows
    is zero."""
    act = _ACTIVATIONS[activation]
    cap, H, width, wide = _product_sizes(x, w, layout, activation)
    bf, dev, i = torch.bfloat16, x.device, x.get_device()
    if not (grad.dtype is bf and grad.get_device() == i and grad.is_contiguous() and grad.shape == (cap, width)):
        _refuse_tensors((grad, "grad", bf, dev, (cap, width)))
    if act == N.EP_ACT_SWIGLU:
        if preact is None:
            raise ValueError("swiglu needs preact")
        if not (preact.dtype is bf and preact.get_device() == i and preact.is_contiguous()
                and preact.shape == (cap, wide)):
            _refuse_tensors((preact, "preact", bf, dev, (cap, wide)))
        if grad_preact is None:
            grad_preact = _empty((cap, wide), bf, dev, stream)
        else:
            _refuse_tensors((grad_preact, "grad_preact", bf, dev, (cap, wide)))
    else:
        preact = grad_preact = None
    if not need_x:
        grad_x = None
    elif grad_x is None:
        grad_x = _empty((cap, H), bf, dev, stream)
    else:
        _refuse_tensors((grad_x, "grad_x", bf, dev, (cap, H)))
    if not need_w:
        grad_w = None
    elif grad_w is None:
        grad_w = _empty(w.shape, bf, dev, stream)
    else:
        _refuse_tensors((grad_w, "grad_w", bf, dev, w.shape))
    lay = layout.c_struct()
    _launch(i, "ep_expert_product_backward", _product_backward_args(
        grad.data_ptr(), x.data_ptr(), w.data_ptr(), cap, layout.num_tokens, H, layout.num_experts,
        C.addressof(lay), width, act, 0 if preact is None else preact.data_ptr(),
        0 if grad_preact is None else grad_preact.data_ptr(),
        0 if grad_x is None else grad_x.data_ptr(), 0 if grad_w is None else grad_w.data_ptr()), stream)
    return grad_x, grad_w


@lru_cache(maxsize=256)
def ep_adapter_workspace_bytes(num_rows: int, hidden: int, rank: int) -> int:
    return int(N.load().ep_adapter_workspace_bytes(num_rows, hidden, rank))


def ep_adapter_product(x: torch.Tensor, w: torch.Tensor, lora_a: torch.Tensor, lora_b: torch.Tensor,
                       adapter_idx: torch.Tensor, adapter_scale: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                       error_word: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x w^T plus, for each row, its own adapter's low-rank term
    ``scale[a] * (x A_a^T) B_a^T`` with a = ``adapter_idx`` (int64 [T], -1 =
    none).  ``x`` bf16 [T, H], ``w`` bf16 [N, H], ``lora_a`` bf16 [A, r, H],
    ``lora_b`` bf16 [A, N, r], ``adapter_scale`` fp32 [A] (1 when not given).
    An index outside [-1, A) counts as -1 and sets EP_ERRBIT_BAD_INDEX in
    ``error_word`` (int32 [1], if given).  Returns bf16 [T, N]."""
    bf = torch.bfloat16
    _want(x, "x", bf)
    if x.dim() != 2 or w.dim() != 2 or lora_a.dim() != 3:
        raise ValueError("x must be [rows, hidden], w [outputs, hidden], lora_a [adapters, rank, hidden]")
    T, H = x.shape
    A, r, _ = lora_a.shape
    width = w.shape[0]
    dev, i = x.device, x.get_device()
    if not (w.dtype is bf and lora_a.dtype is bf and lora_b.dtype is bf and adapter_idx.dtype is torch.int64
            and w.get_device() == i and lora_a.get_device() == i and lora_b.get_device() == i
            and adapter_idx.get_device() == i and w.is_contiguous() and lora_a.is_contiguous()
            and lora_b.is_contiguous() and adapter_idx.is_contiguous() and w.shape == (width, H)
            and lora_a.shape == (A, r, H) and lora_b.shape == (A, width, r) and adapter_idx.shape == (T,)):
        _refuse_tensors((w, "w", bf, dev, (width, H)), (lora_a, "lora_a", bf, dev, (A, r, H)),
                        (lora_b, "lora_b", bf, dev, (A, width, r)),
                        (adapter_idx, "adapter_idx", torch.int64, dev, (T,)))
    if adapter_scale is not None and not (
            adapter_scale.dtype is torch.float32 and adapter_scale.get_device() == i
            and adapter_scale.is_contiguous() and adapter_scale.shape == (A,)):
        _refuse_tensors((adapter_scale, "adapter_scale", torch.float32, dev, (A,)))
    if error_word is not None:
        _want(error_word, "error_word", torch.int32, dev)
    if out is None:
        out = _empty((T, width), bf, dev, stream)
    else:
        _refuse_tensors((out, "out", bf, dev, (T, width)))
    if workspace is None:
        nbytes = ep_adapter_workspace_bytes(T, H, r) or 16
        workspace = _empty(nbytes, torch.uint8, dev, stream)
    else:
        _want(workspace, "workspace", torch.uint8, dev)
        nbytes = workspace.numel()
    _launch(i, "ep_adapter_product", _adapter_args(
        x.data_ptr(), T, H, w.data_ptr(), width, lora_a.data_ptr(), lora_b.data_ptr(), A, r,
        adapter_idx.data_ptr(), 0 if adapter_scale is None else adapter_scale.data_ptr(),
        out.data_ptr(), workspace.data_ptr(), nbytes, 0 if error_word is None else error_word.data_ptr()),
        stream)
    return out


# ------------------- the block around the layer: losses, norm, shared product

@dataclass
class Balance:
    """A batch's balance and z loss, and what they were made of."""
    losses: torch.Tensor  # fp32 [2]: balance, z
    counts: torch.Tensor  # int32 [S, E]: choices of each expert
    probs: torch.Tensor   # fp32 [S, E]: its mean score
    slopes: torch.Tensor  # fp32 [S, E]: the balance loss's derivative for a token's score


_TYPES = {torch.float32: N.EP_TYPE_FP32, torch.bfloat16: N.EP_TYPE_BF16}
_DENSE_ACTIVATIONS = {None: N.EP_ACT_NONE, "swiglu": N.EP_ACT_SWIGLU, "relu": N.EP_ACT_RELU, "silu": N.EP_ACT_SILU,
                      "gelu": N.EP_ACT_GELU, "gelu_tanh": N.EP_ACT_GELU_TANH}
_balance_args = N.packer(N.ep_balance_loss_args_t)
_balance_backward_args = N.packer(N.ep_balance_loss_backward_args_t)
_norm_args = N.packer(N.ep_layer_norm_args_t)
_norm_backward_args = N.packer(N.ep_layer_norm_backward_args_t)
_dense_args = N.packer(N.ep_dense_product_args_t)
_dense_backward_args = N.packer(N.ep_dense_product_backward_args_t)


def _good(t, dtype, i, shape):
    """A contiguous tensor of this type and shape on device ``i``."""
    return t.dtype is dtype and t.get_device() == i and t.is_contiguous() and t.shape == shape


def _address(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _given(t, name, dtype, dev, shape):
    """An optional tensor, refused if it is not so."""
    if t is not None and not (isinstance(t, torch.Tensor) and _good(t, dtype, dev.index, shape)):
        _refuse_tensors((t, name, dtype, dev, shape))


def _target(t, name, dtype, dev, shape, stream):
    """An output: checked if it is given, else a new tensor."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev) if stream is None else _empty(shape, dtype, dev, stream)
    _given(t, name, dtype, dev, shape)
    return t


def _scratch(workspace, nbytes, dev, stream):
    """A workspace and its bytes."""
    if workspace is None:
        return _empty(nbytes or 16, torch.uint8, dev, stream), nbytes or 16
    _want(workspace, "workspace", torch.uint8, dev)
    return workspace, workspace.numel()


def _rows(x: torch.Tensor, name: str, dtypes) -> tuple:
    """Rows, their length and their distance in a matrix [T, H] of a type in
    ``dtypes`` (rows may be apart, a row's entries may not)."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {x.dtype}")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must have two dimensions")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    T, H = shape
    if x.is_contiguous():
        return T, H, H
    apart, step = x.stride()
    if (H > 1 and step != 1) or (T > 1 and apart < H):
        raise ValueError(f"a row of {name} must be contiguous, and rows must not overlap")
    return T, H, apart if T > 1 else H


def _sequences(seq_offsets, dev) -> int:
    if seq_offsets is None:
        return 1
    _want(seq_offsets, "seq_offsets", torch.int32, dev)
    if seq_offsets.dim() != 1 or seq_offsets.shape[0] < 2:
        raise ValueError("seq_offsets must be [num_sequences + 1]")
    return seq_offsets.shape[0] - 1


@lru_cache(maxsize=256)
def ep_balance_workspace_bytes(num_tokens: int, num_experts: int, num_sequences: int) -> int:
    return int(N.load().ep_balance_workspace_bytes(num_tokens, num_experts, num_sequences))


def ep_balance_loss(logits: torch.Tensor, topk_idx: torch.Tensor, score: str = "softmax",
                    seq_offsets: Optional[torch.Tensor] = None, out: Optional[Balance] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> Balance:
    """The router's balance and z loss, and each expert's counts, from the
    gate's logits (as ``ep_route`` takes them) and the choice (int64 [T, K]).

    With ``seq_offsets`` (int32 [S + 1], ascending) the sequences
    ``[seq_offsets[s], seq_offsets[s + 1])`` are balanced one by one and the
    losses averaged; tokens in none of them take no part.  ``score`` is
    "softmax", or "sigmoid" (divided by its sum).  ``losses`` are the mean of
    E times the sum of each expert's share of the choices times its mean score
    (1 when balanced), and the mean square of the logits' log-sum-exp.
    """
    T, E, apart = _logits_sizes(logits)
    dev, i = logits.device, logits.get_device()
    S = _sequences(seq_offsets, dev)
    if topk_idx.dim() != 2 or not _good(topk_idx, torch.int64, i, (T, topk_idx.shape[1])):
        _refuse_tensors((topk_idx, "topk_idx", torch.int64, dev, (T, topk_idx.shape[-1])))
    if out is None:  # (views of one tensor take longer than tensors of their own)
        out = Balance(_empty(2, torch.float32, dev, stream), _empty((S, E), torch.int32, dev, stream),
                      _empty((S, E), torch.float32, dev, stream), _empty((S, E), torch.float32, dev, stream))
    else:
        _refuse_tensors((out.losses, "losses", torch.float32, dev, (2,)), (out.counts, "counts", torch.int32, dev, (S, E)),
                        (out.probs, "probs", torch.float32, dev, (S, E)),
                        (out.slopes, "slopes", torch.float32, dev, (S, E)))
    workspace, nbytes = _scratch(workspace, ep_balance_workspace_bytes(T, E, S) if workspace is None else 0, dev, stream)
    _launch(i, "ep_balance_loss", _balance_args(
        logits.data_ptr(), _LOGITS[logits.dtype], apart, topk_idx.data_ptr(), T, E, topk_idx.shape[1], _SCORES[score],
        _address(seq_offsets), S, out.losses.data_ptr(), out.counts.data_ptr(), out.probs.data_ptr(),
        out.slopes.data_ptr(), workspace.data_ptr(), nbytes), stream)
    return out


def ep_balance_loss_backward(grad_losses: torch.Tensor, logits: torch.Tensor, balance: Balance, score: str = "softmax",
                             seq_offsets: Optional[torch.Tensor] = None, add: Optional[torch.Tensor] = None,
                             out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gradient of ``ep_balance_loss``'s losses for the logits ([T, E],
    the logits' dtype), given theirs (fp32 [2]) and what the forward call
    returned, plus ``add`` ([T, E], for one what ``ep_route_backward`` gave).
    ``out`` may be ``add`` or ``logits``.  The choice is held fixed."""
    T, E, apart = _logits_sizes(logits)
    dev, i = logits.device, logits.get_device()
    S = _sequences(seq_offsets, dev)
    if not (_good(grad_losses, torch.float32, i, (2,)) and _good(balance.slopes, torch.float32, i, (S, E))):
        _refuse_tensors((grad_losses, "grad_losses", torch.float32, dev, (2,)),
                        (balance.slopes, "balance.slopes", torch.float32, dev, (S, E)))
    dtype, shape = logits.dtype, (T, E)
    if not ((add is None or _good(add, dtype, i, shape)) and (out is None or _good(out, dtype, i, shape))):
        _refuse_tensors((add, "add", dtype, dev, shape), (out, "out", dtype, dev, shape))
    if out is None:
        out = _empty(shape, dtype, dev, stream)
    _launch(i, "ep_balance_loss_backward", _balance_backward_args(
        grad_losses.data_ptr(), logits.data_ptr(), _LOGITS[dtype], apart, T, E, _SCORES[score],
        0 if seq_offsets is None else seq_offsets.data_ptr(), S, balance.slopes.data_ptr(),
        0 if add is None else add.data_ptr(), out.data_ptr()), stream)
    return out


def _norm_params(weight, bias, H, dev) -> torch.dtype:
    """The type of a norm's weight and bias, checked."""
    dtype = torch.float32
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            if t.dtype not in _TYPES:
                raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
            dtype = t.dtype
            break
    _given(weight, "weight", dtype, dev, (H,))
    _given(bias, "bias", dtype, dev, (H,))
    return dtype


def ep_layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                  eps: float = 1e-5, out: Optional[torch.Tensor] = None, mean: Optional[torch.Tensor] = None,
                  rstd: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Layer norm of the rows of ``x`` (bf16 or fp32 [T, H]; rows may be a
    slice of wider ones), times ``weight`` plus ``bias`` (fp32 or bf16 [H],
    both alike).  Returns [T, H] in x's type; ``mean`` and ``rstd`` (fp32 [T])
    receive the rows' statistics, which the backward pass needs."""
    T, H, apart = _rows(x, "x", _TYPES)
    dev, i, dtype, f32 = x.device, x.get_device(), x.dtype, torch.float32
    first = bias if weight is None else weight
    params = f32 if first is None else first.dtype
    if not (params in _TYPES and (weight is None or _good(weight, params, i, (H,)))
            and (bias is None or _good(bias, params, i, (H,)))
            and (mean is None or _good(mean, f32, i, (T,))) and (rstd is None or _good(rstd, f32, i, (T,)))):
        _norm_params(weight, bias, H, dev)
        _refuse_tensors((mean, "mean", f32, dev, (T,)), (rstd, "rstd", f32, dev, (T,)))
    if out is None:
        out = _empty((T, H), dtype, dev, stream)
    elif not _good(out, dtype, i, (T, H)):
        _refuse_tensors((out, "out", dtype, dev, (T, H)))
    _launch(i, "ep_layer_norm", _norm_args(
        x.data_ptr(), _TYPES[dtype], apart, T, H, 0 if weight is None else weight.data_ptr(),
        0 if bias is None else bias.data_ptr(), _TYPES[params], eps, out.data_ptr(), 0 if mean is None else mean.data_ptr(),
        0 if rstd is None else rstd.data_ptr()), stream)
    return out


@lru_cache(maxsize=256)
def ep_layer_norm_workspace_bytes(num_rows: int, hidden: int) -> int:
    return int(N.load().ep_layer_norm_workspace_bytes(num_rows, hidden))


def ep_layer_norm_backward(grad: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                           weight: Optional[torch.Tensor] = None, add: Optional[torch.Tensor] = None,
                           grad_x: Optional[torch.Tensor] = None, grad_weight: Optional[torch.Tensor] = None,
                           grad_bias: Optional[torch.Tensor] = None, need_x: bool = True, need_params: bool = True,
                           workspace: Optional[torch.Tensor] = None, stream=None):
    """(grad_x, grad_weight, grad_bias) of ``ep_layer_norm`` for the output's
    gradient ``grad`` ([T, H], x's type) and the statistics that the forward
    call kept; what is not needed is None.  ``add`` ([T, H], x's type: the
    gradient of a residual around the norm) is added to grad_x.  The
    parameters' gradients (fp32 sums over the rows) have the weight's type,
    fp32 without one, or that of the tensors given for them."""
    T, H, apart = _rows(x, "x", _TYPES)
    dev, i = x.device, x.get_device()
    dtype, f32 = x.dtype, torch.float32
    if not (_good(grad, dtype, i, (T, H)) and _good(mean, f32, i, (T,)) and _good(rstd, f32, i, (T,))):
        _refuse_tensors((grad, "grad", dtype, dev, (T, H)), (mean, "mean", f32, dev, (T,)), (rstd, "rstd", f32, dev, (T,)))
    params = f32 if weight is None else weight.dtype
    if weight is not None and not (params in _TYPES and _good(weight, params, i, (H,))):
        _norm_params(weight, None, H, dev)
    if weight is None and need_params and (grad_weight is not None or grad_bias is not None):
        params = _norm_params(grad_weight, grad_bias, H, dev)
    if add is not None and not _good(add, dtype, i, (T, H)):
        _refuse_tensors((add, "add", dtype, dev, (T, H)))
    if not need_x:
        grad_x = None
    elif grad_x is None:
        grad_x = _empty((T, H), dtype, dev, stream)
    elif not _good(grad_x, dtype, i, (T, H)):
        _refuse_tensors((grad_x, "grad_x", dtype, dev, (T, H)))
    nbytes = 0
    if need_params:
        grad_weight = _target(grad_weight, "grad_weight", params, dev, (H,), stream)
        grad_bias = _target(grad_bias, "grad_bias", params, dev, (H,), stream)
        workspace, nbytes = _scratch(workspace, ep_layer_norm_workspace_bytes(T, H) if workspace is None else 0, dev, stream)
    else:
        grad_weight = grad_bias = workspace = None
    _launch(i, "ep_layer_norm_backward", _norm_backward_args(
        grad.data_ptr(), x.data_ptr(), _TYPES[dtype], apart, T, H, mean.data_ptr(), rstd.data_ptr(), _address(weight),
        _TYPES[params], _address(add), _address(grad_x), _address(grad_weight), _address(grad_bias), _address(workspace),
        nbytes), stream)
    return grad_x, grad_weight, grad_bias


def _dense_sizes(x, w, activation) -> tuple:
    """(rows, hidden, x's row distance, width, wide) of a shared product."""
    bf = torch.bfloat16
    T, H, apart = _rows(x, "x", (bf,))
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be [outputs, hidden]")
    wide = w.shape[0]
    if not _good(w, bf, x.get_device(), (wide, H)):
        _refuse_tensors((w, "w", bf, x.device, (wide, H)))
    if activation == "swiglu":
        if wide % 2:
            raise ValueError("w must have an even number of outputs with swiglu")
        return T, H, apart, wide // 2, wide
    return T, H, apart, wide, wide


def ep_dense_product(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                     activation: Optional[str] = None, residual: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, preact: Optional[torch.Tensor] = None,
                     out_dtype: torch.dtype = torch.bfloat16, error_word: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """act(x w^T + bias) + residual, a product shared by all rows.

    ``x`` bf16 [T, H] (rows may be a slice of wider ones, a multiple of 8
    apart; H is one too), ``w`` bf16 [N, H], ``bias`` fp32 or bf16 [N].  ``activation`` is
    None, "relu", "silu", "gelu" (by erf), "gelu_tanh", or "swiglu": silu of
    the first half of the outputs times the second, [T, N/2].  ``residual``
    (bf16 like the output's shape) may be ``out``.  The output is bf16, or
    fp32 with ``out_dtype`` (a gate's logits); sums are fp32, rounded once.
    ``preact`` (bf16 [T, N]) receives x w^T + bias, which the backward pass of
    an activation needs."""
    act = _DENSE_ACTIVATIONS[activation]
    T, H, apart, width, wide = _dense_sizes(x, w, activation)
    bf, dev, i = torch.bfloat16, x.device, x.get_device()
    bias_type = N.EP_TYPE_FP32
    if bias is not None:
        if bias.dtype not in _TYPES:
            raise TypeError(f"bias must be float32 or bfloat16, got {bias.dtype}")
        if not _good(bias, bias.dtype, i, (wide,)):
            _refuse_tensors((bias, "bias", bias.dtype, dev, (wide,)))
        bias_type = _TYPES[bias.dtype]
    if out is not None:
        out_dtype = out.dtype
    if out_dtype not in _TYPES:
        raise TypeError(f"the output must be float32 or bfloat16, not {out_dtype}")
    if not ((residual is None or _good(residual, bf, i, (T, width))) and (preact is None or _good(preact, bf, i, (T, wide)))):
        _refuse_tensors((residual, "residual", bf, dev, (T, width)), (preact, "preact", bf, dev, (T, wide)))
    if error_word is not None:
        _want(error_word, "error_word", torch.int32, dev)
    if out is None:
        out = _empty((T, width), out_dtype, dev, stream)
    elif not _good(out, out_dtype, i, (T, width)):
        _refuse_tensors((out, "out", out_dtype, dev, (T, width)))
    _launch(i, "ep_dense_product", _dense_args(
        x.data_ptr(), apart, T, H, w.data_ptr(), width, 0 if bias is None else bias.data_ptr(), bias_type, act,
        0 if residual is None else residual.data_ptr(), out.data_ptr(), _TYPES[out_dtype],
        0 if preact is None else preact.data_ptr(), 0 if error_word is None else error_word.data_ptr()), stream)
    return out


@lru_cache(maxsize=256)
def ep_dense_workspace_bytes(num_rows: int, hidden: int, width: int, activation: Optional[str] = None) -> int:
    return int(N.load().ep_dense_workspace_bytes(num_rows, hidden, width, _DENSE_ACTIVATIONS[activation]))


def ep_dense_product_backward(grad: torch.Tensor, x: torch.Tensor, w: torch.Tensor, activation: Optional[str] = None,
                              preact: Optional[torch.Tensor] = None, bias_dtype: Optional[torch.dtype] = None,
                              grad_x: Optional[torch.Tensor] = None, grad_w: Optional[torch.Tensor] = None,
                              grad_bias: Optional[torch.Tensor] = None, need_x: bool = True, need_w: bool = True,
                              grad_preact: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                              error_word: Optional[torch.Tensor] = None, stream=None):
    """(grad_x, grad_w, grad_bias) of ``ep_dense_product`` for the output's
    gradient ``grad`` ([T, width], bf16 or fp32); what is not needed is None.
    The bias's is computed for a ``bias_dtype`` (or a ``grad_bias`` tensor).
    With an activation ``preact`` is what the forward pass kept;
    ``grad_preact`` (bf16 [T, N], N rounded up to a multiple of 8, allocated
    when not given and needed) receives its gradient, rounded as the products
    take it.  A residual's gradient is
    ``grad`` itself."""
    act = _DENSE_ACTIVATIONS[activation]
    T, H, apart, width, wide = _dense_sizes(x, w, activation)
    bf, dev, i = torch.bfloat16, x.device, x.get_device()
    if not isinstance(grad, torch.Tensor) or grad.dtype not in _TYPES:
        raise TypeError("grad must be a float32 or bfloat16 tensor")
    given = grad.dtype
    if not _good(grad, given, i, (T, width)):
        _refuse_tensors((grad, "grad", given, dev, (T, width)))
    if act:
        if preact is None:
            raise ValueError(f"{activation} needs preact")
        if not _good(preact, bf, i, (T, wide)):
            _refuse_tensors((preact, "preact", bf, dev, (T, wide)))
    else:
        preact = None
    kept = 0  # bytes of the scratch tensor for grad_preact
    pitch = (wide + 7) // 8 * 8
    if grad_preact is not None:
        _given(grad_preact, "grad_preact", bf, dev, (T, pitch))
    elif (act or given is not bf or width % 8) and (need_x or need_w):
        kept = (T * pitch * 2 + 255) // 256 * 256
    x_at = w_at = bias_at = 0
    if need_x:
        grad_x = _target(grad_x, "grad_x", bf, dev, (T, H), stream)
        x_at = grad_x.data_ptr()
    else:
        grad_x = None
    if need_w:
        grad_w = _target(grad_w, "grad_w", bf, dev, (wide, H), stream)
        w_at = grad_w.data_ptr()
    else:
        grad_w = None
    if grad_bias is not None:
        bias_dtype = grad_bias.dtype
    if bias_dtype is not None:
        if bias_dtype not in _TYPES:
            raise TypeError(f"the bias must be float32 or bfloat16, not {bias_dtype}")
        grad_bias = _target(grad_bias, "grad_bias", bias_dtype, dev, (wide,), stream)
        bias_at = grad_bias.data_ptr()
    if error_word is not None:
        _want(error_word, "error_word", torch.int32, dev)
    if workspace is None:
        nbytes = max(ep_dense_workspace_bytes(T, H, width, activation), 16)
        scratch = _empty(kept + nbytes, torch.uint8, dev, stream)
        made = scratch.data_ptr()
        at = made + kept
    else:
        _want(workspace, "workspace", torch.uint8, dev)
        at, nbytes = workspace.data_ptr(), workspace.numel()
        scratch = _empty(kept, torch.uint8, dev, stream) if kept else None
        made = _address(scratch)
    _launch(i, "ep_dense_product_backward", _dense_backward_args(
        grad.data_ptr(), _TYPES[given], x.data_ptr(), apart, T, H, w.data_ptr(), width, act,
        0 if preact is None else preact.data_ptr(), made if kept else _address(grad_preact), x_at, w_at, bias_at,
        N.EP_TYPE_FP32 if bias_dtype is None else _TYPES[bias_dtype], at, nbytes, _address(error_word)), stream)
    return grad_x, grad_w, grad_bias


def ep_selftest_bounded_waits(device=None, stream=None) -> dict:
    """The library's self-test of its bounded device waits (about one second
    of GPU time): an mbarrier wait that nothing completes and a grid barrier
    that one block never reaches must both give up after the wait limit.
    Waits for the stream, then returns ``{"gave_up": [mbarrier, grid barrier],
    "elapsed_ns": [...], "error_word": ...}``."""
    dev = torch.device("cuda" if device is None else device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    gave_up = torch.full((2,), -1, dtype=torch.int32, device=dev)
    elapsed = torch.zeros(2, dtype=torch.int64, device=dev)
    _call(dev, "ep_selftest_bounded_waits", _ptr(err), _ptr(gave_up), _ptr(elapsed), _stream(stream, dev))
    (torch.cuda.current_stream(dev) if stream is None else stream).synchronize()
    return {"gave_up": gave_up.tolist(), "elapsed_ns": elapsed.tolist(),
            "error_word": int(err.item()) & 0xffffffff}
