"""Refusals of the router, the experts' products and the adapters: reported
on the host, before any CUDA call (no GPU needed)."""
import ctypes as C

import pytest
import torch

import combine_ep_get_layout_gb300 as ep
from combine_ep_get_layout_gb300 import _native as N

P = 0x20000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from combine_ep_get_layout_gb300 import build
    build.build()
    return N.load()


def refused(lib, fn, args, needle, status):
    s = getattr(lib, fn)(C.byref(args), None)
    assert lib.ep_status_str(s).decode() == status, lib.ep_last_error()
    assert needle in lib.ep_last_error().decode()


BAD, LIMIT = "EP_ERR_INVALID_ARG", "EP_ERR_UNSUPPORTED"


@pytest.mark.parametrize("kw,needle,status", [
    (dict(num_tokens=-1), "num_tokens", BAD), (dict(num_experts=0), "num_experts", BAD),
    (dict(num_experts=4097, row_stride=5000, num_groups=1), "num_experts", LIMIT), (dict(num_topk=0), "num_topk", BAD),
    (dict(num_topk=65), "num_topk", BAD), (dict(num_topk=33), "num_topk", LIMIT), (dict(score=2), "score", BAD),
    (dict(logits_type=5), "logits_type", BAD), (dict(row_stride=63), "row_stride", BAD),
    (dict(num_groups=0), "num_groups", BAD), (dict(num_experts=640, row_stride=640, num_groups=65), "num_groups", LIMIT),
    (dict(num_groups=7), "multiple", BAD), (dict(topk_groups=9), "topk_groups", BAD),
    (dict(topk_groups=0), "topk_groups", BAD), (dict(group_top=3), "group_top", BAD),
    (dict(logits=None), "logits is NULL", BAD), (dict(logits=P + 2), "logits is not 4-byte", BAD),
    (dict(bias=P + 1), "bias", BAD), (dict(topk_idx=P + 4), "topk_idx", BAD),
    (dict(topk_weights=None), "topk_weights is NULL", BAD),
])
def test_route_refuses(lib, kw, needle, status):
    a = dict(logits=P, logits_type=0, row_stride=64, num_tokens=10, num_experts=64, num_topk=4, score=0, bias=None,
             num_groups=8, topk_groups=2, group_top=1, renormalize=1, weight_scale=1.0, topk_idx=P, topk_weights=P)
    a.update(kw)
    refused(lib, "ep_route", N.ep_route_args_t(**a), needle, status)


@pytest.mark.parametrize("kw,needle,status", [
    (dict(num_tokens=-1), "num_tokens", BAD), (dict(num_topk=33), "num_topk", LIMIT), (dict(score=-1), "score", BAD),
    (dict(grad_weights=None), "grad_weights is NULL", BAD), (dict(topk_idx=P + 4), "topk_idx", BAD),
    (dict(grad_logits=None), "grad_logits is NULL", BAD), (dict(logits_type=1, logits=P + 1), "logits is not 2-byte", BAD),
    (dict(row_stride=1), "row_stride", BAD),
])
def test_route_backward_refuses(lib, kw, needle, status):
    a = dict(grad_weights=P, logits=P, logits_type=0, row_stride=64, topk_idx=P, num_tokens=10, num_experts=64,
             num_topk=4, score=0, renormalize=1, weight_scale=1.0, grad_logits=P)
    a.update(kw)
    refused(lib, "ep_route_backward", N.ep_route_backward_args_t(**a), needle, status)


SIZES = [
    (dict(recv_capacity=-1), "recv_capacity", BAD), (dict(num_tokens=-1), "num_tokens", BAD),
    (dict(num_experts=0), "num_experts", BAD), (dict(num_experts=4097), "num_experts", LIMIT),
    (dict(hidden=0), "hidden", BAD), (dict(hidden=100), "multiple of 8", BAD), (dict(hidden=16392), "hidden", LIMIT),
    (dict(width=4), "width", BAD), (dict(width=60), "multiple of 8", BAD), (dict(width=16392), "width", LIMIT),
    (dict(activation=3), "activation", BAD), (dict(x=None), "x is NULL", BAD), (dict(x=P + 8), "x is not 16-byte", BAD),
    (dict(w=None), "w is NULL", BAD), (dict(layout=None), "layout is NULL", BAD),
    (dict(layout="offset"), "expert_offset is NULL", BAD),
]


def layout(kind):
    if kind is None:
        return None
    return C.pointer(N.ep_expanded_layout_t(P, None if kind == "offset" else P, P, P))


@pytest.mark.parametrize("kw,needle,status", SIZES + [
    (dict(out=None), "out is NULL", BAD), (dict(preact=P + 4), "preact", BAD)])
def test_product_refuses(lib, kw, needle, status):
    a = dict(x=P, recv_capacity=100, num_tokens=10, hidden=64, num_experts=4, layout="ok", w=P, width=64, activation=1,
             out=P, preact=None)
    a.update(kw)
    a["layout"] = layout(a["layout"])
    refused(lib, "ep_expert_product", N.ep_expert_product_args_t(**a), needle, status)


@pytest.mark.parametrize("kw,needle,status", SIZES + [
    (dict(grad=None), "grad is NULL", BAD), (dict(preact=None), "preact is NULL", BAD),
    (dict(grad_preact=None), "grad_preact is NULL", BAD), (dict(grad_w=P + 2), "grad_w", BAD)])
def test_product_backward_refuses(lib, kw, needle, status):
    a = dict(grad=P, x=P, w=P, recv_capacity=100, num_tokens=10, hidden=64, num_experts=4, layout="ok", width=64,
             activation=1, preact=P, grad_preact=P, grad_x=P, grad_w=P)
    a.update(kw)
    a["layout"] = layout(a["layout"])
    refused(lib, "ep_expert_product_backward", N.ep_expert_product_backward_args_t(**a), needle, status)


@pytest.mark.parametrize("kw,needle,status", [
    (dict(num_rows=-1), "num_rows", BAD), (dict(hidden=12), "multiple of 8", BAD), (dict(width=0), "width", BAD),
    (dict(rank=4), "rank", BAD), (dict(rank=12), "rank", BAD), (dict(rank=136), "rank", LIMIT),
    (dict(num_adapters=0), "num_adapters", BAD), (dict(num_adapters=5000), "num_adapters", LIMIT),
    (dict(x=P + 4), "x is not 16-byte", BAD), (dict(lora_a=None), "lora_a is NULL", BAD),
    (dict(lora_b=P + 2), "lora_b", BAD), (dict(adapter_idx=P + 4), "adapter_idx", BAD), (dict(out=None), "out is NULL", BAD),
    (dict(workspace=None), "workspace is NULL", BAD), (dict(workspace_bytes=8), "workspace_bytes", BAD),
    (dict(error_word=P + 2), "error_word", BAD),
])
def test_adapter_refuses(lib, kw, needle, status):
    a = dict(x=P, num_rows=10, hidden=64, w=P, width=64, lora_a=P, lora_b=P, num_adapters=4, rank=16, adapter_idx=P,
             adapter_scale=None, out=P, workspace=P, workspace_bytes=1 << 20, error_word=None)
    a.update(kw)
    refused(lib, "ep_adapter_product", N.ep_adapter_product_args_t(**a), needle, status)


def test_null_arguments(lib):
    for fn in ("ep_route", "ep_route_backward", "ep_expert_product", "ep_expert_product_backward", "ep_adapter_product"):
        assert lib.ep_status_str(getattr(lib, fn)(None, None)).decode() == BAD
        assert "args is NULL" in lib.ep_last_error().decode()


def test_workspace_sizes(lib):
    assert lib.ep_adapter_workspace_bytes(100, 512, 16) >= 100 * 16 * 2
    for bad in ((-1, 512, 16), (10, 4, 16), (10, 512, 4), (10, 512, 136), (10, 16392, 16)):
        assert lib.ep_adapter_workspace_bytes(*bad) == 0


def test_the_binding_checks_tensors():
    """Types, devices and shapes, before the library is reached."""
    bf = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="logits"):
        ep.ep_route(torch.zeros((4, 8), dtype=torch.float64), 2)
    with pytest.raises(ValueError, match="logits must be a CUDA tensor"):
        ep.ep_route(torch.zeros((4, 8)), 2)
    with pytest.raises(ValueError, match="logits must be"):
        ep.ep_route(torch.zeros(8), 2)
    with pytest.raises(TypeError, match="x must be"):  # dispatched fp8 rows are not taken
        ep.ep_expert_product(torch.zeros((4, 64), dtype=torch.float8_e4m3fn), bf, None)
    with pytest.raises(KeyError):
        ep.ep_expert_product(bf, bf, None, activation="relu")
    with pytest.raises(TypeError, match="x must be"):
        ep.ep_adapter_product(torch.zeros((4, 64)), bf, bf, bf, torch.zeros(4, dtype=torch.int64))


class OnDevice:
    """A tensor as the binding looks at it, on a device that need not be there."""

    def __init__(self, shape, index, dtype=torch.bfloat16):
        self.shape, self.dtype, self.is_cuda, self.index = torch.Size(shape), dtype, True, index
        self.device = torch.device("cuda", index)

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True


@pytest.mark.parametrize("away", ["num_rows_per_expert", "expert_offset", "error_word"])
@pytest.mark.parametrize("where", ["cuda:1", "cpu"])
def test_a_layout_of_another_device_is_refused(away, where):
    """The kernels read the layout's tensors where the rows are."""
    x, w, grad = OnDevice((8, 64), 0), OnDevice((4, 32, 64), 0), OnDevice((8, 32), 0)
    there = {n: OnDevice((1,), 0, torch.int32) for n in
             ("num_rows_per_expert", "expert_offset", "token_slot", "error_word", "workspace")}
    there[away] = OnDevice((1,), 1, torch.int32) if where == "cuda:1" else torch.zeros(1, dtype=torch.int32)
    lay = ep.ExpandedLayout(**there, num_tokens=4, num_topk=2, num_experts=4, expert_alignment=1)
    with pytest.raises(ValueError, match=f"layout.{away} is on {where}, expected cuda:0"):
        ep.ep_expert_product(x, w, lay)
    with pytest.raises(ValueError, match=f"layout.{away} is on {where}, expected cuda:0"):
        ep.ep_expert_product_backward(grad, x, w, lay)


@pytest.mark.parametrize("cls", [N.ep_route_args_t, N.ep_route_backward_args_t, N.ep_expert_product_args_t,
                                 N.ep_expert_product_backward_args_t, N.ep_adapter_product_args_t])
def test_packed_arguments_are_the_structures_bytes(cls):
    """Every field at its place: the structure read back from the bytes."""
    values = [0.5 + i if t is C.c_float else 1000 + 7 * i for i, (_, t) in enumerate(cls._fields_)]
    got = cls.from_buffer_copy(N.packer(cls)(*values))
    for (name, t), want in zip(cls._fields_, values):
        v = getattr(got, name)
        assert (C.cast(v, C.c_void_p).value if issubclass(t, C._Pointer) else v) == want, name
