"""Refusals of the balance loss, the layer norm and the shared product:
reported on the host, before any CUDA call (no GPU needed)."""
import ctypes as C

import pytest
import torch

import combine_ep_get_layout_gb300 as ep
from combine_ep_get_layout_gb300 import _native as N

P = 0x20000  # never dereferenced: validation fails first
BAD, LIMIT = "EP_ERR_INVALID_ARG", "EP_ERR_UNSUPPORTED"
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from combine_ep_get_layout_gb300 import build
    build.build()
    return N.load()


def refused(lib, fn, args, needle, status):
    s = getattr(lib, fn)(C.byref(args), None)
    assert lib.ep_status_str(s).decode() == status, lib.ep_last_error()
    assert needle in lib.ep_last_error().decode()


LOGITS = [
    (dict(num_tokens=-1), "num_tokens", BAD), (dict(num_experts=0), "num_experts", BAD),
    (dict(num_experts=4097, row_stride=5000), "num_experts", LIMIT), (dict(score=2), "score", BAD),
    (dict(logits_type=3), "logits_type", BAD), (dict(row_stride=63), "row_stride", BAD),
    (dict(num_sequences=0), "num_sequences", BAD), (dict(num_sequences=65537), "num_sequences", LIMIT),
    (dict(num_sequences=4, seq_offsets=None), "seq_offsets is NULL", BAD), (dict(seq_offsets=P + 2), "seq_offsets", BAD),
    (dict(logits=None), "logits is NULL", BAD), (dict(logits=P + 2), "logits is not 4-byte", BAD),
    (dict(logits=P + 1, logits_type=1), "logits is not 2-byte", BAD),
]


@pytest.mark.parametrize("kw,needle,status", LOGITS + [
    (dict(num_topk=0), "num_topk", BAD), (dict(num_topk=65), "num_topk", BAD), (dict(num_topk=33), "num_topk", LIMIT),
    (dict(topk_idx=None), "topk_idx is NULL", BAD), (dict(topk_idx=P + 4), "topk_idx", BAD),
    (dict(losses=None), "losses is NULL", BAD), (dict(counts=P + 1), "counts", BAD), (dict(probs=None), "probs is NULL", BAD),
    (dict(slopes=P + 2), "slopes", BAD), (dict(workspace=None), "workspace is NULL", BAD),
    (dict(workspace=P + 8), "workspace is not 16-byte", BAD), (dict(workspace_bytes=64), "workspace_bytes", BAD),
])
def test_balance_refuses(lib, kw, needle, status):
    a = dict(logits=P, logits_type=0, row_stride=64, topk_idx=P, num_tokens=10, num_experts=64, num_topk=4, score=0,
             seq_offsets=P, num_sequences=2, losses=P, counts=P, probs=P, slopes=P, workspace=P, workspace_bytes=1 << 24)
    a.update(kw)
    refused(lib, "ep_balance_loss", N.ep_balance_loss_args_t(**a), needle, status)


@pytest.mark.parametrize("kw,needle,status", LOGITS + [
    (dict(grad_losses=None), "grad_losses is NULL", BAD), (dict(slopes=None), "slopes is NULL", BAD),
    (dict(add=P + 2), "add", BAD), (dict(grad_logits=None), "grad_logits is NULL", BAD),
])
def test_balance_backward_refuses(lib, kw, needle, status):
    a = dict(grad_losses=P, logits=P, logits_type=0, row_stride=64, num_tokens=10, num_experts=64, score=0, seq_offsets=P,
             num_sequences=2, slopes=P, add=None, grad_logits=P)
    a.update(kw)
    refused(lib, "ep_balance_loss_backward", N.ep_balance_loss_backward_args_t(**a), needle, status)


ROWS = [
    (dict(num_rows=-1), "num_rows", BAD), (dict(hidden=0), "hidden", BAD), (dict(hidden=16385, row_stride=20000), "hidden", LIMIT),
    (dict(type=2), "type", BAD), (dict(param_type=-1), "param_type", BAD), (dict(row_stride=63), "row_stride", BAD),
    (dict(x=None), "x is NULL", BAD), (dict(x=P + 1), "x is not 2-byte", BAD), (dict(weight=P + 2), "weight is not 4-byte", BAD),
]


@pytest.mark.parametrize("kw,needle,status", ROWS + [
    (dict(bias=P + 1, param_type=1), "bias is not 2-byte", BAD), (dict(out=None), "out is NULL", BAD),
    (dict(mean=P + 2), "mean", BAD), (dict(rstd=P + 1), "rstd", BAD), (dict(eps=0.0), "eps", BAD), (dict(eps=-1e-5), "eps", BAD),
    (dict(eps=NAN), "eps", BAD), (dict(eps=INF), "eps", BAD), (dict(x=P, out=P, row_stride=128), "out is x", BAD),
])
def test_norm_refuses(lib, kw, needle, status):
    a = dict(x=P, type=1, row_stride=64, num_rows=10, hidden=64, weight=P, bias=P, param_type=0, eps=1e-5, out=P + 0x10000,
             mean=None, rstd=None)
    a.update(kw)
    refused(lib, "ep_layer_norm", N.ep_layer_norm_args_t(**a), needle, status)


@pytest.mark.parametrize("kw,needle,status", ROWS + [
    (dict(grad=None), "grad is NULL", BAD), (dict(mean=None), "mean is NULL", BAD), (dict(rstd=P + 2), "rstd", BAD),
    (dict(add=P + 1), "add", BAD), (dict(grad_x=P + 1), "grad_x", BAD), (dict(grad_weight=P + 2), "grad_weight", BAD),
    (dict(grad_bias=P + 1), "grad_bias", BAD), (dict(grad_x=P, row_stride=128), "grad_x is x", BAD),
    (dict(workspace=None), "workspace is NULL", BAD), (dict(workspace_bytes=100), "workspace_bytes", BAD),
])
def test_norm_backward_refuses(lib, kw, needle, status):
    a = dict(grad=P, x=P, type=1, row_stride=64, num_rows=10, hidden=64, mean=P, rstd=P, weight=P, param_type=0, add=None,
             grad_x=P + 0x10000, grad_weight=P, grad_bias=P, workspace=P, workspace_bytes=1 << 24)
    a.update(kw)
    refused(lib, "ep_layer_norm_backward", N.ep_layer_norm_backward_args_t(**a), needle, status)


PRODUCT = [
    (dict(num_rows=-1), "num_rows", BAD), (dict(hidden=4), "hidden", BAD), (dict(hidden=60), "multiple of 8", BAD),
    (dict(hidden=16392, row_stride=16392), "hidden", LIMIT), (dict(width=0), "width", BAD), (dict(width=-8), "width", BAD),
    (dict(width=16385), "width", LIMIT), (dict(activation=6), "activation", BAD), (dict(activation=-1), "activation", BAD),
    (dict(row_stride=56), "row_stride", BAD), (dict(row_stride=68), "multiple of 8", BAD), (dict(bias_type=2), "bias_type", BAD),
    (dict(x=P + 8), "x is not 16-byte", BAD), (dict(w=None), "w is NULL", BAD), (dict(w=P + 2), "w is not 16-byte", BAD),
    (dict(error_word=P + 2), "error_word", BAD),
]


@pytest.mark.parametrize("kw,needle,status", PRODUCT + [
    (dict(out_type=3), "out_type", BAD), (dict(x=None), "x is NULL", BAD), (dict(bias=P + 2), "bias is not 4-byte", BAD),
    (dict(residual=P + 8), "residual", BAD), (dict(out=None), "out is NULL", BAD), (dict(out=P + 4), "out is not 16-byte", BAD),
    (dict(preact=P + 2), "preact", BAD), (dict(residual=P, out=P, out_type=0), "residual (bf16) is out", BAD),
])
def test_dense_refuses(lib, kw, needle, status):
    a = dict(x=P, row_stride=64, num_rows=10, hidden=64, w=P, width=64, bias=P, bias_type=0, activation=1, residual=None,
             out=P + 0x10000, out_type=1, preact=None, error_word=None)
    a.update(kw)
    refused(lib, "ep_dense_product", N.ep_dense_product_args_t(**a), needle, status)


@pytest.mark.parametrize("kw,needle,status", PRODUCT + [
    (dict(grad_type=2), "grad_type", BAD), (dict(grad=None), "grad is NULL", BAD), (dict(preact=None), "preact is NULL", BAD),
    (dict(grad_preact=None), "grad_preact is NULL", BAD), (dict(activation=0, grad_type=0, grad_preact=None), "grad_preact is NULL", BAD),
    (dict(activation=0, width=60, grad_preact=None), "grad_preact is NULL", BAD),
    (dict(grad_x=P + 8), "grad_x", BAD), (dict(grad_w=P + 2), "grad_w", BAD), (dict(grad_bias=P + 2), "grad_bias", BAD),
    (dict(workspace=None), "workspace is NULL", BAD), (dict(workspace_bytes=16), "workspace_bytes", BAD),
])
def test_dense_backward_refuses(lib, kw, needle, status):
    a = dict(grad=P, grad_type=1, x=P, row_stride=64, num_rows=10, hidden=64, w=P, width=64, activation=4, preact=P,
             grad_preact=P, grad_x=P, grad_w=P, grad_bias=P, bias_type=0, workspace=P, workspace_bytes=1 << 24, error_word=None)
    a.update(kw)
    refused(lib, "ep_dense_product_backward", N.ep_dense_product_backward_args_t(**a), needle, status)


def test_null_arguments(lib):
    for fn in ("ep_balance_loss", "ep_balance_loss_backward", "ep_layer_norm", "ep_layer_norm_backward", "ep_dense_product",
               "ep_dense_product_backward"):
        assert lib.ep_status_str(getattr(lib, fn)(None, None)).decode() == BAD
        assert "args is NULL" in lib.ep_last_error().decode()


def test_workspaces(lib):
    assert lib.ep_balance_workspace_bytes(1000, 64, 3) > 0 and lib.ep_layer_norm_workspace_bytes(1000, 64) > 0
    assert lib.ep_dense_workspace_bytes(1000, 64, 64, 1) >= lib.ep_dense_workspace_bytes(1000, 64, 64, 0) > 0
    for bad in ((-1, 64, 1), (5, 0, 1), (5, 5000, 1), (5, 64, 0), (5, 64, 65537)):
        assert lib.ep_balance_workspace_bytes(*bad) == 0
    for bad in ((-1, 64), (5, 0), (5, 16385)):
        assert lib.ep_layer_norm_workspace_bytes(*bad) == 0
    for bad in ((-1, 64, 64, 0), (5, 0, 64, 0), (5, 64, 16392, 0)):
        assert lib.ep_dense_workspace_bytes(*bad) == 0


def test_tensors_off_the_gpu_are_refused():
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((8, 64), dtype=torch.bfloat16)
    logits, idx = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int64)
    one = torch.zeros(4)
    b = ep.Balance(torch.zeros(2), torch.zeros((1, 8), dtype=torch.int32), torch.zeros((1, 8)), torch.zeros((1, 8)))
    for call in (lambda: ep.ep_layer_norm(x), lambda: ep.ep_layer_norm_backward(x, x, one, one),
                 lambda: ep.ep_dense_product(x, w), lambda: ep.ep_dense_product_backward(x[:, :8], x, w),
                 lambda: ep.ep_balance_loss(logits, idx), lambda: ep.ep_balance_loss_backward(torch.zeros(2), logits, b)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_too_many_rows(lib):
    many = 2 ** 30 + 1
    balance = dict(logits=P, row_stride=1, num_tokens=many, num_experts=1, num_sequences=1)
    norm = dict(x=P, row_stride=1, num_rows=many, hidden=1)
    dense = dict(x=P, row_stride=8, num_rows=many, hidden=8, w=P, width=1)
    for fn, args in (("ep_balance_loss", dict(balance, num_topk=1)), ("ep_balance_loss_backward", balance),
                     ("ep_layer_norm", dict(norm, eps=1e-5)), ("ep_layer_norm_backward", norm),
                     ("ep_dense_product", dense), ("ep_dense_product_backward", dense)):
        refused(lib, fn, getattr(N, fn + "_args_t")(**args), f"{many} > {2 ** 30}", LIMIT)
    assert lib.ep_balance_workspace_bytes(many, 1, 1) == lib.ep_layer_norm_workspace_bytes(many, 1) == 0
    assert lib.ep_dense_workspace_bytes(many, 8, 1, 0) == lib.ep_dense_workspace_bytes(5, 12, 8, 0) == 0


AT = [P + i * 0x10000 for i in range(10)]


@pytest.mark.parametrize("kw,needle", [
    (dict(out=AT[0]), "out is x"), (dict(preact=AT[3]), "out is preact"), (dict(preact=AT[0]), "preact is x"),
    (dict(preact=AT[4]), "preact is residual"),
])
def test_dense_refuses_an_output_that_is_an_operand(lib, kw, needle):
    a = dict(x=AT[0], row_stride=64, num_rows=10, hidden=64, w=AT[1], width=64, bias=AT[2], activation=2, residual=AT[4],
             out=AT[3], out_type=1, preact=AT[5])
    a.update(kw)
    refused(lib, "ep_dense_product", N.ep_dense_product_args_t(**a), needle, BAD)


@pytest.mark.parametrize("kw,needle", [
    (dict(grad_x=AT[0]), "grad_x is grad"), (dict(grad_x=AT[1]), "grad_x is x"), (dict(grad_x=AT[4]), "grad_x is grad_preact"),
    (dict(grad_w=AT[2]), "grad_w is w"), (dict(grad_w=AT[1]), "grad_w is x"), (dict(grad_preact=AT[0]), "grad_preact is grad"),
    (dict(grad_preact=AT[3]), "grad_preact is preact"), (dict(grad_preact=AT[1]), "grad_preact is x"),
])
def test_dense_backward_refuses_an_output_that_is_an_operand(lib, kw, needle):
    a = dict(grad=AT[0], grad_type=1, x=AT[1], row_stride=64, num_rows=10, hidden=64, w=AT[2], width=64, activation=2,
             preact=AT[3], grad_preact=AT[4], grad_x=AT[5], grad_w=AT[6], grad_bias=AT[7], workspace=AT[8],
             workspace_bytes=1 << 24)
    a.update(kw)
    refused(lib, "ep_dense_product_backward", N.ep_dense_product_backward_args_t(**a), needle, BAD)


def test_balance_backward_refuses_logits_apart_as_output(lib):
    refused(lib, "ep_balance_loss_backward", N.ep_balance_loss_backward_args_t(
        grad_losses=AT[0], logits=AT[1], row_stride=128, num_tokens=10, num_experts=64, num_sequences=1, slopes=AT[2],
        grad_logits=AT[1]), "grad_logits is logits", BAD)
