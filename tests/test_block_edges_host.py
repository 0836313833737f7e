"""The shared product refuses every output that begins at an operand or at
another output (no GPU needed: reported before any CUDA call)."""
import ctypes as C
import itertools

import pytest

from combine_ep_get_layout_gb300 import _native as N

P = 0x20000  # never dereferenced: validation fails first
BAD = "EP_ERR_INVALID_ARG"


@pytest.fixture(scope="module")
def lib():
    from combine_ep_get_layout_gb300 import build
    build.build()
    return N.load()


FORWARD = {n: P + i * 0x10000 for i, n in enumerate(["x", "w", "bias", "residual", "error_word", "out", "preact"])}
BACKWARD = {n: P + i * 0x10000 for i, n in enumerate(
    ["grad", "x", "w", "preact", "error_word", "grad_x", "grad_w", "grad_bias", "grad_preact", "workspace"])}


def pairs(names, outputs, allowed=()):
    """(an output, what it must not be), each once."""
    return [(a, b) for a, b in itertools.permutations(names, 2)
            if a in outputs and (a, b) not in allowed and not (b in outputs and outputs.index(b) < outputs.index(a))]


def refused(lib, fn, args, a, b):
    s = getattr(lib, fn)(C.byref(args), None)
    said = lib.ep_last_error().decode()
    assert lib.ep_status_str(s).decode() == BAD, said
    assert f"{a} is {b}" in said


@pytest.mark.parametrize("a,b", pairs(FORWARD, ["out", "preact"], [("out", "residual")]))
def test_an_output_of_the_product(lib, a, b):
    at = dict(FORWARD)
    at[a] = at[b]
    refused(lib, "ep_dense_product", N.ep_dense_product_args_t(
        row_stride=64, num_rows=10, hidden=64, width=64, activation=2, out_type=1, **at), a, b)


@pytest.mark.parametrize("a,b", pairs(BACKWARD, ["grad_x", "grad_w", "grad_bias", "grad_preact", "workspace"]))
def test_an_output_of_the_gradients(lib, a, b):
    at = dict(BACKWARD)
    at[a] = at[b]
    refused(lib, "ep_dense_product_backward", N.ep_dense_product_backward_args_t(
        grad_type=1, row_stride=64, num_rows=10, hidden=64, width=64, activation=2, workspace_bytes=1 << 24, **at), a, b)


@pytest.mark.parametrize("a,b", [("grad_w", "w"), ("grad_w", "grad_bias"), ("grad_w", "workspace"), ("grad_bias", "w"),
                                 ("grad_bias", "workspace")])
def test_without_rows_the_parameters_gradients_are_still_written(lib, a, b):
    at = dict(BACKWARD, grad=None, x=None, preact=None, grad_x=None, grad_preact=None)
    at[a] = at[b]
    refused(lib, "ep_dense_product_backward", N.ep_dense_product_backward_args_t(
        grad_type=1, row_stride=64, num_rows=0, hidden=64, width=64, activation=2, workspace_bytes=1 << 24, **at), a, b)
