"""The product shared by all rows, with its epilogue, and its gradients,
against plain 64-bit implementations.

Tolerances, fixed before any run.  The tensor cores add the products of 16
inner elements to an fp32 sum, whose rounding (or cutting off) is 2^-23 of
the sum of absolute values S at most, each of n / 16 times, and at most eight
parts of the inner dimension are joined: a = 2^-23 (n/16 + 24) S.  Activations
change by at most 1.13 times what z does, and are evaluated to 2^-16 of their
value (the documented bound of the exponential they take) and 2^-20 |z|; the
result is rounded to its type.  A gradient of z is rounded to bf16 where it is
computed: 2^-8 of it enters the products' bounds; for the bias it is summed
before: 2^-24 (T/16 + 400) of the absolute values for at least 32 slices of
rows (T alone below 400), and the activation's own error.
"""
import math

import pytest
import torch

import combine_ep_get_layout_gb300 as ep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
ACTS = [None, "relu", "silu", "gelu", "gelu_tanh", "swiglu"]
F = torch.nn.functional
FUNCTIONS = {None: lambda z: z, "relu": F.relu, "silu": F.silu, "gelu": F.gelu,
             "gelu_tanh": lambda z: F.gelu(z, approximate="tanh"),
             "swiglu": lambda z: F.silu(z.chunk(2, dim=1)[0]) * z.chunk(2, dim=1)[1]}


def half(t):
    return torch.finfo(t).eps / 2


def make(T, H, W, act, params=F32, residual=False, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    wide = 2 * W if act == "swiglu" else W

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    return (normal(T, H).to(BF16), (normal(wide, H) / math.sqrt(H)).to(BF16),
            None if params is None else (0.5 * normal(wide)).to(params), normal(T, W).to(BF16) if residual else None)


def check_forward(x, w, bias, act, residual, out, preact=None):
    H = x.shape[1]
    z = x.double() @ w.double().T
    off = 2 * U * (H / 16 + 24) * (x.double().abs() @ w.double().abs().T)
    if bias is not None:
        z = z + bias.double()
        off = off + U * (z.abs() + bias.double().abs())
    if preact is not None:
        assert ((preact.double() - z).abs() <= half(BF16) * z.abs() + 1.01 * off + 1e-38).all()
    y = FUNCTIONS[act](z)
    if act == "swiglu":
        (g, u), (og, ou) = z.chunk(2, dim=1), off.chunk(2, dim=1)
        off = 1.13 * og * u.abs() + F.silu(g).abs() * ou + 1.13 * og * ou + 2.0 ** -15 * y.abs()
    elif act is not None:
        off = 1.13 * off + 2.0 ** -16 * y.abs() + 2.0 ** -20 * z.abs()
    if residual is not None:
        y = y + residual.double()
        off = off + U * (y.abs() + residual.double().abs())
    tol = half(out.dtype) * y.abs() + 1.01 * off + 1e-38
    err = (out.double() - y).abs()
    assert (err <= tol).all(), float((err / tol).max())


def check_backward(grad, x, w, act, preact, got, bias):
    T, H = x.shape
    g64 = grad.double()
    if act is None:
        d, off = g64, 0 * g64
    else:
        z = preact.double().requires_grad_(True)
        d, = torch.autograd.grad(FUNCTIONS[act](z), z, g64)
        z = z.detach()
        size = g64.abs() if act != "swiglu" else torch.cat(
            [g64.abs() * z.chunk(2, dim=1)[1].abs(), g64.abs() * F.silu(z.chunk(2, dim=1)[0]).abs()], 1)
        off = 2.0 ** -15 * size
    made = act is not None or grad.dtype is not BF16
    total = off + (half(BF16) * (d.abs() + off) if made else 0.0)
    wide = d.shape[1]
    if got[0] is not None:
        want = d @ w.double()
        tol = half(BF16) * want.abs() + total @ w.double().abs() + 2 * U * (wide / 16 + 24) * (d.abs() @ w.double().abs())
        err = (got[0].double() - want).abs()
        assert (err <= 1.01 * tol + 1e-38).all(), ("x", float((err / tol).max()))
    if got[1] is not None:
        want = d.T @ x.double()
        tol = half(BF16) * want.abs() + total.T @ x.double().abs() + 2 * U * (T / 16 + 24) * (d.abs().T @ x.double().abs())
        err = (got[1].double() - want).abs()
        assert (err <= 1.01 * tol + 1e-38).all(), ("w", float((err / tol).max()))
    if bias is not None:
        want = d.sum(0)
        tol = half(got[2].dtype) * want.abs() + off.sum(0) + U * min(T, T / 16 + 400) * d.abs().sum(0)
        err = (got[2].double() - want).abs()
        assert (err <= 1.01 * tol + 1e-38).all(), ("bias", float((err / tol).max()))
    else:
        assert got[2] is None


SHAPES = [(1, 8, 8), (1, 512, 256), (2, 64, 128), (5, 72, 40), (17, 136, 264), (31, 2048, 136), (33, 256, 520), (64, 1024, 96),
          (100, 96, 2056), (129, 128, 128), (255, 264, 248), (256, 512, 256), (300, 512, 1032), (513, 4096, 64), (700, 192, 200),
          (1021, 1000, 328), (2050, 64, 72), (8, 16384, 16), (9, 16, 16384), (1, 8, 1), (40, 64, 3), (33, 256, 60), (700, 128, 225),
          (300, 512, 259), (1500, 64, 130), (5, 72, 1001)]


@pytest.mark.parametrize("T,H,W", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_against_64_bits(T, H, W, act):
    params = [F32, BF16, None][(T + W // 8) % 3]
    for out_dtype in (BF16, F32):
        x, w, bias, residual = make(T, H, W, act, params, residual=(T + H // 8 + (out_dtype is F32)) % 2 == 0, seed=T)
        preact = torch.full((T, w.shape[0]), 9.0, dtype=BF16, device=DEV)
        out = ep.ep_dense_product(x, w, bias, activation=act, residual=residual, preact=preact, out_dtype=out_dtype)
        assert out.dtype is out_dtype
        check_forward(x, w, bias, act, residual, out, preact)
        grad = torch.randn((T, W), device=DEV).to(out_dtype)
        got = ep.ep_dense_product_backward(grad, x, w, activation=act, preact=preact if act else None, bias_dtype=params)
        check_backward(grad, x, w, act, preact, got, bias)


@pytest.mark.parametrize("T,H,W,act", [(24, 4096, 4096, None), (1000, 7168, 256, None), (600, 2048, 1408, "swiglu"),
                                       (4093, 512, 1000, "gelu"), (3000, 1024, 2048, "silu")])
def test_ordinary_sizes(T, H, W, act):
    x, w, bias, residual = make(T, H, W, act, F32, True, seed=1)
    preact = torch.empty((T, w.shape[0]), dtype=BF16, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = ep.ep_dense_product(x, w, bias, activation=act, residual=residual, preact=preact, error_word=err)
    check_forward(x, w, bias, act, residual, out, preact)
    grad = torch.randn((T, W), device=DEV).to(BF16)
    got = ep.ep_dense_product_backward(grad, x, w, activation=act, preact=preact if act else None, bias_dtype=F32, error_word=err)
    check_backward(grad, x, w, act, preact, got, bias)
    assert int(err) == 0


def test_every_row_counts():
    """Small whole numbers: every sum is exact, so a row or an inner element
    that is left out, or taken twice, shows."""
    g = torch.Generator(device=DEV).manual_seed(2)
    for T, H, W in ((1, 64, 8), (37, 72, 24), (1000, 200, 136), (4100, 136, 264), (513, 1032, 8), (9000, 64, 64), (800, 72, 61),
                    (1300, 136, 299)):
        x = torch.randint(-2, 3, (T, H), generator=g, device=DEV).to(BF16)
        w = torch.randint(-2, 3, (W, H), generator=g, device=DEV).to(BF16)
        bias = torch.randint(-9, 10, (W,), generator=g, device=DEV).to(F32)
        out = ep.ep_dense_product(x, w, bias, out_dtype=F32)
        assert torch.equal(out.double(), x.double() @ w.double().T + bias.double())
        grad = torch.randint(-2, 3, (T, W), generator=g, device=DEV).to(BF16)
        dx, dw, db = ep.ep_dense_product_backward(grad, x, w, bias_dtype=F32)
        assert torch.equal(dx, (grad.double() @ w.double()).to(BF16))
        assert torch.equal(dw, (grad.double().T @ x.double()).to(BF16))
        assert torch.equal(db.double(), grad.double().sum(0))
        relu = ep.ep_dense_product_backward(grad.float(), x, w, activation="relu", preact=out.to(BF16), bias_dtype=F32)
        d = torch.where(out > 0, grad.float(), 0.0).double()
        assert torch.equal(relu[0], (d @ w.double()).to(BF16)) and torch.equal(relu[1], (d.T @ x.double()).to(BF16))
        assert torch.equal(relu[2].double(), d.sum(0))


def test_parts_and_given_tensors():
    x, w, bias, residual = make(90, 256, 128, "gelu", BF16, True)
    preact = torch.empty((90, 128), dtype=BF16, device=DEV)
    ep.ep_dense_product(x, w, bias, activation="gelu", preact=preact)
    grad = torch.randn((90, 128), device=DEV).to(BF16)
    full = ep.ep_dense_product_backward(grad, x, w, activation="gelu", preact=preact, bias_dtype=BF16)
    for need_x, need_w, b in ((True, False, None), (False, True, BF16), (False, False, BF16), (False, False, None)):
        got = ep.ep_dense_product_backward(grad, x, w, activation="gelu", preact=preact, bias_dtype=b, need_x=need_x, need_w=need_w)
        for p, q, need in zip(got, full, (need_x, need_w, b is not None)):
            assert torch.equal(p, q) if need else p is None
    mine = [torch.empty_like(t) for t in full]
    scratch = torch.empty(ep.ep_dense_workspace_bytes(90, 256, 128, "gelu"), dtype=torch.uint8, device=DEV)
    got = ep.ep_dense_product_backward(grad, x, w, activation="gelu", preact=preact, grad_x=mine[0], grad_w=mine[1],
                                       grad_bias=mine[2], workspace=scratch, grad_preact=torch.empty_like(preact))
    assert all(p is m and torch.equal(p, q) for p, m, q in zip(got, mine, full))


def test_given_outputs_set_the_type():
    x, w, bias, residual = make(77, 128, 96, "relu", F32, True)
    for dtype in (F32, BF16):
        out = torch.full((77, 96), 5.0, dtype=dtype, device=DEV)
        assert ep.ep_dense_product(x, w, bias, activation="relu", residual=residual, out=out) is out
        check_forward(x, w, bias, "relu", residual, out)


def test_the_widest():
    """16 384 outputs, and as many gates beside them."""
    for act in (None, "swiglu"):
        x, w, bias, residual = make(3, 64, 16384, act, BF16, True)
        preact = torch.empty((3, w.shape[0]), dtype=BF16, device=DEV)
        out = ep.ep_dense_product(x, w, bias, activation=act, residual=residual, preact=preact)
        check_forward(x, w, bias, act, residual, out, preact)
        grad = torch.randn((3, 16384), device=DEV)
        got = ep.ep_dense_product_backward(grad, x, w, activation=act, preact=preact if act else None, bias_dtype=BF16)
        check_backward(grad, x, w, act, preact, got, bias)


def test_residual_in_place():
    for act in (None, "swiglu"):
        x, w, bias, residual = make(333, 512, 264, act, F32, True)
        want = ep.ep_dense_product(x, w, bias, activation=act, residual=residual)
        r = residual.clone()
        assert ep.ep_dense_product(x, w, bias, activation=act, residual=r, out=r) is r
        assert torch.equal(r, want)


def test_rows_of_wider_ones():
    big = torch.randn((70, 1024), device=DEV).to(BF16)
    for first, H in ((0, 256), (64, 512), (8, 136)):
        _, w, bias, residual = make(70, H, 264, "silu", F32, True)
        x = big[:, first:first + H]
        preact = torch.empty((70, 264), dtype=BF16, device=DEV)
        out = ep.ep_dense_product(x, w, bias, activation="silu", residual=residual, preact=preact)
        assert torch.equal(out, ep.ep_dense_product(x.contiguous(), w, bias, activation="silu", residual=residual))
        grad = torch.randn((70, 264), device=DEV).to(BF16)
        got = ep.ep_dense_product_backward(grad, x, w, activation="silu", preact=preact, bias_dtype=F32)
        want = ep.ep_dense_product_backward(grad, x.contiguous(), w, activation="silu", preact=preact, bias_dtype=F32)
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_rows_that_are_not_finite_stay_with_themselves():
    x, w, bias, residual = make(300, 256, 128, "silu", F32, True)
    clean = ep.ep_dense_product(x, w, bias, activation="silu", residual=residual)
    x[7, 3], x[280, 5] = math.nan, math.inf
    out = ep.ep_dense_product(x, w, bias, activation="silu", residual=residual)
    good = [i for i in range(300) if i not in (7, 280)]
    assert torch.equal(out[good], clean[good]) and torch.isnan(out[7]).all()
    grad = torch.randn((300, 128), device=DEV).to(BF16)
    grad[9, 1] = math.nan
    dx, dw, db = ep.ep_dense_product_backward(grad, x, w, bias_dtype=F32)
    assert torch.isnan(dx[9]).all() and torch.isfinite(dx[[i for i in range(300) if i != 9]].float()).all()
    assert torch.isnan(db[1]) and torch.isfinite(db[2:]).all()


def test_activations_far_out():
    """Large and tiny preactivations of either sign, forward and backward."""
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-4, -1e-4, 0.5, -0.5, 3.0, -3.0, 5.5, -5.5, 9.0, -9.0, 14.0, -14.0, 40.0,
                      -40.0, 100.0, -100.0, 1e4, -1e4, 1e30, -1e30], device=DEV).to(BF16)
    T = z.numel()
    x = torch.zeros((T, 64), dtype=BF16, device=DEV)
    x[:, 0] = z
    w = torch.zeros((8, 64), dtype=BF16, device=DEV)
    w[:, 0] = 1.0
    for act in ACTS[1:-1]:
        preact = torch.empty((T, 8), dtype=BF16, device=DEV)
        out = ep.ep_dense_product(x, w, activation=act, preact=preact, out_dtype=F32)
        assert torch.equal(preact, z[:, None].expand(T, 8))
        want = FUNCTIONS[act](z.double())[:, None]
        assert ((out - want).abs() <= 2.0 ** -16 * want.abs() + 2.0 ** -20 * z.double().abs()[:, None] + 1e-37).all(), act
        one = torch.ones((T, 8), device=DEV)
        db = [ep.ep_dense_product_backward(one[i:i + 1], x[i:i + 1], w, activation=act, preact=preact[i:i + 1].contiguous(),
                                           bias_dtype=F32, need_x=False, need_w=False)[2][0] for i in range(T)]
        zz = z.double().requires_grad_(True)
        d, = torch.autograd.grad(FUNCTIONS[act](zz).sum(), zz)
        ok = torch.isfinite(d)
        got = torch.stack(db).double()
        assert ((got - d).abs() <= 2.0 ** -15)[ok].all() and torch.isfinite(got).all(), act


@pytest.mark.parametrize("width", [8, 5])
def test_swiglu_gradient_far_out(width):
    """Large gates of either sign under large gradients: products whose value
    is 0 have no infinite part."""
    gate = torch.tensor([1e38, -1e38, 1e30, -1e30, 200.0, -200.0, -90.0, 0.0], device=DEV)
    T = gate.numel()
    x, w = torch.zeros((T, 64), dtype=BF16, device=DEV), torch.zeros((2 * width, 64), dtype=BF16, device=DEV)
    preact = torch.cat([gate[:, None].expand(T, width), torch.full((T, width), 0.5, device=DEV)], 1).to(BF16)
    for grad in (1.0, 1e4):
        g, u = preact[:, 0].double(), 0.5
        s = torch.sigmoid(g)
        want = torch.cat([(grad * u * s * (1 + g * (1 - s)))[:, None], (grad * g * s)[:, None]], 1)
        for i in range(T):
            db = ep.ep_dense_product_backward(torch.full((1, width), grad, device=DEV), x[i:i + 1], w, activation="swiglu",
                                              preact=preact[i:i + 1].clone(), bias_dtype=F32, need_x=False,
                                              need_w=False)[2].view(2, width).double()
            for h in range(2):
                top = float(want[i, h])
                if abs(top) < 3e38:
                    assert ((db[h] - top).abs() <= 2.0 ** -15 * max(abs(top), grad)).all(), (grad, float(g[i]), h, db[h], top)


def test_no_rows():
    x, w, bias, _ = make(0, 64, 40, None)
    assert ep.ep_dense_product(x, w, bias).shape == (0, 40)
    dx, dw, db = ep.ep_dense_product_backward(torch.empty((0, 40), dtype=BF16, device=DEV), x, w, bias_dtype=F32)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    x, w, bias, _ = make(0, 64, 40, "swiglu")
    pre = torch.empty((0, 80), dtype=BF16, device=DEV)
    dx, dw, db = ep.ep_dense_product_backward(torch.empty((0, 40), device=DEV), x, w, activation="swiglu", preact=pre, bias_dtype=BF16)
    assert dw.shape == (80, 64) and (dw == 0).all() and (db == 0).all()


def test_gradient_by_differences():
    """Central differences of the 64-bit definition, h = 1e-4, against the
    gradients: off by the rounding of d and of the result, 2^-8 each."""
    for act in ACTS:
        x, w, bias, _ = make(5, 16, 8, act, F32, seed=3)
        preact = torch.empty((5, w.shape[0]), dtype=BF16, device=DEV)
        ep.ep_dense_product(x, w, bias, activation=act, preact=preact)
        grad = torch.randn((5, 8), device=DEV).to(BF16)
        got = ep.ep_dense_product_backward(grad, x, w, activation=act, preact=preact, bias_dtype=F32)
        base = preact.double() - x.double() @ w.double().T  # the definition at the kept preactivations
        for which, at in ((0, (0, 3)), (0, (4, 15)), (1, (2, 7)), (1, (7, 0))):
            v = []
            for h in (1e-4, -1e-4):
                args = [x.double(), w.double()]
                args[which] = args[which].clone()
                args[which][at] += h
                v.append(float((FUNCTIONS[act](args[0] @ args[1].T + base) * grad.double()).sum()))
            size = float(grad.double().abs().sum() * 4)
            assert abs((v[0] - v[1]) / 2e-4 - float(got[which][at])) < 2.0 ** -7 * size


def test_the_same_bits_and_captured():
    x, w, bias, residual = make(700, 512, 392, "swiglu", F32, True)
    grad = torch.randn((700, 392), device=DEV).to(BF16)
    preact = torch.empty((700, 784), dtype=BF16, device=DEV)

    def step():
        out = ep.ep_dense_product(x, w, bias, activation="swiglu", residual=residual, preact=preact)
        return (out, *ep.ep_dense_product_backward(grad, x, w, activation="swiglu", preact=preact, bias_dtype=F32))

    want = step()
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(want, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = ep.ep_dense_product(x, w, bias, activation="swiglu", residual=residual, stream=side)
    got = ep.ep_dense_product_backward(grad, x, w, activation="swiglu", preact=preact, bias_dtype=F32, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0]) and all(torch.equal(p, q) for p, q in zip(got, want[1:]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.normal_()
    grad.normal_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, step()))


def test_more_than_2_31_elements():
    """Rows and outputs whose offsets pass 2^31 elements."""
    T, H, W = 2 ** 31 // 2048 + 300, 2048, 2048
    try:
        x = torch.zeros((T, H), dtype=BF16, device=DEV)
        out = torch.empty((T, W), dtype=BF16, device=DEV)
    except torch.OutOfMemoryError:
        pytest.skip("no room")
    x[-5:].normal_()
    _, w, bias, _ = make(1, H, W, None)
    ep.ep_dense_product(x, w, bias, out=out, residual=x)
    assert torch.equal(out[0], bias.to(BF16))
    check_forward(x[-5:], w, bias, None, x[-5:], out[-5:])
    dx, dw, db = ep.ep_dense_product_backward(x, x, w, bias_dtype=F32, grad_x=out)
    check_backward(x[-5:], x[-5:], w, None, None, (dx[-5:], dw, db), bias)
    assert (dx[:1000] == 0).all()


def test_refusals():
    x, w, bias, residual = make(10, 64, 40, None, F32, True)
    grad = torch.randn((10, 40), device=DEV).to(BF16)
    for error, call in [
            (TypeError, lambda: ep.ep_dense_product(x.float(), w)), (TypeError, lambda: ep.ep_dense_product(x, w.float())),
            (ValueError, lambda: ep.ep_dense_product(x, w[:, :32])), (ValueError, lambda: ep.ep_dense_product(x, w[0])),
            (ep.EPError, lambda: ep.ep_dense_product(x, w[:0])), (ep.EPError, lambda: ep.ep_dense_product(x[:, :60].contiguous(), w[:, :60].contiguous())),
            (ValueError, lambda: ep.ep_dense_product(x.T, w)), (KeyError, lambda: ep.ep_dense_product(x, w, activation="tanh")),
            (ValueError, lambda: ep.ep_dense_product(x, w, bias[:8])), (TypeError, lambda: ep.ep_dense_product(x, w, bias.half())),
            (ValueError, lambda: ep.ep_dense_product(x, w, residual=residual[:5])),
            (TypeError, lambda: ep.ep_dense_product(x, w, residual=residual.float())),
            (TypeError, lambda: ep.ep_dense_product(x, w, out_dtype=torch.float16)),
            (ValueError, lambda: ep.ep_dense_product(x, w, preact=torch.empty((10, 80), dtype=BF16, device=DEV))),
            (ValueError, lambda: ep.ep_dense_product(x, w, out=torch.empty((11, 40), dtype=BF16, device=DEV))),
            (ValueError, lambda: ep.ep_dense_product(x, w[:39], activation="swiglu")),
            (ep.EPError, lambda: ep.ep_dense_product(torch.zeros((4, 100), dtype=BF16, device=DEV)[:, :64], w)),
            (ValueError, lambda: ep.ep_dense_product_backward(grad, x, w, activation="gelu")),
            (ValueError, lambda: ep.ep_dense_product_backward(grad[:5], x, w)),
            (TypeError, lambda: ep.ep_dense_product_backward(grad.half(), x, w)),
            (TypeError, lambda: ep.ep_dense_product_backward(grad, x, w, bias_dtype=torch.float16)),
            (ep.EPError, lambda: ep.ep_dense_product_backward(grad, x, w, bias_dtype=F32, workspace=torch.empty(16, dtype=torch.uint8, device=DEV)))]:
        with pytest.raises(error):
            call()
