"""Layer norm and its gradients against plain 64-bit implementations.

Tolerances, fixed before any run.  A row's sum over at least 32 lanes has
H/32 + 32 roundings at most: c = 2^-24 (H/32 + 32) of the sum of absolute
values.  The mean is off by c mean|x|; a difference x - mean by that and
2^-23 (|x| + |mean|); the variance, relative, by 2c and twice the relative
error of its differences; the rest follows by the formulas, with the type's
rounding at the end.  A parameter's gradient sums T terms in slices of at
least T/512 rows and then the slices: 2^-24 (T/8 + 640) of the sum of
absolute values (T alone below 640).
"""
import math

import pytest
import torch

import combine_ep_get_layout_gb300 as ep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-5
U = 2.0 ** -24


def half(t):
    return torch.finfo(t).eps / 2


def statistics64(x):
    mean = x.mean(1, keepdim=True)
    return mean, ((x - mean) ** 2).mean(1, keepdim=True).add(EPS).rsqrt()


def check_forward(x, w, b, out, mean, rstd):
    H = x.shape[1]
    x64 = x.double()
    one = torch.ones(H, device=DEV, dtype=torch.float64)
    w64 = one if w is None else w.double()
    b64 = 0 * one if b is None else b.double()
    m, r = statistics64(x64)
    c = U * (H / 32 + 32)
    off_m = c * x64.abs().mean(1, keepdim=True)
    off_d = off_m + 2 * U * (x64.abs() + m.abs())  # of a difference
    # relative, of rstd: half of the variance's
    off_r = c + (((x64 - m).abs() * off_d).mean(1, keepdim=True) + (off_d ** 2).mean(1, keepdim=True)) * r ** 2 + 4 * U
    y = (x64 - m) * r * w64 + b64
    tol = half(out.dtype) * y.abs() + w64.abs() * r * off_d * 1.01 + ((x64 - m) * r * w64).abs() * (off_r + 4 * U) \
        + 4 * U * (y.abs() + b64.abs()) + 1e-38
    assert ((out.double() - y).abs() <= tol).all(), float(((out.double() - y).abs() / tol).max())
    if mean is not None:
        assert ((mean.double() - m[:, 0]).abs() <= off_m[:, 0] + 1e-38).all()
        assert ((rstd.double() - r[:, 0]).abs() <= (off_r * r)[:, 0]).all()


def backward64(g, x, mean, rstd, w, add):
    """The gradients with the given statistics, and bounds of their errors."""
    T, H = x.shape
    x, g, m, r = x.double(), g.double(), mean.double()[:, None], rstd.double()[:, None]
    w = torch.ones(H, device=DEV, dtype=torch.float64) if w is None else w.double()
    n = (x - m) * r
    off_n = 2 * U * (x.abs() + m.abs()) * r + 2 * U * n.abs()
    gw = g * w
    a, b = gw.mean(1, keepdim=True), (gw * n).mean(1, keepdim=True)
    c = U * (H / 32 + 34)
    off_a = c * gw.abs().mean(1, keepdim=True)
    off_b = c * (gw * n).abs().mean(1, keepdim=True) + (gw.abs() * off_n).mean(1, keepdim=True)
    d = r * (gw - a - n * b)
    tol = r * (off_a + off_b * n.abs() + off_n * b.abs() + 6 * U * (gw.abs() + a.abs() + (n * b).abs()))
    if add is not None:
        d = d + add.double()
        tol = tol + 2 * U * add.double().abs()
    t = U * min(T, T / 8 + 640)
    return d, tol, (g * n).sum(0), (g.abs() * off_n).sum(0) + (t + 2 * U) * (g * n).abs().sum(0), g.sum(0), t * g.abs().sum(0)


def check_backward(g, x, mean, rstd, w, add, got):
    d, tol, dw, tol_w, db, tol_b = backward64(g, x, mean, rstd, w, add)
    for name, v, want, t in (("x", got[0], d, tol), ("weight", got[1], dw, tol_w), ("bias", got[2], db, tol_b)):
        t = t * 1.01 + half(v.dtype) * want.abs() + 1e-38
        err = (v.double() - want).abs()
        assert (err <= t).all(), (name, float((err / t).max()))


def make(T, H, dtype, params, seed=0, shift=0.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    size = torch.exp(torch.randn(H, generator=g, device=DEV) * 0.5)
    x = (torch.randn((T, H), generator=g, device=DEV) * size + shift * torch.randn((T, 1), generator=g, device=DEV)).to(dtype)
    w = (1 + 0.2 * torch.randn(H, generator=g, device=DEV)).to(params)
    b = (0.1 * torch.randn(H, generator=g, device=DEV)).to(params)
    grad = torch.randn((T, H), generator=g, device=DEV).to(dtype)
    add = torch.randn((T, H), generator=g, device=DEV).to(dtype)
    return x, w, b, grad, add


def run(x, w, b, grad, add, **kw):
    T = x.shape[0]
    mean, rstd = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    out = ep.ep_layer_norm(x, w, b, eps=EPS, mean=mean, rstd=rstd)
    check_forward(x, w, b, out, mean, rstd)
    got = ep.ep_layer_norm_backward(grad, x, mean, rstd, w, add=add, **kw)
    check_backward(grad, x, mean, rstd, w, add, got)
    return out, mean, rstd, got


SHAPES = [(1, 1), (1, 8), (3, 2), (7, 31), (64, 33), (13, 64), (5, 100), (129, 128), (300, 250), (31, 256), (1000, 264),
          (9, 512), (17, 1000), (40, 1024), (333, 1032), (6, 2047), (77, 2048), (500, 4096), (3, 4104), (21, 5120), (2, 7167),
          (400, 7168), (10, 8192), (4, 10000), (19, 12288), (3, 16383), (30, 16384), (2049, 72)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dtype,params", [(torch.bfloat16, torch.float32), (torch.float32, torch.float32),
                                          (torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16)])
def test_against_64_bits(T, H, dtype, params):
    x, w, b, grad, add = make(T, H, dtype, params, seed=T + H)
    run(x, w, b, grad, add if (T + H) % 2 else None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_without_parameters(dtype):
    x, w, b, grad, add = make(50, 320, dtype, dtype)
    for weight, bias in ((None, None), (w, None), (None, b)):
        mean, rstd = torch.empty(50, device=DEV), torch.empty(50, device=DEV)
        check_forward(x, weight, bias, ep.ep_layer_norm(x, weight, bias, mean=mean, rstd=rstd), mean, rstd)
        got = ep.ep_layer_norm_backward(grad, x, mean, rstd, weight)
        assert got[1].dtype is got[2].dtype is (torch.float32 if weight is None else dtype)
        check_backward(grad, x, mean, rstd, weight, None, got)
    check_forward(x, w, b, ep.ep_layer_norm(x, w, b), None, None)  # statistics not kept
    mean = torch.empty(50, device=DEV)
    assert ep.ep_layer_norm(x, w, b, mean=mean) is not None  # one of them


def test_parts_of_the_gradients():
    x, w, b, grad, add = make(70, 512, torch.bfloat16, torch.float32)
    out, mean, rstd, full = run(x, w, b, grad, add)
    dx, dw, db = ep.ep_layer_norm_backward(grad, x, mean, rstd, w, add=add, need_params=False)
    assert dw is None and db is None and torch.equal(dx, full[0])
    dx, dw, db = ep.ep_layer_norm_backward(grad, x, mean, rstd, w, need_x=False)
    assert dx is None and torch.equal(dw, full[1]) and torch.equal(db, full[2])
    dw = torch.empty(512, device=DEV, dtype=torch.bfloat16)
    db = torch.empty(512, device=DEV, dtype=torch.bfloat16)
    got = ep.ep_layer_norm_backward(grad, x, mean, rstd, None, grad_weight=dw, grad_bias=db)
    assert got[1] is dw and got[2] is db
    check_backward(grad, x, mean, rstd, None, None, got)


def test_in_place():
    """out over x, grad_x over grad or add."""
    for dtype, H in ((torch.bfloat16, 1024), (torch.float32, 99)):
        x, w, b, grad, add = make(200, H, dtype, torch.float32)
        out, mean, rstd, (dx, dw, db) = run(x, w, b, grad, add)
        y = x.clone()
        assert ep.ep_layer_norm(y, w, b, eps=EPS, out=y) is y
        assert torch.equal(y, out)
        for over in ("grad", "add"):
            g, a = grad.clone(), add.clone()
            got = ep.ep_layer_norm_backward(g, x, mean, rstd, w, add=a, grad_x=g if over == "grad" else a)
            assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,wide,first", [(256, 512, 64), (256, 300, 0), (256, 264, 8), (100, 131, 3), (2000, 2001, 1)])
def test_rows_of_wider_ones(dtype, H, wide, first):
    big = torch.randn((37, wide), device=DEV).to(dtype)
    x, w, b, grad, add = make(37, H, dtype, torch.float32)
    x = big[:, first:first + H]
    keep = big.clone()
    run(x, w, b, grad, add)
    assert torch.equal(big, keep)


def test_tensors_off_16_bytes():
    """Tensors that start at an element that is not 16-byte aligned."""
    for dtype in (torch.bfloat16, torch.float32):
        x, w, b, grad, add = make(23, 640, dtype, dtype)

        def off(t):
            flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:]
            return flat.view(t.shape).copy_(t)

        want = run(x, w, b, grad, add)
        for i in range(5):
            args = [off(t) if i == j else t for j, t in enumerate((x, w, b, grad, add))]
            run(*args)
        out = off(x)
        ep.ep_layer_norm(x, w, b, eps=EPS, out=out)
        assert ((out.double() - want[0].double()).abs() <= 2 * half(dtype) * want[0].double().abs() + 1e-5).all()


def test_rows_that_are_not_finite_stay_with_themselves():
    x, w, b, grad, add = make(40, 512, torch.float32, torch.float32)
    clean = run(x, w, b, grad, add)
    y = x.clone()
    y[3, 100] = math.nan
    y[17, 5] = math.inf
    y[39] = -math.inf
    mean, rstd = torch.empty(40, device=DEV), torch.empty(40, device=DEV)
    out = ep.ep_layer_norm(y, w, b, eps=EPS, mean=mean, rstd=rstd)
    bad = [3, 17, 39]
    good = [i for i in range(40) if i not in bad]
    assert torch.isnan(out[bad]).all(1).sum() == 3 or not torch.isfinite(out[bad]).all(1).any()
    assert torch.equal(out[good], clean[0][good]) and torch.equal(mean[good], clean[1][good])
    dx, dw, db = ep.ep_layer_norm_backward(grad, y, mean, rstd, w, add=add)
    assert torch.equal(dx[good], clean[3][0][good])


def test_constant_rows_and_far_means():
    """A constant row's output is the bias; a mean 2^12 times the deviation
    costs that factor of the differences' rounding, as the bounds say."""
    w, b = torch.ones(768, device=DEV) * 1.5, torch.randn(768, device=DEV)
    x = torch.full((4, 768), 7.0, device=DEV)
    x[1] = 0.0
    x[2] = -1e30
    mean, rstd = torch.empty(4, device=DEV), torch.empty(4, device=DEV)
    out = ep.ep_layer_norm(x, w, b, eps=EPS, mean=mean, rstd=rstd)
    assert torch.equal(out[:2], b.expand(2, -1)) and torch.equal(mean[:2], x[:2, 0])
    g = torch.Generator(device=DEV).manual_seed(4)
    x = 4096.0 + torch.randn((20, 1000), generator=g, device=DEV)
    run(x, torch.ones(1000, device=DEV), torch.zeros(1000, device=DEV), torch.randn((20, 1000), device=DEV), None)


def test_no_rows():
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.empty((0, 96), device=DEV, dtype=dtype)
        w = torch.ones(96, device=DEV)
        none = torch.empty(0, device=DEV)
        assert ep.ep_layer_norm(x, w, w, mean=none, rstd=none).shape == (0, 96)
        dx, dw, db = ep.ep_layer_norm_backward(x, x, none, none, w)
        assert dx.shape == (0, 96) and (dw == 0).all() and (db == 0).all()


def test_gradient_by_differences():
    """Central differences of the 64-bit definition: h = 1e-5 leaves h^2 and
    1e-16 / h of the values' scale, 1e-9 and 1e-11."""
    x, w, b, grad, _ = make(6, 24, torch.float32, torch.float32, seed=12)
    mean, rstd = torch.empty(6, device=DEV), torch.empty(6, device=DEV)
    ep.ep_layer_norm(x, w, b, eps=EPS, mean=mean, rstd=rstd)
    got = ep.ep_layer_norm_backward(grad, x, mean, rstd, w)

    def f(x, w, b):
        m, r = statistics64(x)
        return float((((x - m) * r * w + b) * grad.double()).sum())

    base = [x.double(), w.double(), b.double()]
    for which, at in ((0, (0, 0)), (0, (3, 17)), (0, (5, 23)), (1, (0,)), (1, (20,)), (2, (7,))):
        v = []
        for h in (1e-5, -1e-5):
            args = [t.clone() for t in base]
            args[which][at] += h
            v.append(f(*args))
        assert abs((v[0] - v[1]) / 2e-5 - float(got[which][at])) < 1e-4


def test_the_same_bits_and_captured():
    x, w, b, grad, add = make(1500, 1024, torch.bfloat16, torch.float32)
    mean, rstd = torch.empty(1500, device=DEV), torch.empty(1500, device=DEV)

    def step():
        out = ep.ep_layer_norm(x, w, b, mean=mean, rstd=rstd)
        return (out, *ep.ep_layer_norm_backward(grad, x, mean, rstd, w, add=add))

    want = step()
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(want, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = ep.ep_layer_norm(x, w, b, stream=side)
    got = ep.ep_layer_norm_backward(grad, x, mean, rstd, w, add=add, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0]) and all(torch.equal(p, q) for p, q in zip(got, want[1:]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.normal_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, step()))


def test_more_than_2_31_elements():
    """Rows whose offsets pass 2^31 elements: the last ones as the same rows by themselves."""
    T, H = 2 ** 31 // 8192 + 5, 8192
    try:
        x = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
        out, grad, dx = torch.empty_like(x), torch.zeros_like(x), torch.empty_like(x)
    except torch.OutOfMemoryError:
        pytest.skip("no room")
    x[:-7] = 0
    x[-7:].normal_()
    grad[-7:].normal_()
    w, b = torch.rand(H, device=DEV) + 0.5, torch.randn(H, device=DEV)
    mean, rstd = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    ep.ep_layer_norm(x, w, b, out=out, mean=mean, rstd=rstd)
    assert torch.equal(out[-7:], ep.ep_layer_norm(x[-7:], w, b))
    _, dw, db = ep.ep_layer_norm_backward(grad, x, mean, rstd, w, grad_x=dx)
    small = ep.ep_layer_norm_backward(grad[-7:], x[-7:], mean[-7:], rstd[-7:], w)
    assert torch.equal(dx[-7:], small[0]) and (dx[:100] == 0).all()
    check_backward(grad[-7:], x[-7:], mean[-7:], rstd[-7:], w, None, (dx[-7:], dw, db))


def test_refusals():
    x, w, b, grad, add = make(10, 64, torch.bfloat16, torch.float32)
    m = torch.empty(10, device=DEV)
    for error, call in [
            (TypeError, lambda: ep.ep_layer_norm(x.half(), w, b)), (TypeError, lambda: ep.ep_layer_norm(x, w, b.bfloat16())),
            (TypeError, lambda: ep.ep_layer_norm(x, w.half(), b)), (ValueError, lambda: ep.ep_layer_norm(x, w[:60], b)),
            (ValueError, lambda: ep.ep_layer_norm(x[0], w, b)), (ValueError, lambda: ep.ep_layer_norm(x.T, w[:10], b[:10])),
            (ep.EPError, lambda: ep.ep_layer_norm(x, w, b, eps=0.0)), (ep.EPError, lambda: ep.ep_layer_norm(x, w, b, eps=math.nan)),
            (TypeError, lambda: ep.ep_layer_norm(x, w, b, mean=m.double())),
            (TypeError, lambda: ep.ep_layer_norm(x, w, b, out=grad.float())),
            (ValueError, lambda: ep.ep_layer_norm(x, w.cpu(), b)),
            (TypeError, lambda: ep.ep_layer_norm_backward(grad.float(), x, m, m, w)),
            (ValueError, lambda: ep.ep_layer_norm_backward(grad, x, m[:5], m, w)),
            (ValueError, lambda: ep.ep_layer_norm_backward(grad, x, m, m, w, add=add[:5])),
            (TypeError, lambda: ep.ep_layer_norm_backward(grad, x, m, m, w, grad_bias=torch.empty(64, device=DEV).bfloat16())),
            (ep.EPError, lambda: ep.ep_layer_norm_backward(grad, x, m, m, w, workspace=torch.empty(16, dtype=torch.uint8, device=DEV)))]:
        with pytest.raises(error):
            call()
    wide = torch.randn((4, 16384 + 8), device=DEV)
    with pytest.raises(ep.EPError):
        ep.ep_layer_norm(wide)
