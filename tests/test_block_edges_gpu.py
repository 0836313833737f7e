"""Edges of the block's operators: more choices than 32 bits count, gradients over
logits that are not of whole 16 bytes, rows beside masked ones, rows whose mean
is far above their deviation, a product's ``grad_preact`` whatever else is
asked for, the far tail of GELU, what ReLU cuts off.
"""
import math

import pytest
import torch

import combine_ep_get_layout_gb300 as ep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


# ------------------------------------------------------------ balance loss

@pytest.mark.parametrize("tokens", [2 ** 28, 2 ** 29, 2 ** 29 + 1000])
@pytest.mark.parametrize("split", [False, True])
def test_more_choices_than_32_bits_count(tokens, split):
    """2^31 choices and more, equal scores: the loss is 1 and every quotient a
    power of two or near it.  p = 1/8; a sum of it is rounded at each of at
    most 600 joins of segments."""
    E = K = 8
    try:
        l = torch.zeros((tokens, E), dtype=BF16, device=DEV)
        idx = torch.arange(K, device=DEV).expand(tokens, K).contiguous()
    except torch.OutOfMemoryError:
        pytest.skip("no room")
    cuts = [0, 3, tokens - 500, tokens] if split else [0, tokens]
    off = torch.tensor(cuts, dtype=torch.int32, device=DEV)
    b = ep.ep_balance_loss(l, idx, seq_offsets=off)
    n = (off[1:] - off[:-1]).double()[:, None]
    near = 600 * U
    assert torch.equal(b.counts.double(), n.expand(-1, E))
    assert ((b.probs.double() - 1 / E).abs() <= near / E).all()
    assert ((b.slopes.double() * n * (len(cuts) - 1) - 1).abs() <= 8 * U).all()
    assert abs(float(b.losses[0]) - 1.0) <= 2 * near
    grad = ep.ep_balance_loss_backward(torch.tensor([1.0, 0.0], device=DEV), l, b, seq_offsets=off)
    assert float(grad.abs().max()) <= near  # balanced: nothing pulls


def test_an_expert_named_more_often_than_32_bits_count():
    """All choices name one expert: its share is 1, its count stops at the type's end."""
    T, K, E = 2 ** 28 + 77, 8, 8
    try:
        l = torch.zeros((T, E), dtype=BF16, device=DEV)
        idx = torch.full((T, K), 3, dtype=torch.int64, device=DEV)
    except torch.OutOfMemoryError:
        pytest.skip("no room")
    b = ep.ep_balance_loss(l, idx)
    want = torch.zeros(E, dtype=torch.int32, device=DEV)
    want[3] = 2 ** 31 - 1
    assert torch.equal(b.counts[0], want)
    assert abs(float(b.losses[0]) - 1.0) <= 1200 * U
    assert abs(float(b.slopes[0, 3]) * T / E - 1.0) <= 8 * U and float(b.slopes.sum()) == float(b.slopes[0, 3])


def logits_of(T, E, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    l = (torch.randn((T, E), generator=g, device=DEV) * 1.5).to(dtype)
    return l, torch.argsort(l.float(), dim=1, descending=True)[:, :min(4, E)].contiguous()


@pytest.mark.parametrize("T,E", [(18, 63), (50, 63), (45, 101), (1021, 255), (301, 301), (77, 999), (5, 2047), (40, 9)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_over_logits_off_16_bytes(T, E, dtype, score):
    """In place, rows that are not of whole 16 bytes, masked first rows: the bits of the call that writes elsewhere."""
    l, idx = logits_of(T, E, dtype, T)
    l[::32] = -math.inf
    b = ep.ep_balance_loss(l, idx, score=score)
    g = torch.tensor([0.7, 0.3], device=DEV)
    add = (torch.randn((T, E), device=DEV) * 1e-3).to(dtype)
    for more in (None, add):
        want = ep.ep_balance_loss_backward(g, l, b, score=score, add=more)
        for _ in range(5):
            mine = l.clone()
            assert torch.equal(ep.ep_balance_loss_backward(g, mine, b, score=score, add=more, out=mine), want)
            if more is not None:
                mine = more.clone()
                assert torch.equal(ep.ep_balance_loss_backward(g, l, b, score=score, add=mine, out=mine), want)


EDGES = [(8, 8), (18, 60), (50, 64), (45, 100), (77, 200), (50, 256), (37, 300), (40, 512), (20, 1000), (6, 2048)]


@pytest.mark.parametrize("T,E", EDGES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_row_does_not_change_with_its_neighbours(T, E, dtype, score):
    """The same bits beside rows that are masked, NaN or huge.  A sequence a
    token, so that ``probs`` are one row's scores."""
    l, idx = logits_of(T, E, dtype, T + E)
    off = torch.arange(T + 1, dtype=torch.int32, device=DEV)
    g = torch.tensor([0.7, 0.3], device=DEV)
    other = l.clone()
    strange = [i for i in (0, 5, 7, 17, 34, 44, T - 2) if i < T]
    for i, value in zip(strange, [-math.inf, math.nan, 3e38, -math.inf, -90.0, -math.inf, -math.inf]):
        other[i] = value
    keep = [i for i in range(T) if i not in strange]
    b = ep.ep_balance_loss(l, idx, score=score, seq_offsets=off)
    c = ep.ep_balance_loss(other, idx, score=score, seq_offsets=off)
    assert torch.equal(b.probs[keep], c.probs[keep])
    d, e = (ep.ep_balance_loss_backward(g, x, b, score=score, seq_offsets=off) for x in (l, other))
    assert torch.equal(d[keep], e[keep])


# -------------------------------------------------------------- layer norm

NORMS = [(1, 8), (9, 31), (13, 64), (50, 300), (20, 768), (300, 1000), (3, 2047), (200, 4096), (9, 7168), (5, 8200), (40, 10000),
         (700, 16384)]


@pytest.mark.parametrize("T,H", NORMS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_of_constant_rows(T, H, dtype):
    """n is 0 exactly, whatever the level, so the weight's gradient is too, and
    grad_x is rstd (g w - mean(g w)): H/32 + 40 roundings of a sum of absolute
    values.  The last rows' mean times rstd passes fp32's end."""
    g = torch.Generator(device=DEV).manual_seed(T + H)
    level = (torch.tensor([1000.1, -7.3, 0.0, 1e6, 1e30], device=DEV).repeat(T // 5 + 1)[:T]).to(dtype)
    x = level[:, None].expand(T, H).contiguous()
    grad = torch.randn((T, H), generator=g, device=DEV).to(dtype)
    w = 1 + 0.2 * torch.randn(H, generator=g, device=DEV)
    mean = level.float()
    for eps in (1e-5, 1e-30):
        rstd = torch.full((T,), eps ** -0.5, device=DEV)
        dx, dw, db = ep.ep_layer_norm_backward(grad, x, mean, rstd, w)
        assert (dw == 0).all()
        gw = grad.double() * w.double()
        want = rstd.double()[:, None] * (gw - gw.mean(1, keepdim=True))
        tol = rstd.double()[:, None] * U * ((H / 32 + 40) * gw.abs().mean(1, keepdim=True) + 6 * gw.abs())
        assert ((dx.double() - want).abs() <= tol + torch.finfo(dtype).eps / 2 * want.abs()).all()


@pytest.mark.parametrize("T,H", NORMS)
@pytest.mark.parametrize("ratio", [30.0, 3e3, 3e5])
def test_gradients_of_rows_with_a_far_mean(T, H, ratio):
    """With the statistics as given, n = (x - mean) rstd has the roundings of
    a difference, a factor and a product: 3 U |n|, however far the mean.  The
    sums as in the tests of the norm: H/32 + 34 roundings of a row's, of a
    parameter's T at most (T/8 + 640 from there)."""
    g = torch.Generator(device=DEV).manual_seed(T + H)
    x = ratio + torch.randn((T, H), generator=g, device=DEV)
    grad, w = torch.randn((T, H), generator=g, device=DEV), 1 + 0.2 * torch.randn(H, generator=g, device=DEV)
    mean, rstd = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    ep.ep_layer_norm(x, w, mean=mean, rstd=rstd)
    dx, dw, db = ep.ep_layer_norm_backward(grad, x, mean, rstd, w)
    m, r = mean.double()[:, None], rstd.double()[:, None]
    n = (x.double() - m) * r
    gw = grad.double() * w.double()
    a, b = gw.mean(1, keepdim=True), (gw * n).mean(1, keepdim=True)
    c = U * (H / 32 + 34)
    want = r * (gw - a - n * b)
    off_a = c * gw.abs().mean(1, keepdim=True)
    off_b = (c + 4 * U) * (gw * n).abs().mean(1, keepdim=True)
    tol = r * (off_a + off_b * n.abs() + U * (6 * gw.abs() + 6 * a.abs() + 9 * (n * b).abs()))
    assert ((dx.double() - want).abs() <= 1.01 * tol + U * want.abs()).all()
    t = U * (min(T, T / 8 + 640) + 6)
    assert ((dw.double() - (grad.double() * n).sum(0)).abs() <= 1.01 * t * (grad.double() * n).abs().sum(0)).all()


# ---------------------------------------------------------- shared product

@pytest.mark.parametrize("width", [16, 12])
@pytest.mark.parametrize("act", [None, "silu", "swiglu"])
@pytest.mark.parametrize("grad_type", [BF16, F32])
def test_grad_preact_is_written_whatever_is_needed(act, grad_type, width):
    g = torch.Generator(device=DEV).manual_seed(5)
    wide = width * (2 if act == "swiglu" else 1)
    pitch = (wide + 7) // 8 * 8
    x = torch.randn((40, 64), generator=g, device=DEV).to(BF16)
    w = torch.randn((wide, 64), generator=g, device=DEV).to(BF16)
    grad = torch.randn((40, width), generator=g, device=DEV).to(grad_type)
    preact = torch.randn((40, wide), generator=g, device=DEV).to(BF16)
    z = preact.double().requires_grad_(True)
    F = torch.nn.functional
    y = F.silu(z) if act == "silu" else F.silu(z[:, :width]) * z[:, width:] if act else z
    want, = torch.autograd.grad(y, z, grad.double())
    for needs in [dict(need_x=False, need_w=False), dict(need_x=False, need_w=False, bias_dtype=F32), dict(need_w=False),
                  dict(need_x=False), dict(bias_dtype=F32)]:
        kept = torch.full((40, pitch), math.nan, dtype=BF16, device=DEV)
        got = ep.ep_dense_product_backward(grad, x, w, activation=act, preact=preact if act else None, grad_preact=kept, **needs)
        assert [t is not None for t in got] == [needs.get("need_x", True), needs.get("need_w", True), "bias_dtype" in needs]
        # a sigmoid's 2^-16, and the rounding to bf16
        assert ((kept[:, :wide].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -14) * want.abs() + 1e-3 * 2.0 ** -14).all()


def gelu64(z):
    """GELU and its derivative, relatively right in the tail: by erfc."""
    tail = 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
    density = torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return z * tail, tail + z * density, density


def tail_points():
    z = torch.cat([torch.linspace(-12.5, 12.5, 1601), torch.tensor([-0.0, 1e-6, -1e-6, -13.0, 13.0, 100.0, -100.0, 1e30, -1e30])])
    return z.to(BF16).to(DEV)


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("params", [None, F32])
def test_gelu_keeps_its_relative_accuracy_in_the_tail(out_dtype, params):
    """z itself is exact (one product by 1).  The normal integral's tail is a
    fit of 2^-22, an exponential of 2^-22, whose argument z^2/2 is rounded
    twice, and a dozen roundings: 2^-24 (24 + 2 z^2), relative."""
    z = tail_points()
    x = torch.zeros((z.numel(), 8), dtype=BF16, device=DEV)
    x[:, 0] = z
    w = torch.zeros((3, 8), dtype=BF16, device=DEV)
    w[:, 0] = 1.0
    out = ep.ep_dense_product(x, w, None if params is None else torch.zeros(3, device=DEV), activation="gelu", out_dtype=out_dtype)
    z = z.double()[:, None]
    want = gelu64(z)[0]
    tol = (U * (24 + 2 * z ** 2) + torch.finfo(out_dtype).eps / 2) * want.abs() + 1e-37
    tol = torch.where(torch.isfinite(tol), tol, 0.0)
    # beyond 13 the density leaves fp32's normal numbers
    far = z < -13.1
    err = (out.double() - want).abs()
    assert (err <= torch.where(far, 1e-36, tol)).all(), float((err / tol)[~far.expand_as(err)].max())


@pytest.mark.parametrize("width", [8, 3])
def test_gelu_derivative_in_the_tail(width):
    """A row at a time, so that the bias's gradient (fp32) is the derivative:
    the two terms' bounds as above."""
    z = tail_points()
    for i in range(0, z.numel() - width, width):
        at = z[i:i + width].clone()
        w = torch.zeros((width, 8), dtype=BF16, device=DEV)
        x, one = torch.zeros((1, 8), dtype=BF16, device=DEV), torch.ones((1, width), device=DEV)
        got = ep.ep_dense_product_backward(one, x, w, activation="gelu", preact=at[None], bias_dtype=F32)[2]
        v = at.double()
        y, d, density = gelu64(v)
        tol = U * (24 + 2 * v ** 2) * (torch.where(v != 0, (y / v).abs(), 0.5) + (v * density).abs()) + 1e-36
        assert ((got.double() - d).abs() <= torch.where(v.abs() > 20, 1e-36, tol)).all()


@pytest.mark.parametrize("width", [16, 5])
@pytest.mark.parametrize("grad_type", [BF16, F32])
def test_relu_lets_nothing_through_where_it_is_closed(grad_type, width):
    """Infinities and NaN of the output's gradient in places whose output was cut to 0."""
    g = torch.Generator(device=DEV).manual_seed(9)
    T, H, pitch = 70, 64, (width + 7) // 8 * 8
    x = torch.randn((T, H), generator=g, device=DEV).to(BF16)
    w = torch.randn((width, H), generator=g, device=DEV).to(BF16)
    preact = torch.randn((T, width), generator=g, device=DEV).to(BF16)
    preact[3] = 0.0
    preact[4] = -0.0
    grad = torch.randn((T, width), generator=g, device=DEV).to(grad_type)
    closed = preact <= 0
    clean = torch.where(closed, torch.zeros_like(grad), grad)
    for value in (math.inf, -math.inf, math.nan):
        kept = torch.empty((T, pitch), dtype=BF16, device=DEV)
        given = torch.where(closed, torch.full_like(grad, value), grad)
        got = ep.ep_dense_product_backward(given, x, w, activation="relu", preact=preact, bias_dtype=F32, grad_preact=kept)
        want = ep.ep_dense_product_backward(clean, x, w, activation="relu", preact=preact, bias_dtype=F32)
        assert (kept[:, :width][closed] == 0).all()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
