"""The experts' products and their gradients against plain 64-bit products.

Tolerances, fixed before any run.  A sum of n products of bf16 numbers (each
product exact in fp32) kept in fp32 errs by at most n * 2^-23 times the sum of
the products' absolute values S (2^-23 a step: the tensor cores may truncate
where fp32 arithmetic rounds); the result is rounded once to bf16.  Rounding
is monotone, so a result has to lie between the bf16 roundings of the 64-bit
value less and plus the bound.  silu has a slope of at most 1.1.
"""
import math

import pytest
import torch

import combine_ep_get_layout_gb300 as ep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rows_and_layout(T, K, E, H, align=1, seed=0, masked=0.0, only=None):
    """A routing (distinct experts a token; `only`: the experts that may be
    named), its expanded layout and rows; padding and unused rows are NaN."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    names = torch.arange(E, device=DEV) if only is None else torch.tensor(only, device=DEV)
    K = min(K, len(names))
    idx = names[torch.rand((T, len(names)), generator=g, device=DEV).argsort(1)[:, :K]]
    idx[torch.rand((T, K), generator=g, device=DEV) < masked] = -1
    idx = idx.contiguous()
    lay = ep.ep_get_layout_expanded(idx, E, align)
    cap = lay.capacity_bound()
    x = torch.full((cap, H), math.nan, dtype=torch.bfloat16, device=DEV)
    slot = lay.token_slot.reshape(-1).long()
    used = slot[slot >= 0]
    x[used] = torch.randn((len(used), H), generator=g, device=DEV).to(torch.bfloat16)
    return lay, x, used, g


def segments(lay):
    return list(zip(lay.expert_offset[:-1].tolist(), lay.num_rows_per_expert.tolist()))


def weights(g, E, N, H):
    return (torch.randn((E, N, H), generator=g, device=DEV) / math.sqrt(H)).to(torch.bfloat16)


def fp32_sum(a, b):
    """(a b^T, bound of an fp32 sum's error) in 64 bits."""
    return a.double() @ b.double().T, a.shape[1] * 2.0 ** -23 * (a.double().abs() @ b.double().abs().T)


def close(got, want, tol):
    low, high = ((want + s * tol).to(torch.bfloat16) for s in (-1, 1))
    assert bool(((low <= got) & (got <= high)).all()), float(((got.double() - want).abs() / (tol + 2.0 ** -8 * want.abs())).max())


SIZES = [
    # T, K, E, H, width, align, masked
    (1, 1, 1, 8, 8, 1, 0.0),
    (1, 2, 8, 64, 72, 1, 0.0),
    (5, 3, 16, 200, 136, 4, 0.3),
    (40, 2, 4, 256, 128, 16, 0.0),
    (129, 4, 4, 72, 264, 1, 0.0),
    (300, 2, 2, 136, 520, 128, 0.0),
    (600, 3, 5, 328, 104, 1, 0.1),
    (257, 1, 1, 1000, 256, 1, 0.0),
    (64, 6, 64, 512, 256, 8, 0.0),
    (700, 8, 300, 128, 64, 1, 0.2),
]


@pytest.mark.parametrize("T,K,E,H,width,align,masked", SIZES)
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_product(T, K, E, H, width, align, masked, act):
    lay, x, used, g = rows_and_layout(T, K, E, H, align, T + E, masked)
    wide = 2 * width if act else width
    w = weights(g, E, wide, H)
    out = torch.full((x.shape[0], width), 7.0, dtype=torch.bfloat16, device=DEV)
    pre = torch.full((x.shape[0], wide), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_product(x, w, lay, activation=act, out=out, preact=pre)
    again = ep.ep_expert_product(x, w, lay, activation=act)
    assert lay.errors() == 0
    assert torch.equal(out[used], again[used])
    untouched = torch.ones(x.shape[0], dtype=torch.bool, device=DEV)
    untouched[used] = False
    assert bool((out[untouched] == 7.0).all()) and bool((pre[untouched] == 7.0).all())
    for e, (a, n) in enumerate(segments(lay)):
        h, tol = fp32_sum(x[a:a + n], w[e])
        close(pre[a:a + n], h, tol)
        if act is None:
            close(out[a:a + n], h, tol)
        else:
            gate, up, tg, tu = h[:, :width], h[:, width:], tol[:, :width], tol[:, width:]
            s = gate * torch.sigmoid(gate)
            close(out[a:a + n], s * up, 1.1 * tg * (up.abs() + tu) + s.abs() * tu + 1e-6 * (s * up).abs())


@pytest.mark.parametrize("T,K,E,H,width,align,masked", SIZES)
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_gradients(T, K, E, H, width, align, masked, act):
    lay, x, used, g = rows_and_layout(T, K, E, H, align, T + 3 * E, masked)
    wide = 2 * width if act else width
    w = weights(g, E, wide, H)
    grad = torch.full((x.shape[0], width), math.nan, dtype=torch.bfloat16, device=DEV)
    grad[used] = torch.randn((len(used), width), generator=g, device=DEV).to(torch.bfloat16)
    pre = gp = None
    if act:
        pre = torch.full((x.shape[0], wide), math.nan, dtype=torch.bfloat16, device=DEV)
        ep.ep_expert_product(x, w, lay, activation=act, preact=pre)
        gp = torch.full((x.shape[0], wide), math.nan, dtype=torch.bfloat16, device=DEV)
    grad_x = torch.full((x.shape[0], H), 7.0, dtype=torch.bfloat16, device=DEV)
    grad_w = torch.full((E, wide, H), math.nan, dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_product_backward(grad, x, w, lay, activation=act, preact=pre, grad_x=grad_x, grad_w=grad_w,
                                  grad_preact=gp)
    again = ep.ep_expert_product_backward(grad, x, w, lay, activation=act, preact=pre)
    assert torch.equal(grad_x[used], again[0][used]) and torch.equal(grad_w, again[1])
    only_x = ep.ep_expert_product_backward(grad, x, w, lay, activation=act, preact=pre, need_w=False)
    only_w = ep.ep_expert_product_backward(grad, x, w, lay, activation=act, preact=pre, need_x=False)
    assert only_x[1] is None and only_w[0] is None
    assert torch.equal(only_x[0][used], grad_x[used]) and torch.equal(only_w[1], grad_w)
    untouched = torch.ones(x.shape[0], dtype=torch.bool, device=DEV)
    untouched[used] = False
    assert bool((grad_x[untouched] == 7.0).all())
    for e, (a, n) in enumerate(segments(lay)):
        d = grad[a:a + n]
        if act:  # the gradient through the activation, checked by itself
            p = pre[a:a + n].double()
            gate, up = p[:, :width], p[:, width:]
            sig = torch.sigmoid(gate)
            dg = d.double() * up * sig * (1 + gate * (1 - sig))
            close(gp[a:a + n, :width], dg, 1e-6 * (d.double() * up * sig).abs() * (1 + gate.abs()))
            close(gp[a:a + n, width:], d.double() * gate * sig, 1e-6 * (d.double() * gate * sig).abs())
            d = gp[a:a + n]
        want, tol = fp32_sum(d, w[e].T)
        close(grad_x[a:a + n], want, tol)
        want, tol = fp32_sum(d.T, x[a:a + n].T)
        close(grad_w[e], want, tol)


def test_gradients_against_differences():
    """A central difference of the 64-bit forward along random directions.
    The kernel's gradients carry bf16 roundings of the preactivation, its
    gradient and the results (4 of 2^-9, averaging over the sum): 2^-8 of the
    norm of the summed terms."""
    lay, x, used, g = rows_and_layout(30, 2, 4, 64, 1, 9)
    width = 48
    w = weights(g, 4, 2 * width, 64)
    pre = torch.zeros((x.shape[0], 2 * width), dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_product(x, w, lay, activation="swiglu", preact=pre)
    grad = torch.randn((x.shape[0], width), generator=g, device=DEV).to(torch.bfloat16)
    grad_x, grad_w = ep.ep_expert_product_backward(grad, x, w, lay, activation="swiglu", preact=pre)

    def f(xx, ww):
        total = 0.0
        for e, (a, n) in enumerate(segments(lay)):
            h = xx[a:a + n] @ ww[e].T
            total = total + (torch.nn.functional.silu(h[:, :width]) * h[:, width:] * grad[a:a + n].double()).sum()
        return float(total)

    xd, wd, step = x.double(), w.double(), 1e-5
    for _ in range(3):
        vx = torch.randn(x.shape, generator=g, device=DEV).double()
        vw = torch.randn(w.shape, generator=g, device=DEV).double()
        want = (f(xd + step * vx, wd) - f(xd - step * vx, wd)) / (2 * step)
        terms = grad_x.double() * vx
        assert abs(float(terms.sum()) - want) <= 2.0 ** -8 * float(terms.norm()) * 4
        want = (f(xd, wd + step * vw) - f(xd, wd - step * vw)) / (2 * step)
        terms = grad_w.double() * vw
        assert abs(float(terms.sum()) - want) <= 2.0 ** -8 * float(terms.norm()) * 4


@pytest.mark.parametrize("T,K,E,H,width,only", [(1021, 1, 1, 2048, 1000, None), (1024, 2, 4, 1024, 512, None),
                                                (600, 1, 2, 1024, 264, [1]), (2100, 1, 3, 512, 72, [0, 2]),
                                                (70, 1, 1, 4096, 8, None), (330, 1, 2, 4096, 136, [0])])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_few_experts(T, K, E, H, width, only, act):
    """Few tiles, which are cut narrower or shared by pairs, also where some
    experts get nothing and the others more than was reckoned with."""
    lay, x, used, g = rows_and_layout(T, K, E, H, 1, T, only=only)
    wide = 2 * width if act else width
    w = weights(g, E, wide, H)
    pre = torch.empty((x.shape[0], wide), dtype=torch.bfloat16, device=DEV)
    out = ep.ep_expert_product(x, w, lay, activation=act, preact=pre)
    assert torch.equal(out[used], ep.ep_expert_product(x, w, lay, activation=act)[used])
    grad = torch.randn((x.shape[0], width), generator=g, device=DEV).to(torch.bfloat16)
    gp = torch.zeros_like(pre)
    grad_x, grad_w = ep.ep_expert_product_backward(grad, x, w, lay, activation=act, preact=pre, grad_preact=gp)
    assert lay.errors() == 0
    for e, (a, n) in enumerate(segments(lay)):
        h, tol = fp32_sum(x[a:a + n], w[e])
        close(pre[a:a + n], h, tol)
        if act is None:
            close(out[a:a + n], h, tol)
        else:
            gate, up, tg, tu = h[:, :width], h[:, width:], tol[:, :width], tol[:, width:]
            s = gate * torch.sigmoid(gate)
            close(out[a:a + n], s * up, 1.1 * tg * (up.abs() + tu) + s.abs() * tu + 1e-6 * (s * up).abs())
        d = (gp if act else grad)[a:a + n]
        want, tol = fp32_sum(d, w[e].T)
        close(grad_x[a:a + n], want, tol)
        want, tol = fp32_sum(d.T, x[a:a + n].T)
        close(grad_w[e], want, tol)


@pytest.mark.parametrize("act", [None, "swiglu"])
def test_experts_without_rows(act):
    lay, x, used, g = rows_and_layout(50, 2, 16, 128, 1, 4, only=[3, 9, 10])
    w = weights(g, 16, 128, 128)
    w[0], w[15] = math.nan, math.inf  # weights that no row meets
    width = 64 if act else 128
    pre = torch.empty((x.shape[0], 128), dtype=torch.bfloat16, device=DEV)
    out = ep.ep_expert_product(x, w, lay, activation=act, preact=pre)
    assert torch.isfinite(out[used]).all()
    grad = torch.randn((x.shape[0], width), generator=g, device=DEV).to(torch.bfloat16)
    grad_x, grad_w = ep.ep_expert_product_backward(grad, x, w, lay, activation=act, preact=pre)
    assert torch.isfinite(grad_x[used]).all()
    empty = [e for e in range(16) if e not in (3, 9, 10)]
    assert bool((grad_w[empty] == 0).all()) and bool((grad_w[3] != 0).any())


def test_counts_beyond_num_tokens_are_cut_and_flagged():
    """A layout whose counts belong to more tokens than it says: rows past
    num_tokens an expert are skipped and flagged, the others computed."""
    lay, x, used, g = rows_and_layout(100, 1, 2, 64, 1, 12)
    w = weights(g, 2, 64, 64)
    want = ep.ep_expert_product(x, w, lay)
    assert lay.errors() == 0
    lay.num_tokens = 20
    out = torch.full((x.shape[0], 64), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_product(x, w, lay, out=out)
    assert lay.errors() == ep.EP_ERRBIT_CAPACITY
    for a, n in segments(lay):
        keep = min(n, 20)
        assert torch.equal(out[a:a + keep], want[a:a + keep]) and bool((out[a + keep:a + n] == 7.0).all())


def test_no_tokens():
    idx = torch.empty((0, 2), dtype=torch.int64, device=DEV)
    lay = ep.ep_get_layout_expanded(idx, 4, 1)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    w = torch.randn((4, 32, 64), device=DEV).to(torch.bfloat16)
    assert ep.ep_expert_product(x, w, lay).shape == (0, 32)
    gx, gw = ep.ep_expert_product_backward(torch.empty((0, 32), dtype=torch.bfloat16, device=DEV), x, w, lay)
    assert gx.shape == (0, 64) and bool((gw == 0).all())


def test_nan_and_infinity_stay_in_their_rows():
    """A row's NaN reaches its own outputs and no other row's."""
    lay, x, used, g = rows_and_layout(90, 2, 3, 136, 1, 5)
    w = weights(g, 3, 64, 136)
    want = ep.ep_expert_product(x, w, lay)
    bad = used[:5]
    y = x.clone()
    y[bad[0]] = math.nan
    y[bad[1]] = math.inf
    got = ep.ep_expert_product(y, w, lay)
    rest = used[~torch.isin(used, bad[:2])]
    assert torch.equal(got[rest], want[rest])
    assert torch.isnan(got[bad[0]]).all() and not torch.isfinite(got[bad[1]]).any()
    # an infinite gradient in one expert's row leaves the other experts' weights alone
    grad = torch.randn((x.shape[0], 64), generator=g, device=DEV).to(torch.bfloat16)
    _, gw = ep.ep_expert_product_backward(grad, x, w, lay, need_x=False)
    a, n = segments(lay)[1]
    grad[a] = math.inf
    _, gw2 = ep.ep_expert_product_backward(grad, x, w, lay, need_x=False)
    assert torch.equal(gw[[0, 2]], gw2[[0, 2]])


def test_rows_past_the_capacity_are_flagged_and_skipped():
    lay, x, used, g = rows_and_layout(64, 2, 4, 64, 1, 6)
    w = weights(g, 4, 64, 64)
    want = ep.ep_expert_product(x, w, lay)
    assert lay.errors() == 0
    cap = 70  # of 128 rows
    out = torch.full((128, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_product(x[:cap], w, lay, out=out[:cap])
    assert lay.errors() == ep.EP_ERRBIT_CAPACITY
    assert torch.equal(out[:cap], want[:cap]) and bool((out[cap:] == 7.0).all())


CUT = [
    # rows of each expert, capacity, H, width
    ((300, 300, 300, 300), 1080, 1024, 4096),      # tiles of 160 columns, the cut one of 192
    ((260, 260), 516, 256, 8192),                  # 160, 256
    ((300, 1, 300), 481, 6144, 4104),              # the rows' gradient too
    ((390,) * 16, 390 * 15 + 230, 1032, 704),      # 224, 256
    ((65, 400, 260, 500), 700, 328, 264),          # one cut, one without a row
    ((300, 300, 300, 300), 1080, 1024, 512),       # tiles cut narrower
]


def counted_layout(counts):
    """The layout of one choice a token: the first tokens the first expert's, and so on."""
    idx = torch.cat([torch.full((n,), e) for e, n in enumerate(counts)])[:, None].to(DEV).contiguous()
    lay = ep.ep_get_layout_expanded(idx, len(counts))
    assert lay.num_rows_per_expert.tolist() == list(counts)
    return lay


@pytest.mark.parametrize("counts,cap,H,width", CUT)
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_a_capacity_that_cuts_an_expert(counts, cap, H, width, act):
    """Hundreds of rows an expert, and a capacity inside one's segment, whose
    tiles may then be wider than the whole ones': every row below the capacity
    is right, in the outputs and in the rows' and the weights' gradients, and
    no row past it is touched."""
    g = torch.Generator(device=DEV).manual_seed(sum(counts) + cap)
    x = torch.randn((sum(counts), H), generator=g, device=DEV).to(torch.bfloat16)
    lay = counted_layout(counts)
    wide = 2 * width if act else width
    w = weights(g, len(counts), wide, H)
    out = torch.full((len(x), width), 7.0, dtype=torch.bfloat16, device=DEV)
    pre = torch.full((len(x), wide), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_product(x[:cap], w, lay, activation=act, out=out[:cap], preact=pre[:cap])
    assert lay.errors() == ep.EP_ERRBIT_CAPACITY
    assert bool((out[cap:] == 7.0).all()) and bool((pre[cap:] == 7.0).all())
    grad = torch.randn((len(x), width), generator=g, device=DEV).to(torch.bfloat16)
    grad_x = torch.full((len(x), H), 7.0, dtype=torch.bfloat16, device=DEV)
    gp = torch.zeros_like(pre)
    _, grad_w = ep.ep_expert_product_backward(grad[:cap], x[:cap], w, lay, activation=act, preact=pre[:cap] if act else None,
                                              grad_x=grad_x[:cap], grad_preact=gp[:cap] if act else None)
    assert lay.errors() == ep.EP_ERRBIT_CAPACITY and bool((grad_x[cap:] == 7.0).all())
    for e, (a, n) in enumerate(segments(lay)):
        here = slice(a, max(a, min(a + n, cap)))
        h, tol = fp32_sum(x[here], w[e])
        close(pre[here], h, tol)
        if act is None:
            close(out[here], h, tol)
        else:
            gate, up, tg, tu = h[:, :width], h[:, width:], tol[:, :width], tol[:, width:]
            s = gate * torch.sigmoid(gate)
            close(out[here], s * up, 1.1 * tg * (up.abs() + tu) + s.abs() * tu + 1e-6 * (s * up).abs())
        d = (gp if act else grad)[here]
        want, tol = fp32_sum(d, w[e].T)
        close(grad_x[here], want, tol)
        want, tol = fp32_sum(d.T, x[here].T)
        close(grad_w[e], want, tol)


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("what", ["no capacity", "no tokens"])
def test_rows_that_are_all_skipped_are_flagged(what, act):
    """A capacity of no rows, and a layout whose num_tokens says none: the
    layout's rows are skipped and flagged as any others, and gradients of the
    weights are zero."""
    lay, x, used, g = rows_and_layout(64, 2, 4, 64, 1, 6)
    w = weights(g, 4, 64, 64)
    width = 32 if act else 64
    if what == "no capacity":
        x = x[:0]
    else:
        lay.num_tokens = 0
    out = torch.full((x.shape[0], width), 7.0, dtype=torch.bfloat16, device=DEV)
    pre = torch.full((x.shape[0], 64), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_product(x, w, lay, activation=act, out=out, preact=pre)
    assert lay.errors() == ep.EP_ERRBIT_CAPACITY and bool((out == 7.0).all()) and bool((pre == 7.0).all())
    for need_x, need_w in ((True, False), (False, True), (True, True)):
        lay.error_word.zero_()
        grad_x = torch.full((x.shape[0], 64), 7.0, dtype=torch.bfloat16, device=DEV) if need_x else None
        _, grad_w = ep.ep_expert_product_backward(out, x, w, lay, activation=act, preact=pre if act else None,
                                                  grad_x=grad_x, need_x=need_x, need_w=need_w)
        assert lay.errors() == ep.EP_ERRBIT_CAPACITY
        assert not need_x or bool((grad_x == 7.0).all())
        assert not need_w or bool((grad_w == 0).all())


def test_another_stream():
    lay, x, used, g = rows_and_layout(512, 4, 8, 512, 1, 8)
    w = weights(g, 8, 512, 512)
    want = ep.ep_expert_product(x, w, lay, activation="swiglu")
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y = x * 1.0
        ep.ep_expert_product(y, w, lay, activation="swiglu", out=out)
    s.synchronize()
    assert torch.equal(out[used], want[used])


def delay(stream):
    """Some 10 ms of work on a stream."""
    with torch.cuda.stream(stream):
        m = torch.ones((4096, 4096), device=DEV)
        for _ in range(8):
            m = m @ m * 1e-4


def test_what_a_call_allocates_belongs_to_its_stream():
    """Memory that a call takes and gives back for itself is not handed to
    the current stream while the call's own stream still uses it."""
    lay, x, used, g = rows_and_layout(512, 4, 8, 512, 1, 8)
    w = weights(g, 8, 1024, 512)
    grad = torch.randn((x.shape[0], 512), generator=g, device=DEV).to(torch.bfloat16)
    pre = torch.empty((x.shape[0], 1024), dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_product(x, w, lay, activation="swiglu", preact=pre)
    want = ep.ep_expert_product_backward(grad, x, w, lay, activation="swiglu", preact=pre)
    out = [torch.empty_like(t) for t in want]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    delay(s)
    ep.ep_expert_product_backward(grad, x, w, lay, activation="swiglu", preact=pre, grad_x=out[0], grad_w=out[1],
                                  stream=s)
    held = [torch.zeros_like(pre) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(out[0][used], want[0][used]) and torch.equal(out[1], want[1])
    assert not any(t.any() for t in held)


@pytest.mark.parametrize("act", [None, "swiglu"])
def test_offsets_past_32_bits(act):
    """Rows, weights and their gradients of more than 2^31 elements each; the
    last of them are checked."""
    E, H, wide = 9, 16384, 16384
    width = wide // 2 if act else wide
    lay, x, used, g = rows_and_layout(70000, 2, E, H, 1, 1)
    w = torch.randn((E, wide, H), generator=g, device=DEV, dtype=torch.bfloat16) / 128
    pre = torch.empty((x.shape[0], wide), dtype=torch.bfloat16, device=DEV) if act else None
    out = ep.ep_expert_product(x, w, lay, activation=act, preact=pre)
    assert lay.errors() == 0 and x.numel() > 2 ** 31 and w.numel() > 2 ** 31
    first, n = segments(lay)[-1]
    end = first + n
    last = slice(end - 16, end)
    h, tol = fp32_sum(x[last], w[-1])
    if act is None:
        close(out[last], h, tol)
    else:
        close(pre[last], h, tol)
        gate, up, tg, tu = h[:, :width], h[:, width:], tol[:, :width], tol[:, width:]
        s = gate * torch.sigmoid(gate)
        close(out[last], s * up, 1.1 * tg * (up.abs() + tu) + s.abs() * tu + 1e-6 * (s * up).abs())
    grad = out.normal_(generator=g)
    gp = torch.empty_like(pre) if act else None
    grad_x, grad_w = ep.ep_expert_product_backward(grad, x, w, lay, activation=act, preact=pre, grad_preact=gp)
    d = gp if act else grad
    want, tol = fp32_sum(d[last], w[-1].T)
    close(grad_x[last], want, tol)
    want, tol = fp32_sum(d[first:end, -16:].T, x[first:end].T)
    close(grad_w[-1, -16:], want, tol)
    del x, w, pre, out, grad, gp, grad_x, grad_w, d, want, tol, h
    torch.cuda.empty_cache()


def test_a_layer_end_to_end():
    """Router, expanded layout, dispatch, both products, combine: the whole
    layer against 64 bits.  The hidden rows are rounded to bf16 once, as the
    reference's are, then each output and the combine once more: 3 roundings
    of 2^-9 against the sum of absolute terms."""
    T, H, F, E, K = 200, 128, 192, 16, 4
    g = torch.Generator(device=DEV).manual_seed(31)
    x = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    gate = (torch.randn((E, H), generator=g, device=DEV) / math.sqrt(H)).to(torch.bfloat16)
    w1, w2 = weights(g, E, 2 * F, H), weights(g, E, H, F)
    logits = x.float() @ gate.float().T
    r = ep.ep_route(logits, K, score="sigmoid", num_groups=4, topk_groups=2, group_top=2)
    lay = ep.ep_get_layout_expanded(r.topk_idx, E, 8)
    d = ep.ep_dispatch_expanded(x, r.topk_idx, r.topk_weights, lay, 4)
    hidden = ep.ep_expert_product(d.recv_x, w1, lay, activation="swiglu")
    y = ep.ep_expert_product(hidden, w2, lay)
    out = ep.ep_combine_expanded(y, lay, r.topk_idx, r.topk_weights)
    want = torch.zeros((T, H), dtype=torch.float64, device=DEV)
    size = torch.zeros_like(want)
    for k in range(K):
        e = r.topk_idx[:, k]
        h = torch.einsum("th,tnh->tn", x.double(), w1.double()[e])
        h = torch.nn.functional.silu(h[:, :F]) * h[:, F:]
        p = r.topk_weights[:, k:k + 1].double()
        want += p * torch.einsum("tf,thf->th", h, w2.double()[e])
        size += p * torch.einsum("tf,thf->th", h.abs(), w2.double()[e].abs())
    err = (out.double() - want).abs()
    assert bool((err <= 3 * 2.0 ** -9 * size).all())
