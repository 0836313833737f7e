"""The router and its gradient against plain 64-bit implementations.

Tolerances, fixed before any run.  Indices are equal, except in rows where two
different keys lie closer than fp32 resolves (they are skipped, and few).
A weight is a quotient of positive fp32 sums: an exponential costs 2 ulp plus
the rounding of its argument (|l - m| ulp), a sum of n terms over 32 lanes
n/32 + 5 roundings, so 2^-24 * (32 + n/32 + 4 * max|l|), relative.
A gradient adds differences of such terms, so the same bound on the sum of
the absolute values of its terms; bf16 gradients add their rounding, 2^-8.
"""
import math
import threading

import numpy as np
import pytest
import torch

import combine_ep_get_layout_gb300 as ep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def scores64(l, score):
    """p of fp32 logits (numpy, [T, E]) in 64 bits; masked entries 0."""
    l = l.astype(np.float64)
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max))
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(np.isneginf(l), 0.0, 1.0 / (1.0 + np.exp(-l)))
    m = l.max(1, keepdims=True)
    m = np.where(np.isneginf(m), 0.0, m)
    e = np.exp(l - m)
    s = e.sum(1, keepdims=True)
    return e / np.where(s > 0, s, 1.0)


def route64(l, K, score, bias, G, Gk, top, renorm, scale):
    """(idx, weights, rows whose choice fp32 cannot resolve)."""
    T, E = l.shape
    masked = np.isnan(l) | np.isneginf(l)
    p = scores64(l, score)
    by_logit = bias is None and (G == 1 or top == 1)
    key = np.minimum(l.astype(np.float64), np.finfo(np.float32).max) if by_logit else p + (0.0 if bias is None else bias.astype(np.float64))
    key = np.where(masked, -np.inf, key)
    close = np.zeros(T, bool)

    def gaps(values, n):
        v = -np.sort(-values, axis=1)[:, :n]
        with np.errstate(invalid="ignore"):
            d = v[:, :-1] - v[:, 1:]
            size = 1.0 if bias is not None else np.abs(v[:, :-1])
            return ((d > 0) & (d < 4e-6 * size)).any(1)

    if G > 1:
        per = key.reshape(T, G, E // G)
        best = -np.sort(-per, axis=2)[:, :, :top]
        score_g = np.where(np.isneginf(best[:, :, 0]), -np.inf, np.where(np.isneginf(best), 0.0, best).sum(2))
        if not by_logit:
            close |= gaps(score_g, Gk + 1)
        order = np.argsort(-score_g, axis=1, kind="stable")[:, :Gk]
        keep = np.zeros((T, G), bool)
        np.put_along_axis(keep, order, True, 1)
        key = np.where(np.repeat(keep, E // G, 1), key, -np.inf)
    if not by_logit:
        close |= gaps(key, K + 1)
    idx = np.argsort(-key, axis=1, kind="stable")[:, :K]
    none = np.isneginf(np.take_along_axis(key, idx, 1))
    lm = np.where(masked, -np.inf, np.minimum(l.astype(np.float64), np.finfo(np.float32).max))
    chosen = np.where(none, -np.inf, np.take_along_axis(lm, idx, 1))
    if renorm:  # shares of the chosen, the largest exponential taken out: sigmoid(l) = exp(min(l, 0)) / (1 + exp(-|l|))
        low = np.minimum(chosen, 0.0) if score == "sigmoid" else chosen
        m = low.max(1, keepdims=True)
        e = np.exp(low - np.where(np.isneginf(m), 0.0, m))
        if score == "sigmoid":
            e = e / (1.0 + np.exp(-np.abs(chosen)))
        w = e / np.where(e.sum(1, keepdims=True) > 0, e.sum(1, keepdims=True), 1.0)
    else:
        w = np.where(none, 0.0, np.take_along_axis(p, idx, 1))
    return np.where(none, -1, idx), scale * w, close


def weight_tolerance(l):
    fin = l[np.isfinite(l) & (np.abs(l) < 1e3)]
    return 2.0 ** -24 * (32 + l.shape[1] / 32 + 4 * (np.abs(fin).max() if fin.size else 0.0))


def make_logits(T, E, dtype, seed, lattice=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, E), generator=g) * 1.5
    if lattice:  # few distinct values: many ties
        x = torch.round(x * 2) / 2
    return x.to(dtype)


def check(logits, K, score="softmax", bias=None, G=1, Gk=1, top=1, renorm=True, scale=1.0):
    r = ep.ep_route(logits.to(DEV), K, score=score, bias=None if bias is None else bias.to(DEV), num_groups=G,
                    topk_groups=Gk, group_top=top, renormalize=renorm, weight_scale=scale)
    l = logits.float().numpy()
    idx, w, close = route64(l, K, score, None if bias is None else bias.numpy(), G, Gk, top, renorm, scale)
    got_i, got_w = r.topk_idx.cpu().numpy(), r.topk_weights.cpu().numpy()
    assert close.mean() < 0.05 or len(close) < 40
    ok = ~close
    np.testing.assert_array_equal(got_i[ok], idx[ok])
    np.testing.assert_allclose(got_w[ok], w[ok], rtol=weight_tolerance(l), atol=1e-37)
    return r


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 8, 8), (3, 7, 3), (13, 64, 6), (37, 33, 32), (130, 256, 8),
                                   (257, 257, 5), (70, 512, 10), (9, 520, 8), (5, 1000, 32), (3, 4096, 8)])
def test_sizes_and_types(T, E, K, score, dtype):
    for renorm, bias in ((True, None), (False, None), (True, "b"), (False, "b")):
        b = torch.randn(E, generator=torch.Generator().manual_seed(5)) * 0.1 if bias else None
        check(make_logits(T, E, dtype, T + E), K, score, b, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,Gk,K", [(64, 8, 4, 6), (256, 8, 3, 8), (256, 64, 2, 8), (96, 3, 2, 32), (40, 40, 5, 4),
                                      (1024, 16, 16, 8), (72, 2, 1, 16)])
@pytest.mark.parametrize("top", [1, 2])
def test_groups(E, G, Gk, K, top, score):
    bias = torch.randn(E, generator=torch.Generator().manual_seed(7)) * 0.1
    for b in (None, bias):
        check(make_logits(150, E, torch.float32, E + G), K, score, b, G, Gk, top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,Gk,top", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
def test_ties_go_to_the_lowest_index(G, Gk, top, score):
    check(make_logits(200, 64, torch.float32, 1, lattice=True), 8, score, None, G, Gk, top)
    check(torch.zeros((4, 64)), 8, score, None, G, Gk, top)
    check(torch.zeros((4, 64)), 8, score, torch.zeros(64), G, Gk, top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("G,Gk,top", [(1, 1, 1), (8, 2, 2)])
def test_masks_and_extremes(score, bias, G, Gk, top):
    E, K = 64, 8
    x = make_logits(64, E, torch.float32, 3)
    low = torch.finfo(torch.float32).min
    x[0] = -math.inf                      # nothing offered
    x[1] = low                            # the type's lowest value everywhere: offered, and equal
    x[2, :60] = -math.inf                 # fewer offered than asked
    x[3, ::2] = math.nan
    x[4] = math.nan
    x[5, 7] = math.inf
    x[6, 7] = math.inf
    x[6, 9] = math.inf
    x[7] = 1e30 * torch.sign(x[7])
    x[8, 5:] = low
    x[9] = -200.0                         # sigmoid underflows
    x[10:20].masked_fill_(torch.rand((10, E), generator=torch.Generator().manual_seed(2)) < 0.9, -math.inf)
    b = torch.randn(E, generator=torch.Generator().manual_seed(7)) * 0.1 if bias else None
    r = check(x, K, score, b, G, Gk, top)
    idx, w = r.topk_idx.cpu(), r.topk_weights.cpu()
    assert (idx[0] == -1).all() and (w[0] == 0).all() and (idx[4] == -1).all()
    assert torch.isfinite(w).all()
    check(x, K, score, b, G, Gk, top, renorm=False)


def test_rows_may_be_a_slice_of_wider_ones():
    wide = make_logits(50, 96, torch.float32, 4).to(DEV)
    part = wide[:, 16:80]
    a = ep.ep_route(part, 6)
    b = ep.ep_route(part.contiguous(), 6)
    assert torch.equal(a.topk_idx, b.topk_idx) and torch.equal(a.topk_weights, b.topk_weights)
    odd = wide.to(torch.bfloat16)[:, 3:40]  # rows start at odd places
    a, b = ep.ep_route(odd, 5), ep.ep_route(odd.contiguous(), 5)
    assert torch.equal(a.topk_idx, b.topk_idx) and torch.equal(a.topk_weights, b.topk_weights)
    g = torch.randn((50, 5), device=DEV)
    ga = ep.ep_route_backward(g, odd, a.topk_idx, renormalize=False)
    gb = ep.ep_route_backward(g, odd.contiguous(), a.topk_idx, renormalize=False)
    assert torch.equal(ga, gb)


def test_no_tokens_and_other_streams():
    r = ep.ep_route(torch.empty((0, 16), device=DEV), 4)
    assert r.topk_idx.shape == (0, 4)
    assert ep.ep_route_backward(torch.empty((0, 4), device=DEV), torch.empty((0, 16), device=DEV),
                                torch.empty((0, 4), dtype=torch.int64, device=DEV)).shape == (0, 16)
    x = make_logits(3000, 256, torch.float32, 8).to(DEV)
    want = ep.ep_route(x, 8, score="sigmoid")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = ep.Routing(torch.zeros((3000, 8), dtype=torch.int64, device=DEV), torch.zeros((3000, 8), device=DEV))
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        y = x * 1.0
        ep.ep_route(y, 8, score="sigmoid", out=out)
    s.synchronize()
    assert torch.equal(out.topk_idx, want.topk_idx) and torch.equal(out.topk_weights, want.topk_weights)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,Gk,top,K", [(8, 1, 1, 1, 3), (33, 1, 1, 1, 8), (40, 5, 2, 2, 6), (60, 3, 2, 1, 4), (60, 15, 6, 2, 16)])
@pytest.mark.parametrize("bias", [False, True])
def test_a_token_goes_to_the_same_experts_in_any_batch(E, G, Gk, top, K, score, bias):
    """Many near ties: the logits come in pairs a few units in the last place
    apart, with the same bias.  Few tokens and many take different kernels,
    which compare the same keys."""
    g = torch.Generator().manual_seed(E + K)
    half = E // 2
    x = make_logits(6000, E, torch.float32, E + G)
    x[:, half:2 * half] = x[:, :half] * (1.0 + torch.randint(-3, 4, (6000, half), generator=g) * 2.0 ** -23)
    x[::7].masked_fill_(torch.rand(x[::7].shape, generator=g) < 0.3, -math.inf)
    b = None
    if bias:
        b = torch.randn(E, generator=g) * 0.05
        b[half:2 * half] = b[:half]
        b = b.to(DEV)
    x = x.to(DEV)
    how = dict(score=score, bias=b, num_groups=G, topk_groups=Gk, group_top=top)
    whole = ep.ep_route(x, K, **how).topk_idx
    for n in (1, 700, 4096):
        part = torch.cat([ep.ep_route(x[i:i + n], K, **how).topk_idx for i in range(0, 6000 if n > 1 else 20, n)])
        assert torch.equal(part, whole[:len(part)]), int((part != whole[:len(part)]).any(1).sum())


def test_threads_with_other_counts_of_experts():
    """Calls with more and with fewer experts from several threads at once:
    none refuses another's launch, whose shared memory goes by its experts."""
    errors, results = [], {}

    def go(name, x):
        try:
            out = ep.ep_route(x, 4)
            for _ in range(4000):
                ep.ep_route(x, 4, out=out)
            results[name] = out
        except ep.EPError as e:
            errors.append(str(e))

    x = {n: make_logits(8, n, torch.float32, n).to(DEV) for n in (4096, 3100, 4095, 3073)}
    want = {n: ep.ep_route(v, 4) for n, v in x.items()}
    torch.cuda.synchronize()
    threads = [threading.Thread(target=go, args=item) for item in x.items()]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    assert all(torch.equal(results[n].topk_idx, want[n].topk_idx) for n in x)


def test_many_tokens_feed_the_layout():
    """More tokens than one wave of warps, and the outputs in the form the
    layout takes."""
    T, E, K = 70001, 64, 4
    x = make_logits(T, E, torch.float32, 11)
    r = check(x, K)
    lay = ep.ep_get_layout(r.topk_idx, E, 8)
    assert lay.errors() == 0
    assert int(lay.num_tokens_per_expert.sum()) == T * K


# ------------------------------------------------------------------ gradient

def weights64(l, idx, score, renorm, scale):
    """The weights of a fixed choice as a differentiable 64-bit function."""
    there = idx >= 0
    p = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)
    w = torch.where(there, p.gather(1, idx.clamp_min(0)), 0.0)
    if renorm:
        s = w.sum(1, keepdim=True)
        w = w / torch.where(s > 0, s, 1.0)
    return scale * w


def grad_bound(l, idx, g, score, renorm, scale):
    """Sums of the absolute values of a gradient's terms (64-bit)."""
    there = idx >= 0
    d = torch.where(there, g.abs() * scale, 0.0)
    p = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)
    w = torch.where(there, p.gather(1, idx.clamp_min(0)), 0.0)
    if renorm:
        s = w.sum(1, keepdim=True)
        s = torch.where(s > 0, s, 1.0)
        d = (d + (d * w / s).sum(1, keepdim=True)) / s
    dense = torch.zeros_like(l).scatter_add(1, idx.clamp_min(0), torch.where(there, d, 0.0))
    if score == "sigmoid":
        return dense * p
    return p * (dense + (dense * p).sum(1, keepdim=True))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (5, 7, 3), (33, 64, 6), (129, 256, 8), (65, 257, 1), (7, 520, 32),
                                   (3, 4096, 8), (700, 40, 10)])
def test_gradient(T, E, K, renorm, score, dtype):
    logits = make_logits(T, E, dtype, T + K)
    g = torch.Generator().manual_seed(T)
    idx = torch.rand((T, E), generator=g).argsort(1)[:, :K].contiguous()
    idx[torch.rand((T, K), generator=g) < 0.2] = -1
    if T > 2:
        idx[1] = -1
    grad = torch.randn((T, K), generator=g)
    got = ep.ep_route_backward(grad.to(DEV), logits.to(DEV), idx.to(DEV), score=score, renormalize=renorm,
                               weight_scale=1.5)
    assert got.dtype == dtype
    x = logits.double().requires_grad_(True)
    (weights64(x, idx, score, renorm, 1.5) * grad.double()).sum().backward()
    want = x.grad
    l = logits.float().numpy()
    tol = 2 * weight_tolerance(l) * grad_bound(logits.double(), idx, grad.double(), score, renorm, 1.5)
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
    err = (got.cpu().double() - want).abs()
    assert bool((err <= tol + 1e-37).all()), float((err - tol).max())
    if K == 1 and renorm:
        assert bool((got == 0).all())  # a single weight is constant


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    """Central differences of the 64-bit weights along random directions:
    their error is O(h^2) = 1e-8 of the third derivative, below fp32's."""
    T, E, K, h = 40, 32, 5, 1e-4
    logits = make_logits(T, E, torch.float32, 21)
    r = ep.ep_route(logits.to(DEV), K, score=score, renormalize=renorm)
    idx = r.topk_idx.cpu()
    g = torch.Generator().manual_seed(3)
    grad = torch.randn((T, K), generator=g)
    got = ep.ep_route_backward(grad.to(DEV), logits.to(DEV), r.topk_idx, score=score, renormalize=renorm).cpu().double()
    for _ in range(4):
        v = torch.randn((T, E), generator=g).double()
        f = [(weights64(logits.double() + s * h * v, idx, score, renorm, 1.0) * grad.double()).sum(1) for s in (1, -1)]
        want = (f[0] - f[1]) / (2 * h)
        np.testing.assert_allclose((got * v).sum(1).numpy(), want.numpy(), rtol=1e-4, atol=2e-5)


def test_gradient_of_masked_and_bad_choices():
    """Slots of -1, outside [0, E) or naming a masked expert contribute
    nothing; an expert named twice receives both; a row without choices is 0."""
    E = 16
    logits = make_logits(4, E, torch.float32, 2)
    logits[2, 3] = -math.inf
    logits[3] = -math.inf
    idx = torch.tensor([[1, 1, 2], [-1, 99, -7], [3, 4, -1], [0, 1, 2]])
    grad = torch.tensor([[1.0, 2.0, 0.5]] * 4)
    for score in ("softmax", "sigmoid"):
        got = ep.ep_route_backward(grad.to(DEV), logits.to(DEV), idx.to(DEV), score=score, renormalize=False).cpu()
        assert torch.isfinite(got).all()
        assert (got[1] == 0).all() and (got[3] == 0).all()
        x = logits[:1].double().requires_grad_(True)
        (weights64(x, idx[:1], score, False, 1.0) * grad[:1].double()).sum().backward()
        np.testing.assert_allclose(got[:1].numpy(), x.grad.numpy(), rtol=2e-5, atol=1e-6)
        assert got[2, 3] == 0 and got[2, 4] != 0


# ---------------------------------------- enough tokens for a lane a token

MANY = 2051


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K", [(1, 1), (8, 8), (7, 3), (64, 6), (33, 16), (256, 8), (257, 5), (384, 10), (1000, 12),
                                 (1024, 1), (100, 17)])
def test_many_sizes_and_types(E, K, score, dtype):
    b = torch.randn(E, generator=torch.Generator().manual_seed(5)) * 0.1
    x = make_logits(MANY, E, dtype, E)
    x[5] = -math.inf
    x[6, E // 2:] = -math.inf
    for renorm, bias in ((True, None), (False, None), (True, b), (False, b)):
        check(x, K, score, bias, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,Gk,K", [(64, 8, 4, 6), (256, 8, 3, 8), (256, 64, 2, 8), (96, 3, 2, 16), (40, 40, 5, 4),
                                      (1024, 16, 16, 8), (72, 2, 1, 16), (72, 6, 3, 7)])
@pytest.mark.parametrize("top", [1, 2])
def test_many_groups(E, G, Gk, K, top, score):
    bias = torch.randn(E, generator=torch.Generator().manual_seed(7)) * 0.1
    for b in (None, bias):
        x = make_logits(MANY, E, torch.float32, E + G)
        x[3] = -math.inf
        x[4, E // 4:] = -math.inf
        check(x, K, score, b, G, Gk, top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,Gk,top", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
def test_many_ties_and_extremes(G, Gk, top, score):
    """Ties; logits that differ by less than a key's upper bits; masks, the
    type's lowest value, infinities and NaN."""
    E, K = 64, 8
    x = make_logits(MANY, E, torch.float32, 1, lattice=True)
    x[100:200] = 0.0
    x[200:] = torch.where(torch.rand((MANY - 200, 1), generator=torch.Generator().manual_seed(1)) < 0.5, x[200:],
                          1.0 + torch.randint(0, 40, (MANY - 200, E), generator=torch.Generator().manual_seed(2)) * 2.0 ** -22)
    low = torch.finfo(torch.float32).min
    x[0], x[1], x[2, :60], x[3, ::2], x[4] = -math.inf, low, -math.inf, math.nan, math.nan
    x[5, 7] = x[6, 7] = x[6, 9] = math.inf
    x[7] = 1e30 * torch.sign(x[7])
    x[8, 5:] = low
    x[9] = -200.0
    if G == 1 or top == 1:
        check(x, K, score, None, G, Gk, top)  # compared as logits: exact
    check(x[:200].repeat(11, 1), K, score, None, G, Gk, top)
    check(x[:200].repeat(11, 1), K, score, torch.zeros(E), G, Gk, top)


def test_the_two_forms_agree():
    """The same rows by a warp a token and by a lane a token: bit for bit the
    choice, where keys are logits, and the weights within their bound."""
    x = make_logits(MANY, 128, torch.float32, 13).to(DEV)
    many = ep.ep_route(x, 7)
    few = [ep.ep_route(x[i:i + 500], 7) for i in range(0, MANY, 500)]
    assert torch.equal(many.topk_idx, torch.cat([r.topk_idx for r in few]))
    torch.testing.assert_close(many.topk_weights, torch.cat([r.topk_weights for r in few]), rtol=4e-6, atol=0)
    part = make_logits(MANY, 160, torch.bfloat16, 14).to(DEV)[:, 5:133]  # rows that start at odd places
    a, b = ep.ep_route(part, 7), ep.ep_route(part.contiguous(), 7)
    assert torch.equal(a.topk_idx, b.topk_idx) and torch.equal(a.topk_weights, b.topk_weights)


@pytest.mark.parametrize("T,E,apart,K", [(70000, 64, 32768, 6), (540000, 4000, 4000, 3)])
@pytest.mark.parametrize("renorm", [True, False])
def test_offsets_past_32_bits(T, E, apart, K, renorm):
    """Logits of more than 2^31 elements: the last rows are copies of the
    first and give the same."""
    wide = torch.zeros((T, apart), dtype=torch.float32, device=DEV)
    assert wide.numel() > 2 ** 31
    n = 5000
    some = make_logits(n, E, torch.float32, 3).to(DEV)
    wide[:n, :E] = some
    wide[-n:, :E] = some
    r = ep.ep_route(wide[:, :E], K, renormalize=renorm)
    few = ep.ep_route(some, K, renormalize=renorm)
    for rows in (slice(0, n), slice(T - n, T)):
        assert torch.equal(r.topk_idx[rows], few.topk_idx) and torch.equal(r.topk_weights[rows], few.topk_weights)
    d = torch.randn((n, K), generator=torch.Generator(device=DEV).manual_seed(4), device=DEV)
    all_d = torch.zeros((T, K), device=DEV)
    all_d[:n] = d
    all_d[-n:] = d
    want = ep.ep_route_backward(d, some, few.topk_idx, renormalize=renorm)
    got = ep.ep_route_backward(all_d, wide[:, :E], r.topk_idx, renormalize=renorm)
    assert torch.equal(got[:n], want) and torch.equal(got[-n:], want)
    del wide, got, r
    torch.cuda.empty_cache()
