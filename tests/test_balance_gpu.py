"""The router's balance and z loss, their counts and gradients, against plain
64-bit implementations.

Tolerances, fixed before any run.  A score p is a quotient of positive fp32
sums: its exponential costs 4 ulp and the rounding of its argument (up to
4 |l - m| ulp), the sum of E terms over at least 8 lanes E/8 + 8 roundings:
r = 2^-24 (40 + E/8 + 4 max|l - m|), relative.  A mean over n tokens adds n
roundings at most.  That a token is missing would hide in that, so one-hot
rows, whose scores are 0 and 1 and whose sums are exact, are compared for
equality.  A gradient adds products of such terms: the same bound on the sum
of the terms' absolute values, and its type's rounding.
"""
import math

import numpy as np
import pytest
import torch

import combine_ep_get_layout_gb300 as ep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def scores64(l, score):
    """(p, softmax, log-sum-exp, sigmoid) of logits [T, E] in 64 bits; what is masked is 0."""
    l = l.double()
    l = torch.where(torch.isnan(l), -math.inf, l.clamp(max=torch.finfo(torch.float32).max))
    dead = torch.isneginf(l).all(1, keepdim=True)
    safe = torch.where(dead, 0.0, l)
    soft = torch.where(dead, 0.0, torch.softmax(safe, 1))
    lse = torch.where(dead[:, 0], 0.0, torch.logsumexp(safe, 1))
    sig = torch.where(torch.isneginf(l), 0.0, torch.sigmoid(l))
    if score == "softmax":
        return soft, soft, lse, sig
    # in logarithms, so that tiny scores do not vanish together
    p = torch.where(dead, 0.0, torch.softmax(torch.where(dead, 0.0, torch.nn.functional.logsigmoid(l)), 1))
    return p, soft, lse, sig


def spans(offsets, T):
    o = [0, T] if offsets is None else offsets.tolist()
    return list(zip(o, o[1:]))


def balance64(l, idx, score, offsets):
    T, E = l.shape
    p, soft, lse, sig = scores64(l, score)
    parts = spans(offsets, T)
    full = sum(b > a for a, b in parts)
    tokens = sum(b - a for a, b in parts)
    counts = torch.zeros((len(parts), E), dtype=torch.int64, device=l.device)
    probs = torch.zeros((len(parts), E), dtype=torch.float64, device=l.device)
    slopes = torch.zeros_like(probs)
    z = 0.0
    for s, (a, b) in enumerate(parts):
        if b == a:
            continue
        c = idx[a:b].reshape(-1)
        c = c[(c >= 0) & (c < E)]
        counts[s] = torch.bincount(c, minlength=E)
        probs[s] = p[a:b].mean(0)
        if c.numel():
            slopes[s] = E * counts[s].double() / c.numel() / full / (b - a)
        z += float((lse[a:b] ** 2).sum())
    n = torch.tensor([b - a for a, b in parts], device=l.device, dtype=torch.float64)
    losses = torch.tensor([float((slopes * probs * n[:, None]).sum()), z / max(1, tokens)], dtype=torch.float64, device=l.device)
    return losses, counts, probs, slopes


def gradient64(l, slopes, g, score, offsets, add):
    """(the gradient, the sum of its terms' absolute values)."""
    T, E = l.shape
    p, soft, lse, sig = scores64(l, score)
    d, size = torch.zeros((2, T, E), dtype=torch.float64, device=l.device)
    tokens = sum(b - a for a, b in spans(offsets, T))
    for s, (a, b) in enumerate(spans(offsets, T)):
        if b == a:
            continue
        w = slopes[s].double() * float(g[0])
        dot = (p[a:b] * w).sum(1, keepdim=True)
        side = 1.0 - sig[a:b] if score == "sigmoid" else torch.ones_like(p[a:b])
        zpart = float(g[1]) * 2.0 / tokens * lse[a:b, None] * soft[a:b]
        d[a:b] = p[a:b] * (w - dot) * side + zpart
        size[a:b] = p[a:b] * (w.abs() + (p[a:b] * w.abs()).sum(1, keepdim=True)) * side + zpart.abs()
    if add is not None:
        d, size = d + add.double(), size + add.double().abs()
    return d, size


def rough(l):
    """r of the docstring."""
    f = l.float()
    f = f[torch.isfinite(f)]
    wide = float(f.max() - f.min()) if f.numel() else 0.0
    return 2.0 ** -24 * (40 + l.shape[1] / 8 + 4 * (wide + (float(f.abs().max()) if f.numel() else 0.0)))


def make(T, E, K, dtype, seed=0, masked=0.0, spread=1.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    l = (torch.randn((T, E), generator=g, device=DEV) * spread).to(dtype)
    if masked:
        l[torch.rand(l.shape, generator=g, device=DEV) < masked] = -math.inf
    idx = torch.argsort(l.float(), dim=1, descending=True)[:, :K].contiguous()
    idx[torch.rand(idx.shape, generator=g, device=DEV) < masked] = -1
    return l, idx


def check(l, idx, score, offsets=None, add=None, grad=(0.7, -0.2), **kw):
    b = ep.ep_balance_loss(l, idx, score=score, seq_offsets=offsets, **kw)
    losses, counts, probs, slopes = balance64(l, idx, score, offsets)
    assert torch.equal(b.counts.long(), counts)
    T, r = l.shape[0], rough(l)
    lengths = torch.tensor([x - a for a, x in spans(offsets, T)], device=DEV, dtype=torch.float64)[:, None]
    assert ((b.probs - probs).abs() <= (r + (lengths + 2) * 2.0 ** -24) * probs + 1e-38).all()
    assert ((b.slopes - slopes).abs() <= 2.0 ** -21 * slopes).all()
    lse = scores64(l, score)[2]
    # a log-sum-exp is off by ulps of its two terms
    top = float(lse.abs().max()) if T else 0.0
    assert abs(float(b.losses[0] - losses[0])) <= (r + (T + 70 + l.shape[1]) * 2.0 ** -24) * float(losses[0])
    assert abs(float(b.losses[1] - losses[1])) <= 2 * top * (r + 2.0 ** -22 * (top + 1)) + (T + 70) * 2.0 ** -24 * float(losses[1])
    g = torch.tensor(grad, device=DEV)
    got = ep.ep_balance_loss_backward(g, l, b, score=score, seq_offsets=offsets, add=add)
    want, size = gradient64(l, slopes, grad, score, offsets, add)
    half = torch.finfo(l.dtype).eps / 2
    err = (got.double() - want).abs()
    assert (err <= half * want.abs() + 4 * (r + 2.0 ** -20) * size + 1e-38).all(), float((err / (size + 1e-300)).max())
    return b, got


SHAPES = [(1, 1, 1), (1, 8, 2), (3, 7, 3), (13, 64, 6), (64, 60, 4), (255, 128, 8), (257, 33, 5), (1000, 256, 8),
          (129, 1000, 10), (70, 1024, 4), (33, 1027, 3), (40, 4096, 32), (5, 2048, 8), (2000, 16, 2), (777, 512, 9)]


@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_one_sequence(T, E, K, dtype, score):
    l, idx = make(T, E, K, dtype, seed=T + E)
    check(l, idx, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,offsets", [
    (100, 64, [0, 40, 40, 97]), (100, 64, [3, 4, 90]), (700, 24, [0, 1, 2, 3, 333, 333, 334, 700]),
    (5, 8, [0, 0, 0, 5]), (50, 128, [50, 50]), (50, 128, [0, 0]), (300, 256, list(range(0, 301, 3))),
    (4096, 32, [0, 1000, 1001, 4000]), (1500, 1300, [7, 700, 1400]), (900, 8, [0, 256, 512, 768]),
    (5000, 100, list(range(0, 5001, 10))), (3000, 40, [0, 2000, 2000, *range(2001, 2900)]),
    (300, 16, [0] * 900 + [7] * 50 + list(range(8, 290)) + [290] * 700), (1281, 64, [0, 640, 1281]), (1280, 64, [1, 640, 1279])])
def test_sequences(T, E, offsets, score):
    l, idx = make(T, E, min(4, E), torch.float32, seed=T, masked=0.1)
    add = torch.randn((T, E), device=DEV) * 1e-3
    b, got = check(l, idx, score, torch.tensor(offsets, dtype=torch.int32, device=DEV), add)
    outside = torch.ones(T, dtype=torch.bool)
    outside[offsets[0]:offsets[-1]] = False
    assert torch.equal(got[outside.to(DEV)], add[outside.to(DEV)])  # rows of no sequence, left as they were


def test_every_token_counts():
    """One-hot rows: scores are 0 and 1, and the sums of them exact."""
    for T, E, offsets in ((1, 3, None), (31, 8, None), (5003, 16, None), (1025, 257, [0, 5, 600, 1020]), (65536, 64, None)):
        hot = torch.randint(0, E, (T,), device=DEV)
        l = torch.full((T, E), -math.inf, device=DEV)
        l[torch.arange(T, device=DEV), hot] = 3.0
        off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)
        for score in ("softmax", "sigmoid"):
            b = ep.ep_balance_loss(l, hot[:, None].contiguous(), score=score, seq_offsets=off)
            n = torch.tensor([x - a for a, x in spans(off, T)], device=DEV, dtype=torch.float32)[:, None]
            counts = balance64(l, hot[:, None], score, off)[1]
            assert torch.equal(b.counts.long(), counts)
            assert torch.equal(b.probs, counts.float() / n)
            assert float(b.losses[1]) == 9.0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_rows(score, dtype):
    """Rows without an expert, rows of NaN, the type's lowest value, large logits of either sign."""
    l, idx = make(90, 40, 4, dtype, seed=3, masked=0.3)
    l[5] = -math.inf
    l[6] = math.nan
    l[7, ::2] = math.nan
    l[8] = torch.finfo(dtype).min
    l[9] = torch.finfo(dtype).min
    l[9, 3] = 2.0
    l[11] = -90.0
    l[12] = 80.0
    idx[5:7] = -1
    b = ep.ep_balance_loss(l, idx, score=score)
    losses, counts, probs, slopes = balance64(l, idx, score, None)
    # the rows of huge logits are off by more than the others' bound
    assert torch.equal(b.counts.long(), counts)
    r = 2.0 ** -24 * (40 + 5 + 4 * 180 + 90)
    assert ((b.probs - probs).abs() <= r * probs + 1e-38).all()
    g = torch.tensor([1.0, 0.0], device=DEV)
    got = ep.ep_balance_loss_backward(g, l, b, score=score)
    assert torch.isfinite(got[[5, 6, 7, 9, 11, 12]].float()).all()
    assert (got[5:7] == 0).all() and (got[7, ::2] == 0).all()
    want, size = gradient64(l, slopes, (1.0, 0.0), score, None, None)
    keep = [i for i in range(90) if i != 8]
    half = torch.finfo(dtype).eps / 2
    assert ((got.double() - want).abs() <= half * want.abs() + 4 * (r + 2.0 ** -20) * size + 1e-38)[keep].all()


def test_an_infinite_logit_counts_as_the_largest():
    l, idx = make(10, 16, 2, torch.float32)
    l[4, 3] = math.inf
    m = l.clone()
    m[4, 3] = torch.finfo(torch.float32).max
    for score in ("softmax", "sigmoid"):
        a, b = (ep.ep_balance_loss(x, idx, score=score) for x in (l, m))
        assert torch.equal(a.probs, b.probs) and torch.isfinite(a.probs).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("base", [1e5, 1e7, 1.7e7, 1e9, 1e12, 1e20, 0.9e30])
def test_large_logits(base, dtype, score):
    """Ties at the largest of huge logits (the rest far below it): scores are
    quotients of few equal numbers, 64 roundings of 2^-24 and those of the
    exponentials' 2 ulp."""
    T, E = 40, 96
    l = torch.full((T, E), base, device=DEV)
    l[1::2, 5:] = base * 0.75
    l[2::4] *= -1
    l[3::4] *= -1
    l = l.to(dtype)
    idx = torch.zeros((T, 1), dtype=torch.int64, device=DEV)
    b = ep.ep_balance_loss(l, idx, score=score)
    losses, counts, probs, slopes = balance64(l, idx, score, None)
    near = 2.0 ** -18
    assert torch.equal(b.counts.long(), counts)
    assert ((b.probs - probs).abs() <= near * probs).all()
    for i in range(2):
        assert abs(float(b.losses[i]) - min(float(losses[i]), math.inf)) <= near * float(losses[i]) or float(losses[i]) > 3e38
    grad = (0.7, 1e-3)
    got = ep.ep_balance_loss_backward(torch.tensor(grad, device=DEV), l, b, score=score)
    want, size = gradient64(l, slopes, grad, score, None, None)
    assert ((got.double() - want).abs() <= torch.finfo(dtype).eps / 2 * want.abs() + near * size + 1e-38).all()


def test_choices_outside_and_named_twice():
    l, idx = make(40, 12, 3, torch.float32)
    idx[0] = torch.tensor([5, 5, 5], device=DEV)
    idx[1] = torch.tensor([12, -7, 2 ** 40], device=DEV)
    idx[2] = -1
    check(l, idx, "softmax")
    idx[:] = -1
    b, _ = check(l, idx, "softmax")
    assert float(b.losses[0]) == 0.0 and (b.slopes == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_wider_ones(dtype):
    for E, wide, first in ((64, 96, 8), (64, 67, 1), (63, 80, 0)):
        big = torch.randn((50, wide), device=DEV).to(dtype)
        l = big[:, first:first + E]
        idx = torch.argsort(l.float(), dim=1, descending=True)[:, :4].contiguous()
        b, g = check(l, idx, "softmax")
        b2, g2 = check(l.contiguous(), idx, "softmax")
        assert ((b.probs - b2.probs).abs() <= 2 * rough(l) * b2.probs).all()


def test_no_tokens():
    l = torch.empty((0, 8), device=DEV)
    idx = torch.empty((0, 2), dtype=torch.int64, device=DEV)
    for off in (None, torch.zeros(4, dtype=torch.int32, device=DEV)):
        b = ep.ep_balance_loss(l, idx, seq_offsets=off)
        assert (b.losses == 0).all() and (b.counts == 0).all() and (b.probs == 0).all() and (b.slopes == 0).all()
        assert ep.ep_balance_loss_backward(torch.ones(2, device=DEV), l, b, seq_offsets=off).shape == (0, 8)


@pytest.mark.parametrize("offsets", [[0, 30, 20, 50], [-5, 10, 50], [0, 20, 60], [2 ** 31 - 1, -2 ** 31, 7]])
def test_offsets_out_of_order_are_loud(offsets):
    """Nothing is read or written out of range for them (every access is cut to the tensors)."""
    l, idx = make(50, 16, 2, torch.float32)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    b = ep.ep_balance_loss(l, idx, seq_offsets=off)
    assert torch.isnan(b.losses).all()
    ep.ep_balance_loss_backward(torch.ones(2, device=DEV), l, b, seq_offsets=off)
    torch.cuda.synchronize()


@pytest.mark.parametrize("E", [16, 300, 2048])
def test_offsets_out_of_order_in_a_large_batch(E):
    l, idx = make(4000, E, 2, torch.float32)
    for offsets in ([0, 3000, 10, 4000], [5, 2 ** 31 - 1, -3, 4000], [4000, 0], [3999, 4001], [0, 1, 0, 1, 0, 1, 4000]):
        off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        b = ep.ep_balance_loss(l, idx, seq_offsets=off)
        assert torch.isnan(b.losses).all()
        ep.ep_balance_loss_backward(torch.ones(2, device=DEV), l, b, seq_offsets=off)
    torch.cuda.synchronize()


def test_given_tensors_are_used_again():
    for T, E in ((900, 64), (5000, 256), (300, 1500)):
        shared = torch.empty(ep.ep_balance_workspace_bytes(T, E, 3), dtype=torch.uint8, device=DEV).fill_(255)
        off = torch.tensor([0, T // 3, T // 3, T], dtype=torch.int32, device=DEV)
        out = None
        for seed in range(3):
            l, idx = make(T, E, 3, torch.float32, seed=seed)
            want = ep.ep_balance_loss(l, idx, seq_offsets=off)
            got = ep.ep_balance_loss(l, idx, seq_offsets=off, out=out, workspace=shared)
            assert out is None or got is out
            out = got
            for name in ("losses", "counts", "probs", "slopes"):
                assert torch.equal(getattr(got, name), getattr(want, name))
            g = torch.tensor([1.0, 0.1], device=DEV)
            d = ep.ep_balance_loss_backward(g, l, got, seq_offsets=off)
            mine = l.clone()  # the gradient over the logits themselves
            assert torch.equal(ep.ep_balance_loss_backward(g, mine, got, seq_offsets=off, out=mine), d)


def test_gradient_by_differences():
    """(f(x + h e) - f(x - h e)) / 2h of the 64-bit losses themselves: h = 1e-4 leaves h^2 f'''/6, below 1e-8 of
    the losses' scale, and 1e-16 / h of cancellation."""
    l, idx = make(7, 10, 3, torch.float32, seed=8, masked=0.1)
    off = torch.tensor([0, 4, 7], dtype=torch.int32, device=DEV)
    for score in ("softmax", "sigmoid"):
        b = ep.ep_balance_loss(l, idx, score=score, seq_offsets=off)
        got = ep.ep_balance_loss_backward(torch.tensor([1.0, 0.5], device=DEV), l, b, score=score, seq_offsets=off)
        for t, e in ((0, 1), (3, 9), (4, 0), (6, 5)):
            if torch.isneginf(l[t, e]):
                assert float(got[t, e]) == 0.0
                continue
            f = []
            for h in (1e-4, -1e-4):
                m = l.double()
                m[t, e] += h
                x = balance64(m, idx, score, off)[0]
                f.append(float(x[0] + 0.5 * x[1]))
            assert abs((f[0] - f[1]) / 2e-4 - float(got[t, e])) < 1e-6


def test_add_in_place_and_the_same_bits():
    l, idx = make(3000, 256, 8, torch.bfloat16)
    first = ep.ep_balance_loss(l, idx, score="sigmoid")
    g = torch.tensor([0.01, 0.001], device=DEV)
    add = (torch.randn(l.shape, device=DEV) * 1e-4).to(l.dtype)
    want = ep.ep_balance_loss_backward(g, l, first, score="sigmoid", add=add)
    for _ in range(3):
        b = ep.ep_balance_loss(l, idx, score="sigmoid")
        for name in ("losses", "counts", "probs", "slopes"):
            assert torch.equal(getattr(b, name), getattr(first, name))
        out = add.clone()
        assert ep.ep_balance_loss_backward(g, l, b, score="sigmoid", add=out, out=out) is out
        assert torch.equal(out, want)


def test_more_than_two_gigabytes_apart():
    """Rows whose offsets pass 2^31 elements."""
    try:
        big = torch.zeros((3, 2 ** 30 + 64), dtype=torch.bfloat16, device=DEV)
    except torch.OutOfMemoryError:
        pytest.skip("no room")
    l = big[:, :64]
    l.copy_(torch.randn((3, 64), device=DEV))
    idx = torch.argsort(l.float(), dim=1, descending=True)[:, :4].contiguous()
    check(l, idx, "softmax")


def test_captured_and_on_another_stream():
    l, idx = make(500, 64, 4, torch.float32)
    off = torch.tensor([0, 100, 480], dtype=torch.int32, device=DEV)
    g = torch.ones(2, device=DEV)

    def step():
        b = ep.ep_balance_loss(l, idx, seq_offsets=off)
        return b.losses, b.counts, b.probs, b.slopes, ep.ep_balance_loss_backward(g, l, b, seq_offsets=off)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = ep.ep_balance_loss(l, idx, seq_offsets=off, stream=side)
    d = ep.ep_balance_loss_backward(g, l, b, seq_offsets=off, stream=side)
    side.synchronize()
    assert torch.equal(b.losses, want[0]) and torch.equal(d, want[4])
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    l.normal_()
    idx.random_(-1, 64)
    off[1] = 333
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, step()):
        assert torch.equal(a, b)


def test_refusals():
    l, idx = make(10, 8, 2, torch.float32)
    b = ep.ep_balance_loss(l, idx)
    g = torch.ones(2, device=DEV)
    for error, call in [
            (TypeError, lambda: ep.ep_balance_loss(l.half(), idx)), (TypeError, lambda: ep.ep_balance_loss(l, idx.int())),
            (ValueError, lambda: ep.ep_balance_loss(l, idx[:5])), (ValueError, lambda: ep.ep_balance_loss(l.T, idx)),
            (KeyError, lambda: ep.ep_balance_loss(l, idx, score="relu")),
            (TypeError, lambda: ep.ep_balance_loss(l, idx, seq_offsets=torch.tensor([0, 10], device=DEV))),
            (ValueError, lambda: ep.ep_balance_loss(l, idx, seq_offsets=torch.zeros(1, dtype=torch.int32, device=DEV))),
            (ValueError, lambda: ep.ep_balance_loss(l, idx, seq_offsets=torch.zeros(2, dtype=torch.int32))),
            (ep.EPError, lambda: ep.ep_balance_loss(l, idx, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))),
            (ValueError, lambda: ep.ep_balance_loss(l, idx, seq_offsets=torch.zeros(4, dtype=torch.int32, device=DEV), out=b)),
            (TypeError, lambda: ep.ep_balance_loss_backward(g.double(), l, b)),
            (ValueError, lambda: ep.ep_balance_loss_backward(g, l[:, :4], b)),
            (TypeError, lambda: ep.ep_balance_loss_backward(g, l, b, add=l.bfloat16())),
            (ValueError, lambda: ep.ep_balance_loss_backward(g, l, b, out=torch.empty((10, 9), device=DEV)))]:
        with pytest.raises(error):
            call()
