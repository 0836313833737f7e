"""Edges of the block's operators: more choices than 32 bits count, gradients over
logits that are not of whole 16 bytes, rows beside masked ones.
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
