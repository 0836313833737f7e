"""A shared projection with low-rank adapters against 64 bits.

Tolerances, fixed before any run: fp32 sums of n products err by at most
n * 2^-23 of the sum of absolute values (as in test_product_gpu.py); the low
row (x A^T, times the scale) may be rounded to bf16 before it meets B, at most
half a unit in the last of 8 binary places, 2^-8 of each of its terms; the
result is rounded once (between the roundings of the value less and plus the
bound, as rounding is monotone).
"""
import math

import pytest
import torch

import combine_ep_get_layout_gb300 as ep

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(T, H, N, A, r, seed, spread):
    g = torch.Generator(device=DEV).manual_seed(seed)
    bf = torch.bfloat16
    x = torch.randn((T, H), generator=g, device=DEV).to(bf)
    w = (torch.randn((N, H), generator=g, device=DEV) / math.sqrt(H)).to(bf)
    a = (torch.randn((A, r, H), generator=g, device=DEV) / math.sqrt(H)).to(bf)
    b = (torch.randn((A, N, r), generator=g, device=DEV) / math.sqrt(r)).to(bf)
    s = torch.rand(A, generator=g, device=DEV) + 0.5
    if spread == "none":
        idx = torch.full((T,), -1, device=DEV)
    elif spread == "one":
        idx = torch.full((T,), A - 1, device=DEV)
    elif spread == "runs":
        idx = (torch.arange(T, device=DEV) * A // max(T, 1)) - int(A > 1)
    else:
        idx = torch.randint(-1, A, (T,), generator=g, device=DEV)
    return x, w, a, b, idx, s


def check(x, w, a, b, idx, s, out):
    H, r = x.shape[1], a.shape[1]
    xd, wd = x.double(), w.double()
    want = xd @ wd.T
    tol = H * 2.0 ** -23 * (xd.abs() @ wd.abs().T)
    for k in idx.unique().tolist():
        if not 0 <= k < a.shape[0]:
            continue
        at = (idx == k).nonzero()[:, 0]
        f = 1.0 if s is None else float(s[k])
        low = f * (xd[at] @ a[k].double().T)
        low_tol = f * H * 2.0 ** -23 * (xd[at].abs() @ a[k].double().abs().T) + 2.0 ** -8 * low.abs()
        want[at] += low @ b[k].double().T
        tol[at] += (low_tol + (r + H) * 2.0 ** -23 * low.abs()) @ b[k].double().abs().T
    low, high = ((want + s * tol).to(torch.bfloat16) for s in (-1, 1))
    assert bool(((low <= out) & (out <= high)).all()), float(((out.double() - want).abs() / (tol + 2.0 ** -8 * want.abs())).max())


@pytest.mark.parametrize("T,H,N,A,r", [(1, 8, 8, 1, 8), (1, 4096, 512, 3, 16), (7, 200, 136, 4, 16), (32, 512, 1000, 24, 16),
                                       (64, 256, 72, 64, 8), (130, 136, 264, 5, 24), (300, 512, 512, 9, 32),
                                       (513, 72, 640, 2, 64), (257, 328, 128, 40, 128), (1021, 256, 1000, 40, 40),
                                       (90, 2048, 2056, 10, 16)])
@pytest.mark.parametrize("spread", ["rows", "runs", "one", "none"])
def test_adapters(T, H, N, A, r, spread):
    x, w, a, b, idx, s = make(T, H, N, A, r, T + A, spread)
    out = ep.ep_adapter_product(x, w, a, b, idx, s)
    check(x, w, a, b, idx, s, out)
    again = ep.ep_adapter_product(x, w, a, b, idx, s)
    assert torch.equal(out, again)
    check(x, w, a, b, idx, None, ep.ep_adapter_product(x, w, a, b, idx))


@pytest.mark.parametrize("T,H,N,A,r", [(1100, 4096, 128, 5, 32), (2100, 1024, 72, 40, 64), (1500, 2048, 2048, 300, 48),
                                       (4200, 4096, 1032, 3, 8), (2600, 4096, 264, 20, 16)])
@pytest.mark.parametrize("spread", ["rows", "runs", "one"])
def test_many_rows(T, H, N, A, r, spread):
    """Sizes at which the low rows come from stacked adapters."""
    x, w, a, b, idx, s = make(T, H, N, A, r, T + A, spread)
    idx[7], idx[T - 1] = -1, A
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = ep.ep_adapter_product(x, w, a, b, idx, s, error_word=word)
    assert int(word) == ep.EP_ERRBIT_BAD_INDEX
    check(x, w, a, b, idx, s, out)
    assert torch.equal(out, ep.ep_adapter_product(x, w, a, b, idx, s))


def test_bad_indices_count_as_none_and_are_flagged():
    x, w, a, b, idx, s = make(40, 128, 64, 4, 16, 3, "rows")
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = ep.ep_adapter_product(x, w, a, b, idx, s, error_word=word)
    assert int(word) == 0
    bad = idx.clone()
    bad[5], bad[17], bad[18] = 4, -2, 1 << 40
    got = ep.ep_adapter_product(x, w, a, b, bad, s, error_word=word)
    assert int(word) == ep.EP_ERRBIT_BAD_INDEX
    rest = [i for i in range(40) if i not in (5, 17, 18)]
    assert torch.equal(got[rest], want[rest])
    check(x, w, a, b, bad, s, got)


def test_unused_adapters_and_other_rows_do_not_leak():
    """NaN in adapters that no row names, or in another row, reaches no row."""
    x, w, a, b, idx, s = make(70, 128, 136, 6, 16, 4, "rows")
    idx = torch.where(idx == 2, -1, idx)
    want = ep.ep_adapter_product(x, w, a, b, idx, s)
    a[2], b[2], s[2] = math.nan, math.inf, math.nan
    got = ep.ep_adapter_product(x, w, a, b, idx, s)
    assert torch.equal(got, want)
    x[11] = math.nan
    got = ep.ep_adapter_product(x, w, a, b, idx, s)
    rest = [i for i in range(70) if i != 11]
    assert torch.equal(got[rest], want[rest]) and torch.isnan(got[11]).all()


@pytest.mark.parametrize("T,H,N,A,r", [(3, 512, 136, 3, 8), (32, 4096, 520, 24, 16), (70, 128, 264, 6, 128),
                                       (300, 256, 512, 40, 24), (1100, 4096, 128, 5, 32)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_an_up_projection_that_is_not_finite_stays_with_its_rows(T, H, N, A, r, value):
    """Rows of other adapters, and outputs that it does not reach, keep their
    bits; its own get what the formula gives (the sign too, where the low
    value's sign is certain)."""
    x, w, a, b, idx, s = make(T, H, N, A, r, T, "rows")
    idx[0], idx[1], idx[2] = 1, 0, 1
    clean = ep.ep_adapter_product(x, w, a, b, idx, s)
    b[1, 5, r - 1], b[1, N - 1, 0], b[A - 1, N // 2] = value, value, -value
    got = ep.ep_adapter_product(x, w, a, b, idx, s)
    reached = torch.zeros((T, N), dtype=torch.bool, device=DEV)
    for k, n in ((1, 5), (1, N - 1), (A - 1, N // 2)):
        reached[(idx == k).nonzero()[:, 0], n] = True
    assert torch.equal(got[~reached], clean[~reached])
    assert reached.any() and not torch.isfinite(got[reached]).any()
    if math.isinf(value):
        for n, i in ((5, r - 1), (N - 1, 0)):
            at = (idx == 1).nonzero()[:, 0]
            low = x[at].double() @ a[1, i].double()
            sure = low.abs() > H * 2.0 ** -23 * (x[at].double().abs() @ a[1, i].double().abs())
            assert torch.equal(got[at[sure], n].double(), low[sure].sign() * value)
    assert torch.equal(got.nan_to_num(nan=7.0), ep.ep_adapter_product(x, w, a, b, idx, s).nan_to_num(nan=7.0))


@pytest.mark.parametrize("T,H,N,A,r", [(3, 512, 136, 3, 8), (32, 4096, 520, 24, 16), (300, 256, 512, 40, 24),
                                       (1100, 4096, 128, 5, 32)])
def test_infinite_low_values_meet_infinite_up_projections(T, H, N, A, r):
    """Infinity times infinity is infinity, of the product's sign: a low value
    that overflows meets an infinite up-projection, and finite ones."""
    x, w, a, b, idx, s = make(T, H, N, A, r, T + 1, "rows")
    idx[0], idx[1], idx[2] = 1, 1, 0
    i = r - 2
    a[1, i] = 0.0
    a[1, i, 0] = 3e38
    x[:, 0] = 0.25
    x[0, 0], x[1, 0] = 16.0, -16.0  # times 3e38 and a scale of 0.5 or more: infinite
    clean = ep.ep_adapter_product(x, w, a, b, idx, s)
    finite = b[1, :, i].clone()
    assert bool((finite != 0).all())
    b[1, 5, i], b[1, 70, i], b[1, N - 1, i] = math.inf, -math.inf, math.inf
    got = ep.ep_adapter_product(x, w, a, b, idx, s)
    sign = b[1, :, i].double().sign() * math.inf
    assert torch.equal(got[0].double(), sign) and torch.equal(got[1].double(), -sign)
    own = (idx == 1).nonzero()[:, 0]
    own = own[own > 1]  # their low value is finite and positive
    for n in (5, 70, N - 1):
        assert bool((got[own, n].double() == sign[n]).all())
    rest = (idx != 1).nonzero()[:, 0]
    assert len(rest) and torch.isfinite(clean[rest]).all() and torch.equal(got[rest], clean[rest])


def test_no_rows_and_another_stream():
    x, w, a, b, idx, s = make(0, 64, 32, 2, 8, 5, "rows")
    assert ep.ep_adapter_product(x, w, a, b, idx, s).shape == (0, 32)
    x, w, a, b, idx, s = make(200, 512, 512, 8, 16, 6, "rows")
    want = ep.ep_adapter_product(x, w, a, b, idx, s)
    out = torch.zeros_like(want)
    ws = torch.empty(ep.ep_adapter_workspace_bytes(200, 512, 16), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        y = x * 1.0
        ep.ep_adapter_product(y, w, a, b, idx, s, out=out, workspace=ws)
    st.synchronize()
    assert torch.equal(out, want)


def test_what_a_call_allocates_belongs_to_its_stream():
    """The workspace that a call takes for itself is not handed to the current
    stream while the call's own stream still uses it."""
    x, w, a, b, idx, s = make(300, 512, 512, 8, 16, 6, "rows")
    want = ep.ep_adapter_product(x, w, a, b, idx, s)
    out = torch.zeros_like(want)
    nbytes = ep.ep_adapter_workspace_bytes(300, 512, 16)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        m = torch.ones((4096, 4096), device=DEV)
        for _ in range(8):
            m = m @ m * 1e-4
    ep.ep_adapter_product(x, w, a, b, idx, s, out=out, stream=st)
    held = [torch.zeros(nbytes, dtype=torch.uint8, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and not any(t.any() for t in held)


def test_offsets_past_32_bits():
    """Rows and results of more than 2^31 elements, then adapters of as many."""
    T, H, r = 132000, 16384, 16
    g = torch.Generator(device=DEV).manual_seed(1)
    bf = torch.bfloat16
    x = torch.randn((T, H), generator=g, device=DEV, dtype=bf)
    w = torch.randn((H, H), generator=g, device=DEV, dtype=bf) / 128
    a = torch.randn((5, r, H), generator=g, device=DEV, dtype=bf) / 128
    b = torch.randn((5, H, r), generator=g, device=DEV, dtype=bf) / 4
    idx = torch.randint(-1, 5, (T,), generator=g, device=DEV)
    out = ep.ep_adapter_product(x, w, a, b, idx)
    assert x.numel() > 2 ** 31
    last = slice(T - 24, T)
    check(x[last], w, a, b, idx[last], None, out[last])
    del a, b, out
    # 4096 adapters of rank 128: only those that are named are filled
    x, A, r = x[last].clone(), 4096, 128
    a = torch.empty((A, r, H), dtype=bf, device=DEV)
    b = torch.empty((A, H, r), dtype=bf, device=DEV)
    assert a.numel() > 2 ** 32
    idx = torch.tensor([-1, 0, 1023, 1024, 2047, 4094, 4095, 4095], device=DEV).repeat(3)
    for k in idx.unique().tolist():
        if k >= 0:
            a[k] = torch.randn((r, H), generator=g, device=DEV, dtype=bf) / 128
            b[k] = torch.randn((H, r), generator=g, device=DEV, dtype=bf) / 8
    check(x, w, a, b, idx, None, ep.ep_adapter_product(x, w, a, b, idx))
    del x, w, a, b
    torch.cuda.empty_cache()
