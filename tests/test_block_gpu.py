"""The norm, the gate, the router with its losses, the experts' products, the
combine and the shared product run together as a training block, and their
gradients agree with differentiation in 64 bits; two streams, capture, and
all of it in one graph."""
import os
import sys

import pytest
import torch

import combine_ep_get_layout_gb300 as ep

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
BF16 = torch.bfloat16


def block64(block, x, idx, offsets):
    """(out, losses, logits, the leaves) in 64 bits at a fixed choice."""
    F = torch.nn.functional
    names = ("norm_weight", "norm_bias", "gate", "w1", "w2", "s1", "s1_bias", "s2", "s2_bias")
    leaf = {n: getattr(block, n).double().requires_grad_(True) for n in names}
    leaf["x"] = x.double().requires_grad_(True)
    n = F.layer_norm(leaf["x"], (x.shape[1],), leaf["norm_weight"], leaf["norm_bias"], 1e-5)
    logits = n @ leaf["gate"].T
    sig = torch.sigmoid(logits)
    p = sig.gather(1, idx)
    p = p / p.sum(1, keepdim=True)
    out = leaf["x"]
    for k in range(idx.shape[1]):
        gate, up = torch.einsum("th,tnh->tn", n, leaf["w1"][idx[:, k]]).chunk(2, dim=1)
        out = out + p[:, k:k + 1] * torch.einsum("tf,thf->th", F.silu(gate) * up, leaf["w2"][idx[:, k]])
    gate, up = (n @ leaf["s1"].T + leaf["s1_bias"]).chunk(2, dim=1)
    out = out + (F.silu(gate) * up) @ leaf["s2"].T + leaf["s2_bias"]
    E, o = logits.shape[1], offsets.tolist()
    balance, parts = 0.0, 0
    score = sig / sig.sum(1, keepdim=True)
    for a, b in zip(o, o[1:]):
        if b > a:
            parts += 1
            share = torch.bincount(idx[a:b].reshape(-1), minlength=E).double() / idx[a:b].numel()
            balance = balance + E * (share * score[a:b].mean(0)).sum()
    z = (torch.logsumexp(logits, 1)[o[0]:o[-1]] ** 2).mean()
    return out, torch.stack([balance / parts, z]), leaf


def test_block_against_64_bits():
    """The output passes at most five bf16 roundings in a chain (the norm, the
    preactivation, the hidden row, the expert's output, the sum), a gradient
    ten (those of the norm, the preactivation and the hidden row, the weighted
    gradient, the hidden row's gradient, the preactivation's, the row's, the
    logits' where they enter a product, the sum over rows, the result):
    2^-9 of the norm each, root mean square."""
    import moe_layer
    block = moe_layer.MoEBlock(256, 128, 16, topk=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((150, 256), generator=g, device="cuda").to(BF16)
    grad = torch.randn((150, 256), generator=g, device="cuda").to(BF16)
    coef = torch.tensor([3.0, 0.5], device="cuda")
    offsets = torch.tensor([0, 70, 70, 141], dtype=torch.int32, device="cuda")
    kept = {}
    out, losses = block.forward(x, offsets, kept)
    grads = block.backward(grad, coef, kept)
    assert kept["layout"].errors() == 0
    want, want_losses, leaf = block64(block, x, kept["routing"].topk_idx, offsets)
    assert float((out.double() - want.detach()).norm() / want.detach().norm()) < 5 * 2.0 ** -9
    assert ((losses.double() - want_losses.detach()).abs() < 2 * 2.0 ** -9 * want_losses.detach().abs()).all()
    ((want * grad.double()).sum() + (want_losses * coef.double()).sum()).backward()
    for name, v in leaf.items():
        off = float((grads[name].double() - v.grad).norm() / v.grad.norm())
        assert off < 10 * 2.0 ** -9, (name, off)


def test_blocks_on_two_streams():
    import moe_layer
    blocks = [moe_layer.MoEBlock(256, 128, 8, seed=s) for s in (1, 2)]
    g = torch.Generator(device="cuda").manual_seed(9)
    xs = [torch.randn((400, 256), generator=g, device="cuda").to(BF16) for _ in blocks]
    grads = [torch.randn((400, 256), generator=g, device="cuda").to(BF16) for _ in blocks]
    coef = torch.tensor([1.0, 0.1], device="cuda")

    def step(i):
        kept = {}
        out, losses = blocks[i].forward(xs[i], None, kept)
        return [out, losses, *blocks[i].backward(grads[i], coef, kept).values()]

    want = [step(0), step(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(i))
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(run, want[i]))


def test_two_graphs_and_an_eager_step():
    """Two captured steps of the new operators with workspaces of their own,
    replayed at once on two streams beside an eager one: nothing is shared."""
    def make(seed, T):
        g = torch.Generator(device="cuda").manual_seed(seed)
        t = dict(x=torch.randn((T, 512), generator=g, device="cuda").to(BF16), w=torch.randn((64, 512), generator=g, device="cuda").to(BF16) / 22,
                 b=torch.randn(64, generator=g, device="cuda"), nw=torch.rand(512, generator=g, device="cuda"),
                 mean=torch.empty(T, device="cuda"), rstd=torch.empty(T, device="cuda"), coef=torch.ones(2, device="cuda"))

        def step():
            n = ep.ep_layer_norm(t["x"], t["nw"], mean=t["mean"], rstd=t["rstd"])
            logits = ep.ep_dense_product(n, t["w"], t["b"], out_dtype=torch.float32)
            r = ep.ep_route(logits, 4)
            b = ep.ep_balance_loss(logits, r.topk_idx)
            d = ep.ep_balance_loss_backward(t["coef"], logits, b)
            dn, dw, db = ep.ep_dense_product_backward(d, n, t["w"], bias_dtype=torch.float32)
            dx, gw, gb = ep.ep_layer_norm_backward(dn, t["x"], t["mean"], t["rstd"], t["nw"])
            return logits, b.losses, b.counts, d, dw, db, dx, gw, gb
        return t, step

    parts = [make(s, T) for s, T in ((1, 3000), (2, 777), (3, 2000))]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _, step in parts:
            step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _, step in parts[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    for t, _ in parts:
        t["x"].normal_()
    want = [step() for _, step in parts]
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        with torch.cuda.stream(streams[2]):
            eager = parts[2][1]()
    torch.cuda.synchronize()
    for got, w in zip([*outs, eager], want):
        assert all(torch.equal(a, b) for a, b in zip(got, w))


def test_captured_without_a_call_before():
    """In a process of its own: the first calls are the captured ones."""
    import subprocess
    code = """
import torch, combine_ep_get_layout_gb300 as ep
ep.library_path()
x = torch.randn((500, 1024), device="cuda").bfloat16(); g = torch.randn_like(x)
w = torch.randn((72, 1024), device="cuda").bfloat16(); gw = torch.randn((500, 72), device="cuda").bfloat16()
l = torch.randn((4000, 256), device="cuda"); idx = torch.argsort(l, 1)[:, :2].contiguous()
m, r, one = torch.zeros(500, device="cuda"), torch.ones(500, device="cuda"), torch.ones(2, device="cuda")
torch.cuda.synchronize()
def step():
    n = ep.ep_layer_norm(x, mean=m, rstd=r)
    b = ep.ep_balance_loss(l, idx)
    return (n, ep.ep_dense_product(n, w, out_dtype=torch.float32), b.losses, ep.ep_balance_loss_backward(one, l, b),
            *ep.ep_layer_norm_backward(g, x, m, r), *ep.ep_dense_product_backward(gw, x, w, bias_dtype=torch.float32))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, step()))
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and "captured" in p.stdout, p.stderr[-2000:]


def test_calls_from_two_threads():
    """Each with its own stream and sizes: limits of shared memory, messages
    and tensors belong to the call."""
    import threading
    want, got, errors = {}, {}, []

    def work(i, store):
        try:
            g = torch.Generator(device="cuda").manual_seed(i)
            T, H = (300, 4096) if i else (50, 264)
            x = torch.randn((T, H), generator=g, device="cuda").to(BF16)
            w = torch.randn((72, H), generator=g, device="cuda").to(BF16)
            l = torch.randn((T, 512 if i else 12), generator=g, device="cuda")
            mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
            out = []
            for _ in range(20):
                n = ep.ep_layer_norm(x, mean=mean, rstd=rstd)
                idx = ep.ep_route(l, 3).topk_idx
                out.append((n, ep.ep_dense_product(n, w, activation="gelu"), ep.ep_balance_loss(l, idx).losses,
                            *ep.ep_layer_norm_backward(n, x, mean, rstd)))
            torch.cuda.current_stream().synchronize()
            store[i] = out
        except Exception as e:  # reported by the test
            errors.append(e)

    for i in range(2):
        work(i, want)

    def thread(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            work(i, got)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for i in range(2):
        for a, b in zip(got[i], want[i]):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
