"""The example layer runs the router, the layout, dispatch, products, adapters
and combine together, and its gradients agree with 64-bit differentiation."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_example_output():
    """Five bf16 roundings of 2^-9 (root mean square) lie between input and
    output: the hidden rows, the experts' outputs, the low rows, the shared
    projection and the result."""
    import moe_layer
    off, out, kept, grads = moe_layer.main(["--tokens", "333"])
    assert kept["layout"].errors() == 0
    assert off < 5 * 2.0 ** -9
    assert all(torch.isfinite(v).all() for v in grads.values())


def test_example_gradients():
    """Against torch's differentiation of the layer in 64 bits at the kept
    routing.  Every gradient passes at most five bf16 roundings (the rows'
    gradient, the hidden rows, the preactivation, its gradient, the result):
    5 * 2^-9 of its norm."""
    import moe_layer
    layer = moe_layer.MoELayer(128, 64, 8, topk=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((70, 128), generator=g, device="cuda").to(torch.bfloat16)
    grad = torch.randn((70, 128), generator=g, device="cuda").to(torch.bfloat16)
    kept = {}
    layer.forward(x, torch.full((70,), -1, device="cuda"), kept)
    got = layer.backward(grad, kept)
    idx = kept["routing"].topk_idx
    w1, w2, logits = (t.double().requires_grad_(True) for t in (layer.w1, layer.w2, kept["logits"]))
    p = torch.sigmoid(logits).gather(1, idx)
    p = p / p.sum(1, keepdim=True)
    out = 0.0
    for k in range(3):
        gate, up = torch.einsum("th,tnh->tn", x.double(), w1[idx[:, k]]).chunk(2, dim=1)
        out = out + p[:, k:k + 1] * torch.einsum("tf,thf->th", torch.nn.functional.silu(gate) * up, w2[idx[:, k]])
    (out * grad.double()).sum().backward()
    for name, want in (("w1", w1.grad), ("w2", w2.grad), ("logits", logits.grad)):
        off = float((got[name].double() - want).norm() / want.norm())
        assert off < 5 * 2.0 ** -9, (name, off)


def test_two_streams_at_once():
    """Two layers' products and adapters on two streams, interleaved by the
    device as it likes: the outputs equal the ones of a single stream."""
    import moe_layer
    layers = [moe_layer.MoELayer(256, 128, 8, seed=s) for s in (1, 2)]
    g = torch.Generator(device="cuda").manual_seed(9)
    xs = [torch.randn((500, 256), generator=g, device="cuda").to(torch.bfloat16) for _ in layers]
    requests = [torch.randint(-1, 8, (500,), generator=g, device="cuda") for _ in layers]
    want = [m.forward(x, r) for m, x, r in zip(layers, xs, requests)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(layers[i].forward(xs[i], requests[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in range(2) for o in got[i])


def test_a_captured_layer_replays():
    """The calls allocate nothing in the library and are captured into a
    graph; a replay on new inputs gives what direct calls give."""
    import combine_ep_get_layout_gb300 as ep
    import moe_layer
    layer = moe_layer.MoELayer(256, 128, 8)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((64, 256), generator=g, device="cuda").to(torch.bfloat16)
    request = torch.randint(-1, 8, (64,), generator=g, device="cuda")
    logits = torch.randn((64, 8), generator=g, device="cuda")

    def step():
        r = ep.ep_route(logits, 2)
        return r.topk_idx, r.topk_weights, ep.ep_adapter_product(x, layer.shared, layer.lora_a, layer.lora_b, request)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.normal_(generator=g)
    logits.normal_(generator=g)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, step()):
        assert torch.equal(a, b)
