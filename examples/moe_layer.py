"""A mixture-of-experts layer with a shared projection and low-rank adapters,
from the gate's logits to the combined output, and its training step.

    python examples/moe_layer.py [--tokens N] [--hidden N] [--width N] [--experts N]

Serving (``forward``): the router picks each token's experts, the expanded
layout groups the rows by expert, the dispatch copies them, two products with
SiLU gating between run over them, and the combine adds them up by their
weights.  A shared projection runs beside it, with each request's own adapter.

Training (``backward``): the gradients of both products, of the gate weights
and of the router's logits, for the loss ``sum(out * grad_out)``.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import combine_ep_get_layout_gb300 as ep  # noqa: E402

BF16 = torch.bfloat16


class MoELayer:
    """Weights of one layer: the gate [E, H] with its balance bias [E], the
    experts' w1 [E, 2F, H] and w2 [E, H, F], a shared projection [H, H] with
    adapters A [N, r, H], B [N, H, r] and scales [N]."""

    def __init__(self, hidden, width, experts, topk=4, ranks=4, adapters=8, rank=16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape):
            return (torch.randn(shape, generator=g, device=device) / math.sqrt(shape[-1])).to(BF16)

        self.experts, self.topk, self.ranks = experts, topk, ranks
        self.gate, self.bias = normal(experts, hidden), torch.zeros(experts, device=device)
        self.w1, self.w2 = normal(experts, 2 * width, hidden), normal(experts, hidden, width)
        self.shared = normal(hidden, hidden)
        self.lora_a, self.lora_b = normal(adapters, rank, hidden), normal(adapters, hidden, rank)
        self.scale = torch.ones(adapters, device=device)

    def forward(self, x, request, keep=None):
        """x bf16 [T, H]; request int64 [T]: each row's adapter, -1 = none.
        Returns bf16 [T, H]; ``keep`` (a dict) receives what backward needs."""
        logits = x.float() @ self.gate.float().T
        routing = ep.ep_route(logits, self.topk, score="sigmoid", bias=self.bias, num_groups=self.ranks,
                              topk_groups=max(1, self.ranks // 2), group_top=2)
        layout = ep.ep_get_layout_expanded(routing.topk_idx, self.experts)
        rows = ep.ep_dispatch_expanded(x, routing.topk_idx, None, layout, self.ranks).recv_x
        preact = None
        if keep is not None:
            preact = torch.empty((rows.shape[0], self.w1.shape[1]), dtype=BF16, device=x.device)
        hidden = ep.ep_expert_product(rows, self.w1, layout, activation="swiglu", preact=preact)
        y = ep.ep_expert_product(hidden, self.w2, layout)
        beside = ep.ep_adapter_product(x, self.shared, self.lora_a, self.lora_b, request, self.scale)
        out = ep.ep_combine_expanded(y, layout, routing.topk_idx, routing.topk_weights, bias0=beside)
        if keep is not None:
            keep.update(logits=logits, routing=routing, layout=layout, rows=rows, preact=preact, hidden=hidden, y=y)
        return out

    def backward(self, grad_out, kept):
        """The gradients of w1, w2 and of the logits for the output's gradient
        (bf16 [T, H]); the routed path only."""
        k = kept
        r, layout = k["routing"], k["layout"]
        slot = layout.token_slot.long()  # [T, K], -1 = no row
        there = slot >= 0
        at = slot.clamp_min(0)
        # of the combine: each row's gradient is its token's times its weight,
        # and a weight's the product of its row with its token's gradient
        grad_y = torch.zeros_like(k["y"])
        grad_rows = (r.topk_weights[:, :, None] * grad_out.float()[:, None, :]).to(BF16)
        grad_y[slot[there]] = grad_rows[there]
        grad_weights = (k["y"].float()[at] * grad_out.float()[:, None, :]).sum(2).masked_fill(~there, 0.0)
        grad_hidden, grad_w2 = ep.ep_expert_product_backward(grad_y, k["hidden"], self.w2, layout)
        _, grad_w1 = ep.ep_expert_product_backward(grad_hidden, k["rows"], self.w1, layout, activation="swiglu",
                                                   preact=k["preact"], need_x=False)
        grad_logits = ep.ep_route_backward(grad_weights, k["logits"], r.topk_idx, score="sigmoid")
        return {"w1": grad_w1, "w2": grad_w2, "logits": grad_logits}


def plain(layer, x, request, routing):
    """The same output by loops of products in 64 bits, for a fixed routing."""
    w1, w2, xd = layer.w1.double(), layer.w2.double(), x.double()
    out = xd @ layer.shared.double().T
    for a in range(layer.lora_a.shape[0]):
        at = (request == a).nonzero()[:, 0]
        out[at] += layer.scale[a].double() * (xd[at] @ layer.lora_a[a].double().T) @ layer.lora_b[a].double().T
    for e in range(layer.experts):
        token, k = (routing.topk_idx == e).nonzero(as_tuple=True)
        gate, up = (xd[token] @ w1[e].T).chunk(2, dim=1)
        y = (torch.nn.functional.silu(gate) * up) @ w2[e].T
        out.index_add_(0, token, routing.topk_weights[token, k].double()[:, None] * y)
    return out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=1000)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--experts", type=int, default=16)
    a = ap.parse_args(argv)
    layer = MoELayer(a.hidden, a.width, a.experts)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((a.tokens, a.hidden), generator=g, device="cuda").to(BF16)
    request = torch.randint(-1, 8, (a.tokens,), generator=g, device="cuda")
    kept = {}
    out = layer.forward(x, request, kept)
    want = plain(layer, x, request, kept["routing"])
    off = float((out.double() - want).norm() / want.norm())
    grads = layer.backward(torch.randn((a.tokens, a.hidden), generator=g, device="cuda").to(BF16), kept)
    print(f"{a.tokens} tokens: output {tuple(out.shape)}, {off:.1e} from 64 bits; gradients "
          + ", ".join(f"{n} {tuple(v.shape)}" for n, v in grads.items()))
    return off, out, kept, grads


if __name__ == "__main__":
    main()
