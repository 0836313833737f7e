"""A mixture-of-experts layer with a shared projection and low-rank adapters,
from the gate's logits to the combined output, and its training step.

    python examples/moe_layer.py [--tokens N] [--hidden N] [--width N] [--experts N]
                                 (hidden and width in multiples of 8)

Serving (``forward``): the router picks each token's experts, the expanded
layout groups the rows by expert, the dispatch copies them, two products with
SiLU gating between run over them, and the combine adds them up by their
weights.  A shared projection runs beside it, with each request's own adapter.

Training (``backward``): the gradients of both products, of the gate weights
and of the router's logits, for the loss ``sum(out * grad_out)``.

``MoEBlock`` is the block around such a layer as it is trained: layer norm,
the gate, the routed experts beside a shared one, the residual, and the losses
that keep the router balanced, with the gradients of all of it.
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
        logits = ep.ep_dense_product(x, self.gate, out_dtype=torch.float32)
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

    def backward(self, grad_out, kept, need_rows=False):
        """The gradients of w1, w2 and of the logits for the output's gradient
        (bf16 [T, H]); the routed path only.  With ``need_rows`` also that of
        the dispatched rows."""
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
        grad_x, grad_w1 = ep.ep_expert_product_backward(grad_hidden, k["rows"], self.w1, layout, activation="swiglu",
                                                        preact=k["preact"], need_x=need_rows)
        grad_logits = ep.ep_route_backward(grad_weights, k["logits"], r.topk_idx, score="sigmoid")
        grads = {"w1": grad_w1, "w2": grad_w2, "logits": grad_logits}
        if need_rows:
            grads["rows"] = grad_x
        return grads


class MoEBlock(MoELayer):
    """``x + experts(norm(x)) + shared(norm(x))`` with the router's losses: the
    layer's gate and experts, a norm's weight and bias [H], and a shared
    expert's s1 [2F, H] with bias, s2 [H, F] with bias."""

    def __init__(self, hidden, width, experts, topk=4, ranks=4, seed=0, device="cuda"):
        super().__init__(hidden, width, experts, topk, ranks, seed=seed, device=device)
        g = torch.Generator(device=device).manual_seed(seed + 1)
        self.norm_weight = 1.0 + 0.1 * torch.randn(hidden, generator=g, device=device)
        self.norm_bias = 0.1 * torch.randn(hidden, generator=g, device=device)
        self.s1 = (torch.randn((2 * width, hidden), generator=g, device=device) / math.sqrt(hidden)).to(BF16)
        self.s2 = (torch.randn((hidden, width), generator=g, device=device) / math.sqrt(width)).to(BF16)
        self.s1_bias = 0.1 * torch.randn(2 * width, generator=g, device=device)
        self.s2_bias = 0.1 * torch.randn(hidden, generator=g, device=device)

    def forward(self, x, seq_offsets=None, keep=None):
        """x bf16 [T, H], seq_offsets int32 [S + 1] of the sequences packed in
        it (None: one).  Returns (out bf16 [T, H], the balance and z loss fp32
        [2]); ``keep`` (a dict) receives what backward needs."""
        T, dev = x.shape[0], x.device
        mean, rstd = torch.empty(T, device=dev), torch.empty(T, device=dev)
        n = ep.ep_layer_norm(x, self.norm_weight, self.norm_bias, mean=mean, rstd=rstd)
        logits = ep.ep_dense_product(n, self.gate, out_dtype=torch.float32)
        routing = ep.ep_route(logits, self.topk, score="sigmoid", bias=self.bias)
        balance = ep.ep_balance_loss(logits, routing.topk_idx, score="sigmoid", seq_offsets=seq_offsets)
        layout = ep.ep_get_layout_expanded(routing.topk_idx, self.experts)
        rows = ep.ep_dispatch_expanded(n, routing.topk_idx, None, layout, self.ranks).recv_x
        preact = torch.empty((rows.shape[0], self.w1.shape[1]), dtype=BF16, device=dev)
        hidden = ep.ep_expert_product(rows, self.w1, layout, activation="swiglu", preact=preact)
        y = ep.ep_expert_product(hidden, self.w2, layout)
        routed = ep.ep_combine_expanded(y, layout, routing.topk_idx, routing.topk_weights, bias0=x)
        shared_preact = torch.empty((T, self.s1.shape[0]), dtype=BF16, device=dev)
        shared = ep.ep_dense_product(n, self.s1, self.s1_bias, activation="swiglu", preact=shared_preact)
        out = ep.ep_dense_product(shared, self.s2, self.s2_bias, residual=routed)
        if keep is not None:
            keep.update(x=x, mean=mean, rstd=rstd, n=n, logits=logits, routing=routing, balance=balance, layout=layout,
                        rows=rows, preact=preact, hidden=hidden, y=y, shared_preact=shared_preact, shared=shared,
                        seq_offsets=seq_offsets)
        return out, balance.losses

    def backward(self, grad_out, grad_losses, kept):
        """The gradients of every parameter and of x, for those of the output
        (bf16 [T, H]) and of the losses (fp32 [2])."""
        k = kept
        grad_shared, s2, s2_bias = ep.ep_dense_product_backward(grad_out, k["shared"], self.s2, bias_dtype=torch.float32)
        n_shared, s1, s1_bias = ep.ep_dense_product_backward(grad_shared, k["n"], self.s1, activation="swiglu",
                                                             preact=k["shared_preact"], bias_dtype=torch.float32)
        grads = super().backward(grad_out, k, need_rows=True)
        logits = ep.ep_balance_loss_backward(grad_losses, k["logits"], k["balance"], score="sigmoid",
                                             seq_offsets=k["seq_offsets"], add=grads["logits"])
        n_gate, gate, _ = ep.ep_dense_product_backward(logits, k["n"], self.gate)
        # the sum of a token's rows, and the two others
        grad_n = ep.ep_combine_expanded(grads["rows"], k["layout"], bias0=n_shared, bias1=n_gate)
        x, norm_weight, norm_bias = ep.ep_layer_norm_backward(grad_n, k["x"], k["mean"], k["rstd"], self.norm_weight,
                                                              add=grad_out)
        return {"x": x, "norm_weight": norm_weight, "norm_bias": norm_bias, "gate": gate, "w1": grads["w1"],
                "w2": grads["w2"], "s1": s1, "s1_bias": s1_bias, "s2": s2, "s2_bias": s2_bias, "logits": logits}


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
    block, kept_block = MoEBlock(a.hidden, a.width, a.experts), {}
    y, losses = block.forward(x, None, kept_block)
    grad = torch.randn((a.tokens, a.hidden), generator=g, device="cuda").to(BF16)
    block_grads = block.backward(grad, torch.tensor([1e-2, 1e-3], device="cuda"), kept_block)
    print(f"block: output {tuple(y.shape)}, balance and z loss {losses.tolist()}; gradients " + ", ".join(block_grads))
    return off, out, kept, grads


if __name__ == "__main__":
    main()
