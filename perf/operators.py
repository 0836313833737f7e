"""The operators measured around the expert-parallel path, as cases.

Five operators of a mixture-of-experts layer, next to the layout, dispatch and
combine that move its rows:

  route              the gate's logits to the experts and weights of each token
  route_backward     the gradient of those weights with respect to the logits
  product            each expert's rows times its weights (plain, or gated by SiLU)
  product_backward   the gradients of that product for the rows and the weights
  adapters           a shared projection plus each row's own low-rank adapter

Every case names sizes; ``prepare`` makes its inputs on the GPU from a seed,
``run`` makes one pass (the package's calls where ``own`` is true, elementary
torch operations in 32 bits where it is not), ``exact`` gives the same outputs
from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64, I64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int64, torch.int32


# ------------------------------------------------------------------- cases

def listed():
    return [
        # One decoding step of a small batch: the router's latency.
        dict(name="route_decode", op="route", tokens=13, experts=64, topk=6, score="softmax", bias=False,
             groups=1, topk_groups=1, group_top=1, renorm=True, dtype="bf16", masked=0.0),
        # A training batch with balance biases and a limit of four of the eight ranks a token.
        dict(name="route_train", op="route", tokens=65536, experts=256, topk=8, score="sigmoid", bias=True,
             groups=8, topk_groups=4, group_top=2, renorm=True, dtype="fp32", masked=0.0),
        # The backward pass of an ordinary batch, an odd count of tokens, weights not renormalised.
        dict(name="route_backward_dense", op="route_backward", tokens=4093, experts=64, topk=6,
             score="softmax", renorm=False, dtype="bf16", masked=0.1),
        # The backward pass of the training batch.
        dict(name="route_backward_train", op="route_backward", tokens=65536, experts=256, topk=8,
             score="sigmoid", renorm=True, dtype="fp32", masked=0.0),
        # Serving: a few tokens over many experts; reading the weights is the work.
        dict(name="product_decode", op="product", tokens=24, topk=6, experts=64, hidden=4096, width=1408,
             act="swiglu", align=1, zipf=0.0, masked=0.0),
        # A prompt's first half of the expert, gate and up in one product.
        dict(name="product_prefill", op="product", tokens=4096, topk=6, experts=64, hidden=4096, width=1408,
             act="swiglu", align=1, zipf=0.0, masked=0.0),
        # The second half over many experts: a short inner size and wide rows out.
        dict(name="product_down", op="product", tokens=8192, topk=8, experts=256, hidden=512, width=7168,
             act="none", align=16, zipf=0.0, masked=0.0),
        # The smallest training step, with masked choices.
        dict(name="product_backward_small", op="product_backward", tokens=128, topk=2, experts=16, hidden=256,
             width=136, act="swiglu", align=8, zipf=0.0, masked=0.1),
        # A training batch with skewed routing and masked choices.
        dict(name="product_backward_train", op="product_backward", tokens=4096, topk=6, experts=64, hidden=4096,
             width=1408, act="swiglu", align=1, zipf=0.6, masked=0.1),
        # One decoding step of 32 requests with two dozen adapters.
        dict(name="adapters_decode", op="adapters", rows=32, hidden=4096, width=4096, adapters=24, rank=16,
             spread="rows", none=0.1),
        # Prompts in chunks beside decoding rows, an odd count of rows, a narrow projection.
        dict(name="adapters_mixed", op="adapters", rows=1021, hidden=4096, width=1000, adapters=40, rank=8,
             spread="mixed", none=0.1),
        # Long prompts of a few requests.
        dict(name="adapters_prefill", op="adapters", rows=8192, hidden=7168, width=4096, adapters=8, rank=32,
             spread="runs", none=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _eights(rng, lo, hi):
    return max(8, _log(rng, lo, hi) // 8 * 8)


def draw(rng):
    op = rng.choice(["route", "route_backward", "product", "product_backward", "adapters"])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 2, 4, 8]) if op == "route" else 1
        experts = groups * max(1, _log(rng, 8, 512) // groups)
        topk = rng.randint(1, min(10, experts))
        tokens = _log(rng, 1, 65536 * 256 // max(256, experts))
        case = dict(op=op, tokens=tokens, experts=experts, topk=topk, score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.6, dtype=rng.choice(["fp32", "bf16"]), masked=rng.choice([0.0, 0.0, 0.1]))
        if op == "route":
            case.update(bias=rng.random() < 0.5, groups=groups, topk_groups=rng.randint(1, groups),
                        group_top=rng.choice([1, 2]))
        return case
    if op in ("product", "product_backward"):
        act = rng.choice(["none", "swiglu"])
        most = 3e11 if op == "product" else 1.2e11
        while True:
            case = dict(op=op, tokens=_log(rng, 1, 8192), topk=rng.randint(1, 8), experts=_log(rng, 8, 256),
                        hidden=_eights(rng, 64, 7168), width=_eights(rng, 64, 4096), act=act,
                        align=rng.choice([1, 1, 8, 16, 128]), zipf=rng.choice([0.0, 0.0, 1.2]),
                        masked=rng.choice([0.0, 0.0, 0.1]))
            weights = case["experts"] * case["hidden"] * case["width"] * (2 if act == "swiglu" else 1)
            rows = case["tokens"] * case["topk"]
            # the padded batch of the plain form stays within a few GB too
            if 2.0 * rows * weights / case["experts"] <= most and weights <= 1.1e9 and rows * case["hidden"] <= 3e8 \
                    and (case["zipf"] == 0.0 or rows * case["experts"] * (case["hidden"] + 4 * case["width"]) <= 1.2e10):
                return case
    while True:
        case = dict(op=op, rows=_log(rng, 1, 8192), hidden=_eights(rng, 64, 7168), width=_eights(rng, 64, 7168),
                    adapters=_log(rng, 1, 64), rank=rng.choice([8, 16, 24, 32, 64]),
                    spread=rng.choice(["rows", "mixed", "runs"]), none=rng.choice([0.0, 0.1, 1.0 / 3]))
        if case["rows"] * case["hidden"] * case["width"] <= 8192 * 7168 * 4096 and \
                (case["spread"] != "rows" or case["rows"] <= 512):
            return case


# ------------------------------------------------------------------- inputs

def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + salt)
    return g


def _normal(g, shape, dtype=F32, std=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=F32).mul_(std).to(dtype)


def _type(case):
    return BF16 if case["dtype"] == "bf16" else F32


def _logits(g, case, rows):
    """The gate's logits; a masked expert (not offered to a token) has -infinity."""
    x = _normal(g, (rows, case["experts"]), _type(case), 1.5)
    if case["masked"]:
        x.masked_fill_(torch.rand(x.shape, generator=g, device=DEV) < case["masked"], -math.inf)
    return x


def _scores64(case, logits):
    x = logits.to(F64)
    return torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1).nan_to_num(0.0)


def _by_logit(case):
    """Without biases, and with groups judged by their best expert, the scores' order is the logits' order."""
    return not case["bias"] and (case["groups"] == 1 or case["group_top"] == 1)


def _selection64(case, logits, bias):
    """(the experts' keys, the groups' scores or None), in 64 bits, masked ones at -infinity."""
    key = logits.to(F64) if _by_logit(case) else _scores64(case, logits)
    if case["bias"]:
        key = key + bias.to(F64)
    key = key.masked_fill(torch.isneginf(logits), -math.inf)
    if case["groups"] == 1:
        return key, None
    per = key.view(key.shape[0], case["groups"], -1)
    top = torch.sort(per, dim=2, descending=True, stable=True)[0][:, :, :case["group_top"]]
    return key, torch.where(torch.isneginf(top[:, :, :1]), top[:, :, :1], top.masked_fill(torch.isneginf(top), 0.0)).sum(2)


def _chosen64(case, key, group):
    """Keys of the experts in groups that were not chosen at -infinity."""
    if group is None:
        return key
    order = torch.sort(group, dim=1, descending=True, stable=True)[1][:, :case["topk_groups"]]
    keep = torch.zeros_like(group, dtype=torch.bool).scatter_(1, order, True)
    return key.masked_fill(~keep.repeat_interleave(key.shape[1] // case["groups"], 1), -math.inf)


def _near_tie(case, logits, bias):
    """Rows whose choice hangs on less than 32 bits resolve: two different keys closer than their rounding."""
    key, group = _selection64(case, logits, bias)
    bad = torch.zeros(key.shape[0], dtype=torch.bool, device=DEV)
    lists = [(_chosen64(case, key, group), case["topk"] + 1)]
    if group is not None:
        lists.append((group, case["topk_groups"] + 1))
    if _by_logit(case):
        return bad  # logits are compared as they are: a tie is a tie
    for values, n in lists:
        v = torch.sort(values, dim=1, descending=True)[0][:, :n]
        gap = v[:, :-1] - v[:, 1:]
        size = 0.3 if case["bias"] else v[:, :-1].abs()
        bad |= ((gap > 0) & (gap < 4e-6 * size)).any(1)
    return bad


def _prepare_route(case, seed):
    g = _gen(seed, 1)
    s = {"logits": _logits(g, case, case["tokens"]),
         "bias": _normal(g, (case["experts"],), F32, 0.05) if case["bias"] else None}
    for _ in range(50):
        bad = _near_tie(case, s["logits"], s["bias"])
        n = int(bad.sum())
        if not n:
            break
        s["logits"][bad] = _logits(g, case, n)
    return s


def _prepare_route_backward(case, seed):
    g = _gen(seed, 2)
    logits = _logits(g, case, case["tokens"])
    value, idx = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    idx = torch.where(torch.isneginf(value), -1, idx)[:, :case["topk"]].contiguous()
    return {"logits": logits, "topk_idx": idx, "grad": _normal(g, (case["tokens"], case["topk"]))}


def _routing(g, case):
    """topk_idx int64 [T, K]: distinct experts a token, uniform or skewed, some choices masked (-1)."""
    T, E, K = case["tokens"], case["experts"], min(case["topk"], case["experts"])
    key = torch.rand((T, E), generator=g, device=DEV).clamp_min_(1e-20).log_().neg_().log_().neg_()
    if case["zipf"]:
        order = torch.randperm(E, generator=g, device=DEV)
        key = key - case["zipf"] * torch.log(order.to(F32) + 1.0)
    idx = torch.sort(key, dim=1, descending=True)[1][:, :K]
    if case["masked"]:
        idx = idx.masked_fill(torch.rand(idx.shape, generator=g, device=DEV) < case["masked"], -1)
    return idx.contiguous()


def _expanded(idx, E, align):
    """The expanded layout of a routing: rows grouped by expert, each group's start rounded up to `align`."""
    flat = idx.reshape(-1)
    hot = flat[:, None] == torch.arange(E, device=DEV)
    counts = hot.sum(0)
    offset = torch.zeros(E + 1, dtype=I64, device=DEV)
    offset[1:] = ((counts + align - 1) // align * align).cumsum(0)
    nth = (hot.to(I32).cumsum(0, dtype=I32).gather(1, flat.clamp_min(0)[:, None])[:, 0] - 1).to(I64)
    slot = torch.where(flat >= 0, offset[flat.clamp_min(0)] + nth, -1)
    return counts, offset, slot.reshape(idx.shape)


def _prepare_product(case, seed):
    g = _gen(seed, 3)
    T, E, align = case["tokens"], case["experts"], case["align"]
    idx = _routing(g, case)
    counts, offset, slot = _expanded(idx, E, align)
    K = idx.shape[1]
    cap = T * K + E * (align - 1)
    H, W = case["hidden"], case["width"]
    N = 2 * W if case["act"] == "swiglu" else W
    x = torch.zeros((cap, H), dtype=BF16, device=DEV)
    rows = slot.reshape(-1)
    token = torch.arange(T, device=DEV).repeat_interleave(K)[rows >= 0]
    x[rows[rows >= 0]] = _normal(g, (T, H), BF16)[token]
    w = torch.empty((E, N, H), dtype=BF16, device=DEV)
    step = max(1, (1 << 28) // (N * H))
    for e in range(0, E, step):
        w[e:e + step] = _normal(g, (min(step, E - e), N, H), BF16, 1.0 / math.sqrt(H))
    s = {"T": T, "K": K, "E": E, "align": align, "max_rows": max(1, int(counts.max())),
         "num_rows_per_expert": counts.to(I32), "expert_offset": offset.to(I32), "token_slot": slot.to(I32),
         "error_word": torch.zeros(1, dtype=I32, device=DEV), "workspace": torch.zeros(256, dtype=torch.uint8, device=DEV),
         "x": x, "w": w, "act": case["act"], "rows": rows, "hosts": counts.tolist(), "starts": offset.tolist()}
    if case["op"] == "product":
        s["out"] = torch.zeros((cap, W), dtype=BF16, device=DEV)
        return s
    grad = torch.zeros((cap, W), dtype=BF16, device=DEV)
    grad[rows[rows >= 0]] = _normal(g, (int((rows >= 0).sum()), W), BF16)
    s["grad"] = grad
    s["grad_x"] = torch.zeros((cap, H), dtype=BF16, device=DEV)
    s["grad_w"] = torch.zeros((E, N, H), dtype=BF16, device=DEV)
    if case["act"] == "swiglu":  # what the forward pass kept
        pre = torch.zeros((cap, N), dtype=BF16, device=DEV)
        for e, (a, n) in enumerate(zip(s["starts"], s["hosts"])):
            pre[a:a + n] = (x[a:a + n] @ w[e].T)
        s["preact"] = pre
    return s


def _prepare_adapters(case, seed):
    g = _gen(seed, 4)
    T, K, N, A, r = case["rows"], case["hidden"], case["width"], case["adapters"], case["rank"]
    if case["spread"] == "rows":  # decoding: every row its own request
        idx = torch.randint(0, A, (T,), generator=g, device=DEV)
        idx[torch.rand(T, generator=g, device=DEV) < case["none"]] = -1
    else:
        # requests of many rows one after the other; "mixed": the last eighth are decoding rows
        cuts = max(1, T // 300) if case["spread"] == "mixed" else min(max(1, T // 64), A)
        place = torch.sort(torch.randint(0, T, (cuts,), generator=g, device=DEV))[0]
        owner = torch.randint(0, A, (cuts + 1,), generator=g, device=DEV)
        owner[torch.rand(cuts + 1, generator=g, device=DEV) < case["none"]] = -1
        idx = owner[torch.searchsorted(place, torch.arange(T, device=DEV), right=True)]
        if case["spread"] == "mixed":
            tail = T // 8
            idx[T - tail:] = torch.randint(0, A, (tail,), generator=g, device=DEV)
    return {"x": _normal(g, (T, K), BF16), "w": _normal(g, (N, K), BF16, 1.0 / math.sqrt(K)),
            "lora_a": _normal(g, (A, r, K), BF16, 1.0 / math.sqrt(K)),
            "lora_b": _normal(g, (A, N, r), BF16, 0.5 / math.sqrt(r)),
            "scale": torch.rand(A, generator=g, device=DEV) + 0.5, "adapter_idx": idx.contiguous()}


def prepare(case, seed):
    s = {"route": _prepare_route, "route_backward": _prepare_route_backward, "product": _prepare_product,
         "product_backward": _prepare_product, "adapters": _prepare_adapters}[case["op"]](case, seed)
    s["case"] = case
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


# The plain forms: 32 bits, rounded once at the end.

def _scores(case, x):
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.amax(1, keepdim=True).clamp_min(-3.0e38)
    e = torch.exp(x - top)
    return e / e.sum(1, keepdim=True).clamp_min(1e-38)


def _plain_route(s):
    case, x = s["case"], s["logits"].float()
    p = _scores(case, x)
    key = x if _by_logit(case) else p if s["bias"] is None else p + s["bias"]
    none = torch.isneginf(x)
    key = key.masked_fill(none, -math.inf)
    if case["groups"] > 1:
        per = key.view(x.shape[0], case["groups"], -1)
        top = torch.sort(per, dim=2, descending=True, stable=True)[0][:, :, :case["group_top"]]
        lost = torch.isneginf(top)
        group = top.masked_fill(lost, 0.0).sum(2).masked_fill(lost[:, :, 0], -math.inf)
        order = torch.sort(group, dim=1, descending=True, stable=True)[1][:, :case["topk_groups"]]
        keep = torch.zeros_like(group, dtype=torch.bool).scatter(1, order, True)
        key = torch.where(keep[:, :, None], per, -math.inf).view(x.shape)
    value, idx = torch.sort(key, dim=1, descending=True, stable=True)
    value, idx = value[:, :case["topk"]], idx[:, :case["topk"]]
    empty = torch.isneginf(value)
    w = p.gather(1, idx).masked_fill(empty, 0.0)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return {"topk_idx": torch.where(empty, -1, idx), "topk_weights": 2.5 * w}


def _plain_route_backward(s):
    case, x, idx = s["case"], s["logits"].float(), s["topk_idx"]
    p = _scores(case, x)
    empty = idx < 0
    at = idx.clamp_min(0)
    w = p.gather(1, at).masked_fill(empty, 0.0)
    d = (2.5 * s["grad"]).masked_fill(empty, 0.0)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        u = torch.where(total > 0, w / total, 0.0)
        d = torch.where(total > 0, (d - (d * u).sum(1, keepdim=True)) / total, 0.0)
    d = d.masked_fill(empty, 0.0)
    dense = torch.zeros_like(p).scatter_add(1, at, d)
    if case["score"] == "sigmoid":
        g = dense * p * (1.0 - p)
    else:
        g = p * (dense - (dense * p).sum(1, keepdim=True))
    return {"grad_logits": g.to(s["logits"].dtype)}


def _padded(s, rows, idx, valid):
    """[E, M, n] in 32 bits: each expert's rows of `rows`, zeros after its last."""
    return rows[idx.clamp(max=rows.shape[0] - 1)].float() * valid[:, :, None]


def _places(s):
    j = torch.arange(s["max_rows"], device=DEV)
    return s["expert_offset"][:-1, None].long() + j, j < s["num_rows_per_expert"][:, None]


def _unpadded(s, padded, idx, valid):
    """Back to [cap, n]: the rows where the layout has them, zeros elsewhere."""
    cap = s["x"].shape[0]
    out = torch.zeros((cap + 1, padded.shape[2]), dtype=BF16, device=DEV)
    out[torch.where(valid, idx, cap).reshape(-1)] = padded.reshape(-1, padded.shape[2]).to(BF16)
    return out[:cap]


def _plain_product(s):
    idx, valid = _places(s)
    h = torch.bmm(_padded(s, s["x"], idx, valid), s["w"].float().transpose(1, 2))
    if s["act"] == "swiglu":
        gate, up = h.chunk(2, dim=2)
        h = gate / (1.0 + torch.exp(-gate)) * up
    return {"out": _unpadded(s, h, idx, valid)}


def _plain_product_backward(s):
    idx, valid = _places(s)
    g = _padded(s, s["grad"], idx, valid)
    if s["act"] == "swiglu":
        gate, up = _padded(s, s["preact"], idx, valid).chunk(2, dim=2)
        sig = 1.0 / (1.0 + torch.exp(-gate))
        g = torch.cat([g * up * sig * (1.0 + gate * (1.0 - sig)), g * gate * sig], 2)
    grad_x = _unpadded(s, torch.bmm(g, s["w"].float()), idx, valid)
    grad_w = torch.bmm(g.transpose(1, 2), _padded(s, s["x"], idx, valid)).to(BF16)
    return {"grad_x": grad_x, "grad_w": grad_w}


def _plain_adapters(s):
    x, idx = s["x"].float(), s["adapter_idx"]
    A, r, K = s["lora_a"].shape
    every = (x @ s["lora_a"].float().view(A * r, K).T).view(-1, A, r)
    mine = (idx[:, None] == torch.arange(A, device=DEV)) * s["scale"]
    low = (every * mine[:, :, None]).view(-1, A * r)
    y = x @ s["w"].float().T + low @ s["lora_b"].float().transpose(1, 2).reshape(A * r, -1)
    return {"out": y.to(BF16)}


_plain = {"route": _plain_route, "route_backward": _plain_route_backward, "product": _plain_product,
          "product_backward": _plain_product_backward, "adapters": _plain_adapters}


# The package's calls.

def _own_route(s):
    import combine_ep_get_layout_gb300 as ep
    c = s["case"]
    r = ep.ep_route(s["logits"], c["topk"], score=c["score"], bias=s["bias"], num_groups=c["groups"],
                    topk_groups=c["topk_groups"], group_top=c["group_top"], renormalize=c["renorm"], weight_scale=2.5)
    return {"topk_idx": r.topk_idx, "topk_weights": r.topk_weights}


def _own_route_backward(s):
    import combine_ep_get_layout_gb300 as ep
    c = s["case"]
    g = ep.ep_route_backward(s["grad"], s["logits"], s["topk_idx"], score=c["score"], renormalize=c["renorm"],
                             weight_scale=2.5)
    return {"grad_logits": g}


def _layout(s):
    import combine_ep_get_layout_gb300 as ep
    return ep.ExpandedLayout(s["num_rows_per_expert"], s["expert_offset"], s["token_slot"], s["error_word"],
                             s["workspace"], s["T"], s["K"], s["E"], s["align"])


def _own_product(s):
    import combine_ep_get_layout_gb300 as ep
    act = None if s["act"] == "none" else s["act"]
    return {"out": ep.ep_expert_product(s["x"], s["w"], _layout(s), activation=act, out=s["out"])}


def _own_product_backward(s):
    import combine_ep_get_layout_gb300 as ep
    act = None if s["act"] == "none" else s["act"]
    grad_x, grad_w = ep.ep_expert_product_backward(s["grad"], s["x"], s["w"], _layout(s), activation=act,
                                                   preact=s.get("preact"), grad_x=s["grad_x"], grad_w=s["grad_w"])
    return {"grad_x": grad_x, "grad_w": grad_w}


def _own_adapters(s):
    import combine_ep_get_layout_gb300 as ep
    return {"out": ep.ep_adapter_product(s["x"], s["w"], s["lora_a"], s["lora_b"], s["adapter_idx"], s["scale"])}


_own = {"route": _own_route, "route_backward": _own_route_backward, "product": _own_product,
        "product_backward": _own_product_backward, "adapters": _own_adapters}


# --------------------------------------------------------- what a pass needs

def _rows(case):
    return case["tokens"] * min(case["topk"], case["experts"]) * (1.0 - case["masked"])


def work(case):
    if case["op"] in ("route", "route_backward"):
        n = case["tokens"] * case["experts"]
        size = 2 if case["dtype"] == "bf16" else 4
        if case["op"] == "route":
            return {"bytes": n * size + case["tokens"] * case["topk"] * 12 + (4 * case["experts"] if case["bias"] else 0),
                    "flops": 4.0 * n}
        return {"bytes": 2 * n * size + case["tokens"] * case["topk"] * 12, "flops": 6.0 * n}
    if case["op"] in ("product", "product_backward"):
        rows, E, H, W = _rows(case), case["experts"], case["hidden"], case["width"]
        N = 2 * W if case["act"] == "swiglu" else W
        used = E * (1.0 - (1.0 - 1.0 / E) ** rows)  # experts with a row
        if case["op"] == "product":
            return {"bytes": 2 * (rows * (H + W) + used * N * H), "flops": 2.0 * rows * N * H}
        pre = N if case["act"] == "swiglu" else 0
        return {"bytes": 2 * (rows * (2 * H + W + pre) + used * N * H + E * N * H), "flops": 4.0 * rows * N * H}
    T, K, N, A, r = case["rows"], case["hidden"], case["width"], case["adapters"], case["rank"]
    if case["spread"] == "rows":
        used = A * (1.0 - (1.0 - 1.0 / A) ** (T * (1.0 - case["none"])))
    else:
        used = min(A, 1)
    return {"bytes": 2 * (T * (K + N) + N * K + used * r * (K + N)) + 8 * T,
            "flops": 2.0 * T * K * N + 2.0 * T * (1.0 - case["none"]) * r * (K + N)}


# ----------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        key, group = _selection64(case, s["logits"], s["bias"])
        key = _chosen64(case, key, group)
        order = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :case["topk"]]
        there = ~torch.isneginf(key.gather(1, order))
        w = _scores64(case, s["logits"]).gather(1, order) * there
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
        return {"topk_idx": torch.where(there, order, -1), "topk_weights": 2.5 * w}
    if case["op"] == "route_backward":
        # by torch's own differentiation of the definition
        x = s["logits"].to(F64).requires_grad_(True)
        there = s["topk_idx"] >= 0
        p = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
        w = torch.where(there, p.gather(1, s["topk_idx"].clamp_min(0)), 0.0)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
        (2.5 * w * s["grad"].to(F64)).sum().backward()
        return {"grad_logits": x.grad.nan_to_num(0.0)}
    if case["op"] == "product":
        out = torch.zeros(s["out"].shape, dtype=F64, device=DEV)
        for e, (a, n) in enumerate(zip(s["starts"], s["hosts"])):
            h = s["x"][a:a + n].to(F64) @ s["w"][e].to(F64).T
            if case["act"] == "swiglu":
                h = h[:, :case["width"]] * torch.sigmoid(h[:, :case["width"]]) * h[:, case["width"]:]
            out[a:a + n] = h
        return {"out": out}
    if case["op"] == "product_backward":
        grad_x = torch.zeros(s["x"].shape, dtype=F64, device=DEV)
        grad_w = torch.zeros(s["w"].shape, dtype=F64, device=DEV)
        for e, (a, n) in enumerate(zip(s["starts"], s["hosts"])):
            g = s["grad"][a:a + n].to(F64)
            if case["act"] == "swiglu":
                h = s["preact"][a:a + n].to(F64).requires_grad_(True)
                y = torch.nn.functional.silu(h[:, :case["width"]]) * h[:, case["width"]:]
                g, = torch.autograd.grad(y, h, g)
            grad_x[a:a + n] = g @ s["w"][e].to(F64)
            grad_w[e] = g.T @ s["x"][a:a + n].to(F64)
        return {"grad_x": grad_x, "grad_w": grad_w}
    x, idx = s["x"].to(F64), s["adapter_idx"]
    y = x @ s["w"].to(F64).T
    for k in range(case["adapters"]):
        at = (idx == k).nonzero()[:, 0]
        y[at] += float(s["scale"][k]) * (x[at] @ s["lora_a"][k].to(F64).T) @ s["lora_b"][k].to(F64).T
    return {"out": y}
