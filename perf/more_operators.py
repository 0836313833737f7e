"""The operators of a mixture-of-experts block's training step that stand
beside the router, the experts' products and the combine, as cases.

  balance  the router's balance loss and z loss, with each expert's counts,
           over sequences of a packed batch, and their gradient for the logits
  norm     layer norm of the block's rows, and its gradients for the rows
           (the residual's gradient added) and for its weight and bias
  dense    a product shared by all rows, x w^T, with bias, activation and
           residual in its epilogue: the gate, a shared expert; and its
           gradients for the rows, the weights and the bias

A case has ``backward``: whether it is the operator or its gradients.  Every
case names sizes; ``prepare`` makes its inputs on the GPU from a seed, ``run``
makes one pass (the package's calls where ``own`` is true, elementary torch
operations in 32 bits where it is not), ``exact`` gives the same outputs from
the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64, I64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int64, torch.int32
TYPES = {"bf16": BF16, "fp32": F32}
EPS = 1e-5


# ------------------------------------------------------------------- cases

def listed():
    return [
        # The losses of a fine-tuning step's small batch: bf16 logits, some experts masked, an odd count.
        dict(name="balance_small", op="balance", backward=False, tokens=1021, experts=64, topk=6, sequences=1,
             score="softmax", dtype="bf16", masked=0.1),
        # The losses of a training batch, balanced sequence by sequence, the end of the batch padding.
        dict(name="balance_train", op="balance", backward=False, tokens=65536, experts=256, topk=8, sequences=16,
             score="sigmoid", dtype="fp32", masked=0.0),
        # Their gradient on top of the gate weights' own.
        dict(name="balance_backward_train", op="balance", backward=True, tokens=65536, experts=256, topk=8,
             sequences=16, score="softmax", dtype="fp32", masked=0.0, add=True),
        # One decoding step's rows: the norm's latency.
        dict(name="norm_decode", op="norm", backward=False, rows=13, hidden=4096, dtype="bf16", params="bf16"),
        # A training batch's rows before the gate.
        dict(name="norm_train", op="norm", backward=False, rows=8192, hidden=7168, dtype="bf16", params="fp32"),
        # The gradients of a small batch kept in 32 bits, an odd count of rows.
        dict(name="norm_backward_odd", op="norm", backward=True, rows=1021, hidden=4096, dtype="fp32", params="fp32",
             add=False),
        # The gradients of the training batch, the residual's gradient added.
        dict(name="norm_backward_train", op="norm", backward=True, rows=8192, hidden=7168, dtype="bf16", params="fp32",
             add=True),
        # One decoding step of a small batch through an output projection: reading the weights is the work.
        dict(name="dense_decode", op="dense", backward=False, rows=24, hidden=4096, width=4096, act="none", bias=True,
             residual=True, out="bf16", params="bf16"),
        # The gate of a training batch: few outputs, kept in 32 bits for the router.
        dict(name="dense_gate", op="dense", backward=False, rows=8192, hidden=7168, width=256, act="none", bias=False,
             residual=False, out="fp32", params="fp32"),
        # A prompt through a shared expert's first half, the gate and what it multiplies, with biases.
        dict(name="dense_prefill", op="dense", backward=False, rows=4093, hidden=4096, width=2816, act="swiglu",
             bias=True, residual=False, out="bf16", params="fp32"),
        # The gradients of a small feed-forward's first half, an odd count of rows.
        dict(name="dense_backward_small", op="dense", backward=True, rows=333, hidden=512, width=1408, act="gelu",
             bias=True, out="bf16", params="bf16"),
        # The gradients of a training batch through a shared expert's first half.
        dict(name="dense_backward_train", op="dense", backward=True, rows=8192, hidden=4096, width=2048, act="swiglu",
             bias=True, out="bf16", params="fp32"),
    ]


ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _eights(rng, lo, hi):
    return max(8, _log(rng, lo, hi) // 8 * 8)


def draw(rng):
    op = rng.choice(["balance", "norm", "dense"])
    backward = rng.random() < 0.5
    if op == "balance":
        experts = _log(rng, 8, 512)
        case = dict(op=op, backward=backward, tokens=_log(rng, 1, 65536 * 256 // max(256, experts)), experts=experts,
                    topk=rng.randint(1, min(10, experts)), sequences=rng.choice([1, 1, _log(rng, 2, 64)]),
                    score=rng.choice(["softmax", "sigmoid"]), dtype=rng.choice(["fp32", "bf16"]),
                    masked=rng.choice([0.0, 0.0, 0.1]))
        if backward:
            case["add"] = rng.random() < 0.5
        return case
    if op == "norm":
        hidden = _eights(rng, 64, 16384) if rng.random() < 0.8 else _log(rng, 33, 8191) | 1
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        most = 8192 * 7168 // (2 if dtype == "fp32" else 1) // (1 if hidden % 8 == 0 else 4)
        case = dict(op=op, backward=backward, rows=_log(rng, 1, min(65536, most // hidden)), hidden=hidden, dtype=dtype,
                    params=rng.choice(["bf16", "fp32"]))
        if backward:
            case["add"] = rng.random() < 0.5
        return case
    while True:
        act = rng.choice(ACTS)
        case = dict(op=op, backward=backward, rows=_log(rng, 1, 8192), hidden=_eights(rng, 64, 7168),
                    width=_eights(rng, 64, 7168), act=act, bias=rng.random() < 0.6,
                    out=rng.choice(["bf16", "bf16", "fp32"]), params=rng.choice(["bf16", "fp32"]))
        if not backward:
            case["residual"] = rng.random() < 0.5
        if work(case)["flops"] <= 2.7e11 and case["rows"] * case["width"] * (2 if act == "swiglu" else 1) <= 3e7:
            return case


# ------------------------------------------------------------------- inputs

def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + salt)
    return g


def _normal(g, shape, dtype=F32, std=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=F32).mul_(std).to(dtype)


def _prepare_balance(case, seed):
    g = _gen(seed, 11)
    T, E, K, S = case["tokens"], case["experts"], case["topk"], case["sequences"]
    # some experts are favoured, which is what the loss is for
    x = (_normal(g, (T, E), F32, 1.5) + _normal(g, (E,), F32, 0.5)).to(TYPES[case["dtype"]])
    if case["masked"]:
        x.masked_fill_(torch.rand(x.shape, generator=g, device=DEV) < case["masked"], -math.inf)
    value, idx = torch.sort(x.float(), dim=1, descending=True, stable=True)
    idx = torch.where(torch.isneginf(value), -1, idx)[:, :K].contiguous()
    s = {"logits": x, "topk_idx": idx, "seq_offsets": None}
    if S > 1:  # sequences of random lengths, empty ones among them when there are few tokens; padding behind the last
        used = T - T // 32
        cuts = torch.sort(torch.randint(0, used + 1, (S - 1,), generator=g, device=DEV))[0]
        s["seq_offsets"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), used)]).to(I32)
    if case["backward"]:
        s["grad_losses"] = torch.rand(2, generator=g, device=DEV) * 0.01 + 0.001
        s["add"] = _normal(g, (T, E), x.dtype, 0.01 / T) if case["add"] else None
        s.update(_losses(case, s))  # what the forward pass gave
    return s


def _prepare_norm(case, seed):
    g = _gen(seed, 12)
    T, H, dtype, params = case["rows"], case["hidden"], TYPES[case["dtype"]], TYPES[case["params"]]
    # rows of a residual stream: channels of different sizes, a mean of their own
    size = torch.exp(_normal(g, (H,), F32, 0.5))
    x = (_normal(g, (T, H)) * size + _normal(g, (T, 1), F32, 0.5)).to(dtype)
    s = {"x": x, "weight": (1.0 + _normal(g, (H,), F32, 0.2)).to(params), "bias": _normal(g, (H,), params, 0.1)}
    if case["backward"]:
        s["grad"] = _normal(g, (T, H), dtype)
        s["add"] = _normal(g, (T, H), dtype) if case["add"] else None
        s["mean"], s["rstd"] = _statistics(x.float())
    else:
        s["mean"], s["rstd"] = torch.zeros(T, device=DEV), torch.zeros(T, device=DEV)
    return s


def _prepare_dense(case, seed):
    g = _gen(seed, 13)
    T, H, W = case["rows"], case["hidden"], case["width"]
    N = 2 * W if case["act"] == "swiglu" else W
    s = {"x": _normal(g, (T, H), BF16), "w": _normal(g, (N, H), BF16, 1.0 / math.sqrt(H)),
         "bias": _normal(g, (N,), TYPES[case["params"]], 0.5) if case["bias"] else None}
    if case["backward"]:
        s["grad"] = _normal(g, (T, W), TYPES[case["out"]])
        s["preact"] = None
        if case["act"] != "none":  # what the forward pass kept
            z = s["x"].float() @ s["w"].float().T
            s["preact"] = (z if s["bias"] is None else z + s["bias"].float()).to(BF16)
    else:
        s["residual"] = _normal(g, (T, W), BF16) if case["residual"] else None
    return s


def prepare(case, seed):
    s = {"balance": _prepare_balance, "norm": _prepare_norm, "dense": _prepare_dense}[case["op"]](case, seed)
    s["case"] = case
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    return (_own if own else _plain)[case["op"], case["backward"]](state)


# The plain forms: 32 bits, rounded once at the end.

def _scores(case, x):
    """(the scores that are averaged, the softmax, its log of the sum), a masked expert's at 0; a row without
    experts counts as zeros."""
    top = x.amax(1, keepdim=True)
    top = torch.where(torch.isneginf(top), 0.0, top)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    soft = torch.where(total > 0, e / total, 0.0)
    lse = torch.where(total > 0, torch.log(total) + top, 0.0)
    if case["score"] == "softmax":
        return soft, soft, lse
    s = 1.0 / (1.0 + torch.exp(-x))
    total = s.sum(1, keepdim=True)
    return torch.where(total > 0, s / total, 0.0), soft, lse


def _segments(s):
    """The sequences' borders, each token's sequence (none: their number) and the sequences' lengths."""
    T = s["logits"].shape[0]
    off = s["seq_offsets"]
    off = torch.tensor([0, T], device=DEV) if off is None else off.to(I64)
    t = torch.arange(T, device=DEV)
    of = (t[:, None] >= off[None, 1:]).sum(1)
    return off, of, off[1:] - off[:-1]


def _losses(case, s):
    off, of, lengths = _segments(s)
    S, E = lengths.shape[0], case["experts"]
    p, _, lse = _scores(case, s["logits"].float())
    inside = of < S
    idx = s["topk_idx"]
    flat = torch.where(idx >= 0, of[:, None] * E + idx, (S + 1) * E)
    counts = torch.zeros((S + 1) * E + 1, dtype=I64, device=DEV).scatter_add_(0, flat.reshape(-1), torch.ones_like(flat).reshape(-1))
    counts = counts[:S * E].view(S, E)
    # the sums run in 64 bits: a batch has many tokens
    probs = torch.zeros((S + 1, E), dtype=F64, device=DEV).index_add_(0, of, p.to(F64))[:S]
    probs = probs / lengths.clamp_min(1)[:, None]
    chosen, full = counts.sum(1, keepdim=True), (lengths > 0).sum()
    share = torch.where(chosen > 0, counts.to(F64) / chosen.clamp_min(1), 0.0) * E / full.clamp_min(1)
    z = (lse[:, 0].to(F64) ** 2 * inside).sum() / inside.sum().clamp_min(1)
    return {"losses": torch.stack([(share * probs).sum(), z]).float(), "counts": counts.to(I32), "probs": probs.float(),
            "slopes": (share / lengths.clamp_min(1)[:, None]).float()}


def _plain_balance(s):
    return _losses(s["case"], s)


def _plain_balance_backward(s):
    case = s["case"]
    off, of, lengths = _segments(s)
    x = s["logits"].float()
    p, soft, lse = _scores(case, x)
    inside = (of < lengths.shape[0])[:, None]
    slope = torch.cat([s["slopes"], torch.zeros_like(s["slopes"][:1])])[of] * s["grad_losses"][0]
    d = p * (slope - (p * slope).sum(1, keepdim=True))
    if case["score"] == "sigmoid":
        d = d * (1.0 / (1.0 + torch.exp(x)))
    d = d + s["grad_losses"][1] * 2.0 / inside.sum().clamp_min(1) * lse * soft
    d = torch.where(inside, d, 0.0)
    if s["add"] is not None:
        d = s["add"].float() + d
    return {"grad_logits": d.to(s["logits"].dtype)}


def _statistics(x):
    mean = x.mean(1)
    return mean, 1.0 / torch.sqrt(((x - mean[:, None]) ** 2).mean(1) + EPS)


def _plain_norm(s):
    x = s["x"].float()
    mean, rstd = _statistics(x)
    y = (x - mean[:, None]) * rstd[:, None] * s["weight"].float() + s["bias"].float()
    return {"out": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_norm_backward(s):
    x, g = s["x"].float(), s["grad"].float()
    n = (x - s["mean"][:, None]) * s["rstd"][:, None]
    gw = g * s["weight"].float()
    d = (gw - gw.mean(1, keepdim=True) - n * (gw * n).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["add"] is not None:
        d = d + s["add"].float()
    # long sums over the rows, in 64 bits
    return {"grad_x": d.to(s["x"].dtype), "grad_weight": (g * n).sum(0, dtype=F64).to(s["weight"].dtype),
            "grad_bias": g.sum(0, dtype=F64).to(s["bias"].dtype)}


def _activate(act, z):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "swiglu":
        gate, up = z.chunk(2, dim=1)
        return gate / (1.0 + torch.exp(-gate)) * up
    return z


def _activate_backward(act, z, g):
    if act == "relu":
        return torch.where(z > 0, g, 0.0)
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-z))
        return g * sig * (1.0 + z * (1.0 - sig))
    if act == "gelu":
        return g * (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return g * (0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z))
    if act == "swiglu":
        gate, up = z.chunk(2, dim=1)
        sig = 1.0 / (1.0 + torch.exp(-gate))
        return torch.cat([g * up * sig * (1.0 + gate * (1.0 - sig)), g * gate * sig], 1)
    return g


def _plain_dense(s):
    case = s["case"]
    z = s["x"].float() @ s["w"].float().T
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _activate(case["act"], z)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"out": y.to(TYPES[case["out"]])}


def _plain_dense_backward(s):
    case = s["case"]
    z = None if s["preact"] is None else s["preact"].float()
    d = _activate_backward(case["act"], z, s["grad"].float())
    out = {"grad_x": (d @ s["w"].float()).to(BF16), "grad_w": (d.T @ s["x"].float()).to(BF16)}
    if s["bias"] is not None:
        out["grad_bias"] = d.sum(0, dtype=F64).to(s["bias"].dtype)
    return out


_plain = {("balance", False): _plain_balance, ("balance", True): _plain_balance_backward,
          ("norm", False): _plain_norm, ("norm", True): _plain_norm_backward,
          ("dense", False): _plain_dense, ("dense", True): _plain_dense_backward}


# The package's calls.

def _own_balance(s):
    import combine_ep_get_layout_gb300 as ep
    b = ep.ep_balance_loss(s["logits"], s["topk_idx"], score=s["case"]["score"], seq_offsets=s["seq_offsets"])
    return {"losses": b.losses, "counts": b.counts, "probs": b.probs, "slopes": b.slopes}


def _own_balance_backward(s):
    import combine_ep_get_layout_gb300 as ep
    b = ep.Balance(s["losses"], s["counts"], s["probs"], s["slopes"])
    g = ep.ep_balance_loss_backward(s["grad_losses"], s["logits"], b, score=s["case"]["score"],
                                    seq_offsets=s["seq_offsets"], add=s["add"])
    return {"grad_logits": g}


def _own_norm(s):
    import combine_ep_get_layout_gb300 as ep
    y = ep.ep_layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, mean=s["mean"], rstd=s["rstd"])
    return {"out": y, "mean": s["mean"], "rstd": s["rstd"]}


def _own_norm_backward(s):
    import combine_ep_get_layout_gb300 as ep
    d, w, b = ep.ep_layer_norm_backward(s["grad"], s["x"], s["mean"], s["rstd"], s["weight"], add=s["add"])
    return {"grad_x": d, "grad_weight": w, "grad_bias": b}


def _act(case):
    return None if case["act"] == "none" else case["act"]


def _own_dense(s):
    import combine_ep_get_layout_gb300 as ep
    c = s["case"]
    return {"out": ep.ep_dense_product(s["x"], s["w"], s["bias"], activation=_act(c), residual=s["residual"],
                                       out_dtype=TYPES[c["out"]])}


def _own_dense_backward(s):
    import combine_ep_get_layout_gb300 as ep
    c = s["case"]
    d, w, b = ep.ep_dense_product_backward(s["grad"], s["x"], s["w"], activation=_act(c), preact=s["preact"],
                                           bias_dtype=None if s["bias"] is None else s["bias"].dtype)
    out = {"grad_x": d, "grad_w": w}
    if b is not None:
        out["grad_bias"] = b
    return out


_own = {("balance", False): _own_balance, ("balance", True): _own_balance_backward,
        ("norm", False): _own_norm, ("norm", True): _own_norm_backward,
        ("dense", False): _own_dense, ("dense", True): _own_dense_backward}


# --------------------------------------------------------- what a pass needs

SIZE = {"bf16": 2, "fp32": 4}


def work(case):
    if case["op"] == "balance":
        n, k, se = case["tokens"] * case["experts"], case["tokens"] * case["topk"], case["sequences"] * case["experts"]
        size = SIZE[case["dtype"]]
        if case["backward"]:
            return {"bytes": n * size * (3 if case["add"] else 2) + 4 * se, "flops": 10.0 * n}
        return {"bytes": n * size + 8 * k + 12 * se, "flops": 6.0 * n}
    if case["op"] == "norm":
        T, H, size = case["rows"], case["hidden"], SIZE[case["dtype"]]
        params = H * SIZE[case["params"]]
        if case["backward"]:
            return {"bytes": T * H * size * (4 if case["add"] else 3) + 8 * T + 3 * params, "flops": 14.0 * T * H}
        return {"bytes": 2 * T * H * size + 8 * T + 2 * params, "flops": 8.0 * T * H}
    T, H, W = case["rows"], case["hidden"], case["width"]
    N = 2 * W if case["act"] == "swiglu" else W
    bias = N * SIZE[case["params"]] if case["bias"] else 0
    if case["backward"]:
        kept = 0 if case["act"] == "none" else T * N * 2
        return {"bytes": 4 * T * H + 4 * N * H + T * W * SIZE[case["out"]] + kept + bias, "flops": 4.0 * T * H * N}
    rest = T * W * (SIZE[case["out"]] + (2 if case["residual"] else 0))
    return {"bytes": 2 * (T * H + N * H) + rest + bias, "flops": 2.0 * T * H * N}


# ----------------------------------------------- the definitions in 64 bits

def _exact_balance(case, s, logits):
    """The losses as functions of the logits, one sequence after the other."""
    T, E = logits.shape
    off = [0, T] if s["seq_offsets"] is None else s["seq_offsets"].tolist()
    dead = torch.isneginf(s["logits"]).all(1)
    soft = torch.softmax(logits, 1) if case["score"] == "softmax" else torch.sigmoid(logits)
    if case["score"] == "sigmoid":
        soft = soft / torch.where(dead, 1.0, soft.sum(1))[:, None]
    soft = torch.where(dead[:, None], 0.0, soft)
    z = torch.where(dead, 0.0, torch.logsumexp(logits, 1)) ** 2
    full = sum(b > a for a, b in zip(off, off[1:]))
    balance, counts, probs, slopes = 0.0, [], [], []
    for a, b in zip(off, off[1:]):
        chosen = s["topk_idx"][a:b].reshape(-1)
        chosen = chosen[chosen >= 0]
        n = torch.bincount(chosen, minlength=E)
        mean = soft[a:b].sum(0) / max(1, b - a)
        share = n.to(F64) / max(1, chosen.numel()) * E
        balance = balance + (share * mean).sum() / max(1, full)
        counts.append(n.to(I32))
        probs.append(mean)
        slopes.append(share / max(1, full) / max(1, b - a))
    z = z[off[0]:off[-1]].sum() / max(1, off[-1] - off[0])
    return balance, z, {"counts": torch.stack(counts), "probs": torch.stack(probs), "slopes": torch.stack(slopes)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "balance":
        if not case["backward"]:
            b, z, rest = _exact_balance(case, s, s["logits"].to(F64))
            return {"losses": torch.stack([b, z]), **rest}
        # by torch's own differentiation of the definition; a row without experts has no gradient
        x = torch.where(torch.isneginf(s["logits"]).all(1, keepdim=True), 0.0, s["logits"].to(F64)).requires_grad_(True)
        b, z, _ = _exact_balance(case, s, x)
        d, = torch.autograd.grad(s["grad_losses"][0].to(F64) * b + s["grad_losses"][1].to(F64) * z, x)
        d = d.nan_to_num(0.0)
        return {"grad_logits": d if s["add"] is None else d + s["add"].to(F64)}
    if case["op"] == "norm":
        x = s["x"].to(F64)
        if not case["backward"]:
            var, mean = torch.var_mean(x, 1, correction=0)
            rstd = (var + EPS).rsqrt()
            y = torch.addcmul(s["bias"].to(F64), (x - mean[:, None]) * rstd[:, None], s["weight"].to(F64))
            return {"out": y, "mean": mean, "rstd": rstd}
        # with the statistics that the forward pass kept
        g, w = s["grad"].to(F64), s["weight"].to(F64)
        mean, rstd = s["mean"].to(F64)[:, None], s["rstd"].to(F64)[:, None]
        n = (x - mean) * rstd
        H = x.shape[1]
        dn = g * w
        d = rstd / H * (H * dn - dn.sum(1, keepdim=True) - n * (dn * n).sum(1, keepdim=True))
        return {"grad_x": d if s["add"] is None else d + s["add"].to(F64), "grad_weight": (g * n).sum(0), "grad_bias": g.sum(0)}
    F = torch.nn.functional
    acts = {"none": lambda z: z, "relu": F.relu, "silu": F.silu, "gelu": F.gelu,
            "gelu_tanh": lambda z: F.gelu(z, approximate="tanh"),
            "swiglu": lambda z: F.silu(z[:, :case["width"]]) * z[:, case["width"]:]}
    x, w = s["x"].to(F64), s["w"].to(F64)
    if not case["backward"]:
        z = x @ w.T if s["bias"] is None else torch.addmm(s["bias"].to(F64), x, w.T)
        y = acts[case["act"]](z)
        return {"out": y if s["residual"] is None else y + s["residual"].to(F64)}
    d = s["grad"].to(F64)
    if case["act"] != "none":
        z = s["preact"].to(F64).requires_grad_(True)
        d, = torch.autograd.grad(acts[case["act"]](z), z, d)
    out = {"grad_x": d @ w, "grad_w": d.T @ x}
    if s["bias"] is not None:
        out["grad_bias"] = d.sum(0)
    return out
