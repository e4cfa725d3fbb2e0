"""The operators around an MoE block's experts, as cases that can be timed and compared.

* ``norm`` / ``norm_backward``: what leaves a block scaled, gated, normalised and added to the
  residual stream, and the stream normalised for the next block, in one pass; and its gradients;
* ``balance``: per-expert counts, mean probabilities, the balance loss and the z-loss of a
  router's logits, over one batch or over the ragged sequences of it;
* ``route_backward``: the gradient of router weights and of both losses with respect to the logits;
* ``mm`` / ``moe_mm``: products of FP8 rows with FP8 weights (128 x 128 block scales) that end in a
  bias, an activation, a scale and a residual.

``run`` computes them in a plain form (elementary torch operations) or, where ``own``
is true, through this repository's package.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
BLOCK = 128           # values that share an activation scale; rows and columns that share a weight scale
E4M3_MAX = 448.0
EPS = 1e-6


def listed():
    return [
        # one token of a decode step: the MoE layer's fp32 output into the fp16 stream, and the next block's norm
        {"name": "norm_decode", "op": "norm", "tokens": 1, "hidden": 4096, "y": "f32", "h": "f16", "x": "f16",
         "gain": "f16", "post": False, "gate": "none", "sigmoid": False, "scale": 1.0, "residual_scale": 1.0},
        # a prompt of 2048 tokens: the block's output is normalised too and scaled per channel
        {"name": "norm_prefill", "op": "norm", "tokens": 2048, "hidden": 4096, "y": "bf16", "h": "bf16", "x": "bf16",
         "gain": "bf16", "post": True, "gate": "channel", "sigmoid": False, "scale": 1.0, "residual_scale": 1.0},
        # the gradients of the same pass in training
        {"name": "norm_backward", "op": "norm_backward", "tokens": 2048, "hidden": 4096, "y": "bf16", "h": "bf16",
         "x": "bf16", "gain": "bf16", "post": True, "gate": "channel", "sigmoid": False, "scale": 1.0,
         "residual_scale": 1.0},
        # an odd batch with the stream in fp32 and a sigmoid gate per value
        {"name": "norm_backward_gated", "op": "norm_backward", "tokens": 2047, "hidden": 2048, "y": "bf16", "h": "f32",
         "x": "bf16", "gain": "f32", "post": False, "gate": "full", "sigmoid": True, "scale": 0.5,
         "residual_scale": 1.0},
        # one short sequence, 128 experts: latency counts
        {"name": "balance_short", "op": "balance", "tokens": 129, "experts": 128, "topk": 8, "sequences": 0,
         "scoring": "softmax", "bias": True},
        # a training batch of ragged sequences, score routing over 256 experts
        {"name": "balance_sequences", "op": "balance", "tokens": 16384, "experts": 256, "topk": 6, "sequences": 9,
         "scoring": "sqrtsoftplus", "bias": False},
        # the gradient of the router weights of a small batch
        {"name": "route_backward_short", "op": "route_backward", "tokens": 129, "experts": 128, "topk": 8,
         "sequences": 0, "scoring": "softmax", "bias": True, "losses": False, "out": "f32", "scale": 1.0},
        # a training batch: router weights, balance loss over ragged sequences and z-loss in one gradient
        {"name": "route_backward_train", "op": "route_backward", "tokens": 16384, "experts": 256, "topk": 6,
         "sequences": 9, "scoring": "softmax_then_bias", "bias": False, "losses": True, "out": "f32", "scale": 1.0},
        # one token through a dense 4096 x 4096 projection into the residual stream: bound by reading the weight
        {"name": "mm_residual_decode", "op": "mm", "out": "f16", "m": 1, "n": 4096, "k": 4096, "act": "none",
         "bias": True, "residual": True, "scale": 1.0},
        # a prompt through the first projection of an ungated feed-forward block
        {"name": "mm_gelu_prefill", "op": "mm", "out": "bf16", "m": 2048, "n": 4096, "k": 4096, "act": "gelu",
         "bias": True, "residual": False, "scale": 1.0},
        # experts with biases: the fused gate and up projections of a decode batch
        {"name": "moe_mm_bias_decode", "op": "moe_mm", "out": "bf16", "tokens": 32, "experts": 128, "topk": 8,
         "n": 1536, "k": 2048, "act": "swiglu", "bias": True, "residual": False, "scale": 1.0},
        # ... and the down projections of a ragged prefill batch, about 128 rows an expert, with a residual per row
        {"name": "moe_mm_residual_prefill", "op": "moe_mm", "out": "bf16", "tokens": 2047, "experts": 128, "topk": 8,
         "n": 2048, "k": 768, "act": "none", "bias": True, "residual": True, "scale": 0.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_once(rng):
    op = rng.choice(["norm", "norm_backward", "norm", "norm_backward", "balance", "route_backward", "mm", "moe_mm"])
    if op in ("norm", "norm_backward"):
        y, h, x = rng.choice([("f16",) * 3, ("bf16",) * 3, ("f32",) * 3, ("f32", "f16", "f16"), ("bf16", "f32", "bf16"),
                              ("f16", "f32", "f16"), ("f32", "bf16", "f32")])
        gate = rng.choice(["none", "token", "channel", "full"])
        return {"op": op, "tokens": _log(rng, 1, 8192), "hidden": 8 * _log(rng, 16, 1024), "y": y, "h": h, "x": x,
                "gain": rng.choice([x, "f32"]), "post": rng.random() < 0.5, "gate": gate,
                "sigmoid": gate != "none" and rng.random() < 0.5, "scale": rng.choice([1.0, 0.5, 0.22]),
                "residual_scale": rng.choice([1.0, 1.0, 1.5])}
    if op in ("balance", "route_backward"):
        experts = _log(rng, 8, 1024)
        scoring = rng.choice(["softmax", "softmax_then_bias", "sqrtsoftplus"])
        c = {"op": op, "tokens": _log(rng, 1, 16384), "experts": experts, "topk": rng.randint(1, 8),
             "sequences": rng.choice([0, 0, 1, 3, 17, 64]), "scoring": scoring, "bias": rng.random() < 0.5}
        if op == "route_backward":
            c.update(losses=rng.random() < 0.7, out=rng.choice(["f32", "f32", "bf16", "f16"]),
                     scale=rng.choice([1.0, 2.5]) if scoring == "sqrtsoftplus" else 1.0)
        return c
    out = rng.choice(["f16", "bf16", "f32"])
    act = rng.choice(["none", "swiglu", "silu", "gelu", "gelu_tanh", "relu", "relu2"])
    n = 256 * rng.randint(1, 16) if act == "swiglu" else _log(rng, 128, 4096)
    c = {"op": op, "out": out, "n": n, "act": act, "bias": rng.random() < 0.7, "residual": rng.random() < 0.5,
         "scale": rng.choice([1.0, 0.5])}
    if op == "mm":
        return dict(c, m=_log(rng, 1, 2048), k=16 * _log(rng, 16, 256))
    return dict(c, tokens=_log(rng, 1, 2048), experts=_log(rng, 8, 128), topk=rng.randint(1, 8),
                k=16 * _log(rng, 16, 128))


def draw(rng):
    most = {}
    for c in listed():
        for key, v in work(c).items():
            most[c["op"], key] = max(most.get((c["op"], key), 0), v)
    while True:
        c = _draw_once(rng)
        if all(v <= most[c["op"], key] for key, v in work(c).items()):
            return c


# ---------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rows(g, shape):
    """Activations: normal values over channels of unequal size, as hidden states have them."""
    return _randn(g, *shape) * torch.exp(0.7 * _randn(g, shape[-1]))


def _fp8_rows(g, rows, k):
    """FP8 activation rows [rows, k] and their scales [rows, ceil(k / 128)]."""
    kb = -(-k // BLOCK)
    x = torch.zeros(rows, kb * BLOCK, device="cuda")
    x[:, :k] = _rows(g, (rows, k))
    x = x.view(rows, kb, BLOCK)
    scales = (x.abs().amax(-1) / E4M3_MAX).clamp(min=2.0 ** -126)
    q = (x / scales[..., None]).to(torch.float8_e4m3fn).view(rows, kb * BLOCK)
    return q[:, :k].contiguous(), scales.contiguous()


def _fp8_weight(g, mats, n, k):
    """FP8 weights [mats, n, k] and their scales [mats, ceil(n / 128), ceil(k / 128)]."""
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    w = torch.empty(mats, n, k, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(mats, nb, kb, device="cuda")
    step = max(1, (1 << 28) // (nb * kb * BLOCK * BLOCK))
    for e in range(0, mats, step):
        c = min(step, mats - e)
        v = _randn(g, c, nb, BLOCK, kb, BLOCK)
        v *= torch.exp(0.3 * _randn(g, c, nb, 1, kb, 1)) / math.sqrt(k)
        s = v.abs().amax((2, 4)) / E4M3_MAX
        q = (v / s[:, :, None, :, None]).to(torch.float8_e4m3fn).view(c, nb * BLOCK, kb * BLOCK)
        w[e:e + c] = q[:, :n, :k]
        scales[e:e + c] = s
    return w, scales


def _scores(logits, bias, scoring):
    """What a router selects by, for making ids: largest first."""
    if scoring == "softmax":
        return logits if bias is None else logits + bias
    s = torch.softmax(logits, 1) if scoring == "softmax_then_bias" else torch.sqrt(torch.log1p(torch.exp(logits)))
    return s if bias is None else s + bias


def _sequence_offsets(g, tokens, sequences):
    """Ragged lengths that add up to the tokens; one of many is empty, and a few rows at the end belong to none."""
    cuts = torch.sort(torch.randint(0, tokens + 1, (sequences - 1,), generator=g, device="cuda")).values
    if sequences > 4:
        cuts[2] = cuts[1]
    end = tokens - (tokens // 50 if sequences > 1 else 0)
    o = torch.zeros(sequences + 1, dtype=torch.int32, device="cuda")
    o[1:sequences] = cuts.clamp(max=end).int()
    o[sequences] = end
    return o


def _norm_inputs(g, case):
    t, h = case["tokens"], case["hidden"]
    gd = DTYPES[case["gain"]]
    s = {"y": _rows(g, (t, h)).to(DTYPES[case["y"]]), "h": (2 * _rows(g, (t, h))).to(DTYPES[case["h"]]),
         "gain": (1 + 0.1 * _randn(g, h)).to(gd), "gate": None,
         "post_gain": (1 + 0.1 * _randn(g, h)).to(gd) if case["post"] else None}
    # per value in the rows' own type; per channel with the gains; per token as a projection of 32 bits leaves it
    shape, dt = {"none": (None, None), "token": ((t, 1), torch.float32), "channel": ((h,), gd),
                 "full": ((t, h), DTYPES[case["y"]])}[case["gate"]]
    if shape:
        s["gate"] = _randn(g, *shape).to(dt)
    return s


def _norm_args(s):
    c = s["case"]
    return {"gain": s["gain"], "post_gain": s["post_gain"], "gate": s["gate"], "gate_sigmoid": c["sigmoid"],
            "scale": c["scale"], "residual_scale": c["residual_scale"], "eps": EPS}


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op in ("norm", "norm_backward"):
        t, h = case["tokens"], case["hidden"]
        s.update(_norm_inputs(g, case))
        if op == "norm":
            s["h_out"] = torch.empty_like(s["h"])
            s["x"] = torch.empty(t, h, dtype=DTYPES[case["x"]], device="cuda")
            return s
        s["h_out"] = s.pop("h")                      # the backward pass reads the stream behind the block
        s["dh_out"] = _rows(g, (t, h)).to(s["h_out"].dtype)
        s["dx"] = _rows(g, (t, h)).to(DTYPES[case["x"]])
        s["dy"], s["dh"] = torch.empty_like(s["y"]), torch.empty_like(s["h_out"])
        s["dgain"] = torch.empty(h, device="cuda")
        s["dpost_gain"] = torch.empty(h, device="cuda") if case["post"] else None
        s["dgate"] = None
        if s["gate"] is not None:
            s["dgate"] = torch.empty_like(s["gate"], dtype=s["gate"].dtype if case["gate"] == "full" else torch.float32)
        if own:
            import block_quantized_moe_gather_gb300 as bq
            s["workspace"] = torch.empty(bq.residual_norm_backward_workspace_bytes(t, h), dtype=torch.uint8,
                                         device="cuda")
        return s
    if op in ("balance", "route_backward"):
        t, e, k = case["tokens"], case["experts"], case["topk"]
        popular = 0.5 * _randn(g, e)                 # some experts are liked by every token
        s["logits"] = 1.5 * _randn(g, t, e) + popular
        s["bias"] = 0.2 * _randn(g, e) if case["bias"] else None
        s["ids"] = torch.topk(_scores(s["logits"], s["bias"], case["scoring"]), k, 1).indices.int().contiguous()
        s["offsets"] = _sequence_offsets(g, t, case["sequences"]) if case["sequences"] else None
        groups = max(1, case["sequences"])
        s["counts"] = torch.zeros(groups, e, dtype=torch.int32, device="cuda")
        if op == "balance":
            s["probs"], s["losses"] = torch.empty(groups, e, device="cuda"), torch.empty(2, device="cuda")
            if own:
                import block_quantized_moe_gather_gb300 as bq
                s["workspace"] = torch.empty(bq.moe_balance_workspace_bytes(t, e, groups), dtype=torch.uint8,
                                             device="cuda")
            return s
        s["counts"] = _counts(s)
        s["dweights"] = _randn(g, t, k)
        s["dlosses"] = torch.tensor([30.0, 3.0], device="cuda") * (1 + 0.1 * _randn(g, 2)) if case["losses"] else None
        s["dlogits"] = torch.zeros(t, e, dtype=DTYPES[case["out"]], device="cuda")
        s["dbias"] = torch.empty(e, device="cuda") if _bias_learns(case) else None
        if own:
            import block_quantized_moe_gather_gb300 as bq
            s["workspace"] = torch.empty(bq.moe_route_backward_workspace_bytes(t, e), dtype=torch.uint8, device="cuda")
        return s
    n, k = case["n"], case["k"]
    cols = n // 2 if case["act"] == "swiglu" else n
    rows = case["m"] if op == "mm" else case["tokens"] * case["topk"]
    mats = 1 if op == "mm" else case["experts"]
    s["x"], s["xs"] = _fp8_rows(g, rows, k)
    s["w"], s["ws"] = _fp8_weight(g, mats, n, k)
    s["bias"] = 0.5 * _randn(g, mats, n) if case["bias"] else None
    s["residual"] = (2 * _rows(g, (rows, cols))).to(DTYPES[case["out"]]) if case["residual"] else None
    s["out"] = torch.empty(rows, cols, dtype=DTYPES[case["out"]], device="cuda")
    if op == "mm":
        s["w"], s["ws"], s["bias"] = s["w"][0], s["ws"][0], s["bias"][0] if case["bias"] else None
        return s
    ids = torch.topk(_randn(g, case["tokens"], mats), min(case["topk"], mats), 1).indices.reshape(-1)
    counts = torch.bincount(ids, minlength=mats)
    s["offsets"] = torch.zeros(mats + 1, dtype=torch.int32, device="cuda")
    s["offsets"][1:] = torch.cumsum(counts, 0)
    # what a program that pads the experts to the longest of them keeps: the experts that have rows, each
    # sorted row's place among them, and the longest expert's length
    s["active"] = torch.nonzero(counts).view(-1)
    slot = torch.cumsum((counts > 0).long(), 0) - 1
    s["row_slot"] = slot[torch.sort(ids).values]
    s["row_pos"] = torch.arange(rows, device="cuda") - s["offsets"][s["active"]].long()[s["row_slot"]]
    s["longest"] = int(counts.max())
    return s


# ---------------------------------------------------------------- plain forms
def _bias_learns(case):
    """A bias that is added to the logits is part of the weights; one that is added to scores only selects."""
    return case["bias"] and case["scoring"] == "softmax"


def _inverse_rms(v):
    return torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)


def _gate_of(s):
    if s["gate"] is None:
        return None
    g = s["gate"].float()
    return 1 / (1 + torch.exp(-g)) if s["case"]["sigmoid"] else g


def _plain_norm(s):
    c = s["case"]
    b = s["y"].float()
    if c["post"]:
        b = b * _inverse_rms(b) * s["post_gain"].float()
    g = _gate_of(s)
    if g is not None:
        b = b * g
    h = c["residual_scale"] * s["h"].float() + c["scale"] * b
    x = h * _inverse_rms(h) * s["gain"].float()
    return h.to(s["h"].dtype), x.to(s["x"].dtype)


def _norm_gradient(v, r, gain, d):
    """Gradient of gain * v * r, r = 1 / rms(v), with respect to v."""
    d = d * gain
    return r * d - v * (r * r * r * (d * v).mean(-1, keepdim=True))


def _plain_norm_backward(s):
    c = s["case"]
    y, h, dx = s["y"].float(), s["h_out"].float(), s["dx"].float()
    r = _inverse_rms(h)
    dgain = (dx * h * r).sum(0)
    dh = s["dh_out"].float() + _norm_gradient(h, r, s["gain"].float(), dx)
    b, ry, post = y, None, None
    if c["post"]:
        ry, post = _inverse_rms(y), s["post_gain"].float()
        b = y * ry * post
    g, dgate, db = _gate_of(s), None, c["scale"] * dh
    if g is not None:
        dgate = db * b
        if c["sigmoid"]:
            dgate = dgate * g * (1 - g)
        if c["gate"] != "full":
            dgate = dgate.sum(1, keepdim=True) if c["gate"] == "token" else dgate.sum(0)
        dgate = dgate.to(s["dgate"].dtype)
        db = db * g
    dpost = None
    if c["post"]:
        dpost = (db * y * ry).sum(0)
        db = _norm_gradient(y, ry, post, db)
    return db.to(s["y"].dtype), (c["residual_scale"] * dh).to(s["h_out"].dtype), dgain, dpost, dgate


def _sequence_of_rows(s):
    """Each row's sequence, and whether it has one."""
    t = s["logits"].shape[0]
    if s["offsets"] is None:
        return torch.zeros(t, dtype=torch.long, device="cuda"), torch.ones(t, dtype=torch.bool, device="cuda")
    row = torch.arange(t, device="cuda")
    o = s["offsets"].long()
    at = (row[:, None] >= o[None, 1:]).sum(1)
    return at.clamp(max=o.numel() - 2), (row >= o[0]) & (row < o[-1])


def _counts(s):
    at, valid = _sequence_of_rows(s)
    groups, e = s["counts"].shape
    pairs = (at[:, None] * e + s["ids"].long())[valid].reshape(-1)
    return torch.bincount(pairs, minlength=groups * e).view(groups, e).int()


def _lengths(s):
    if s["offsets"] is None:
        return torch.full((1,), float(s["logits"].shape[0]), device="cuda")
    return (s["offsets"][1:] - s["offsets"][:-1]).float()


def _logits_and_probabilities(s):
    z = s["logits"]
    if _bias_learns(s["case"]):
        z = z + s["bias"]
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    if s["case"]["scoring"] != "sqrtsoftplus":
        return z, lse, e / total, e / total, None, None
    score = torch.sqrt(z.clamp(min=0) + torch.log1p(torch.exp(-z.abs())))
    slope = 0.5 / (1 + torch.exp(-z)) / score        # d score / d logit
    whole = score.sum(1, keepdim=True)
    return z, lse, e / total, score / whole, slope, whole


def _plain_balance(s):
    at, valid = _sequence_of_rows(s)
    z, lse, _, p, _, _ = _logits_and_probabilities(s)
    n = _lengths(s)
    counts = _counts(s)
    probs = torch.zeros(counts.shape, device="cuda")
    probs.index_add_(0, at[valid], p[valid])
    probs = probs / n.clamp(min=1)[:, None]
    share = counts.float() * (counts.shape[1] / s["case"]["topk"]) / n.clamp(min=1)[:, None]
    balance = (share * probs).sum() / (n > 0).sum().clamp(min=1)
    square = (lse * lse)[valid].sum() / n.sum().clamp(min=1)
    return counts, probs, torch.stack([balance, square])


def _plain_route_backward(s):
    c = s["case"]
    at, valid = _sequence_of_rows(s)
    z, lse, soft, p, slope, whole = _logits_and_probabilities(s)
    d = torch.zeros_like(z)
    ids, dw = s["ids"].long(), s["dweights"]
    if c["scoring"] == "sqrtsoftplus":
        d.scatter_(1, ids, dw * c["scale"] * slope.gather(1, ids))
    else:
        zs = z.gather(1, ids)
        w = torch.exp(zs - zs.amax(1, keepdim=True))
        w = w / w.sum(1, keepdim=True)
        d.scatter_(1, ids, w * (dw - (w * dw).sum(1, keepdim=True)))
    if c["losses"]:
        n = _lengths(s)
        weight = s["dlosses"][0] * (c["experts"] / c["topk"]) / (n > 0).sum().clamp(min=1) / (n * n).clamp(min=1)
        a = (s["counts"].float() * weight[:, None])[at]
        a = a - (p * a).sum(1, keepdim=True)
        d = d + (p * a if slope is None else a / whole * slope)
        d = d + soft * lse * (2 * s["dlosses"][1] / n.sum().clamp(min=1))
    d = d * valid[:, None]
    return d.to(s["dlogits"].dtype), d.sum(0) if _bias_learns(c) else None


def _grouped(x):
    """Rows in fp32 as [rows, ceil(k / 128), 128], the last group filled up with zeros."""
    rows, k = x.shape
    kb = -(-k // BLOCK)
    if kb * BLOCK == k:
        return x.float().view(rows, kb, BLOCK)
    out = torch.zeros(rows, kb * BLOCK, device=x.device)
    out[:, :k] = x.float()
    return out.view(rows, kb, BLOCK)


def _dequantised_rows(q, scales):
    rows, k = q.shape
    return (_grouped(q) * scales[..., None]).view(rows, -1)[:, :k]


def _dequantised_weight(w, scales):
    n, k = w.shape[-2:]
    return w.float() * scales.repeat_interleave(BLOCK, -1)[..., :k].repeat_interleave(BLOCK, -2)[..., :n, :]


def _activation(v, act):
    if act == "swiglu":
        gate, up = v.chunk(2, -1)
        return gate / (1 + torch.exp(-gate)) * up
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if act in ("relu", "relu2"):
        v = v.clamp(min=0)
        return v * v if act == "relu2" else v
    return v


def _plain_product(s):
    c = s["case"]
    x = _dequantised_rows(s["x"], s["xs"])
    if s["op"] == "mm":
        v = x @ _dequantised_weight(s["w"], s["ws"]).t()
        if s["bias"] is not None:
            v = v + s["bias"]
    else:
        padded = torch.zeros(s["active"].numel(), s["longest"], x.shape[1], device=x.device)
        padded[s["row_slot"], s["row_pos"]] = x
        w = _dequantised_weight(s["w"].view(torch.uint8)[s["active"]].view(torch.float8_e4m3fn), s["ws"][s["active"]])
        v = torch.bmm(padded, w.transpose(1, 2))[s["row_slot"], s["row_pos"]]
        if s["bias"] is not None:
            v = v + s["bias"][s["active"]][s["row_slot"]]
    v = c["scale"] * _activation(v, c["act"])
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(s["out"].dtype)


def run(state):
    s, op = state, state["op"]
    if not own:
        return {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "balance": _plain_balance,
                "route_backward": _plain_route_backward, "mm": _plain_product, "moe_mm": _plain_product}[op](s)
    import block_quantized_moe_gather_gb300 as bq
    c = s["case"]
    if op == "norm":
        return bq.residual_norm(s["y"], s["h"], s["h_out"], s["x"], **_norm_args(s))
    if op == "norm_backward":
        bq.residual_norm_backward(s["y"], s["h_out"], s["dh_out"], s["dx"], s["dy"], s["dh"], **_norm_args(s),
                                  dgain=s["dgain"], dpost_gain=s["dpost_gain"], dgate=s["dgate"],
                                  workspace=s["workspace"])
        return s["dy"], s["dh"], s["dgain"], s["dpost_gain"], s["dgate"]
    if op == "balance":
        bq.moe_balance_loss(s["logits"], s["ids"], s["counts"], s["probs"], s["losses"], s["workspace"],
                            bias=s["bias"] if _bias_learns(c) else None, scoring=bq.SCORING_BY_NAME[c["scoring"]],
                            seq_offsets=s["offsets"])
        return s["counts"], s["probs"], s["losses"]
    if op == "route_backward":
        bq.moe_route_backward(s["logits"], s["ids"], s["dweights"], s["dlogits"],
                              bias=s["bias"] if _bias_learns(c) else None, scoring=bq.SCORING_BY_NAME[c["scoring"]],
                              scale=c["scale"], counts=s["counts"] if c["losses"] else None, dlosses=s["dlosses"],
                              seq_offsets=s["offsets"], dbias=s["dbias"], workspace=s["workspace"])
        return s["dlogits"], s["dbias"]
    more = {"act": c["act"], "bias": s["bias"], "residual": s["residual"], "scale": c["scale"]}
    if op == "mm":
        return bq.mm_fp8_b128(s["x"], s["xs"], s["w"], s["ws"], s["out"], **more)
    return bq.moe_mm_fp8_b128(s["x"], s["xs"], s["offsets"], s["w"], s["ws"], s["out"], **more)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("norm", "norm_backward"):
        t, h = case["tokens"], case["hidden"]
        ys, hs, xs = SIZE[case["y"]], SIZE[case["h"]], SIZE[case["x"]]
        gate = {"none": 0, "token": 4 * t, "channel": SIZE[case["gain"]] * h, "full": ys * t * h}[case["gate"]]
        gains = (1 + case["post"]) * h * SIZE[case["gain"]]
        if op == "norm":
            return {"bytes": t * h * (ys + 2 * hs + xs) + gate + gains, "flops": 9 * t * h}
        dgate = gate if case["gate"] in ("none", "token", "full") else 4 * h
        return {"bytes": t * h * (2 * ys + 3 * hs + xs) + gate + dgate + gains + (1 + case["post"]) * 4 * h,
                "flops": 24 * t * h}
    if op in ("balance", "route_backward"):
        t, e, k, g = case["tokens"], case["experts"], case["topk"], max(1, case["sequences"])
        if op == "balance":
            return {"bytes": 4 * t * (e + k) + 8 * g * e, "flops": 8 * t * e}
        return {"bytes": t * e * (4 + SIZE[case["out"]]) + 8 * t * k + (4 * g * e if case["losses"] else 0),
                "flops": (14 if case["losses"] else 2) * t * e}
    n, k = case["n"], case["k"]
    cols = n // 2 if case["act"] == "swiglu" else n
    if op == "mm":
        rows, mats = case["m"], 1
    else:
        rows = case["tokens"] * case["topk"]
        # the experts that a uniform routing reaches
        mats = case["experts"] * (1 - (1 - case["topk"] / case["experts"]) ** case["tokens"])
    kb, nb = -(-k // BLOCK), -(-n // BLOCK)
    return {"bytes": int(rows * (k + 4 * kb) + mats * (n * k + 4 * nb * kb + (4 * n if case["bias"] else 0))
                         + rows * cols * SIZE[case["out"]] * (1 + case["residual"])),
            "flops": 2 * rows * n * k}


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_stream(case, y, h, post_gain, gate):
    branch = y
    if post_gain is not None:
        branch = post_gain * y / torch.sqrt(torch.mean(y ** 2, 1, keepdim=True) + EPS)
    if gate is not None:
        branch = branch * (torch.sigmoid(gate) if case["sigmoid"] else gate)
    return case["residual_scale"] * h + case["scale"] * branch


def _exact_normed(h, gain):
    return gain * h / torch.sqrt(torch.mean(h ** 2, 1, keepdim=True) + EPS)


def _exact_norm(s):
    d = {n: None if s[n] is None else s[n].double() for n in ("y", "h", "gain", "post_gain", "gate")}
    h = _exact_stream(s["case"], d["y"], d["h"], d["post_gain"], d["gate"])
    return h, _exact_normed(h, d["gain"])


def _exact_norm_backward(s):
    """By differentiation of the definition; the stream that the norm reads is an input of its own."""
    case = s["case"]
    leaf = {n: None if s[n] is None else s[n].double().requires_grad_()
            for n in ("y", "h_out", "gain", "post_gain", "gate")}
    x = _exact_normed(leaf["h_out"], leaf["gain"])
    dh, dgain = torch.autograd.grad(x, [leaf["h_out"], leaf["gain"]], s["dx"].double())
    dh = dh + s["dh_out"].double()
    before = torch.zeros_like(dh).requires_grad_()
    stream = _exact_stream(case, leaf["y"], before, leaf["post_gain"], leaf["gate"])
    wanted = [t for t in (leaf["y"], before, leaf["post_gain"], leaf["gate"]) if t is not None]
    found = dict(zip(map(id, wanted), torch.autograd.grad(stream, wanted, dh)))
    dpost, dgate = (None if leaf[n] is None else found[id(leaf[n])] for n in ("post_gain", "gate"))
    return found[id(leaf["y"])], found[id(before)], dgain, dpost, dgate


def _exact_router(s, logits, bias):
    """Per row: the probabilities of the balance loss and the squared log-sum-exp; the router's selected weights."""
    scoring = s["case"]["scoring"]
    z = logits + bias if bias is not None else logits
    lse = torch.logsumexp(z, 1)
    ids = s["ids"].long()
    if scoring == "sqrtsoftplus":
        # softplus in 64 bits, without torch's cut-off
        score = torch.sqrt(torch.logaddexp(z, torch.zeros_like(z)))
        return score / score.sum(1, keepdim=True), lse ** 2, score.gather(1, ids)
    p = torch.exp(z - lse[:, None])
    chosen = torch.exp(z.gather(1, ids) - torch.logsumexp(z.gather(1, ids), 1, keepdim=True))
    return p, lse ** 2, chosen


def _exact_ranges(s):
    t = s["logits"].shape[0]
    o = [0, t] if s["offsets"] is None else s["offsets"].tolist()
    return list(zip(o[:-1], o[1:]))


def _exact_losses(s, p, square, counts):
    """The two losses; `counts` as a list of 64-bit rows."""
    parts, rows = [], 0
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for (a, b), c in zip(_exact_ranges(s), counts):
        if a == b:
            continue
        f = c * s["case"]["experts"] / (s["case"]["topk"] * (b - a))
        parts.append((f * p[a:b].mean(0)).sum())
        total = total + square[a:b].sum()
        rows += b - a
    balance = sum(parts) / len(parts) if parts else torch.zeros((), dtype=torch.float64, device="cuda")
    return balance, total / max(1, rows)


def _exact_balance(s):
    p, square, _ = _exact_router(s, s["logits"].double(), s["bias"].double() if _bias_learns(s["case"]) else None)
    groups, e = s["counts"].shape
    counts = torch.zeros(groups, e, dtype=torch.int32, device="cuda")
    probs = torch.zeros(groups, e, dtype=torch.float64, device="cuda")
    for i, (a, b) in enumerate(_exact_ranges(s)):
        if b > a:
            counts[i] = torch.histc(s["ids"][a:b].double(), e, -0.5, e - 0.5).int()
            probs[i] = p[a:b].mean(0)
    return counts, probs, torch.stack(_exact_losses(s, p, square, counts.double()))


def _exact_route_backward(s):
    logits = s["logits"].double().requires_grad_()
    bias = s["bias"].double().requires_grad_() if _bias_learns(s["case"]) else None
    p, square, chosen = _exact_router(s, logits, bias)
    ranges = _exact_ranges(s)
    first, last = ranges[0][0], ranges[-1][1]
    chosen = chosen * s["case"]["scale"]
    total = (chosen * s["dweights"].double())[first:last].sum()
    if s["case"]["losses"]:
        balance, z = _exact_losses(s, p, square, s["counts"].double())
        total = total + s["dlosses"][0].double() * balance + s["dlosses"][1].double() * z
    d = torch.autograd.grad(total, [logits] + ([bias] if bias is not None else []))
    return d[0], d[1] if bias is not None else None


def _exact_e4m3(codes):
    """FP8 e4m3 bytes as 64-bit values, from their bits."""
    b = codes.view(torch.uint8).long()
    e, m = ((b & 127) >> 3).double(), (b & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e - 7))
    return torch.where(b > 127, -v, v)


def _exact_rows(x, xs, w, ws, bias):
    """Block by block: the 64-bit sum over 128 columns, times the two scales."""
    x, w = _exact_e4m3(x), _exact_e4m3(w)
    v = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device="cuda")
    block = torch.arange(w.shape[0], device="cuda") // BLOCK
    for b in range(xs.shape[1]):
        part = x[:, b * BLOCK:(b + 1) * BLOCK] @ w[:, b * BLOCK:(b + 1) * BLOCK].t()
        v += part * xs[:, b].double()[:, None] * ws[:, b].double()[block][None, :]
    return v if bias is None else v + bias.double()


def _exact_activation(v, act):
    if act == "swiglu":
        half = v.shape[1] // 2
        return v[:, :half] * torch.sigmoid(v[:, :half]) * v[:, half:]
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    if act == "relu":
        return torch.relu(v)
    return torch.relu(v) ** 2 if act == "relu2" else v


def _exact_product(s):
    if s["op"] == "mm":
        v = _exact_rows(s["x"], s["xs"], s["w"], s["ws"], s["bias"])
    else:
        o = s["offsets"].tolist()
        v = torch.cat([_exact_rows(s["x"][a:b], s["xs"][a:b], s["w"][e], s["ws"][e],
                                   None if s["bias"] is None else s["bias"][e])
                       for e, (a, b) in enumerate(zip(o[:-1], o[1:])) if b > a])
    v = s["case"]["scale"] * _exact_activation(v, s["case"]["act"])
    return v if s["residual"] is None else v + s["residual"].double()


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "balance": _exact_balance,
            "route_backward": _exact_route_backward, "mm": _exact_product, "moe_mm": _exact_product}[case["op"]](s)
