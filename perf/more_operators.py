"""Cases of a decoder's feed-forward and projections over weights of few bits: the router of a mixture of
experts, the layer of its experts (affine codes), the quantization of activations and weights to 8-bit
floating point with a scale for each block of 128, and the product of such operands.

`run` computes a case in its plain form (elementary torch operations in float32, or float64 next to a
border between two choices or two codes) or, where `own` is true, through the package's entry points.
`exact` computes the same outputs in float64 from the definitions."""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_F8 = torch.float8_e4m3fn
_BLOCK = 128


def listed():
    return [
        # A decode step's routing: 128 experts, 8 of them for each token.
        dict(name="route_decode", op="route", tokens=64, experts=128, top_k=8, scoring="softmax", bias=False,
             renormalize=True, scale=1.0, dtype="bf16", masked=0.0),
        # A prompt's routing, logits kept in float32.
        dict(name="route_prompt", op="route", tokens=16384, experts=128, top_k=8, scoring="softmax", bias=False,
             renormalize=True, scale=1.0, dtype="f32", masked=0.0),
        # Independent scores with a balancing bias that only the choice sees, some experts switched off.
        dict(name="route_balanced", op="route", tokens=4097, experts=253, top_k=6, scoring="sigmoid", bias=True,
             renormalize=True, scale=2.5, dtype="f16", masked=0.05),
        # One user's next token through the experts of one layer: the call whose latency counts.
        dict(name="moe_one", op="moe", tokens=1, experts=128, top_k=8, hidden=768, width=2048, bits=4, group=64,
             dtype="bf16", elsewhere=0.0, resid=True),
        # A decode step of a busy server.
        dict(name="moe_batch", op="moe", tokens=64, experts=128, top_k=8, hidden=768, width=2048, bits=4, group=64,
             dtype="bf16", elsewhere=0.0, resid=True),
        # Sizes that are no multiple of a tile, straddling codes, a part of the experts on another machine.
        dict(name="moe_odd", op="moe", tokens=37, experts=60, top_k=4, hidden=1408, width=2080, bits=6, group=32,
             dtype="f16", elsewhere=0.25, resid=False),
        # A prompt's tokens through the same layer.
        dict(name="moe_prompt", op="moe", tokens=2048, experts=128, top_k=8, hidden=768, width=2048, bits=4, group=64,
             dtype="bf16", elsewhere=0.0, resid=True),
        # A prompt's activations on their way into a product.
        dict(name="quantize_prompt", op="quantize", rows=8192, cols=4096, block_rows=1, dtype="bf16"),
        # A weight taken into the format as it is loaded.
        dict(name="quantize_weight", op="quantize", rows=4096, cols=14336, block_rows=128, dtype="bf16"),
        # One token's projection.
        dict(name="product_one", op="product", m=1, n=4096, k=4096, dtype="bf16"),
        # A decode batch's up projection, a ragged number of rows.
        dict(name="product_batch", op="product", m=61, n=14336, k=4096, dtype="f16"),
        # A prompt's down projection.
        dict(name="product_prompt", op="product", m=2048, n=4096, k=14336, dtype="bf16"),
    ]


def _span(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["route", "moe", "moe", "quantize", "product", "product"])
    while True:
        if op == "route":
            experts = _span(rng, 4, 512)
            c = dict(op=op, tokens=_span(rng, 1, 16384), experts=experts, top_k=rng.randint(1, min(8, experts)),
                     scoring=rng.choice(["softmax", "softmax", "sigmoid"]), bias=rng.random() < 0.4,
                     renormalize=rng.random() < 0.7, scale=rng.choice([1.0, 1.0, 2.5]),
                     dtype=rng.choice(["bf16", "f16", "f32"]), masked=rng.choice([0.0, 0.0, 0.05, 0.9]))
            if c["tokens"] * experts <= 4 << 20:
                return c
        elif op == "moe":
            group = rng.choice([32, 64, 64, 128])
            experts = _span(rng, 2, 128)
            c = dict(op=op, tokens=_span(rng, 1, 4096), experts=experts, top_k=rng.randint(1, min(8, experts)),
                     hidden=group * _span(rng, 1, 2048 // group), width=group * _span(rng, 1, 4096 // group),
                     bits=rng.choice([2, 3, 4, 4, 4, 5, 6, 8]), group=group, dtype=rng.choice(["bf16", "bf16", "f16"]),
                     elsewhere=rng.choice([0.0, 0.0, 0.0, 0.5]), resid=rng.random() < 0.5)
            w = work(c)
            if w["flops"] <= 1.5e11 and experts * c["hidden"] * c["width"] <= 1 << 28 and w["bytes"] >= 1e4:
                return c
        elif op == "quantize":
            c = dict(op=op, rows=_span(rng, 1, 16384), cols=_span(rng, 16, 16384), block_rows=rng.choice([1, 1, 128]),
                     dtype=rng.choice(["bf16", "f16", "f32"]))
            if c["rows"] * c["cols"] <= 1 << 26:
                return c
        else:
            c = dict(op=op, m=_span(rng, 1, 8192), n=_span(rng, 64, 16384), k=_span(rng, 64, 16384),
                     dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
            if rng.random() < 0.7:
                c["k"] = max(1, c["k"] // 128) * 128
            if 2 * c["m"] * c["n"] * c["k"] <= 2.4e11:
                return c


def _blocks(n):
    return -(-n // _BLOCK)


def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        return {"bytes": t * e * size[case["dtype"]] + 8 * t * k + (4 * e if case["bias"] else 0), "flops": 0}
    if case["op"] == "moe":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        rows = t * k * (1 - case["elsewhere"])
        used = e * (1 - (1 - rows / t / e) ** t)  # experts that some token has chosen, on average
        weights = 3 * case["hidden"] * case["width"] * (case["bits"] / 8 + 4 / case["group"])
        return {"bytes": used * weights + t * case["width"] * (6 if case["resid"] else 4) + 8 * t * k,
                "flops": 6 * rows * case["hidden"] * case["width"]}
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        scales = -(-case["rows"] // case["block_rows"]) * _blocks(case["cols"])
        return {"bytes": n * (size[case["dtype"]] + 1) + 4 * scales, "flops": 0}
    m, n, k = case["m"], case["n"], case["k"]
    return {"bytes": m * k + n * k + 4 * _blocks(k) * (m + _blocks(n)) + m * n * size[case["dtype"]],
            "flops": 2 * m * n * k}


def _prepare_route(case, gen):
    t, e = case["tokens"], case["experts"]
    x = 2.0 * torch.randn(t, e, generator=gen, device="cuda") + 0.5 * torch.randn(e, generator=gen, device="cuda")
    if case["masked"]:
        x[torch.rand(t, e, generator=gen, device="cuda") < case["masked"]] = -torch.inf
        x[::97] = -torch.inf  # tokens to which no expert is left
    bias = 0.1 * torch.randn(e, generator=gen, device="cuda") if case["bias"] else None
    return dict(case=case, logits=x.to(_TYPES[case["dtype"]]), bias=bias)


def _affine(n_experts, rows, cols, case, gen):
    """Random codes with scales and biases that give weights of variance 1 / cols around 0."""
    dt, bits = _TYPES[case["dtype"]], case["bits"]
    words = torch.randint(-(1 << 31), 1 << 31, (n_experts, rows, cols * bits // 32), generator=gen, device="cuda",
                          dtype=torch.int32)
    top = (1 << bits) - 1
    shape = (n_experts, rows, cols // case["group"])
    step = math.sqrt(12 / (top * (top + 2)) / cols)  # variance of a uniform code: top (top + 2) / 12
    scales = step * (0.5 + torch.rand(shape, generator=gen, device="cuda"))
    biases = -scales * top / 2 * (0.9 + 0.2 * torch.rand(shape, generator=gen, device="cuda"))
    return words, scales.to(dt), biases.to(dt)


def _prepare_moe(case, gen):
    t, e, k, h, w = (case[x] for x in ("tokens", "experts", "top_k", "hidden", "width"))
    dt = _TYPES[case["dtype"]]
    chosen = torch.rand(t, e, generator=gen, device="cuda").topk(k, dim=1).indices.int()
    chosen[torch.rand(t, k, generator=gen, device="cuda") < case["elsewhere"]] = -1
    weights = torch.rand(t, k, generator=gen, device="cuda").softmax(-1)
    return dict(case=case, x=torch.randn(t, w, generator=gen, device="cuda").to(dt), experts=chosen, weights=weights,
                gate=_affine(e, h, w, case, gen), up=_affine(e, h, w, case, gen), down=_affine(e, w, h, case, gen),
                resid=torch.randn(t, w, generator=gen, device="cuda").to(dt) if case["resid"] else None)


def _prepare_quantize(case, gen):
    x = torch.randn(case["rows"], case["cols"], generator=gen, device="cuda")
    if case["block_rows"] == 1:  # activations: rows of different size, a few channels far above the others
        x *= torch.exp(torch.randn(case["rows"], 1, generator=gen, device="cuda"))
        x[:, ::211] *= 30
    else:
        x *= 0.02
    return dict(case=case, x=x.to(_TYPES[case["dtype"]]))


def _codes(rows, cols, gen):
    """Codes as a block's largest value at 448 leaves them, normally distributed."""
    return (130 * torch.randn(rows, cols, generator=gen, device="cuda")).clamp_(-448, 448).to(_F8)


def _prepare_product(case, gen):
    m, n, k = case["m"], case["n"], case["k"]
    scales = (0.5 + torch.rand(m, _blocks(k), generator=gen, device="cuda")) / 130
    return dict(case=case, x=_codes(m, k, gen), x_scales=scales, w=_codes(n, k, gen),
                w_scales=(0.5 + torch.rand(_blocks(n), _blocks(k), generator=gen, device="cuda")) / 130 / math.sqrt(k))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"route": _prepare_route, "moe": _prepare_moe, "quantize": _prepare_quantize,
            "product": _prepare_product}[case["op"]](case, gen)


def _plain_route(s):
    c = s["case"]
    kind = torch.float64 if c["bias"] else torch.float32  # a score next to another decides who is chosen
    x = s["logits"].to(kind)
    if c["scoring"] == "softmax":
        top = x.amax(-1, keepdim=True)
        e = torch.where(top == -torch.inf, 0.0, (x - top).exp())
        score = e / e.sum(-1, keepdim=True).clamp(min=1e-300 if c["bias"] else 1e-37)
    else:
        score = 1 / (1 + (-x).exp())
    key = torch.where(x == -torch.inf, x, score + s["bias"].to(kind)) if c["bias"] else x
    chosen = key.sort(dim=-1, descending=True, stable=True).indices[:, :c["top_k"]]
    w = score.gather(1, chosen)
    if c["renormalize"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return (w * c["scale"]).float(), chosen.int()


def _dense(weight, e, bits, group):
    """Expert e's weight in float32: codes from each row's little-endian bit stream."""
    words, scales, biases = (t[e] for t in weight)
    words = words.long() & 0xFFFFFFFF
    cols = words.shape[1] * 32 // bits
    at = torch.arange(cols, device=words.device) * bits
    lo, shift = at >> 5, at & 31
    hi = (lo + 1).clamp(max=words.shape[1] - 1)
    codes = ((words[:, lo] >> shift) | (words[:, hi] << (32 - shift))) & ((1 << bits) - 1)
    wide = codes.float().view(-1, cols // group, group)
    return (wide * scales.float()[..., None] + biases.float()[..., None]).view(-1, cols)


def _plain_moe(s):
    c = s["case"]
    x, k = s["x"].float(), c["top_k"]
    flat = s["experts"].reshape(-1).long()
    order = flat.argsort(stable=True)
    counts = torch.bincount(flat + 1, minlength=c["experts"] + 1).tolist()
    y = torch.zeros_like(x) if s["resid"] is None else s["resid"].float()
    at = counts[0]  # rows of experts that are elsewhere add nothing here
    for e, n in enumerate(counts[1:]):
        if not n:
            continue
        rows = order[at:at + n]
        at += n
        token = rows // k
        g = x[token] @ _dense(s["gate"], e, c["bits"], c["group"]).T
        u = x[token] @ _dense(s["up"], e, c["bits"], c["group"]).T
        d = (g / (1 + (-g).exp()) * u) @ _dense(s["down"], e, c["bits"], c["group"]).T
        y.index_add_(0, token, d * s["weights"].reshape(-1)[rows, None])
    return y.to(s["x"].dtype)


def _padded(x, rows, cols):
    """x with zeros up to whole blocks, as [row blocks, rows, column blocks, cols]."""
    n, k = x.shape
    full = torch.zeros(-(-n // rows) * rows, -(-k // cols) * cols, dtype=x.dtype, device=x.device)
    full[:n, :k] = x
    return full.view(-1, rows, full.shape[1] // cols, cols)


def _plain_quantize(s):
    c = s["case"]
    x = _padded(s["x"].double(), c["block_rows"], _BLOCK)  # a quotient next to a border between two codes
    scale = (x.abs().amax((1, 3)) / 448).float()
    q = (x / scale.double()[:, None, :, None]).float()
    q = torch.where(scale[:, None, :, None] == 0, 0.0, q).clamp(-448, 448)
    codes = q.reshape(-1, q.shape[2] * _BLOCK)[:c["rows"], :c["cols"]].contiguous().to(_F8)
    return codes, scale


def _plain_product(s):
    c = s["case"]
    x = s["x"].float() * s["x_scales"].repeat_interleave(_BLOCK, 1)[:, :c["k"]]
    each = s["w_scales"].repeat_interleave(_BLOCK, 0)[:c["n"]].repeat_interleave(_BLOCK, 1)[:, :c["k"]]
    w = s["w"].float() * each
    return (x @ w.T).to(_TYPES[c["dtype"]])


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"route": _plain_route, "moe": _plain_moe, "quantize": _plain_quantize,
                "product": _plain_product}[c["op"]](s)
    import quantized_matmul_mlx_amd as qaff
    if c["op"] == "route":
        return qaff.moe_route(s["logits"], c["top_k"], bias=s["bias"], scoring=c["scoring"],
                              renormalize=c["renormalize"], scale=c["scale"])
    if c["op"] == "moe":
        return qaff.moe_ffn(s["x"], s["experts"], s["weights"], s["gate"], s["up"], s["down"], c["group"], c["bits"],
                            resid=s["resid"])
    if c["op"] == "quantize":
        return qaff.block_quantize(s["x"], block_rows=c["block_rows"])
    return qaff.block_qmm(s["x"], s["x_scales"], s["w"], s["w_scales"], out_dtype=_TYPES[c["dtype"]])


def _exact_route(s):
    c = s["case"]
    x = s["logits"].double()
    empty = torch.isneginf(x).all(-1)
    score = torch.sigmoid(x)
    if c["scoring"] == "softmax":
        score = torch.where(empty[:, None], 0.0, torch.softmax(torch.where(empty[:, None], 0.0, x), -1))
    rank = x.clone()
    if c["bias"]:
        rank = score + s["bias"].double()
        rank[torch.isneginf(x)] = -torch.inf
    experts, weights = [], []
    left = torch.ones_like(rank, dtype=torch.bool)
    index = torch.arange(c["experts"], device=x.device)
    for _ in range(c["top_k"]):  # the largest that is left, the first of equal ones
        best = torch.where(left, rank, -torch.inf).amax(-1, keepdim=True)
        first = torch.where(left & (rank == best), index, c["experts"]).amin(-1, keepdim=True)
        left.scatter_(1, first, False)
        experts.append(first)
        weights.append(score.gather(1, first))
    w = torch.cat(weights, 1)
    if c["renormalize"]:
        w = w / torch.where(w.sum(-1, keepdim=True) > 0, w.sum(-1, keepdim=True), 1.0)
    return w * c["scale"], torch.cat(experts, 1).int()


def _exact_weight(weight, e, bits, group):
    words, scales, biases = (t[e] for t in weight)
    bit = torch.arange(32, device=words.device, dtype=torch.int32)
    stream = (words[:, :, None] >> bit & 1).reshape(words.shape[0], -1, bits)  # a row's bits, a code each
    codes = (stream.double() * 2.0 ** torch.arange(bits, device=words.device)).sum(-1)
    group_of = torch.arange(codes.shape[1], device=words.device) // group
    return codes * scales.double()[:, group_of] + biases.double()[:, group_of]


def _exact_moe(s):
    c = s["case"]
    x = s["x"].double()
    y = torch.zeros_like(x) if s["resid"] is None else s["resid"].double()
    for e in range(c["experts"]):
        mine = s["experts"] == e
        token = mine.any(-1).nonzero().squeeze(1)
        if token.numel():
            share = (mine[token] * s["weights"][token].double()).sum(-1, keepdim=True)
            gate, up, down = (_exact_weight(s[k], e, c["bits"], c["group"]) for k in ("gate", "up", "down"))
            pre = x[token] @ gate.T
            y[token] += share * ((pre * torch.sigmoid(pre) * (x[token] @ up.T)) @ down.T)
    return y


def _exact_quantize(s):
    """The scale is float32(largest / 448), a code the nearest 8-bit value, of two the even one, of the
    float32 quotient by it."""
    c = s["case"]
    x, br = s["x"].double(), c["block_rows"]
    scales = torch.empty(-(-c["rows"] // br), _blocks(c["cols"]), device="cuda")
    codes = torch.empty_like(x)
    for j in range(_blocks(c["cols"])):
        part = x[:, j * _BLOCK:(j + 1) * _BLOCK]
        top = part.abs().amax(1)
        if br > 1:
            top = torch.stack([t.max() for t in top.split(br)])
        scales[:, j] = (top / 448).float()
        scale = scales[:, j].double().repeat_interleave(br)[:c["rows"], None]
        q = torch.where(scale > 0, part / scale, 0.0).float().double().clamp(-448, 448)
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)  # of the value's binade
        codes[:, j * _BLOCK:(j + 1) * _BLOCK] = torch.round(q / step) * step
    return codes, scales.double()


def _exact_product(s):
    c = s["case"]
    y = torch.zeros(c["m"], c["n"], dtype=torch.float64, device="cuda")
    rows = torch.arange(c["n"], device="cuda") // _BLOCK
    for j in range(_blocks(c["k"])):
        part = slice(j * _BLOCK, min(c["k"], (j + 1) * _BLOCK))
        sums = s["x"][:, part].double() @ s["w"][:, part].double().T
        y += s["x_scales"][:, j].double()[:, None] * sums * s["w_scales"][rows, j].double()
    return y


def exact(case, seed):
    return {"route": _exact_route, "moe": _exact_moe, "quantize": _exact_quantize,
            "product": _exact_product}[case["op"]](prepare(case, seed))
