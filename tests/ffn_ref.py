"""Plain float64 forms of the feed-forward operators, with bounds of the rounding errors their kernels may
make: half a step of each rounding (u) and float32 sums."""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
F32 = 2.0 ** -24


def codes_of(words, bits):
    """[..., words] int32 -> [..., cols] codes: a little-endian bit stream a row."""
    b = (words[..., None] >> torch.arange(32, device=words.device, dtype=torch.int32)) & 1
    b = b.reshape(*words.shape[:-1], -1, bits).long()
    return (b << torch.arange(bits, device=words.device)).sum(-1)


def dense(weight, bits, group):
    """(packed, scales, biases) -> float64 weights and |s| (2 B + c) + |b|, what a kernel's sums may hold of a
    weight in magnitude (B up to 1024: codes enter as B + c)."""
    words, s, b = weight
    c = codes_of(words, bits).double()
    s, b = (t.double().repeat_interleave(group, -1) for t in (s, b))
    return s * c + b, s.abs() * (2048 + c) + b.abs()


def random_weight(gen, experts, rows, cols, bits, group, dtype, device="cuda"):
    words = torch.randint(-(1 << 31), 1 << 31, (experts, rows, cols * bits // 32), generator=gen, dtype=torch.int64)
    top = (1 << bits) - 1
    step = (12 / (top * (top + 2)) / cols) ** 0.5
    s = step * (0.5 + torch.rand(experts, rows, cols // group, generator=gen))
    s = torch.where(torch.rand(s.shape, generator=gen) < 0.5, s, -s)
    b = -s * top / 2 * (0.8 + 0.4 * torch.rand(s.shape, generator=gen))
    return words.int().to(device), s.to(dtype).to(device), b.to(dtype).to(device)


def route(logits, top_k, bias=None, scoring="softmax", renormalize=True, scale=1.0):
    """float64 weights, experts, and the weights' bound."""
    x = logits.double().cpu()
    x = torch.where(x.isnan(), -torch.inf, x)
    top = x.amax(-1, keepdim=True)
    none = top == -torch.inf
    if scoring == "softmax":
        e = torch.where(none, 0.0, torch.where(x == top, 1.0, (x - top).exp()))
        total = e.sum(-1, keepdim=True)
        score = torch.where(total > 0, e / total, 0.0)
    else:
        score = 1 / (1 + (-x).exp())
    key = x if bias is None else torch.where(x == -torch.inf, x, score + bias.double().cpu())
    key = torch.where(key.isnan(), -torch.inf, key)
    chosen = key.sort(dim=-1, descending=True, stable=True).indices[..., :top_k]
    w = score.gather(-1, chosen)
    # exponent: the difference's rounding; then exp (2 steps), sums, a quotient and the factor
    gap = torch.where(chosen >= 0, (x.gather(-1, chosen) - (top if scoring == "softmax" else 0)).abs(), 0.0)
    rel = (gap.nan_to_num(0, 0, 0) + 2 * x.shape[-1] ** 0.5 + 16) * 2 * F32
    if renormalize:
        s = w.sum(-1, keepdim=True)
        w = torch.where(s > 0, w / s, 0.0)
        rel = rel + rel.amax(-1, keepdim=True)
    w = w * scale
    return w, chosen.int(), w.abs() * rel + 1e-37


def moe(x, experts, weights, gate, up, down, group, bits, resid=None):
    """float64 y and its bound. The products' sums are float32: at most k / 16 + 32 roundings one after
    another, each half a step of a partial sum no larger than the sum of magnitudes; silu(g) u is rounded
    to x's type; silu's exponential and quotient are good to 8 steps."""
    u = HALF[x.dtype]
    n_experts, hidden, width = gate[0].shape[0], gate[0].shape[1], x.shape[-1]
    y = torch.zeros(x.shape, dtype=torch.float64, device=x.device) if resid is None else resid.double().clone()
    err = y.abs() * F32
    xs = x.double()
    for e in range(n_experts):
        mine = experts == e
        token = mine.any(-1).nonzero().squeeze(1)
        if not token.numel():
            continue
        share = (mine[token] * weights[token].double()).sum(-1, keepdim=True)
        mag = (mine[token] * weights[token].double().abs()).sum(-1, keepdim=True)
        (wg, ag), (wu, au), (wd, ad) = (dense(tuple(t[e] for t in w), bits, group) for w in (gate, up, down))
        xa = xs[token]
        g, v = xa @ wg.T, xa @ wu.T
        dg, dv = ((xa.abs() @ a.T) * (width / 16 + 32) * F32 for a in (ag, au))
        sig = torch.sigmoid(g)
        h = g * sig * v
        slope = (sig * (1 + g * (1 - sig))).abs() + dg  # silu' (its own slope is at most 1/2)
        dh = slope * v.abs() * dg + (g * sig).abs() * dv + dg * dv + h.abs() * (u + 16 * F32) + TINY[x.dtype]
        y[token] += share * (h @ wd.T)
        err[token] += mag * (dh @ wd.abs().T + (h.abs() + dh) @ ad.T * (hidden / 16 + 32) * F32)
        err[token] += mag * (h.abs() @ wd.abs().T) * experts.shape[-1] * F32
    return y, err + u * (y.abs() + err) + TINY[x.dtype]


def quantize(x, block_rows=1):
    """Codes (float8 on the CPU) and scales, by the formula in float32 (IEEE quotients)."""
    x = x.float().cpu()
    rows, cols = x.shape
    nb, kb = -(-rows // block_rows), -(-cols // 128)
    full = torch.zeros(nb * block_rows, kb * 128)
    full[:rows, :cols] = x
    tiles = full.view(nb, block_rows, kb, 128)
    scale = tiles.abs().amax((1, 3)) / 448
    q = tiles / scale[:, None, :, None]
    q = torch.where(scale[:, None, :, None] == 0, 0.0, q).clamp(-448, 448)
    return q.reshape(nb * block_rows, -1)[:rows, :cols].contiguous().to(torch.float8_e4m3fn), scale


def product(x, xs, w, ws, dtype, eights=False):
    """float64 y and its bound: float32 sums of at most 128 terms a block, scaled and added block by block.
    With `eights`, sums of the 8-bit matrix instructions: of each eight products, those beside the largest lose
    less than 2^-13 of its power of two (seven of them)."""
    m, k = x.shape
    n = w.shape[0]
    a = x.double() * xs.double().repeat_interleave(128, 1)[:, :k]
    b = w.double() * ws.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    y = a @ b.T
    err = (a.abs() @ b.abs().T) * (k / 128 + 128 + 4) * F32
    if eights:
        for at in range(0, k, 8):
            err += 7 * 2.0 ** -13 * (a[:, None, at:at + 8] * b[None, :, at:at + 8]).abs().amax(-1)
    return y, err + HALF[dtype] * (y.abs() + err) + TINY[dtype]
