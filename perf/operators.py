"""Cases of the serving operators around a paged cache: the plan of a step (block tables and slot
maps), rotary positions with the write into the cache, and attention of the new tokens over it.

`run` computes a case in its plain form (elementary torch operations in float32, or float64 for the
angles) or, where `own` is true, through the package's entry points. `exact` computes the same
outputs in float64 from the definitions."""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # A decode step of a busy server: one new token per request, contexts up to 8 K.
        dict(name="plan_decode", op="plan", requests=64, chunks=0, new=1, cached=8192, page=16, lens_seed=1),
        # A step that admits prompts: a thousand requests, 160 of them with a chunk of the prompt.
        dict(name="plan_admit", op="plan", requests=1021, chunks=160, new=511, cached=16384, page=32, lens_seed=2),
        # The new tokens of a decode step (32 query heads and 8 cache heads of a 4096-wide model).
        dict(name="rope_decode", op="rope", tokens=64, heads=32, kv_heads=8, dim=128, rot=128, axes=1,
             interleaved=False, traditional=False, page=16, far=131072, dtype="bf16"),
        # A long prompt's tokens.
        dict(name="rope_prompt", op="rope", tokens=8192, heads=32, kv_heads=8, dim=128, rot=128, axes=1,
             interleaved=False, traditional=False, page=16, far=131072, dtype="bf16"),
        # Image and video tokens: time, height and width positions interleaved over the pairs.
        dict(name="rope_axes", op="rope", tokens=4101, heads=28, kv_heads=4, dim=128, rot=128, axes=3,
             interleaved=True, traditional=False, page=16, far=32768, dtype="f16"),
        # One user's next token over a short context: the smallest call.
        dict(name="attn_one", op="attention", requests=1, chunks=0, new=1, cached=777, heads=32, kv_heads=8, dim=128,
             page=16, window=0, dtype="bf16", lse=False, lens_seed=6),
        # A decode step of a busy server, contexts of 1 K to 8 K.
        dict(name="attn_decode", op="attention", requests=64, chunks=0, new=1, cached=8192, heads=32, kv_heads=8,
             dim=128, page=16, window=0, dtype="bf16", lse=False, lens_seed=7),
        # Two users deep in a long document: few rows, a long cache.
        dict(name="attn_far", op="attention", requests=2, chunks=0, new=1, cached=120001, heads=32, kv_heads=8,
             dim=128, page=64, window=0, dtype="f16", lse=False, lens_seed=8),
        # A few short prompts packed into one call.
        dict(name="attn_short", op="attention", requests=3, chunks=3, new=333, cached=0, heads=32, kv_heads=8,
             dim=128, page=16, window=0, dtype="bf16", lse=False, lens_seed=9),
        # A long prompt in one piece.
        dict(name="attn_prompt", op="attention", requests=1, chunks=1, new=8192, cached=0, heads=32, kv_heads=8,
             dim=128, page=16, window=0, dtype="bf16", lse=False, lens_seed=10),
        # A chunk of a long prompt over what is cached of it, with the sums a caller needs to join parts.
        dict(name="attn_chunk", op="attention", requests=1, chunks=1, new=512, cached=32768, heads=32, kv_heads=8,
             dim=128, page=32, window=0, dtype="bf16", lse=True, lens_seed=11),
        # Chunked prefill beside decoding requests, a window of 1 K keys, 64-wide heads.
        dict(name="attn_mixed", op="attention", requests=33, chunks=2, new=1111, cached=6000, heads=24, kv_heads=4,
             dim=64, page=32, window=1024, dtype="f16", lse=False, lens_seed=12),
    ]


def _span(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    n = min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))
    return n + 1 if n == 3 * 1024 else n


def draw(rng):
    op = rng.choice(["plan", "rope", "attention", "attention"])
    seed = rng.randrange(1, 1 << 30)
    if op == "plan":
        while True:
            r = _span(rng, 1, 1024)
            c = dict(op=op, requests=r, chunks=rng.choice([0, r, rng.randint(0, r)]), new=_span(rng, 1, 2048),
                     cached=_span(rng, 1, 65536), page=rng.choice([8, 16, 32, 64, 128]), lens_seed=seed)
            if sum(_lens(c)[1]) <= 98304:
                return c
    if op == "rope":
        kv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 96, 128, 128, 256])
        axes = rng.choice([1, 1, 3])
        while True:
            c = dict(op=op, tokens=_span(rng, 1, 16384), heads=kv * rng.choice([1, 4, 7, 8]), kv_heads=kv, dim=dim,
                     rot=dim if axes > 1 else rng.choice([dim, dim, dim // 2]), axes=axes,
                     interleaved=axes > 1 and rng.random() < 0.5, traditional=rng.random() < 0.3,
                     page=rng.choice([16, 32, 64]), far=_span(rng, 1024, 1 << 20), dtype=rng.choice(["bf16", "f16"]))
            if work(c)["bytes"] <= 250e6:
                return c
    while True:
        kind = rng.choice(["decode", "prompt", "chunk", "mixed"])
        r = _span(rng, 1, 64) if kind in ("decode", "mixed") else rng.randint(1, 4)
        kv = rng.choice([1, 2, 4, 8])
        c = dict(op=op, requests=r,
                 chunks={"decode": 0, "prompt": r, "chunk": r, "mixed": min(r, rng.randint(1, 3))}[kind],
                 new=1 if kind == "decode" else _span(rng, 2, 8192), cached=0 if kind == "prompt" else _span(rng, 1, 131072),
                 heads=kv * rng.choice([1, 4, 7, 8]), kv_heads=kv, dim=rng.choice([64, 96, 128, 128, 256]),
                 page=rng.choice([8, 16, 32, 64, 128]), window=rng.choice([0, 0, 0, 512, 4096]),
                 dtype=rng.choice(["bf16", "f16"]), lse=rng.random() < 0.25, lens_seed=seed)
        w = work(c)
        plain = sum(n * (k + n) for k, n in zip(*_lens(c))) * c["heads"] * c["dim"]  # what the plain form multiplies
        if w["flops"] <= 5.5e11 and w["bytes"] <= 2.5e9 and plain <= 2.75e11:
            return c


def _lens(case):
    """Cached and new tokens of each request. The first request has the lengths the case names, the
    others between an eighth of them and all; the last `chunks` requests bring a chunk of tokens
    (the others one each)."""
    rng = random.Random(case["lens_seed"])
    r, first = case["requests"], case["requests"] - case["chunks"]
    cached = [case["cached"] if b == 0 else rng.randint(case["cached"] // 8, case["cached"]) for b in range(r)]
    new = [1 if b < first else case["new"] if b == first else rng.randint(max(1, case["new"] // 8), case["new"])
           for b in range(r)]
    return cached, new


def _pages(tokens, page):
    return -(-tokens // page)


def work(case):
    if case["op"] == "plan":
        cached, new = _lens(case)
        fresh = sum(_pages(c + n, case["page"]) - _pages(c, case["page"]) for c, n in zip(cached, new))
        return {"bytes": 20 * case["requests"] + 12 * sum(new) + 8 * fresh + 8, "flops": 0}
    if case["op"] == "rope":
        t, row = case["tokens"], (case["heads"] + 2 * case["kv_heads"]) * case["dim"]
        turned = (case["heads"] + case["kv_heads"]) * case["rot"] // 2
        return {"bytes": t * (4 * row + 4 * case["axes"] + 8) + 2 * case["rot"], "flops": 6 * t * turned}
    cached, new = _lens(case)
    win = case["window"] or 1 << 62
    pairs = keys = 0
    for c, n in zip(cached, new):
        short = min(n, max(0, win - c))  # queries that see less than a whole window
        pairs += short * c + short * (short + 1) // 2 + (n - short) * min(win, c + n)
        keys += min(c + n, win + n - 1)
    q = sum(new) * case["heads"] * case["dim"]
    size = 4 * q + 4 * keys * case["kv_heads"] * case["dim"] + 4 * keys // case["page"] + 8 * case["requests"]
    return {"bytes": size + (4 * sum(new) * case["heads"] if case["lse"] else 0),
            "flops": 4 * case["dim"] * case["heads"] * pairs}


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype).cuda()


def _tables(cached, new, page, gen, spare=4):
    """Shuffled pages for every request: the table (padded with 0), its width and the pool's size."""
    need = [_pages(c + n, page) for c, n in zip(cached, new)]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=gen, device="cuda", dtype=torch.int32)
    width = max(need) + 1
    starts = _ints([sum(need[:b]) for b in range(len(need))])[:, None]
    col = torch.arange(width, device="cuda", dtype=torch.int32)[None]
    live = col < _ints(need)[:, None]
    table = torch.where(live, order[(starts + col).clamp(max=pool - 1).long()], torch.zeros_like(order[:1]))
    return table.contiguous(), pool


def _prepare_plan(case, gen):
    cached, new = _lens(case)
    page = case["page"]
    table, pool = _tables(cached, new, page, gen)
    have = _ints([_pages(c, page) for c in cached])[:, None]
    col = torch.arange(table.shape[1], device="cuda")[None]
    total = sum(new)
    fresh = sum(_pages(c + n, page) - _pages(c, page) for c, n in zip(cached, new))
    return dict(case=case, cached=_ints(cached), new=_ints(new), table=torch.where(col < have, table, -1).int().contiguous(),
                free=torch.randperm(fresh + 64, generator=gen, device="cuda").int() + pool, page=page, tokens=total)


def _sections(case):
    half = case["rot"] // 2
    if case["axes"] == 1:
        return None
    side = half * 5 // 16  # for 64 pairs: 24 of time, 20 of height, 20 of width
    return (half - 2 * side, side, side)


def _prepare_rope(case, gen):
    t, h, kv, d, page = (case[k] for k in ("tokens", "heads", "kv_heads", "dim", "page"))
    dt = _TYPES[case["dtype"]]
    qkv = torch.randn(t, h + 2 * kv, d, generator=gen, device="cuda").to(dt)  # one projection's rows
    pages = _pages(t, page) + 3
    shape = (t,) if case["axes"] == 1 else (case["axes"], t)
    half = case["rot"] // 2
    return dict(case=case, q=qkv[:, :h], k=qkv[:, h:h + kv], v=qkv[:, h + kv:],
                positions=torch.randint(0, case["far"], shape, generator=gen, device="cuda", dtype=torch.int32),
                inv_freq=(500000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float(),
                slots=torch.randperm(pages * page, generator=gen, device="cuda")[:t],
                k_cache=torch.zeros(pages, kv, page, d, dtype=dt, device="cuda"),
                v_cache=torch.zeros(pages, kv, page, d, dtype=dt, device="cuda"), sections=_sections(case))


def _prepare_attention(case, gen):
    cached, new = _lens(case)
    h, kv, d, page = (case[k] for k in ("heads", "kv_heads", "dim", "page"))
    dt = _TYPES[case["dtype"]]
    table, pool = _tables(cached, new, page, gen)
    total = sum(new)
    q = torch.randn(total, h, d, generator=gen, device="cuda").to(dt)
    k, v = (torch.empty(pool, kv, page, d, dtype=dt, device="cuda").normal_(generator=gen) for _ in range(2))
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return dict(case=case, q=q, k_cache=k, v_cache=v, table=table, cu=_ints(cu),
                kv_lens=_ints([c + n for c, n in zip(cached, new)]), max_new=max(new), lens=(cached, new), starts=cu)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"plan": _prepare_plan, "rope": _prepare_rope, "attention": _prepare_attention}[case["op"]](case, gen)


def _plain_plan(s):
    cached, new, page, total = s["cached"].long(), s["new"].long(), s["page"], s["tokens"]
    zero = torch.zeros(1, dtype=torch.long, device=new.device)
    cu = torch.cat([zero, new.cumsum(0)])
    have = (cached + page - 1) // page
    need = torch.where(new > 0, (cached + new + page - 1) // page - have, 0)
    first = torch.cat([zero, need.cumsum(0)])
    col = torch.arange(s["table"].shape[1], device=new.device)[None] - have[:, None]
    fresh = (col >= 0) & (col < need[:, None])
    at = (first[:-1, None] + col).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][at], s["table"])
    t = torch.arange(total, device=new.device)
    req = torch.searchsorted(cu, t, right=True) - 1
    pos = cached[req] + t - cu[req]
    slots = table[req, pos // page].long() * page + pos % page
    return cu.int(), (cached + new).int(), pos.int(), slots, first[-1:].int(), table


def _axis_of_pair(case, half, device):
    i = torch.arange(half, device=device)
    if case["axes"] == 1:
        return torch.zeros_like(i)
    sec = _sections(case)
    if case["interleaved"]:
        a = i % len(sec)
        return torch.where(i < len(sec) * torch.tensor(sec, device=device)[a], a, 0)
    return torch.cat([torch.full((n,), a, device=device) for a, n in enumerate(sec)])


def _turn(x, cos, sin, rot, traditional):
    half = rot // 2
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if traditional else (x[..., :half], x[..., half:rot])
    y = x.clone()
    left, right = a * cos - b * sin, b * cos + a * sin
    if traditional:
        y[..., 0:rot:2], y[..., 1:rot:2] = left, right
    else:
        y[..., :half], y[..., half:rot] = left, right
    return y


def _plain_rope(s):
    c = s["case"]
    pos = s["positions"].double().reshape(-1, c["tokens"])
    angle = pos[_axis_of_pair(c, c["rot"] // 2, pos.device)].T * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out = _turn(s["q"].float(), cos, sin, c["rot"], c["traditional"]).to(s["q"].dtype)
    k = _turn(s["k"].float(), cos, sin, c["rot"], c["traditional"]).to(s["k"].dtype)
    page, off = s["slots"] // c["page"], s["slots"] % c["page"]
    s["k_cache"][page, :, off] = k
    s["v_cache"][page, :, off] = s["v"]
    return out, s["k_cache"], s["v_cache"]


def _plain_attention(s):
    c = s["case"]
    h, kv, d, win = c["heads"], c["kv_heads"], c["dim"], c["window"]
    g = h // kv
    out = torch.empty_like(s["q"])
    lse = torch.empty(out.shape[:2], dtype=torch.float32, device=out.device)
    for b, (past, n) in enumerate(zip(*s["lens"])):
        total = past + n
        pages = s["table"][b, :_pages(total, c["page"])].long()
        k, v = (x[pages].transpose(0, 1).reshape(kv, -1, d)[:, :total].float().contiguous()
                for x in (s["k_cache"], s["v_cache"]))
        kt = k.transpose(1, 2).contiguous()
        for at in range(0, n, 1024):  # so many query rows at a time
            m = min(1024, n - at)
            rows = slice(s["starts"][b] + at, s["starts"][b] + at + m)
            x = s["q"][rows].float().reshape(m, kv, g, d).permute(1, 2, 0, 3).reshape(kv, g * m, d)
            score = torch.matmul(x, kt).reshape(kv, g, m, total) * (1 / math.sqrt(d))
            p = torch.arange(past + at, past + at + m, device=x.device)[:, None]
            j = torch.arange(total, device=x.device)[None]
            hidden = j > p
            if win:
                hidden |= j <= p - win
            score.masked_fill_(hidden, float("-inf"))
            top = score.amax(-1, keepdim=True)
            e = score.sub_(top).exp_()
            z = e.sum(-1, keepdim=True)
            o = torch.matmul(e.reshape(kv, g * m, total), v).reshape(kv, g, m, d) / z
            out[rows] = o.permute(2, 0, 1, 3).reshape(m, h, d).to(out.dtype)
            lse[rows] = (top + z.log()).squeeze(-1).permute(2, 0, 1).reshape(m, h)
    return (out, lse) if c["lse"] else out


def run(state):
    c = state["case"]
    if not own:
        return {"plan": _plain_plan, "rope": _plain_rope, "attention": _plain_attention}[c["op"]](state)
    import quantized_matmul_mlx_amd as qaff
    s = state
    if c["op"] == "plan":
        p = qaff.paged_plan(s["cached"], s["new"], s["free"], s["table"], s["page"], s["tokens"])
        return p.cu_new, p.kv_lens, p.positions, p.slots, p.pages_used, s["table"]
    if c["op"] == "rope":
        out = qaff.rope_append(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["slots"], s["k_cache"],
                               s["v_cache"], sections=s["sections"], interleaved=c["interleaved"],
                               traditional=c["traditional"])
        return out, s["k_cache"], s["v_cache"]
    return qaff.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_lens"],
                                max_new=s["max_new"], window=c["window"], return_lse=c["lse"])


def _exact_plan(s):
    cached, new, page, table, free = (s[k].tolist() if torch.is_tensor(s[k]) else s[k]
                                      for k in ("cached", "new", "page", "table", "free"))
    cu, kv, pos, slots, used = [0], [], [], [], 0
    for b, (c, n) in enumerate(zip(cached, new)):
        for t in range(n):
            p = c + t
            if p % page == 0:  # the first token of a page takes the next free one
                table[b][p // page] = free[used]
                used += 1
            pos.append(p)
            slots.append(table[b][p // page] * page + p % page)
        cu.append(cu[-1] + n)
        kv.append(c + n)
    return _ints(cu), _ints(kv), _ints(pos), _ints(slots, torch.int64), _ints([used]), _ints(table)


def _exact_rope(s):
    c = s["case"]
    half, t = c["rot"] // 2, c["tokens"]
    sec = _sections(c)
    pos = s["positions"].cpu().double().reshape(-1, t)
    phase = torch.empty(t, half, dtype=torch.float64)
    for i in range(half):
        if sec is None:
            a = 0
        elif c["interleaved"]:
            a = i % 3 if i // 3 < sec[i % 3] else 0
        else:
            a = 0 if i < sec[0] else 1 if i < sec[0] + sec[1] else 2
        phase[:, i] = pos[a] * s["inv_freq"][i].double().item()
    turn = torch.polar(torch.ones_like(phase), phase).cuda()[:, None]
    lead = [(2 * i, 2 * i + 1) if c["traditional"] else (i, i + half) for i in range(half)]
    first, second = (torch.tensor(x, device="cuda") for x in zip(*lead))

    def turned(x):
        y = x.double().clone()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    flat = s["slots"] // c["page"], slice(None), s["slots"] % c["page"]
    kc[flat], vc[flat] = turned(s["k"]), s["v"].double()
    return turned(s["q"]), kc, vc


def _exact_attention(s):
    c = s["case"]
    h, kv, d = c["heads"], c["kv_heads"], c["dim"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(out.shape[:2], dtype=torch.float64, device="cuda")
    for b, (past, n) in enumerate(zip(*s["lens"])):
        key = torch.arange(past + n, device="cuda")
        page, off = s["table"][b].long()[key // c["page"]], key % c["page"]
        for i in range(kv):
            k, v = s["k_cache"][page, i, off].double(), s["v_cache"][page, i, off].double()
            for head in range(i * (h // kv), (i + 1) * (h // kv)):
                for at in range(0, n, 2048):
                    rows = torch.arange(at, min(at + 2048, n), device="cuda")
                    w = (s["q"][s["starts"][b] + rows, head].double() @ k.T) * d ** -0.5
                    own_key = past + rows[:, None]
                    seen = key[None] <= own_key
                    if c["window"]:
                        seen &= own_key - key[None] < c["window"]
                    w = torch.where(seen, w, -torch.inf)
                    total = torch.logsumexp(w, -1)
                    out[s["starts"][b] + rows, head] = torch.exp(w - total[:, None]) @ v
                    lse[s["starts"][b] + rows, head] = total
    return (out, lse) if c["lse"] else out


def exact(case, seed):
    return {"plan": _exact_plan, "rope": _exact_rope, "attention": _exact_attention}[case["op"]](prepare(case, seed))
