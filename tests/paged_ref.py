"""Plain float64 forms of the paged-cache operators, on the CPU, one request and one row at a time,
with the error that the kernels' roundings allow. No code of the library."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
F32 = 2.0 ** -24


def plan(cached, new, free, tables, page, rows):
    """Token by token: (cu, kv, positions, slots, used, tables)."""
    tables = [list(r) for r in tables]
    width = len(tables[0]) if tables else 0
    cu, kv, pos, slots, used = [0], [], [], [], 0
    for b, (c, n) in enumerate(zip(cached, new)):
        c, n = max(c, 0), max(n, 0)
        have = -(-c // page)
        for p in range(c, c + n):
            at = p // page
            in_rows = len(pos) < rows
            if p % page == 0 and at >= have:
                entry = free[used] if used < len(free) and at < width else -1
                used += 1
                if at < width and in_rows:
                    tables[b][at] = entry
                page_id = entry
            elif at < have:
                page_id = tables[b][at] if at < width else -1
            if in_rows:
                pos.append(p)
                slots.append(page_id * page + p % page if page_id >= 0 else -1)
        cu.append(cu[-1] + n)
        kv.append(c + n)
    pad = rows - len(pos)
    return cu, kv, pos + [0] * pad, slots + [-1] * pad, used, tables


def rope(x, positions, inv_freq, axis, traditional):
    """x [tokens, heads, dim], positions [axes, tokens], axis of each pair -> (turned, allowed error)."""
    y, tol = x.double().clone(), torch.zeros_like(x.double())
    half = inv_freq.numel()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if traditional else (i, i + half)
        ang = positions[axis[i]].double() * inv_freq[i].double()
        c, s = ang.cos()[:, None], ang.sin()[:, None]
        u, v = x[..., a].double(), x[..., b].double()
        y[..., a], y[..., b] = u * c - v * s, v * c + u * s
        # sine and cosine in float32 (fraction of a turn, the function: 4 steps), two products and a sum
        tol[..., a] = tol[..., b] = 8 * F32 * (u.abs() + v.abs())
    # the rounding at the end, half a step of the type (and of its smallest value)
    tol += torch.where(tol > 0, y.abs() * HALF_STEP[x.dtype] + (2.0 ** -25 if x.dtype == torch.float16 else 0.0), 0.0)
    return y, tol


def attention(q, k_cache, v_cache, tables, cu, kv_lens, scale, causal=True, window=0):
    """(out, lse, allowed error of out, allowed error of lse); rows that see no key are zeros and
    -inf, rows that see a key on a page outside the pool NaN."""
    tokens, heads, dim = q.shape
    pages, kv_heads, page, _ = k_cache.shape
    group = heads // kv_heads
    u = HALF_STEP[q.dtype]
    out = torch.zeros(tokens, heads, dim, dtype=torch.float64)
    lse = torch.full((tokens, heads), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(len(kv_lens)):
        n, kv = cu[b + 1] - cu[b], kv_lens[b]
        if n <= 0 or kv <= 0:
            continue
        j = torch.arange(kv)
        entry = j // page
        width = tables.shape[1]
        ids = torch.where(entry < width, tables[b][entry.clamp(max=width - 1)].long(), -1)
        good = (ids >= 0) & (ids < pages)
        ids = torch.where(good, ids, 0)
        k = k_cache[ids, :, j % page].double()  # [kv, kv_heads, dim]
        v = v_cache[ids, :, j % page].double()
        pos = kv - n + torch.arange(n)
        seen = torch.ones(n, kv, dtype=torch.bool)
        if causal:
            seen &= j[None] <= pos[:, None]
        if window:
            seen &= j[None] > pos[:, None] - window
        for h in range(heads):
            kh, vh = k[:, h // group], v[:, h // group]
            qh = q[cu[b]:cu[b + 1], h].double()
            for i in range(n):
                w = seen[i]
                if not w.any():
                    continue
                row = cu[b] + i
                if not good[w].all():
                    out[row, h], lse[row, h] = math.nan, math.nan
                    continue
                s = (kh[w] @ qh[i]) * scale
                lse[row, h] = torch.logsumexp(s, 0)
                p = torch.exp(s - lse[row, h])
                out[row, h] = p @ vh[w]
                # a score: dim products summed in float32, then the scaling and the exponential's argument
                ds = ((dim + 4) * F32 * (kh[w].abs() @ qh[i].abs()) * scale).max() + 8 * F32 * (1 + s.abs().max())
                count = int(w.sum())
                size = p @ vh[w].abs()
                # probabilities off by their scores' error and one rounding to the type (float16: its
                # smallest step, 2^-32 of the largest probability), sums in float32, the last rounding
                tol[row, h] = ((1.01 * u + 2 * ds + (count + 8) * F32) * size + u * out[row, h].abs()
                               + (2.0 ** -32 * vh[w].abs().sum(0) + 2.0 ** -25 if q.dtype == torch.float16 else 0.0))
                ltol[row, h] = 2 * ds + (count + 8) * F32 + 4 * F32 * (1 + lse[row, h].abs())
    return out, lse, tol, ltol
