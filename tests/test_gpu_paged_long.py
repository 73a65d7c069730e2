"""Paged attention over tables so long that a row's parts are joined in several stretches, and over many
requests whose keys are cut finer: against float64 sums over all keys at once."""
import math
import random

import pytest
import torch

import paged_ref as ref
import quantized_matmul_mlx_amd as qaff
from gpu_util import banner
from test_gpu_paged import BF, HF, ints

pytestmark = pytest.mark.gpu


def wanted(q, k, v, scale):
    """One request's last rows q [n, heads, dim] over keys and values [kv, kv_heads, dim] of types like q's:
    (out, lse, allowed error of out, of lse), the errors counted as in paged_ref.attention."""
    n, heads, dim = q.shape
    kv, kv_heads = k.shape[:2]
    u = ref.HALF_STEP[q.dtype]
    x, kd, vd = q.double(), k.double(), v.double()
    seen = torch.arange(kv)[None] <= (kv - n + torch.arange(n))[:, None]
    count = seen.sum(1)[:, None]
    out, lse = torch.empty(n, heads, dim, dtype=torch.float64), torch.empty(n, heads, dtype=torch.float64)
    tol, ltol = torch.empty_like(out), torch.empty_like(lse)
    for h in range(heads):
        hk = h // (heads // kv_heads)
        s = (x[:, h] @ kd[:, hk].T * scale).masked_fill(~seen, -math.inf)
        lse[:, h] = torch.logsumexp(s, 1)
        p = torch.exp(s - lse[:, h, None])
        out[:, h] = p @ vd[:, hk]
        size = p @ vd[:, hk].abs()
        most = (x[:, h].abs() @ kd[:, hk].abs().T * scale).masked_fill(~seen, 0).amax(1)
        top = s.masked_fill(~seen, 0).abs().amax(1)
        ds = (dim + 4) * ref.F32 * most + 8 * ref.F32 * (1 + top)
        small = 2.0 ** -32 * (seen.double() @ vd[:, hk].abs()) + 2.0 ** -25 if q.dtype == HF else 0.0
        tol[:, h] = (1.01 * u + 2 * ds[:, None] + (count + 8) * ref.F32) * size + u * out[:, h].abs() + small
        ltol[:, h] = 2 * ds + (count[:, 0] + 8) * ref.F32 + 4 * ref.F32 * (1 + lse[:, h].abs())
    return out, lse, tol, ltol


def check(lens, heads, kv_heads, dim, page, dt, width=None, max_new=None, jump=False, seed=0):
    gen = torch.Generator().manual_seed(seed)
    need = [-(-k // page) for k, _ in lens]
    order = torch.randperm(sum(need) + 2, generator=gen).tolist()
    width = width or max(need) + 1
    tables = torch.tensor([[order.pop() for _ in range(m)] + [-1] * (width - m) for m in need], dtype=torch.int32)
    cu = [0]
    for _, n in lens:
        cu.append(cu[-1] + n)
    q = torch.randn(cu[-1], heads, dim, generator=gen).to(dt)
    pool = sum(need) + 2
    k, v = (torch.randn(pool, kv_heads, page, dim, generator=gen).to(dt) for _ in range(2))
    if jump:  # the largest scores lie in the last stretch of keys: what was joined before is scaled by little
        for b, (kv, _) in enumerate(lens):
            ids = tables[b, :need[b]].long()
            k[ids[-max(1, need[b] // 8):]] *= 6
    out, lse = qaff.paged_attention(q.cuda(), k.cuda(), v.cuda(), tables.cuda(), ints(cu), ints([x for x, _ in lens]),
                                    max_new=max_new or max(n for _, n in lens), return_lse=True)
    out, lse = out.cpu().double(), lse.cpu().double()
    for b, (kv, n) in enumerate(lens):
        ids = tables[b, :need[b]].long()
        kb, vb = (x[ids].transpose(1, 2).reshape(-1, kv_heads, dim)[:kv] for x in (k, v))
        rows = slice(cu[b], cu[b + 1])
        want, wlse, tol, ltol = wanted(q[rows], kb, vb, 1 / math.sqrt(dim))
        assert ((out[rows] - want).abs() <= tol).all(), f"request {b}: out"
        assert ((lse[rows] - wlse).abs() <= ltol).all(), f"request {b}: lse"


# One row over one cache head is cut into as many parts as the chip holds workgroups, twice: more than the
# 512 that a stretch of the join takes. A chunk's tile has parts of 512 keys at least, and a stretch of its
# join takes 32 (heads of up to 64), 64 or 128 of them.
@pytest.mark.parametrize("jump", [False, True])
@pytest.mark.parametrize("dim,dt", [(64, BF), (128, HF), (256, BF)])
@pytest.mark.parametrize("heads", [1, 4])
def test_one_row_over_a_long_table(dim, dt, heads, jump):
    banner(f"long row dim {dim} heads {heads} jump {jump}")
    check([(130001, 1)], heads, 1, dim, 64, dt, jump=jump)


@pytest.mark.parametrize("jump", [False, True])
@pytest.mark.parametrize("dim,keys,dt", [(64, 40007, HF), (128, 70003, BF), (256, 75001, BF)])
def test_a_chunk_over_a_long_table(dim, keys, dt, jump):
    banner(f"long chunk dim {dim} keys {keys} jump {jump}")
    check([(keys, 40)], 1, 1, dim, 16, dt, jump=jump)


def test_two_chunks_over_a_long_table():
    # the join's workgroups walk over several rows each, with several stretches a row
    check([(70003, 40), (33000, 37)], 4, 1, 128, 32, BF)


@pytest.mark.parametrize("dim,heads,kv_heads", [(128, 4, 2), (64, 2, 2), (256, 2, 2)])
@pytest.mark.parametrize("page", [16, 64])
def test_many_requests_over_a_long_table(dim, heads, kv_heads, page):
    # three parts a workgroup slot: more requests than half the slots, a table of 4096 keys or more
    banner(f"long tables of many dim {dim} page {page}")
    rng = random.Random(dim)
    lens = [(rng.choice([1, 17, 100, rng.randint(1, 700)]), 1) for _ in range(300)]
    lens[7] = lens[150] = (4100, 1)
    lens[299] = (9000, 1)
    check(lens, heads, kv_heads, dim, page, BF)


def test_many_requests_and_chunks_over_a_long_table():
    rng = random.Random(9)
    lens = [(rng.randint(1, 500), 1) for _ in range(140)]
    lens[3], lens[77] = (9001, 100), (5000, 33)
    check(lens, 4, 2, 128, 16, HF)
