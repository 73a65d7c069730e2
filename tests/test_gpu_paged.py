"""The paged-cache operators against plain float64 forms (tests/paged_ref.py)."""
import math
import random

import pytest
import torch

import paged_ref as ref
import quantized_matmul_mlx_amd as qaff
from gpu_util import banner

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype).cuda()


# ---- the plan ----

def check_plan(cached, new, page, width=None, n_free=None, rows=None, seed=0):
    rng = random.Random(seed)
    have = [-(-max(c, 0) // page) for c in cached]
    need = [-(-(max(c, 0) + max(n, 0)) // page) for c, n in zip(cached, new)]
    width = max(need, default=0) + 1 if width is None else width
    ids = list(range(sum(need) + 3))
    rng.shuffle(ids)
    tables = []
    for h in have:
        own = [ids.pop() for _ in range(min(h, width))]
        tables.append(own + [-7] * (width - len(own)))
    free = ids if n_free is None else ids[:n_free]
    rows = sum(max(n, 0) for n in new) if rows is None else rows
    want = ref.plan(cached, new, free, tables, page, rows)
    table = ints(tables).reshape(len(cached), width)
    for _ in range(2):  # the step taken again from the same state gives the same plan
        got = qaff.paged_plan(ints(cached), ints(new), ints(free), table, page, rows)
        assert got.cu_new.tolist() == want[0]
        assert got.kv_lens.tolist() == want[1]
        assert got.positions.tolist() == want[2]
        assert got.slots.tolist() == want[3]
        assert got.pages_used.tolist() == [want[4]]
        assert table.tolist() == want[5]


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
def test_plan_edges(page):
    banner(f"plan page {page}")
    check_plan([0, 0, 1, page - 1, page, page + 1, 5 * page, 3], [1, page + 1, 0, 1, 1, 1, 2 * page, page - 3], page)


@pytest.mark.parametrize("requests", [1, 2, 63, 64, 65, 511, 512, 513, 1100])
def test_plan_many_requests(requests):
    banner(f"plan {requests} requests")
    rng = random.Random(requests)
    check_plan([rng.randint(0, 90) for _ in range(requests)], [rng.choice([0, 1, 1, 1, 40]) for _ in range(requests)], 16)


def test_plan_most_requests():
    banner("plan 16384 requests")
    check_plan([(i * 7) % 40 for i in range(16384)], [1] * 16384, 8)


def test_plan_padding_negative_lengths_and_no_tokens():
    check_plan([3, -5, 20], [2, 4, -1], 8, rows=11)
    check_plan([3, 9], [0, 0], 8)
    check_plan([3, 9], [0, 0], 8, rows=5)
    check_plan([3, 9], [4, 30], 8, rows=12)  # fewer rows than tokens


def test_plan_runs_out_of_pages_or_width():
    check_plan([3, 9, 0], [20, 30, 9], 8, n_free=3)
    check_plan([3, 9, 0], [20, 30, 9], 8, n_free=0)
    check_plan([3, 30, 0], [20, 30, 9], 8, width=3)


def test_plan_saturates():
    big = 2**31 - 1
    table = torch.full((2, 4), 5, dtype=torch.int32).cuda()
    got = qaff.paged_plan(ints([big, 0]), ints([big, 3]), ints([1, 2]), table, 8, 4)
    assert got.cu_new.tolist() == [0, big, big] and got.kv_lens.tolist() == [big, 3]
    assert got.positions.tolist() == [big] * 4 and got.slots.tolist() == [-1] * 4


# ---- rotary positions and the cache write ----

def axis_map(half, sections, interleaved):
    if sections is None:
        return [0] * half
    if interleaved:
        a = len(sections)
        return [i % a if i // a < sections[i % a] else 0 for i in range(half)]
    return [x for x, n in enumerate(sections) for _ in range(n)]


def check_rope(tokens, heads, kv_heads, dim, rot, dt, page=16, sections=None, interleaved=False, traditional=False,
               far=1 << 20, fused=True, offset=0, in_place=False, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rows = heads + 2 * kv_heads
    flat = torch.randn(offset + tokens * rows * dim, generator=gen).to(dt)
    dev = flat.cuda()
    if fused:
        x, xd = flat[offset:].view(tokens, rows, dim), dev[offset:].view(tokens, rows, dim)
    else:  # heads outermost: large head strides
        x, xd = (f[offset:].view(rows, tokens, dim).transpose(0, 1) for f in (flat, dev))
    parts = slice(0, heads), slice(heads, heads + kv_heads), slice(heads + kv_heads, rows)
    q, k, v = (x[:, p] for p in parts)
    qd, kd, vd = (xd[:, p] for p in parts)
    axes = 1 if sections is None else len(sections)
    pos = torch.randint(0, far, (axes, tokens), generator=gen, dtype=torch.int32)
    half = rot // 2
    inv = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float()
    pages = -(-tokens // page) + 2
    slots = torch.randperm(pages * page, generator=gen)[:tokens]
    if tokens > 2:
        slots[1], slots[2] = -1, pages * page  # written nowhere
    kc = torch.randn(pages, kv_heads, page, dim, generator=gen).to(dt)
    vc = torch.randn(pages, kv_heads, page, dim, generator=gen).to(dt)
    kcd, vcd = kc.cuda(), vc.cuda()
    if in_place:
        qd = qd.contiguous()
    got = qaff.rope_append(qd, kd, vd, (pos if sections else pos[0]).contiguous().cuda(), inv.cuda(), slots.cuda(), kcd,
                           vcd, sections=sections, interleaved=interleaved, traditional=traditional,
                           out=qd if in_place else None)
    axis = axis_map(half, sections, interleaved)
    want, tol = ref.rope(q, pos, inv, axis, traditional)
    assert got.shape == q.shape and got.dtype == dt
    assert ((got.cpu().double() - want).abs() <= tol).all()
    kw, ktol = ref.rope(k, pos, inv, axis, traditional)
    kc64, vc64, tol64 = kc.double(), vc.double(), torch.zeros_like(kc.double())
    for t in range(tokens):
        s = slots[t].item()
        if 0 <= s < pages * page:
            kc64[s // page, :, s % page], tol64[s // page, :, s % page] = kw[t], ktol[t]
            vc64[s // page, :, s % page] = v[t].double()
    assert ((kcd.cpu().double() - kc64).abs() <= tol64).all()
    assert torch.equal(vcd.cpu().double(), vc64)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("traditional", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (64, 64), (96, 96), (256, 256), (128, 64), (128, 32), (80, 48), (72, 24),
                                     (20, 10), (33, 12), (16, 0), (8, 8), (512, 512)])
def test_rope_sizes(dt, traditional, dim, rot):
    banner(f"rope {dt} {dim} {rot} {traditional}")
    check_rope(37, 8, 2, dim, rot, dt, traditional=traditional)


@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 7, 8, 65, 257])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (28, 4), (7, 1)])
def test_rope_tokens_and_heads(tokens, heads, kv_heads):
    banner(f"rope tokens {tokens} heads {heads}/{kv_heads}")
    check_rope(tokens, heads, kv_heads, 128, 128, BF, page=8)


@pytest.mark.parametrize("sections,interleaved", [((24, 20, 20), False), ((24, 20, 20), True), ((64, 0, 0), True),
                                                  ((0, 64, 0), False), ((32, 32), True), ((31, 33), False),
                                                  ((16, 16, 16, 16), True), ((40, 8, 8, 8), True)])
@pytest.mark.parametrize("traditional", [False, True])
def test_rope_axes(sections, interleaved, traditional):
    banner(f"rope sections {sections} {interleaved}")
    check_rope(19, 6, 2, 128, 128, HF, sections=sections, interleaved=interleaved, traditional=traditional)


def test_rope_strides_alignment_and_in_place():
    for dim, rot in ((128, 128), (64, 32)):
        check_rope(21, 4, 2, dim, rot, BF, fused=False)
        check_rope(21, 4, 2, dim, rot, BF, offset=1)   # not 16-byte aligned
        check_rope(21, 4, 2, dim, rot, HF, offset=4)   # 8-byte aligned
        check_rope(21, 4, 2, dim, rot, HF, in_place=True)
        check_rope(21, 4, 2, dim, rot, BF, in_place=True, traditional=True)


def test_rope_far_positions():
    check_rope(33, 4, 2, 128, 128, BF, far=2**31 - 1)


def test_rope_nothing_to_do():
    check_rope(0, 4, 2, 128, 128, BF)


# ---- attention ----

class Case:
    """Requests with kv_lens[b] keys, of which the last new[b] are this step's, in shuffled pages;
    what no key occupies holds NaN."""

    def __init__(self, lens, heads, kv_heads, dim, page, dt, seed=0, pad_rows=0, spread=1.0, alternate=False):
        gen = torch.Generator().manual_seed(seed)
        self.kv, self.new = [k for k, _ in lens], [n for _, n in lens]
        self.cu = [0]
        for n in self.new:
            self.cu.append(self.cu[-1] + n)
        need = [-(-k // page) for k in self.kv]
        pool = sum(need) + 2
        order = torch.randperm(pool, generator=gen).tolist()
        width = max(need, default=0) + 1
        self.tables = torch.tensor([[order.pop() for _ in range(m)] + [-1] * (width - m) for m in need],
                                   dtype=torch.int32).reshape(len(lens), width)
        self.q = (spread * torch.randn(self.cu[-1] + pad_rows, heads, dim, generator=gen)).to(dt)
        self.k = torch.full((pool, kv_heads, page, dim), math.nan, dtype=dt)
        self.v = self.k.clone()
        for b, n in enumerate(self.kv):
            j = torch.arange(n)
            ids = self.tables[b].long()[j // page]
            self.k[ids, :, j % page] = torch.randn(n, kv_heads, dim, generator=gen).to(dt)
            self.v[ids, :, j % page] = torch.randn(n, kv_heads, dim, generator=gen).to(dt)
        self.alternate = alternate
        self.scale = 1 / math.sqrt(dim)

    def caches(self):
        if not self.alternate:
            return self.k.cuda(), self.v.cuda()
        both = torch.stack([self.k, self.v], 1).cuda()  # K and V pages in turn
        return both[:, 0], both[:, 1]

    def run(self, q=None, **kw):
        k, v = self.caches()
        return qaff.paged_attention(self.q.cuda() if q is None else q, k, v, self.tables.cuda(), ints(self.cu),
                                    ints(self.kv), return_lse=True, **kw)

    def check(self, got, causal=True, window=0, scale=None):
        out, lse = (x.cpu().double() for x in got)
        want, wlse, tol, ltol = ref.attention(self.q, self.k, self.v, self.tables, self.cu, self.kv,
                                              self.scale if scale is None else scale, causal, window)
        same = (out.isnan() & want.isnan()) | ((out - want).abs() <= tol)
        assert same.all(), f"out: {int((~same).sum())} of {same.numel()} off, first at {(~same).nonzero()[0].tolist()}"
        same = (lse.isnan() & wlse.isnan()) | (lse == wlse) | ((lse - wlse).abs() <= ltol)
        assert same.all(), f"lse: {int((~same).sum())} of {same.numel()} off, first at {(~same).nonzero()[0].tolist()}"


DECODE = [(1, 1), (2, 1), (15, 1), (16, 1), (17, 1), (31, 1), (32, 1), (33, 1), (64, 1), (65, 1), (257, 1), (777, 1)]
PROMPTS = [(1, 1), (5, 5), (31, 31), (32, 32), (33, 33), (64, 64), (65, 65), (130, 130)]
CHUNKS = [(300, 37), (6, 1), (0, 0), (400, 3), (129, 128), (70, 70), (511, 66)]


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("dim", [8, 20, 64, 72, 96, 128, 200, 256])
@pytest.mark.parametrize("lens", [DECODE, PROMPTS, CHUNKS], ids=["decode", "prompts", "chunks"])
def test_attention_sizes(dt, dim, lens):
    banner(f"attention {dt} dim {dim} {lens[:2]}")
    c = Case(lens, 4, 2, dim, 16, dt)
    c.check(c.run())


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 4), (7, 1), (14, 2), (8, 1), (32, 1), (33, 1), (40, 1)])
@pytest.mark.parametrize("lens", [DECODE, CHUNKS], ids=["decode", "chunks"])
def test_attention_heads(heads, kv_heads, lens):
    banner(f"attention heads {heads}/{kv_heads}")
    c = Case(lens, heads, kv_heads, 64, 32, BF)
    c.check(c.run())
    c.check(c.run(max_new=max(c.new)))


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("lens", [DECODE, CHUNKS], ids=["decode", "chunks"])
def test_attention_pages(page, lens):
    banner(f"attention page {page}")
    c = Case(lens, 4, 1, 128, page, BF, alternate=True)
    c.check(c.run(max_new=max(c.new)))


@pytest.mark.parametrize("window", [1, 5, 32, 100, 5000])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", [DECODE, CHUNKS], ids=["decode", "chunks"])
def test_attention_masks(window, causal, lens):
    banner(f"attention window {window} causal {causal}")
    c = Case(lens, 4, 2, 64, 16, HF)
    c.check(c.run(window=window, causal=causal, max_new=max(c.new)), causal=causal, window=window)
    c.check(c.run(causal=causal), causal=causal)


def test_attention_rows_that_see_nothing():
    # more new tokens than keys: the first see none; and rows past every request
    c = Case([(0, 3), (2, 5), (40, 90), (0, 0), (7, 1)], 4, 2, 64, 16, BF, pad_rows=9)
    c.check(c.run())
    c.check(c.run(max_new=90))
    c = Case([], 4, 2, 64, 16, BF, pad_rows=5)
    c.check(c.run())


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("new", [1, 20, 130])
def test_attention_long_split(dt, new):
    # long rows, few of them: the keys are split over workgroups and joined
    banner(f"attention split {dt} new {new}")
    c = Case([(2500, new), (611, new)], 4, 2, 128, 16, dt, spread=2.0)
    c.check(c.run(max_new=new))


def test_attention_large_scores():
    # scores of several hundred: the softmax is all but one-hot, and the running maximum jumps
    c = Case([(900, 1), (500, 70)], 4, 2, 64, 16, HF, spread=40.0)
    c.check(c.run())
    c.check(c.run(scale=1.0), scale=1.0)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_attention_keys_out_of_the_window_do_not_enter(bad):
    # bad keys and values that the rows' windows have left behind
    c = Case([(180, 60), (200, 1)], 4, 2, 64, 8, BF)
    clean = ref.attention(c.q, c.k, c.v, c.tables, c.cu, c.kv, c.scale, True, 16)
    for b, j in ((0, 100), (0, 104), (1, 183), (1, 3)):
        page, off = c.tables[b, j // 8].long(), j % 8
        c.v[page, :, off, 5] = bad
        c.k[page, :, off, 6] = bad
    out, lse = (x.cpu().double() for x in c.run(window=16, max_new=60))
    # request 0's positions are 120 to 179, whose windows begin at 105; request 1's window at 184
    assert ((out - clean[0]).abs() <= clean[2]).all()
    assert ((lse - clean[1]).abs() <= clean[3]).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("heads", [2, 8])
def test_attention_later_tokens_values_do_not_enter(bad, heads):
    # a chunk whose later tokens hold bad values: earlier rows must be as if they were not there
    c = Case([(150, 100)], heads, 2, 64, 16, BF)
    ids = c.tables[0].long()
    clean = ref.attention(c.q, c.k, c.v, c.tables, c.cu, c.kv, c.scale)
    for j in (121, 140):
        c.v[ids[j // 16], :, j % 16, 9] = bad
        c.k[ids[j // 16], :, j % 16, 1] = bad
    out, lse = (x.cpu().double() for x in c.run())
    rows = 121 - 50
    assert ((out[:rows] - clean[0][:rows]).abs() <= clean[2][:rows]).all()
    assert ((lse[:rows] - clean[1][:rows]).abs() <= clean[3][:rows]).all()


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_attention_seen_values_enter(bad):
    # a value of infinity (or NaN) that a row sees with a positive weight is the row's result there
    c = Case([(70, 40)], 4, 2, 64, 16, BF)
    ids = c.tables[0].long()
    c.v[ids[45 // 16], :, 45 % 16, 9] = bad
    out = c.run()[0].cpu().double()
    seen = out[45 - 30:, :, 9]
    assert (seen.isnan() if math.isnan(bad) else seen == bad).all()
    assert out[:45 - 30].isfinite().all() and out[:, :, :9].isfinite().all() and out[:, :, 10:].isfinite().all()


@pytest.mark.parametrize("dim", [64, 20])
def test_attention_pages_outside_the_pool(dim):
    c = Case([(100, 1), (100, 60), (90, 1)], 4, 2, dim, 16, BF)
    c.tables[0, 2] = c.k.shape[0]
    c.tables[1, 5] = -3
    c.check(c.run())                      # rows that see the page are NaN, the others exact
    c.check(c.run(window=8), window=8)
    c.kv[2] = 1000                        # keys past the table's width
    c.check(c.run())


@pytest.mark.parametrize("dim", [64, 96, 20])
@pytest.mark.parametrize("stale", [-1, 10**6])
def test_attention_windows_over_released_pages(dim, stale):
    # the pages that every window has left behind are given back: their entries are stale
    c = Case([(700, 1), (300, 5), (640, 80)], 4, 2, dim, 8, HF)
    for b in range(3):
        first = c.kv[b] - c.new[b] - 100 + 1          # the first key that the request's first token sees
        c.tables[b, :first // 8] = stale
    c.check(c.run(window=100, max_new=80), window=100)


@pytest.mark.parametrize("dim", [8, 64, 72, 96, 128, 136, 256])
def test_attention_uses_the_pool_to_its_end(dim):
    # a pool of exactly the pages in use, the last page full, right up to the end of its allocation
    page, pages = 8, 24
    gen = torch.Generator().manual_seed(dim)
    k, v = (torch.randn(pages, 2, page, dim, generator=gen).to(BF) for _ in range(2))
    table = torch.arange(pages, dtype=torch.int32)[None]
    for new in (1, 60):
        q = torch.randn(new, 4, dim, generator=gen).to(BF)
        out = qaff.paged_attention(q.cuda(), k.cuda(), v.cuda(), table.cuda(), ints([0, new]), ints([pages * page]))
        want, _, tol, _ = ref.attention(q, k, v, table, [0, new], [pages * page], 1 / math.sqrt(dim))
        assert ((out.cpu().double() - want).abs() <= tol).all()


def test_attention_without_a_pool():
    # no page at all: every row that sees a key is NaN
    k = torch.empty(0, 2, 16, 64, dtype=BF, device="cuda")
    q = torch.randn(3, 4, 64, device="cuda").to(BF)
    out = qaff.paged_attention(q, k, k.clone(), ints([[0, 1], [0, 0]]), ints([0, 1, 2]), ints([5, 0]))
    assert out[0].isnan().all() and (out[1:] == 0).all()


@pytest.mark.parametrize("dim", [64, 20])
def test_attention_lengths_past_the_table(dim):
    # lengths that no table holds: NaN rows, and no time spent on keys that are not there
    c = Case([(100, 1), (60, 60), (90, 1), (64, 40)], 4, 2, dim, 16, BF)
    whole = c.run()[0].cpu()
    c.kv[0], c.kv[1] = 2**31 - 1, 2**31 - 1
    for kw in (dict(), dict(window=8), dict(max_new=60), dict(causal=False)):
        out, lse = (x.cpu() for x in c.run(**kw))
        assert out[:61].isnan().all() and lse[:61].isnan().all()
        assert out[61:].isfinite().all() and lse[61:].isfinite().all()
    assert torch.equal(c.run()[0].cpu()[61:], whole[61:])


@pytest.mark.parametrize("dim", [128, 64, 24])
def test_attention_strides_and_alignment(dim):
    c = Case(CHUNKS, 4, 2, dim, 16, BF)
    tokens = c.q.shape[0]
    wide = torch.zeros(tokens, 9, dim, dtype=BF)
    wide[:, 2:6] = c.q
    c.check(c.run(q=wide.cuda()[:, 2:6]))
    c.check(c.run(q=c.q.transpose(0, 1).contiguous().cuda().transpose(0, 1)))
    flat = torch.zeros(c.q.numel() + 1, dtype=BF, device="cuda")
    flat[1:] = c.q.reshape(-1).cuda()
    c.check(c.run(q=flat[1:].view(c.q.shape)))


def test_attention_max_new_is_only_a_hint():
    c = Case([(300, 1), (200, 150), (64, 9)], 8, 2, 128, 16, BF)
    for hint in (0, 1, 4, 150, 100000):
        c.check(c.run(max_new=hint))


def test_attention_many_requests():
    rng = random.Random(5)
    c = Case([(rng.randint(1, 60), 1) for _ in range(300)], 2, 1, 64, 8, HF)
    c.check(c.run(max_new=1))
    c = Case([(n, n) for n in (rng.choice([0, 1, 2, 40]) for _ in range(150))], 2, 1, 64, 8, HF)
    c.check(c.run())


@pytest.mark.parametrize("requests", [1, 63, 64, 65, 128, 129])
@pytest.mark.parametrize("new", [1, 50])
def test_attention_requests_and_rows_past_them(requests, new):
    # the search for a row's request takes 64 requests at a time; rows past the last are zeros
    banner(f"attention {requests} requests of {new}")
    rng = random.Random(requests)
    c = Case([(rng.randint(new, 200), new if b % 9 == 0 else 1) for b in range(requests)], 4, 2, 64, 16, BF, pad_rows=70)
    c.check(c.run())
    c.check(c.run(max_new=max(new, 70)))


def test_attention_same_bits_each_time_and_on_another_stream():
    c = Case([(3000, 1), (900, 33), (40, 40)], 8, 2, 128, 16, BF)
    k, v = c.caches()
    args = c.q.cuda(), k, v, c.tables.cuda(), ints(c.cu), ints(c.kv)
    first = qaff.paged_attention(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = qaff.paged_attention(*args)
    side.synchronize()
    assert torch.equal(first, other) and torch.equal(first, qaff.paged_attention(*args))


def test_a_far_page_past_32_bit_offsets():
    # a pool of more than 2^31 elements, of which the first and the last page are used
    page, kv_heads, dim = 256, 8, 128
    size = page * kv_heads * dim
    pages = 2**31 // size + 2
    k = torch.empty(pages, kv_heads, page, dim, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    for x in (k, v):
        x[0], x[-1] = torch.randn_like(x[0]), torch.randn_like(x[0])
    table = ints([[pages - 1, 0]])
    q = torch.randn(1, 8, dim, device="cuda").to(BF)
    out = qaff.paged_attention(q, k, v, table, ints([0, 1]), ints([300]))
    small = [torch.stack([x[-1], x[0]]) for x in (k, v)]
    want, _, tol, _ = ref.attention(q.cpu(), small[0].cpu(), small[1].cpu(), torch.tensor([[0, 1]]), [0, 1], [300],
                                    1 / math.sqrt(dim))
    assert ((out.cpu().double() - want).abs() <= tol).all()
    inv = torch.ones(dim // 2, device="cuda")
    row = torch.randn(1, 8, dim, device="cuda").to(BF)
    last = pages * page - 1
    qaff.rope_append(q, row, row, ints([0]), inv, ints([last], torch.int64), k, v)
    assert torch.equal(k[-1, :, -1], row[0]) and torch.equal(v[-1, :, -1], row[0])


# ---- a step as it is used: plan, cache write, attention; eager and as a graph ----

def step(cached, new, free, table, page, tokens, qkv, heads, inv, k, v):
    p = qaff.paged_plan(cached, new, free, table, page, tokens)
    kv = k.shape[1]
    q = qaff.rope_append(qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:], p.positions, inv, p.slots, k, v)
    return qaff.paged_attention(q, k, v, table, p.cu_new, p.kv_lens, max_new=max(1, tokens))


@pytest.mark.parametrize("chunk", [1, 40])
def test_a_step_in_a_graph_replays_like_eager(chunk):
    heads, kv, dim, page, requests = 8, 2, 128, 16, 3
    gen = torch.Generator(device="cuda").manual_seed(3)
    tokens = chunk * requests
    table = torch.full((requests, 40), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(130, generator=gen, device="cuda").int()
    k = torch.zeros(130, kv, page, dim, dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    inv = (10000.0 ** (-torch.arange(dim // 2, device="cuda") / (dim // 2))).float()
    cached, new = ints([0] * requests), ints([chunk] * requests)
    qkv = torch.zeros(tokens, heads + 2 * kv, dim, dtype=BF, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cached, new, free, table, page, tokens, qkv, heads, inv, k, v)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cached, new, free, table, page, tokens, qkv, heads, inv, k, v)
    table.fill_(-1)
    table2, k2, v2 = table.clone(), k.zero_().clone(), v.zero_().clone()
    left = free.clone()
    for i in range(4):
        qkv.copy_(torch.randn(qkv.shape, generator=gen, device="cuda"))
        eager = step(cached, new, left, table2, page, tokens, qkv, heads, inv, k2, v2)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(k, k2) and torch.equal(v, v2) and torch.equal(table, table2)
        used = requests * (-(-chunk * (i + 1) // page) - -(-chunk * i // page))
        left = torch.cat([left[used:], left[:used]]).contiguous()
        free.copy_(left)
        cached += chunk
