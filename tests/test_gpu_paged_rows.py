"""Every row of paged attention's outputs is written, whatever the requests: through the C ABI, into
outputs that hold NaN before the call."""
import math

import pytest
import torch

import paged_ref as ref
from gpu_util import banner
from quantized_matmul_mlx_amd import _lib
from test_gpu_paged import BF, HF, Case, ints

pytestmark = pytest.mark.gpu


def attend(c, rows, max_new):
    """The case's first `rows` rows of q; (out, lse)."""
    lib = _lib.load()
    k, v = c.caches()
    q, tables, cu, kv = c.q[:rows].cuda().contiguous(), c.tables.cuda(), ints(c.cu), ints(c.kv)
    _, heads, dim = q.shape
    pages, kv_heads, page, _ = k.shape
    out = torch.full_like(q, math.nan)
    lse = torch.full((rows, heads), math.nan, device="cuda")
    size = lib.qaff_paged_attention_workspace_size(rows, heads, kv_heads, dim, page, tables.shape[1], len(c.kv), max_new)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    dtype = _lib.QAFF_F16 if q.dtype == HF else _lib.QAFF_BF16
    st = lib.qaff_paged_attention(q.data_ptr(), dtype, rows, heads, heads * dim, dim, k.data_ptr(), v.data_ptr(), pages,
                                  k.stride(0), kv_heads, dim, page, tables.data_ptr(), tables.shape[1], cu.data_ptr(),
                                  kv.data_ptr(), len(c.kv), max_new, c.scale, 1, 0, ws.data_ptr(), size, out.data_ptr(),
                                  lse.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == _lib.QAFF_OK, lib.qaff_last_error()
    torch.cuda.synchronize()
    return out, lse


# new tokens of each request, heads, kv_heads, rows past the requests, whether max_new is exact
FEW_REQUESTS = [([1, 1, 9], 32, 8, 0, True), ([1, 1, 1, 12], 32, 8, 0, True), ([1, 1, 5], 64, 8, 0, True),
                ([1, 1, 33], 32, 32, 0, True), ([4, 4, 4], 32, 8, 0, False), ([1, 1, 1], 64, 4, 0, False),
                ([1, 1, 1, 1], 64, 4, 0, False), ([1, 1, 1], 32, 8, 9, False), ([1, 1], 32, 8, 9, False),
                ([9, 1], 32, 8, 3, True)]


@pytest.mark.parametrize("new,heads,kv_heads,padding,exact", FEW_REQUESTS, ids=str)
@pytest.mark.parametrize("keys", [50, 2000])
def test_few_requests_of_few_rows(new, heads, kv_heads, padding, exact, keys):
    banner(f"rows new {new} heads {heads}/{kv_heads} padding {padding} keys {keys}")
    c = Case([(keys + 3 * b, n) for b, n in enumerate(new)], heads, kv_heads, 64, 16, BF, pad_rows=padding)
    rows = c.q.shape[0]
    c.check(attend(c, rows, max(new) if exact else rows))


@pytest.mark.parametrize("dim", [64, 128, 20])
@pytest.mark.parametrize("new", [[1] * 12, [20, 90, 70], [200], [3, 1, 150, 1, 1, 80, 1]], ids=str)
@pytest.mark.parametrize("cut", [1, 2, 25])
def test_fewer_rows_than_the_requests_tokens(dim, new, cut):
    # cu_new says where the requests' tokens are, as a plan for fewer rows leaves it: the rows that are
    # there come out as they do among all of them
    banner(f"rows dim {dim} new {new} cut {cut}")
    c = Case([(n + 37 * (b % 4), n) for b, n in enumerate(new)], 4, 2, dim, 16, HF)
    rows = max(1, c.q.shape[0] - cut)
    want, wlse, tol, ltol = (x[:rows] for x in ref.attention(c.q, c.k, c.v, c.tables, c.cu, c.kv, c.scale))
    for max_new in (max(new), rows):
        out, lse = (x.cpu().double() for x in attend(c, rows, max_new))
        assert ((out - want).abs() <= tol).all()
        assert ((lse - wlse).abs() <= ltol).all()


def test_fewer_rows_over_a_cut_table():
    # the same where the keys are cut into parts
    c = Case([(2500, 1), (900, 60)], 4, 2, 128, 16, BF)
    rows = 30
    want, wlse, tol, ltol = (x[:rows] for x in ref.attention(c.q, c.k, c.v, c.tables, c.cu, c.kv, c.scale))
    for max_new in (60, rows):
        out, lse = (x.cpu().double() for x in attend(c, rows, max_new))
        assert ((out - want).abs() <= tol).all()
        assert ((lse - wlse).abs() <= ltol).all()
