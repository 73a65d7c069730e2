"""Views of the caches that are laid out as [pages, kv_heads, page_size, head_dim] in memory are taken,
whatever the strides of their axes of size 1 say; others are refused."""
import pytest
import torch

import quantized_matmul_mlx_amd as qaff
from test_gpu_paged import BF, Case, ints

pytestmark = pytest.mark.gpu


def attend(c, k, v):
    return qaff.paged_attention(c.q.cuda(), k, v, c.tables.cuda(), ints(c.cu), ints(c.kv))


def test_one_cache_head_kept_behind_the_tokens():
    # [pages, page_size, 1, head_dim], as a cache of one head may well be kept
    c = Case([(70, 3), (40, 1)], 4, 1, 64, 16, BF)
    k, v = c.caches()
    want = attend(c, k, v)
    turned = [x.reshape(x.shape[0], 16, 1, 64).transpose(1, 2) for x in (k, v)]
    assert turned[0].shape == k.shape and turned[0].stride() != k.stride()
    assert torch.equal(attend(c, *turned), want)
    assert torch.equal(attend(c, k, turned[1]), want)  # one of them only
    # and as rope_append's target
    row = torch.randn(2, 1, 64, device="cuda").to(BF)
    q = torch.randn(2, 4, 64, device="cuda").to(BF)
    args = q, row, row, ints([5, 9]), torch.ones(32, device="cuda"), ints([3, 20], torch.int64)
    a = qaff.rope_append(*args, k, v)
    k2, v2 = (x.reshape(x.shape[0], 16, 1, 64).transpose(1, 2) for x in (torch.zeros_like(k), torch.zeros_like(v)))
    b = qaff.rope_append(*args, k2, v2)
    assert torch.equal(a, b)
    for page, off in ((0, 3), (1, 4)):
        assert torch.equal(k2[page, :, off], k[page, :, off]) and torch.equal(v2[page, :, off], row[page])


def test_one_page():
    c = Case([(9, 3)], 4, 2, 64, 16, BF)
    c.tables[c.tables >= 0] = 0
    k, v = (torch.randn(1, 2, 16, 64, device="cuda").to(BF) for _ in range(2))
    want = attend(c, k, v)
    odd = [torch.as_strided(x, x.shape, (7, *x.stride()[1:])) for x in (k, v)]  # a stride that no page takes
    assert torch.equal(attend(c, *odd), want) and torch.equal(attend(c, k, odd[1]), want)


def test_layouts_that_differ_are_refused():
    c = Case([(70, 3)], 4, 2, 64, 16, BF)
    k, v = c.caches()
    strided = torch.stack([v, v], 1)[:, 0]  # pages twice as far apart as k's
    with pytest.raises(ValueError, match="strides"):
        attend(c, k, strided)
    with pytest.raises(ValueError, match="contiguous"):
        turned = k.transpose(1, 2).contiguous().transpose(1, 2)
        attend(c, turned, turned)
