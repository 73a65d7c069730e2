"""The example examples/serve_layer.py: a layer's answers do not depend on how a request's tokens are
cut into steps, and the captured decode step does what the eager one does."""
import os
import sys

import pytest
import torch

from gpu_util import banner

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import serve_layer as ex  # noqa: E402

pytestmark = pytest.mark.gpu

WIDTH, LENS, PAGE = 512, [1, 7, 40, 133], 8


def setup(seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    layer = ex.Layer(WIDTH, 8, 2, 64, 1024, gen)
    prompts = [torch.randn(n + 6, WIDTH, generator=gen, device="cuda").bfloat16() for n in LENS]
    return layer, prompts


def cache_of(layer):
    return ex.Cache(layer, sum(-(-(n + 8) // PAGE) for n in LENS) + 2, PAGE, len(LENS), max(LENS) + 8)


def relative(a, b):
    return ((a.double() - b.double()).norm(dim=-1) / b.double().norm(dim=-1)).max().item()


# A layer's output rounds to bf16 (half a step 2^-8) at about ten places one after the other (norms,
# projections, rotary step, attention, residuals, the feed-forward's product); which kernel takes a
# number of rows changes the sums' order and so those roundings. Independent, ten of 2^-8 / sqrt(3)
# on either side are 2^-8 * sqrt(20 / 3) = 2^-6.6 in the norm; three times that is allowed.
TOL = 3 * 2 ** -6.6


@pytest.mark.parametrize("chunk", [5, 64])
def test_chunks_do_not_change_the_answers(chunk):
    banner(f"serve_layer chunk {chunk}")
    layer, prompts = setup()
    whole, cut = cache_of(layer), cache_of(layer)
    a = ex.prefill(layer, whole, prompts, 1000)
    b = ex.prefill(layer, cut, prompts, chunk)
    assert relative(b, a) <= TOL
    assert whole.lens.tolist() == cut.lens.tolist() == [n + 6 for n in LENS]
    # the free lists hold the same number of pages, and no page belongs to two requests
    for c in (whole, cut):
        used = [c.tables[i, :-(-(n + 6) // PAGE)].tolist() for i, n in enumerate(LENS)]
        ids = sum(used, [])
        left = c.free[c.free >= 0].tolist()
        assert len(set(ids)) == len(ids) and min(ids) >= 0
        assert sorted(ids + left) == list(range(c.k.shape[0]))


def test_captured_decode_equals_eager_and_the_prompt():
    banner("serve_layer decode")
    layer, prompts = setup(1)
    eager, captured = cache_of(layer), cache_of(layer)
    start = [p[:-6] for p in prompts]
    want = ex.prefill(layer, cache_of(layer), prompts, 1000)  # the whole prompts at once
    ex.prefill(layer, eager, start, 1000)
    ex.prefill(layer, captured, start, 1000)
    one = torch.ones_like(eager.lens)
    x = torch.zeros(len(LENS), WIDTH, dtype=torch.bfloat16, device="cuda")
    x.copy_(torch.stack([p[-6] for p in prompts]))
    decoder = ex.Decoder(layer, captured, x)
    for i in range(6):
        token = torch.stack([p[i - 6] for p in prompts])
        got = ex.step(layer, eager, token, one, 1)
        torch.cuda.synchronize()
        x.copy_(token)
        decoder.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, got)
        assert torch.equal(eager.tables, captured.tables) and torch.equal(eager.free, captured.free)
    assert relative(got, want) <= TOL
