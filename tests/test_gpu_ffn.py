"""The feed-forward operators on the GPU against float64 (tests/ffn_ref.py, whose tolerances count
roundings): the router, the layer of experts, block quantization and the product of its operands."""
import functools
import zlib

import pytest
import torch

import ffn_ref as ref
import quantized_matmul_mlx_amd as qaff
from gpu_util import banner

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def gen_of(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def check(got, want, bound, what=""):
    got = got.double().cpu()
    want, bound = want.cpu(), bound.cpu()
    assert got.shape == want.shape
    off = (got - want).abs()
    worst = (off / bound).max().item() if off.numel() else 0.0
    print(f"{what} largest error / bound {worst:.3f}", flush=True)
    assert torch.isfinite(got).all() and worst <= 1, f"{what}: {worst} of the bound"


# ---- the router -------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (1, 8, 2), (3, 64, 64), (17, 60, 4), (64, 128, 8), (129, 129, 7),
                                                  (5, 256, 8), (33, 257, 64), (9, 512, 10), (4, 1000, 33), (2, 1024, 1)])
def test_route(dtype, tokens, experts, top_k):
    gen = gen_of("route", tokens, experts)
    logits = (2 * torch.randn(tokens, experts, generator=gen)).to(dtype).cuda()
    bias = 0.1 * torch.randn(experts, generator=gen).cuda()
    for b, scoring, renormalize, scale in [(None, "softmax", True, 1.0), (None, "softmax", False, 2.5),
                                           (None, "sigmoid", True, 2.5), (bias, "sigmoid", True, 1.0),
                                           (bias, "softmax", False, 1.0)]:
        banner(f"route {tokens} x {experts} top {top_k} {dtype} {scoring} bias {b is not None} renorm {renormalize}")
        w, e = qaff.moe_route(logits, top_k, bias=b, scoring=scoring, renormalize=renormalize, scale=scale)
        rw, re, bound = ref.route(logits, top_k, b, scoring, renormalize, scale)
        assert w.dtype == F32 and e.dtype == torch.int32
        assert torch.equal(e.cpu(), re)
        check(w, rw, bound)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_edges(scoring, biased):
    """Ties, switched-off experts, rows with none left, NaN, infinities and the type's lowest value."""
    inf, low = float("inf"), torch.finfo(BF16).min
    rows = [[1.0] * 8, [-inf] * 8, [-inf] * 6 + [2.0, 2.0], [float("nan")] * 8, [low] * 8, [low] * 7 + [0.0],
            [float("nan"), 3.0] * 4, [inf, 1.0, inf, 0.0, -inf, 0.0, 0.0, 0.0], [0.0, -0.0] * 4,
            [88.0, -88.0, 300.0, -300.0, 0.0, 1e30, -1e30, 5.0]]
    logits = torch.tensor(rows).to(BF16).cuda()
    bias = torch.tensor([0.0, 0.5, 0.0, 0.5, -0.5, 0.0, 0.25, 0.0]).cuda() if biased else None
    for renormalize in (True, False):
        w, e = qaff.moe_route(logits, 3, bias=bias, scoring=scoring, renormalize=renormalize)
        rw, re, bound = ref.route(logits, 3, bias, scoring, renormalize)
        assert torch.equal(e.cpu(), re)
        check(w, rw, bound + 1e-30)


def test_route_views_and_shapes():
    gen = gen_of("views")
    wide = torch.randn(7, 40, generator=gen).cuda()
    w, e = qaff.moe_route(wide[:, 3:35], 4)
    rw, re, bound = ref.route(wide[:, 3:35], 4)
    assert torch.equal(e.cpu(), re)
    check(w, rw, bound)
    w, e = qaff.moe_route(torch.randn(2, 3, 16, generator=gen).cuda(), 2)
    assert w.shape == e.shape == (2, 3, 2)
    for shape, k in [((0, 8), 2), ((3, 8), 0), ((0, 0), 0)]:
        w, e = qaff.moe_route(torch.zeros(shape).cuda(), k)
        assert w.shape == e.shape == (shape[0], k)


# ---- the layer of experts ---------------------------------------------------------------------------

def moe_inputs(gen, tokens, experts, top_k, hidden, width, bits, group, dtype, away=0.0):
    chosen = torch.rand(tokens, experts, generator=gen).argsort(-1)[:, :top_k].int()
    chosen[torch.rand(tokens, top_k, generator=gen) < away] = -1
    return dict(x=torch.randn(tokens, width, generator=gen).to(dtype).cuda(), experts=chosen.cuda(),
                weights=torch.rand(tokens, top_k, generator=gen).softmax(-1).cuda(),
                gate=ref.random_weight(gen, experts, hidden, width, bits, group, dtype),
                up=ref.random_weight(gen, experts, hidden, width, bits, group, dtype),
                down=ref.random_weight(gen, experts, width, hidden, bits, group, dtype), group=group, bits=bits)


def run_moe(i, resid=None, out=None):
    return qaff.moe_ffn(i["x"], i["experts"], i["weights"], i["gate"], i["up"], i["down"], i["group"], i["bits"],
                        resid=resid, out=out)


def check_moe(i, resid=None, what=""):
    y = run_moe(i, resid)
    want, bound = ref.moe(i["x"], i["experts"], i["weights"], i["gate"], i["up"], i["down"], i["group"], i["bits"], resid)
    check(y, want, bound, what)
    return y


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("bits", [1, 2, 3, 4, 5, 6, 8])
def test_moe_formats(dtype, group, bits):
    gen = gen_of("moe", group, bits)
    for tokens, experts, top_k, hidden, width in [(1, 4, 2, 128, 256), (1, 12, 3, 384, 640), (21, 3, 2, 384, 640),
                                                  (90, 3, 2, 384, 640)]:
        what = f"moe {bits} bits g{group} {dtype} {tokens} tokens {experts} experts [{hidden}, {width}]"
        banner(what)
        i = moe_inputs(gen, tokens, experts, top_k, hidden, width, bits, group, dtype)
        check_moe(i, resid=torch.randn(tokens, width, generator=gen).to(dtype).cuda(), what=what)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("tokens,experts,top_k,hidden,width,bits,group",
                         [(1, 1, 1, 32, 32, 4, 32), (2, 7, 3, 96, 160, 6, 32), (5, 16, 8, 64, 2080, 4, 32),
                          (40, 2, 1, 1408, 96, 3, 32), (64, 128, 8, 128, 256, 4, 64), (33, 1, 1, 256, 4096, 8, 128),
                          (300, 4, 2, 192, 320, 4, 64), (1000, 5, 3, 64, 128, 4, 64), (7, 60, 4, 352, 416, 5, 32),
                          (3, 2, 2, 128, 8192, 4, 64), (18, 2, 2, 9216, 128, 4, 128), (130, 300, 4, 64, 64, 2, 64), (700, 3, 1, 96, 160, 4, 32),
                          (193, 1, 1, 64, 128, 3, 64), (200, 4, 4, 32, 32, 4, 32), (250, 8, 2, 256, 2176, 6, 128),
                          (130, 5, 2, 1056, 288, 8, 32), (1, 128, 8, 768, 2048, 4, 64), (2, 64, 8, 96, 160, 5, 32),
                          (3, 48, 4, 1056, 288, 8, 32), (1, 300, 60, 64, 128, 3, 64), (1, 4, 1, 4096, 32, 4, 32),
                          (1, 9, 2, 4224, 128, 4, 128), (5, 160, 8, 32, 4160, 2, 32)])
def test_moe_sizes(dtype, tokens, experts, top_k, hidden, width, bits, group):
    gen = gen_of("sizes", tokens, experts, hidden)
    what = f"moe {tokens} tokens {top_k} of {experts} [{hidden}, {width}] {bits} bits g{group} {dtype}"
    banner(what)
    check_moe(moe_inputs(gen, tokens, experts, top_k, hidden, width, bits, group, dtype, away=0.2), what=what)


# ---- block quantization -----------------------------------------------------------------------------

def same_bits(a, b):
    return torch.equal(a.cpu().view(torch.uint8), b.cpu().view(torch.uint8))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 130), (128, 128), (129, 255), (300, 384), (257, 1000), (64, 4096),
                                       (1000, 64), (2, 9), (5, 7)])
def test_quantize(dtype, block_rows, rows, cols):
    gen = gen_of("quantize", rows, cols)
    x = torch.randn(rows, cols, generator=gen) * torch.exp(3 * torch.randn(rows, 1, generator=gen))
    x = x.to(dtype).cuda()
    banner(f"quantize {rows} x {cols} {dtype} blocks of {block_rows}")
    codes, scales = qaff.block_quantize(x, block_rows)
    rc, rs = ref.quantize(x, block_rows)
    assert same_bits(scales, rs)
    assert codes.dtype == torch.float8_e4m3fn and same_bits(codes, rc)


def test_quantize_borders():
    """Quotients on and beside the borders between two codes, the smallest codes, zeros, tiny and huge values."""
    gen = gen_of("borders")
    e = torch.arange(-9, 9).float()
    grid = torch.cat([2.0 ** e * (1 + i / 16) for i in range(16)])
    grid = torch.cat([grid, grid * (1 + 2.0 ** -23), grid * (1 - 2.0 ** -24), -grid])
    grid = grid[torch.randperm(grid.numel(), generator=gen)]
    rows = []
    for scale in (1.0, 2.0 ** -20, 0.3, 1e-30, 3e37, 1e-38, 2.0 ** -140):
        for part in grid.split(127):
            row = torch.zeros(128)
            row[:part.numel()] = part.clamp(-448, 448) * scale
            row[127] = 448 * scale if scale < 1e37 else 3.4e38
            rows.append(row)
    rows.append(torch.zeros(128))
    x = torch.stack(rows).cuda()
    codes, scales = qaff.block_quantize(x)
    rc, rs = ref.quantize(x)
    same = functools.partial(torch.testing.assert_close, rtol=0, atol=0, equal_nan=True)  # NaN where x is infinite
    same(scales.cpu(), rs)
    same(codes.cpu().float(), rc.float())
    codes, scales = qaff.block_quantize(torch.cat([x, x], 1), 128)
    rc, rs = ref.quantize(torch.cat([x, x], 1), 128)
    same(scales.cpu(), rs)
    same(codes.cpu().float(), rc.float())


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_not_finite(block_rows):
    x = torch.randn(256, 512, generator=gen_of("nan")).cuda()
    x[3, 5], x[4, 200], x[140, 300], x[141, 301] = float("nan"), float("inf"), -float("inf"), float("nan")
    codes, scales = qaff.block_quantize(x, block_rows)
    rc, rs = ref.quantize(x, block_rows)
    values = codes.cpu().float() * scales.cpu().repeat_interleave(block_rows, 0).repeat_interleave(128, 1)
    want = rc.float() * rs.repeat_interleave(block_rows, 0).repeat_interleave(128, 1)
    bad = want.isnan()
    assert bad.any() and torch.equal(values.isnan(), bad) and torch.equal(values[~bad], want[~bad])


def test_quantize_views_and_shapes():
    wide = torch.randn(9, 400, generator=gen_of("wide")).to(BF16).cuda()
    part = wide[:, 5:270]
    for block_rows in (1, 128):
        codes, scales = qaff.block_quantize(part, block_rows)
        rc, rs = ref.quantize(part, block_rows)
        assert same_bits(scales, rs) and same_bits(codes, rc)
    codes, scales = qaff.block_quantize(wide.view(3, 3, 400))
    assert codes.shape == (3, 3, 400) and scales.shape == (3, 3, 4)
    for shape in [(0, 256), (4, 0), (0, 0)]:
        codes, scales = qaff.block_quantize(torch.zeros(shape).cuda())
        assert codes.shape == shape and scales.shape == (shape[0], -(-shape[1] // 128))


# ---- the product ------------------------------------------------------------------------------------

def product_inputs(gen, m, n, k):
    x = qaff.block_quantize(torch.randn(m, k, generator=gen).cuda())
    w = qaff.block_quantize((torch.randn(n, k, generator=gen) / max(k, 1) ** 0.5).cuda(), 128)
    return x, w


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 128, 128), (1, 4096, 4096), (2, 130, 300), (15, 48, 4099), (16, 256, 512),
                                   (17, 200, 1000), (33, 384, 2048), (61, 1000, 640), (64, 512, 1536), (100, 129, 160),
                                   (128, 256, 384), (129, 257, 400), (200, 640, 3000), (256, 512, 4096), (300, 300, 129),
                                   (513, 1030, 1040), (1000, 64, 256), (1024, 1024, 1024), (7, 65, 16384)])
def test_product(dtype, m, n, k):
    (x, xs), (w, ws) = product_inputs(gen_of("product", m, n, k), m, n, k)
    what = f"product {m} x {n} x {k} {dtype}"
    banner(what)
    y = qaff.block_qmm(x, xs, w, ws, out_dtype=dtype)
    assert y.dtype == dtype
    many = m > 64 and k % 16 == 0 and dtype != F32  # on the 8-bit matrix instructions
    want, bound = ref.product(x, xs, w, ws, dtype, eights=many)
    check(y, want, bound, what=what)
    # all outputs together: the rounding's root mean square (half a step times sqrt(1/3)), 3e-5 for the sums
    rms = ((y.double() - want).norm() / want.norm()).item()
    assert y.numel() < 1000 or rms <= ref.HALF[dtype] * 0.58 + 3e-5
