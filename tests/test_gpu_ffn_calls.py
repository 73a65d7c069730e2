"""How the feed-forward operators are called on the GPU: together, captured and replayed, on another stream, with
values that are not finite, the same expert twice, empty routings, views and outputs between other memory."""
import pytest
import torch

import ffn_ref as ref
import quantized_matmul_mlx_amd as qaff
from gpu_util import banner
from test_gpu_ffn import BF16, F16, F32, check, gen_of, moe_inputs, product_inputs, run_moe

pytestmark = pytest.mark.gpu

# tokens for each way through the layer: pairs alone, few rows an expert, many
REGIMES = [(1, 16, 4), (24, 6, 3), (200, 4, 2)]


def block(x, router, layer, dense):
    """A decoder layer's feed-forward: an 8-bit projection, the router's logits, the routing and the experts."""
    x = dense.mm(x)
    weights, experts = qaff.moe_route(router.mm(x, out_dtype=F32), 3)
    y = qaff.moe_ffn(x, experts, weights, layer["gate"], layer["up"], layer["down"], layer["group"], layer["bits"], resid=x)
    return y, x, weights, experts


def block_parts(gen, experts=8, hidden=192, width=256):
    layer = moe_inputs(gen, 1, experts, 3, hidden, width, 4, 64, BF16)
    router = qaff.BlockWeight(*qaff.block_quantize((torch.randn(experts, width, generator=gen) / width ** 0.5).cuda(), 128))
    dense = qaff.BlockWeight(*qaff.block_quantize((torch.randn(width, width, generator=gen) / width ** 0.5).cuda(), 128))
    return layer, router, dense


@pytest.mark.parametrize("tokens", [1, 5, 40, 130, 300])
def test_together(tokens):
    gen = gen_of("together", tokens)
    layer, router, dense = block_parts(gen)
    x0 = torch.randn(tokens, 256, generator=gen).to(BF16).cuda()
    banner(f"a feed-forward block of {tokens} tokens")
    y, x, weights, experts = block(x0, router, layer, dense)
    codes, scales = ref.quantize(x0)
    want, bound = ref.product(codes.cuda(), scales.cuda(), dense.codes, dense.scales, BF16, eights=tokens > 64)
    check(x, want, bound, "projection")
    logits = router.mm(x, out_dtype=F32)
    rw, re, rb = ref.route(logits, 3)
    assert torch.equal(experts.cpu(), re)
    check(weights, rw, rb, "weights")
    want, bound = ref.moe(x, experts, weights, layer["gate"], layer["up"], layer["down"], 64, 4, x)
    check(y, want, bound, "layer")


@pytest.mark.parametrize("tokens", [1, 5, 40, 130, 300])
def test_captured(tokens):
    """Replays of a captured block on new inputs, the program's own work between them, against eager calls; and two
    graphs that share the allocator's memory."""
    gen = gen_of("captured", tokens)
    layer, router, dense = block_parts(gen)
    x = torch.randn(tokens, 256, generator=gen).to(BF16).cuda()
    inputs = [torch.randn(tokens, 256, generator=gen).to(BF16).cuda() for _ in range(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(x, router, layer, dense)
    torch.cuda.current_stream().wait_stream(side)
    banner(f"capture with {tokens} tokens")
    pool = torch.cuda.graph_pool_handle()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            out = block(x, router, layer, dense)
        graphs.append((g, out))
    for turn in range(4):
        src = inputs[turn % 3]
        want = [t.clone() for t in block(src, router, layer, dense)]
        torch.cuda.synchronize()
        for g, out in graphs:
            x.copy_(src)
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b)


@pytest.mark.parametrize("tokens", [5, 130])
def test_another_stream_and_two_at_once(tokens):
    gen = gen_of("streams", tokens)
    layer, router, dense = block_parts(gen)
    xs = [torch.randn(tokens, 256, generator=gen).to(BF16).cuda() for _ in range(2)]
    want = [block(x, router, layer, dense)[0].clone() for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(block(x, router, layer, dense)[0])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("tokens,experts,top_k", REGIMES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_moe_routings(tokens, experts, top_k, dtype):
    """The same expert twice in a token, all tokens at one expert, none anywhere, entries far outside, y into resid."""
    i = moe_inputs(gen_of("routings", tokens), tokens, experts, top_k, 160, 288, 4, 32, dtype)
    resid = torch.randn(tokens, 288, generator=gen_of("r", tokens)).to(dtype).cuda()
    for what, chosen in [("twice", torch.zeros(tokens, top_k) + torch.arange(top_k) // 2),
                         ("one", torch.full((tokens, top_k), experts - 1)), ("none", torch.full((tokens, top_k), -1)),
                         ("outside", torch.tensor([experts, -(2 ** 31), 2 ** 31 - 1, 0]).repeat(tokens)[:tokens * top_k]
                          .view(tokens, top_k))]:
        banner(f"moe {what} {tokens} tokens {dtype}")
        i["experts"] = chosen.int().cuda()
        want, bound = ref.moe(i["x"], i["experts"], i["weights"], i["gate"], i["up"], i["down"], 32, 4, resid)
        check(run_moe(i, resid), want, bound, what)
        out = resid.clone()
        assert run_moe(i, out, out=out) is out
        check(out, want, bound, what + " into resid")
    assert torch.equal(run_moe(i | dict(experts=i["experts"] * 0 - 1)), torch.zeros_like(resid))


@pytest.mark.parametrize("tokens,experts,top_k", REGIMES)
@pytest.mark.parametrize("group,bits", [(32, 4), (64, 6), (128, 4)])
def test_moe_not_finite_stays_in_its_row(tokens, experts, top_k, group, bits):
    """Infinite and NaN activations and weights of a token, and a NaN scale of an expert, reach only what they enter."""
    i = moe_inputs(gen_of("nan", tokens, group), tokens, experts, top_k, 256, 384, bits, group, BF16)
    clean = run_moe(i)
    bad = torch.zeros(tokens, dtype=torch.bool)
    if tokens > 3:
        i["x"][1, 5], i["x"][2, 383], i["weights"][3, 0] = float("nan"), float("inf"), float("nan")
        bad[1:4] = True
    i["down"][1][experts - 1, 7, 0] = float("nan")
    banner(f"not finite, {tokens} tokens g{group}")
    y = run_moe(i)
    uses = (i["experts"] == experts - 1).any(-1).cpu()
    good = ~bad
    assert torch.equal(y[good & ~uses], clean[good & ~uses])
    if (good & uses).any():
        rows = y[good & uses].cpu()
        assert rows[:, 7].isnan().all() and not rows[:, :7].isnan().any() and not rows[:, 8:].isnan().any()
    if tokens > 3:
        assert y[1].isnan().any() and not y[2].isfinite().all() and y[3].isnan().all()


@pytest.mark.parametrize("bits", [3, 4, 8])
@pytest.mark.parametrize("tokens,experts,top_k", REGIMES)
def test_moe_scales_of_any_size(tokens, experts, top_k, bits):
    """Scales and biases (and activations) far from 1: each row of a weight and of x keeps its precision."""
    i = moe_inputs(gen_of("scales", tokens, bits), tokens, experts, top_k, 128, 192, bits, 32, BF16)
    for name, power in (("gate", -20), ("up", 12), ("down", 30)):
        w, s, b = i[name]
        row = torch.exp2(torch.randint(-6, 7, s.shape[:2], generator=gen_of(name)).float()).cuda()[..., None] * 2.0 ** power
        i[name] = (w, (s * row).to(BF16), (b * row).to(BF16))
    i["x"] = (i["x"].float() * torch.exp2(torch.randint(-30, 20, (tokens, 1), generator=gen_of("x")).float()).cuda()).to(BF16)
    want, bound = ref.moe(i["x"], i["experts"], i["weights"], i["gate"], i["up"], i["down"], 32, bits)
    check(run_moe(i), want, bound, f"{bits} bits {tokens} tokens")


@pytest.mark.parametrize("bits,group,hidden,width", [(4, 32, 1056, 1536), (4, 32, 1536, 1664), (2, 32, 3040, 1056), (6, 64, 2112, 3840),
                                                     (4, 64, 4096, 2176), (8, 64, 3904, 2112), (3, 128, 4224, 7680), (5, 128, 7808, 4096)])
@pytest.mark.parametrize("tokens", [70, 420])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_moe_many_rows_of_many_groups(bits, group, hidden, width, tokens, dtype):
    """Rows of more groups than the GEMM holds at a time (32), up to and past the borders of what it holds; scales of
    each row grow towards its end, where its largest stands."""
    i = moe_inputs(gen_of("groups", bits, group, hidden, tokens), tokens, 3, 1, hidden, width, bits, group, dtype)
    for name in ("gate", "up", "down"):
        w, s, b = i[name]
        grow = torch.linspace(-3, 1, s.shape[-1], device="cuda").exp2()
        i[name] = (w, (s * grow).to(dtype), (b * grow).to(dtype))
    banner(f"moe {bits} bits g{group} {hidden} x {width}, {tokens} tokens {dtype}")
    want, bound = ref.moe(i["x"], i["experts"], i["weights"], i["gate"], i["up"], i["down"], group, bits)
    check(run_moe(i), want, bound, f"{bits} bits g{group}")


@pytest.mark.parametrize("tokens,experts,top_k", REGIMES)
def test_moe_same_result_each_time_and_nothing_else_written(tokens, experts, top_k):
    i = moe_inputs(gen_of("again", tokens), tokens, experts, top_k, 160, 288, 5, 32, F16)
    buffer = torch.full((tokens + 2, 288), 7.0, dtype=F16, device="cuda")
    first = run_moe(i)
    for _ in range(3):
        run_moe(i, out=buffer[1:-1])
        assert torch.equal(buffer[1:-1], first)
        assert (buffer[0] == 7).all() and (buffer[-1] == 7).all()


@pytest.mark.parametrize("tokens,experts,top_k", REGIMES)
def test_moe_operands_at_odd_addresses(tokens, experts, top_k):
    """x, resid, y, scales and biases 2 bytes past a 16-byte address, codes 4."""
    def shifted(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
        buf[1:].copy_(t.reshape(-1))
        return buf[1:].view(t.shape)
    i = moe_inputs(gen_of("odd", tokens), tokens, experts, top_k, 160, 288, 6, 32, BF16)
    resid = torch.randn(tokens, 288, generator=gen_of("odd")).to(BF16).cuda()
    want = run_moe(i, resid)
    moved = {k: tuple(shifted(t) for t in v) if isinstance(v, tuple) else shifted(v) if torch.is_tensor(v) else v
             for k, v in i.items()}
    out = shifted(torch.zeros_like(resid))
    assert torch.equal(run_moe(moved, shifted(resid), out=out), want)


@pytest.mark.parametrize("m", [1, 16, 17, 33, 64, 65, 128, 200, 600])
@pytest.mark.parametrize("k", [1024, 1040, 1001])
def test_product_calls(m, k):
    """The same result each time, nothing written beside y, rows at odd addresses, NaN codes and scales in their rows."""
    n = 272
    (x, xs), (w, ws) = product_inputs(gen_of("calls", m, k), m, n, k)
    y = qaff.block_qmm(x, xs, w, ws)
    buffer = torch.full((m + 2, n), 7.0, dtype=BF16, device="cuda")
    banner(f"product {m} x {n} x {k}")
    qaff.block_qmm(x, xs, w, ws, out=buffer[1:-1])
    assert torch.equal(buffer[1:-1], y) and (buffer[0] == 7).all() and (buffer[-1] == 7).all()
    odd = torch.empty(x.numel() + 3, dtype=torch.uint8, device="cuda")[3:].view(x.shape)
    odd.copy_(x.view(torch.uint8))
    want, bound = ref.product(x, xs, w, ws, BF16)
    check(qaff.block_qmm(odd.view(torch.float8_e4m3fn), xs, w, ws), want, bound, "odd address")
    nan, inf = x.clone(), xs.clone()
    nan.view(torch.uint8)[m - 1, k - 1] = 0x7F
    got = qaff.block_qmm(nan, xs, w, ws)
    assert got[m - 1].isnan().all() and torch.equal(got[:m - 1], y[:m - 1])
    inf[0, 0] = float("inf")
    got = qaff.block_qmm(x, inf, w, ws)
    assert not got[0].isfinite().any() and torch.equal(got[1:], y[1:])
    wn = w.clone()
    wn.view(torch.uint8)[n - 1, 0] = 0xFF
    got = qaff.block_qmm(x, xs, wn, ws)
    assert got[:, n - 1].isnan().all() and torch.equal(got[:, :n - 1], y[:, :n - 1])


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("m,n,k", [(17, 8200, 16), (20, 8193, 128), (33, 8200, 272), (61, 9000, 384), (64, 16385, 400), (18, 20000, 640),
                                   (65, 200, 144), (66, 129, 896), (128, 300, 1920), (70, 4096, 256), (768, 600, 528)])
def test_product_split(dtype, m, n, k):
    """Few rows against wide weights, and small products: K in two parts, down to one block and to a part without any."""
    (x, xs), (w, ws) = product_inputs(gen_of("split", m, n, k), m, n, k)
    banner(f"product {m} x {n} x {k} {dtype}")
    y = qaff.block_qmm(x, xs, w, ws, out_dtype=dtype)
    want, bound = ref.product(x, xs, w, ws, dtype, eights=dtype != F32)
    check(y, want, bound, f"{m} x {n} x {k}")
    rms = ((y.double() - want).norm() / want.norm()).item()
    assert rms <= ref.HALF[dtype] * 0.58 + 3e-5
    nan = x.clone()
    nan.view(torch.uint8)[m - 1, k - 1] = 0x7F
    got = qaff.block_qmm(nan, xs, w, ws, out_dtype=dtype)
    assert got[m - 1].isnan().all() and torch.equal(got[:m - 1], y[:m - 1])
    scales = xs.clone()
    scales[1, 0] = float("inf")
    got = qaff.block_qmm(x, scales, w, ws, out_dtype=dtype)
    assert not got[1].isfinite().any() and torch.equal(got[2:], y[2:]) and torch.equal(got[0], y[0])


def test_product_shapes():
    (x, xs), (w, ws) = product_inputs(gen_of("shapes"), 6, 130, 300)
    y = qaff.block_qmm(x, xs, w, ws)
    assert torch.equal(qaff.block_qmm(x.view(2, 3, 300), xs.view(2, 3, 3), w, ws), y.view(2, 3, 130))
    assert torch.equal(qaff.block_qmm(x[0], xs[0], w, ws), y[0])
    f8 = torch.float8_e4m3fn
    for m, n, k in [(0, 4, 128), (3, 0, 128), (3, 4, 0)]:
        got = qaff.block_qmm(torch.empty(m, k, dtype=f8).cuda(), torch.ones(m, -(-k // 128)).cuda(),
                             torch.empty(n, k, dtype=f8).cuda(), torch.ones(-(-n // 128), -(-k // 128)).cuda(), out_dtype=F32)
        assert got.shape == (m, n) and (got == 0).all()


def test_refusals():
    i = moe_inputs(gen_of("refuse"), 3, 4, 2, 64, 128, 4, 32, BF16)
    for change, kind in [(dict(x=i["x"].float()), TypeError), (dict(x=i["x"].half()), TypeError),
                         (dict(x=i["x"][:, ::2]), ValueError), (dict(experts=i["experts"].long()), TypeError),
                         (dict(experts=i["experts"][:2]), ValueError), (dict(weights=i["weights"].double()), TypeError),
                         (dict(group=48), ValueError), (dict(bits=7), ValueError), (dict(bits=5), ValueError),
                         (dict(up=i["down"]), ValueError), (dict(gate=i["gate"][:2]), TypeError),
                         (dict(x=i["x"][:, :96].contiguous()), ValueError)]:
        with pytest.raises(kind):
            run_moe(i | change)
    with pytest.raises(ValueError):
        run_moe(i, resid=i["x"][:1])
    with pytest.raises(ValueError):
        run_moe(i, out=torch.empty(3, 64, dtype=BF16, device="cuda"))
    (x, xs), (w, ws) = product_inputs(gen_of("refuse"), 3, 64, 256)
    for args in [(x[:, :128], xs, w, ws), (x, xs[:, :1], w, ws), (x, xs, w, ws.repeat(2, 1)), (x, xs, w[:, :128].contiguous(), ws)]:
        with pytest.raises(ValueError):
            qaff.block_qmm(*args)
    with pytest.raises(TypeError):
        qaff.block_qmm(x, xs, w, ws, out_dtype=torch.int8)
    with pytest.raises(TypeError):
        qaff.block_qmm(x.view(torch.uint8), xs, w, ws)
    with pytest.raises(ValueError):
        qaff.block_quantize(torch.zeros(4, 8).cuda(), 64)
    with pytest.raises(ValueError):
        qaff.block_quantize(torch.zeros(4, 8).cuda().T)
    with pytest.raises(TypeError):
        qaff.block_quantize(torch.zeros(4, 8, dtype=torch.int8).cuda())
    with pytest.raises(ValueError):
        qaff.moe_route(torch.zeros(4, 8).cuda(), 9)
    with pytest.raises(ValueError):
        qaff.moe_route(torch.zeros(4, 8).cuda(), 2, bias=torch.zeros(7).cuda())
    with pytest.raises(qaff.QaffError):
        qaff.moe_route(torch.zeros(4, 1025).cuda(), 2)
