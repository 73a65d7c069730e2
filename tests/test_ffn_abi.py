"""The feed-forward operators' refusals, on the CPU: every case fails validation, or is a no-op that returns
before any launch. The binding refuses CPU tensors and shapes that do not fit."""
import os

import pytest
import torch

import quantized_matmul_mlx_amd as qaff
from quantized_matmul_mlx_amd import _lib

OK, INVALID, UNSUPPORTED = _lib.QAFF_OK, _lib.QAFF_ERR_INVALID_ARGUMENT, _lib.QAFF_ERR_UNSUPPORTED
A, ODD = 0x10000, 0x10001
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from quantized_matmul_mlx_amd import build
        build.build()
    return _lib.load()


def route(lib, **kw):
    a = dict(logits=A, dtype=_lib.QAFF_BF16, tokens=3, experts=8, stride=8, bias=None, sigmoid=0, top_k=2, renorm=1,
             scale=1.0, weights=A, chosen=A)
    assert not set(kw) - set(a)
    return lib.qaff_moe_route(*{**a, **kw}.values(), None)


def moe(lib, **kw):
    a = dict(x=A, dtype=_lib.QAFF_BF16, tokens=3, width=128, hidden=64, chosen=A, weights=A, top_k=2, experts=4, gp=A,
             gs=A, gb=A, up=A, us=A, ub=A, dp=A, ds=A, db=A, group=32, bits=4, resid=None, ws=A, ws_bytes=1 << 40, y=A)
    assert not set(kw) - set(a)
    return lib.qaff_moe_ffn(*{**a, **kw}.values(), None)


def quantize(lib, **kw):
    a = dict(x=A, dtype=_lib.QAFF_BF16, rows=3, cols=200, stride=200, block_rows=1, codes=A, scales=A)
    assert not set(kw) - set(a)
    return lib.qaff_block_quantize(*{**a, **kw}.values(), None)


def product(lib, **kw):
    a = dict(x=A, xs=A, m=3, w=A, ws=A, n=64, k=256, y=A, dtype=_lib.QAFF_BF16)
    assert not set(kw) - set(a)
    return lib.qaff_block_qmm(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("kw", [dict(dtype=9), dict(tokens=-1), dict(experts=-1), dict(stride=-1), dict(top_k=-1),
                                dict(top_k=9), dict(scale=NAN), dict(scale=INF), dict(logits=None), dict(weights=None),
                                dict(chosen=None), dict(logits=ODD), dict(weights=A + 2), dict(chosen=A + 2), dict(bias=A + 2),
                                dict(dtype=_lib.QAFF_F32, logits=A + 2)], ids=str)
def test_route_invalid(lib, kw):
    assert route(lib, **kw) == INVALID
    assert b"qaff_moe_route" in lib.qaff_last_error()


def test_route_unsupported(lib):
    assert route(lib, experts=1025) == UNSUPPORTED
    assert route(lib, experts=1024, top_k=65) == UNSUPPORTED
    assert route(lib, tokens=2**26) == UNSUPPORTED
    assert route(lib, stride=2**32) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(dtype=_lib.QAFF_F32), dict(dtype=9), dict(tokens=-1), dict(width=-128), dict(hidden=-64),
                                dict(top_k=-1), dict(experts=-1), dict(group=0), dict(group=16), dict(group=256),
                                dict(width=144), dict(hidden=48), dict(group=64, hidden=96), dict(x=None), dict(chosen=None),
                                dict(weights=None), dict(y=None), dict(ws=None), dict(ws_bytes=16), dict(x=ODD), dict(y=ODD),
                                dict(resid=ODD), dict(chosen=A + 2), dict(weights=A + 2), dict(ws=A + 8), dict(gp=None),
                                dict(up=None), dict(dp=None), dict(gs=None), dict(us=None), dict(ds=None), dict(gb=None),
                                dict(ub=None), dict(db=None), dict(gp=A + 2), dict(ds=ODD), dict(ub=ODD)], ids=str)
def test_moe_invalid(lib, kw):
    assert moe(lib, **kw) == INVALID
    assert b"qaff_moe_ffn" in lib.qaff_last_error()


@pytest.mark.parametrize("kw", [dict(bits=0), dict(bits=7), dict(bits=9), dict(bits=-4), dict(width=32768 + 32),
                                dict(hidden=32768 + 32), dict(experts=65536), dict(tokens=2**31), dict(tokens=2**30, top_k=2),
                                dict(top_k=65536), dict(tokens=2**30, top_k=1, width=2**14), dict(tokens=2**62, top_k=4)], ids=str)
def test_moe_unsupported(lib, kw):
    assert moe(lib, **kw) == UNSUPPORTED


def test_moe_workspace(lib):
    size = lib.qaff_moe_ffn_workspace_size
    assert size(1, 128, 64, 2, 4, 32, 4) > 0
    for args in [(-1, 128, 64, 2, 4, 32, 4), (1, 130, 64, 2, 4, 32, 4), (1, 128, 64, 2, 4, 33, 4), (1, 128, 64, 2, 4, 32, 7),
                 (0, 128, 64, 2, 4, 32, 4), (1, 128, 64, 0, 4, 32, 4), (1, 128, 64, 2, 0, 32, 4), (2**40, 128, 64, 2, 4, 32, 4)]:
        assert size(*args) == 0
    need = size(3, 128, 64, 2, 4, 32, 4)
    assert moe(lib, ws_bytes=need - 1) == INVALID and b"workspace" in lib.qaff_last_error()


@pytest.mark.parametrize("kw", [dict(dtype=9), dict(rows=-1), dict(cols=-1), dict(stride=-1), dict(block_rows=0),
                                dict(block_rows=64), dict(block_rows=-128), dict(stride=199), dict(x=None), dict(codes=None),
                                dict(scales=None), dict(x=ODD), dict(scales=A + 2), dict(dtype=_lib.QAFF_F32, x=A + 2)], ids=str)
def test_quantize_invalid(lib, kw):
    assert quantize(lib, **kw) == INVALID
    assert b"qaff_block_quantize" in lib.qaff_last_error()


@pytest.mark.parametrize("kw", [dict(rows=2**27), dict(rows=2**32), dict(cols=2**31, stride=2**31), dict(rows=2**62),
                                dict(stride=2**31)], ids=str)
def test_quantize_unsupported(lib, kw):
    assert quantize(lib, **kw) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(dtype=9), dict(m=-1), dict(n=-1), dict(k=-1), dict(x=None), dict(xs=None), dict(w=None),
                                dict(ws=None), dict(y=None), dict(xs=A + 2), dict(ws=A + 2), dict(y=ODD),
                                dict(dtype=_lib.QAFF_F32, y=A + 2)], ids=str)
def test_product_invalid(lib, kw):
    assert product(lib, **kw) == INVALID
    assert b"qaff_block_qmm" in lib.qaff_last_error()


@pytest.mark.parametrize("kw", [dict(m=2**31), dict(n=2**28), dict(k=2**18 + 1), dict(k=2**62)], ids=str)
def test_product_unsupported(lib, kw):
    assert product(lib, **kw) == UNSUPPORTED


def test_empty_calls(lib):
    """Sizes of zero: nothing is launched and no pointer is looked at."""
    assert route(lib, tokens=0, logits=None, weights=None, chosen=None) == OK
    assert route(lib, top_k=0, logits=None, weights=None, chosen=None) == OK
    assert moe(lib, tokens=0, x=None, y=None, ws=None) == OK
    assert moe(lib, width=0, x=None, y=None, ws=None) == OK
    assert quantize(lib, rows=0, x=None, codes=None, scales=None) == OK
    assert quantize(lib, cols=0, x=None, codes=None, scales=None) == OK
    assert product(lib, m=0, x=None, y=None) == OK
    assert product(lib, n=0, w=None, y=None) == OK


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    e = torch.zeros(2, 2, dtype=torch.int32)
    w = (torch.zeros(4, 64, 8, dtype=torch.int32), x, x)
    with pytest.raises(ValueError, match="GPU"):
        qaff.moe_route(x, 2)
    with pytest.raises(ValueError, match="GPU"):
        qaff.moe_ffn(x, e, e.float(), w, w, w, 32, 4)
    with pytest.raises(ValueError, match="GPU"):
        qaff.block_quantize(x)
    f8 = x.to(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="GPU"):
        qaff.block_qmm(f8, x.float(), f8, x.float())
    with pytest.raises(TypeError, match="torch.Tensor"):
        qaff.block_quantize(3)
    with pytest.raises(ValueError, match="scoring"):
        qaff.moe_route(x, 2, scoring="relu")
    with pytest.raises(ValueError, match="scales"):
        qaff.BlockWeight(f8, torch.zeros(2, 1))
