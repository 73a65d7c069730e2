"""The paged-cache operators' refusals, on the CPU: every case fails validation, or is a no-op that
returns before any launch. The binding refuses CPU tensors and shapes that do not fit."""
import ctypes
import math
import os

import pytest
import torch

import quantized_matmul_mlx_amd as qaff
from quantized_matmul_mlx_amd import _lib

OK, INVALID, UNSUPPORTED = _lib.QAFF_OK, _lib.QAFF_ERR_INVALID_ARGUMENT, _lib.QAFF_ERR_UNSUPPORTED
A, ODD = 0x10000, 0x10001


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from quantized_matmul_mlx_amd import build
        build.build()
    return _lib.load()


def plan(lib, **kw):
    a = dict(cached=A, new=A, requests=2, free=A, n_free=4, tables=A, width=3, page=16, tokens=5, cu=A, kv=A, pos=A,
             slots=A, used=A)
    assert not set(kw) - set(a)
    return lib.qaff_paged_plan(*{**a, **kw}.values(), None)


def rope(lib, **kw):
    a = dict(q=A, k=A, v=A, dtype=_lib.QAFF_BF16, tokens=3, heads=4, kv_heads=2, dim=64, q_ts=256, q_hs=64, k_ts=128,
             k_hs=64, v_ts=128, v_hs=64, positions=A, axes=1, sections=None, interleaved=0, traditional=0, inv=A, rot=64,
             slots=A, k_cache=A, v_cache=A, pages=4, page_stride=2048, page=16, out=A)
    assert not set(kw) - set(a)
    a.update(kw)
    if a["sections"] is not None:
        a["sections"] = (ctypes.c_int32 * len(a["sections"]))(*a["sections"])
    return lib.qaff_rope_append(*a.values(), None)


def attention(lib, **kw):
    a = dict(q=A, dtype=_lib.QAFF_F16, tokens=3, heads=4, q_ts=256, q_hs=64, k_cache=A, v_cache=A, pages=4,
             page_stride=2048, kv_heads=2, dim=64, page=16, tables=A, width=3, cu=A, kv=A, requests=2, max_new=3,
             scale=0.125, causal=1, window=0, ws=A, ws_bytes=1 << 40, out=A, lse=None)
    assert not set(kw) - set(a)
    return lib.qaff_paged_attention(*{**a, **kw}.values(), None)


@pytest.mark.parametrize("call", [plan, rope, attention])
@pytest.mark.parametrize("page", [-16, 0, 1, 4, 12, 24, 512])
def test_page_sizes(lib, call, page):
    assert call(lib, page=page) == UNSUPPORTED
    assert b"page size" in lib.qaff_last_error()


@pytest.mark.parametrize("kw", [dict(requests=-1), dict(n_free=-1), dict(width=-1), dict(tokens=-1), dict(cached=None),
                                dict(new=None), dict(free=None), dict(tables=None), dict(cu=None), dict(kv=None),
                                dict(pos=None), dict(slots=None), dict(used=None), dict(cached=ODD), dict(new=ODD),
                                dict(free=ODD), dict(tables=ODD), dict(cu=ODD), dict(kv=ODD), dict(pos=ODD),
                                dict(slots=A + 4), dict(used=ODD)], ids=str)
def test_plan_invalid(lib, kw):
    assert plan(lib, **kw) == INVALID
    assert b"qaff_paged_plan" in lib.qaff_last_error()


def test_plan_unsupported(lib):
    assert plan(lib, requests=16385) == UNSUPPORTED
    assert plan(lib, tokens=2**31) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(dtype=_lib.QAFF_F32), dict(dtype=9), dict(tokens=-1), dict(heads=-1),
                                dict(kv_heads=-1), dict(dim=-1), dict(q_ts=-1), dict(q_hs=-1), dict(k_ts=-1),
                                dict(k_hs=-1), dict(v_ts=-1), dict(v_hs=-1), dict(rot=63), dict(rot=66), dict(rot=-2),
                                dict(axes=0), dict(axes=5), dict(axes=2), dict(axes=2, sections=(16, 15)),
                                dict(axes=2, sections=(33, -1)), dict(axes=1, sections=(31,)),
                                dict(axes=3, sections=(8, 12, 12), interleaved=1), dict(pages=-1), dict(page_stride=-1),
                                dict(page_stride=2047), dict(q=None), dict(k=None), dict(v=None), dict(positions=None),
                                dict(inv=None), dict(slots=None), dict(k_cache=None), dict(v_cache=None), dict(out=None),
                                dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(positions=A + 2), dict(inv=A + 2),
                                dict(slots=A + 4), dict(k_cache=ODD), dict(v_cache=ODD), dict(out=ODD)], ids=str)
def test_rope_invalid(lib, kw):
    assert rope(lib, **kw) == INVALID
    assert b"qaff_rope_append" in lib.qaff_last_error()


def test_rope_unsupported_and_no_ops(lib):
    assert rope(lib, dim=514, q_hs=514, page_stride=1 << 20) == UNSUPPORTED
    assert rope(lib, tokens=2**31) == UNSUPPORTED
    assert rope(lib, pages=2**31) == UNSUPPORTED
    assert rope(lib, tokens=0, q=None, k=None, v=None, positions=None, slots=None, out=None) == OK
    assert rope(lib, heads=0, kv_heads=0, q=None) == OK


@pytest.mark.parametrize("kw", [dict(dtype=_lib.QAFF_F32), dict(dtype=-1), dict(tokens=-1), dict(heads=-1),
                                dict(kv_heads=-1), dict(kv_heads=0), dict(kv_heads=3), dict(dim=-1), dict(requests=-1),
                                dict(width=-1), dict(window=-1), dict(max_new=-1), dict(q_ts=-1), dict(q_hs=-1),
                                dict(pages=-1), dict(page_stride=2047), dict(scale=0.0), dict(scale=-1.0),
                                dict(scale=math.inf), dict(scale=math.nan), dict(q=None), dict(k_cache=None),
                                dict(v_cache=None), dict(tables=None), dict(cu=None), dict(kv=None), dict(out=None),
                                dict(q=ODD), dict(k_cache=ODD), dict(v_cache=ODD), dict(tables=ODD), dict(cu=ODD),
                                dict(kv=ODD), dict(out=ODD), dict(lse=ODD)], ids=str)
def test_attention_invalid(lib, kw):
    assert attention(lib, **kw) == INVALID
    assert b"qaff_paged_attention" in lib.qaff_last_error()


def test_attention_unsupported_and_no_ops(lib):
    assert attention(lib, dim=264, page_stride=1 << 20) == UNSUPPORTED
    assert attention(lib, requests=65537) == UNSUPPORTED
    assert attention(lib, tokens=2**29) == UNSUPPORTED
    assert attention(lib, width=2**27) == UNSUPPORTED
    assert attention(lib, width=2**26) == UNSUPPORTED
    assert attention(lib, pages=2**31) == UNSUPPORTED
    assert attention(lib, tokens=0, q=None, out=None) == OK
    assert attention(lib, heads=0, kv_heads=0, q=None, out=None) == OK


def test_grids_that_no_launch_holds(lib):
    # 2^32 threads or more: refused before any launch
    assert rope(lib, tokens=2**24) == UNSUPPORTED                                       # a workgroup of 256 a token
    assert rope(lib, tokens=2**24, dim=62, rot=62, q_ts=248, q_hs=62) == UNSUPPORTED    # element by element
    assert b"2^32" in lib.qaff_last_error()
    assert attention(lib, tokens=2**24, dim=62, q_ts=248, q_hs=62) == UNSUPPORTED       # a wave a row
    assert b"2^32" in lib.qaff_last_error()


def test_attention_workspace(lib):
    size = lib.qaff_paged_attention_workspace_size
    for bad in ((-1, 8, 2, 64, 16, 3, 2, 1), (3, 8, 3, 64, 16, 3, 2, 1), (3, 8, 2, 300, 16, 3, 2, 1),
                (3, 8, 2, 64, 17, 3, 2, 1), (3, 8, 2, 64, 16, 3, 70000, 1)):
        assert size(*bad) == 0
    need = size(2, 8, 2, 64, 16, 4096, 2, 1)
    big = dict(tokens=2, heads=8, kv_heads=2, width=4096, max_new=1)
    if need:
        assert attention(lib, **big, ws_bytes=need - 1) == INVALID
        assert attention(lib, **big, ws=None, ws_bytes=need) == INVALID
        assert attention(lib, **big, ws=A + 8, ws_bytes=need) == INVALID


def test_binding_refuses_cpu_tensors_and_other_types():
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        qaff.paged_plan(i32, i32, i32, i32[None], 16, 4)
    x = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    cache = torch.zeros(2, 4, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        qaff.rope_append(x, x, x, i32, torch.zeros(32), torch.zeros(3, dtype=torch.int64), cache, cache)
    with pytest.raises(ValueError, match="GPU"):
        qaff.paged_attention(x, cache, cache, i32[None], i32, i32)
    with pytest.raises(TypeError):
        qaff.paged_attention([1.0], cache, cache, i32[None], i32, i32)
