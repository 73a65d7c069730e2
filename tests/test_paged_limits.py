"""Sizes of a paged cache whose product leaves 64 bits are refused, on the CPU."""
import pytest

from quantized_matmul_mlx_amd import _lib
from test_paged_abi import attention, lib, rope  # noqa: F401


@pytest.mark.parametrize("kv_heads", [2**31, 2**46, 2**60, 2**63 - 1])
def test_cache_heads(lib, kv_heads):  # noqa: F811
    # 2^46 heads of 256 values in pages of 256: 2^62 elements a page; 2^60: 2^76, which wraps to 0
    assert attention(lib, heads=0, kv_heads=kv_heads, dim=256, page=256, page_stride=2**62) == _lib.QAFF_ERR_UNSUPPORTED
    assert b"cache heads" in lib.qaff_last_error()
    assert rope(lib, heads=0, kv_heads=kv_heads, page_stride=2**62) == _lib.QAFF_ERR_UNSUPPORTED


def test_cache_heads_without_query_heads(lib):  # noqa: F811
    assert attention(lib, heads=0, kv_heads=2**31 - 1, pages=1) == _lib.QAFF_OK
    assert attention(lib, heads=0, kv_heads=2**31 - 1) == _lib.QAFF_ERR_INVALID_ARGUMENT  # pages overlap
