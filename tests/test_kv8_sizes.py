"""Sizes that the 8-bit cache's write and read do not take, refused before any device work
(no GPU; the pointers are made up and never followed)."""
import pytest

from autoregressive_tts_decode_gb300 import q3tts
from tests.test_kv8_abi import cache, lib, read, write  # noqa: F401


@pytest.mark.parametrize("fn", [write, read])
@pytest.mark.parametrize("heads,page", [(8, 1 << 27), (1, 1 << 30), (1 << 20, 1 << 10)])
def test_pages_of_more_than_32_bits_of_rows(lib, fn, heads, page):  # noqa: F811
    kv = cache(n_kv_heads=heads, page_size=page, block=16, n_pages=2)
    assert fn(lib, kv, pps=1, lda=heads * 64, ldb=heads * 64, b=1 << 46) == q3tts.ERR_UNSUPPORTED


@pytest.mark.parametrize("hd,block", [(128, 1 << 24), (64, 1 << 25)])
def test_blocks_of_more_than_32_bits_of_codes(lib, hd, block):  # noqa: F811
    kv = cache(n_kv_heads=1, page_size=block, block=block, n_pages=1, head_dim=hd)
    assert write(lib, kv, pps=1) == q3tts.ERR_UNSUPPORTED
