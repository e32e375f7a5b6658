"""What the cached chain and the operators around the cache refuse beyond
missing and misaligned arrays, on the host: sizes that a kernel behind the
entry point does not cover, and operands that lie in one another."""
import ctypes

import pytest

from tests.test_kv_host import NULL, SHAPE, addr, api  # noqa: F401  (api: the fixture)


@pytest.mark.parametrize("hidden,status", [(32768, NULL), (32896, SHAPE), (65536, SHAPE)])
def test_cached_chain_refuses_rows_past_the_norms(api, hidden, status):  # noqa: F811
    """Up to 32768 columns the missing tables are what is refused."""
    buf = api.ChainBuffers(*[addr(i) for i in range(1, 10)], 2, hidden, 128, 64, 512)
    c = api.ChainCache(x=addr(10), q=addr(11), k=addr(12))
    layers, cached = (api.ChainLayer * 1)(), (api.CachedLayer * 1)()
    rc = api.tw_decoder_chain_cached(layers, cached, 1, ctypes.byref(buf), ctypes.byref(c), addr(13), 1 << 30, None)
    assert rc == status, api.tw_last_error()
    assert status != SHAPE or b"hidden" in api.tw_last_error()
