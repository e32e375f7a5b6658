"""What the cache operators and the residual norms refuse, on the host: the C
entry points check their arguments before they touch a device."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def api():
    from ternary_weight_decoder_b200 import build
    build.build()
    from ternary_weight_decoder_b200 import api as a
    return a


NULL, SHAPE, ALIGN, BUFSIZE, NONFINITE, UNSUPPORTED = 1, 2, 3, 4, 5, 9
A = 0x10000000   # addresses, 256 MB apart; nothing is read there


def addr(i):
    return A + i * 0x10000000


def cache(api, **over):
    f = dict(k=addr(1), v=addr(2), k_scale=None, v_scale=None, num_pages=10, page_size=16, kv_heads=2,
             head_dim=128, page_stride=16 * 256, token_stride=256, head_stride=128, dtype=0)
    f.update(over)
    return api.KVCacheStruct(**f)


ASSIGN = dict(lengths=addr(1), delta=addr(2), requests=4, page_size=16, block_table=addr(3), max_pages=8,
              table_stride=8, free_pages=addr(4), free_capacity=32, free_count=addr(5), lengths_out=addr(6),
              free_count_out=addr(7), slots=addr(8), positions=addr(9), request_of_row=addr(10), rows=64,
              row_start=addr(11), stream=None)


@pytest.mark.parametrize("bad,status", [
    (dict(lengths=None), NULL), (dict(slots=None), NULL), (dict(requests=0), SHAPE), (dict(requests=8193), SHAPE),
    (dict(page_size=0), SHAPE), (dict(table_stride=7), SHAPE), (dict(rows=-1), SHAPE), (dict(free_capacity=0), SHAPE),
    (dict(max_pages=0), SHAPE), (dict(lengths=addr(1) + 2), ALIGN), (dict(delta=addr(6)), SHAPE),
    (dict(slots=addr(9) + 16), SHAPE), (dict(lengths_out=addr(1) + 4), SHAPE), (dict(free_pages=addr(3) + 64), SHAPE),
    (dict(row_start=addr(8) + 4), SHAPE), (dict(free_count_out=addr(4)), SHAPE), (dict(delta=addr(1)), None)])
def test_assign_refuses(api, bad, status):
    rc = api.tw_kv_assign(*dict(ASSIGN, **bad).values())
    assert rc == status if status else rc != 0, api.tw_last_error()
    assert rc == 0 or api.tw_last_error()


def test_assign_may_work_in_place(api):
    """lengths_out = lengths and free_count_out = free_count pass the checks
    (what is left to fail here is the device)."""
    args = dict(ASSIGN, lengths_out=addr(1), free_count_out=addr(5))
    assert api.tw_kv_assign(*dict(args, rows=-1).values()) == SHAPE
    import torch
    if not torch.cuda.is_available():
        assert api.tw_kv_assign(*args.values()) in (6, UNSUPPORTED)


@pytest.mark.parametrize("bad,status", [
    (dict(k=None), NULL), (dict(dtype=3), UNSUPPORTED), (dict(num_pages=0), SHAPE), (dict(page_size=0), SHAPE),
    (dict(kv_heads=0), SHAPE), (dict(head_dim=100), SHAPE), (dict(head_dim=264), SHAPE), (dict(head_dim=0), SHAPE),
    (dict(num_pages=1 << 28), SHAPE), (dict(token_stride=64), SHAPE), (dict(head_stride=132), ALIGN),
    (dict(v=addr(2) + 8), ALIGN), (dict(dtype=2), NULL), (dict(dtype=2, head_dim=72, k_scale=addr(3), v_scale=addr(4)), SHAPE),
    (dict(dtype=2, k_scale=addr(3) + 2, v_scale=addr(4)), ALIGN),
    (dict(dtype=2, k_scale=addr(3), v_scale=addr(4), head_stride=136), ALIGN)])
def test_cache_refused(api, bad, status):
    c = cache(api, **bad)
    rc = api.tw_rope_append(addr(3), 1536, addr(4), 256, addr(5), 256, 8, 12, 128, addr(6), 0, addr(7), addr(8),
                            ctypes.addressof(c), addr(9), 1536, None)
    assert rc == status, api.tw_last_error()
    rc = api.tw_paged_attention(addr(3), 1536, 4, 12, ctypes.addressof(c), addr(4), 8, 8, addr(5), None, 0.1, addr(6),
                                1536, None, addr(7), 1 << 27, None)
    assert rc == status, api.tw_last_error()


APPEND = dict(q=addr(3), ldq=1536, k=addr(4), ldk=256, v=addr(5), ldv=256, rows=8, heads=12, rotary=128,
              inv_freq=addr(6), interleaved=0, positions=addr(7), slots=addr(8), cache=None, q_out=addr(9), ldqo=1536,
              stream=None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), NULL), (dict(v=None), NULL), (dict(q_out=None), NULL), (dict(positions=None), NULL),
    (dict(inv_freq=None), NULL), (dict(rows=0), SHAPE), (dict(heads=0), SHAPE), (dict(heads=13), SHAPE),
    (dict(ldq=1532), SHAPE), (dict(ldk=258), ALIGN), (dict(k=addr(4) + 4), ALIGN), (dict(rotary=132), SHAPE),
    (dict(rotary=12), SHAPE), (dict(rotary=-8), SHAPE), (dict(q_out=addr(3), ldqo=1540), SHAPE),
    (dict(inv_freq=addr(6) + 4), ALIGN), (dict(rotary=1 << 40), SHAPE)])
def test_append_refuses(api, bad, status):
    c = cache(api)
    args = dict(APPEND, cache=ctypes.addressof(c))
    assert api.tw_rope_append(*dict(args, **bad).values()) == status, api.tw_last_error()
    assert api.tw_rope_append(*dict(args, cache=None).values()) == NULL


ATTEND = dict(q=addr(3), ldq=1536, requests=4, heads=12, cache=None, block_table=addr(4), max_pages=8, table_stride=8,
              lengths=addr(5), first=None, scale=0.1, out=addr(6), ldo=1536, lse=None, ws=addr(7), ws_bytes=1 << 27,
              stream=None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(lengths=None), NULL), (dict(block_table=None), NULL),
    (dict(requests=0), SHAPE), (dict(heads=5), SHAPE), (dict(ldo=1000), SHAPE), (dict(ldq=1538), ALIGN),
    (dict(max_pages=0), SHAPE), (dict(table_stride=4), SHAPE), (dict(scale=float("nan")), NONFINITE),
    (dict(ws=None), BUFSIZE), (dict(ws_bytes=16), BUFSIZE), (dict(ws=addr(7) + 8), ALIGN),
    (dict(out=addr(3) + 6144), SHAPE), (dict(lse=addr(8) + 1), ALIGN)])
def test_attention_refuses(api, bad, status):
    c = cache(api)
    args = dict(ATTEND, cache=ctypes.addressof(c))
    assert api.tw_paged_attention(*dict(args, **bad).values()) == status, api.tw_last_error()


def test_attention_workspace_sizes(api):
    f = api.tw_paged_attention_workspace_bytes
    assert f(1, 12, 2, 128) > 0 and f(1, 12, 2, 128) % 16 == 0
    for bad in ((0, 12, 2, 128), (1, 13, 2, 128), (1, 12, 0, 128), (1, 12, 2, 0), (1, 0, 1, 128), (1, 12, 2, 512)):
        assert f(*bad) == 0


def norm_args(api, **over):
    f = dict(x=addr(1), y=addr(2), gate=None, post_weight=None, post_bias=None, pre_weight=addr(3), pre_bias=None,
             h=addr(4), n=addr(5), xq=None, amax=None, qsum=None, M=4, K=1536, ldx=1536, ldy=1536, ldgate=0, ldh=1536,
             ldn=1536, post=0, pre=1, alpha=1.0, eps=1e-6)
    f.update(over)
    return api.NormArgs(**f)


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), NULL), (dict(h=None, n=None), NULL), (dict(xq=addr(6)), NULL), (dict(amax=addr(6)), NULL),
    (dict(qsum=addr(6)), NULL), (dict(M=0), SHAPE), (dict(K=0), SHAPE), (dict(K=32769, ldx=40000, ldy=40000, ldh=40000, ldn=40000), SHAPE),
    (dict(post=3), UNSUPPORTED), (dict(pre=-1), UNSUPPORTED), (dict(pre_bias=addr(6)), SHAPE), (dict(post_weight=addr(6)), SHAPE),
    (dict(y=None, gate=addr(6)), NULL), (dict(y=None, post=1), NULL), (dict(alpha=float("inf")), NONFINITE),
    (dict(eps=-1.0), NONFINITE), (dict(eps=float("nan")), NONFINITE), (dict(ldx=1535), SHAPE), (dict(ldh=8), SHAPE),
    (dict(gate=addr(6), ldgate=5), SHAPE), (dict(x=addr(1) + 2), ALIGN), (dict(h=addr(1) + 16), SHAPE),
    (dict(n=addr(4)), SHAPE), (dict(h=addr(3)), SHAPE), (dict(h=addr(1), ldh=1540), SHAPE),
    (dict(xq=addr(5), amax=addr(7)), SHAPE), (dict(n=None, xq=addr(6), amax=addr(6) + 16), SHAPE)])
def test_norm_refuses(api, bad, status):
    a = norm_args(api, **bad)
    assert api.tw_residual_norm(ctypes.byref(a), None) == status, api.tw_last_error()
    assert api.tw_residual_norm(None, None) == NULL


def test_structs_match_the_header(api):
    assert ctypes.sizeof(api.KVCacheStruct) == 12 * 8
    assert ctypes.sizeof(api.NormArgs) == 19 * 8 + 16
    assert ctypes.sizeof(api.CachedLayer) == 14 * 8
    assert ctypes.sizeof(api.ChainCache) == 13 * 8 + 16 + 16


def test_cached_chain_refuses(api):
    buf = api.ChainBuffers(*[addr(i) for i in range(1, 10)], 2, 256, 128, 64, 512)
    c = api.ChainCache(x=addr(10), q=addr(11), k=addr(12))
    layers, cached = (api.ChainLayer * 1)(), (api.CachedLayer * 1)()
    call = lambda c, n=1: api.tw_decoder_chain_cached(layers, cached, n, ctypes.byref(buf), ctypes.byref(c), addr(13), 1 << 20, None)  # noqa: E731
    assert call(c, 0) == NULL
    assert call(c) == NULL                                   # no tables
    assert call(api.ChainCache(x=addr(10), q=addr(11))) == NULL
    assert call(api.ChainCache(x=addr(10), q=addr(11), k=addr(12) + 4)) == ALIGN
    assert call(api.ChainCache(x=addr(1) + 16, q=addr(11), k=addr(12))) == SHAPE
    assert call(api.ChainCache(x=addr(10), q=addr(10) + 16, k=addr(12))) == SHAPE


def test_python_refuses(api):
    import torch
    x = torch.zeros(2, 128)
    for call in (lambda: api.residual_norm(x), lambda: api.kv_assign(x, x, x, x, x, 16, 2),
                 lambda: api.KVCache(torch.zeros(2, 16, 2, 64, dtype=torch.float16), torch.zeros(2, 16, 2, 64))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
