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


APPEND = dict(q=addr(3), ldq=1536, k=addr(4), ldk=256, v=addr(5), ldv=256, rows=8, heads=12, rotary=128,
              inv_freq=addr(6), interleaved=0, positions=addr(7), slots=addr(8), cache=None, q_out=addr(9), ldqo=1536,
              stream=None)
QKV = dict(ldq=2048, k=addr(3) + 4 * 1536, ldk=2048, v=addr(3) + 4 * 1792, ldv=2048)   # q, k, v: columns of one buffer


def append(api, scaled=False, pools=(2, 128), **over):  # noqa: F811
    hk, d = pools
    c = dict(k=addr(1), v=addr(2), k_scale=None, v_scale=None, num_pages=10, page_size=16, kv_heads=hk, head_dim=d,
             page_stride=16 * hk * d, token_stride=hk * d, head_stride=d, dtype=0)
    if scaled:
        c.update(k_scale=addr(11), v_scale=addr(12), dtype=2)
    c = api.KVCacheStruct(**c)
    return api.tw_rope_append(*dict(APPEND, cache=ctypes.addressof(c), **over).values())


@pytest.mark.parametrize("bad", [
    dict(q_out=addr(3) + 16), dict(q_out=addr(3) + 4 * 1536), dict(q_out=addr(3) - 4 * 1536 * 7),
    dict(q_out=addr(3) + 4 * 1536 * 7), dict(q_out=addr(4)), dict(q_out=addr(5) + 4 * 256 * 7),
    dict(k=addr(9) + 4 * 1536 * 7), dict(v=addr(9) - 16), dict(q_out=addr(4) - 4 * 1536 * 8 + 16),
    dict(QKV, q_out=addr(3) + 16, ldqo=2048), dict(QKV, q_out=addr(3) + 4 * 1536, ldqo=2048),
    dict(QKV, q_out=addr(3) + 4 * 2048 - 16, ldqo=2048), dict(QKV, q_out=addr(3) + 4 * 1536, ldqo=1536),
    dict(q=addr(3), ldq=4096, q_out=addr(3) + 4 * 3584, ldqo=4096),
    dict(q=addr(3), ldq=4096, q_out=addr(3) + 4 * 2048, ldqo=2048),
    dict(q_out=addr(1)), dict(q_out=addr(2) + 2 * (10 * 16 * 256) - 16), dict(q_out=addr(1) - 4 * 1536 * 8 + 16),
    dict(scaled=True, q_out=addr(11)), dict(scaled=True, q_out=addr(12) + 4 * 316), dict(q_out=addr(7)),
    dict(q_out=addr(8) + 16), dict(q_out=addr(6) + 496)])
def test_append_refuses_outputs_in_its_operands(api, bad):  # noqa: F811
    assert append(api, **bad) == SHAPE, api.tw_last_error()
    assert b"overlaps" in api.tw_last_error()


@pytest.mark.parametrize("good", [
    dict(), dict(q_out=addr(3)), dict(QKV, q_out=addr(3), ldqo=2048), dict(q_out=addr(3) + 4 * 1536 * 8),
    dict(QKV, q_out=addr(3) + 4 * 2048 * 8, ldqo=1536), dict(q_out=addr(4) - 4 * 1536 * 8),
    dict(QKV, ldq=4096, ldk=4096, ldv=4096, q_out=addr(3) + 4 * 2048, ldqo=4096),
    dict(QKV, ldq=4096, ldk=4096, ldv=4096, q_out=addr(3) - 4 * 1536, ldqo=4096),
    dict(q=addr(3), ldq=6144, q_out=addr(3) + 4 * 1536, ldqo=6144), dict(rows=1, q_out=addr(3) + 4 * 1536),
    dict(rotary=0, inv_freq=addr(9)), dict(q_out=addr(1) + 2 * 10 * 16 * 256), dict(k=addr(9) - 4 * 256 * 8),
    dict(rows=2, q=addr(3), ldq=8192, k=addr(3) + 4 * 1536, ldk=12288, q_out=addr(3) + 4 * 2048, ldqo=4096)])
def test_append_takes_rows_side_by_side(api, good):  # noqa: F811
    """What shares no byte passes the checks (what is left to fail here is the device)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("addresses of nothing: checked where nothing can be launched")
    assert append(api, **good) in (6, 9), api.tw_last_error()


@pytest.mark.parametrize("seed", range(4))
def test_append_overlap_is_that_of_the_bytes(api, seed):  # noqa: F811
    """Random rows of q, k, v and q_out in one buffer, against the columns that each touches."""
    import random

    import torch
    if torch.cuda.is_available():
        pytest.skip("addresses of nothing: checked where nothing can be launched")
    rng = random.Random(seed)
    seen = [0, 0]
    for _ in range(400):
        rows, heads = rng.randrange(1, 6), rng.randrange(1, 4)
        same = 4 * rng.randrange(2 * heads, 16)
        put = {}
        for name, width in (("q", 8 * heads), ("k", 8), ("v", 8), ("q_out", 8 * heads)):
            ld = same if rng.random() < 0.6 else width + 4 * rng.randrange(0, 12)
            put[name] = (4 * rng.randrange(0, 80), max(ld, width), width)
        if put["q"][0] == put["q_out"][0]:
            continue
        touch = {n: {a + i * ld + c for i in range(rows) for c in range(w)} for n, (a, ld, w) in put.items()}
        want = any(touch["q_out"] & touch[n] for n in "qkv")
        at = {n: addr(20) + 4 * a for n, (a, _, _) in put.items()}
        rc = append(api, rows=rows, heads=heads, rotary=8, ldq=put["q"][1], ldk=put["k"][1], ldv=put["v"][1],
                    ldqo=put["q_out"][1], pools=(1, 8), **at)
        assert (rc == SHAPE) == want and rc in (SHAPE, 6, 9), (rc, put, rows, api.tw_last_error())
        seen[want] += 1
    assert min(seen) > 50


ATTEND = dict(q=addr(3), ldq=1536, requests=4, heads=12, cache=None, block_table=addr(4), max_pages=8, table_stride=8,
              lengths=addr(5), first=addr(8), scale=0.1, out=addr(6), ldo=1536, lse=addr(9), ws=addr(7), ws_bytes=1 << 27,
              stream=None)


@pytest.mark.parametrize("bad", [
    dict(lse=addr(6) + 64), dict(lse=addr(3)), dict(lse=addr(5) + 12), dict(lse=addr(8) - 188), dict(lse=addr(7) + 32),
    dict(lse=addr(1)), dict(lse=addr(11) + 4), dict(out=addr(2) + 512), dict(out=addr(4)), dict(out=addr(5) - 16),
    dict(out=addr(7) + 4096), dict(out=addr(12)), dict(ws=addr(3) + 64), dict(ws=addr(9) + 16), dict(ws=addr(1) + 16),
    dict(ws=addr(4)), dict(lengths=addr(6)), dict(first=addr(9) + 4), dict(block_table=addr(7) + 128)])
def test_attention_refuses_outputs_in_its_operands(api, bad):  # noqa: F811
    c = api.KVCacheStruct(k=addr(1), v=addr(2), k_scale=addr(11), v_scale=addr(12), num_pages=10, page_size=16, kv_heads=2,
                          head_dim=128, page_stride=16 * 256, token_stride=256, head_stride=128, dtype=2)
    args = dict(ATTEND, cache=ctypes.addressof(c))
    assert api.tw_paged_attention(*dict(args, **bad).values()) == SHAPE, api.tw_last_error()
    assert b"overlaps" in api.tw_last_error()


@pytest.mark.parametrize("over,taken", [
    (dict(ldq=3200, out=addr(3) + 4 * 1536, ldo=3200), True), (dict(ldq=3200, out=addr(3) + 4 * 1664, ldo=3200), True),
    (dict(ldq=3200, out=addr(3) + 4 * 1532, ldo=3200), False), (dict(ldq=3200, out=addr(3) + 4 * 1668, ldo=3200), False),
    (dict(ldq=3200, out=addr(3) + 4 * 1536, ldo=1536), False), (dict(out=addr(3)), False)])
def test_attention_takes_rows_side_by_side(api, over, taken):  # noqa: F811
    """Queries and outputs as columns of one buffer."""
    import torch
    if taken and torch.cuda.is_available():
        pytest.skip("addresses of nothing: checked where nothing can be launched")
    c = api.KVCacheStruct(k=addr(1), v=addr(2), num_pages=10, page_size=16, kv_heads=2, head_dim=128, page_stride=16 * 256,
                          token_stride=256, head_stride=128)
    rc = api.tw_paged_attention(*dict(ATTEND, cache=ctypes.addressof(c), **over).values())
    assert rc in (6, 9) if taken else rc == SHAPE, api.tw_last_error()


def test_attention_counts_its_tiles_past_64_bits(api):  # noqa: F811
    """2^24 requests of 2^16 heads with 2^24 tiles of 96 keys each: 2^64 tiles are too many, not none."""
    c = api.KVCacheStruct(k=addr(1), v=addr(2), num_pages=10, page_size=12288, kv_heads=1 << 16, head_dim=8,
                          page_stride=12288 << 19, token_stride=1 << 19, head_stride=8)
    big = dict(requests=1 << 24, heads=1 << 16, ldq=1 << 19, ldo=1 << 19, lse=None, first=None, max_pages=1 << 17,
               table_stride=1 << 17)
    assert api.tw_paged_attention(*dict(ATTEND, cache=ctypes.addressof(c), **big).values()) == SHAPE
    assert b"too many" in api.tw_last_error()
