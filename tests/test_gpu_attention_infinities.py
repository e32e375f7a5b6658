"""Paged attention where visible values, keys or queries are infinite or NaN:
outputs are what the formula makes of them (an infinite value in its column,
no weight for a score of -infinity, NaN where infinities meet)."""
import numpy as np
import pytest

from tests import gpu_util as G
from tests import plain64
from tests.test_gpu_attention import make, rows_of
from tests.test_gpu_kv import i32

pytestmark = pytest.mark.gpu
# (pages of 16 and of 7 keys are read in two ways)
SHAPES = [(12, 2, 128, 16), (4, 2, 64, 7), (9, 3, 80, 16), (8, 1, 256, 7), (2, 1, 64, 64), (20, 2, 128, 7)]
LENGTHS = [40, 1, 700, 0, 9000, 33]


@pytest.fixture(scope="module")
def dev():
    return G.torch_dev()


@pytest.fixture(scope="module")
def api():
    return G.api()


def put(pool, table, r, j, head, c, value):
    """Column c of a request's place j."""
    page = pool.shape[1]
    pool[int(table[r][j // page]), j % page, head, c] = value


def formula(q, k, v, scale):
    """One head: out, lse and their bounds.  Keys with a score of -infinity
    have no weight; what is left is bounded as plain64's, the columns of
    infinite or NaN values apart."""
    with np.errstate(invalid="ignore"):
        s = scale * (k * q).sum(axis=1)
        some = ~(s == -np.inf)
        if not some.any():
            return np.zeros(v.shape[1]), -np.inf, np.zeros(v.shape[1]), 0.0
        if not np.isfinite(s[some]).all():
            return np.full(v.shape[1], np.nan), np.nan, np.zeros(v.shape[1]), 0.0
        p = np.exp(s - s.max())
        out = (p[:, None] * v).sum(axis=0) / p.sum()
    w, lse, tol, tl = plain64.attention(q[None], k[some][:, None], np.where(np.isfinite(v), v, 0)[some][:, None], scale, 1)
    return out, lse[0], tol[0], tl[0]


def check(api, dev, cache, q, table, lengths, heads, first=None):
    d, group = cache.head_dim, heads // cache.kv_heads
    ws = api.paged_attention_workspace(len(lengths), heads, cache)
    args = (G.to_dev(q, dev), cache, i32(table, dev), i32(lengths, dev), None if first is None else i32(first, dev))
    for _ in range(2):
        out, lse = api.paged_attention(*args, ws=ws, return_lse=True)
        api.check()
        out, lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        seen = set()
        for r, n in enumerate(lengths):
            k, v = rows_of(cache, table, r, 0 if first is None else min(max(first[r], 0), n), n)
            for h in range(heads):
                want, wl, tol, tl = formula(q[r, h * d:(h + 1) * d].astype(np.float64), k[:, h // group],
                                            v[:, h // group], d ** -0.5)
                got = out[r, h * d:(h + 1) * d]
                fine = np.isfinite(want)
                seen |= {str(x) for x in np.unique(want[~fine])}
                assert np.array_equal(got[~fine], want[~fine], equal_nan=True), (r, h, got[~fine], want[~fine])
                assert (np.abs(got[fine] - want[fine]) <= tol[fine]).all(), (r, h)
                if np.isfinite(wl):
                    assert abs(lse[r, h] - wl) <= tl, (r, h)
                else:
                    assert np.array_equal(lse[r, h], wl, equal_nan=True), (r, h, lse[r, h])
    return seen


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,hk,d,page", SHAPES)
def test_infinite_values(dev, api, dtype, heads, hk, d, page):
    """+-inf and NaN in columns of their own, and +inf beside -inf in one."""
    cache, q, table = make(api, dev, dtype, LENGTHS, heads, hk, d, page, heads)
    inf, kv = float("inf"), hk - 1
    for r, n in enumerate(LENGTHS):
        if n == 0 or r == 5:
            continue
        put(cache.v, table, r, n // 3, kv, 2, inf)
        put(cache.v, table, r, n // 2, kv, d - 1, -inf)
        put(cache.v, table, r, n - 1, kv, 9, float("nan"))
        if n > 1:
            put(cache.v, table, r, 0, kv, 4, inf)
            put(cache.v, table, r, n - 1, kv, 4, -inf)
    assert check(api, dev, cache, q, table, LENGTHS, heads) == {"inf", "-inf", "nan"}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,hk,d,page", SHAPES)
def test_infinite_keys(dev, api, dtype, heads, hk, d, page):
    """A key of -inf in a column where half of the queries are positive (no
    weight) and half negative (a score of +inf: NaN)."""
    cache, q, table = make(api, dev, dtype, LENGTHS, heads, hk, d, page, heads + 1)
    col = 5
    for r, n in enumerate(LENGTHS):
        sign = np.where(np.arange(heads) % 2 == r % 2, 1, -1)
        q[r, col::d] = sign * (0.5 + np.abs(q[r, col::d]))
        if n and r != 5:
            for j in {n // 3, n - 1}:
                for h in range(hk):
                    put(cache.k, table, r, j, h, col, -float("inf"))
    assert check(api, dev, cache, q, table, LENGTHS, heads) == {"nan"}


@pytest.mark.parametrize("dtype", ["bf16", "f16", "i8"])
@pytest.mark.parametrize("heads,hk,d,page", [s for s in SHAPES if s[2] % 16 == 0])
def test_infinite_queries(dev, api, dtype, heads, hk, d, page):
    """An infinite query times keys of both signs, and one whose scores are all -inf."""
    cache, q, table = make(api, dev, dtype, LENGTHS, heads, hk, d, page, heads + 2)
    q[0, 3], q[2, d - 1], q[4, 0], q[4, (heads - 1) * d + 7] = np.inf, -np.inf, np.nan, np.inf
    q[5, 11] = -np.inf
    for j in range(LENGTHS[5]):
        put(cache.k, table, 5, j, 0, 11, 1 + j % 3)
    check(api, dev, cache, q, table, LENGTHS, heads)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("seed", range(6))
def test_infinities_anywhere(dev, api, dtype, seed):
    """Many requests with windows, a few runs' ends in each, infinities at random places seen or not."""
    rng = np.random.default_rng(100 + seed)
    heads, hk, d, page = SHAPES[seed]
    count = int(rng.integers(20, 90))
    lengths = [int(n) for n in rng.integers(0, int(rng.choice([200, 700, 2500])), count)]
    first = [int(rng.integers(-5, n + 3)) if rng.random() < 0.5 else 0 for n in lengths]
    cache, q, table = make(api, dev, dtype, lengths, heads, hk, d, page, seed, first=first)
    for _ in range(count):
        r = int(rng.integers(0, count))
        if lengths[r]:
            j, h, c = int(rng.integers(0, lengths[r])), int(rng.integers(0, hk)), int(rng.integers(0, d))
            put(cache.k if rng.random() < 0.3 else cache.v, table, r, j, h, c, float(rng.choice([np.inf, -np.inf])))
    check(api, dev, cache, q, table, lengths, heads, first)


def test_fp16_keys_past_its_range(dev, api):
    """Values past 65504 become infinite in an fp16 cache, and its outputs in their column."""
    import torch
    page, hk, d, n = 16, 2, 64, 50
    cache = api.KVCache.empty(8, page, hk, d, torch.float16, dev)
    rng = np.random.default_rng(8)
    k, v = (rng.standard_normal((n, hk * d)).astype(np.float32) for _ in range(2))
    v[20, 3], v[21, d + 5] = 1e5, -1e6
    q = rng.standard_normal((n, 4 * d)).astype(np.float32)
    api.rope_append(G.to_dev(q, dev), G.to_dev(k, dev), G.to_dev(v, dev), i32(range(n), dev), i32(range(n), dev), cache)
    out = api.paged_attention(G.to_dev(q[-1:], dev), cache, i32([[0, 1, 2, 3]], dev), i32([n], dev))
    api.check()
    out = out.cpu().numpy().reshape(4, d)
    want = np.zeros((4, d))
    want[:2, 3], want[2:, 5] = np.inf, -np.inf
    assert np.array_equal(np.where(np.isinf(out), out, 0), want) and not np.isnan(out).any()
