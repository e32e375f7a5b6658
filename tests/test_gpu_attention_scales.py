"""Paged attention on codes where visible values have a scale of 0 (as the
append writes for a row of zeros): such a key counts in the sum of weights and
gives nothing to the values, whatever the other keys' scales are."""
import numpy as np
import pytest

from tests import gpu_util as G
from tests import plain64
from tests.test_gpu_attention import make, rows_of, scales_of
from tests.test_gpu_kv import i32

pytestmark = pytest.mark.gpu
SHAPES = [(4, 2, 64, 16), (12, 2, 128, 7), (8, 1, 256, 32)]


@pytest.fixture(scope="module")
def dev():
    return G.torch_dev()


@pytest.fixture(scope="module")
def api():
    return G.api()


def zero_keys(cache, table, r, places, kv=slice(None)):
    """Values of these places of a request become zeros with a scale of 0."""
    for j in places:
        page, at = int(table[r][j // cache.page_size]), j % cache.page_size
        cache.v[page, at, kv] = 0
        cache.v_scale[page, at, kv] = 0


def check(api, dev, cache, q, table, lengths, heads, dominant=False):
    """Against the plain form, a zero scale standing for no weight times scale
    at all (1e-300 in its bound).  `dominant`: keys of scale 0 may set the
    running maximum, which they do 2^80 below their score.  Then distances of
    up to 80 + 12 + 3 powers of two to it, and the maximum less 12 in a part
    and in the log-sum-exp, are rounded below 128 (half a step: 2^-18 each,
    times ln 2), and the log-sum-exp's product, logarithm and sum below 64
    (2^-19 each): together under 2^-16.  And weights times scales end at
    2^-25 beside a sum of 2^(80 + 12) at least: 2^-117 for each key's code."""
    out, lse = api.paged_attention(G.to_dev(q, dev), cache, i32(table, dev), i32(lengths, dev), return_lse=True)
    api.check()
    out, lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    d = cache.head_dim
    for r, n in enumerate(lengths):
        k, v = rows_of(cache, table, r, 0, n)
        s = scales_of(cache, table, r, 0, n)
        vs = np.where(s > 0, s, 1e-300)
        want, wl, tol, tl = plain64.attention(q[r].reshape(heads, d).astype(np.float64), k, v, d ** -0.5, heads, vs)
        if dominant:
            codes = np.abs(v / vs[..., None]).sum(axis=0).repeat(heads // cache.kv_heads, axis=0)
            tol, tl = tol + 2.0 ** -16 * np.abs(want) + 2.0 ** -117 * codes, tl + 2.0 ** -16
        err = np.abs(out[r].reshape(heads, d) - want)
        assert (err <= tol).all(), (r, n, float((err / np.maximum(np.abs(want), 1e-300)).max()))
        assert (np.abs(lse[r] - wl) <= tl).all(), (r, n, float(np.abs(lse[r] - wl).max()))


@pytest.mark.parametrize("heads,hk,d,page", SHAPES)
@pytest.mark.parametrize("power", [-58, -40, -32, -24, -8, 20])
def test_one_zero_scale_among_small_ones(dev, api, heads, hk, d, page, power):
    """One key of scale 0 in each request, the others' scales within a factor of four."""
    lengths = [32, 200, 1, 5000, 33]
    cache, q, table = make(api, dev, "i8", lengths, heads, hk, d, page, 40 + d, poison=False)
    rng = np.random.default_rng(d)
    cache.v_scale.copy_(G.to_dev(2.0 ** (power + 2 * rng.random(tuple(cache.v_scale.shape))).astype(np.float32), dev))
    for r, n in enumerate(lengths):
        if n > 1:
            zero_keys(cache, table, r, [int(rng.integers(0, n))])
    check(api, dev, cache, q, table, lengths, heads)


@pytest.mark.parametrize("heads,hk,d,page", SHAPES)
@pytest.mark.parametrize("far", [20.0, 45.0, 100.0, 300.0])
@pytest.mark.parametrize("power", [-50, -6])
def test_zero_scale_with_the_highest_score(dev, api, heads, hk, d, page, far, power):
    """A key of scale 0 whose score is far above every other one's (in powers of e)."""
    lengths = [64, 300, 3000]
    cache, q, table = make(api, dev, "i8", lengths, heads, hk, d, page, 50 + d, poison=False)
    cache.v_scale.fill_(2.0 ** power)
    q = np.ones_like(q) + 0.01 * q
    for r, n in enumerate(lengths):
        zero_keys(cache, table, r, [n // 2])
        page_of, at = int(table[r][(n // 2) // page]), (n // 2) % page
        cache.k[page_of, at] = 100
        cache.k_scale[page_of, at] = far / (100 * d ** 0.5)
    check(api, dev, cache, q, table, lengths, heads, dominant=True)


def test_every_scale_zero(dev, api):
    """Nothing but zeros to sum: out is 0, the log-sum-exp that of the scores."""
    import torch
    lengths = [1, 40, 2000]
    cache, q, table = make(api, dev, "i8", lengths, 12, 2, 128, 16, 60, poison=False)
    cache.v.zero_()
    cache.v_scale.zero_()
    out = api.paged_attention(G.to_dev(q, dev), cache, i32(table, dev), i32(lengths, dev))
    assert not bool(torch.any(out))
    check(api, dev, cache, q, table, lengths, 12, dominant=True)
    # and in one KV head alone
    cache.v[:, :, 1] = 3
    cache.v_scale[:, :, 1] = 0.01
    check(api, dev, cache, q, table, lengths, 12, dominant=True)


@pytest.mark.parametrize("heads,hk,d,page", SHAPES)
@pytest.mark.parametrize("low,high", [(-62, -60), (-85, -75), (-126, -100), (-126, -122), (-126, 0)])
def test_scales_below_the_products_range(dev, api, heads, hk, d, page, low, high):
    """Scales of all keys far below 1: sums stay finite, outputs within 2^-117 of the sum of weights."""
    lengths = [64, 1, 300, 6000]
    cache, q, table = make(api, dev, "i8", lengths, heads, hk, d, page, 70 + d, poison=False)
    rng = np.random.default_rng(d)
    cache.v_scale.copy_(G.to_dev((2.0 ** rng.uniform(low, high, tuple(cache.v_scale.shape))).astype(np.float32), dev))
    check(api, dev, cache, q, table, lengths, heads, dominant=True)


def test_tiny_values_appended_and_read(dev, api):
    """Scales as the append makes them from values of 1e-20 and 1e-35, beside a row of zeros."""
    import torch
    page, hk, d, n = 16, 2, 64, 40
    cache = api.KVCache.empty(4, page, hk, d, torch.int8, dev)
    rng = np.random.default_rng(5)
    k, v = (rng.standard_normal((n, hk * d)).astype(np.float32) for _ in range(2))
    v[:20] *= 1e-20
    v[20:] *= 1e-35
    v[7] = 0
    q = rng.standard_normal((n, 4 * d)).astype(np.float32)
    api.rope_append(G.to_dev(q, dev), G.to_dev(k, dev), G.to_dev(v, dev), i32(range(n), dev), i32(range(n), dev), cache)
    for length in (n, 8, 1):
        check(api, dev, cache, q[-1:], np.arange(4)[None], [length], 4, dominant=True)
    check(api, dev, cache, q[-1:], np.array([[2, 1, 0, 3]]), [13], 4, dominant=True)   # the smallest alone
