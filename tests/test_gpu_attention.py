"""Paged attention of one new token per request against a plain form in 64
bits: types, head layouts, lengths, page sizes, strides, masks that leave
nothing, what masked places hold, long caches, graphs and streams."""
import numpy as np
import pytest

from tests import gpu_util as G
from tests import plain64
from tests.test_gpu_kv import i32

pytestmark = pytest.mark.gpu
SHAPES = [(12, 2, 128), (2, 1, 128), (8, 8, 64), (14, 2, 64), (9, 3, 80), (8, 1, 256), (16, 1, 128),
          (40, 2, 96), (1, 1, 16), (5, 5, 48), (20, 1, 256), (6, 2, 32), (3, 1, 8), (4, 2, 24), (2, 1, 200),
          (3, 3, 240), (32, 32, 64), (7, 1, 112)]


@pytest.fixture(scope="module")
def dev():
    return G.torch_dev()


@pytest.fixture(scope="module")
def api():
    return G.api()


def make(api, dev, dtype, lengths, heads, hk, d, page, seed, first=None, order="pth", spread=1.0, poison=True):
    """A cache whose unused places hold NaN (codes: 127 with a NaN scale), q, table and the request's rows."""
    import torch
    rng = np.random.default_rng(seed)
    T = dict(bf16=torch.bfloat16, f16=torch.float16, i8=torch.int8)[dtype]
    need = [-(-n // page) for n in lengths]
    pages, width = sum(need) + 2, max(max(need), 1) + 1
    ids = rng.permutation(pages)
    table = np.full((len(lengths), width), 2 ** 30)      # behind a request's pages: no page
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
    size = dict(p=pages, t=page, h=hk)
    shape = [size[c] for c in order] + [d]
    perm = [order.index(c) for c in "pth"] + [3]
    seen = np.zeros((pages, page), bool)
    for r, n in enumerate(lengths):
        for j in range(0 if first is None else max(first[r], 0), n):
            seen[table[r, j // page], j % page] = True
    seen = G.to_dev(seen, dev)
    pools, scales = [], [None, None]
    for i in range(2):
        x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dev).permute(perm)
        if dtype == "i8":
            x = (x * 40).round().clamp(-127, 127)
            s = G.to_dev((rng.random((pages, page, hk)) * 0.05 + 0.002).astype(np.float32), dev)
            scales[i] = torch.where(seen[..., None], s, float("nan")) if poison else s
            x = torch.where(seen[..., None, None], x, 127) if poison else x
        elif poison:
            x = torch.where(seen[..., None, None], x, float("nan"))
        pool = torch.empty(shape, dtype=T, device=dev).permute(perm)
        pool.copy_(x)
        pools.append(pool)
    cache = api.KVCache(*pools, *scales)
    q = spread * rng.standard_normal((len(lengths), heads * d)).astype(np.float32)
    return cache, q, table


def rows_of(cache, table, r, lo, hi):
    """Keys and values of a request's places lo..hi - 1, in 64 bits."""
    j = np.arange(lo, hi)
    page, off = table[r][j // cache.page_size], j % cache.page_size
    out = []
    for pool, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        import torch
        p, o = torch.from_numpy(page).to(pool.device), torch.from_numpy(off).to(pool.device)
        x = pool[p, o].double()
        if s is not None:
            x = x * s[p, o].double()[..., None]
        out.append(x.cpu().numpy())
    return out


def scales_of(cache, table, r, lo, hi):
    """The scales of the values of a request's places, or None."""
    if cache.v_scale is None:
        return None
    j = np.arange(lo, hi)
    return cache.v_scale.cpu().numpy().astype(np.float64)[table[r][j // cache.page_size], j % cache.page_size]


def check_all(api, cache, q, table, lengths, first, out, lse, heads, scale=None):
    d = cache.head_dim
    scale = d ** -0.5 if scale is None else scale
    out, lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    for r, n in enumerate(lengths):
        lo = 0 if first is None else min(max(first[r], 0), n)
        k, v = rows_of(cache, table, r, lo, n)
        w, wl, tol, tl = plain64.attention(q[r].reshape(heads, d).astype(np.float64), k, v, scale, heads,
                                           scales_of(cache, table, r, lo, n))
        got = out[r].reshape(heads, d)
        assert (np.abs(got - w) <= tol).all(), (r, n, float((np.abs(got - w) - tol).max()))
        if n > lo:
            assert (np.abs(lse[r] - wl) <= tl).all(), (r, n)
        else:
            assert (got == 0).all() and (lse[r] == -np.inf).all()


LENGTHS = [1, 0, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 1025]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "i8"])
@pytest.mark.parametrize("heads,hk,d", SHAPES)
def test_attention_shapes(dev, api, dtype, heads, hk, d):
    if dtype == "i8" and d % 16:
        pytest.skip("codes come in 16-byte rows")
    page = 16 if heads % 2 else 7
    cache, q, table = make(api, dev, dtype, LENGTHS, heads, hk, d, page, heads + d, order="pht" if hk == 2 else "pth")
    out, lse = api.paged_attention(G.to_dev(q, dev), cache, i32(table, dev), i32(LENGTHS, dev), return_lse=True)
    api.check()
    check_all(api, cache, q, table, LENGTHS, None, out, lse, heads)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "i8"])
@pytest.mark.parametrize("page", [1, 3, 16, 48, 64, 256])
def test_attention_masks_and_pages(dev, api, dtype, page):
    rng = np.random.default_rng(page)
    lengths = [int(n) for n in rng.integers(1, 700, 19)] + [64, 128, 5]
    first = [int(rng.integers(0, n)) for n in lengths]
    first[0], first[1], first[2], first[3] = lengths[0], lengths[1] + 40, -5, lengths[3] - 1
    cache, q, table = make(api, dev, dtype, lengths, 12, 2, 128, page, page, first=first)
    out, lse = api.paged_attention(G.to_dev(q, dev), cache, i32(table, dev), i32(lengths, dev),
                                   first=i32(first, dev), scale=0.3, return_lse=True)
    api.check()
    check_all(api, cache, q, table, lengths, first, out, lse, 12, scale=0.3)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "i8"])
def test_attention_long_and_peaked(dev, api, dtype):
    """Lengths that are split over the whole GPU, and scores of up to +-60."""
    lengths = [20000, 1, 3333]
    cache, q, table = make(api, dev, dtype, lengths, 12, 2, 128, 64, 5, spread=8.0)
    ws = api.paged_attention_workspace(3, 12, cache)
    args = (G.to_dev(q, dev), cache, i32(table, dev), i32(lengths, dev))
    out, lse = api.paged_attention(*args, ws=ws, return_lse=True)
    api.check()
    check_all(api, cache, q, table, lengths, None, out, lse, 12)
    for _ in range(3):   # the same bits again, from the same workspace
        o2, l2 = api.paged_attention(*args, ws=ws, return_lse=True)
        assert bool((o2 == out).all()) and bool((l2 == lse).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "i8"])
def test_attention_many_requests(dev, api, dtype):
    rng = np.random.default_rng(11)
    lengths = [int(n) for n in np.exp(rng.uniform(0, np.log(600), 1500))]
    lengths[7::50] = [0] * len(lengths[7::50])
    cache, q, table = make(api, dev, dtype, lengths, 4, 2, 64, 16, 12)
    out, lse = api.paged_attention(G.to_dev(q, dev), cache, i32(table, dev), i32(lengths, dev), return_lse=True)
    api.check()
    check_all(api, cache, q, table, lengths, None, out, lse, 4)


def test_attention_extreme_queries(dev, api):
    """Queries far from 1: small ones stay exact, large ones pick one key."""
    import torch
    for dtype, mul in (("f16", 1e-6), ("f16", 3e4), ("bf16", 1e5), ("i8", 1e4), ("bf16", 0.0)):
        cache, q, table = make(api, dev, dtype, [100, 37], 6, 2, 64, 16, 3, spread=mul)
        out, lse = api.paged_attention(G.to_dev(q, dev), cache, i32(table, dev), i32([100, 37], dev), return_lse=True)
        api.check()
        assert torch.isfinite(out).all()
        check_all(api, cache, q, table, [100, 37], None, out, lse, 6)


def test_attention_code_scales(dev, api):
    """Scales of codes from 2^-40 to 2^10, and zero where every code is zero."""
    cache, q, table = make(api, dev, "i8", [200, 5], 4, 2, 64, 16, 9, poison=False)
    rng = np.random.default_rng(1)
    cache.v_scale.copy_(G.to_dev(2.0 ** rng.uniform(-40, 10, tuple(cache.v_scale.shape)).astype(np.float32), dev))
    zero = G.to_dev(rng.random(tuple(cache.v_scale.shape)) < 0.2, dev)
    cache.v[zero] = 0
    cache.v_scale[zero] = 0
    out, lse = api.paged_attention(G.to_dev(q, dev), cache, i32(table, dev), i32([200, 5], dev), return_lse=True)
    api.check()
    check_all(api, cache, q, table, [200, 5], None, out, lse, 4)


def test_attention_nan_stays_in_its_request(dev, api):
    import torch
    lengths = [50, 70, 64]
    cache, q, table = make(api, dev, "bf16", lengths, 4, 2, 64, 16, 4)
    want = api.paged_attention(G.to_dev(q, dev), cache, i32(table, dev), i32(lengths, dev))
    cache.k[int(table[1][2]), 3, 0, 5] = float("nan")     # a visible key of request 1, KV head 0
    got = api.paged_attention(G.to_dev(q, dev), cache, i32(table, dev), i32(lengths, dev))
    api.check()
    assert torch.equal(got[[0, 2]], want[[0, 2]])
    assert torch.isnan(got[1, :128]).all() and torch.equal(got[1, 128:], want[1, 128:])


def test_attention_bad_pages_and_lengths(dev, api):
    import torch
    lengths = [40, 20]
    cache, q, table = make(api, dev, "f16", lengths, 2, 1, 64, 16, 6)
    x = G.to_dev(q, dev)
    want = api.paged_attention(x, cache, i32(table, dev), i32(lengths, dev))
    bad = table.copy()
    bad[0, 1] = cache.num_pages
    bad[0, 2] = -1
    got = api.paged_attention(x, cache, i32(bad, dev), i32(lengths, dev))
    with pytest.raises(api.TernaryError, match="TW_ERR_CORRUPT"):
        api.check()
    assert torch.isfinite(got).all() and torch.equal(got[1], want[1])
    got = api.paged_attention(x, cache, i32(table[:, :2], dev), i32([1 << 30, 20], dev))
    with pytest.raises(api.TernaryError, match="TW_ERR_CORRUPT"):
        api.check()
    assert torch.equal(got[1], want[1])
    assert (api.paged_attention(x, cache, i32(table, dev), i32([-3, 0], dev)) == 0).all()
    api.check()


def test_attention_strided_rows_and_one_row(dev, api):
    import torch
    lengths = [33, 100, 64]
    cache, q, table = make(api, dev, "bf16", lengths, 12, 2, 128, 16, 8)
    wide = torch.zeros(3, 12 * 128 + 64, device=dev)
    wide[:, 32:32 + 12 * 128] = G.to_dev(q, dev)
    t = torch.full((3, table.shape[1] + 5), -1, dtype=torch.int32, device=dev)
    t[:, :table.shape[1]] = i32(table, dev)
    into = torch.full((3, 12 * 128 + 8), 7.0, device=dev)
    out, lse = api.paged_attention(wide[:, 32:32 + 12 * 128], cache, t[:, :table.shape[1]], i32(lengths, dev),
                                   out=into[:, 4:4 + 12 * 128], return_lse=True)
    api.check()
    check_all(api, cache, q, table, lengths, None, out, lse, 12)
    assert (into[:, :4] == 7).all() and (into[:, 4 + 12 * 128:] == 7).all()
    one, lse1 = api.paged_attention(G.to_dev(q[1:2], dev), cache, i32(table[1:2], dev), i32(lengths[1:2], dev), return_lse=True)
    check_all(api, cache, q[1:2], table[1:2], lengths[1:2], None, one, lse1, 12)


def test_attention_offsets_past_32_bits(dev, api):
    """Pools of more than 2^31 elements, the request's pages at their end."""
    import torch
    pages, page, hk, d = 2 ** 31 // (64 * 2 * 128) + 4, 64, 2, 128
    k = torch.zeros((pages, page, hk, d), dtype=torch.int8, device=dev)
    v = torch.zeros_like(k)
    ks, vs = (torch.full((pages, page, hk), 0.01, device=dev) for _ in range(2))
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    for pool in (k, v):
        pool[-3:] = torch.randint(-127, 128, (3, page, hk, d), device=dev, generator=g, dtype=torch.int8)
    cache = api.KVCache(k, v, ks, vs)
    table = np.array([[pages - 1, pages - 3, pages - 2]])
    q = np.random.default_rng(2).standard_normal((1, 12 * d)).astype(np.float32)
    out, lse = api.paged_attention(G.to_dev(q, dev), cache, i32(table, dev), i32([190], dev), return_lse=True)
    # and a new key at the very last slot
    x = torch.randn(1, hk * d, device=dev)
    api.rope_append(G.to_dev(q, dev), x, x, i32([0], dev), i32([pages * page - 1], dev), cache)
    api.check()
    assert int(k[-1, -1].abs().max()) == 127
    k[-1, -1] = 0   # (place 63 of the request's first page)
    cache2 = api.KVCache(k, v, ks, vs)
    out, lse = api.paged_attention(G.to_dev(q, dev), cache2, i32(table, dev), i32([190], dev), return_lse=True)
    api.check()
    check_all(api, cache2, q, table, [190], None, out, lse, 12)


def test_attention_on_streams(dev, api):
    """Two calls at once on their own streams and workspaces, beside a third on the current stream."""
    import torch
    lengths = [5000, 3, 800]
    cache, q, table = make(api, dev, "bf16", lengths, 12, 2, 128, 16, 21)
    x, t, n = G.to_dev(q, dev), i32(table, dev), i32(lengths, dev)
    want = api.paged_attention(x, cache, t, n)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(20):
        outs += [api.paged_attention(x, cache, t, n, stream=s) for s in streams]
        outs.append(api.paged_attention(x, cache, t, n))
    torch.cuda.synchronize()
    api.check()
    assert all(torch.equal(o, want) for o in outs)


def test_step_in_a_graph(dev, api):
    """A whole step -- assign, append, attend -- captured once and replayed
    follows the same steps run one by one."""
    import torch
    n, page, width, heads, hk, d = 5, 4, 12, 6, 2, 64
    inv = G.to_dev(10000.0 ** (-np.arange(32) / 32.0), dev)

    def state():
        s = dict(cache=api.KVCache.empty(n * width, page, hk, d, torch.bfloat16, dev))
        s["lengths"], s["count"] = i32([0, 3, 9, 1, 4], dev), i32([n * width - 7], dev)
        table = np.full((n, width), -1)
        table[1, 0], table[2, :3], table[3, 0], table[4, 0] = 59, [58, 57, 56], 55, 54
        s["table"], s["free"] = i32(table, dev), i32(list(range(53)) + [0] * 7, dev)
        s["x"] = torch.zeros(n, (heads + 2 * hk) * d, device=dev)
        s["ws"] = api.paged_attention_workspace(n, heads, s["cache"])
        return s

    def step(s):
        a = api.kv_assign(s["lengths"], ones, s["table"], s["free"], s["count"], page, n + 2,
                          lengths_out=s["lengths"], free_count_out=s["count"])
        q, k, v = s["x"].split([heads * d, hk * d, hk * d], dim=1)
        q = api.rope_append(q, k, v, a.positions[:n], a.slots[:n], s["cache"], inv_freq=inv)
        return api.paged_attention(q, s["cache"], s["table"], s["lengths"], ws=s["ws"])

    ones = i32([1] * n, dev)
    xs = [torch.randn(n, (heads + 2 * hk) * d, device=dev) for _ in range(12)]
    eager, graphed = state(), state()
    want = []
    for x in xs:
        eager["x"].copy_(x)
        want.append(step(eager).clone())
    side = torch.cuda.Stream()
    warm = state()
    with torch.cuda.stream(side):
        step(warm)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(graphed)
    for x, w in zip(xs, want):
        graphed["x"].copy_(x)
        g.replay()
        assert torch.equal(out, w)
    api.check()
    assert torch.equal(graphed["lengths"], eager["lengths"]) and torch.equal(graphed["table"], eager["table"])


@pytest.mark.parametrize("dtype", ["bf16", "i8"])
def test_attention_large_pages_and_all_heads(dev, api, dtype):
    """Pages of more keys than a tile, and a layer of 64 query heads over one KV head."""
    lengths = [3000, 700, 0, 4096, 4097]
    for heads, hk, d, page in ((64, 1, 64, 2048), (16, 16, 128, 4096), (9, 3, 128, 1000)):
        cache, q, table = make(api, dev, dtype, lengths, heads, hk, d, page, heads)
        out, lse = api.paged_attention(G.to_dev(q, dev), cache, i32(table, dev), i32(lengths, dev), return_lse=True)
        api.check()
        check_all(api, cache, q, table, lengths, None, out, lse, heads)


def test_two_graphs_and_eager_share_a_workspace(dev, api):
    """Captured calls of different shapes on one workspace, replayed in turn with eager ones on one stream."""
    import torch
    lengths = [9000, 17, 400]
    ws, calls = None, []
    for dtype, heads, hk, d in (("bf16", 12, 2, 128), ("i8", 8, 8, 64)):
        cache, q, table = make(api, dev, dtype, lengths, heads, hk, d, 16, d)
        args = (G.to_dev(q, dev), cache, i32(table, dev), i32(lengths, dev))
        ws = api.paged_attention_workspace(3, heads, cache) if ws is None else ws
        want = api.paged_attention(*args, ws=ws)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            out = api.paged_attention(*args, ws=ws)
        calls.append((g, out, want, args))
    for _ in range(4):
        for g, out, want, args in calls:
            out.zero_()
            g.replay()
            assert torch.equal(out, want)
            assert torch.equal(api.paged_attention(*args, ws=ws), want)
    api.check()
    assert int(ws[:3 * 512 * 8 * 4].any()) == 0   # the counters are zero again


def test_attention_refuses_wrong_tensors(dev, api):
    import torch
    cache, q, table = make(api, dev, "bf16", [40, 20], 2, 1, 64, 16, 6)
    x, t, n = G.to_dev(q, dev), i32(table, dev), i32([40, 20], dev)
    good = (x, cache, t, n)
    ok = api.paged_attention(*good)
    for bad, kind in ((dict(q=x.double()), TypeError), (dict(q=x.cpu()), ValueError), (dict(q=x[0]), ValueError),
                      (dict(q=x[:, :100]), ValueError), (dict(block_table=t.long()), TypeError),
                      (dict(block_table=t[:1]), ValueError), (dict(block_table=t.t()), ValueError),
                      (dict(lengths=n[:1]), ValueError), (dict(lengths=n.cpu()), ValueError), (dict(first=n.float()), TypeError),
                      (dict(out=x[:, :64]), ValueError), (dict(out=x), api.TernaryError), (dict(lse=n), TypeError),
                      (dict(ws=torch.zeros(16, dtype=torch.uint8, device=dev)), api.TernaryError),
                      (dict(scale=float("inf")), api.TernaryError), (dict(scale="a"), TypeError)):
        kw = dict(q=x, cache=cache, block_table=t, lengths=n)
        kw.update(bad)
        with pytest.raises(kind):
            api.paged_attention(**kw)
    assert torch.equal(api.paged_attention(*good), ok)
    wide = torch.zeros(2, 2 ** 20, dtype=torch.int32, device=dev)   # 2 x 2^20 pages of 2^15 keys
    big = api.KVCache(*[torch.zeros(1, 2 ** 15, 1, 64, dtype=torch.bfloat16, device=dev) for _ in range(2)])
    many = torch.zeros(300, 64, device=dev)
    with pytest.raises(api.TernaryError, match="too many"):
        api.paged_attention(many, big, wide[:1].expand(300, 2 ** 20).contiguous(), i32([1] * 300, dev))
    api.check()


def test_pools_with_strides_past_32_bits(dev, api):
    """Two pages 2^32 bytes apart: appended to, then attended over, as in a dense pool."""
    import torch
    d, page, far = 64, 16, 2 ** 32
    pools = [torch.zeros(far + page * d, dtype=torch.int8, device=dev).as_strided((2, page, 1, d), (far, d, d, 1)) for _ in range(2)]
    scales = [torch.zeros(2, page, 1, device=dev) for _ in range(4)]
    cache = api.KVCache(*pools, *scales[:2])
    dense = api.KVCache(*[torch.zeros(2, page, 1, d, dtype=torch.int8, device=dev) for _ in range(2)], *scales[2:])
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    x = torch.randn(31, d, device=dev, generator=g)
    inv = G.to_dev(100.0 ** (-np.arange(32) / 32.0), dev)
    slots = i32(list(range(16, 32)) + list(range(15)), dev)
    outs = []
    for c in (cache, dense):
        q = api.rope_append(x, x, x, i32(range(31), dev), slots, c, inv_freq=inv)
        outs.append(api.paged_attention(q[:1], c, i32([[1, 0]], dev), i32([31], dev)))
    api.check()
    assert torch.equal(outs[0], outs[1]) and float(outs[0].abs().max()) > 0
    assert torch.equal(cache.k[1], dense.k[1]) and torch.equal(cache.v[0], dense.v[0])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "i8"])
@pytest.mark.parametrize("heads,hk,d", [(8, 1, 128), (7, 1, 64), (9, 1, 128), (15, 1, 64), (3, 1, 256), (8, 1, 256)])
def test_attention_joins_of_every_head_count(dev, api, dtype, heads, hk, d):
    """One to eight heads of a unit, in more pieces than one join takes."""
    lengths = [14000, 5, 0, 3500]
    cache, q, table = make(api, dev, dtype, lengths, heads, hk, d, 64, heads * d)
    ws = api.paged_attention_workspace(len(lengths), heads, cache)
    args = (G.to_dev(q, dev), cache, i32(table, dev), i32(lengths, dev))
    out, lse = api.paged_attention(*args, ws=ws, return_lse=True)
    api.check()
    check_all(api, cache, q, table, lengths, None, out, lse, heads)
    o2, l2 = api.paged_attention(*args, ws=ws, return_lse=True)
    assert bool((o2 == out).all()) and bool((l2 == lse).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "i8"])
@pytest.mark.parametrize("heads,hk,d,page", [(14, 2, 64, 16), (8, 8, 64, 48), (6, 2, 32, 32), (4, 4, 48, 5)])
def test_attention_masks_in_short_rows(dev, api, dtype, heads, hk, d, page):
    """Sixteens of keys of which none is visible beside others, what the masked places hold being NaN."""
    rng = np.random.default_rng(d + page)
    lengths = [int(n) for n in rng.integers(1, 900, 24)] + [16, 17, 32, 33, 48, 49]
    first = [int(rng.integers(0, n)) for n in lengths]
    first[:4] = [lengths[0], max(lengths[1] - 3, 0), 16, -1]
    cache, q, table = make(api, dev, dtype, lengths, heads, hk, d, page, heads, first=first)
    args = (G.to_dev(q, dev), cache, i32(table, dev), i32(lengths, dev))
    for _ in range(3):
        out, lse = api.paged_attention(*args, first=i32(first, dev), return_lse=True)
        api.check()
        check_all(api, cache, q, table, lengths, first, out, lse, heads)


@pytest.mark.parametrize("seed", range(12))
def test_attention_runs_of_few_tiles(dev, api, seed):
    """Lengths of a few tiles each, so many that blocks have one to five: ends of runs next to ends of requests."""
    rng = np.random.default_rng(seed)
    count, top = int(rng.integers(40, 260)), int(rng.choice([150, 250, 400, 700, 1500]))
    lengths = [int(n) for n in rng.integers(1, top, count)]
    lengths[::17] = [0] * len(lengths[::17])
    heads, hk, d = [(8, 1, 64), (4, 2, 128), (2, 1, 256)][seed % 3]
    dtype = ["f16", "i8", "bf16"][seed // 3 % 3]
    cache, q, table = make(api, dev, dtype, lengths, heads, hk, d, 32, seed, poison=False)
    ws = api.paged_attention_workspace(count, heads, cache)
    args = (G.to_dev(q, dev), cache, i32(table, dev), i32(lengths, dev))
    out, lse = api.paged_attention(*args, ws=ws, return_lse=True)
    api.check()
    check_all(api, cache, q, table, lengths, None, out, lse, heads)
    o2, l2 = api.paged_attention(*args, ws=ws, return_lse=True)
    assert bool((o2 == out).all()) and bool((l2 == lse).all())
    assert not bool(ws[:3 * 512 * 8 * 4].any())   # the counters are zero between calls
