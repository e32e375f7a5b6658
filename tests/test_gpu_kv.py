"""Block tables and slots from request lengths, and the rotation of new tokens
with their write into the cache, against plain forms in 64 bits."""
import numpy as np
import pytest

from tests import gpu_util as G
from tests import plain64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return G.torch_dev()


@pytest.fixture(scope="module")
def api():
    return G.api()


def i32(a, dev):
    import torch
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)


def _server(rng, n, page, width, top):
    """Requests with pages, and a free list of the rest."""
    lengths = rng.integers(0, top + 1, n)
    lengths[rng.random(n) < 0.2] = 0
    pages = rng.permutation(n * width)
    table = np.full((n, width), -7)
    used = 0
    for r in range(n):
        k = -(-lengths[r] // page)
        table[r, :k] = pages[used:used + k]
        used += k
    free = np.full(n * width, -9)
    free[:n * width - used] = pages[used:]
    return lengths, table, free, n * width - used


def _compare(api, dev, lengths, delta, table, free, count, page, rows, in_place=False, stride=0):
    import torch
    want = plain64.assign(lengths.tolist(), delta.tolist(), table.tolist(), free.tolist(), count, page, rows)
    wide = torch.full((table.shape[0], table.shape[1] + stride), -3, dtype=torch.int32, device=dev)
    t = wide[:, :table.shape[1]]
    t.copy_(i32(table, dev))
    ln, f, c = i32(lengths, dev), i32(free, dev), i32([count], dev)
    a = api.kv_assign(ln, i32(delta, dev), t, f, c, page, rows,
                      lengths_out=ln if in_place else None, free_count_out=c if in_place else None)
    fits = want is not None
    if fits:
        api.check()
    else:
        with pytest.raises(api.TernaryError):
            api.check()
        want = dict(lengths=lengths, free_count=[count], block_table=table, free_pages=free,
                    slots=[-1] * rows, positions=[0] * rows, requests=[-1] * rows,
                    row_start=[0] * (len(lengths) + 1))
    got = dict(a._asdict(), block_table=t, free_pages=f)
    for name, w in want.items():
        assert np.array_equal(got[name].cpu().numpy(), np.asarray(w).astype(np.int64)), name
    assert (wide[:, table.shape[1]:] == -3).all()
    if not in_place:
        assert np.array_equal(ln.cpu().numpy(), lengths) and int(c) == count
    return fits


@pytest.mark.parametrize("n,page,width", [(1, 16, 1), (1, 1, 40), (3, 16, 5), (31, 7, 9), (32, 16, 20),
                                          (513, 64, 3), (1025, 16, 12), (8192, 16, 2)])
@pytest.mark.parametrize("kind", ["step", "turn", "nothing", "release"])
def test_assign(dev, api, n, page, width, kind):
    rng = np.random.default_rng(n * 7 + page)
    top = page * width
    lengths, table, free, count = _server(rng, n, page, width, top)
    if kind == "step":
        lengths = np.minimum(lengths, top - 1)
        delta = np.ones(n, np.int64)
    elif kind == "turn":
        delta = rng.integers(-top, top + 1, n)
        delta = np.minimum(delta, top - lengths)
    elif kind == "nothing":
        delta = np.zeros(n, np.int64)
    else:
        delta = np.full(n, -2 ** 31)
    rows = int(np.maximum(np.minimum(lengths + delta, top) - lengths, 0).sum()) + (n % 5)
    assert _compare(api, dev, lengths, delta, table, free, count, page, rows, stride=n % 3)
    assert _compare(api, dev, lengths, delta, table, free, count, page, rows, in_place=True)


def test_assign_takes_all_or_nothing(dev, api):
    lengths, delta = np.array([3, 0, 20]), np.array([6, 5, 1])
    table = np.array([[4, -1, -1, -1], [-1] * 4, [7, 8, 9, -1]])
    free = np.array([5, 2, 3, 0, 0, 0, 0, 0])
    assert _compare(api, dev, lengths, delta, table, free, 3, 8, 12)           # takes the last page
    assert not _compare(api, dev, lengths, delta, table, free, 1, 8, 12)       # one page too few
    assert not _compare(api, dev, lengths, delta, table, free, 3, 8, 11)       # one row too few
    assert not _compare(api, dev, lengths, np.array([30, 0, 0]), table, free, 3, 8, 64)   # table too narrow
    assert not _compare(api, dev, np.array([-1, 0, 0]), delta, table, free, 3, 8, 64)
    assert not _compare(api, dev, lengths, delta, table, free, -1, 8, 64)
    assert not _compare(api, dev, lengths, delta, table, free, 9, 8, 64)
    # pages come back and are taken in the same step
    assert _compare(api, dev, lengths, np.array([10, 0, -20]), table, free, 0, 8, 10)


def test_assign_error_codes(dev, api):
    one = i32([0], dev)
    for delta, count, status in (([9], [0], "TW_ERR_BUFSIZE"), ([9], [-1], "TW_ERR_CORRUPT")):
        api.kv_assign(one, i32(delta, dev), i32([[0, 0]], dev), i32([0, 1], dev), i32(count, dev), 8, 16)
        with pytest.raises(api.TernaryError, match=status):
            api.check()


def test_assign_without_rows(dev, api):
    assert _compare(api, dev, np.array([5, 9]), np.array([-5, -1]), np.array([[0, 1], [2, 3]]),
                    np.array([0] * 4), 0, 8, 0)


# ------------------------------------------------------- rotate and append
def _pool(torch, dev, pages, page, hk, d, dtype, order):
    """Pools with the given order of dimensions in memory, filled with a pattern."""
    size = dict(p=pages, t=page, h=hk)
    base = [torch.full([size[c] for c in order] + [d], 3, dtype=dtype, device=dev) for _ in range(2)]
    perm = [order.index(c) for c in "pth"] + [3]
    return [b.permute(perm) for b in base]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "i8"])
@pytest.mark.parametrize("rows,heads,hk,d,rot,inter,order", [
    (1, 12, 2, 128, 128, False, "pth"), (33, 12, 2, 128, 128, True, "pht"), (7, 9, 3, 80, 40, False, "pth"),
    (130, 4, 4, 64, 64, False, "pth"), (5, 8, 1, 256, 256, False, "pht"), (3, 2, 1, 16, 8, True, "pth"),
    (9, 3, 3, 96, 0, False, "pht"), (40, 8, 1, 256, 128, True, "pth")])
def test_rope_append(dev, api, dtype, rows, heads, hk, d, rot, inter, order):
    import torch
    rng = np.random.default_rng(rows + heads)
    page = 8 if rows % 2 else 5
    pages = -(-rows // page) + 2
    T = dict(bf16=torch.bfloat16, f16=torch.float16, i8=torch.int8)[dtype]
    k, v = _pool(torch, dev, pages, page, hk, d, T, order)
    before = [k.clone(), v.clone()]
    scales = [torch.full((pages, page, hk), -1.0, device=dev) for _ in range(2)] if dtype == "i8" else [None, None]
    cache = api.KVCache(k, v, *scales)
    qkv = rng.standard_normal((rows, (heads + 2 * hk) * d)).astype(np.float32)
    qkv[rows // 2, heads * d:heads * d + d] = 0           # a key of zeros
    x = G.to_dev(qkv, dev)
    q, kn, vn = x.split([heads * d, hk * d, hk * d], dim=1)
    slots = rng.permutation(pages * page)[:rows]
    skip = rng.random(rows) < 0.2
    slots[skip] = -1
    pos = rng.integers(0, 2 ** 20, rows)
    pos[0] = 0
    inv = 10000.0 ** (-np.arange(rot // 2) * 2 / max(rot, 1))
    args = (i32(pos, dev), i32(slots, dev), cache)
    kw = dict(inv_freq=G.to_dev(inv, dev) if rot else None, interleaved=inter)
    out = api.rope_append(q, kn, vn, *args, **kw)
    api.check()
    want, tol = plain64.rotate(qkv[:, :heads * d].reshape(rows, heads, d), pos, inv, inter)
    assert (np.abs(out.cpu().numpy().reshape(want.shape) - want) <= tol + 1e-45).all()
    kw64 = plain64.rotate(qkv[:, heads * d:(heads + hk) * d].reshape(rows, hk, d), pos, inv, inter)
    v64 = qkv[:, (heads + hk) * d:].reshape(rows, hk, d).astype(np.float64)
    for pool, old, sc, (w, t) in ((k, before[0], scales[0], kw64), (v, before[1], scales[1], (v64, 0 * v64))):
        flat = pool.reshape(-1, hk, d).double().cpu().numpy()
        keep = np.setdiff1d(np.arange(pages * page), slots[slots >= 0])
        assert np.array_equal(flat[keep], old.reshape(-1, hk, d).double().cpu().numpy()[keep])
        got, w, t = flat[slots[~skip]], w[~skip], t[~skip]
        if dtype == "i8":
            s = sc.reshape(-1, hk).cpu().numpy().astype(np.float64)
            assert (s[keep] == -1).all()
            s = s[slots[~skip]][..., None]
            top = np.abs(w).max(axis=2, keepdims=True)
            assert (np.abs(s - top / 127) <= (t.max(axis=2, keepdims=True) + 2.0 ** -23 * top) / 127).all()
            # half a code, and the roundings of scale and product (2^-24 each of up to 127 codes)
            assert (np.abs(got * s - w) <= (0.5 + 127 * 4 * 2.0 ** -24) * s + 2 * t.max(axis=2, keepdims=True)).all()
            assert (np.abs(got) <= 127).all()
        else:
            half = plain64.HALF[dtype]
            assert (np.abs(got - w) <= half * np.abs(w) + t * (1 + half) + 2.0 ** -25).all()
    # in place, on a strided q
    assert torch.equal(api.rope_append(q, kn, vn, *args, q_out=q, **kw), out)
    assert q.data_ptr() == x.data_ptr()
    api.check()


def test_append_skips_bad_slots(dev, api):
    import torch
    cache = api.KVCache.empty(2, 4, 1, 16, torch.float16, dev)
    x = torch.randn(3, 16, device=dev)
    out = api.rope_append(x, x, x, i32([0, 1, 2], dev), i32([8, 2, 2 ** 31 - 1], dev), cache)
    with pytest.raises(api.TernaryError, match="TW_ERR_CORRUPT"):
        api.check()
    assert torch.equal(out, x)
    flat = cache.k.reshape(8, 16)
    assert torch.equal(flat[2], x[1].half()) and int((flat != 0).any(dim=1).sum()) == 1


def test_kv_refuses_wrong_tensors(dev, api):
    import torch
    z, t = i32([0, 0], dev), i32([[0, 0], [0, 0]], dev)
    good = dict(lengths=z, delta=i32([1, 1], dev), block_table=t, free_pages=i32([0, 1, 2], dev),
                free_count=i32([3], dev), page_size=4, rows=4)
    for bad, kind in ((dict(delta=z[:1]), ValueError), (dict(lengths=z.long()), TypeError), (dict(rows=-1), ValueError),
                      (dict(block_table=t[:1]), ValueError), (dict(page_size=0), api.TernaryError),
                      (dict(free_count=z), ValueError), (dict(delta=z), api.TernaryError), (dict(page_size="x"), TypeError),
                      (dict(lengths_out=good["delta"]), api.TernaryError)):
        with pytest.raises(kind):
            api.kv_assign(**dict(good, **bad))
    a = api.kv_assign(**good)
    api.check()
    assert a.slots.tolist() == [8, 4, -1, -1] and a.row_start.tolist() == [0, 1, 2]
    cache = api.KVCache.empty(2, 4, 1, 16, torch.float16, dev)
    x = torch.randn(2, 16, device=dev)
    for bad, kind in ((dict(k=x[:, :8]), ValueError), (dict(positions=z.float()), TypeError), (dict(slots=z[:1]), ValueError),
                      (dict(inv_freq=torch.ones(8, device=dev)), TypeError), (dict(q_out=x[:1]), ValueError),
                      (dict(inv_freq=torch.ones(3, dtype=torch.float64, device=dev)), api.TernaryError), (dict(q=x[:, :12]), ValueError)):
        kw = dict(q=x, k=x, v=x, positions=z, slots=i32([-1, -1], dev), cache=cache)
        with pytest.raises(kind):
            api.rope_append(**dict(kw, **bad))
    two = torch.zeros(2, 4, 2, 16, dtype=torch.float16, device=dev)
    for k, v in ((cache.k, cache.v[:1]), (cache.k.float(), cache.v.float()), (two.transpose(2, 3), two.transpose(2, 3))):
        with pytest.raises((TypeError, ValueError)):
            api.KVCache(k, v)
    with pytest.raises(ValueError):
        api.KVCache(torch.zeros(2, 4, 1, 16, dtype=torch.int8, device=dev), torch.zeros(2, 4, 1, 16, dtype=torch.int8, device=dev))
    with pytest.raises(api.TernaryError, match="head_dim"):   # pools of heads of one column
        thin = api.KVCache(cache.k.transpose(2, 3), cache.v.transpose(2, 3))
        api.rope_append(x, x, x, z, i32([-1, -1], dev), thin)
    with pytest.raises(ValueError, match="expanded"):
        api.KVCache(cache.k.expand(2, 4, 3, 16), cache.v.expand(2, 4, 3, 16))


def test_assign_flags_pages_that_are_none(dev, api):
    """A row whose page, in the table or in the list, cannot be one gets no slot; the other rows do."""
    for table, free in (([[-5, 0], [3, 0]], [1, 2]), ([[7, 0], [3, 0]], [1, 2 ** 30])):
        a = api.kv_assign(i32([3, 2], dev), i32([2, 1], dev), i32(table, dev), i32(free, dev), i32([2], dev), 4, 3)
        with pytest.raises(api.TernaryError, match="TW_ERR_CORRUPT"):
            api.check()
        assert a.slots.tolist() == ([-1, 8, 14] if table[0][0] < 0 else [31, -1, 14])


def test_outputs_are_tensors_of_their_own(dev, api):
    """Under gradients, without them and in inference mode; no output is a view of another."""
    import torch
    x = torch.randn(3, 64, device=dev)
    w = torch.rand(64, device=dev).requires_grad_()
    seen = []
    for mode in (torch.enable_grad, torch.no_grad, torch.inference_mode):
        with mode():
            lengths, table = i32([0, 15, 3], dev), i32([[-1, -1], [4, -1], [2, -1]], dev)
            a = api.kv_assign(lengths, i32([2, 2, 1], dev), table, i32([1, 0, 3, 5], dev), i32([4], dev), 16, 6)
            r = api.residual_norm(x, x, pre="rms", pre_weight=w)
            api.check()
            assert all(not t.requires_grad and t._base is None for t in (*a, r.h, r.n))
            before = [t.clone() for t in a]
            a.slots.add_(1)
            a.lengths.zero_()
            for t, b in zip(a[1:2] + a[3:], before[1:2] + before[3:]):
                assert torch.equal(t, b)
            seen.append((before, r.n.clone()))
            if mode is torch.enable_grad:   # what autograd saves of an output stays usable
                (r.n * w).sum().backward()
                n64 = r.n.double()   # three summands: two roundings of at most their sizes' sum
                assert ((w.grad - n64.sum(0)).abs() <= 2 * 2 ** -24 * n64.abs().sum(0)).all()
    for before, n in seen[1:]:
        assert torch.equal(n, seen[0][1]) and all(torch.equal(p, q) for p, q in zip(before, seen[0][0]))
