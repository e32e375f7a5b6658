"""The decoder-layer chain with its cache and norms: every step checked on the
GPU's own input of that step, over a prompt-less generation of several
tokens, against the operators' plain forms and the projections' oracle."""
import numpy as np
import pytest

from oracle import oracle as orc
from tests import gpu_util as G
from tests import plain64
from tests.test_gpu_attention import check_all
from tests.test_gpu_chain import PROJ, _shapes
from tests.test_gpu_kv import i32
from ternary_weight_decoder_b200 import synth

pytestmark = pytest.mark.gpu
SMALL = (256, 128, 64, 512)           # 4 query heads over 2 KV heads
QWEN = (1536, 256, 128, 8960)


@pytest.fixture(scope="module")
def dev():
    return G.torch_dev()


@pytest.fixture(scope="module")
def api():
    return G.api()


def _build(api, dev, M, dims, n_layers, dtype, seed):
    import torch
    hidden, kv, hd, inter = dims
    rng = np.random.default_rng(seed)
    gpu, oracle = [], []
    for li in range(n_layers):
        g, o = {}, {}
        for pi, name in enumerate(PROJ):
            W = synth.weights(seed + li, 60 + pi, *_shapes(hidden, kv, inter)[name])
            packed, _, wscale = G.ternarize_gpu(W, dev)
            g[name], o[name] = (packed, wscale), orc.ternarize(W)
        gpu.append(g)
        oracle.append(o)
    width, page = 8, 4
    s = dict(table=torch.full((M, width), -1, dtype=torch.int32, device=dev), page=page,
             free=i32(rng.permutation(M * width), dev), count=i32([M * width], dev),
             lengths=i32([0] * M, dev), positions=i32([0] * M, dev), slots=i32([0] * M, dev),
             inv=1e6 ** (-np.arange(hd // 2) * 2 / hd))
    caches = [api.KVCache.empty(M * width, page, kv // hd, hd, dtype, dev) for _ in range(n_layers)]
    norms = [tuple(G.to_dev((1 + 0.1 * rng.standard_normal(hidden)).astype(np.float32), dev) for _ in range(2))
             for _ in range(n_layers)]
    out = G.to_dev((1 + 0.1 * rng.standard_normal(hidden)).astype(np.float32), dev)
    chain = api.CachedDecoderChain(gpu, M, hidden, kv, hd, inter, dev, caches, norms, out,
                                   G.to_dev(s["inv"], dev), s["table"], s["lengths"], s["positions"], s["slots"])
    return chain, oracle, s


def _assign(api, s, M, delta=None):
    a = api.kv_assign(s["lengths"], i32([1] * M, s["lengths"].device) if delta is None else delta, s["table"],
                      s["free"], s["count"], s["page"], M, lengths_out=s["lengths"], free_count_out=s["count"])
    s["positions"].copy_(a.positions)
    s["slots"].copy_(a.slots)


def _np(t):
    return t.cpu().numpy()


def _proj(x, codes, y, ctx):
    G.assert_y_close(_np(y), orc.ternary_linear(_np(x), *codes)["y"], ctx)


def _rms(x, w, got):
    n, dn = plain64.norm(_np(x).astype(np.float64), 0.0 * _np(x), "rms", _np(w).astype(np.float64), None, 1e-6)
    assert (np.abs(_np(got) - n) <= dn).all()


@pytest.mark.parametrize("M,dims,dtype", [(1, SMALL, "bf16"), (5, SMALL, "f16"), (12, SMALL, "i8"), (3, QWEN, "bf16")])
def test_cached_chain_steps(dev, api, M, dims, dtype):
    """One layer: each buffer left behind by the run follows from the others."""
    import torch
    T = dict(bf16=torch.bfloat16, f16=torch.float16, i8=torch.int8)[dtype]
    chain, oracle, s = _build(api, dev, M, dims, 1, T, 70 + M)
    hidden, kv, hd, inter = dims
    heads, hk = hidden // hd, kv // hd
    for step in range(6):
        _assign(api, s, M)
        x0 = G.to_dev(synth.activations(80 + step, 0, M, hidden), dev)
        chain.x.copy_(x0)
        for name in ("h", "q", "k", "v", "a", "o", "h1", "g", "u", "act", "d"):
            getattr(chain, name).fill_(float("nan"))
        api.decoder_chain_cached(chain)
        api.check()
        h_in = api.residual_norm(x0, pre="rms", pre_weight=chain.norms[0][0]).n
        _rms(x0, chain.norms[0][0], h_in)
        for n in ("k", "v"):
            _proj(h_in, oracle[0][n], getattr(chain, n), n)
        # q is rotated in place: rotate the projection of the same input
        packed, wscale = chain.layers[0]["q"]
        q = _np(api.ternary_linear(h_in, packed, wscale, hidden)).reshape(M, heads, hd)
        want, tol = plain64.rotate(q, [step] * M, s["inv"], False)
        assert (np.abs(_np(chain.q).reshape(want.shape) - want) <= tol).all()
        lengths = [step + 1] * M
        assert _np(s["lengths"]).tolist() == lengths
        lse = torch.empty(M, heads, device=dev)
        a = api.paged_attention(chain.q, chain.caches[0], s["table"], s["lengths"], lse=lse)
        assert torch.equal(a, chain.a)
        check_all(api, chain.caches[0], _np(chain.q), _np(s["table"]), lengths, None, a, lse, heads)
        _proj(chain.a, oracle[0]["o"], chain.o, "o")
        x1 = x0 + chain.o
        _rms(x1, chain.norms[0][1], chain.h1)
        _proj(chain.h1, oracle[0]["gate"], chain.g, "gate")
        _proj(chain.h1, oracle[0]["up"], chain.u, "up")
        _proj(chain.act, oracle[0]["down"], chain.d, "down")
        assert torch.equal(chain.x, x1 + chain.d)
        _rms(chain.x, chain.norm_out, chain.h)


def test_cached_chain_layers_follow_each_other(dev, api):
    """Two layers in one call give what two one-layer chains give in turn, and
    a replayed graph of the whole step gives the same bytes."""
    import torch
    M, dims = 4, SMALL
    two, _, s2 = _build(api, dev, M, dims, 2, torch.bfloat16, 90)
    hidden, kv, hd, inter = dims
    ones = []
    for li in range(2):
        t = dict(s2, lengths=i32([0] * M, dev))
        cache = [api.KVCache.empty(M * 8, 4, kv // hd, hd, torch.bfloat16, dev)]
        ones.append(api.CachedDecoderChain([two.layers[li]], M, hidden, kv, hd, inter, dev, cache, [two.norms[li]],
                                           two.norms[1][0] if li == 0 else two.norm_out, two.inv_freq, s2["table"],
                                           s2["lengths"], s2["positions"], s2["slots"]))
    xs = [G.to_dev(synth.activations(95 + i, 0, M, hidden), dev) for i in range(5)]
    got = []
    for x in xs:
        _assign(api, s2, M)
        two.x.copy_(x)
        api.decoder_chain_cached(two)
        ones[0].x.copy_(x)
        api.decoder_chain_cached(ones[0])
        ones[1].x.copy_(ones[0].x)
        api.decoder_chain_cached(ones[1])
        api.check()
        assert torch.equal(two.x, ones[1].x) and torch.equal(two.h, ones[1].h)
        for i in range(2):
            assert torch.equal(two.caches[i].k, ones[i].caches[0].k)
        got.append((two.x.clone(), two.h.clone()))
    # the same five steps from a graph, on a fresh state
    rerun, _, s = _build(api, dev, M, dims, 2, torch.bfloat16, 90)
    delta = i32([1] * M, dev)
    inp = torch.zeros_like(xs[0])
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        _assign(api, s, M, delta)
        rerun.x.copy_(inp)
        api.decoder_chain_cached(rerun)
    for x, (wx, wh) in zip(xs, got):
        inp.copy_(x)
        g.replay()
        assert torch.equal(rerun.x, wx) and torch.equal(rerun.h, wh)
    api.check()


def test_cached_chain_padded_batch(dev, api):
    """A row that is padding (no slot, length 0) changes nothing of the others
    and leaves the caches alone."""
    import torch
    M = 3
    full, _, s = _build(api, dev, M, SMALL, 1, torch.float16, 120)
    x = G.to_dev(synth.activations(121, 0, M, SMALL[0]), dev)
    delta = i32([1, 0, 1], dev)
    a = api.kv_assign(s["lengths"], delta, s["table"], s["free"], s["count"], s["page"], M, lengths_out=s["lengths"],
                      free_count_out=s["count"])
    # rows are packed by kv_assign: put each beside its request
    s["slots"].copy_(torch.stack([a.slots[0], a.slots[2], a.slots[1]]))
    full.x.copy_(x)
    api.decoder_chain_cached(full)
    api.check()
    assert (full.a[1] == 0).all() and torch.isfinite(full.x).all()
    used = (full.caches[0].k.reshape(-1, 2 * 64) != 0).any(dim=1)
    assert int(used.sum()) == 2
