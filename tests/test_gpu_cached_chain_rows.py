"""The cached chain where some of its requests take no token: rows unpacked from
kv_assign's as the chain's documentation says, over caches of different lengths."""
import numpy as np
import pytest

from tests import gpu_util as G
from tests import plain64
from tests.test_gpu_attention import check_all
from tests.test_gpu_cached_chain import SMALL, _build
from tests.test_gpu_kv import i32
from ternary_weight_decoder_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return G.torch_dev()


@pytest.fixture(scope="module")
def api():
    return G.api()


@pytest.mark.parametrize("takes", [[1, 0, 1, 1, 0], [0, 0, 0, 1, 0], [0, 1, 0, 0, 1], [1, 1, 1, 1, 1], [0, 0, 0, 0, 0]])
def test_requests_without_a_token(dev, api, takes):
    import torch
    M, (hidden, kv, hd, inter) = 5, SMALL
    heads, hk = hidden // hd, kv // hd
    chain, _, s = _build(api, dev, M, SMALL, 1, torch.bfloat16, 130)
    before = [3, 0, 9, 5, 14]
    assign = dict(lengths_out=s["lengths"], free_count_out=s["count"])
    api.kv_assign(s["lengths"], i32(before, dev), s["table"], s["free"], s["count"], s["page"], sum(before), **assign)
    cache = chain.caches[0]
    g = torch.Generator(device=dev)
    g.manual_seed(7)
    for pool in (cache.k, cache.v):
        pool.copy_(torch.randn(pool.shape, device=dev, generator=g))
    old = [cache.k.clone(), cache.v.clone()]
    a = api.kv_assign(s["lengths"], i32(takes, dev), s["table"], s["free"], s["count"], s["page"], M, **assign)
    row = a.row_start[:M].long().clamp(max=M - 1)
    took = a.row_start[1:] > a.row_start[:-1]
    s["slots"].copy_(torch.where(took, a.slots[row], -1))
    s["positions"].copy_(torch.where(took, a.positions[row], s["lengths"] - 1))
    assert took.int().tolist() == takes
    now = [n + t for n, t in zip(before, takes)]
    assert s["positions"].tolist() == [n - 1 for n in now]
    x = G.to_dev(synth.activations(131, 0, M, hidden), dev)
    chain.x.copy_(x)
    api.decoder_chain_cached(chain)
    api.check()

    # q and k are the projections of the same input, turned to each request's own place
    h = api.residual_norm(x, pre="rms", pre_weight=chain.norms[0][0]).n
    turned = {}
    for name, n in (("q", heads), ("k", hk)):
        packed, wscale = chain.layers[0][name]
        y = api.ternary_linear(h, packed, wscale, n * hd).cpu().numpy().reshape(M, n, hd)
        turned[name] = plain64.rotate(y, [n - 1 for n in now], s["inv"], False)
    want, tol = turned["q"]
    assert (np.abs(chain.q.cpu().numpy().reshape(want.shape) - want) <= tol).all()
    # each new key and value lies at its request's place; nothing else has changed
    table, page = s["table"].cpu().numpy(), s["page"]
    want, tol = turned["k"]
    for r, t in enumerate(takes):
        if t:
            at = int(table[r, before[r] // page]), before[r] % page
            got = cache.k[at].double().cpu().numpy()
            assert (np.abs(got - want[r]) <= tol[r] + plain64.HALF["bf16"] * (np.abs(want[r]) + tol[r])).all(), r
            assert torch.equal(cache.v[at], chain.v[r].reshape(hk, hd).bfloat16()), r
            for pool, kept in zip((cache.k, cache.v), old):
                kept[at] = pool[at]
    assert torch.equal(cache.k, old[0]) and torch.equal(cache.v, old[1])
    # and every row, idle ones too, attends over what its request holds
    lse = torch.empty(M, heads, device=dev)
    out = api.paged_attention(chain.q, cache, s["table"], s["lengths"], lse=lse)
    assert torch.equal(out, chain.a)
    check_all(api, cache, chain.q.cpu().numpy(), table, now, None, out, lse, heads)
