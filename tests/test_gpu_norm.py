"""Residual sums with the norms, gate and scale around them, against a plain
form in 64 bits; the codes against the library's own quantisation, bit for bit."""
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


def _case(rng, m, k, post, pre, gate, bias=True):
    c = dict(x=rng.standard_normal((m, k)), y=3 * rng.standard_normal((m, k)) + 0.5)
    for side, kind in (("post", post), ("pre", pre)):
        c[side + "_weight"] = 1 + 0.2 * rng.standard_normal(k) if kind else None
        c[side + "_bias"] = rng.standard_normal(k) if kind == "layer" and bias else None
    c["gate"] = dict(none=None, channel=rng.standard_normal(k), token=rng.standard_normal((m, k)))[gate]
    return {n: None if v is None else v.astype(np.float32) for n, v in c.items()}


def _run(api, dev, c, post, pre, alpha, eps, **kw):
    t = {n: None if v is None else G.to_dev(v, dev) for n, v in c.items()}
    x, y = t.pop("x"), t.pop("y")
    return api.residual_norm(x, y, post=post, pre=pre, alpha=alpha, eps=eps, **t, **kw)


def _want(c, post, pre, alpha, eps):
    d = {n: None if v is None else v.astype(np.float64) for n, v in c.items()}
    return plain64.residual_norm(d["x"], d["y"], post, d["post_weight"], d["post_bias"], d["gate"],
                                 np.float64(np.float32(alpha)), pre, d["pre_weight"], d["pre_bias"],
                                 np.float64(np.float32(eps)))


def _close(got, want, tol):
    got = got.cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("m,k", [(1, 1), (3, 2), (1, 1536), (32, 1536), (5, 1537), (2, 8960), (3, 8959),
                                 (2, 32768), (2, 20001), (300, 64), (7, 130), (2, 16384),
                                 (150, 1536), (148, 4), (2, 4096), (2, 6000), (2, 8000), (2, 12000), (2, 14000), (2, 17000), (2, 3001)])
@pytest.mark.parametrize("post,pre,gate", [(None, "rms", "none"), ("rms", "rms", "channel"),
                                           ("layer", "layer", "token"), ("rms", None, "token"),
                                           (None, "layer", "none")])
def test_residual_norm(dev, api, m, k, post, pre, gate):
    c = _case(np.random.default_rng(m * 31 + k), m, k, post, pre, gate, bias=k % 3 != 0)
    r = _run(api, dev, c, post, pre, 0.7, 1e-5)
    api.check()
    h, n, dh, dn = _want(c, post, pre, 0.7, 1e-5)
    _close(r.h, h, dh)
    if pre:
        _close(r.n, n, dn)
    else:
        assert r.n is None


@pytest.mark.parametrize("m,k", [(1, 128), (33, 1536), (4, 8960), (3, 1541), (1, 5)])
def test_codes_are_those_of_quantize_act(dev, api, m, k):
    import torch
    c = _case(np.random.default_rng(k), m, k, "rms", "layer", "channel")
    plain = _run(api, dev, c, "rms", "layer", 1.0, 1e-6)
    codes = _run(api, dev, c, "rms", "layer", 1.0, 1e-6, quantize=True)
    api.check()
    assert codes.n is None and torch.equal(codes.h, plain.h)
    n = plain.n.cpu().numpy()
    amax = np.abs(n).max(axis=1)
    assert np.array_equal(codes.amax.cpu().numpy(), amax)
    want = np.clip(np.rint(n * (np.float32(127) / amax)[:, None]), -128, 127).astype(np.int8)
    assert np.array_equal(codes.xq.cpu().numpy(), want)
    assert np.array_equal(codes.qsum.cpu().numpy(), want.astype(np.int32).sum(axis=1))
    if k % 128 == 0:
        xq, am, qs = api.quantize_act(plain.n)
        assert torch.equal(xq, codes.xq) and torch.equal(am, codes.amax) and torch.equal(qs, codes.qsum)


def test_codes_of_a_zero_row(dev, api):
    import torch
    x = torch.zeros(2, 256, device=dev)
    r = api.residual_norm(x, pre="rms", quantize=True)
    api.check()
    assert (r.xq == 0).all() and (r.amax == 0).all() and (r.qsum == 0).all() and r.h is x


def test_norm_alone_and_in_place(dev, api):
    import torch
    c = _case(np.random.default_rng(4), 9, 1536, "rms", "rms", "channel")
    want = _run(api, dev, c, "rms", "rms", 0.5, 1e-6)
    x, y = G.to_dev(c["x"], dev), G.to_dev(c["y"], dev)
    w = {n: G.to_dev(c[n], dev) for n in ("post_weight", "gate", "pre_weight")}
    r = api.residual_norm(x, y, post="rms", pre="rms", alpha=0.5, h=x, n=y, **w)
    assert r.h is x and r.n is y and torch.equal(x, want.h) and torch.equal(y, want.n)
    # without y: the norm of x alone, x returned as it is
    a = api.residual_norm(x, pre="rms", pre_weight=w["pre_weight"])
    assert a.h is x and torch.equal(a.n, want.n)
    b = api.residual_norm(x, pre="rms", pre_weight=w["pre_weight"], h=torch.empty_like(x))
    assert torch.equal(b.h, x) and torch.equal(b.n, want.n)
    api.check()


def test_norm_strided_rows(dev, api):
    import torch
    for off in (0, 4, 3):   # aligned and unaligned rows of wider buffers
        c = _case(np.random.default_rng(off), 6, 1536, "layer", "rms", "token")
        want = _run(api, dev, c, "layer", "rms", 0.25, 1e-6)
        wide = {}
        for name in ("x", "y", "gate"):
            t = torch.full((6, 1536 + 12 + off), 9.0, device=dev)
            t[:, off:off + 1536] = G.to_dev(c[name], dev)
            wide[name] = t[:, off:off + 1536]
        h, n = (torch.full((6, 1536 + 12 + off), 9.0, device=dev) for _ in range(2))
        r = api.residual_norm(wide["x"], wide["y"], post="layer", pre="rms", alpha=0.25, gate=wide["gate"],
                              post_weight=G.to_dev(c["post_weight"], dev), post_bias=G.to_dev(c["post_bias"], dev),
                              pre_weight=G.to_dev(c["pre_weight"], dev), h=h[:, off:off + 1536], n=n[:, off:off + 1536])
        api.check()
        hh, nn, dh, dn = _want(c, "layer", "rms", 0.25, 1e-6)
        _close(r.h, hh, dh)
        _close(r.n, nn, dn)
        for t in (h, n):
            assert (t[:, :off] == 9).all() and (t[:, off + 1536:] == 9).all()
        if off != 3:
            assert torch.equal(r.h, want.h) and torch.equal(r.n, want.n)


def test_layer_norm_far_from_zero(dev, api):
    """A mean 3000 times the deviation: the centred values are summed."""
    rng = np.random.default_rng(3)
    c = _case(rng, 4, 1536, None, "layer", "none")
    c["x"] = (3000 + rng.standard_normal((4, 1536))).astype(np.float32)
    c["y"] = np.zeros((4, 1536), np.float32)
    r = _run(api, dev, c, None, "layer", 1.0, 1e-6)
    api.check()
    h, n, dh, dn = _want(c, None, "layer", 1.0, 1e-6)
    _close(r.n, n, dn)


def test_codes_feed_a_projection(dev, api):
    """Norm with codes, then the ternary layer on them, is the ternary layer on the norm's output."""
    import torch
    from ternary_weight_decoder_b200 import synth
    W = synth.weights(1, 1, 256, 1536)
    packed, _, wscale = G.ternarize_gpu(W, dev)
    for m in (3, 200):
        c = _case(np.random.default_rng(m), m, 1536, None, "rms", "none")
        r = _run(api, dev, c, None, "rms", 1.0, 1e-6, quantize=True)
        p = _run(api, dev, c, None, "rms", 1.0, 1e-6)
        a = api.ternary_linear_q(r.xq, r.amax, r.qsum, packed, wscale, 256)
        b = api.ternary_linear(p.n, packed, wscale, 256)
        api.check()
        assert torch.equal(a, b)


def test_norm_refuses_wrong_tensors(dev, api):
    import torch
    x, w = torch.randn(4, 256, device=dev), torch.ones(256, device=dev)
    for kw, kind in ((dict(y=x.half()), TypeError), (dict(y=x[:2]), ValueError), (dict(y=x.cpu()), ValueError),
                     (dict(y=x, gate=w[:8]), ValueError), (dict(pre_weight=w[:100]), ValueError), (dict(pre="batch"), ValueError),
                     (dict(pre_weight=torch.ones(512, device=dev)[::2]), ValueError), (dict(pre=None), ValueError),
                     (dict(quantize=True, n=x), ValueError), (dict(gate=w), api.TernaryError),
                     (dict(pre_bias=w), api.TernaryError), (dict(y=x, h=x[:, :128]), ValueError),
                     (dict(y=x, alpha=float("nan")), api.TernaryError), (dict(y=x, h=torch.zeros(1, 256, device=dev).expand(4, 256)), api.TernaryError)):
        with pytest.raises(kind):
            api.residual_norm(x, **kw)
    with pytest.raises(ValueError):
        api.residual_norm(x[0])
    api.check()


def test_norm_on_another_stream(dev, api):
    import torch
    x, y = torch.randn(64, 1536, device=dev), torch.randn(64, 1536, device=dev)
    want = api.residual_norm(x, y)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [api.residual_norm(x, y, stream=s) for _ in range(10)]
    s.synchronize()
    assert all(torch.equal(g.n, want.n) and torch.equal(g.h, want.h) for g in got)


@pytest.mark.parametrize("m,k", [(150, 1), (150, 256), (150, 171), (1800, 171), (1800, 256), (150, 301), (150, 513),
                                 (150, 1025), (150, 1537), (150, 2049), (150, 2561), (150, 4097), (150, 6145),
                                 (150, 8193), (150, 20001), (2, 1025), (2, 4097), (2, 8193), (150, 2052),
                                 (150, 4100), (150, 6148), (150, 8196), (150, 10244), (150, 12292), (150, 16388),
                                 (2, 4100), (2, 8196), (2, 16388)])
def test_norm_and_codes_at_every_row_shape(dev, api, m, k):
    """Widths on both sides of where threads and columns a thread change, for few rows and for many."""
    c = _case(np.random.default_rng(m + k), m, k, "layer", "rms", "token")
    r = _run(api, dev, c, "layer", "rms", -1.3, 1e-5)
    codes = _run(api, dev, c, "layer", "rms", -1.3, 1e-5, quantize=True)
    api.check()
    h, n, dh, dn = _want(c, "layer", "rms", -1.3, 1e-5)
    _close(r.h, h, dh)
    _close(r.n, n, dn)
    got = r.n.cpu().numpy()
    amax = np.abs(got).max(axis=1)
    assert np.array_equal(codes.amax.cpu().numpy(), amax)
    scale = np.divide(np.float32(127), amax, out=np.zeros_like(amax), where=amax > 0)
    want = np.clip(np.rint(got * scale[:, None]), -128, 127).astype(np.int8)
    assert np.array_equal(codes.xq.cpu().numpy(), want)
    assert np.array_equal(codes.qsum.cpu().numpy(), want.astype(np.int32).sum(axis=1))
