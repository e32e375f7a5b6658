"""What the binding of the cache operators and the norms does with Python objects."""
import numpy as np
import pytest

from tests import gpu_util as G
from tests.test_gpu_attention import make
from tests.test_gpu_kv import i32

pytestmark = pytest.mark.gpu


class NoTruth:
    def __bool__(self):
        raise ArithmeticError("neither")


@pytest.fixture(scope="module")
def dev():
    return G.torch_dev()


@pytest.fixture(scope="module")
def api():
    return G.api()


def test_flags_without_a_truth_value(dev, api):
    """The object's own error comes, and nothing is launched."""
    import torch
    cache, q, table = make(api, dev, "bf16", [20, 3], 4, 2, 64, 16, 1, poison=False)
    q, table, lengths = G.to_dev(q, dev), i32(table, dev), i32([20, 3], dev)
    out = torch.full_like(q, 7.0)
    kv = torch.ones(2, 128, device=dev)
    kept = cache.k.clone()
    x = torch.ones(2, 64, device=dev)
    n = torch.full_like(x, 7.0)
    for call in (lambda: api.paged_attention(q, cache, table, lengths, out=out, return_lse=NoTruth()),
                 lambda: api.rope_append(q, kv, kv, lengths, lengths, cache, interleaved=NoTruth(), q_out=out),
                 lambda: api.residual_norm(x, x, n=n, quantize=NoTruth())):
        with pytest.raises(ArithmeticError, match="neither"):
            call()
    assert (out == 7).all() and (n == 7).all() and torch.equal(cache.k, kept)
    api.check()
    assert np.isfinite(api.paged_attention(q, cache, table, lengths).cpu().numpy()).all()
