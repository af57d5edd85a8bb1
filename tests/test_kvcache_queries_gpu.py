"""Attention over the quantised cache with queries at the ends of bf16's range, against 64 bits (the tolerance of
test_kvcache_scales_gpu: it is relative to the scores and holds at any size of query and key)."""
import pytest
import torch

from io_aware_exact_25_b200 import binding
from test_kvcache_gpu import DTYPES, FP8, Batch
from test_kvcache_scales_gpu import GROUPS, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("g", GROUPS)
@pytest.mark.parametrize("power", [-124, -100, -40, 40, 100, 118, 123])
def test_large_queries_of_small_keys_and_small_queries_of_large_keys(dtype, g, power):
    """q times 2^power and the keys' scales times 2^-power: the scores are those of power 0."""
    for d in (64, 128):
        x = Batch(dtype, d, 16, 1, g, q=[4, 1], lens=[200, 33], seed=11)
        x.q.mul_(2.0 ** power)
        x.cache.k_scale.mul_(2.0 ** -power)
        assert x.q.isfinite().all()
        check(x, *x.run())


@pytest.mark.parametrize("g", GROUPS)
def test_queries_of_different_size_in_one_tile(g):
    x = Batch(FP8, 128, 32, 1, g, q=[4, 3], lens=[200, 64], seed=12)
    size = torch.exp2(torch.randint(-60, 6, (x.T, x.g, 1), generator=torch.Generator().manual_seed(2)).float()).cuda()
    x.q.copy_(x.q.float() * size)
    check(x, *x.run())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("g", GROUPS)
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_an_infinity_in_a_query_spoils_that_query(dtype, g, bad):
    """Its scores are infinities of either sign or NaN, all of one sign here, and a softmax of those is NaN; a query that
    sees no key has zeros all the same."""
    x = Batch(dtype, 64, 16, 1, g, q=[4, 2, 1], lens=[70, 1, 20], seed=13)
    x.cache.k[..., 9].copy_(torch.ones((), device="cuda"))
    clean, clean_lse = x.run()
    x.q[1, g - 1, 9] = bad  # sees 68 keys
    x.q[4, 0, 9] = bad      # sees none
    x.q[6, 0, 9] = bad
    o, lse = x.run()
    for t, h in ((1, g - 1), (6, 0)):
        assert o[t, h].isnan().all() and lse[h, t].isnan()
        o[t, h], lse[h, t] = clean[t, h], clean_lse[h, t]
    assert (o[4] == 0).all() and torch.equal(o, clean) and torch.equal(lse, clean_lse)
    assert binding.device_error() == 0
