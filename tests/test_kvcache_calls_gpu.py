"""What the cache's Python calls accept and refuse (GPU tensors; test_kvcache_abi has the C entry points' refusals)."""
import pytest
import torch

from io_aware_exact_25_b200 import binding
from io_aware_exact_25_b200.kvcache import KVCache, flash_attention_kvcache
from test_kvcache_gpu import FP8, INT8, Batch

pytestmark = pytest.mark.gpu


def attend(x, max_seqlen_q, **kw):
    return flash_attention_kvcache(x.q, x.cache, x.table_dev, x.seqlens, cu_seqlens_q=x.cu, max_seqlen_q=max_seqlen_q,
                                   return_lse=True, **kw)


@pytest.mark.parametrize("n", [0, -1, -(1 << 32)])
def test_a_bound_that_leaves_no_query_is_refused(n):
    """It would return outputs that nothing wrote."""
    x = Batch(INT8, 64, 16, 1, 2, q=[2, 1], lens=[20, 32], seed=1)
    with pytest.raises(ValueError):
        attend(x, n)
    with pytest.raises(ValueError):
        binding.fwd_kvcache(x.q, x.cache.buffers, x.table_dev, x.seqlens, n, cu_seqlens_q=x.cu)
    with pytest.raises(ValueError):
        flash_attention_kvcache(x.q, x.cache, x.table_dev, x.seqlens, max_seqlen_q=n)


@pytest.mark.parametrize("n", [2, 3, 1 << 24, (1 << 24) + 1, (1 << 31) - 1, 1 << 31, 1 << 32, (1 << 32) + 1, 1 << 62])
@pytest.mark.parametrize("prefix", [0, 16])
def test_a_generous_bound_changes_nothing(n, prefix):
    x = Batch(FP8, 64, 16, 1, 2, q=[2, 1], lens=[20, 32], prefix=prefix, seed=2)
    o, lse = attend(x, 2, prefix_len=prefix)
    o2, lse2 = attend(x, n, prefix_len=prefix)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    x.check(o, lse)
