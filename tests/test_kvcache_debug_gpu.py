"""The quantised cache's entry points through the bounds-checking build (as test_debug_build_gpu has the others'): no check
fails, and results equal the release build's bit for bit."""
import pytest
import torch

from io_aware_exact_25_b200 import binding
from io_aware_exact_25_b200.kvcache import KVCache, flash_attention_kvcache
from test_debug_build_gpu import _run_both
from test_kvcache_gpu import DTYPES, FP8, INT8, Batch

pytestmark = pytest.mark.gpu


def _equal(ref, got):
    for r, g in zip(ref, got):
        assert torch.equal(r.nan_to_num(-1.0), g.nan_to_num(-1.0)) and torch.equal(r.isnan(), g.isnan())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,page,Hkv", [(64, 16, 3), (128, 128, 2), (128, 32, 16)])
def test_append_and_read(dtype, d, page, Hkv):
    new, past = [5, 0, 1, 130, 17], [3, 9, 64, 0, 100]
    gen = torch.Generator().manual_seed(d + page)
    T, pages = sum(new) + 3, 240 // page + 1
    table = torch.randperm(5 * pages, generator=gen).to(torch.int32).view(5, pages).cuda()
    cu = (torch.tensor([0] + new).cumsum(0) + 1).to(torch.int32).cuda()  # rows of no sequence at both ends
    starts = torch.tensor(past, dtype=torch.int32).cuda()
    wide = torch.randn((T, 2 * Hkv + 1, d), generator=gen).to(torch.bfloat16).cuda()

    def run():
        cache = KVCache(5 * pages, Hkv, d, page, dtype)
        cache.append(wide[:, :Hkv], wide[:, Hkv + 1:], table, starts, cu_seqlens=cu)
        out = torch.zeros((T, 2 * Hkv, d), dtype=torch.bfloat16, device="cuda")
        binding.kv_read(cache.buffers, table, T, starts, cu, k=out[:, :Hkv], v=out[:, Hkv:])
        one = torch.zeros((5, 2, Hkv, d), dtype=torch.bfloat16, device="cuda")
        binding.kv_read(cache.buffers, table, 5, starts, k=one[:, 0], v=one[:, 1])
        return cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale, out, one

    _equal(*_run_both(run))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kw", [
    dict(d=128, page=16, Hkv=2, g=4, q=[1] * 7, lens=[1, 17, 700, 0, 5000, 33, 128]),           # 4 rows
    dict(d=64, page=64, Hkv=3, g=3, q=[5, 1, 0, 2], lens=[300, 1, 9, 2000]),                    # 15 rows
    dict(d=128, page=32, Hkv=1, g=24, q=[1] * 5, lens=[900, 40, 0, 3000, 128]),                 # 24 rows, few items
    dict(d=64, page=16, Hkv=8, g=6, q=[5, 3] * 16, lens=[70 * i + 5 for i in range(32)]),       # 30 rows, more items than SMs
    dict(d=128, page=128, Hkv=2, g=2, q=[300, 7, 1], lens=[900, 200, 64]),                      # several row tiles
    dict(d=64, page=32, Hkv=4, g=2, q=[1] * 200, lens=[(37 * i) % 500 for i in range(200)]),    # more items than CTAs
])
@pytest.mark.parametrize("causal", [True, False])
def test_attention(dtype, kw, causal):
    x = Batch(dtype, seed=61, **kw)
    (o, lse), got = _run_both(lambda: x.run(causal))
    _equal((o, lse), got)
    x.check(o, lse, causal=causal)


@pytest.mark.parametrize("kw", [
    dict(dtype=INT8, d=128, page=16, Hkv=2, g=4, q=[1] * 3, lens=[100, 64, 70], prefix=64),
    dict(dtype=FP8, d=64, page=32, Hkv=2, g=4, q=[1, 3, 0, 2] * 5, lens=[1000 + 31 * i for i in range(20)], prefix=960),
    dict(dtype=INT8, d=128, page=64, Hkv=1, g=3, q=[100, 200], lens=[700, 640], prefix=512),
    dict(dtype=FP8, d=128, page=16, Hkv=2, g=4, q=[2, 1, 3], lens=[100, 0, 40], prefix=64),
])
@pytest.mark.parametrize("causal", [True, False])
def test_shared_prefix(kw, causal):
    x = Batch(seed=62, **kw)
    (o, lse), got = _run_both(lambda: x.run(causal))
    _equal((o, lse), got)
    x.check(o, lse, causal=causal)


def test_uniform_batch_and_strided_output():
    x = Batch(INT8, 64, 16, 2, 4, q=[3, 3], lens=[50, 20], seed=63)

    def run():
        out = torch.zeros((6, 9, 64), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((8, 6), device="cuda")
        binding.fwd_kvcache(x.q, x.cache.buffers, x.table_dev, x.seqlens, 3, o=out[:, 1:], lse=lse)
        return out, lse, flash_attention_kvcache(x.q.view(2, 3, 8, 64), x.cache, x.table_dev, x.seqlens)

    _equal(*_run_both(run))
