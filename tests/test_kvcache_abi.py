"""Refusals of the quantised key/value cache's entry points (no GPU needed, no kernel launched)."""
import ctypes

import pytest
import torch

from io_aware_exact_25_b200 import binding, kvcache
from io_aware_exact_25_b200.build import build


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load()


INV, UNS, ALI, WSP, BIG = (binding.FA_ERR_INVALID_ARG, binding.FA_ERR_UNSUPPORTED, binding.FA_ERR_ALIGNMENT,
                           binding.FA_ERR_WORKSPACE, binding.FA_ERR_TOO_LARGE)


def cache(k=16, v=16, ks=16, vs=16, pages=4, page=16, heads=2, d=64, fmt=0):
    return binding.FaKvCache(k, v, ks, vs, pages, page, heads, d, fmt)


def strides(n=128, h=64):
    return (binding.FaStrides * 2)(binding.FaStrides(0, h, n), binding.FaStrides(0, h, n))


CACHES = [
    (dict(page=8), INV), (dict(page=48), INV), (dict(page=256), INV), (dict(page=0), INV), (dict(pages=0), INV),
    (dict(pages=-1), INV), (dict(heads=0), INV), (dict(d=96), UNS), (dict(d=256), UNS), (dict(fmt=2), INV),
    (dict(fmt=-1), INV), (dict(k=None), INV), (dict(vs=None), INV), (dict(k=8), ALI), (dict(ks=4), ALI),
    (dict(pages=1 << 27, page=16, heads=1), BIG), (dict(heads=1 << 17), BIG),
]


def rows(lib, fn, c=None, k=16, v=16, st=None, table=16, pages=4, stride=4, starts=16, cu=16, B=2, T=8):
    c = cache() if c is None else c
    return getattr(lib, fn)(ctypes.byref(c), k, v, strides() if st is None else st, table, pages, stride, starts, cu, B,
                            T, None)


def attend(lib, c=None, q=16, o=16, lse=16, st=None, table=16, pages=4, stride=4, lens=16, cu=16, B=2, Hq=4, T=2,
           mq=1, scale=0.1, causal=1, prefix=0, ws=16, wsb=1 << 40):
    c = cache() if c is None else c
    return lib.fa_fwd_kvcache(q, o, lse, strides() if st is None else st, ctypes.byref(c), table, pages, stride, lens,
                              cu, B, Hq, T, mq, scale, causal, prefix, ws, wsb, None)


@pytest.mark.parametrize("kw,status", CACHES)
def test_caches_are_checked_by_every_entry_point(lib, kw, status):
    c = cache(**kw)
    assert rows(lib, "fa_kv_append", c) == status
    assert rows(lib, "fa_kv_read", c) == status
    assert attend(lib, c, Hq=4 * max(1, kw.get("heads", 2))) == status


@pytest.mark.parametrize("fn", ["fa_kv_append", "fa_kv_read"])
@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INV), (dict(T=-1), INV), (dict(pages=-1), INV), (dict(pages=0), INV), (dict(stride=3), INV),
    (dict(table=None), INV), (dict(cu=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(k=8), ALI),
    (dict(table=2), ALI), (dict(starts=2), ALI), (dict(cu=2), ALI), (dict(st=strides(n=4)), ALI),
    (dict(st=strides(h=-64)), ALI), (dict(B=1 << 25), BIG), (dict(T=(1 << 30) + 1), BIG),
    (dict(B=0), binding.FA_OK), (dict(T=0), binding.FA_OK),
])
def test_rows(lib, fn, kw, status):
    assert rows(lib, fn, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(Hq=3), INV), (dict(Hq=-4), INV), (dict(B=-1), INV), (dict(T=-1), INV), (dict(mq=-1), INV),
    (dict(scale=0.0), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(causal=2), INV),
    (dict(prefix=-16), INV), (dict(prefix=8), INV), (dict(prefix=80), INV), (dict(cu=None, T=3), INV),
    (dict(q=None), INV), (dict(o=None), INV), (dict(lens=None), INV), (dict(table=None), INV), (dict(stride=2), INV),
    (dict(q=8), ALI), (dict(o=4), ALI), (dict(lse=2), ALI), (dict(lens=3), ALI), (dict(st=strides(n=12)), ALI),
    (dict(ws=None), WSP), (dict(wsb=100), WSP), (dict(ws=24), ALI), (dict(T=(1 << 24) + 1), BIG),
    (dict(mq=(1 << 24) + 1), BIG), (dict(Hq=1 << 17), BIG),
    (dict(B=0), binding.FA_OK), (dict(Hq=0), binding.FA_OK), (dict(T=0), binding.FA_OK), (dict(mq=0), binding.FA_OK),
])
def test_attention(lib, kw, status):
    assert attend(lib, **kw) == status


def test_workspace_size(lib):
    size = binding.fwd_kvcache_workspace_size
    assert size(0, 4, 2, 64, 2, 1) == 0 and size(2, 3, 2, 64, 2, 1) == 0 and size(2, 4, 2, 96, 2, 1) == 0
    for d in (64, 128):
        plain, shared = size(4, 16, 4, d, 4, 1), size(4, 16, 4, d, 4, 1, 1024)
        assert 0 < plain < shared
        assert size(1, 16, 4, d, 1, 1, 1024) == size(1, 16, 4, d, 1, 1)  # nothing is shared by one sequence
    assert attend(lib, wsb=size(2, 4, 2, 64, 2, 1) - 1) == WSP


def test_the_python_layer_refuses_what_is_not_on_a_gpu():
    t = torch.zeros((2, 2, 16, 64), dtype=torch.int8)
    s = torch.zeros((2, 2, 16))
    with pytest.raises(ValueError, match="CUDA"):
        kvcache.KVCache.from_tensors(t, t, s, s)
    for kw in (dict(page_size=8), dict(head_dim=96), dict(num_pages=0), dict(dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            kvcache.KVCache(**{"num_pages": 2, "num_kv_heads": 2, "head_dim": 64, **kw})
