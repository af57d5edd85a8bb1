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


def moved(t):
    """The same values in views that the kernels cannot address: off by one element, and (one token, or one head) with
    a stride that nothing is reached by."""
    flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:] = t.flatten()
    out = [flat[1:].view(t.shape)]
    room = torch.zeros(t.numel() + 64, dtype=t.dtype, device=t.device)
    for dim in (0, 1):
        if t.shape[dim] == 1:
            stride = list(t.stride())
            stride[dim] = 13
            out.append(room.as_strided(t.shape, stride).copy_(t))
    for v in out:
        assert torch.equal(v, t) and not binding._rows_usable(v)
    return out


@pytest.mark.parametrize("T,Hkv", [(3, 2), (1, 2), (3, 1), (1, 1)])
def test_inputs_that_the_kernels_cannot_address_are_copied(T, Hkv):
    x = Batch(INT8, 64, 16, Hkv, 1, q=[T], lens=[40], seed=3)
    o, lse = attend(x, T)
    for q in moved(x.q):
        o2, lse2 = flash_attention_kvcache(q, x.cache, x.table_dev, x.seqlens, cu_seqlens_q=x.cu, max_seqlen_q=T,
                                           return_lse=True)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    k, v = (torch.randn((T, Hkv, 64), device="cuda").to(torch.bfloat16) for _ in "kv")
    want = KVCache(1, Hkv, 64, 16, INT8)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    want.append(k, v, table, cu_seqlens=x.cu)
    for k2, v2 in zip(moved(k), moved(v)):
        for given in ((k2, v), (k, v2), (k2, v2)):
            got = KVCache(1, Hkv, 64, 16, INT8)
            got.append(*given, table, cu_seqlens=x.cu)
            assert all(torch.equal(getattr(got, n), getattr(want, n)) for n in ("k", "v", "k_scale", "v_scale"))
    assert binding.device_error() == 0


def test_keys_and_values_that_want_a_gradient_are_refused():
    """As queries are: nothing of the cache is differentiated."""
    cache = KVCache(1, 2, 64, 16, INT8)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    x = torch.ones((1, 2, 64), device="cuda").to(torch.bfloat16)
    grad = x.clone().requires_grad_()
    for k, v in ((grad, x), (x, grad), (grad, grad * 2)):
        with pytest.raises(ValueError, match="no backward"):
            cache.append(k, v, table)
        assert (cache.k_scale == 0).all()
        with torch.no_grad():
            cache.append(k, v, table)
        cache.append(k.detach(), v.detach(), table)
        assert (cache.k_scale[0, :, 0] > 0).all()
        cache.k_scale.zero_()


SHAPES = [  # each kernel and both phases of a shared prefix
    dict(d=128, page=16, Hkv=2, g=4, q=[1] * 5, lens=[700, 80, 300, 65, 1500], prefix=64),
    dict(d=64, page=32, Hkv=2, g=4, q=[1] * 20, lens=[1000 + 7 * i for i in range(20)], prefix=960),
    dict(d=128, page=64, Hkv=1, g=8, q=[5, 3, 4], lens=[900, 70, 2000]),
    dict(d=128, page=64, Hkv=2, g=2, q=[200, 33], lens=[900, 1300]),
]


@pytest.mark.parametrize("kw", SHAPES)
@pytest.mark.parametrize("dtype", [INT8, FP8])
def test_captured_calls_follow_their_lengths(kw, dtype):
    """A captured call replayed with other lengths and queries, an eager one and another graph's between its replays."""
    x = Batch(dtype, seed=71, **kw)
    full = list(x.lens)
    graphs = []
    x.run()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = x.run()
        graphs.append((g, out))
    shorter = [max(n - 17 - 5 * i, kw.get("prefix", 0) // 2 + nq) for i, (n, nq) in enumerate(zip(full, x.q_lens))]
    gen = torch.Generator().manual_seed(3)
    for i, lens in enumerate((full, shorter, [nq for nq in x.q_lens], full)):
        x.lens = lens
        x.seqlens.copy_(torch.tensor(lens, dtype=torch.int32))
        x.q.copy_(torch.randn(x.q.shape, generator=gen))
        want, want_lse = x.run()
        x.check(want, want_lse)
        for g, (o, lse) in (graphs if i % 2 else graphs[::-1]):
            o.fill_(7)
            g.replay()
            assert torch.equal(o, want) and torch.equal(lse, want_lse)
    assert binding.device_error() == 0


def test_every_shape_at_once_on_streams_of_its_own():
    xs = [Batch(dtype, seed=72, **kw) for kw in SHAPES for dtype in (INT8, FP8)]
    want = [x.run() for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[] for _ in xs]
    for _ in range(6):
        for x, s, out in zip(xs, streams, got):
            with torch.cuda.stream(s):
                out.append(x.run())
    torch.cuda.synchronize()
    for w, out in zip(want, got):
        for o, lse in out:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])
    assert binding.device_error() == 0


def test_a_page_that_a_sequence_holds_twice():
    """Nothing says that a table's pages are different ones."""
    x = Batch(INT8, 128, 16, 2, 4, q=[2, 1], lens=[100, 50], seed=73)
    x.table[0, 3], x.table[1, 1] = x.table[0, 1], x.table[0, 2]
    x.table_dev = x.table.cuda()
    x.check(*x.run())


@pytest.mark.parametrize("kw", SHAPES)
def test_a_page_outside_the_cache_spoils_its_sequence_only(kw):
    """It is reported and not touched (device error 5); the other sequences' results stand."""
    x = Batch(INT8, seed=74, **kw)
    o, lse = x.run()
    b, last = len(x.lens) - 1, (x.lens[-1] - 1) // x.page
    rows = x.T - x.q_lens[-1]
    for bad in (x.cache.num_pages, -1, (1 << 31) - 1, -(1 << 31)):
        table = x.table_dev.clone()
        table[b, last] = bad
        o2, lse2 = flash_attention_kvcache(x.q, x.cache, table, x.seqlens, cu_seqlens_q=x.cu, max_seqlen_q=max(x.q_lens),
                                           prefix_len=x.prefix, return_lse=True)
        assert binding.device_error() == 5
        assert torch.equal(o[:rows], o2[:rows]) and torch.equal(lse[:, :rows], lse2[:, :rows])


@pytest.mark.parametrize("g", [2, 40])
@pytest.mark.parametrize("prefix", [0, 32])
@pytest.mark.parametrize("cu", [[0, 3, 1, 4], [-5, 2, 3, 4], [0, 2, 3, 9], [4, 3, 2, 1], [0, 1 << 30, 3, 4]])
def test_offsets_out_of_order_are_reported(g, prefix, cu):
    """Device error 3; what they leave of the tensors is read and written inside them."""
    x = Batch(FP8, 64, 16, 1, g, q=[2, 1, 1], lens=[40, 70, 33], prefix=prefix, seed=75)
    room = torch.full((3, 4, g, 64), 5.0, device="cuda").to(torch.bfloat16)
    lse = torch.full((3, g, 4), 5.0, device="cuda")
    binding.fwd_kvcache(x.q, x.cache.buffers, x.table_dev, x.seqlens, 2,
                        cu_seqlens_q=torch.tensor(cu, dtype=torch.int32).cuda(), prefix_len=prefix, o=room[1], lse=lse[1])
    assert binding.device_error() == 3
    for t in (room, lse):
        assert (t[0] == 5).all() and (t[2] == 5).all()
