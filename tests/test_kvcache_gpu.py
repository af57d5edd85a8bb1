"""The quantised key/value cache and the attention that reads it, against plain 64-bit implementations.

Tolerances are derived, not fitted.  For row i of one head, with x the fp64 scores, p their softmax, N keys:
  scores    the products are exact (f16 operands, up to 11 + 8 significant bits) and summed in fp32: at most
            4 (d + 16) 2^-24 X, X = max_j scale sum_c |q_c k_jc|, with the factor 4 for a tensor core that truncates
            instead of rounding; q's f16 form is exact above 2^-14 of the row's largest entry and off by at most
            2^-24 of it below: 2^-24 Y, Y = max_j scale max_c |q_c| sum_c |k_jc|; the exponent argument and the
            exponential add 2^-21 (1 + max |x|).  Their sum is delta.
  o         2^-8 |o| (the output's bf16 rounding) + A (r 2^-11 + 2 delta), A = sum_j p_j |v_j|.  r counts the f16
            roundings, of p, and above 16 rows per key head of the value's scale and of the scaled value: 1 or 3; the
            latter two are also off by at most 2^-25 V where they leave f16's normal range, 2^-22 below the largest
            scale.  + N 2^-32 V for probabilities below f16's normal range (each off by at most 2^-25 on a
            scale where the row sum is at least 2^7), V = max |v|, + 2^-20 A for fp32 sums and the merge.
  lse       delta + 2^-20 (1 + |lse|)
The cache's codes have to equal those of the exact quotient bit for bit; scales are one fp32 division, so they do too.
"""
import math

import pytest
import torch

from io_aware_exact_25_b200 import binding
from io_aware_exact_25_b200.kvcache import KVCache, flash_attention_kvcache

pytestmark = pytest.mark.gpu

TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
INT8, FP8 = torch.int8, torch.float8_e4m3fn


def quantise(x, dtype):
    """Codes and scales of bf16 rows by the definition: the exact quotient in 64 bits (its distance from a border
    between two codes is 0 or above 2^-17 of its value, so 64 bits decide it), half to even."""
    x = x.double()
    amax = x.abs().amax(-1, keepdim=True)
    y = torch.where(amax > 0, x * TOP[dtype] / amax.clamp_min(1e-300), torch.zeros_like(x))
    code = torch.round(y).to(torch.int8) if dtype == INT8 else y.float().to(FP8)
    return code, (amax[..., 0] / TOP[dtype]).float()


def poison(cache):
    """Slots never written: NaN scales, and codes whose bytes are e4m3's NaN."""
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        c.view(torch.uint8).fill_(0x7f)
        s.fill_(float("nan"))


def make_table(B, pages_each, num_pages, shared, gen):
    order = torch.randperm(num_pages, generator=gen).to(torch.int32)
    table = torch.full((B, max(pages_each + [1])), -1, dtype=torch.int32)
    at = shared
    for b in range(B):
        n = pages_each[b]
        s = min(shared, n)
        table[b, :s] = order[:s]
        table[b, s:n] = order[at:at + n - s]
        at += n - s
    assert at <= num_pages
    return table


class Batch:
    """A filled cache and its queries."""

    def __init__(self, dtype=INT8, d=128, page=16, Hkv=2, g=4, q=(1,), lens=(40,), prefix=0, seed=0, scale=1.0,
                 heavy=False):
        gen = torch.Generator().manual_seed(seed)
        self.B, self.q_lens, self.lens, self.prefix = len(lens), list(q), list(lens), prefix
        self.Hkv, self.g, self.d, self.page = Hkv, g, d, page
        each = [-(-n // page) for n in lens]
        shared = prefix // page
        num = sum(each) + shared + 2
        self.cache = KVCache(num, Hkv, d, page, dtype)
        poison(self.cache)
        self.table = make_table(self.B, each, num, shared, gen)
        for b, n in enumerate(lens):
            first = min(prefix, n) if b > 0 else 0
            for name in ("k", "v"):
                x = torch.randn((n - first, Hkv, d), generator=gen) * scale
                if heavy:  # rows of very different size, a few large channels
                    x = x * torch.exp2(torch.randint(-12, 13, (n - first, Hkv, 1), generator=gen).float())
                    x[..., ::16] *= 8
                code, sc = quantise(x.to(torch.bfloat16), dtype)
                pos = torch.arange(first, n)
                if name == "k" and heavy:
                    code, sc = quantise((x / x.abs().amax(-1, keepdim=True).clamp_min(1e-9) * 3).to(torch.bfloat16),
                                        dtype)
                pg, sl = self.table[b][pos // page].long().cuda(), (pos % page).cuda()
                getattr(self.cache, name).view(torch.uint8)[pg, :, sl] = code.view(torch.uint8).cuda()
                getattr(self.cache, name + "_scale")[pg, :, sl] = sc.cuda()
        # a sequence inside a longer prefix than its own keys still names the shared pages
        self.T = sum(q)
        self.cu = torch.tensor([0] + list(q)).cumsum(0).to(torch.int32).cuda()
        self.q = (torch.randn((self.T, Hkv * g, d), generator=gen) * scale).to(torch.bfloat16).cuda()
        self.table_dev = self.table.cuda()
        self.seqlens = torch.tensor(lens, dtype=torch.int32).cuda()

    def values(self, name, b):
        """fp64 [n, Hkv, d]"""
        n = self.lens[b]
        pos = torch.arange(n)
        pg, sl = self.table[b][pos // self.page].long().cuda(), (pos % self.page).cuda()
        code = getattr(self.cache, name)[pg, :, sl].float().double()
        return code * getattr(self.cache, name + "_scale")[pg, :, sl].double()[..., None]

    def run(self, causal=True, prefix=None, **kw):
        return flash_attention_kvcache(self.q, self.cache, self.table_dev, self.seqlens, cu_seqlens_q=self.cu,
                                       max_seqlen_q=max(self.q_lens), causal=causal, return_lse=True,
                                       prefix_len=self.prefix if prefix is None else prefix, **kw)

    def check(self, o, lse, causal=True, scale=None):
        scale = scale or 1.0 / math.sqrt(self.d)
        wide = max(self.q_lens + [self.T if self.prefix else 0]) * self.g > 16
        r, sub = (3, 2.0 ** -25) if wide else (1, 0.0)
        t = 0
        for b, (nq, n) in enumerate(zip(self.q_lens, self.lens)):
            k, v = self.values("k", b), self.values("v", b)
            for h in range(self.Hkv * self.g):
                if nq == 0:
                    continue
                q = self.q[t:t + nq, h].double()
                kk, vv = k[:, h // self.g], v[:, h // self.g]
                end = (n - nq + 1 + torch.arange(nq)).clamp(0, n).cuda() if causal else torch.full((nq,), n).cuda()
                sees = torch.arange(n).cuda()[None] < end[:, None]
                got, got_lse = o[t:t + nq, h].double(), lse[h, t:t + nq].double()
                empty = end == 0
                assert (got[empty] == 0).all() and (got_lse[empty] == -math.inf).all()
                if n == 0 or empty.all():
                    continue
                x = (q @ kk.t() * scale).masked_fill(~sees, -math.inf)
                ref_lse = torch.logsumexp(x, 1)
                p = torch.exp(x - ref_lse[:, None]).masked_fill(~sees, 0)
                ref = p @ vv
                A = p @ vv.abs()
                X = ((q.abs() @ kk.abs().t()) * scale).masked_fill(~sees, 0).amax(1)
                Y = (q.abs().amax(1, keepdim=True) * kk.abs().sum(1)[None] * scale).masked_fill(~sees, 0).amax(1)
                big = x.abs().masked_fill(~sees, 0).amax(1)
                delta = 4 * (self.d + 16) * 2.0 ** -24 * X + 2.0 ** -24 * Y + 2.0 ** -21 * (1 + big)
                V = torch.stack([vv[s].abs().max() if s.any() else vv.new_zeros(()) for s in sees])
                tol = 2.0 ** -8 * ref.abs() + A * (r * 2.0 ** -11 + 2.0 ** -20 + 2 * delta)[:, None] \
                    + ((n * 2.0 ** -32 + sub) * V)[:, None]
                ok = ~empty
                bad = (got - ref).abs()[ok] - tol[ok]
                assert not torch.isnan(got[ok]).any()
                assert (bad <= 0).all(), (b, h, bad.max().item(), (got - ref).abs()[ok].max().item())
                assert ((got_lse - ref_lse).abs()[ok] <= (delta + 2.0 ** -20 * (1 + ref_lse.abs()))[ok]).all()
            t += nq
        assert binding.device_error() == 0


DTYPES = [pytest.param(INT8, id="int8"), pytest.param(FP8, id="fp8")]


# ------------------------------------------------------------ append and read

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,page,Hkv,new,past", [
    (128, 16, 1, [1], [0]),
    (128, 16, 8, [1] * 5, [0, 15, 16, 17, 300]),
    (64, 32, 3, [5, 1, 70, 33], [0, 31, 32, 7]),
    (128, 64, 5, [130, 0, 1, 64], [63, 5, 0, 64]),
    (64, 128, 16, [257, 3], [127, 128]),
    (64, 16, 2, [0, 0, 9, 0, 40, 0], [3, 4, 5, 6, 7, 8]),
    (128, 32, 1, [1] * 70, list(range(70))),
])
def test_append_codes_are_exact_and_read_returns_their_values(dtype, d, page, Hkv, new, past):
    gen = torch.Generator().manual_seed(sum(new) + d)
    B, T = len(new), sum(new)
    each = [-(-(n + p) // page) for n, p in zip(new, past)]
    cache = KVCache(sum(each) + 2, Hkv, d, page, dtype)
    poison(cache)
    table = make_table(B, each, sum(each) + 2, 0, gen)
    k = torch.randn((T, Hkv, d), generator=gen).to(torch.bfloat16)
    v = (torch.randn((T, Hkv, d), generator=gen) * torch.exp2(torch.randint(-40, 40, (T, Hkv, 1), generator=gen).float()))
    v = v.to(torch.bfloat16)
    k[0, 0] = 0                                  # a row of zeros
    k[-1, -1, :] = 0
    k[-1, -1, 3] = 2.0                           # one entry
    v[0, 0, :] = torch.tensor([1.0, 0.5, -0.5, -1.0]).repeat(d // 4)  # 127 / 2 lies on a border
    expect = {n: getattr(cache, n).clone() for n in ("k", "v", "k_scale", "v_scale")}
    t = 0
    for b in range(B):
        pos = torch.arange(past[b], past[b] + new[b])
        pg, sl = table[b][pos // page].long().cuda(), (pos % page).cuda()
        for name, x in (("k", k), ("v", v)):
            code, sc = quantise(x[t:t + new[b]], dtype)
            expect[name].view(torch.uint8)[pg, :, sl] = code.view(torch.uint8).cuda()
            expect[name + "_scale"][pg, :, sl] = sc.cuda()
        t += new[b]
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
    starts = torch.tensor(past, dtype=torch.int32).cuda()
    cache.append(k.cuda(), v.cuda(), table.cuda(), starts, cu_seqlens=cu)
    for name in ("k", "v"):
        assert torch.equal(getattr(cache, name).view(torch.uint8), expect[name].view(torch.uint8)), name
        a, e = getattr(cache, name + "_scale"), expect[name + "_scale"]
        assert torch.equal(a.isnan(), e.isnan()) and torch.equal(a.nan_to_num(-1), e.nan_to_num(-1)), name
    kr, vr = cache.read(table.cuda(), cu, T, starts=starts)
    for x, r in ((k, kr), (v, vr)):
        code, sc = quantise(x, dtype)
        assert torch.equal(r, (code.float() * sc[..., None]).to(torch.bfloat16).cuda())
    assert binding.device_error() == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_quotient_of_two_bf16_significands_is_rounded_exactly(dtype):
    """amax runs over all 128 significands, x over all 128 at twelve smaller exponents, both signs: every way a bf16
    quotient can lie on or near a border."""
    sig = torch.arange(128, 256).float()
    rows = []
    for e in range(12):
        rows.append(torch.stack([sig] * 128) * 2.0 ** -(e + 1))
    x = torch.cat([torch.cat([r, -r], 1) for r in rows])              # [12 * 128, 256]
    a = sig.repeat(12)                                                # a row's amax; every entry is at most half of 2a
    x = torch.minimum(x, a[:, None])
    x = torch.cat([x[:, :127], a[:, None], x[:, 127:254], a[:, None]], 1).reshape(-1, 1, 128).to(torch.bfloat16)
    T = x.shape[0]
    cache = KVCache(-(-T // 128), 1, 128, 128, dtype)
    table = torch.arange(cache.num_pages, dtype=torch.int32)[None].cuda()
    cu = torch.tensor([0, T], dtype=torch.int32).cuda()
    cache.append(x.cuda(), -x.cuda(), table, cu_seqlens=cu)
    code, sc = quantise(x, dtype)
    got = cache.k.reshape(-1, 128)[:T]
    assert torch.equal(got.view(torch.uint8), code[:, 0].view(torch.uint8).cuda())
    ncode, _ = quantise(-x, dtype)
    assert torch.equal(cache.v.reshape(-1, 128)[:T].view(torch.uint8), ncode[:, 0].view(torch.uint8).cuda())
    assert torch.equal(cache.k_scale.reshape(-1)[:T], sc[:, 0].cuda())


@pytest.mark.parametrize("dtype", DTYPES)
def test_extreme_rows(dtype):
    """The largest and smallest bf16 numbers, and rows that hold an infinity or a NaN."""
    d = 64
    top = torch.finfo(torch.bfloat16).max
    tiny = 2.0 ** -133  # the smallest subnormal
    rows = [torch.full((d,), top), torch.full((d,), tiny), torch.full((d,), -2.0 ** -126),
            torch.linspace(-top, top, d), torch.linspace(-1e-38, 1e-38, d)]
    bad = [torch.ones(d), torch.ones(d), torch.ones(d)]
    bad[0][5], bad[1][0], bad[2][63] = float("inf"), float("nan"), float("-inf")
    x = torch.stack(rows + bad)[:, None].to(torch.bfloat16)
    T = x.shape[0]
    cache = KVCache(1, 1, d, 16, dtype)
    table = torch.zeros((1, 1), dtype=torch.int32).cuda()
    cu = torch.tensor([0, T], dtype=torch.int32).cuda()
    cache.append(x.cuda(), x.cuda(), table, cu_seqlens=cu)
    k, v = cache.read(table, cu, T)
    good = x.isfinite().all(-1)[:, 0].cuda()  # (the span from -top to top is itself infinite in fp32: its row is not)
    assert int(good.sum()) == 4 and torch.equal(k[good], v[good]) and k[~good].isnan().all() and v[~good].isnan().all()
    # one step of the row's codes: amax / 127 (half of it), or 2^-4 of the value (its half step) plus e4m3's smallest
    ref = x.cuda()[good].double()
    amax = ref.abs().amax(-1, keepdim=True)
    step = amax / 254 if dtype == INT8 else ref.abs() * 2.0 ** -4 + amax * 2.0 ** -10 / 448
    # bf16 rounding of the value, and the scale's own rounding where it is subnormal (2^-149 on each code)
    tol = step + 2.0 ** -8 * ref.abs() + 2.0 ** -133 + TOP[dtype] * 2.0 ** -149
    assert ((k[good].double() - ref).abs() <= tol).all()


def test_append_and_read_strided_views_and_rows_of_no_sequence():
    gen = torch.Generator(device="cuda").manual_seed(5)
    Hkv, d, T = 3, 128, 20
    qkv = torch.randn((T, 2 * Hkv + 6, d), generator=gen, device="cuda").to(torch.bfloat16)
    k, v = qkv[:, :Hkv], qkv[:, Hkv + 1:2 * Hkv + 1]
    cache = KVCache(4, Hkv, d, 16, INT8)
    poison(cache)
    table = torch.tensor([[2, 0], [1, 3]], dtype=torch.int32).cuda()
    cu = torch.tensor([2, 9, 17], dtype=torch.int32).cuda()  # rows 0, 1 and 17.. belong to no sequence
    cache.append(k, v, table, cu_seqlens=cu)
    assert int((~cache.k_scale.isnan()).sum()) == 15 * Hkv
    out = torch.full((T, 2 * Hkv, d), 7.0, device="cuda").to(torch.bfloat16)
    binding.kv_read(cache.buffers, table, T, cu_seqlens=cu, k=out[:, :Hkv], v=out[:, Hkv:])
    assert (out[:2] == 7).all() and (out[17:] == 7).all()
    for x, y in ((k, out[:, :Hkv]), (v, out[:, Hkv:])):
        code, sc = quantise(x[2:17], INT8)
        assert torch.equal(y[2:17], (code.float() * sc[..., None]).to(torch.bfloat16))
    # a transposed view is copied, not misread
    kt = k.transpose(0, 1).contiguous().transpose(0, 1)
    c2 = KVCache(4, Hkv, d, 16, INT8)
    poison(c2)
    c2.append(kt, torch.empty((Hkv, d, T), dtype=torch.bfloat16, device="cuda").permute(2, 0, 1).copy_(v), table,
              cu_seqlens=cu)
    assert torch.equal(c2.k, cache.k) and torch.equal(c2.v, cache.v)


def test_pages_outside_the_cache_are_reported_and_not_touched():
    Hkv, d = 2, 64
    x = torch.ones((4, Hkv, d), device="cuda").to(torch.bfloat16)
    cache = KVCache(2, Hkv, d, 16, INT8)
    starts = torch.zeros(4, dtype=torch.int32).cuda()
    table = torch.tensor([[0], [2], [-1], [1]], dtype=torch.int32).cuda()
    cache.append(x, x, table, starts)
    assert binding.device_error() == 5
    assert int((cache.k_scale != 0).sum()) == 2 * Hkv
    cu = torch.arange(5, dtype=torch.int32).cuda()
    k, v = cache.read(table, cu, 4)
    assert binding.device_error() == 5
    assert (k[1] == 0).all() and (k[2] == 0).all() and (k[0] == 1).all() and (v[3] == 1).all()
    # positions past the table, and before it
    cache.append(x, x, table, torch.tensor([16, 3, -1, 1], dtype=torch.int32).cuda())
    assert binding.device_error() == 5


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_one_token(dtype, d, page):
    """The single-token form at lengths around every border: slices of 32, units of 128, pages."""
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 500, 1025]
    x = Batch(dtype, d, page, Hkv=2, g=4, q=[1] * len(lens), lens=lens, seed=page + d)
    x.check(*x.run())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Hkv,g", [(1, 1), (3, 1), (2, 3), (1, 7), (2, 16), (1, 17), (1, 32), (1, 33), (2, 71), (1, 128)])
def test_groups_of_heads(dtype, Hkv, g):
    x = Batch(dtype, 128, 16, Hkv, g, q=[1, 1, 1], lens=[3, 130, 700], seed=g)
    x.check(*x.run())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,page,Hkv,g,q,lens", [
    (128, 32, 2, 4, [2, 4, 1, 3], [2, 300, 129, 64]),
    (64, 16, 3, 1, [5, 1, 16, 9], [5, 1, 200, 33]),
    (128, 64, 2, 6, [5, 4, 3, 2, 1], [50, 1000, 3, 2, 128]),
    (128, 16, 1, 8, [40, 3], [40, 90]),
    (64, 128, 2, 3, [100, 7, 1], [333, 7, 128]),
    (128, 64, 4, 1, [257, 128, 300], [600, 128, 1300]),
    (64, 32, 1, 5, [333], [2000]),
])
def test_several_tokens(dtype, causal, d, page, Hkv, g, q, lens):
    x = Batch(dtype, d, page, Hkv, g, q=q, lens=lens, seed=sum(q))
    x.check(*x.run(causal), causal=causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("g", [2, 20])
def test_rows_and_sequences_that_see_nothing(causal, g):
    """No keys, fewer keys than queries (the first queries see none), sequences without queries."""
    x = Batch(INT8, 128, 16, 2, g, q=[1, 3, 0, 5, 2, 0], lens=[0, 1, 9, 2, 40, 0], seed=3)
    x.check(*x.run(causal), causal=causal)


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_short_sequences_and_one_long(dtype):
    """More sequences than a block has threads; one of them as long as all the others."""
    gen = torch.Generator().manual_seed(9)
    lens = torch.randint(0, 40, (400,), generator=gen).tolist()
    lens[137] = 9000
    x = Batch(dtype, 64, 16, 1, 2, q=[1] * 400, lens=lens, seed=1)
    x.check(*x.run())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("g,q", [(4, 1), (8, 40)])
def test_rows_of_very_different_size(dtype, g, q):
    """Key and value rows whose scales span 2^24, and a few large channels."""
    x = Batch(dtype, 128, 32, 2, g, q=[q, q], lens=[700, 1500], seed=8, heavy=True)
    x.check(*x.run())


@pytest.mark.parametrize("g", [4, 40])
def test_peaked_and_flat_rows(g):
    """Scores so large that one key takes everything, and so small that all keys weigh the same."""
    for scale in (6.0, 1e-4):
        x = Batch(INT8, 128, 64, 2, g, q=[1, 2], lens=[300, 777], seed=4, scale=scale)
        x.check(*x.run())


def test_long_cache_past_32_bit_offsets():
    """A cache of more than 2^31 bytes of codes whose last pages are the ones in use."""
    Hkv, d, page = 8, 128, 128
    pages = (1 << 31) // (Hkv * page * d) + 40
    cache = KVCache(pages, Hkv, d, page, FP8)
    gen = torch.Generator().manual_seed(0)
    L = 2500
    n = -(-L // page)
    table = (pages - 1 - torch.arange(n, dtype=torch.int32))[None]
    k, v = (torch.randn((L, Hkv, d), generator=gen).to(torch.bfloat16) for _ in "kv")
    cu = torch.tensor([0, L], dtype=torch.int32).cuda()
    cache.append(k.cuda(), v.cuda(), table.cuda(), cu_seqlens=cu)
    kr, vr = cache.read(table.cuda(), cu, L)
    code, sc = quantise(k, FP8)
    assert torch.equal(kr, (code.float() * sc[..., None]).to(torch.bfloat16).cuda())
    for nq in (1, 50):
        x = Batch.__new__(Batch)
        x.B, x.q_lens, x.lens, x.prefix, x.Hkv, x.g, x.d, x.page, x.T = 1, [nq], [L], 0, Hkv, 2, d, page, nq
        x.cache, x.table, x.table_dev = cache, table, table.cuda()
        x.cu, x.seqlens = torch.tensor([0, nq], dtype=torch.int32).cuda(), torch.tensor([L], dtype=torch.int32).cuda()
        x.q = torch.randn((nq, 2 * Hkv, d), generator=gen).to(torch.bfloat16).cuda()
        x.check(*x.run())


@pytest.mark.parametrize("dtype", DTYPES)
def test_infinities_and_nan_stay_with_the_rows_that_see_them(dtype):
    """A key or value row with a NaN makes NaN of the queries that see it and of no others."""
    x = Batch(dtype, 64, 16, 1, 2, q=[4, 4, 1], lens=[70, 70, 70], seed=2)
    clean, clean_lse = x.run()
    for name, b in (("k_scale", 0), ("v_scale", 1)):
        pos = 68  # seen by the last two of four queries
        getattr(x.cache, name)[x.table[b, pos // 16].item(), :, pos % 16] = float("nan")
    x.q[8, 1, 7] = float("nan")
    o, lse = x.run()
    assert o[2:4].isnan().all() and o[6:8].isnan().all() and o[8, 1].isnan().all()
    assert lse[:, 2:4].isnan().all() and not lse[:, 4:8].isnan().any()
    for rows in (slice(0, 2), slice(4, 6)):
        assert torch.equal(o[rows], clean[rows]) and torch.equal(lse[:, rows], clean_lse[:, rows])
    assert torch.equal(o[8, 0], clean[8, 0])


def test_uniform_batch_forms_views_and_untouched_rows():
    x = Batch(INT8, 128, 16, 2, 4, q=[3, 3], lens=[50, 20], seed=6)
    o, lse = x.run()
    q4 = x.q.view(2, 3, 8, 128)
    o4 = flash_attention_kvcache(q4, x.cache, x.table_dev, x.seqlens)
    assert torch.equal(o4.view(6, 8, 128), o)
    # q and o as strided views, a wider block table, rows of no sequence left alone
    wide = torch.randn((10, 12, 128), device="cuda").to(torch.bfloat16)
    wide[2:8, 2:10] = x.q
    out = torch.full((10, 9, 128), 5.0, device="cuda").to(torch.bfloat16)
    table = torch.full((2, 11), -9, dtype=torch.int32, device="cuda")
    table[:, 3:3 + x.table.shape[1]] = x.table_dev
    cu = torch.tensor([2, 5, 8], dtype=torch.int32).cuda()
    l2 = torch.full((8, 10), 3.0, device="cuda")
    binding.fwd_kvcache(wide[:, 2:10], x.cache.buffers, table[:, 3:], x.seqlens, 3, cu_seqlens_q=cu,
                        o=out[:, :8], lse=l2)
    assert torch.equal(out[2:8, :8], o) and torch.equal(l2[:, 2:8], lse)
    assert (out[:2] == 5).all() and (out[8:] == 5).all() and (out[:, 8] == 5).all()
    assert (l2[:, :2] == 3).all() and (l2[:, 8:] == 3).all()
    # non-contiguous heads are copied
    qt = x.q.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(flash_attention_kvcache(qt, x.cache, x.table_dev, x.seqlens, cu_seqlens_q=x.cu, max_seqlen_q=3), o)


# -------------------------------------------------------------- shared prefix

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,page,Hkv,g,q,prefix,own", [
    (128, 16, 2, 4, [1] * 3, 16, [1, 5, 40]),
    (64, 16, 4, 4, [1] * 8, 2048, [1, 2, 17, 33, 64, 100, 128, 129]),
    (128, 64, 1, 1, [1] * 40, 192, list(range(1, 41))),
    (128, 32, 2, 8, [1] * 33, 480, [7 * (i % 13) + 1 for i in range(33)]),
    (128, 128, 2, 2, [3, 1, 0, 5], 384, [3, 200, 7, 130]),
    (64, 32, 1, 6, [30, 50, 1], 1024, [30, 300, 1]),
    (128, 16, 8, 4, [1] * 2, 4000, [1, 900]),
])
def test_shared_prefix(dtype, d, page, Hkv, g, q, prefix, own):
    x = Batch(dtype, d, page, Hkv, g, q=q, lens=[prefix + n for n in own], prefix=prefix, seed=prefix)
    o, lse = x.run()
    x.check(o, lse)
    x.check(*x.run(prefix=0))
    x.check(*x.run(causal=False), causal=False)


def test_shared_prefix_longer_than_some_sequences():
    """A padded slot without keys, a sequence inside the prefix, one that ends with it: their queries see what their
    own lengths allow."""
    x = Batch(INT8, 128, 16, 2, 4, q=[2, 1, 3, 2, 1], lens=[100, 0, 40, 64, 65], prefix=64, seed=12)
    for causal in (True, False):
        x.check(*x.run(causal), causal=causal)


def test_shared_prefix_of_one_sequence_and_untouched_rows():
    x = Batch(INT8, 128, 16, 2, 4, q=[1], lens=[100], prefix=64, seed=13)
    assert torch.equal(x.run()[0], x.run(prefix=0)[0])
    x = Batch(FP8, 64, 16, 2, 4, q=[1, 2], lens=[100, 90], prefix=64, seed=14)
    x.check(*x.run())
    out = torch.full((6, 8, 64), 5.0, device="cuda").to(torch.bfloat16)
    l2 = torch.full((8, 6), 3.0, device="cuda")
    q = torch.zeros((6, 8, 64), device="cuda").to(torch.bfloat16)
    q[1:4] = x.q
    binding.fwd_kvcache(q, x.cache.buffers, x.table_dev, x.seqlens, 2, cu_seqlens_q=x.cu + 1, o=out,
                        lse=l2, prefix_len=64)
    x.check(out[1:4], l2[:, 1:4])  # (not to the bit: 24 rows may take another kernel than 12)
    assert (out[0] == 5).all() and (out[4:] == 5).all() and (l2[:, 0] == 3).all() and (l2[:, 4:] == 3).all()


# ------------------------------------------------ together, and as programs run

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,Hkv,g", [(128, 2, 4), (64, 1, 3)])
def test_a_prompt_and_its_answers(dtype, d, Hkv, g):
    """As a server uses them: a shared prompt is appended once and attended in chunks, then several answers are
    decoded from its pages with the prefix shared, each step appending a token and attending.  Each step is
    checked against the 64-bit attention over the cache, and the cache against what was appended."""
    gen = torch.Generator().manual_seed(d + g)
    page, P, A, steps = 16, 150, 4, 20
    whole = P // page                                # pages of the prompt that are full, shared by the answers
    cache = KVCache(64, Hkv, d, page, dtype)
    poison(cache)
    x = Batch.__new__(Batch)
    x.Hkv, x.g, x.d, x.page, x.cache, x.prefix = Hkv, g, d, page, cache, 0
    table = torch.arange(16, dtype=torch.int32)[None]
    x.table, x.table_dev = table, table.cuda()
    k, v = (torch.randn((P, Hkv, d), generator=gen).to(torch.bfloat16).cuda() for _ in "kv")
    for first, n in ((0, 70), (70, 80)):             # two chunks
        cu = torch.tensor([0, n], dtype=torch.int32).cuda()
        start = torch.tensor([first], dtype=torch.int32).cuda()
        cache.append(k[first:first + n], v[first:first + n], x.table_dev, start, cu_seqlens=cu)
        x.q = torch.randn((n, Hkv * g, d), generator=gen).to(torch.bfloat16).cuda()
        x.q_lens, x.lens, x.cu, x.seqlens, x.T = [n], [first + n], cu, start + n, n
        x.check(*x.run())
    # the answers: the full pages are shared, the prompt's tail is written to each answer's own page
    table = torch.full((A, 16), -1, dtype=torch.int32)
    table[:, :whole] = torch.arange(whole, dtype=torch.int32)
    for a in range(A):
        table[a, whole:whole + 3] = torch.arange(16 + 3 * a, 19 + 3 * a, dtype=torch.int32)
    x.table, x.table_dev, x.prefix = table, table.cuda(), whole * page
    tail = P - whole * page
    kt, vt = k[whole * page:].repeat(A, 1, 1), v[whole * page:].repeat(A, 1, 1)
    cache.append(kt, vt, x.table_dev, torch.full((A,), whole * page, dtype=torch.int32).cuda(),
                 cu_seqlens=(torch.arange(A + 1, dtype=torch.int32) * tail).cuda())
    lens = torch.full((A,), P, dtype=torch.int32).cuda()
    x.q_lens, x.cu, x.T = [1] * A, torch.arange(A + 1, dtype=torch.int32).cuda(), A
    for step in range(steps):
        kn, vn = (torch.randn((A, Hkv, d), generator=gen).to(torch.bfloat16).cuda() for _ in "kv")
        cache.append(kn, vn, x.table_dev, lens)
        lens = lens + 1
        x.q = torch.randn((A, Hkv * g, d), generator=gen).to(torch.bfloat16).cuda()
        x.seqlens, x.lens = lens, [P + step + 1] * A
        x.check(*x.run())
    kr, _ = cache.read(x.table_dev, torch.tensor([0, P, P, P, P], dtype=torch.int32).cuda(), P)
    code, sc = quantise(k, dtype)
    assert torch.equal(kr, (code.float() * sc[..., None]).to(torch.bfloat16))


def test_two_runs_are_equal_and_the_workspace_does_not_matter():
    for kw in (dict(q=[1] * 5, lens=[900, 30, 5000, 64, 700]), dict(q=[60, 3], lens=[900, 4000], g=3),
               dict(q=[1] * 20, lens=[600 + i for i in range(20)], prefix=512)):
        x = Batch(INT8, 128, 64, 2, seed=21, **{"g": 4, **kw})
        o, lse = x.run()
        need = binding.fwd_kvcache_workspace_size(x.B, x.Hkv * x.g, x.Hkv, 128, x.T, max(x.q_lens), x.prefix)
        for fill in (0, 255):
            ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            o2, lse2 = x.run(workspace=ws)
            assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_captured_steps_follow_lengths_tables_and_contents():
    """Append and attention captured once and replayed over several steps, two graphs in turn."""
    x = Batch(INT8, 128, 16, 2, 4, q=[1] * 3, lens=[30, 200, 75], seed=31)
    room = torch.full((3, 40), 0, dtype=torch.int32)
    room[:, :x.table.shape[1]] = x.table.clamp_min(0)
    cache = KVCache(140, 2, 128, 16, INT8)
    room = torch.arange(120, dtype=torch.int32).view(3, 40)
    x.cache, x.table, x.table_dev = cache, room, room.cuda()
    gen = torch.Generator().manual_seed(1)
    k, v = (torch.randn((305, 2, 128), generator=gen).to(torch.bfloat16).cuda() for _ in "kv")
    cache.append(k, v, x.table_dev, cu_seqlens=torch.tensor([0, 30, 230, 305], dtype=torch.int32).cuda())
    lens = torch.tensor([30, 200, 75], dtype=torch.int32).cuda()
    kn, vn = torch.zeros((3, 2, 128), dtype=torch.bfloat16).cuda(), torch.zeros((3, 2, 128), dtype=torch.bfloat16).cuda()
    x.seqlens = lens
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.append(kn, vn, x.table_dev, lens)
        x.run()
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cache.append(kn, vn, x.table_dev, lens)
            lens.add_(1)
            out = x.run()
        graphs.append((g, out))
    n = [30, 200, 75]
    for step in range(6):
        if step == 3:
            lens[0] += 90
            n[0] += 90
            fill = [torch.randn((90, 2, 128), generator=gen).to(torch.bfloat16).cuda() for _ in "kv"]
            cache.append(*fill, x.table_dev[:1], (lens[:1] - 90).contiguous(),
                         cu_seqlens=torch.tensor([0, 90], dtype=torch.int32).cuda())
        kn.copy_(torch.randn((3, 2, 128), generator=gen))
        vn.copy_(torch.randn((3, 2, 128), generator=gen))
        x.q.copy_(torch.randn((3, 8, 128), generator=gen))
        g, out = graphs[step % 2]
        g.replay()
        n = [i + 1 for i in n]
        x.lens = n
        x.check(*out)


def test_calls_on_other_streams():
    """Two batches at once on two streams, and a call told its stream."""
    xs = [Batch(INT8, 128, 64, 2, 4, q=[1] * 4, lens=[3000, 10, 700, 64], seed=40 + i) for i in range(2)]
    ref = [x.run() for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            if i == 0:
                with torch.cuda.stream(s):
                    outs[i].append(xs[i].run())
            else:
                outs[i].append(xs[i].run(stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in outs[i]:
            assert torch.equal(o, ref[i][0]) and torch.equal(lse, ref[i][1])
    # a layout that is copied first, on the stream the call was given
    q = xs[0].q.view(4, 1, 8, 128).transpose(2, 3).contiguous().transpose(2, 3)
    torch.cuda.synchronize()
    o = flash_attention_kvcache(q, xs[0].cache, xs[0].table_dev, xs[0].seqlens, stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(o.view(4, 8, 128), ref[0][0])


def test_empty_calls():
    x = Batch(INT8, 64, 16, 1, 2, q=[1, 1], lens=[20, 32], seed=51)
    c, dev = x.cache, "cuda"
    no_rows = torch.empty((0, 1, 64), dtype=torch.bfloat16, device=dev)
    zero = torch.zeros(3, dtype=torch.int32, device=dev)
    before = c.k_scale.clone()
    c.append(no_rows, no_rows, x.table_dev, cu_seqlens=zero)
    k, v = c.read(x.table_dev, zero, 0)
    assert k.shape == v.shape == (0, 1, 64)
    assert torch.equal(before.nan_to_num(-1), c.k_scale.nan_to_num(-1))
    o, lse = flash_attention_kvcache(torch.empty((0, 2, 64), dtype=torch.bfloat16, device=dev), c, x.table_dev, x.seqlens,
                                     cu_seqlens_q=zero, max_seqlen_q=1, return_lse=True)
    assert o.shape == (0, 2, 64) and lse.shape == (2, 0)
    none = torch.empty((0,), dtype=torch.int32, device=dev)
    o = flash_attention_kvcache(torch.empty((0, 1, 2, 64), dtype=torch.bfloat16, device=dev), c,
                                torch.empty((0, 2), dtype=torch.int32, device=dev), none)
    assert o.shape == (0, 1, 2, 64)
    assert binding.device_error() == 0


def test_python_refusals():
    x = Batch(INT8, 64, 16, 2, 2, q=[1, 1], lens=[20, 32], seed=52)
    ok = dict(cu_seqlens_q=x.cu, max_seqlen_q=1)
    call = lambda q=x.q, table=x.table_dev, lens=x.seqlens, **kw: flash_attention_kvcache(q, x.cache, table, lens,
                                                                                          **{**ok, **kw})
    call()
    for bad in (dict(q=x.q.float()), dict(q=x.q[:, :3]), dict(q=x.q[..., :32]), dict(table=x.table_dev.long()),
                dict(table=x.table_dev[0]), dict(table=x.table_dev[:1].expand(2, -1)), dict(lens=x.seqlens[:1]),
                dict(lens=x.seqlens.long()), dict(cu_seqlens_q=x.cu[:2]), dict(max_seqlen_q=None),
                dict(prefix_len=8), dict(prefix_len=1 << 20), dict(prefix_len=-16),
                dict(q=x.q.clone().requires_grad_()), dict(table=x.table),
                dict(q=x.q.view(1, 2, 4, 64)), dict(workspace=torch.empty(16, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(binding.FaError):
        call(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(binding.FaError):
        call(scale=-1.0)
    kv = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    for args in ((kv.float(), kv), (kv[:, :1], kv), (kv, kv[:1]), (kv[:1], kv[:1])):
        with pytest.raises(ValueError):
            x.cache.append(*args, x.table_dev)
    with pytest.raises(ValueError):
        KVCache.from_tensors(x.cache.k, x.cache.v.view(FP8), x.cache.k_scale, x.cache.v_scale)
    with pytest.raises(ValueError):
        KVCache.from_tensors(x.cache.k[:, :, :15], x.cache.v[:, :, :15], x.cache.k_scale, x.cache.v_scale)
    assert binding.device_error() == 0


@pytest.mark.parametrize("g", [2, 20, 80])
def test_an_infinite_scale_spoils_only_the_rows_that_see_it(g):
    x = Batch(INT8, 128, 16, 1, g, q=[4, 2], lens=[200, 64], seed=53)
    clean, clean_lse = x.run()
    x.cache.v_scale[x.table[0, 198 // 16].item(), :, 198 % 16] = float("inf")
    o, lse = x.run()
    assert not o[2:4].isfinite().any() and torch.equal(lse, clean_lse)
    assert torch.equal(o[:2], clean[:2]) and torch.equal(o[4:], clean[4:])


def test_lengths_out_of_range_are_clamped_and_reported():
    x = Batch(INT8, 64, 16, 1, 2, q=[1, 1], lens=[20, 32], seed=50)
    x.seqlens = torch.tensor([20, 1 << 30], dtype=torch.int32).cuda()
    o, lse = x.run()
    assert binding.device_error() == 3
    x.check(o, lse)  # the second length is clamped to the table's 32 positions
    x.seqlens = torch.tensor([-4, 32], dtype=torch.int32).cuda()
    o, lse = x.run()
    assert binding.device_error() == 3 and (o[0] == 0).all()
    x.seqlens = torch.tensor([20, 32], dtype=torch.int32).cuda()
    bad = x.table_dev.clone()
    bad[1, 1] = 1 << 20
    flash_attention_kvcache(x.q, x.cache, bad, x.seqlens)
    assert binding.device_error() == 5


def test_outputs_whose_rows_the_kernels_cannot_address_are_refused():
    """A given output is written in place, so nothing can be copied for it: other strides are an error, and a strided
    one that can be addressed is written where it says."""
    x = Batch(INT8, 64, 16, 2, 2, q=[1, 1], lens=[20, 32], seed=54)
    b, dev = x.cache.buffers, "cuda"
    want, _ = x.run()
    attend = lambda o: binding.fwd_kvcache(x.q, b, x.table_dev, x.seqlens, 1, cu_seqlens_q=x.cu, o=o)
    bf16 = dict(dtype=torch.bfloat16, device=dev)
    apart = torch.zeros((2, 4, 64, 2), **bf16)[..., 0]     # last stride 2
    turned = torch.zeros((2, 64, 4), **bf16).transpose(1, 2)
    narrow = torch.zeros((2, 4, 68), **bf16)[..., :64]     # rows 136 bytes apart
    shifted = torch.zeros(2 * 4 * 64 + 1, **bf16)[1:].view(2, 4, 64)
    for o in (apart, turned, narrow, shifted):
        with pytest.raises(ValueError):
            attend(o)
        assert (o == 0).all()
        kv = o[:, :2]
        for given in (dict(k=kv), dict(v=kv)):
            with pytest.raises(ValueError):
                binding.kv_read(b, x.table_dev, 2, cu_seqlens=x.cu, **given)
    wide = torch.zeros((2, 4, 128), **bf16)
    attend(wide[..., :64])
    assert torch.equal(wide[..., :64].reshape(want.shape), want) and (wide[..., 64:] == 0).all()
    assert binding.device_error() == 0
