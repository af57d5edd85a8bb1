"""Attention over the quantised cache where the values' scales differ widely, against 64 bits.

A query's result depends on the keys that it sees and on no others, however large the scale of a value next to them that
a causal mask or a shorter length hides.  Tolerance, for row i of one head, with the names of test_kvcache_gpu's header
(x, p, A, delta): the codes enter the products as they are, and a value's scale multiplies its probability in fp32 before
the one rounding of the two to f16, 2^-11.  Below f16's normal range that rounding is off by at most 2^-25 where the row
sum is at least 2^7 on the scale of a power of two P <= 2 max_j vs_j over the keys that the row sees; a row's largest code
is top (127, 448), so each of N keys adds at most 2^-32 P top <= 2^-31 V, V = max |v| over the keys that the row sees:
  |o - ref| <= 2^-8 |ref| + A (2^-11 + 2^-20 + 2 delta) + N 2^-31 V
"""
import math

import pytest
import torch

from io_aware_exact_25_b200 import binding
from test_kvcache_gpu import DTYPES, FP8, INT8, Batch

pytestmark = pytest.mark.gpu

GROUPS = [2, 20, 80]  # with four queries 8, 80 and 320 rows per key head: each of the kernels


def check(x, o, lse, causal=True):
    scale = 1.0 / math.sqrt(x.d)
    t = 0
    for b, (nq, n) in enumerate(zip(x.q_lens, x.lens)):
        k, v = x.values("k", b), x.values("v", b)
        i = torch.arange(nq, device="cuda")
        end = (n - nq + 1 + i).clamp(0, n) if causal else torch.full((nq,), n, device="cuda")
        sees = torch.arange(n, device="cuda")[None] < end[:, None]
        # [heads, queries, ...]
        q, got, got_lse = x.q[t:t + nq].double().transpose(0, 1), o[t:t + nq].double().transpose(0, 1), lse[:, t:t + nq].double()
        kk, vv = (y.transpose(0, 1).repeat_interleave(x.g, 0) for y in (k, v))
        s = (q @ kk.mT * scale).masked_fill(~sees, -math.inf)
        ref_lse = torch.logsumexp(s, 2)
        p = torch.exp(s - ref_lse[..., None]).masked_fill(~sees, 0)
        ref, A = p @ vv, p @ vv.abs()
        X = ((q.abs() @ kk.abs().mT) * scale).masked_fill(~sees, 0).amax(2)
        Y = (q.abs().amax(2, keepdim=True) * kk.abs().sum(2)[:, None] * scale).masked_fill(~sees, 0).amax(2)
        big = s.abs().masked_fill(~sees, 0).amax(2)
        delta = 4 * (x.d + 16) * 2.0 ** -24 * X + 2.0 ** -24 * Y + 2.0 ** -21 * (1 + big)
        V = (vv.abs().amax(2)[:, None] * sees).amax(2)
        tol = 2.0 ** -8 * ref.abs() + A * (2.0 ** -11 + 2.0 ** -20 + 2 * delta)[..., None] + (n * 2.0 ** -31 * V)[..., None]
        off = (got - ref).abs()
        assert got.isfinite().all(), b
        assert (off <= tol).all(), (b, (off / tol).max().item())
        assert ((got_lse - ref_lse).abs() <= delta + 2.0 ** -20 * (1 + ref_lse.abs())).all(), b
        t += nq
    assert binding.device_error() == 0


def scale_value(x, b, pos, factor):
    x.cache.v_scale[x.table[b, pos // x.page].item(), :, pos % x.page] *= factor


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("g", GROUPS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [20, 40, 110])
def test_values_that_a_query_does_not_see(dtype, g, d, power):
    """The last keys' values are up to 2^110 times the others'; the first queries do not see them."""
    for n in (200, 132, 128):
        x = Batch(dtype, d, 16, 1, g, q=[4, 2], lens=[n, 64], seed=power)
        scale_value(x, 0, n - 2, 2.0 ** power)
        scale_value(x, 0, n - 1, 2.0 ** (power // 2))
        check(x, *x.run())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("g", GROUPS)
@pytest.mark.parametrize("causal", [True, False])
def test_values_of_a_prefix_past_a_short_sequence(dtype, g, causal):
    """Sequences that end inside the shared prefix, before a value of 2^40 times the others' size."""
    x = Batch(dtype, 128, 16, 2, g, q=[2, 1, 1], lens=[300, 100, 161], prefix=256, seed=3)
    scale_value(x, 0, 150, 2.0 ** 40)
    check(x, *x.run(causal), causal)
    x = Batch(dtype, 64, 32, 1, g, q=[2, 1, 1], lens=[300, 130, 31], prefix=256, seed=4)
    scale_value(x, 0, 131, 2.0 ** 40)
    scale_value(x, 0, 31, 2.0 ** 60)
    check(x, *x.run(causal), causal)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("g", GROUPS)
@pytest.mark.parametrize("power", [-110, -60, -33, -31, 31, 33, 60, 110])
def test_values_all_large_or_all_small(dtype, g, power):
    x = Batch(dtype, 64, 16, 1, g, q=[4, 1], lens=[300, 20], seed=5)
    x.cache.v_scale.mul_(2.0 ** power)
    check(x, *x.run())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("g", GROUPS)
def test_scales_that_grow_along_the_keys(dtype, g):
    """From 2^-100 to 2^100 over the keys, in steps of a slice and of a key, and falling again."""
    for step in (1, 17, 64):
        x = Batch(dtype, 128, 32, 1, g, q=[3], lens=[1300], seed=6)
        up = -100 + torch.div(torch.arange(1300), step, rounding_mode="floor") * (200 * step / 650)
        up = torch.minimum(torch.minimum(up, 200 - up), torch.tensor(100.0))
        page, slot = x.table[0][torch.arange(1300) // 32].long().cuda(), torch.arange(1300).cuda() % 32
        x.cache.v_scale[page, :, slot] *= torch.exp2(up)[:, None].cuda()
        check(x, *x.run())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [16, 40, 160])
def test_one_key_is_its_value(dtype, d, g):
    """A query of one key returns the value, rounded once to f16 on the way: the codes and their scale enter exactly."""
    x = Batch(dtype, d, 16, 1, g, q=[1] * 96, lens=[1] * 96, seed=7)
    check(x, *x.run())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [16, 40, 160])
def test_a_value_next_to_a_border_of_bf16(dtype, d, g):
    """Values above the middle of 1 and 1 + 2^-7 by 1.1 to 2 times 2^-11: one rounding to f16 does not carry them to the
    other side, two or three do."""
    x = Batch(dtype, d, 16, 1, g, q=[1] * 256, lens=[1] * 256, seed=17)
    over = torch.linspace(1.1, 2.0, 256, dtype=torch.float64) * 2.0 ** -11
    for b in range(256):
        page = x.table[b, 0].item()
        code = (3 + 2 * b) % 64 + 64 if dtype == INT8 else 1.0 + b % 8 / 8
        x.cache.v[page, :, 0] = torch.tensor(code, dtype=torch.float32).to(dtype).cuda()
        x.cache.v_scale[page, :, 0] = float((1 + 2.0 ** -8) * (1 + over[b]) / code)
    check(x, *x.run())


@pytest.mark.parametrize("g", GROUPS)
def test_all_values_zero(g):
    x = Batch(INT8, 64, 16, 1, g, q=[4], lens=[150], seed=8)
    x.cache.v_scale.masked_fill_(~x.cache.v_scale.isnan(), 0.0)
    o, lse = x.run()
    assert (o == 0).all()
    check(x, o, lse)


@pytest.mark.parametrize("g", GROUPS)
def test_scales_that_are_not_finite_among_large_ones(g):
    """A NaN and an infinite scale spoil the queries that see them, whatever else the tile holds."""
    x = Batch(FP8, 128, 16, 1, g, q=[4], lens=[140], seed=9)
    scale_value(x, 0, 139, 2.0 ** 50)
    clean, clean_lse = x.run()
    for bad in (float("nan"), float("inf")):
        x.cache.v_scale[x.table[0, 138 // 16].item(), :, 138 % 16] = bad
        o, lse = x.run()
        assert not o[2:].isfinite().any() and torch.equal(lse, clean_lse)
        assert torch.equal(o[:2], clean[:2])
