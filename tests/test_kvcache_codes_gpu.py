"""Codes and scales of the quantised cache at every magnitude of bf16, bit for bit against the exact quotients."""
import pytest
import torch

from io_aware_exact_25_b200 import binding
from io_aware_exact_25_b200.kvcache import KVCache
from test_kvcache_gpu import DTYPES, quantise

pytestmark = pytest.mark.gpu

# exponents of a row's largest entry: both ends of the normal range, where the kernel changes its scaling, and the middle
TOP_EXPONENTS = [127, 126, 125, 124, 120, 60, 0, -60, -98, -99, -100, -101, -118, -119, -124, -125, -126]


def rows_of(top):
    """Rows [., 128] whose largest entry runs over all significands at exponent `top` and whose other entries over all
    significands, of both signs, at `top` and twelve smaller exponents (no entry is larger than the row's largest)."""
    sig = torch.arange(128, 256, dtype=torch.float64) * 2.0 ** -7
    amax = sig * 2.0 ** top
    out = []
    for e in range(13):
        x = torch.minimum((sig * 2.0 ** (top - e))[None].expand(128, -1), amax[:, None])  # [amax, x]
        x = torch.cat([x, -x], 1)                                                          # 256 entries a largest
        for part in x.split(127, 1):
            part = torch.cat([part, part.new_zeros((128, 127 - part.shape[1]))], 1)
            at = 37 + 11 * e % 64  # where the largest entry stands
            out.append(torch.cat([part[:, :at], amax[:, None], part[:, at:]], 1))
    x = torch.cat(out).to(torch.bfloat16)
    assert x.isfinite().all()
    return x


def check_rows(x, dtype):
    T = x.shape[0]
    cache = KVCache(-(-T // 128), 1, 128, 128, dtype)
    table = torch.arange(cache.num_pages, dtype=torch.int32)[None].cuda()
    cu = torch.tensor([0, T], dtype=torch.int32).cuda()
    x = x[:, None].cuda()
    cache.append(x, -x.flip(0), table, cu_seqlens=cu)
    for got, got_scale, want in ((cache.k, cache.k_scale, x), (cache.v, cache.v_scale, -x.flip(0))):
        code, scale = quantise(want[:, 0], dtype)
        wrong = (got.reshape(-1, 128)[:T].view(torch.uint8) != code.view(torch.uint8))
        assert not wrong.any(), (int(wrong.sum()), want[:, 0][wrong][:4].tolist(), want[:, 0].abs().amax(1)[wrong.any(1)][:4].tolist())
        assert torch.equal(got_scale.reshape(-1)[:T], scale)
    assert binding.device_error() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("top", TOP_EXPONENTS)
def test_codes_at_every_magnitude(dtype, top):
    check_rows(rows_of(top), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_subnormal_rows(dtype):
    """Rows of bf16's subnormals, whose significands have from one to seven bits."""
    a = torch.arange(1, 128, dtype=torch.float64)
    x = torch.minimum(a[None].expand(127, -1), a[:, None]) * 2.0 ** -133
    x = torch.cat([x, x[:, :1] * 0], 1)
    x[:, 127] = a * 2.0 ** -133
    check_rows(torch.cat([x, -x]).to(torch.bfloat16), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_small_and_ordinary_rows_side_by_side(dtype):
    """Rows of every magnitude in one call, so that a warp holds several, a NaN and an infinity among them."""
    x = torch.cat([rows_of(t)[::97] for t in (127, 0, -126, 126, -100)])
    x = x[torch.randperm(x.shape[0], generator=torch.Generator().manual_seed(1))]
    T, H = x.shape[0] // 6, 6
    x = x[:T * H].view(T, H, 128).clone()
    x[3, 2, 5], x[5, 4, 0] = float("inf"), float("nan")
    cache = KVCache(-(-T // 64), H, 128, 64, dtype)
    table = torch.arange(cache.num_pages, dtype=torch.int32)[None].cuda()
    cu = torch.tensor([0, T], dtype=torch.int32).cuda()
    cache.append(x.cuda(), x.cuda(), table, cu_seqlens=cu)
    good = x.isfinite().all(-1)
    assert int((~good).sum()) == 2
    code, scale = quantise(x[good].cuda(), dtype)
    for got, got_scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        got = got.transpose(1, 2).reshape(-1, H, 128)[:T]
        got_scale = got_scale.transpose(1, 2).reshape(-1, H)[:T]
        assert torch.equal(got.view(torch.uint8)[good.cuda()], code.view(torch.uint8))
        assert torch.equal(got_scale[good.cuda()], scale) and got_scale[~good.cuda()].isnan().all()
