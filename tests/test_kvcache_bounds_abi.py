"""Sizes that the cache's C entry points refuse or take for an empty problem (no GPU needed, no kernel launched)."""
import pytest

from io_aware_exact_25_b200 import binding
from test_kvcache_abi import INV, attend, lib  # noqa: F401  (lib is the fixture)


@pytest.mark.parametrize("kw,status", [
    (dict(mq=0, cu=None), INV),                       # one max_q for all, and it does not give total_q
    (dict(mq=0, cu=None, T=0), binding.FA_OK),
    (dict(mq=1, cu=None, T=0), binding.FA_OK),
    (dict(mq=0, cu=None, B=0), binding.FA_OK),
    (dict(mq=0), binding.FA_OK),                      # no sequence has queries; the rows are of no sequence
])
def test_no_queries(lib, kw, status):  # noqa: F811
    assert attend(lib, **kw) == status
