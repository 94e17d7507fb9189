"""The binding's parameter helpers of the 8-bit paged cache: what is left out is refused like what is wrong (host only)."""
import pytest

from dictionary_sparse_kv_gb300 import fadkv as F


def test_scales_and_tables_that_are_left_out_are_refused():
    torch = pytest.importorskip("torch")
    pool = torch.zeros((5, 2, 32, 64), dtype=torch.int8)
    k = torch.zeros((3, 2, 64), dtype=torch.float16)
    q = torch.zeros((4, 6, 64), dtype=torch.float16)
    s = torch.ones((5, 2, 2))
    table = torch.zeros((4, 9), dtype=torch.int32)
    full = torch.zeros((8, 2, 32, 64))
    for call in (lambda: F.append8_params(k, k, pool), lambda: F.append8_params(k, k, pool, "head", None, pool, s),
                 lambda: F.read8_params(pool, None, full, table), lambda: F.read8_params(pool, s, full, None),
                 lambda: F.paged8_params(q, q, pool, None, "head", table), lambda: F.paged8_params(q, q, pool, s)):
        with pytest.raises(ValueError):
            call()
    assert F.append8_params(k, k, pool, k_scales=s).block == 16 and F.paged8_params(q, q, pool, s, block_table=table).max_pages == 9
