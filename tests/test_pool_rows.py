"""A pool whose K and V rows cannot be counted in 32 bits with a sign, as the
coordinates of tensor copies are, is refused before anything is allocated."""
import pytest

from tests.test_packed_api import hk  # noqa: F401


@pytest.mark.parametrize("page,pages", [(64, 1 << 24), (16, 1 << 26), (1 << 20, 1 << 10), (128, (1 << 31) - 1)])
def test_rows_past_31_bits_are_refused(hk, page, pages):
    cfg = hk.CacheConfig(num_layers=1, batch=1, num_q_heads=4, num_kv_heads=2, head_dim=64, dtype="bf16", num_sink=0,
                         recent_window=0, budgets=[32, 32], max_tokens=128, page_tokens=page, pool_pages=pages)
    with pytest.raises(hk.HikvError, match="pool") as e:
        hk.hikv_create_cache(cfg)
    assert e.value.status == hk.HIKV_ERR_UNSUPPORTED
