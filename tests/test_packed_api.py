"""Refusals of the packed-batch entry points that need no device."""
import ctypes

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def hk():
    from tests.conftest import build_native
    build_native()
    import importance_aware_kv_gb300 as hk
    return hk


@pytest.fixture
def cache(hk):
    """The binding's object without a cache behind it: its own checks run first."""
    c = hk.Cache.__new__(hk.Cache)
    c.cfg = hk.CacheConfig(num_layers=1, batch=2, num_q_heads=4, num_kv_heads=2, head_dim=64, dtype="bf16",
                           num_sink=0, recent_window=0, budgets=[8, 8], max_tokens=16)
    c.h, c.device_index, c._torch_dtype = None, 0, torch.bfloat16
    return c


def test_null_cache_is_refused(hk):
    lib, r = hk._lib, hk.hikv_rows(16, 64, 64)
    n = (ctypes.c_int32 * 1)(1)
    p = ctypes.byref(r)
    assert lib.hikv_append_packed(None, 0, n, p, p, None, None, None, None) == hk.HIKV_ERR_INVALID_ARG
    assert lib.hikv_attend_packed(None, 0, n, p, p, None) == hk.HIKV_ERR_INVALID_ARG
    assert lib.hikv_drop(None, 0, 1, n, None) == hk.HIKV_ERR_INVALID_ARG
    assert lib.hikv_device_view(None, None) == hk.HIKV_ERR_INVALID_ARG
    assert "device_view" in hk.hikv_last_error()


@pytest.mark.parametrize("counts", [[1.0, 2.0], [True, False], ["a", "b"]])
def test_counts_are_whole_numbers(cache, counts):
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        cache.append_packed(x, x, counts)
    with pytest.raises(TypeError):
        cache.attend_packed(x, x, counts)


@pytest.mark.parametrize("counts", [[1], [1, 1, 1], [[1, 2]], [-2, 1], [1 << 31, 0]])
def test_counts_fit_the_batch(cache, counts):
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: cache.append_packed(x, x, counts), lambda: cache.attend_packed(x, x, counts),
                 lambda: cache.drop(counts)):
        with pytest.raises(ValueError):
            call()


def test_host_tensors_are_refused(hk, cache):
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="CUDA"):
        cache.append_packed(x, x, np.array([1, 2]))
    with pytest.raises(TypeError, match="CUDA"):
        cache.attend_packed(x, x, torch.tensor([1, 2]))
    with pytest.raises(TypeError, match="CUDA"):
        hk.Rope(torch.zeros(4, 32), torch.zeros(4, 32))
