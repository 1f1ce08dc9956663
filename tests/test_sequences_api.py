"""Refusals of the window, tree and copy entry points that need no device."""
import ctypes

import numpy as np
import pytest
import torch

from tests.test_packed_api import cache, hk  # noqa: F401


def test_null_cache_is_refused(hk):
    lib, r = hk._lib, hk.hikv_rows(16, 64, 64)
    n = (ctypes.c_int32 * 1)(1)
    p = ctypes.byref(r)
    bad = hk.HIKV_ERR_INVALID_ARG
    assert lib.hikv_attend_window(None, 0, n, n, 0, p, p, None) == bad
    assert lib.hikv_attend_tree(None, 0, n, n, 1, p, p, None) == bad
    assert lib.hikv_append_tree(None, 0, n, n, p, p, None, None, None, None) == bad
    assert lib.hikv_tree_masks(None, n, n, n, 1, n, None) == bad
    assert lib.hikv_accept(None, 0, 1, n, n, n, None) == bad
    assert lib.hikv_fork(None, 0, 1, n, None, None) == bad
    assert "fork" in hk.hikv_last_error()


class NoTree:
    ntok, device_index, mask, depth, counts = [1, 2], 0, torch.zeros(3, 1, dtype=torch.int32), None, None


def test_lists_are_whole_numbers(cache):
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    for bad in ([1.0, 2.0], ["a", "b"], [True, False]):
        with pytest.raises(TypeError):
            cache.fork(bad)
        with pytest.raises(TypeError):
            cache.fork([0, 1], same=bad)
        with pytest.raises(TypeError):
            cache.accept(bad, [[], []])
        with pytest.raises(TypeError):
            cache.accept([2, 2], [bad, []])
        with pytest.raises(TypeError):
            cache.attend_window(x, x, [1, 2], bad)


def test_lists_fit_the_batch(cache):
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    for bad in ([1], [0, 1, 0], [[0, 1]], [1 << 31, 0]):
        for call in (lambda: cache.fork(bad), lambda: cache.fork([0, 1], same=bad), lambda: cache.accept(bad, [[], []]),
                     lambda: cache.attend_window(x, x, [1, 2], bad)):
            with pytest.raises(ValueError):
                call()
    with pytest.raises(ValueError):
        cache.accept([1, 1], [[0]])
    with pytest.raises(ValueError):
        cache.accept([1, 1], [[1 << 40], []])


def test_host_tensors_are_refused(hk, cache):
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="CUDA"):
        cache.attend_window(x, x, [1, 2], np.int64(4))
    with pytest.raises(TypeError, match="CUDA"):
        cache.tree(torch.zeros(3, dtype=torch.int32), [1, 2])
    with pytest.raises(TypeError, match="CUDA"):
        hk.Tree([1, 2], torch.zeros(3, 1, dtype=torch.int32))
    with pytest.raises(TypeError, match="CUDA"):
        cache.attend_tree(x, x, NoTree)
    with pytest.raises(ValueError, match="no depth"):
        cache.append_tree(x, x, NoTree, None)
