"""The binding's own part of the window, tree and copy entry points, with the
C calls and the device tensors stood in for: no device is needed."""
import array
import ctypes
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from tests.test_packed_api import cache, hk  # noqa: F401


class DeviceTensor:
    """What the binding asks of a CUDA tensor."""

    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.dtype, self.is_cuda, self.device = torch.Size(shape), dtype, True, "cuda:0"
        self.streams = []

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 1 << 20

    def stride(self):
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s)

    def new_empty(self, shape):
        return DeviceTensor(*shape, dtype=self.dtype)

    def record_stream(self, stream):
        self.streams.append(stream)


@pytest.fixture
def calls(hk, cache, monkeypatch):
    """Calls on a batch of two: the host counts that each C call reads, by name."""
    read = {}

    def c_call(name, at):
        def call(*args):
            read[name] = list((ctypes.c_int32 * 2).from_address(args[at]))
            return hk.HIKV_OK
        return call

    where = {"hikv_tree_masks": 1, "hikv_append_tree": 2, "hikv_attend_tree": 2, "hikv_accept": 3}
    monkeypatch.setattr(hk, "_lib", SimpleNamespace(**{n: c_call(n, at) for n, at in where.items()}))
    monkeypatch.setattr(cache, "_int32", torch.int32, raising=False)
    monkeypatch.setattr(cache, "_row_args", [hk.hikv_rows() for _ in range(4)], raising=False)
    monkeypatch.setattr(cache, "_row_refs", [ctypes.byref(r) for r in cache._row_args], raising=False)
    monkeypatch.setattr(cache, "_stream_int", lambda stream: stream or 0)
    return read


def in_int32(kind, values):
    return {"array": lambda: np.array(values, dtype=np.int32), "tensor": lambda: torch.tensor(values, dtype=torch.int32),
            "buffer": lambda: array.array("i", values), "list": lambda: list(values)}[kind]()


@pytest.mark.parametrize("kind", ["array", "tensor", "buffer", "list"])
def test_a_tree_has_counts_of_its_own(cache, calls, kind):
    """The caller's counts are filled again for the next step while the tree lives."""
    n = in_int32(kind, [3, 4])
    tree = cache.tree(DeviceTensor(7, dtype=torch.int32), n)
    assert calls["hikv_tree_masks"] == [3, 4]
    n[0], n[1] = 12, 1
    kv, q, out = DeviceTensor(7, 2, 64), DeviceTensor(7, 4, 64), DeviceTensor(7, 4, 64)
    rope = SimpleNamespace(device_index=0, ref=None)
    cache.append_tree(kv, kv, tree, rope, q=q, q_out=out)
    cache.attend_tree(q, out, tree)
    cache.accept(tree, [[0], [1, 3]])
    assert calls == {name: [3, 4] for name in calls} and len(calls) == 4
    assert list(tree.ntok) == [3, 4]
    with pytest.raises(TypeError):   # (and what a tree says of itself is not what the calls read)
        tree.ntok[0] = 12


def test_the_default_stream_is_no_new_stream(hk, cache, calls, monkeypatch):
    """Given by its handle, 0, which torch takes as "any stream" where it makes
    one from a handle."""
    used = []

    def external(handle, device=None):
        assert handle != 0
        return handle

    class On:
        def __init__(self, stream):
            used.append(stream)

        def __enter__(self):
            pass

        def __exit__(self, *a):
            pass

    monkeypatch.setattr(cache, "_stream_int", lambda stream: 5 if stream is None else stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch.cuda, "stream", On)
    tree = cache.tree(DeviceTensor(7, dtype=torch.int32), [3, 4], stream=0)
    assert used == ["default"]
    q, out = DeviceTensor(7, 4, 64), DeviceTensor(7, 4, 64)
    cache.attend_tree(q, out, tree, stream=0)
    assert set(tree.mask.streams) <= {"default"}


def test_a_tree_is_held_for_every_stream_that_uses_it(hk, cache, calls, monkeypatch):
    """Its tensors are memory of the stream it was made on: any other one's use
    of them, given by handle or the current one, is known to the allocator."""
    current = [7]
    monkeypatch.setattr(cache, "_stream_int", lambda stream: current[0] if stream is None else stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s, device=None: s)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: 0)
    tree = cache.tree(DeviceTensor(7, dtype=torch.int32), [3, 4])
    kv, q, out = DeviceTensor(7, 2, 64), DeviceTensor(7, 4, 64), DeviceTensor(7, 4, 64)
    rope = SimpleNamespace(device_index=0, ref=None)

    def use(stream=None):
        cache.append_tree(kv, kv, tree, rope, q=q, q_out=out, stream=stream)
        cache.attend_tree(q, out, tree, stream=stream)

    use()
    use(7)
    assert set(tree.mask.streams) <= {7} and set(tree.depth.streams) <= {7}
    use(9)
    current[0] = 11
    use()
    current[0] = 0
    use()
    for t in (tree.mask, tree.depth):
        assert set(t.streams) - {7} == {9, 11, 0}


def test_sink_is_a_whole_number(cache):
    """Checked as the windows are, before the tensors."""
    x = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    for bad in (3.9, "4", True, None, [4], np.float32(4), np.bool_(True)):
        with pytest.raises(TypeError, match="sink"):
            cache.attend_window(x, x, [1, 2], 4, sink=bad)
    for bad in (1 << 31, 1 << 63, -(1 << 31) - 1, np.int64(1 << 40)):
        with pytest.raises(ValueError, match="sink"):
            cache.attend_window(x, x, [1, 2], 4, sink=bad)
    for good in (0, 4, np.int32(4), np.uint8(4), 0x7FFFFFFF, torch.tensor(4)):   # (as far as the host tensors)
        with pytest.raises(TypeError, match="CUDA"):
            cache.attend_window(x, x, [1, 2], 4, sink=good)
