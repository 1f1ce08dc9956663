"""GPU tests of the window, tree and copy entry points where a caller's
buffers, streams or heads differ from the plain case.  Results against 64 bits
with the tolerances of tests/test_gpu_sequences.py."""
import numpy as np
import pytest
import torch

from tests.test_gpu_packed import DEV, gen_of, hk, make, rnd, tables  # noqa: F401
from tests.test_gpu_sequences import check, fill, paths_of, queries, random_tree, tree_sees

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["array", "tensor"])
def test_counts_that_are_filled_again(hk, kind):
    """The counts a tree was made from serve the next step while the tree lives."""
    new, held = [9, 0, 40], [70, 3, 200]
    gen, cpu = gen_of(60), torch.Generator().manual_seed(60)
    cache = make(hk, 3, 8, 2, 64, "bf16", 512)
    fill(cache, gen, [held])
    parents = [random_tree(cpu, n) for n in new]
    counts = np.array(new, dtype=np.int32) if kind == "array" else torch.tensor(new, dtype=torch.int32)
    tree = cache.tree(torch.tensor(sum(parents, []), dtype=torch.int32, device=DEV), counts)
    counts[:] = 1
    cos, sin = tables(512, 64)
    k, v = (rnd(gen, sum(new), 2, 64, dtype="bf16") for _ in range(2))
    q, out = queries(cache, gen, sum(new))
    cache.append_tree(k, v, tree, hk.Rope(cos, sin), q=q, q_out=q)
    cache.attend_tree(q, out, tree)
    check(cache, q, out, new, tree_sees([paths_of(p) if p else torch.zeros(0, 0, dtype=torch.bool) for p in parents], held))
    cache.accept(tree, [[0], [], [0, 1]])
    assert cache.lengths().reshape(3, 2).tolist() == [[71] * 2, [3] * 2, [202] * 2]
    cache.device_status()


def stream_of_memory(t):
    """The stream that the allocator's segment of t belongs to."""
    at = t.data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"])


def test_memory_of_a_tree_belongs_to_its_stream(hk):
    """The default stream given by handle while another one is current, and the
    other way round."""
    cache = make(hk, 2, 4, 2, 64, "bf16", 64)
    parent = torch.tensor([-1, 0, 0, -1, 0], dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        by_handle, by_stream = cache.tree(parent, [3, 2], stream=0), cache.tree(parent, [3, 2], stream=torch.cuda.default_stream())
    beside = cache.tree(parent, [3, 2], stream=side)
    torch.cuda.synchronize()
    for tree, stream in ((by_handle, 0), (by_stream, 0), (beside, side.cuda_stream)):
        assert stream_of_memory(tree.mask) == stream and stream_of_memory(tree.depth) == stream
        assert tree.mask.flatten().tolist() == [1, 3, 5, 1, 3] and tree.depth.tolist() == [0, 1, 1, 0, 1]


@pytest.mark.parametrize("given", [False, True])
def test_a_tree_made_on_one_stream_and_used_on_another(hk, given):
    """Its memory is not given out again on the stream it was made on while the
    other one's work on it waits."""
    cache = make(hk, 1, 4, 2, 64, "bf16", 128)
    gen = gen_of(61)
    fill(cache, gen, [[40], [33]])
    parent = torch.tensor(random_tree(torch.Generator().manual_seed(61), 33), dtype=torch.int32, device=DEV)
    q, out = queries(cache, gen, 33)
    made, used = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    tree = cache.tree(parent, [33], stream=made)
    shapes, at = [tree.mask.shape, tree.depth.shape], tree.mask.data_ptr()
    used.wait_stream(made)
    if given:
        with torch.cuda.stream(used):
            torch.cuda._sleep(200_000_000)
        cache.attend_tree(q, out, tree, stream=used)
    else:
        with torch.cuda.stream(used):
            torch.cuda._sleep(200_000_000)
            cache.attend_tree(q, out, tree)
    del tree
    with torch.cuda.stream(made):
        again = [torch.empty(s, dtype=torch.int32, device=DEV).fill_(-1) for s in shapes]
    assert not used.query() and at not in [x.data_ptr() for x in again]
    torch.cuda.synchronize()
    check(cache, q, out, [33], tree_sees([paths_of(parent.tolist())], [40]))


def test_a_tree_made_before_a_capture(hk):
    """On the current stream, used by a captured call on the capture's and by an
    eager one beside it; given up before the eager call's work is done."""
    cache = make(hk, 2, 8, 2, 128, "bf16", 256)
    gen, cpu = gen_of(64), torch.Generator().manual_seed(64)
    new, held = [33, 7], [100, 0]
    fill(cache, gen, [held, new])
    parents = [random_tree(cpu, n) for n in new]
    sees = tree_sees([paths_of(p) for p in parents], held)
    tree = cache.tree(torch.tensor(sum(parents, []), dtype=torch.int32, device=DEV), new)
    q, out = queries(cache, gen, sum(new))
    eager = torch.full_like(q, 7.0)
    cache.attend_tree(q, eager, tree)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attend_tree(q, out, tree)
    graph.replay()
    out2 = out.clone()
    q.copy_(torch.randn(q.shape, generator=gen, device=DEV))
    graph.replay()
    cache.attend_tree(q, eager, tree)
    check(cache, q, out, new, sees)
    assert torch.equal(out, eager) and not torch.equal(out, out2)
    graph.reset()
    del graph, tree
    torch.cuda.synchronize()
    check(cache, q, eager, new, sees)
