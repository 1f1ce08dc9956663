"""GPU tests of the window, tree and copy entry points where a caller's
buffers, streams or heads differ from the plain case.  Results against 64 bits
with the tolerances of tests/test_gpu_sequences.py."""
import ctypes

import numpy as np
import pytest
import torch

from tests.test_gpu_packed import DEV, DT, gen_of, hk, make, rnd, slots, tables  # noqa: F401
from tests.test_gpu_sequences import (bits_of, check, fill, paths_of, queries, random_tree, tree_sees,
                                      window_sees)

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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("held", [0, 130, 9000])
def test_logits_of_minus_infinity_are_seen(hk, dtype, held):
    """A row all of whose seen logits overflow to -inf has no softmax (0 / 0), in a
    tree as in the other calls; one that sees nothing is zero; the others are
    what they are without it."""
    n, g = 70, gen_of(65)
    cache = make(hk, 1, 8, 1, 64, dtype, held + n)
    low = torch.full((max(held, n), 1, 64), -3e38, device=DEV, dtype=DT[dtype])
    v = rnd(g, held + n, 1, 64, dtype=dtype)
    if held:
        cache.append_packed(low[:held], v[:held], [held])
    cache.append_packed(low[:n], v[held:], [n])
    q = torch.zeros(n, 8, 64, device=DEV, dtype=DT[dtype])
    q[7], q[33:36], q[69] = 3e38, 3e38, 3e38
    m = torch.eye(n, dtype=torch.bool)
    m[34] = False          # sees nothing but what is in front
    m[40] = False
    tree = hk.Tree([n], bits_of(m, 3).to(DEV))
    out = torch.full_like(q, 7.0)
    before = cache.kernel_launches()
    cache.attend_tree(q, out, tree)
    assert held < 9000 or cache.kernel_launches() - before == 2
    causal, window = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
    cache.attend_packed(q, causal, [n])
    cache.attend_window(q, window, [n], 1)
    lost = torch.zeros(n, dtype=torch.bool, device=DEV)
    lost[[7, 33, 34, 35, 69]] = True
    for x in (causal, window):
        assert bool(torch.isnan(x[lost]).all()) and bool(torch.isfinite(x[~lost]).all())
    if held == 0:
        assert bool((out[[34, 40]] == 0).all())
        lost[34] = False
    assert bool(torch.isnan(out[lost]).all()) and bool(torch.isfinite(out[~lost]).all())
    # equal logits: the mean of what is seen
    k = torch.cat([torch.ones(n, held, dtype=torch.bool), m], 1).double().to(DEV)
    mean = (k @ v[:, 0].double()) / k.sum(1, keepdim=True).clamp_min(1)
    size = (k @ v[:, 0].double().abs()) / k.sum(1, keepdim=True).clamp_min(1)
    h = torch.finfo(DT[dtype]).eps / 2
    tol = (2 * (held + n) * 2.0 ** -24 + 8 * 2.0 ** -24 + (h if dtype == "bf16" else 0)) * size + h * mean.abs()
    err = (out.double() - mean[:, None]).abs()
    assert bool((err <= tol[:, None])[~lost].all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_split_rows_that_see_nothing(hk, dtype):
    """Nothing in front of a long tree whose keys are split over work items."""
    n, gen, cpu = 1900, gen_of(66), torch.Generator().manual_seed(66)
    cache = make(hk, 1, 2, 1, 64, dtype, n)
    fill(cache, gen, [[n]])
    m = torch.rand(n, n, generator=cpu) < 0.01
    m[:, 300:600] = False
    m[[0, 5, 127, 128, 1000, n - 1]] = False
    m[77], m[78] = False, False
    m[77, n - 1] = m[78, 0] = True      # one key each, in the last and the first part
    tree = hk.Tree([n], bits_of(m, 60).to(DEV))
    q, out = queries(cache, gen, n)
    before = cache.kernel_launches()
    cache.attend_tree(q, out, tree)
    assert cache.kernel_launches() - before == 2
    check(cache, q, out, [n], tree_sees([m], [0]))
    blind = ~m.any(1).to(DEV)
    assert int(blind.sum()) >= 6 and bool((out[blind] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_minus_infinity_in_front_of_larger_logits(hk, dtype):
    """Rows whose only logit is -inf, in the first tile of keys, between rows
    whose maximum moves in every later one."""
    n, g = 400, gen_of(67)
    cache = make(hk, 1, 2, 1, 64, dtype, n)
    k = torch.zeros(n, 1, 64, device=DEV, dtype=DT[dtype])
    k[:128] = -3e38
    k[128:, 0, 0] = 10.0 * torch.arange(n - 128, device=DEV)
    v = rnd(g, n, 1, 64, dtype=dtype)
    cache.append_packed(k, v, [n])
    m = torch.zeros(n, n, dtype=torch.bool)
    m[:, 128:] = True
    odd = torch.arange(1, n, 2)
    m[odd] = False
    m[odd, odd % 128] = True
    m[7] = False
    tree = hk.Tree([n], bits_of(m, 13).to(DEV))
    q = torch.zeros(n, 2, 64, device=DEV, dtype=DT[dtype])
    q[:, :, 0] = 1.0
    plain, out = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
    tame = q.clone()
    tame[odd] = 0.0
    cache.attend_tree(tame, plain, tree)
    check(cache, tame, plain, [n], tree_sees([m], [0]))
    q[odd] = 3e38
    cache.attend_tree(q, out, tree)
    assert torch.equal(out[::2], plain[::2]) and bool((out[7] == 0).all())
    lost = odd[odd != 7].to(DEV)
    assert bool(torch.isnan(out[lost]).all())


class Refused:
    """While this lasts nothing can be launched on the default stream: a stream
    that it waits for is being captured.  A host error, no work on the device."""

    def __enter__(self):
        self.cu, self.s = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p()
        assert self.cu.cuStreamCreate(ctypes.byref(self.s), 0) == 0
        assert self.cu.cuStreamBeginCapture_v2(self.s, 2) == 0

    def __exit__(self, *a):
        graph = ctypes.c_void_p()
        self.cu.cuStreamEndCapture(self.s, ctypes.byref(graph))   # (an error: the capture is lost)
        if graph.value:
            self.cu.cuGraphDestroy(graph)
        assert self.cu.cuStreamDestroy_v2(self.s) == 0


def test_a_failed_launch_is_not_the_next_calls_error(hk):
    """The next call, of another kind, is carried out and says so."""
    cfg = dict(budgets=[24, 30], num_sink=2, recent_window=8)
    cache, other = (make(hk, 2, 4, 2, 64, "bf16", 128, **cfg) for _ in range(2))
    new = [40, 33]
    for c in (cache, other):
        fill(c, gen_of(69), [new])
    q, out = queries(cache, gen_of(69), sum(new))
    torch.cuda.synchronize()
    for call in (lambda c: c.evict(), lambda c: c.append(*(torch.ones(1, 2, 2, 3, 64, device=DEV, dtype=torch.bfloat16),) * 2),
                 lambda c: c.decode_step(q[None, :2].contiguous(), out[None, :2].contiguous()), lambda c: c.evict(),
                 lambda c: c.drop()):
        with Refused(), pytest.raises(hk.HikvError, match="fork: launch") as e:
            cache.fork([0, 0])
        assert e.value.status == hk.HIKV_ERR_CUDA
        call(cache)
        call(other)
        assert cache.lengths().tolist() == other.lengths().tolist()
        for u in range(4):
            assert all(torch.equal(x, y) for x, y in zip(slots(cache, u), slots(other, u)))
    cache.device_status()


def test_a_failed_launch_says_which_call_and_that_it_was_the_launch(hk):
    """And leaves the cache as it was."""
    cache = make(hk, 2, 4, 2, 64, "bf16", 128)
    gen, new = gen_of(68), [5, 3]
    fill(cache, gen, [[20, 9], new])
    parent = torch.tensor([-1, 0, 0, 1, 1, -1, 0, 0], dtype=torch.int32, device=DEV)
    tree, rope = cache.tree(parent, new), hk.Rope(*tables(128, 64))
    k, v = (rnd(gen, 8, 2, 64, dtype="bf16") for _ in range(2))
    q, out = queries(cache, gen, 8)
    torch.cuda.synchronize()
    want = cache.lengths().tolist()
    assert torch.cuda.current_stream().cuda_stream == 0
    for name, call in (("append_packed", lambda: cache.append_packed(k, v, new)),
                       ("attend_packed", lambda: cache.attend_packed(q, out, new)),
                       ("attend_window", lambda: cache.attend_window(q, out, new, 4)),
                       ("tree_masks", lambda: cache.tree(parent, new)),
                       ("append_tree", lambda: cache.append_tree(k, v, tree, rope)),
                       ("attend_tree", lambda: cache.attend_tree(q, out, tree)),
                       ("accept", lambda: cache.accept(tree, [[0, 1], [0]])),
                       ("fork", lambda: cache.fork([0, 0])),
                       ("drop", lambda: cache.drop([1, 1]))):
        with Refused(), pytest.raises(hk.HikvError, match=name + ": launch") as e:
            call()
        assert e.value.status == hk.HIKV_ERR_CUDA
        assert cache.lengths().tolist() == want
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())
    cache.attend_tree(q, out, tree)
    check(cache, q, out, new, tree_sees([paths_of([-1, 0, 0, 1, 1]), paths_of([-1, 0, 0])], [20, 9]))
    cache.device_status()


# Cut caches: budgets per head, tokens appended since; few queries, so that the
# keys are split over work items
UNEVEN = [("bf16", 128, 8, [6000, 700]), ("bf16", 64, 2, [3100, 40, 5000]), ("f32", 64, 4, [6000, 700]),
          ("f32", 128, 8, [129, 4000])]


def uneven(hk, dtype, d, group, budgets, held, since, new, gen):
    cache = make(hk, len(held), group * len(budgets), len(budgets), d, dtype, max(map(sum, zip(held, since, new))),
                 budgets=budgets, num_sink=4, recent_window=16)
    fill(cache, gen, [held])
    cache.evict()
    fill(cache, gen, [since, new])
    n = cache.lengths().reshape(len(held), -1)
    assert any(len(set(row)) > 1 for row in n.tolist())
    return cache


@pytest.mark.parametrize("dtype,d,group,budgets", UNEVEN)
@pytest.mark.parametrize("new", [[1], [5, 3], [37, 0, 1]])
def test_tree_split_over_heads_of_unequal_length(hk, dtype, d, group, budgets, new):
    gen, cpu = gen_of(62 + sum(new)), torch.Generator().manual_seed(62)
    held, since = [7000, 900, 6500][:len(new)], [0, 77, 300][:len(new)]
    cache = uneven(hk, dtype, d, group, budgets, held, since, new, gen)
    masks = [torch.rand(n, n, generator=cpu) < 0.5 for n in new]
    tree = hk.Tree(new, torch.cat([bits_of(m, 2) for m in masks]).to(DEV))
    q, out = queries(cache, gen, sum(new))
    before = cache.kernel_launches()
    cache.attend_tree(q, out, tree)
    assert cache.kernel_launches() - before == 2
    check(cache, q, out, new, tree_sees(masks, held))
    before = cache.kernel_launches()
    cache.attend_packed(q, out, new)
    assert cache.kernel_launches() - before == 2
    check(cache, q, out, new, lambda b, g, n, pos: pos[None] <= int(pos.max()) - new[b] + 1
          + torch.arange(new[b], device=DEV)[:, None])
    cache.device_status()


@pytest.mark.parametrize("dtype,d,group,budgets", UNEVEN)
@pytest.mark.parametrize("new", [[1], [5, 3], [37, 0, 1]])
def test_window_split_over_heads_of_unequal_length(hk, dtype, d, group, budgets, new):
    """A window for every head inside what was appended since the cut; head 0
    sees all that it holds."""
    gen = gen_of(63 + sum(new))
    held, since = [7000, 900, 6500][:len(new)], [2600, 2500, 2700][:len(new)]
    cache = uneven(hk, dtype, d, group, budgets, held, since, new, gen)
    for windows, sink in (([0, 2400, 1100], 4), ([2400, 2400, 2400], 0), ([1500, 0, 7], 3)):
        windows = windows[:len(budgets)]
        q, out = queries(cache, gen, sum(new))
        before = cache.kernel_launches()
        cache.attend_window(q, out, new, windows, sink)
        assert cache.kernel_launches() - before == 2
        check(cache, q, out, new, window_sees(new, windows, sink))
    cache.device_status()


@pytest.mark.parametrize("layer0,nlayers", [(1, 0x7FFFFFFF), (0x7FFFFFFF, 1), (2, 1), (0, 3), (-1, 1), (1, 0), (1, -1)])
def test_layers_out_of_range_are_refused(hk, layer0, nlayers):
    """Their sum past 32 bits among them."""
    cache = make(hk, 2, 4, 2, 64, "bf16", 64, layers=2)
    fill(cache, gen_of(70), [[9, 5]])
    at = dict(layer0=layer0, nlayers=nlayers)
    for call in (lambda: cache.drop([1, 1], **at), lambda: cache.accept([2, 1], [[0], [0]], **at),
                 lambda: cache.fork([0, 0], **at), lambda: cache.evict(**at)):
        with pytest.raises(hk.HikvError) as e:
            call()
        assert e.value.status == hk.HIKV_ERR_INVALID_ARG
    assert cache.lengths().tolist() == [9, 9, 5, 5, 0, 0, 0, 0]
