"""GPU tests of sliding windows with visible first tokens
(hikv_attend_window), trees of drafted tokens (hikv_tree_masks,
hikv_append_tree, hikv_attend_tree, hikv_accept) and copies of sequences
(hikv_fork), each against a plain computation in 64 bits.

Tolerances are those of the packed calls (h = half a step of the cache dtype,
u = 2^-24): rotation h |y| + 3 u (|a c| + |b s|); attention, with e = 2 d u
scale max over what is seen of sum |q k|,
    (expm1(2 e) + 2 n u + 8 u + h) sum p |v| + h |o|
(h of the probabilities in bf16 only).  What is moved or copied is equal.
"""
import math

import pytest
import torch

from tests.test_gpu_packed import (DEV, DT, HALF, SHAPES, U, close_rot, gen_of, hk, make, rnd, rotated,  # noqa: F401
                                   slots, tables)

pytestmark = pytest.mark.gpu


def check(cache, q, out, nq, sees, layer=0):
    """out against softmax attention in 64 bits; sees(b, g, n, pos): bool
    [nq[b]][n], what each query sees of unit (b, g)'s n slots.  A non-finite V
    element that is seen joins the sum as it is; one that is not has no part."""
    c = cache.cfg
    dtype, d, hkv, G = c.dtype, c.head_dim, c.num_kv_heads, c.num_q_heads // c.num_kv_heads
    scale = c.scale or 1.0 / math.sqrt(d)
    r = 0
    for b, t in enumerate(nq):
        for g in range(hkv if t else 0):
            u = (layer * c.batch + b) * hkv + g
            k, v, pos = slots(cache, u)
            n = k.shape[0]
            seen_all = sees(b, g, n, pos)
            kd = torch.where(torch.isfinite(k), k, 0).double()
            vd = torch.where(torch.isfinite(v), v, 0).double()
            odd = torch.where(torch.isfinite(v), 0, v).double()
            has_odd = bool((odd != 0).any())
            for i0 in range(0, t, 512):
                m = min(512, t - i0)
                seen = seen_all[i0:i0 + m]
                x = q[r + i0:r + i0 + m, g * G:(g + 1) * G].double()
                z = torch.einsum("mgd,nd->mgn", x, kd) * scale
                hide = ~seen[:, None]
                e = 2 * d * U * scale * torch.einsum("mgd,nd->mgn", x.abs(), kd.abs()).masked_fill(hide, 0).amax(-1)
                z = z.masked_fill(hide, -math.inf)
                top = z.amax(-1, keepdim=True)
                p = torch.exp(z - torch.where(top == -math.inf, 0, top))
                p = p / p.sum(-1, keepdim=True).clamp_min(1e-300)
                o, mag = p @ vd, p @ vd.abs()
                f = torch.expm1(2 * e) + 2 * n * U + 8 * U + (HALF[dtype] if dtype == "bf16" else 0.0)
                tol = f[..., None] * mag + HALF[dtype] * o.abs()
                got = out[r + i0:r + i0 + m, g * G:(g + 1) * G].double()
                if has_odd:
                    extra = torch.zeros(m, d, dtype=torch.float64, device=DEV)
                    for s in torch.nonzero((odd != 0).any(-1)).flatten().tolist():
                        extra += torch.where(seen[:, s:s + 1], odd[s], 0)
                    bad = ~torch.isfinite(extra)[:, None].expand_as(got)
                    assert torch.equal(got[bad].nan_to_num(9.0), extra[:, None].expand_as(got)[bad].nan_to_num(9.0))
                    got, o = got.masked_fill(bad, 0), o.masked_fill(bad, 0)
                err = (got - o).abs()
                assert bool((err <= tol).all()), (b, g, i0, float((err - tol).max()), int((~(err <= tol)).sum()))
        r += t


def window_sees(nq, windows, sink):
    def sees(b, g, n, pos):
        w = windows[g]
        mine = int(pos.max()) - nq[b] + 1 + torch.arange(nq[b], device=DEV)[:, None]
        ok = pos[None] <= mine
        return ok & ((pos[None] > mine - w) | (pos[None] < sink)) if w else ok
    return sees


def fill(cache, gen, parts):
    """Random tokens appended part by part."""
    c = cache.cfg
    for n in parts:
        t = sum(n)
        if t:
            cache.append_packed(rnd(gen, t, c.num_kv_heads, c.head_dim, dtype=c.dtype),
                                rnd(gen, t, c.num_kv_heads, c.head_dim, dtype=c.dtype), n)


def queries(cache, gen, total):
    c = cache.cfg
    q = rnd(gen, total, c.num_q_heads, c.head_dim, dtype=c.dtype)
    return q, torch.full_like(q, 7.0)


# ---------------------------------------------------------------------------
# windows
# ---------------------------------------------------------------------------
WINDOWS = [([1], [0], 1, 0), ([5], [0], 1, 1), ([1], [700], 300, 4), ([130, 0, 1, 257], [0, 9, 1300, 64], 64, 4),
           ([700], [0], 100, 0), ([300, 33], [500, 1000], 129, 70), ([64], [3000], 1000, 4), ([1, 2], [4096, 63], 63, 1),
           ([200], [100], 5000, 3), ([257], [0], 1, 200), ([40], [90], 2, 128)]


@pytest.mark.parametrize("dtype,d,hq,hkv", SHAPES)
@pytest.mark.parametrize("new,held,window,sink", WINDOWS)
def test_window(hk, dtype, d, hq, hkv, new, held, window, sink):
    gen = gen_of(sum(new) + 13 * hq + d + window)
    cache = make(hk, len(new), hq, hkv, d, dtype, max(a + b for a, b in zip(new, held)))
    fill(cache, gen, (held, new))
    q, out = queries(cache, gen, sum(new))
    cache.attend_window(q, out, new, window, sink)
    cache.device_status()
    check(cache, q, out, new, window_sees(new, [window] * hkv, sink))


@pytest.mark.parametrize("dtype,page,shared", [("bf16", 16, True), ("bf16", 32, False), ("bf16", 128, True),
                                               ("bf16", 256, False), ("f32", 16, True)])
def test_window_over_pages_of_any_size(hk, dtype, page, shared):
    new, held = [70, 1, 300], [333, 800, 5]
    cap = 832
    per = -(-cap // page)
    kw = dict(pool_pages=3 * 2 * per - 1) if shared else {}
    cache = make(hk, 3, 8, 2, 128, dtype, cap, page_tokens=page, **kw)
    gen = gen_of(page)
    for n in ([100, 7, 0], [233, 793, 5], new):   # shared: the rows' pages interleave
        fill(cache, gen, [n])
    for window, sink in ((50, 5), (17, 0), (256, 129)):
        q, out = queries(cache, gen, sum(new))
        cache.attend_window(q, out, new, window, sink)
        check(cache, q, out, new, window_sees(new, [window] * 2, sink))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_window_of_its_own_for_every_head(hk, dtype):
    new, held = [150, 1, 40], [0, 900, 300]
    windows = [0, 1, 33, 200, 128, 1000, 7]
    cache = make(hk, 3, 14, 7, 64, dtype, 1024)
    gen = gen_of(21)
    fill(cache, gen, (held, new))
    for sink in (0, 4):
        q, out = queries(cache, gen, sum(new))
        cache.attend_window(q, out, new, windows, sink)
        check(cache, q, out, new, window_sees(new, windows, sink))


def test_window_that_hides_nothing_is_causal_attention(hk):
    new, held = [65, 3], [700, 20]
    cache = make(hk, 2, 8, 2, 128, "bf16", 1024)
    gen = gen_of(22)
    fill(cache, gen, (held, new))
    q, out = queries(cache, gen, sum(new))
    cache.attend_packed(q, out, new)
    for window, sink in ((0, 0), (765, 0), (700, 65), (2 ** 31 - 1, 2 ** 31 - 1)):
        got = torch.full_like(q, 7.0)
        cache.attend_window(q, got, new, window, sink)
        assert torch.equal(got, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_window_hides_what_is_not_finite(hk, dtype):
    """NaN keys and infinite values outside a window touch nothing, inside it
    the rows that see them."""
    new, held = [200, 1], [333, 600]
    cache = make(hk, 2, 8, 2, 64, dtype, 640)
    gen = gen_of(23)
    fill(cache, gen, (held, new))
    w = cache.device_view()
    pt = w["pages"].shape[2]

    def put(u, s, kind, col, x):
        w["pages"][int(w["page_table"][u, s // pt]), kind, s % pt, col] = x

    window, sink = 40, 3
    for s in (3, 100, 292):          # keys that no query sees (the first query's window starts at slot 294)
        put(0, s, 0, 5, math.nan)
    for s in (4, 50, 200, 293):
        put(0, s, 1, 9, math.inf)
        put(1, s, 1, 10, math.nan)
    put(0, 300, 1, 11, math.inf)     # seen by the first queries, not by the last
    put(0, 420, 1, 12, -math.inf)    # by some in the middle
    put(0, 425, 1, 12, math.inf)
    put(0, 430, 1, 13, math.nan)
    put(0, 1, 1, 14, math.inf)       # a first token: by all
    put(1, 532, 1, 15, math.inf)     # the newest token: by the last query
    put(2, 560, 1, 3, math.inf)      # hidden from the single query, seen by it
    put(2, 561, 1, 4, math.inf)
    q, out = queries(cache, gen, sum(new))
    cache.attend_window(q, out, new, window, sink)
    check(cache, q, out, new, window_sees(new, [window] * 2, sink))


def test_window_over_a_cut_unit(hk):
    gen = gen_of(24)
    cache = make(hk, 1, 4, 2, 64, "bf16", 512, budgets=[100, 60], num_sink=4, recent_window=16)
    fill(cache, gen, [[300]])
    cache.evict()
    fill(cache, gen, [[90], [30]])
    q, out = queries(cache, gen, 30)
    cache.attend_window(q, out, [30], [91, 40], 4)   # 30 + 91 - 1 newest tokens are in order
    check(cache, q, out, [30], window_sees([30], [91, 40], 4))
    cache.attend_window(q, out, [30], [0, 1], 2)
    check(cache, q, out, [30], window_sees([30], [0, 1], 2))
    for windows, sink in (([92, 40], 4), ([91, 40], 5), ([0, 2 ** 31 - 1], 0)):
        with pytest.raises(hk.HikvError) as e:
            cache.attend_window(q, out, [30], windows, sink)
        assert e.value.status == hk.HIKV_ERR_STATE


@pytest.mark.parametrize("dtype,hq,hkv", [("bf16", 8, 1), ("bf16", 4, 4), ("f32", 8, 1)])
def test_window_split_over_work_items(hk, dtype, hq, hkv):
    """Few rows over a long window: the keys are split and joined."""
    gen = gen_of(25)
    for new, held, window, sink in (([1], [9000], 6000, 4), ([3], [9000], 8000, 300), ([50], [5000], 4000, 0)):
        cache = make(hk, 1, hq, hkv, 128, dtype, 9088)
        fill(cache, gen, (held, new))
        q, out = queries(cache, gen, sum(new))
        before = cache.kernel_launches()
        cache.attend_window(q, out, new, window, sink)
        assert cache.kernel_launches() - before == 2   # split, and the join
        check(cache, q, out, new, window_sees(new, [window] * hkv, sink))


# ---------------------------------------------------------------------------
# trees
# ---------------------------------------------------------------------------
def random_tree(g, n):
    """Parents of n nodes, several roots among them."""
    u = torch.rand(n, generator=g).tolist()
    return [min(i - 1, int(x * (i + 1)) - 1) for i, x in enumerate(u)]


def paths_of(parent):
    m = torch.zeros(len(parent), len(parent), dtype=torch.bool)
    for i, p in enumerate(parent):
        if p >= 0:
            m[i] = m[p]
        m[i, i] = True
    return m


def bits_of(m, words):
    """bool [rows][cols] as int32 words."""
    x = torch.zeros(m.shape[0], 32 * words, dtype=torch.int64)
    x[:, :m.shape[1]] = m
    x = (x.view(-1, words, 32) << torch.arange(32)).sum(-1)
    return torch.where(x >= 1 << 31, x - (1 << 32), x).to(torch.int32)


def tree_sees(masks, held):
    def sees(b, g, n, pos):
        t = masks[b].shape[0]   # (whatever the unit holds in front of them)
        return torch.cat([torch.ones(t, n - t, dtype=torch.bool, device=DEV), masks[b].to(DEV)], 1)
    return sees


TREES = [([1], [0]), ([1, 0, 5], [0, 9, 0]), ([26, 32, 33, 64], [97, 0, 128, 700]), ([65, 7], [0, 2000]), ([63], [3001]),
         ([127, 128, 129], [1, 127, 255]), ([300], [40])]


@pytest.mark.parametrize("dtype,d,hq,hkv", SHAPES)
@pytest.mark.parametrize("new,held", TREES)
def test_tree(hk, dtype, d, hq, hkv, new, held):
    gen, cpu = gen_of(sum(new) + 17 * hq + d), torch.Generator().manual_seed(sum(new))
    cache = make(hk, len(new), hq, hkv, d, dtype, max(a + b for a, b in zip(new, held)))
    fill(cache, gen, (held, new))
    parents = [random_tree(cpu, n) for n in new]
    flat = torch.tensor([p for t in parents for p in t], dtype=torch.int32, device=DEV)
    tree = cache.tree(flat, new)
    masks = [paths_of(p) for p in parents]
    words = -(-max(new) // 32)
    assert torch.equal(tree.mask.cpu(), torch.cat([bits_of(m, words) for m in masks]))
    assert torch.equal(tree.depth.cpu(), torch.cat([m.sum(1) - 1 for m in masks]).int())
    q, out = queries(cache, gen, sum(new))
    cache.attend_tree(q, out, tree)
    cache.device_status()
    check(cache, q, out, new, tree_sees(masks, held))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("held", [[0, 70, 0], [300, 0, 129]])
def test_masks_of_any_shape(hk, dtype, held):
    """Rows that see later nodes or nothing at all; spare words and bits past
    the nodes are ignored."""
    new = [40, 77, 3]
    gen, cpu = gen_of(31), torch.Generator().manual_seed(5)
    cache = make(hk, 3, 8, 2, 64, dtype, 512)
    fill(cache, gen, (held, new))
    masks = [torch.rand(n, n, generator=cpu) < 0.3 for n in new]
    masks[0][7] = False
    masks[1][0] = False
    masks[2][:] = False
    words = torch.randint(-2 ** 31, 2 ** 31, (sum(new), 5), generator=cpu, dtype=torch.int64)
    r = 0
    for m in masks:
        n = m.shape[0]
        full = torch.ones(n, 160, dtype=torch.int64) * ((words[r:r + n, :, None] >> torch.arange(32)) & 1).view(n, 160)
        full[:, :n] = m
        words[r:r + n] = bits_of(full.bool(), 5).long()
        r += n
    tree = hk.Tree(new, words.to(torch.int32).to(DEV))
    q, out = queries(cache, gen, sum(new))
    cache.attend_tree(q, out, tree)
    check(cache, q, out, new, tree_sees(masks, held))
    for b, (m, h) in enumerate(zip(masks, held)):
        rows = out[sum(new[:b]):sum(new[:b + 1])]
        if h == 0:
            assert bool((rows[~m.any(1).to(DEV)] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_split_over_work_items(hk, dtype):
    gen, cpu = gen_of(32), torch.Generator().manual_seed(6)
    for new, held in (([20], [9000]), ([5, 64], [6000, 7001])):
        cache = make(hk, len(new), 8, 1, 128, dtype, 9088)
        fill(cache, gen, (held, new))
        masks = [torch.rand(n, n, generator=cpu) < 0.5 for n in new]
        words = -(-max(new) // 32)
        tree = hk.Tree(new, torch.cat([bits_of(m, words) for m in masks]).to(DEV))
        q, out = queries(cache, gen, sum(new))
        before = cache.kernel_launches()
        cache.attend_tree(q, out, tree)
        assert cache.kernel_launches() - before == 2
        check(cache, q, out, new, tree_sees(masks, held))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_hides_what_is_not_finite(hk, dtype):
    new, held = [70], [100]
    gen, cpu = gen_of(33), torch.Generator().manual_seed(7)
    cache = make(hk, 1, 8, 2, 64, dtype, 256)
    fill(cache, gen, (held, new))
    m = torch.rand(70, 70, generator=cpu) < 0.5
    m[:, 13] = m[:, 60] = False                # nobody sees these
    w = cache.device_view()
    pt = w["pages"].shape[2]

    def put(u, s, kind, col, x):
        w["pages"][int(w["page_table"][u, s // pt]), kind, s % pt, col] = x

    put(0, 113, 0, 1, math.nan)
    put(0, 160, 1, 2, math.nan)
    put(0, 120, 1, 3, math.inf)
    put(0, 121, 1, 3, -math.inf)
    put(0, 169, 1, 4, math.nan)
    put(1, 5, 1, 5, math.inf)                  # in front of the tree: seen by all
    put(1, 100, 1, 6, -math.inf)
    tree = hk.Tree(new, bits_of(m, 3).to(DEV))
    q, out = queries(cache, gen, 70)
    cache.attend_tree(q, out, tree)
    check(cache, q, out, new, tree_sees([m], held))


@pytest.mark.parametrize("dtype,d,hq,hkv", [("bf16", 128, 8, 2), ("f32", 64, 4, 2)])
def test_long_masks(hk, dtype, d, hq, hkv):
    """Masks of many words a row: most key tiles are the tree's own."""
    new, held = [1500, 0, 333], [100, 7, 2000]
    gen, cpu = gen_of(39), torch.Generator().manual_seed(19)
    cache = make(hk, 3, hq, hkv, d, dtype, 2368)
    fill(cache, gen, (held, new))
    masks = [torch.rand(n, n, generator=cpu) < 0.2 for n in new]
    tree = hk.Tree(new, torch.cat([bits_of(m, 48) for m in masks]).to(DEV))
    q, out = queries(cache, gen, sum(new))
    cache.attend_tree(q, out, tree)
    check(cache, q, out, new, tree_sees(masks, held))


def test_bad_parents_are_reported(hk):
    cache = make(hk, 2, 4, 2, 64, "bf16", 64)
    parent = torch.tensor([-1, 0, 2, 9, -2, 0, 0], dtype=torch.int32, device=DEV)   # nodes 2, 3 and 4 of the first
    tree = cache.tree(parent, [5, 2])
    with pytest.raises(hk.HikvError) as e:
        cache.device_status()
    assert e.value.status == hk.HIKV_ERR_STATE
    assert tree.mask.flatten().tolist() == [1, 3, 4, 8, 16, 1, 3]
    assert tree.depth.tolist() == [0, 1, 0, 0, 0, 0, 1]   # (the second sequence's first node names itself)


def test_trees_of_more_sequences_than_a_launch_takes(hk):
    B, cpu = 600, torch.Generator().manual_seed(8)
    cache = make(hk, B, 2, 1, 64, "bf16", 64, page_tokens=16)
    new = [(5 * b) % 40 for b in range(B)]
    parents = [random_tree(cpu, n) for n in new]
    tree = cache.tree(torch.tensor([p for t in parents for p in t], dtype=torch.int32, device=DEV), new)
    masks = [paths_of(p) for p in parents]
    assert torch.equal(tree.mask.cpu(), torch.cat([bits_of(m, 2) for m in masks]))
    gen = gen_of(34)
    fill(cache, gen, [new])
    q, out = queries(cache, gen, sum(new))
    cache.attend_tree(q, out, tree)
    check(cache, q, out, new, tree_sees(masks, [0] * B))
    keep = [list(range(0, n, 3)) for n in new]
    before = [slots(cache, u) for u in range(0, B, 37)]
    cache.accept(tree, keep)
    for u, (k, v, _) in zip(range(0, B, 37), before):
        k1, v1, p1 = slots(cache, u)
        assert torch.equal(k1, k[keep[u]]) and torch.equal(v1, v[keep[u]]) and p1.tolist() == list(range(len(keep[u])))


@pytest.mark.parametrize("dtype,d,hq,hkv,rot,interleaved,shared", [
    ("bf16", 128, 8, 2, 128, False, False), ("bf16", 64, 16, 2, 64, True, True), ("f32", 64, 4, 2, 32, True, False),
    ("f32", 128, 8, 1, 128, False, True)])
def test_a_verified_step_leaves_what_its_accepted_tokens_would(hk, dtype, d, hq, hkv, rot, interleaved, shared):
    """Two layers: trees appended (rotated by depth), attended, their paths
    accepted: as if the path's tokens alone had been appended."""
    held, new = [60, 0, 131, 7, 9], [33, 5, 64, 0, 1]
    cap = 256
    kw = dict(page_tokens=16, pool_pages=2 * 5 * hkv * 16 - 1) if shared else {}
    a, b = (make(hk, 5, hq, hkv, d, dtype, cap, layers=2, **kw) for _ in range(2))
    cos, sin = tables(cap, rot)
    rope = hk.Rope(cos, sin, interleaved)
    gen, cpu = gen_of(35), torch.Generator().manual_seed(9)
    parents = [random_tree(cpu, n) for n in new]
    paths = []
    for p in parents:   # the path to the last node, but for one sequence that accepts nothing
        at, path = len(p) - 1, []
        while at >= 0:
            path.insert(0, at)
            at = p[at]
        paths.append(path)
    paths[1] = []
    flat = torch.tensor([p for t in parents for p in t], dtype=torch.int32, device=DEV)
    tree = a.tree(flat, new)
    rows = [sum(new[:i]) + x for i, path in enumerate(paths) for x in path]
    for layer in (0, 1):
        x = rnd(gen, sum(held), hkv, d, dtype=dtype)
        for c in (a, b):
            c.append_packed(x, x, held, layer=layer, rope=rope)
        qkv = rnd(gen, sum(new), hq + 2 * hkv, d, dtype=dtype)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        qo, out = torch.empty(sum(new), hq, d, device=DEV, dtype=DT[dtype]), torch.empty(sum(new), hq, d, device=DEV, dtype=DT[dtype])
        a.append_tree(k, v, tree, rope, layer=layer, q=q, q_out=qo)
        pos = torch.cat([h + paths_of(p).sum(1) - 1 for h, p in zip(held, parents) if p]).to(DEV)
        close_rot(qo, *rotated(q, pos, cos, sin, interleaved), dtype)
        a.attend_tree(qo, out, tree, layer=layer)
        check(a, qo, out, new, tree_sees([paths_of(p) for p in parents], held), layer)
        b.append_packed(k[rows], v[rows], [len(p) for p in paths], layer=layer, rope=rope)
    a.accept(tree, paths)
    a.device_status()
    assert a.lengths().tolist() == b.lengths().tolist()
    for x, y in zip(a.gather(with_kv=True), b.gather(with_kv=True)):
        assert torch.equal(x, y)
    # and the next step goes on from there
    t = rnd(gen, 5, hkv, d, dtype=dtype)
    for c in (a, b):
        c.append_packed(t, t, [1] * 5, layer=1, rope=rope)
    q1, o1 = queries(a, gen, 5)
    o2 = torch.empty_like(o1)
    a.attend_packed(q1, o1, [1] * 5, layer=1)
    b.attend_packed(q1, o2, [1] * 5, layer=1)
    assert torch.equal(o1, o2)


def test_accept_of_long_lists_keeps_scores_and_neighbours(hk):
    """Lists longer than one launch takes, importance moved with its tokens,
    other rows and layers left alone."""
    B, n = 3, 5000
    cache = make(hk, B, 2, 2, 64, "bf16", 5056, layers=2)
    gen = gen_of(36)
    for layer in (0, 1):
        x = rnd(gen, 3 * n, 2, 64)
        cache.append_packed(x, x, [n] * B, layer=layer)
    w = cache.device_view()
    w["importance"].copy_(torch.rand(w["importance"].shape, generator=gen, device=DEV))
    old = [(*slots(cache, u), w["importance"][u].clone()) for u in range(12)]
    keep = [[i for i in range(4900) if i % 3], [], list(range(2000, 4800))]
    cache.accept([4900, 0, 4800], keep, layer0=1, nlayers=1)
    for u, (k, v, p, imp) in enumerate(old):
        layer, b = u // 6, u // 2 % 3
        idx = list(range(n)) if layer == 0 or b == 1 else \
            list(range(n - (4900, 0, 4800)[b])) + [n - (4900, 0, 4800)[b] + i for i in keep[b]]
        k1, v1, p1 = slots(cache, u)
        assert torch.equal(k1, k[idx]) and torch.equal(v1, v[idx])
        assert p1.tolist() == list(range(len(idx)))
        assert torch.equal(w["importance"][u, :len(idx)], imp[idx])


def test_step_in_a_graph(hk):
    """Tree masks, append, attention and acceptance captured once, replayed
    over other trees."""
    new, held, cap = [20, 33], [50, 4], 128
    cache = make(hk, 2, 8, 2, 64, "bf16", cap)
    cos, sin = tables(cap, 64)
    rope = hk.Rope(cos, sin)
    gen, cpu = gen_of(37), torch.Generator().manual_seed(10)
    fill(cache, gen, [held])
    fill(cache, gen, [[2, 3]])
    parent = torch.zeros(53, dtype=torch.int32, device=DEV)
    qkv = torch.zeros(53, 12, 64, device=DEV, dtype=torch.bfloat16)
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    qo, out = torch.empty(53, 8, 64, device=DEV, dtype=torch.bfloat16), torch.empty(53, 8, 64, device=DEV, dtype=torch.bfloat16)
    parents = [random_tree(cpu, n) for n in new]
    parent.copy_(torch.tensor(sum(parents, []), dtype=torch.int32))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            cache.drop([2, 3])
            tree = cache.tree(parent, new)
            cache.append_tree(k, v, tree, rope, q=q, q_out=qo)
            cache.attend_tree(qo, out, tree)
            cache.accept(tree, [[0, 5], [1, 2, 32]])
    torch.cuda.current_stream().wait_stream(s)
    other = make(hk, 2, 8, 2, 64, "bf16", cap)
    for seed in (1, 2):
        cpu.manual_seed(seed)
        parents = [random_tree(cpu, n) for n in new]
        parent.copy_(torch.tensor(sum(parents, []), dtype=torch.int32))
        qkv.copy_(rnd(gen, 53, 12, 64))
        graph.replay()
        torch.cuda.synchronize()
        other.drop()
        other.device_view()["pages"].copy_(cache.device_view()["pages"])
        z = torch.zeros(sum(held), 2, 64, device=DEV, dtype=torch.bfloat16)
        # the same step eagerly over the same held tokens
        keep = cache.device_view()["pages"].clone()
        other.append_packed(z, z, held)
        other.device_view()["pages"].copy_(keep)
        t2 = other.tree(parent, new)
        qo2, out2 = torch.empty_like(qo), torch.empty_like(out)
        other.append_tree(k, v, t2, rope, q=q, q_out=qo2)
        other.attend_tree(qo2, out2, t2)
        other.accept(t2, [[0, 5], [1, 2, 32]])
        assert torch.equal(tree.mask, t2.mask) and torch.equal(qo, qo2) and torch.equal(out, out2)
        for u in range(4):
            for x, y in zip(slots(cache, u), slots(other, u)):
                assert torch.equal(x, y)


@pytest.mark.parametrize("kind", ["window", "tree"])
def test_last_sequences_split_when_rounds_do_not_fill(hk, kind):
    """A few more work items than whole rounds of them: the shortest sequences'
    keys are split, the others' not, each into its own rows."""
    B, hq, hkv = 40, 16, 8
    held = [1700 + 11 * ((17 * b) % B) for b in range(B)]
    new = [0 if b == 5 else 1 + b % 2 for b in range(B)]
    cache = make(hk, B, hq, hkv, 64, "bf16", 2176)
    gen, cpu = gen_of(38), torch.Generator().manual_seed(18)
    fill(cache, gen, (held, new))
    q, out = queries(cache, gen, sum(new))
    before = cache.kernel_launches()
    if kind == "window":
        cache.attend_window(q, out, new, 1500, 4)
        sees = window_sees(new, [1500] * hkv, 4)
    else:
        masks = [torch.rand(n, n, generator=cpu) < 0.6 for n in new]
        cache.attend_tree(q, out, hk.Tree(new, torch.cat([bits_of(m, 1) for m in masks]).to(DEV)))
        sees = tree_sees(masks, held)
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        assert cache.kernel_launches() - before == 2   # 312 items on 152 SMs
    check(cache, q, out, new, sees)


@pytest.mark.parametrize("call", ["packed", "window", "tree"])
def test_non_finite_values_of_every_item_arrive(hk, call):
    """More short items of one row tile than SMs, each with a non-finite value
    in its last tile: the rows get their own, whichever items a CTA takes in
    turn."""
    B, hkv, n = 60, 8, 90
    cache = make(hk, B, 16, hkv, 64, "bf16", 128)
    gen = gen_of(40)
    fill(cache, gen, [[n] * B])
    w = cache.device_view()
    u = torch.arange(B * hkv, device=DEV)
    slot, col = n - 1 - u % 30, u % 64
    value = torch.tensor([math.inf, -math.inf, math.nan], device=DEV)[u % 3]
    pt = w["pages"].shape[2]
    w["pages"][w["page_table"][u, slot // pt].long(), 1, slot % pt, col] = value.bfloat16()
    q, out = queries(cache, gen, B)
    tree = hk.Tree([1] * B, torch.ones(B, 1, dtype=torch.int32, device=DEV))
    run = {"packed": lambda: cache.attend_packed(q, out, [1] * B), "window": lambda: cache.attend_window(q, out, [1] * B, 60, 2),
           "tree": lambda: cache.attend_tree(q, out, tree)}[call]
    for _ in range(30):
        out.fill_(7.0)
        run()
        got = out.view(B * hkv, 2, 64)
        want = torch.zeros(B * hkv, 64, device=DEV)
        want[u, col] = value
        bad = ~torch.isfinite(want)[:, None].expand_as(got)
        assert bool(torch.isfinite(got[~bad]).all())
        assert torch.equal(got[bad].float().nan_to_num(9.0), want[:, None].expand_as(got)[bad].nan_to_num(9.0))


# ---------------------------------------------------------------------------
# copies
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,d,page,shared", [("bf16", 128, 64, False), ("bf16", 64, 16, True), ("f32", 128, 32, True),
                                                 ("f32", 64, 256, False)])
def test_fork(hk, dtype, d, page, shared):
    hkv, L, cap = 2, 3, 512
    held = [200, 3, 0, 511, 64, 129, 65]
    src = [0, 0, 3, -1, 0, 5, 3]
    kw = dict(pool_pages=L * 7 * hkv * -(-cap // page) - 1) if shared else {}
    cache = make(hk, 7, 4, hkv, d, dtype, cap, layers=L, page_tokens=page, **kw)
    gen = gen_of(41)
    for layer in range(L):
        for n in (held[:3] + [0] * 4, [0] * 3 + held[3:]):
            t = sum(n)
            x, y = rnd(gen, t, hkv, d, dtype=dtype), rnd(gen, t, hkv, d, dtype=dtype)
            cache.append_packed(x, y, n, layer=layer)
    w = cache.device_view()
    w["importance"].copy_(torch.rand(w["importance"].shape, generator=gen, device=DEV))
    units = L * 7 * hkv
    old = [(*slots(cache, u), w["importance"][u].clone()) for u in range(units)]
    cache.fork(src, layer0=1, nlayers=2)
    cache.device_status()
    owners = set()
    for u in range(units):
        layer, b, g = u // (7 * hkv), u // hkv % 7, u % hkv
        f = u if layer == 0 or src[b] < 0 else (layer * 7 + src[b]) * hkv + g
        k, v, p, imp = old[f]
        k1, v1, p1 = slots(cache, u)
        assert torch.equal(k1, k) and torch.equal(v1, v) and torch.equal(p1, p)
        n = len(p)
        assert cache.lengths()[u] == n and torch.equal(w["importance"][u, :n], imp[:n])
        pages = w["page_table"][u, :-(-n // page)].tolist()
        assert not owners & set(pages) and min(pages, default=0) >= 0
        owners |= set(pages)
    # a copy goes on by itself
    x = rnd(gen, 7, hkv, d, dtype=dtype)
    cache.append_packed(x, x, [1] * 7, layer=1)
    assert all(torch.equal(slots(cache, (7 + b) * hkv)[0][-1], x[b, 0]) for b in range(7))
    assert all(torch.equal(slots(cache, (14 + b) * hkv)[0], old[(14 + (b if src[b] < 0 else src[b])) * hkv][0])
               for b in range(7))
    cache.device_status()


@pytest.mark.parametrize("same", [[0, 1, 64, 100], [100, 64, 63, 0], [0, 130, 130, 7]])
def test_fork_of_what_differs(hk, same):
    """Slots below `same` are left as they are, the others copied."""
    cache = make(hk, 4, 4, 2, 64, "bf16", 256)
    gen = gen_of(42)
    fill(cache, gen, [[130, 140, 135, 133]])
    old = [slots(cache, u) for u in range(8)]
    cache.fork([0, 0, 0, 0], same=same)
    for b in (1, 2, 3):
        for g in (0, 1):
            k, v, p = slots(cache, 2 * b + g)
            assert len(p) == 130 and torch.equal(p, old[g][2])
            for x, i in ((k, 0), (v, 1)):
                assert torch.equal(x[same[b]:], old[g][i][same[b]:])
                assert torch.equal(x[:same[b]], old[2 * b + g][i][:same[b]])


def test_beams_of_a_shared_pool(hk):
    """Beams that go on from one another, step by step, in a pool that holds
    just what they need: as rows that were given the same tokens."""
    B, prompt, steps = 4, 50, 24
    cap = 96
    cache = make(hk, B, 4, 2, 64, "bf16", cap, page_tokens=16, pool_pages=2 * B * 5)   # 74 tokens: five pages
    gen, cpu = gen_of(43), torch.Generator().manual_seed(11)
    x = rnd(gen, prompt, 2, 64)
    cache.append_packed(x, x, [prompt, 0, 0, 0])
    cache.fork([0] * B)
    history = [[x] for _ in range(B)]
    for step in range(steps):
        t = rnd(gen, B, 2, 64)
        cache.append_packed(t, t, [1] * B)
        for b in range(B):
            history[b].append(t[b:b + 1])
        keep = torch.randperm(B, generator=cpu)[:torch.randint(1, B + 1, (1,), generator=cpu)].tolist()
        src = [b if b in keep else keep[int(torch.randint(0, len(keep), (1,), generator=cpu))] for b in range(B)]
        cache.fork(src, same=[prompt] * B)
        history = [list(history[s]) for s in src]
    cache.device_status()
    for b in range(B):
        for g in range(2):
            k, v, p = slots(cache, 2 * b + g)
            want = torch.cat(history[b])[:, g]
            assert torch.equal(k, want) and torch.equal(v, want) and p.tolist() == list(range(prompt + steps))


def test_fork_of_cut_rows(hk):
    """Rows whose heads hold budgets of their own, forked and decoded on."""
    cfg = dict(budgets=[40, 25], num_sink=2, recent_window=8)
    cache = make(hk, 3, 4, 2, 64, "f32", 128, **cfg)
    gen = gen_of(44)
    fill(cache, gen, [[100, 30, 60]])
    cache.evict()
    cache.fork([0, 0, 0])
    assert cache.lengths().tolist() == [40, 25] * 3
    q, out = rnd(gen, 1, 1, 4, 64, dtype="f32").repeat(1, 3, 1, 1).contiguous(), torch.empty(1, 3, 4, 64, device=DEV)
    kv = rnd(gen, 1, 1, 2, 1, 64, dtype="f32").repeat(1, 3, 1, 1, 1).contiguous()
    for _ in range(5):
        cache.step(kv, kv, q, out)
        assert torch.equal(out[0, 0], out[0, 1]) and torch.equal(out[0, 0], out[0, 2])
    cache.device_status()
    lengths, positions, imp, k, v = cache.gather(with_kv=True)
    for g in (0, 1):
        for x in (positions, imp, k, v):
            assert torch.equal(x[g], x[2 + g]) and torch.equal(x[g], x[4 + g])


def test_fork_of_more_rows_than_a_launch_takes(hk):
    B = 1100
    cache = make(hk, B, 1, 1, 64, "bf16", 32, page_tokens=16, pool_pages=1700)   # what they need in the end
    gen = gen_of(45)
    held = [b % 31 if b % 100 else 30 if b % 200 == 0 else 10 for b in range(B)]
    fill(cache, gen, [held])
    rows = [slots(cache, b) for b in range(0, B, 100)]
    cache.fork([b // 100 * 100 for b in range(B)])
    cache.device_status()
    assert cache.lengths().tolist() == [30 if b // 100 % 2 == 0 else 10 for b in range(B)]
    for b in range(0, B, 7):
        for x, y in zip(slots(cache, b), rows[b // 100]):
            assert torch.equal(x, y)


# ---------------------------------------------------------------------------
# together, strided, far, in debug mode
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,d,hq,hkv,off", [("bf16", 128, 8, 2, 8), ("bf16", 64, 4, 4, 8), ("f32", 64, 8, 1, 4)])
def test_strided_rows_and_what_lies_around_them(hk, dtype, d, hq, hkv, off):
    """q as slices of a projection's output, outputs at 16-byte offsets with
    strides of their own: nothing beside the rows is written."""
    new, held = [37, 0, 70, 1], [300, 20, 5, 64]
    cache = make(hk, 4, hq, hkv, d, dtype, 384)
    gen, cpu = gen_of(61), torch.Generator().manual_seed(13)
    fill(cache, gen, (held, new))
    total = sum(new)
    q = rnd(gen, total, (hq + 2 * hkv) * d, dtype=dtype)[:, :hq * d].unflatten(1, (hq, d))
    parents = [random_tree(cpu, n) for n in new]
    tree = cache.tree(torch.tensor(sum(parents, []), dtype=torch.int32, device=DEV), new)
    for call, sees in ((lambda o: cache.attend_window(q, o, new, 50, 3), window_sees(new, [50] * hkv, 3)),
                       (lambda o: cache.attend_tree(q, o, tree), tree_sees([paths_of(p) for p in parents], held))):
        room = torch.full((total + 2, hq * d + 3 * off), 7.0, device=DEV, dtype=DT[dtype])
        out = room[1:-1, off:off + hq * d].unflatten(1, (hq, d))
        call(out)
        check(cache, q, out, new, sees)
        out.fill_(7.0)
        assert bool((room == 7.0).all())


def test_tree_over_pages_of_any_size(hk):
    for dtype, page, shared in (("bf16", 16, True), ("bf16", 32, False), ("bf16", 256, True), ("f32", 16, True)):
        new, held = [70, 1, 33], [333, 800, 5]
        kw = dict(pool_pages=3 * 2 * -(-832 // page) - 1) if shared else {}
        cache = make(hk, 3, 8, 2, 128, dtype, 832, page_tokens=page, **kw)
        gen, cpu = gen_of(62 + page), torch.Generator().manual_seed(14)
        for n in ([100, 7, 0], [233, 793, 5], new):   # shared: the rows' pages interleave
            fill(cache, gen, [n])
        masks = [torch.rand(n, n, generator=cpu) < 0.5 for n in new]
        tree = hk.Tree(new, torch.cat([bits_of(m, 3) for m in masks]).to(DEV))
        q, out = queries(cache, gen, sum(new))
        cache.attend_tree(q, out, tree)
        check(cache, q, out, new, tree_sees(masks, held))
        old = [slots(cache, u) for u in range(6)]
        keep = [[0, 1, 5, 40, 69], [], [3, 32]]
        cache.accept(tree, keep)
        for u in range(6):
            idx = list(range(held[u // 2])) + [held[u // 2] + i for i in keep[u // 2]]
            k, v, p = slots(cache, u)
            assert torch.equal(k, old[u][0][idx]) and torch.equal(v, old[u][1][idx]) and p.tolist() == list(range(len(idx)))
        cache.device_status()


def test_tree_over_a_cut_unit(hk):
    gen, cpu = gen_of(63), torch.Generator().manual_seed(15)
    cache = make(hk, 2, 8, 2, 64, "bf16", 512, budgets=[100, 60], num_sink=4, recent_window=16)
    fill(cache, gen, [[300, 40]])
    cache.evict()
    fill(cache, gen, [[20, 9]])
    masks = [torch.rand(n, n, generator=cpu) < 0.5 for n in (20, 9)]
    tree = hk.Tree([20, 9], torch.cat([bits_of(m, 1) for m in masks]).to(DEV))
    q, out = queries(cache, gen, 29)
    cache.attend_tree(q, out, tree)
    check(cache, q, out, [20, 9], tree_sees(masks, None))
    cache.accept(tree, [[2, 3], [8]])
    assert cache.lengths().tolist() == [102, 62, 41, 41]
    with pytest.raises(hk.HikvError) as e:
        cache.accept([3, 0], [[0], []])   # the cut has left two in order
    assert e.value.status == hk.HIKV_ERR_STATE


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_fork_tree_and_steps_together(hk, dtype):
    """A prompt read in windows, forked, drafted and verified by trees, decoded
    on: copies that are given the same stay the same as their source, and as a
    cache that was never forked."""
    hq, hkv, d, n = 8, 2, 64, 150
    a, b = make(hk, 3, hq, hkv, d, dtype, 256, page_tokens=16), make(hk, 3, hq, hkv, d, dtype, 256)
    gen, cpu = gen_of(64), torch.Generator().manual_seed(16)
    rope = hk.Rope(*tables(256, d))
    qkv = rnd(gen, n, hq + 2 * hkv, d, dtype=dtype)
    for c in (a, b):
        rows = [n, 0, 0] if c is a else [n] * 3
        x = qkv if c is a else qkv.repeat(3, 1, 1)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        qo, out = torch.empty_like(x[:, :hq]), torch.empty_like(x[:, :hq])
        c.append_packed(k, v, rows, q=q, q_out=qo, rope=rope)
        c.attend_window(qo, out, rows, 40, 4)
        check(c, qo, out, rows, window_sees(rows, [40] * hkv, 4))
    a.fork([0, 0, 0])
    for step in range(3):
        m = (7, 33, 1)[step]
        parent = random_tree(cpu, m)
        path = [i for i in range(m) if paths_of(parent)[-1, i]]
        flat = torch.tensor(parent * 3, dtype=torch.int32, device=DEV)
        x = rnd(gen, m, hq + 2 * hkv, d, dtype=dtype).repeat(3, 1, 1)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        outs = []
        for c in (a, b):
            qo, out = torch.empty_like(x[:, :hq]), torch.empty_like(x[:, :hq])
            tree = c.tree(flat, [m] * 3)
            c.append_tree(k, v, tree, rope, q=q, q_out=qo)
            c.attend_tree(qo, out, tree)
            c.accept(tree, [path] * 3)
            outs.append(out)
        assert torch.equal(*outs) and torch.equal(outs[0][:m], outs[0][m:2 * m]) and torch.equal(outs[0][:m], outs[0][2 * m:])
    q1, kv = rnd(gen, 1, 1, hq, d, dtype=dtype).repeat(1, 3, 1, 1), rnd(gen, 1, 1, hkv, 1, d, dtype=dtype).repeat(1, 3, 1, 1, 1)
    o1, o2 = torch.empty_like(q1), torch.empty_like(q1)
    for _ in range(3):
        a.step(kv, kv, q1, o1)
        b.step(kv, kv, q1, o2)
        assert torch.equal(o1, o2) and torch.equal(o1[0, 0], o1[0, 2])
    for x, y in zip(a.gather(with_kv=True), b.gather(with_kv=True)):
        assert torch.equal(x, y)
    a.device_status()


def test_calls_at_offsets_past_32_bits(hk):
    """A pool of 5 GiB: the last row's pages lie past 2^32 bytes."""
    B, n = 40, 30000
    cache = make(hk, B, 32, 8, 128, "bf16", 32768)
    assert cache.device_view()["pages"].numel() * 2 >= 5 << 30
    gen, cpu = gen_of(65), torch.Generator().manual_seed(17)
    zeros = [0] * (B - 1)
    fill(cache, gen, [[n] + zeros])
    cache.fork([-1] * (B - 1) + [0])
    for g in range(8):
        for x, y in zip(slots(cache, g), slots(cache, (B - 1) * 8 + g)):
            assert torch.equal(x, y)
    new = zeros + [20]
    fill(cache, gen, [new])
    parent = random_tree(cpu, 20)
    tree = cache.tree(torch.tensor(parent, dtype=torch.int32, device=DEV), new)
    q, out = queries(cache, gen, 20)
    cache.attend_tree(q, out, tree)
    check(cache, q, out, new, tree_sees([torch.zeros(0, 0)] * (B - 1) + [paths_of(parent)], None))
    cache.attend_window(q, out, new, 5000, 4)
    check(cache, q, out, new, window_sees(new, [5000] * 8, 4))
    old = slots(cache, (B - 1) * 8 + 7)
    cache.accept(tree, [[]] * (B - 1) + [[4, 19]])
    k, v, _ = slots(cache, (B - 1) * 8 + 7)
    idx = list(range(n)) + [n + 4, n + 19]
    assert torch.equal(k, old[0][idx]) and torch.equal(v, old[1][idx])
    cache.device_status()


@pytest.mark.parametrize("shared", [False, True])
def test_vacated_slots_in_debug_mode(hk, shared, monkeypatch):
    """Slots that acceptance and forks give up read as NaN, and nothing that
    is seen does."""
    monkeypatch.setenv("HIKV_DEBUG", "1")
    kw = dict(page_tokens=16, pool_pages=3 * 2 * 20 - 1) if shared else {}
    cache = make(hk, 3, 4, 2, 64, "bf16", 320, **kw)
    monkeypatch.delenv("HIKV_DEBUG")
    gen = gen_of(66)
    fill(cache, gen, [[100, 300, 20], [40, 0, 0]])
    w = cache.device_view()
    cache.accept([40, 0, 20], [[3, 9], [], []])
    cache.fork([0, 0, 0])
    assert cache.lengths().tolist() == [102] * 6
    for b in range(3):
        for g in (0, 1):
            u = 2 * b + g
            k, v, _ = slots(cache, u)
            assert bool(torch.isfinite(k).all() and torch.isfinite(v).all())
            if b != 2:                              # (row 2 was shorter before)
                assert bool(torch.isnan(w["importance"][u, 102:140]).all()) and bool((w["positions"][u, 102:140] == -1).all())
            if not shared and b != 2:
                assert math.isnan(cache.read_slot(u, 102)[2])
    q, out = queries(cache, gen, 6)
    cache.attend_window(q, out, [2, 2, 2], 30, 4)
    check(cache, q, out, [2, 2, 2], window_sees([2, 2, 2], [30, 30], 4))
    cache.device_status()


# ---------------------------------------------------------------------------
# refusals, streams
# ---------------------------------------------------------------------------
def test_refusals_leave_the_cache_as_it_was(hk):
    cache = make(hk, 2, 4, 2, 64, "bf16", 64, page_tokens=16, pool_pages=10)
    gen = gen_of(51)
    fill(cache, gen, [[30, 5]])
    cos, sin = tables(32, 64)
    rope = hk.Rope(cos, sin)
    x, q, out = rnd(gen, 4, 2, 64), rnd(gen, 4, 4, 64), torch.empty(4, 4, 64, device=DEV, dtype=torch.bfloat16)
    tree = cache.tree(torch.tensor([-1, 0, -1, 0], dtype=torch.int32, device=DEV), [2, 2])
    before = cache.kernel_launches()
    INVALID, STATE, CAP = hk.HIKV_ERR_INVALID_ARG, hk.HIKV_ERR_STATE, hk.HIKV_ERR_CAPACITY
    wide = hk.Tree([2, 2], tree.mask)
    for status, call in [
            (INVALID, lambda: cache.attend_window(q, out, [2, 2], -1)),
            (INVALID, lambda: cache.attend_window(q, out, [2, 2], 4, sink=-1)),
            (INVALID, lambda: cache.attend_window(q, q, [2, 2], 4)),
            (INVALID, lambda: cache.attend_window(q, out, [2, 2], 4, layer=1)),
            (STATE, lambda: cache.attend_window(rnd(gen, 36, 4, 64), torch.empty(36, 4, 64, device=DEV, dtype=torch.bfloat16),
                                                [30, 6], 4)),
            (INVALID, lambda: cache.append_tree(x, x, hk.Tree([3, 1], tree.mask, tree.depth), rope)),   # position 32
            (INVALID, lambda: cache.attend_tree(rnd(gen, 33, 4, 64), torch.empty(33, 4, 64, device=DEV, dtype=torch.bfloat16),
                                                hk.Tree([33, 0], torch.zeros(33, 1, dtype=torch.int32, device=DEV)))),
            (STATE, lambda: cache.attend_tree(rnd(gen, 6, 4, 64), torch.empty(6, 4, 64, device=DEV, dtype=torch.bfloat16),
                                              hk.Tree([0, 6], torch.zeros(6, 1, dtype=torch.int32, device=DEV)))),
            (INVALID, lambda: cache.accept([2, 2], [[0, 2], []])),
            (INVALID, lambda: cache.accept([2, 2], [[1, 0], []])),
            (INVALID, lambda: cache.accept([2, 2], [[0, 0], []])),
            (INVALID, lambda: cache.accept([2, 2], [[-1], []])),
            (INVALID, lambda: cache.accept([2, 2], [[0, 1, 2], []])),
            (STATE, lambda: cache.accept([2, 6], [[0], [0]])),
            (INVALID, lambda: cache.fork([1, 0])),
            (INVALID, lambda: cache.fork([0, 2])),
            (INVALID, lambda: cache.fork([0, -2])),
            (INVALID, lambda: cache.fork([0, 0], same=[0, 6])),
            (INVALID, lambda: cache.fork([0, 0], same=[0, -1])),
            (INVALID, lambda: cache.fork([0, 0], layer0=1, nlayers=1))]:
        with pytest.raises(hk.HikvError) as e:
            call()
        assert e.value.status == status, e.value
    assert cache.kernel_launches() == before
    fill(cache, gen, [[15, 0]])   # three pages a head: 45 tokens, six pages, two of row 1, two free
    before = cache.kernel_launches()
    with pytest.raises(hk.HikvError) as e:
        cache.fork([0, 0])        # four more
    assert e.value.status == CAP
    for call in (lambda: cache.attend_tree(q, out, hk.Tree([2, 3], tree.mask)),
                 lambda: cache.append_tree(x, x, wide, rope), lambda: cache.accept([2, 2], [[0]]),
                 lambda: cache.attend_window(q, out, [2, 2], [1]), lambda: cache.fork([0]),
                 lambda: cache.tree(tree.depth, [2, 3]), lambda: hk.Tree([2, 2], tree.mask, tree.depth[:3])):
        with pytest.raises(ValueError):
            call()
    assert cache.kernel_launches() == before
    assert cache.lengths().tolist() == [45, 45, 5, 5]
    cache.device_status()


def test_windows_of_many_heads(hk):
    """128 KV heads in 16 windows; more are refused."""
    cache = make(hk, 1, 128, 128, 64, "bf16", 96)
    gen = gen_of(55)
    fill(cache, gen, [[70], [20]])
    windows = [(7 * g) % 16 * 5 for g in range(128)]
    q, out = queries(cache, gen, 20)
    cache.attend_window(q, out, [20], windows, 1)
    check(cache, q, out, [20], window_sees([20], windows, 1))
    cache = make(hk, 1, 129, 129, 64, "bf16", 16)
    fill(cache, gen, [[2]])
    q, out = queries(cache, gen, 1)
    with pytest.raises(hk.HikvError) as e:
        cache.attend_window(q, out, [1], 1)
    assert e.value.status == hk.HIKV_ERR_UNSUPPORTED


def test_depths_out_of_range_are_reported(hk):
    cache = make(hk, 1, 4, 2, 64, "bf16", 64)
    cos, sin = tables(4, 64)
    x = rnd(gen_of(52), 4, 2, 64)
    tree = hk.Tree([4], torch.zeros(4, 1, dtype=torch.int32, device=DEV),
                   torch.tensor([0, 4, -1, 2 ** 31 - 1], dtype=torch.int32, device=DEV))
    cache.append_tree(x, x, tree, hk.Rope(cos, sin))
    with pytest.raises(hk.HikvError) as e:
        cache.device_status()
    assert e.value.status == hk.HIKV_ERR_STATE
    k, _, _ = slots(cache, 0)
    y, mag = rotated(x, torch.tensor([0, 3, 0, 3], device=DEV), cos, sin, False)
    close_rot(k[:, None], y[:, :1], mag[:, :1], "bf16")


def test_nothing_to_do(hk):
    cache = make(hk, 2, 4, 2, 64, "bf16", 64)
    fill(cache, gen_of(53), [[3, 4]])
    empty = torch.empty(0, 4, 64, device=DEV, dtype=torch.bfloat16)
    tree = cache.tree(torch.empty(0, dtype=torch.int32, device=DEV), [0, 0])
    before = cache.kernel_launches()
    cache.attend_window(empty, empty, [0, 0], 4)
    cache.attend_tree(empty, empty, tree)
    cache.append_tree(empty[:, :2], empty[:, :2], tree, hk.Rope(*tables(8, 64)))
    cache.accept([0, 0], [[], []])
    cache.fork([0, -1])
    assert cache.kernel_launches() == before and cache.lengths().tolist() == [3, 3, 4, 4]


def test_calls_on_a_stream_of_their_own(hk):
    """Everything on a stream that is not the current one, given by handle."""
    new, held = [9, 40], [300, 20]
    cache = make(hk, 2, 8, 2, 64, "bf16", 384)
    gen, cpu = gen_of(54), torch.Generator().manual_seed(12)
    fill(cache, gen, (held,))
    parents = [random_tree(cpu, n) for n in new]
    flat = torch.tensor(sum(parents, []), dtype=torch.int32, device=DEV)
    x = rnd(gen, 49, 2, 64)
    q, out = queries(cache, gen, 49)
    out2 = torch.full_like(out, 7.0)
    rope = hk.Rope(*tables(384, 64))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        tree = cache.tree(flat, new, stream=stream)
        cache.append_tree(x, x, tree, rope, stream=stream)
        cache.attend_tree(q, out, tree, stream=stream)
        cache.attend_window(q, out2, new, 17, 2, stream=stream)
        s.synchronize()
        check(cache, q, out, new, tree_sees([paths_of(p) for p in parents], held))
        check(cache, q, out2, new, window_sees(new, [17, 17], 2))
        cache.accept(tree, [[], []], stream=stream)
    cache.fork([0, 0], stream=s)
    s.synchronize()
    assert cache.lengths().tolist() == [300] * 4
