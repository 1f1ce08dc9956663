"""GPU tests of the packed-batch entry points: hikv_append_packed (ragged
appends with rotary positions), hikv_attend_packed (causal attention over
the paged cache), hikv_drop and hikv_device_view, each against a plain
computation in 64 bits.

Tolerances (h = half a step of the cache dtype, 2^-8 for bf16 and 2^-24 for
fp32, relative to the value; u = 2^-24):
  * rotation: two products and a sum in fp32, rounded once:
        h |y| + 3 u (|a c| + |b s|);
  * attention: a logit is a sum of d products in fp32, off by at most
    2 d u scale sum |q k| (twice the bound of a rounded sum, since a matrix
    unit may truncate where it aligns; fp32 operands in three bf16 parts lose 3 u
    of each product, far inside that); an error e in every logit moves the
    output by at most (exp(2 e) - 1) sum p |v|; the exponential by 4 u of its
    value; sums of n terms by 2 n u; probabilities rounded to the cache dtype
    in front of the product with V by h each; then the output's rounding:
        (expm1(2 e) + 2 n u + 8 u + h) sum p |v| + h |o|.
"""
import math
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U = 2.0 ** -24
DEV = "cuda:0"


@pytest.fixture(scope="module")
def hk():
    from tests.conftest import build_native
    build_native()
    import importance_aware_kv_gb300 as hk
    return hk


def make(hk, batch, hq=8, hkv=2, d=128, dtype="bf16", cap=512, layers=1, budgets=None, **kw):
    base = dict(num_layers=layers, batch=batch, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, dtype=dtype,
                num_sink=2, recent_window=8, budgets=budgets or [max(10, cap)] * (layers * hkv), max_tokens=cap)
    base.update(kw)
    return hk.Cache(hk.CacheConfig(**base))


def rnd(gen, *shape, dtype="bf16"):
    return torch.randn(*shape, generator=gen, device=DEV).to(DT[dtype])


def gen_of(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def tables(positions, rot, base=10000.0):
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    ang = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * inv
    return ang.cos().float(), ang.sin().float()


def rotated(x, pos, cos, sin, interleaved):
    """x [t][h][d] turned in 64 bits, and sum |terms| of every element."""
    y = x.double().clone()
    mag = torch.zeros_like(y)
    half = cos.shape[1]
    c, s = cos[pos].double()[:, None], sin[pos].double()[:, None]
    i = torch.arange(half, device=DEV)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = x.double()[..., ia], x.double()[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia], mag[..., ib] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return y, mag


def close_rot(got, y, mag, dtype):
    err = (got.double() - y).abs()
    assert bool((err <= HALF[dtype] * y.abs() + 3 * U * mag).all()), err.max()


def slots(cache, u):
    """K, V, positions of unit u by slot, read from its pages."""
    w = cache.device_view()
    n = int(w["lengths"][u])
    pt = cache.cfg.page_tokens or 64
    pages = w["page_table"][u, :-(-n // pt)].long()
    rows = w["pages"][pages]
    k, v = rows[:, 0].reshape(-1, cache.cfg.head_dim)[:n], rows[:, 1].reshape(-1, cache.cfg.head_dim)[:n]
    return k, v, w["positions"][u, :n]


def check_attend(cache, q, out, nq, layer=0):
    """out against softmax attention in 64 bits of each query over the slots
    at positions up to its own."""
    c = cache.cfg
    dtype, d, hkv, G = c.dtype, c.head_dim, c.num_kv_heads, c.num_q_heads // c.num_kv_heads
    scale = c.scale or 1.0 / math.sqrt(d)
    r = 0
    for b, t in enumerate(nq):
        for g in range(hkv if t else 0):
            u = (layer * c.batch + b) * hkv + g
            k, v, pos = slots(cache, u)
            n = k.shape[0]
            newest = int(pos.max())
            kd = torch.where(torch.isfinite(k), k, 0).double()
            vd = torch.where(torch.isfinite(v), v, 0).double()
            for i0 in range(0, t, 512):
                m = min(512, t - i0)
                x = q[r + i0:r + i0 + m, g * G:(g + 1) * G].double()          # [m][G][d]
                z = torch.einsum("mgd,nd->mgn", x, kd) * scale
                e = 2 * d * U * scale * torch.einsum("mgd,nd->mgn", x.abs(), kd.abs()).amax(-1)
                mine = newest - t + 1 + i0 + torch.arange(m, device=DEV)
                seen = (pos[None] <= mine[:, None])[:, None]
                p = torch.softmax(z.masked_fill(~seen, -math.inf), -1)
                o, mag = p @ vd, p @ vd.abs()
                f = torch.expm1(2 * e) + 2 * n * U + 8 * U + (HALF[dtype] if dtype == "bf16" else 0.0)
                got = out[r + i0:r + i0 + m, g * G:(g + 1) * G].double()
                err = (got - o).abs()
                tol = f[..., None] * mag + HALF[dtype] * o.abs()
                assert bool((err <= tol).all()), (b, g, i0, float((err - tol).max()), int((~(err <= tol)).sum()))
        r += t


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,d,hq,hkv,rot,interleaved", [
    ("bf16", 128, 8, 2, 128, False), ("bf16", 128, 8, 8, 64, True), ("bf16", 64, 16, 2, 64, False),
    ("bf16", 64, 2, 2, 16, True), ("f32", 64, 4, 2, 32, True), ("f32", 128, 8, 1, 128, False),
    ("f32", 128, 4, 4, 16, False), ("bf16", 128, 64, 8, 112, False), ("f32", 64, 8, 2, 48, False)])
@pytest.mark.parametrize("shared", [False, True])
def test_append_rotates_packed_sequences(hk, dtype, d, hq, hkv, rot, interleaved, shared):
    lens = [[5, 0, 63, 1, 130], [60, 3, 1, 1, 0], [1, 1, 1, 1, 1]]
    cap = 256
    kw = dict(page_tokens=16, pool_pages=5 * hkv * 16 - 1) if shared else {}
    cache = make(hk, 5, hq, hkv, d, dtype, cap, **kw)
    cos, sin = tables(cap, rot)
    rope = hk.Rope(cos, sin, interleaved)
    gen = gen_of(3)
    ks, vs = [[] for _ in range(5)], [[] for _ in range(5)]
    at = [0] * 5
    for n in lens:
        total = sum(n)
        qkv = rnd(gen, total, hq + 2 * hkv, d, dtype=dtype)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        before = qkv.clone()
        q_out = torch.full((total + 2, hq, d), 7.0, device=DEV, dtype=DT[dtype])
        cache.append_packed(k, v, n, q=q, q_out=q_out[1:-1], rope=rope)
        assert torch.equal(qkv, before)
        assert bool((q_out[0] == 7).all() and (q_out[-1] == 7).all())
        pos = torch.cat([torch.arange(a, a + m, device=DEV) for a, m in zip(at, n)])
        close_rot(q_out[1:-1], *rotated(q, pos, cos, sin, interleaved), dtype)
        # in the place of q
        cache.drop(n)
        cache.append_packed(k, v, n, q=q, q_out=q, rope=rope)
        assert torch.equal(q, q_out[1:-1])
        r = 0
        for b, m in enumerate(n):
            ks[b].append((k[r:r + m], pos[r:r + m]))
            vs[b].append(v[r:r + m])
            at[b] += m
            r += m
    cache.device_status()
    lengths, positions, imp, kc, vc = cache.gather(with_kv=True)
    for b in range(5):
        kb, pb = torch.cat([x[0] for x in ks[b]]), torch.cat([x[1] for x in ks[b]])
        y, mag = rotated(kb, pb, cos, sin, interleaved)
        for g in range(hkv):
            u = b * hkv + g
            assert int(lengths[u]) == at[b]
            assert torch.equal(positions[u, :at[b]].long(), pb)
            assert torch.equal(vc[u, :at[b]], torch.cat(vs[b])[:, g])
            close_rot(kc[u, :at[b]], y[:, g], mag[:, g], dtype)
    assert bool((imp == 0).all())


def test_append_without_rope_equals_plain_append(hk):
    gen = gen_of(5)
    k, v = rnd(gen, 1, 3, 2, 40, 64), rnd(gen, 1, 3, 2, 40, 64)
    a, b = make(hk, 3, 4, 2, 64), make(hk, 3, 4, 2, 64)
    a.append(k, v)
    pk, pv = (t[0].permute(0, 2, 1, 3).reshape(120, 2, 64) for t in (k, v))
    b.append_packed(pk, pv, [40, 40, 40])
    for x, y in zip(a.gather(with_kv=True), b.gather(with_kv=True)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("shared", [False, True])
def test_append_leaves_everything_else_as_it_was(hk, shared):
    kw = dict(page_tokens=16, pool_pages=150) if shared else {}
    cache = make(hk, 4, 4, 2, 64, "bf16", 300, layers=2, budgets=[300] * 4, **kw)
    gen = gen_of(6)
    for layer in (0, 1):
        x = rnd(gen, 100, 2, 64)
        cache.append_packed(x, x, [30, 0, 7, 63], layer=layer)
    w = cache.device_view()
    torch.cuda.synchronize()
    if not shared:
        w["importance"].add_(1.0)
    old = {k: t.clone() for k, t in w.items()}
    new = rnd(gen, 20, 2, 64)
    cache.append_packed(new, new, [0, 18, 2, 0], layer=1)
    touched = {}
    for b, m, h in ((1, 18, 0), (2, 2, 7)):
        for g in range(2):
            touched[8 + 2 * b + g] = (h, h + m)
    for u in range(16):
        lo, hi = touched.get(u, (0, 0))
        assert int(w["lengths"][u]) == int(old["lengths"][u]) + hi - lo
        for name in ("importance", "positions"):
            x, y = w[name][u].clone(), old[name][u].clone()
            x[lo:hi] = y[lo:hi] = 0
            assert torch.equal(x, y)
    pt = cache.cfg.page_tokens
    same = torch.ones(w["pages"].shape[0], 2, pt, dtype=torch.bool, device=DEV)
    for u, (lo, hi) in touched.items():
        for s in range(lo, hi):
            same[int(w["page_table"][u, s // pt]), :, s % pt] = False
    eq = (w["pages"].view(torch.int16) == old["pages"].view(torch.int16)).all(-1)
    assert bool(eq[same].all())


def test_append_and_attend_more_sequences_than_one_launch_takes(hk):
    B = 600
    gen = gen_of(7)
    n = [(7 * b) % 5 for b in range(B)]
    cache = make(hk, B, 2, 1, 64, "bf16", 32, page_tokens=16)
    cos, sin = tables(32, 64)
    total = sum(n)
    q, k, v = rnd(gen, total, 2, 64), rnd(gen, total, 1, 64), rnd(gen, total, 1, 64)
    qo, out = torch.empty_like(q), torch.empty_like(q)
    cache.append_packed(k, v, n, q=q, q_out=qo, rope=hk.Rope(cos, sin))
    assert cache.lengths().tolist() == n and cache.device_view()["lengths"].tolist() == n
    cache.attend_packed(qo, out, n)
    check_attend(cache, qo, out, n)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
SHAPES = [("bf16", 128, 8, 2), ("bf16", 128, 16, 2), ("bf16", 64, 4, 4), ("bf16", 64, 2, 1), ("bf16", 128, 2, 2),
          ("bf16", 64, 8, 1), ("f32", 64, 4, 2), ("f32", 128, 8, 1)]
LENGTHS = [([1], [0]), ([1, 2, 3], [0, 0, 0]), ([127, 128, 129, 0, 1], [0] * 5), ([255, 65], [0, 0]),
           ([700], [0]), ([1, 5, 16], [63, 64, 600]), ([33, 0, 260], [95, 10, 384]), ([1], [2000]), ([7], [5000])]


@pytest.mark.parametrize("dtype,d,hq,hkv", SHAPES)
@pytest.mark.parametrize("new,held", LENGTHS)
def test_attention(hk, dtype, d, hq, hkv, new, held):
    gen = gen_of(sum(new) + 11 * hq + d)
    cap = max(a + b for a, b in zip(new, held))
    cache = make(hk, len(new), hq, hkv, d, dtype, cap)
    for n in (held, new):
        t = sum(n)
        cache.append_packed(rnd(gen, t, hkv, d, dtype=dtype), rnd(gen, t, hkv, d, dtype=dtype), n)
    total = sum(new)
    q = rnd(gen, total, hq, d, dtype=dtype)
    buf = torch.full((total + 2, hq, d), 3.0, device=DEV, dtype=DT[dtype])
    cache.attend_packed(q, buf[1:-1], new)
    cache.device_status()
    assert bool((buf[0] == 3).all() and (buf[-1] == 3).all())
    check_attend(cache, q, buf[1:-1], new)


@pytest.mark.parametrize("page,shared", [(16, False), (16, True), (32, True), (128, False), (256, True), (1024, False)])
def test_attention_page_sizes(hk, page, shared):
    gen = gen_of(page)
    new, held = [50, 200, 1], [77, 0, 511]
    cap = 520
    pages = sum(2 * -(-(a + b) // page) for a, b in zip(new, held)) if shared else 0
    cache = make(hk, 3, 8, 2, 128, "bf16", cap, page_tokens=page, pool_pages=pages)
    for n in (held, new):
        cache.append_packed(rnd(gen, sum(n), 2, 128), rnd(gen, sum(n), 2, 128), n)
    q = rnd(gen, sum(new), 8, 128)
    out = torch.empty_like(q)
    cache.attend_packed(q, out, new)
    cache.device_status()
    check_attend(cache, q, out, new)


def test_attention_strided_rows(hk):
    """q as a slice of a projection, out heads-major, K/V from strided slices."""
    gen = gen_of(21)
    new = [40, 3, 150]
    t = sum(new)
    cache = make(hk, 3, 8, 2, 64)
    qkv = rnd(gen, t, 12 * 64)
    q, k, v = (x.unflatten(1, (-1, 64)) for x in qkv.split([512, 128, 128], 1))
    cache.append_packed(k, v, new)
    out = torch.empty(8, t, 64, device=DEV, dtype=torch.bfloat16).transpose(0, 1)
    cache.attend_packed(q, out, new)
    check_attend(cache, q, out, new)
    qh = q.transpose(0, 1).contiguous().transpose(0, 1)
    again = torch.empty_like(q)
    cache.attend_packed(qh, again, new)
    assert torch.equal(again, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layers_of_their_own(hk, dtype):
    """Three layers at lengths of their own, k rotated without a q, in a cache
    whose decode steps are element-level: attention is exact all the same."""
    gen = gen_of(25)
    cache = make(hk, 2, 4, 2, 64, dtype, 300, layers=3, element_budget=16)
    cos, sin = tables(300, 64)
    lens = [[100, 3], [1, 250], [64, 64]]
    rows = []
    for layer, n in enumerate(lens):
        k, v = rnd(gen, sum(n), 2, 64, dtype=dtype), rnd(gen, sum(n), 2, 64, dtype=dtype)
        cache.append_packed(k, v, np.array(n), layer=layer, rope=hk.Rope(cos, sin))
        rows.append(k)
    assert cache.lengths().tolist() == [x for n in lens for m in n for x in (m, m)]
    for layer in (2, 0, 1):
        n = lens[layer]
        q = rnd(gen, sum(n), 4, 64, dtype=dtype)
        out = torch.empty_like(q)
        cache.attend_packed(q, out, torch.tensor(n), layer=layer)
        check_attend(cache, q, out, n, layer)
        y, mag = rotated(rows[layer], torch.cat([torch.arange(m, device=DEV) for m in n]), cos, sin, False)
        for g in range(2):
            close_rot(slots(cache, 4 * layer + g)[0], y[:n[0], g], mag[:n[0], g], dtype)
    cache.device_status()


@pytest.mark.parametrize("dtype,d,hq,hkv", [("bf16", 128, 8, 2), ("bf16", 64, 16, 2), ("f32", 64, 4, 2)])
@pytest.mark.parametrize("sizes", [[1] * 9, [64, 64, 44], [130, 1, 41]])
def test_chunks_of_a_prompt_give_the_whole(hk, dtype, d, hq, hkv, sizes):
    """Chunk by chunk, cut between chunks for one cache: every chunk against 64 bits."""
    gen = gen_of(31)
    whole = make(hk, 2, hq, hkv, d, dtype, 512)
    cut = make(hk, 2, hq, hkv, d, dtype, 512, budgets=[20 + 9 * g for g in range(hkv)])
    for m in sizes:
        n = [m, max(0, m - 3)]
        t = sum(n)
        k, v, q = rnd(gen, t, hkv, d, dtype=dtype), rnd(gen, t, hkv, d, dtype=dtype), rnd(gen, t, hq, d, dtype=dtype)
        for cache in (whole, cut):
            cache.append_packed(k, v, n)
            out = torch.empty_like(q)
            cache.attend_packed(q, out, n)
            check_attend(cache, q, out, n)
        cut.evict()
    cut.device_status()
    assert cut.lengths().max() <= 20 + 9 * (hkv - 1)


def test_attention_long_cache_few_rows_and_many(hk):
    gen = gen_of(41)
    cache = make(hk, 2, 8, 2, 128, "bf16", 20000)
    held, new = [19000, 777], [17, 900]
    for n in (held, new):
        cache.append_packed(rnd(gen, sum(n), 2, 128), rnd(gen, sum(n), 2, 128), n)
    q = rnd(gen, sum(new), 8, 128)
    out = torch.empty_like(q)
    cache.attend_packed(q, out, new)
    cache.device_status()
    check_attend(cache, q, out, new)
    # the same queries in the other order of work: results do not depend on the run
    again = torch.empty_like(q)
    cache.attend_packed(q, again, new)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype,d,hq,hkv", [("bf16", 128, 8, 2), ("bf16", 64, 8, 1), ("f32", 128, 4, 2), ("f32", 64, 8, 1)])
@pytest.mark.parametrize("new,held,cut", [([3], [9000], None), ([40, 1, 0], [9000, 300, 50], None),
                                          ([5, 70], [7000, 6000], [5000, 100]), ([33], [12000], [40, 9000])])
def test_attention_split_keys(hk, dtype, d, hq, hkv, new, held, cut):
    """Few rows over long keys, which several work items share: heads cut to
    lengths of their own, among them some shorter than one part."""
    gen = gen_of(sum(held) + hq)
    cap = max(a + b for a, b in zip(new, held))
    cache = make(hk, len(new), hq, hkv, d, dtype, cap, budgets=cut[:hkv] if cut else None)
    for i, n in enumerate((held, new)):
        t = sum(n)
        cache.append_packed(rnd(gen, t, hkv, d, dtype=dtype), rnd(gen, t, hkv, d, dtype=dtype), n)
        if i == 0:
            cache.evict()
    q = rnd(gen, sum(new), hq, d, dtype=dtype)
    out = torch.empty_like(q)
    launches = cache.kernel_launches()
    cache.attend_packed(q, out, new)
    # the parts and their join (one head cut to 40 tokens leaves nothing to split)
    assert cache.kernel_launches() == launches + (2 if cache.lengths().max() > 1000 else 1)
    cache.device_status()
    check_attend(cache, q, out, new)


@pytest.mark.parametrize("dtype,d,hq,hkv", [("bf16", 128, 8, 2), ("f32", 64, 4, 2)])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_non_finite_values_in_split_keys(hk, dtype, d, hq, hkv, value, monkeypatch):
    """A non-finite V element among the new tokens of a split call."""
    monkeypatch.setenv("HIKV_DEBUG", "1")
    gen = gen_of(57)
    held, n, bad = 6000, 20, 6009
    k, v = rnd(gen, held + n, hkv, d, dtype=dtype), rnd(gen, held + n, hkv, d, dtype=dtype)
    q = rnd(gen, n, hq, d, dtype=dtype)
    v[bad, :, 5] = value
    cache = make(hk, 1, hq, hkv, d, dtype, 6100)
    cache.append_packed(k, v, [held + n])
    out = torch.empty_like(q)
    cache.attend_packed(q, out, [n])
    head = make(hk, 1, hq, hkv, d, dtype, 6100)
    m = bad - held
    head.append_packed(k[:bad], v[:bad], [bad])
    check_attend(head, q[:m], out[:m], [m])
    assert not bool(torch.isfinite(out[m:, :, 5]).any())
    assert bool(torch.isfinite(out[:, :, [i for i in range(d) if i != 5]]).all())
    cache.device_status()


def test_attention_with_an_unread_error_pending(hk):
    """Another kernel's recorded time-out does not keep the queries from being answered."""
    gen = gen_of(59)
    cache = make(hk, 1, 8, 2)
    x, q = rnd(gen, 100, 2, 128), rnd(gen, 100, 8, 128)
    cache.append_packed(x, x, [100])
    cache.selftest_timeout(1000)
    out = torch.empty_like(q)
    cache.attend_packed(q, out, [100])
    check_attend(cache, q, out, [100])
    with pytest.raises(hk.HikvError) as ei:
        cache.device_status()
    assert ei.value.status == hk.HIKV_ERR_TIMEOUT
    cache.device_status()


def test_attention_large_logits(hk):
    """Rows whose maximum keeps growing along the keys, and far negative ones."""
    gen = gen_of(43)
    n = 900
    for dtype in ("bf16", "f32"):
        cache = make(hk, 1, 4, 1, 128, dtype, n, scale=1.0)
        grow = torch.linspace(0.01, 1.0, n, device=DEV)[:, None, None]
        k = (torch.ones(n, 1, 128, device=DEV) * grow).to(DT[dtype])
        q = torch.cat([torch.ones(n, 2, 128, device=DEV), -torch.ones(n, 2, 128, device=DEV)], 1).to(DT[dtype])
        v = rnd(gen, n, 1, 128, dtype=dtype)
        cache.append_packed(k, v, [n])
        out = torch.empty_like(q)
        cache.attend_packed(q, out, [n])
        check_attend(cache, q, out, [n])


@pytest.mark.parametrize("dtype,d,hq,hkv", [("bf16", 128, 8, 2), ("bf16", 64, 8, 1), ("f32", 64, 4, 2)])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_what_a_query_does_not_see_does_not_touch_it(hk, dtype, d, hq, hkv, value, monkeypatch):
    """Non-finite K and V rows at one position: earlier queries are exact, V's
    own elements non-finite from there on; slots behind the units' ends NaN."""
    monkeypatch.setenv("HIKV_DEBUG", "1")
    gen = gen_of(51)
    n, bad = 391, 200
    for where in ("v", "k"):
        cache = make(hk, 1, hq, hkv, d, dtype, 512)
        k, v = rnd(gen, n, hkv, d, dtype=dtype), rnd(gen, n, hkv, d, dtype=dtype)
        q = rnd(gen, n, hq, d, dtype=dtype)
        (v if where == "v" else k)[bad, :, 3] = value
        cache.append_packed(k, v, [n])
        out = torch.empty_like(q)
        cache.attend_packed(q, out, [n])
        head = make(hk, 1, hq, hkv, d, dtype, 512)
        head.append_packed(k[:bad], v[:bad], [bad])
        check_attend(head, q[:bad], out[:bad], [bad])
        if where == "v":
            assert not bool(torch.isfinite(out[bad:, :, 3]).any())
            if not math.isnan(value):
                assert bool((out[bad:, :, 3] == value).all())
            keep = [i for i in range(d) if i != 3]
            assert bool(torch.isfinite(out[:, :, keep]).all())


def test_attention_past_32_bit_offsets(hk):
    """The last unit's pages start beyond 4 GiB of the pool."""
    gen = gen_of(61)
    cap = 1 << 20
    cache = make(hk, 1, 9, 9, 128, "bf16", cap, budgets=[cap] * 9)
    n = [300]
    k, v, q = (rnd(gen, 300, 9, 128) for _ in range(3))
    cache.append_packed(k, v, n)
    out = torch.empty_like(q)
    cache.attend_packed(q, out, n)
    cache.device_status()
    check_attend(cache, q, out, n)


# ---------------------------------------------------------------------------
# drop
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("debug", [False, True])
def test_drop_then_decode_equals_a_cache_that_never_held_them(hk, debug, monkeypatch):
    if debug:
        monkeypatch.setenv("HIKV_DEBUG", "1")
    gen = gen_of(71)
    caches = [make(hk, 3, 8, 2, 128, "bf16", 200, layers=2, budgets=[100] * 4) for _ in range(2)]
    n = [50, 1, 90]
    for layer in (0, 1):
        k, v = rnd(gen, sum(n), 2, 128), rnd(gen, sum(n), 2, 128)
        for c in caches:
            c.append_packed(k, v, n, layer=layer)
    extra = [20, 3, 0]
    for layer in (0, 1):
        x = rnd(gen, sum(extra), 2, 128)
        caches[0].append_packed(x, x, extra, layer=layer)
    caches[0].drop(extra)
    assert caches[0].lengths().tolist() == caches[1].lengths().tolist()
    for _ in range(30):
        k, v = rnd(gen, 2, 3, 2, 1, 128), rnd(gen, 2, 3, 2, 1, 128)
        q = rnd(gen, 2, 3, 8, 128)
        outs = [torch.empty_like(q) for _ in caches]
        for c, o in zip(caches, outs):
            c.step(k, v, q, o)
        assert torch.equal(*outs)
    for x, y in zip(caches[0].gather(with_kv=True), caches[1].gather(with_kv=True)):
        assert torch.equal(x, y)
    for c in caches:
        c.device_status()


def test_drop_of_all_returns_the_pages(hk):
    gen = gen_of(73)
    cache = make(hk, 2, 4, 2, 64, "bf16", 256, page_tokens=16, pool_pages=20, budgets=[16, 16])
    x = rnd(gen, 150, 2, 64)
    for n in ([150, 0], [0, 150], [70, 80], [150, 0]):
        cache.append_packed(x, x, n)
        cache.evict()
        with pytest.raises(hk.HikvError) as ei:   # cut: nothing of it is in order any more
            cache.drop([1 if m else 0 for m in n])
        assert ei.value.status == hk.HIKV_ERR_STATE
        cache.drop([-1 if m else 0 for m in n])
    assert not cache.lengths().any()
    cache.append_packed(x, x, [150, 0])
    out = torch.empty(150, 4, 64, device=DEV, dtype=torch.bfloat16)
    q = rnd(gen, 150, 4, 64)
    cache.attend_packed(q, out, [150, 0])
    check_attend(cache, q, out, [150, 0])
    cache.drop()
    assert not cache.lengths().any() and not cache.device_view()["lengths"].any()
    cache.device_status()


# ---------------------------------------------------------------------------
# the run of them together, captured, on another stream
# ---------------------------------------------------------------------------
def test_serving_run(hk):
    """Ragged prompts appended with rotation, attended, scored, cut; decode
    steps with rotation; a verification whose tail is rejected; next turn."""
    gen = gen_of(81)
    B, hq, hkv, d = 3, 8, 2, 128
    cache = make(hk, B, hq, hkv, d, "bf16", 400, budgets=[64, 90], max_window_queries=8)
    cos, sin = tables(600, d)
    rope = hk.Rope(cos, sin)

    def turn(n):
        t = sum(n)
        qkv = rnd(gen, t, hq + 2 * hkv, d)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        cache.append_packed(k, v, n, q=q, q_out=q, rope=rope)
        out = torch.empty(t, hq, d, device=DEV, dtype=torch.bfloat16)
        cache.attend_packed(q, out, n)
        check_attend(cache, q, out, n)
        return q, out

    n = [200, 37, 131]
    q, _ = turn(n)
    ends = np.cumsum(n)
    cache.score_window(torch.stack([q[e - 8:e].transpose(0, 1) for e in ends])[None].contiguous())
    cache.evict()
    assert cache.lengths().tolist() == [64, 90, 37, 37, 64, 90]
    for _ in range(4):
        q, _ = turn([1] * B)
        out = torch.empty(1, B, hq, d, device=DEV, dtype=torch.bfloat16)
        cache.decode_step(q[None].contiguous(), out)
        cache.evict()
    turn([5, 5, 5])
    cache.drop([3, 0, 4])
    turn([60, 1, 0])
    cache.drop()
    turn([10, 300, 0])
    cache.device_status()


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 2, 128), ("f32", 4, 2, 64)])
def test_captured_and_replayed(hk, dtype, hq, hkv, d):
    gen = gen_of(91)
    cache = make(hk, 2, hq, hkv, d, dtype, 9000)
    held, n = [8000, 50], [3, 200]
    cache.append_packed(rnd(gen, sum(held), hkv, d, dtype=dtype), rnd(gen, sum(held), hkv, d, dtype=dtype), held)
    t = sum(n)
    cos, sin = tables(9000, d)
    rope = hk.Rope(cos, sin)
    qkv = rnd(gen, t, hq + 2 * hkv, d, dtype=dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    qo, out = torch.empty(2, t, hq, d, device=DEV, dtype=DT[dtype])
    cache.append_packed(k, v, n, q=q, q_out=qo, rope=rope)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def once():
        cache.drop(n)
        cache.append_packed(k, v, n, q=q, q_out=qo, rope=rope)
        cache.attend_packed(qo, out, n)

    with torch.cuda.stream(side):
        once()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            once()
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        qkv.copy_(rnd(gen, t, hq + 2 * hkv, d, dtype=dtype))
        out.zero_()
        graph.replay()
        got = out.clone()
        check_attend(cache, qo, got, n)
        once()   # eager, after the replay
        assert torch.equal(got, out)
    assert cache.lengths().tolist() == [8003] * hkv + [250] * hkv
    assert cache.device_view()["lengths"].tolist() == cache.lengths().tolist()
    cache.device_status()


def test_two_caches_on_two_streams(hk):
    gen = gen_of(95)
    n = [1500, 4, 700]
    t = sum(n)
    data = []
    for _ in range(2):
        c = make(hk, 3, 8, 2, 128, "bf16", 1500)
        k, v, q = rnd(gen, t, 2, 128), rnd(gen, t, 2, 128), rnd(gen, t, 8, 128)
        data.append((c, k, v, q, torch.empty_like(q), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for c, k, v, q, out, s in data:
            c.drop(stream=s)
            c.append_packed(k, v, n, stream=s)
            c.attend_packed(q, out, n, stream=s)
    torch.cuda.synchronize()
    for c, k, v, q, out, s in data:
        check_attend(c, q, out, n)
        c.device_status()


# ---------------------------------------------------------------------------
# refusals: an error, and the cache as it was
# ---------------------------------------------------------------------------
def test_refusals_leave_the_cache_as_it_was(hk):
    gen = gen_of(99)
    cache = make(hk, 2, 4, 2, 64, "bf16", 100, budgets=[40, 40])
    x = rnd(gen, 60, 2, 64)
    cache.append_packed(x, x, [50, 10])
    cos, sin = tables(52, 64)
    rope = hk.Rope(cos, sin)
    q, qo = rnd(gen, 4, 4, 64), torch.zeros(4, 4, 64, device=DEV, dtype=torch.bfloat16)
    y = rnd(gen, 4, 2, 64)
    big = rnd(gen, 60, 2, 64)
    odd = rnd(gen, 4 * 2 * 72 + 8)[4:4 + 4 * 2 * 72].view(4, 2, 72)[..., :64]
    lap = torch.zeros(4 * 4 * 64, device=DEV, dtype=torch.bfloat16).as_strided((4, 4, 64), (64, 64, 1))
    r16 = hk.Rope(*tables(100, 24))

    def err(status, f):
        launches, lens = cache.kernel_launches(), cache.lengths().tolist()
        with pytest.raises(hk.HikvError) as ei:
            f()
        assert ei.value.status == status, str(ei.value)
        assert cache.kernel_launches() == launches and cache.lengths().tolist() == lens

    BAD, CAPA, STATE, UNS = (hk.HIKV_ERR_INVALID_ARG, hk.HIKV_ERR_CAPACITY, hk.HIKV_ERR_STATE,
                             hk.HIKV_ERR_UNSUPPORTED)
    err(BAD, lambda: cache.append_packed(y, y, [4, 0], layer=1))
    err(BAD, lambda: cache.append_packed(y, y, [5, -1]))
    err(BAD, lambda: cache.append_packed(odd, y, [4, 0]))
    err(BAD, lambda: cache.append_packed(y, odd, [4, 0]))
    err(BAD, lambda: cache.append_packed(y, y, [4, 0], q=q, q_out=qo))
    err(BAD, lambda: cache.append_packed(y, y, [4, 0], q=q, q_out=qo, rope=rope))     # position 53 of 52
    err(BAD, lambda: cache.append_packed(y, y, [0, 4], q=q, q_out=lap, rope=rope))
    err(UNS, lambda: cache.append_packed(y, y, [0, 4], rope=r16))
    err(CAPA, lambda: cache.append_packed(big, big, [60, 0]))
    err(BAD, lambda: cache.attend_packed(q, qo, [4, 0], layer=-1))
    err(BAD, lambda: cache.attend_packed(q, q, [4, 0]))
    err(BAD, lambda: cache.attend_packed(q, lap, [4, 0]))
    err(BAD, lambda: cache.attend_packed(q, qo, [5, -1]))
    err(STATE, lambda: cache.attend_packed(rnd(gen, 11, 4, 64), torch.empty(11, 4, 64, device=DEV, dtype=torch.bfloat16),
                                           [0, 11]))
    err(STATE, lambda: cache.drop([0, 11]))
    err(BAD, lambda: cache.drop([0, 0], layer0=1, nlayers=1))
    cache.evict()     # cuts sequence 0 to 40
    err(STATE, lambda: cache.attend_packed(q, qo, [1, 3]))
    err(STATE, lambda: cache.drop([1, 0]))
    cache.append_packed(y, y, [1, 3])
    cache.attend_packed(q, qo, [1, 3])
    check_attend(cache, q, qo, [1, 3])
    for bad in (lambda: cache.append_packed(y.cpu(), y, [4, 0]), lambda: cache.append_packed(y.float(), y, [4, 0]),
                lambda: cache.attend_packed(q, qo.float(), [4, 0])):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: cache.append_packed(y, y, [3, 0]), lambda: cache.append_packed(y, y, [4]),
                lambda: cache.append_packed(y.transpose(1, 2).contiguous().transpose(1, 2), y, [4, 0]),
                lambda: cache.attend_packed(q, qo, [2, 1]), lambda: cache.drop([1])):
        with pytest.raises(ValueError):
            bad()
    cache.append_packed(y[:0], y[:0], [0, 0])
    cache.attend_packed(q[:0], qo[:0], [0, 0])
    cache.device_status()
    cache.close()
    with pytest.raises(hk.HikvError):
        cache.attend_packed(q, qo, [1, 3])


def test_overlapping_rows_are_refused_and_slices_are_not(hk):
    """Written rows that share memory with rows that are read are refused; slices
    of one buffer, tokens or heads outermost, are not."""
    gen = gen_of(101)
    cache = make(hk, 1, 4, 2, 64, "bf16", 400)
    cos, sin = tables(400, 64)
    rope = hk.Rope(cos, sin)
    t = 20
    buf = rnd(gen, t + 1, 8, 64)
    q, k, v = buf[:t, :4], buf[:t, 4:6], buf[:t, 6:]
    for bad in (buf[1:, :4], buf[:t, 1:5], buf[:t, 2:6], buf[:t, 4:], buf[1:, 3:7],
                buf.view(-1)[64:64 + t * 256].view(t, 4, 64)):
        with pytest.raises(hk.HikvError) as ei:
            cache.append_packed(k, v, [t], q=q, q_out=bad, rope=rope)
        assert ei.value.status == hk.HIKV_ERR_INVALID_ARG
    heads = rnd(gen, 8, t, 64).transpose(0, 1)     # head outermost
    cache.append_packed(heads[:, 4:6], heads[:, 6:], [t], q=heads[:, :4], q_out=heads[:, :4], rope=rope)
    cache.append_packed(k, v, [t], q=q, q_out=q, rope=rope)
    for out in (buf[1:, :4], buf[:t, 1:5], q):
        with pytest.raises(hk.HikvError) as ei:
            cache.attend_packed(q, out, [t])
        assert ei.value.status == hk.HIKV_ERR_INVALID_ARG
    q2 = q.clone()
    out = buf[:t, 4:]                              # beside q in its own buffer
    cache.attend_packed(q, out, [t])
    assert torch.equal(q, q2)
    check_attend(cache, q2, out, [t])
    one = rnd(gen, 1, 8, 64)
    cache.append_packed(one[:, 4:6], one[:, 6:], [1], q=one[:, :4], q_out=one[:, :4], rope=rope)
    cache.attend_packed(one[:, :4], one[:, 4:], [1])
    check_attend(cache, one[:, :4], one[:, 4:], [1])
    cache.device_status()
