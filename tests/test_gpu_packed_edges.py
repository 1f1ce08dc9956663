"""GPU tests of the packed-batch entry points at the edges of what they take:
keys on both sides of every page, tile, split and causal edge, values near the
ends of the number range, an unread time-out, broadcast rows.

Bounds on the attention's error (notation of test_gpu_packed.py: h half a step
of the cache dtype, u = 2^-24, e the error of a logit, p the exact weights, o
the exact output).  Numerator and denominator are sums of the weights
p_j (1 + a_j), |a_j| <= a = expm1(2 e) + 8 u, and sum_j p_j (v_j - o) = 0, so
these errors move a row only as far as its values differ.  bf16 rounds the
weights of the numerator once more, by h (fp32: g = 0, else g = h), and takes
the rounded value of the largest, p_m, into the denominator as well:
    |out - o| <= [a sum_j p_j |v_j - o|
                  + g (p_m |v_m - o| + sum_{j != m} p_j |v_j|)] / (1 - a - g)
                 + 2 n u sum_j p_j |v_j| + h |o|.
Norm-wise, with independent roundings of variance below h^2,
    |out - o|^2 <= 2 sum [g^2 (p_m^2 (v_m - o)^2 + sum_{j != m} p_j^2 v_j^2)
                          + a^2 sum_j p_j^2 (v_j - o)^2 + h^2 o^2]
                   + sum [n u (|o| + 4 sqrt(sum_j p_j^2 v_j^2))]^2
(the factor 2 on top of a variance that is at most a third of h^2; the last
term: n additions that each lose u of a partial sum, partial sums at most four
times their random-walk size).
"""
import gc
import math

import pytest
import torch

from tests.test_gpu_packed import DEV, DT, HALF, U, gen_of, hk, make, rnd, slots  # noqa: F401

pytestmark = pytest.mark.gpu


def check_edges(cache, q, out, nq, layer=0, norm=False):
    """out against attention in 64 bits by the bounds above, element by element
    or (norm) over all rows of a sequence and KV head."""
    c = cache.cfg
    dtype, d, hkv, G = c.dtype, c.head_dim, c.num_kv_heads, c.num_q_heads // c.num_kv_heads
    scale = c.scale or 1.0 / math.sqrt(d)
    h, gp = HALF[dtype], HALF[dtype] if dtype == "bf16" else 0.0
    r = 0
    for b, t in enumerate(nq):
        for g in range(hkv if t else 0):
            k, v, pos = slots(cache, (layer * c.batch + b) * hkv + g)
            n = k.shape[0]
            newest = int(pos.max())
            kd, vd = k.double(), v.double()
            total = limit = 0.0
            for i0 in range(0, t, 64):
                m = min(64, t - i0)
                x = q[r + i0:r + i0 + m, g * G:(g + 1) * G].double()
                z = torch.einsum("mgd,nd->mgn", x, kd) * scale
                e = 2 * d * U * scale * torch.einsum("mgd,nd->mgn", x.abs(), kd.abs()).amax(-1)
                mine = newest - t + 1 + i0 + torch.arange(m, device=DEV)
                p = torch.softmax(z.masked_fill(~(pos[None] <= mine[:, None])[:, None], -math.inf), -1)
                o = p @ vd
                a = (torch.expm1(2 * e) + 8 * U)[..., None]
                pm, m_at = p.max(-1, keepdim=True)
                vm = vd[m_at[..., 0]]
                err = (out[r + i0:r + i0 + m, g * G:(g + 1) * G].double() - o).abs()
                if norm:
                    p2 = p * p
                    v2 = p2 @ (vd * vd)
                    spread = v2 - 2 * o * (p2 @ vd) + p2.sum(-1, keepdim=True) * o * o
                    rounded = v2 + pm * pm * ((vm - o).square() - vm.square())
                    limit += float((2 * (gp * gp * rounded + a * a * spread + h * h * o * o)).sum())
                    limit += float((n * U * (o.abs() + 4 * v2.sqrt())).square().sum())
                    total += float(err.square().sum())
                    continue
                spread = torch.stack([(p * (vd[:, j] - o[..., j:j + 1]).abs()).sum(-1) for j in range(d)], -1)
                mag = p @ vd.abs()
                rounded = mag + pm * ((vm - o).abs() - vm.abs())
                tol = ((a * spread + gp * rounded) / (1 - a - gp) + 2 * n * U * mag) * (1 + h) + h * o.abs()
                assert bool((err <= tol).all()), (b, g, i0, float((err - tol).max()), int((~(err <= tol)).sum()))
            assert not norm or total <= limit, (b, g, total, limit)
        r += t


# ---------------------------------------------------------------------------
# every key once: no key missed, taken twice, or seen too early
# ---------------------------------------------------------------------------
def needles(gen, cache, held, new, hq, hkv, d, dtype):
    """Keys of +-1; each query points at two of them with equal logits that
    outweigh all others together: one at an edge and another, far from it.  A
    missed edge key leaves the other's value, one taken twice weighs 2 : 1, and
    a key behind the causal limit shows where the other alone should."""
    lens = [a + b for a, b in zip(held, new)]
    ks = []
    for n in (held, new):
        t = sum(n)
        k = torch.randint(0, 2, (t, hkv, d), generator=gen, device=DEV).mul(2).sub(1).to(DT[dtype])
        cache.append_packed(k, rnd(gen, t, hkv, d, dtype=dtype), n)
        ks.append(k.split(n))
    keys = [torch.cat([a, b]) for a, b in zip(*ks)]
    # slots on both sides of every 16 (pages, tiles of 64 and 128 keys and parts of the keys begin at some)
    edges = [sorted({s for x in range(0, n + 1, 16) for s in (x - 1, x) if 0 <= s < n}) for n in lens]
    G = hq // hkv
    at = 0
    while at < max(len(e) for e in edges):
        q = torch.empty(sum(new), hq, d, device=DEV)
        r = 0
        for b, t in enumerate(new):
            e = torch.tensor(edges[b], device=DEV)
            i = torch.arange(t, device=DEV)[:, None].expand(t, G)
            lim = held[b] + i
            a = e[(at + torch.arange(t * G, device=DEV).view(t, G)) % len(e)]
            # the first two heads also look at the causal limit and right behind it
            a[:, 0] = torch.where(torch.arange(t, device=DEV) % 2 == at % 2, lim[:, 0], a[:, 0])
            if G > 1:
                a[:, 1] = (lim[:, 1] + 1).clamp(max=lens[b] - 1)
            # (the other is always visible: an edge key may not be)
            other = (a + 37 + lens[b] // 2) % (held[b] + i + 1)
            for g in range(hkv):
                q[r:r + t, g * G:(g + 1) * G] = keys[b][a, g].float() + keys[b][other, g].float()
            r += t
        at += sum(new) * G if sum(new) else 1
        yield (2 * q).to(DT[dtype])


@pytest.mark.parametrize("dtype,d,hq,hkv", [("bf16", 128, 8, 2), ("bf16", 128, 8, 1), ("bf16", 64, 4, 2), ("bf16", 128, 2, 2),
                                            ("f32", 64, 4, 2)])
@pytest.mark.parametrize("new,held,page", [([17], [9000], 64), ([40, 1], [5000, 300], 16), ([3, 5], [2000, 2500], 128),
                                           ([130], [1000], 64), ([300, 129], [0, 140], 32), ([700], [0], 256)])
def test_every_edge_key_counts_once(hk, dtype, d, hq, hkv, new, held, page):
    gen = gen_of(sum(held) + d + hq)
    cap = max(a + b for a, b in zip(new, held))
    cache = make(hk, len(new), hq, hkv, d, dtype, cap, page_tokens=page, scale=0.25 if d == 64 else 0.125)
    out = torch.empty(sum(new), hq, d, device=DEV, dtype=DT[dtype])
    for q in needles(gen, cache, held, new, hq, hkv, d, dtype):
        cache.attend_packed(q, out, new)
        check_edges(cache, q, out, new)
    cache.device_status()


@pytest.mark.parametrize("dtype,d,hq,hkv", [("bf16", 128, 8, 2), ("bf16", 64, 8, 1), ("f32", 64, 4, 2)])
@pytest.mark.parametrize("new,held", [([17], [19000]), ([64], [9000]), ([40, 3], [5000, 2000]), ([1000], [0]), ([300, 200], [700, 31])])
def test_error_over_many_keys_is_that_of_rounding(hk, dtype, d, hq, hkv, new, held):
    """Norm-wise: a key or a tile of keys lost somewhere in a long cache is larger than the rounding."""
    gen = gen_of(sum(held) + sum(new) + d)
    cap = max(a + b for a, b in zip(new, held))
    cache = make(hk, len(new), hq, hkv, d, dtype, cap)
    for n in (held, new):
        cache.append_packed(rnd(gen, sum(n), hkv, d, dtype=dtype), rnd(gen, sum(n), hkv, d, dtype=dtype), n)
    q = rnd(gen, sum(new), hq, d, dtype=dtype)
    out = torch.empty_like(q)
    cache.attend_packed(q, out, new)
    cache.device_status()
    check_edges(cache, q, out, new, norm=True)


# ---------------------------------------------------------------------------
# values of every size
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("at", [5, 200, 290])
def test_a_row_that_sees_one_key_returns_its_value(hk, dtype, d, at):
    """One key has all but 300 e^-14 = 0.00025 of a row's weight: the rounding
    of its probability, 2^-8, is in numerator and denominator alike."""
    gen = gen_of(111 + at)
    n, t = 300, 8
    cache = make(hk, 1, 8, 2, d, dtype, n, scale=1.0)
    k = torch.zeros(n, 2, d, device=DEV)
    k[at, :, 0] = 14.0
    v = rnd(gen, n, 2, d, dtype=dtype)
    cache.append_packed(k.to(DT[dtype]), v, [n])
    q = torch.zeros(t, 8, d, device=DEV)
    # logits 14 to 16.3, all bf16 steps of their binade among them; log2 of the weights 20.2 to 23.4
    q[..., 0] = 1.0 + torch.arange(t * 8, device=DEV).view(t, 8) / 384.0
    q = q.to(DT[dtype])
    out = torch.empty_like(q)
    cache.attend_packed(q, out, [t])
    check_edges(cache, q, out, [t])
    cache.device_status()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("size", [1e-25, 1e33, 1e36])
@pytest.mark.parametrize("held", [0, 6000])
def test_values_whose_mean_is_finite(hk, dtype, d, size, held):
    """Logits that grow along the keys by up to 23 in powers of two, and values
    so large that the weights have to stay near one for sums to be finite:
    |v| <= 5 x 10^36, at most 64 keys near the maximum."""
    gen = gen_of(121)
    n, t = held + 300, 9
    cache = make(hk, 1, 8, 2, d, dtype, n, scale=1.0)
    k = torch.full((n, 2, d), 0.0, device=DEV)
    k[:, :, 0] = -30.0
    k[:held + 64, :, 0] = torch.linspace(-40.0, 0.0, held + 64, device=DEV)[:, None]
    k[held + 140:held + 200, :, 0] = 15.0
    v = (rnd(gen, n, 2, d, dtype="f32") * size).to(DT[dtype])
    cache.append_packed(k.to(DT[dtype]), v, [n])
    q = torch.zeros(t, 8, d, device=DEV)
    q[..., 0] = 1.0 - torch.arange(t * 8, device=DEV).view(t, 8) / 100.0
    q = q.to(DT[dtype])
    out = torch.empty_like(q)
    cache.attend_packed(q, out, [t])
    assert bool(torch.isfinite(out).all())
    check_edges(cache, q, out, [t])
    cache.device_status()


@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (128, 8, 1)])
@pytest.mark.parametrize("where", ["q", "k", "v"])
@pytest.mark.parametrize("value", [3.3895314e38, 3.3961775e38, 3.3999e38, 3.4028234663852886e38, -3.4028234663852886e38])
def test_the_largest_fp32_numbers_are_numbers(hk, d, hq, hkv, where, value):
    """Elements of q, k and v up to the largest finite one, whose nearest bf16
    is an infinity: against 2^-124 in a logit, and as one value among others."""
    gen = gen_of(131)
    n = 150
    cache = make(hk, 1, hq, hkv, d, "f32", n)
    k, v, q = rnd(gen, n, hkv, d, dtype="f32"), rnd(gen, n, hkv, d, dtype="f32"), rnd(gen, n, hq, d, dtype="f32")
    if where == "v":
        v[70, :, 5] = value
    else:
        big, small = (q, k) if where == "q" else (k, q)
        big[..., 3] = 0.0
        big[70, :, 3] = value
        small[..., 3] = 2.0 ** -124
    cache.append_packed(k, v, [n])
    out = torch.empty_like(q)
    cache.attend_packed(q, out, [n])
    assert bool(torch.isfinite(out).all())
    check_edges(cache, q, out, [n])
    cache.device_status()


# ---------------------------------------------------------------------------
# an unread time-out of the attention itself
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,d,hq,hkv", [("bf16", 128, 8, 2), ("f32", 64, 4, 2)])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("held,new", [(9000, 3), (100, 3), (0, 200)])
def test_attention_writes_nothing_while_its_timeout_is_unread(hk, dtype, d, hq, hkv, first, held, new, monkeypatch):
    """Split over the keys or not, after another kernel's time-out (first) or alone."""
    gen = gen_of(141)
    cache = make(hk, 1, hq, hkv, d, dtype, 9100)
    for n in (held, new):
        x = rnd(gen, n, hkv, d, dtype=dtype)
        cache.append_packed(x, rnd(gen, n, hkv, d, dtype=dtype), [n])
    q, other = rnd(gen, new, hq, d, dtype=dtype), rnd(gen, new, hq, d, dtype=dtype)
    out = torch.empty_like(q)
    cache.attend_packed(other, out, [new])       # leaves its partial results in the work buffer
    launches = cache.kernel_launches()
    cache.attend_packed(q, out, [new])
    assert cache.kernel_launches() - launches == 2 or held < 9000
    check_edges(cache, q, out, [new])
    if first:
        cache.selftest_timeout(1000)
    monkeypatch.setenv("HIKV_SELFTEST_SITE", "9")
    cache.selftest_timeout(1000)
    out.fill_(7.0)
    cache.attend_packed(q, out, [new])
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())
    with pytest.raises(hk.HikvError) as ei:
        cache.device_status()
    assert ei.value.status == hk.HIKV_ERR_TIMEOUT
    assert ("self-test" if first else "packed attention") in str(ei.value)
    cache.attend_packed(q, out, [new])
    check_edges(cache, q, out, [new])
    cache.device_status()


# ---------------------------------------------------------------------------
# broadcast rows
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_broadcast_k_and_v_enter_and_a_broadcast_q_is_refused(hk, dtype, d):
    gen = gen_of(161)
    t = 70
    cache = make(hk, 1, 8, 2, d, dtype, 200)
    k, v = rnd(gen, t, 1, d, dtype=dtype), rnd(gen, 1, 1, d, dtype=dtype)
    cache.append_packed(k.expand(t, 2, d), v.expand(t, 2, d), [t])
    for g in range(2):
        kc, vc, _ = slots(cache, g)
        assert torch.equal(kc, k[:, 0]) and torch.equal(vc, v[:, 0].expand(t, d))
    q = rnd(gen, t, 1, d, dtype=dtype)
    out = torch.zeros(t, 8, d, device=DEV, dtype=DT[dtype])
    launches = cache.kernel_launches()
    for bad in (q.expand(t, 8, d), q[:1].expand(t, 8, d)):
        with pytest.raises(hk.HikvError, match="q has rows that overlap") as ei:
            cache.attend_packed(bad, out, [t])
        assert ei.value.status == hk.HIKV_ERR_INVALID_ARG
    assert cache.kernel_launches() == launches and not bool(out.any())
    whole = q.expand(t, 8, d).contiguous()
    cache.attend_packed(whole, out, [t])
    check_edges(cache, whole, out, [t])
    cache.device_status()


# ---------------------------------------------------------------------------
# memory
# ---------------------------------------------------------------------------
def test_large_caches_pay_no_memory_for_packed_attention(hk):
    """Where the decode steps' logits buffer (67 MB) holds the partial results
    of split keys (61 MB on 152 SMs), they get no memory of their own."""
    units, cap, G, d, page = 64, 1 << 16, 4, 128, 64
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    make(hk, 1, 8, 2, d, "bf16", 256).close()      # what the first cache of a process loads
    before = torch.cuda.mem_get_info()[0]
    cache = make(hk, 8, 32, 8, d, "bf16", cap, page_tokens=page)
    used = before - torch.cuda.mem_get_info()[0]
    slots = units * cap
    known = slots * (4 * d + 4 * G + 8) + slots // page * 8 + units * (cap // 1024) * 32 * G * 8
    # (buffers are rounded up to 2 MB, some ten of them large)
    assert used < known + (40 << 20), (used - known) / 2 ** 20
    # and they serve both, in turn
    gen = gen_of(171)
    cache.append_packed(rnd(gen, 8 * 3000, 8, d), rnd(gen, 8 * 3000, 8, d), [3000] * 8)
    q, q1 = rnd(gen, 8 * 5, 32, d), rnd(gen, 1, 8, 32, d)
    out, one, other = torch.empty_like(q), torch.empty_like(q1), torch.empty_like(q1)
    launches = cache.kernel_launches()
    cache.attend_packed(q, out, [5] * 8)
    assert cache.kernel_launches() == launches + 2
    cache.decode_step(q1, one)
    for _ in range(10):
        again = torch.empty_like(q)
        cache.decode_step(q1, other)
        cache.attend_packed(q, again, [5] * 8)
        assert torch.equal(again, out) and torch.equal(other, one)
    check_edges(cache, q, out, [5] * 8)
    cache.device_status()
    cache.close()
