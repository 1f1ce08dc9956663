"""What is measured of the packed-prompt operators: appending ragged batches
of tokens to the paged cache with the rotary position rotation on the way,
and causal grouped-query attention of those tokens over the paged cache.

Every case is a dict of plain values.  Sequence lengths are comma-separated
texts: "new" holds the tokens each sequence adds, "held" those it already has
in the cache (for attention the new tokens are in the cache as well, as they
are in a model's layer after the append).
"""
import math

import torch

own = False

PAGE = 64
SINK = 4


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _case(op, new, held=None, hq=32, hkv=8, d=128, dtype="bf16", **kw):
    c = {"op": op, "new": ",".join(map(str, new)), "held": ",".join(map(str, held or [0] * len(new))),
         "hq": hq, "hkv": hkv, "d": d, "dtype": dtype}
    c.update(kw)
    return c


def listed():
    ragged = [1, 17, 333, 1025, 2047, 4000, 0, 640]
    return [
        # a decode step of 64 sequences at positions of their own: one token each,
        # where the call's latency is all there is
        dict(_case("append", [1] * 64, [97 + 13 * i for i in range(64)], rot=128, interleaved=False),
             name="append-step-64-sequences"),
        # a batch of prompts of mixed lengths as a scheduler packs them, an
        # idle sequence among them (Llama-3-8B's heads)
        dict(_case("append", ragged, rot=128, interleaved=False), name="append-ragged-prompts"),
        # a large prefill of four 8K prompts with Llama-3-70B's heads
        dict(_case("append", [8192] * 4, hq=64, rot=128, interleaved=False), name="append-4x8k-70b-heads"),
        # fp32 cache, rotation of half of a row's elements, interleaved pairs
        dict(_case("append", [255, 1, 130, 77, 1001], [5, 0, 300, 64, 31], hq=4, hkv=2, d=64, dtype="f32",
                   rot=32, interleaved=True), name="append-fp32-interleaved"),
        # short prompts of a small model: latency
        dict(_case("attend", [16, 9, 31, 2], hq=4, hkv=2, d=64), name="attend-short-prompts"),
        # one whole 8K prompt, a layer of Llama-3-8B
        dict(_case("attend", [8192]), name="attend-8k-prompt"),
        # the ragged batch of the append case
        dict(_case("attend", ragged), name="attend-ragged-prompts"),
        # a long prompt with Llama-3-70B's groups of eight: arithmetic-bound
        dict(_case("attend", [16384], hq=64), name="attend-16k-prompt-70b-heads"),
        # two prompts' next chunks of 512 tokens over 16K already cached
        dict(_case("attend", [512, 512], [15872, 13007]), name="attend-chunk-over-16k"),
        # checking four drafted tokens and the last accepted one of eight
        # sequences over long contexts: bound by reading the cache
        dict(_case("attend", [5] * 8, [32763, 8187, 16384, 30001, 24571, 12345, 32000, 20480]),
             name="attend-5-drafted-tokens"),
        # a 33-token turn over a cache cut to budgets that differ by head
        dict(_case("attend", [33] * 16, [2100] * 16, cut=True), name="attend-turn-over-cut-heads"),
        # fp32 cache with small heads
        dict(_case("attend", [256, 100, 511, 1], hq=4, hkv=2, d=64, dtype="f32"), name="attend-fp32-prompts"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8, 8])
    hq = hkv * rng.choice([1, 2, 4, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if rng.random() < 0.35:
        b = _log_int(rng, 1, 64)
        total = _log_int(rng, b, 32768)
        new = [max(0, _log_int(rng, 1, max(1, 2 * total // b)) - rng.choice([0, 1])) for _ in range(b)]
        while sum(new) > 32768:
            new = [n // 2 for n in new]
        if sum(new) == 0:
            new[0] = 1
        held = [rng.choice([0, _log_int(rng, 1, 32768 // b)]) for _ in range(b)]
        c = _case("append", new, held, hq=hq, hkv=hkv, d=d, dtype=dtype,
                  rot=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.3)
        return c
    kind = rng.choice(["prompts", "prompts", "chunk", "verify", "cut"])
    if kind == "prompts":
        b = _log_int(rng, 1, 16)
        new = [_log_int(rng, 1, 8192) for _ in range(b)]
        held = [0] * b
    elif kind == "chunk":
        b = _log_int(rng, 1, 4)
        new = [_log_int(rng, 64, 2048) for _ in range(b)]
        held = [_log_int(rng, 64, 24576) for _ in range(b)]
    elif kind == "verify":
        b = _log_int(rng, 1, 16)
        new = [rng.randint(1, 16) for _ in range(b)]
        held = [_log_int(rng, 64, 32768) for _ in range(b)]
    else:
        b = _log_int(rng, 1, 16)
        new = [rng.randint(1, 200) for _ in range(b)]
        held = [_log_int(rng, 256, 4096)] * b
    c = _case("attend", new, held, hq=hq, hkv=hkv, d=d, dtype=dtype)
    if kind == "cut":
        c["cut"] = True
    most = work(_case("attend", [16384], hq=64))["flops"] / (16 if dtype == "f32" else 1)
    while work(c)["flops"] > most:
        new = [max(1, n // 2) for n in new]
        c["new"] = ",".join(map(str, new))
    return c


def _ints(text):
    return [int(x) for x in text.split(",")]


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _budgets(case):
    """Tokens each KV head keeps of the held ones: spread from 64 to 2048."""
    if not case.get("cut"):
        return None
    n = case["hkv"]
    return [max(64, int(2048 * ((i * 5 + 3) % n + 1) / n) - 7 * i) for i in range(n)]


def work(case):
    new, held = _ints(case["new"]), _ints(case["held"])
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    e = 2 if case["dtype"] == "bf16" else 4
    total = sum(new)
    if case["op"] == "append":
        # q, k, v in and out, a table row (cos and sin) a distinct position
        spans = sorted((h, h + n) for h, n in zip(held, new) if n)
        rows, end = 0, 0
        for lo, hi in spans:
            rows += max(0, hi - max(lo, end))
            end = max(end, hi)
        return {"bytes": 2 * total * (hq + 2 * hkv) * d * e + rows * case["rot"] * 4,
                "flops": total * (hq + hkv) * case["rot"] * 3}
    cut = _budgets(case)
    pairs, slots = 0, 0
    for n, h in zip(new, held):
        if n == 0:
            continue
        for g in range(hkv):
            kept = min(h, cut[g]) if cut else h
            pairs += n * kept + n * (n + 1) // 2
            slots += kept + n
    return {"bytes": (2 * total * hq + 2 * slots) * d * e, "flops": 4 * d * pairs * (hq // hkv)}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(0x5EED + seed)
    return g


def _randn(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _tables(positions, rot):
    """cos and sin of position x frequency, the angles in 64 bits."""
    inv = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    ang = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * inv
    return ang.cos().float(), ang.sin().float()


def _append_inputs(case, seed):
    new, held = _ints(case["new"]), _ints(case["held"])
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g = _gen(seed)
    qkv = _randn(g, sum(new), (hq + 2 * hkv) * d, dtype=_dtype(case))
    q, k, v = qkv.split([hq * d, hkv * d, hkv * d], dim=1)   # slices of one projection's output
    cos, sin = _tables(max(h + n for h, n in zip(held, new)), case["rot"])
    return dict(new=new, held=held, q=q.unflatten(1, (hq, d)), k=k.unflatten(1, (hkv, d)),
                v=v.unflatten(1, (hkv, d)), cos=cos, sin=sin)


def _attend_inputs(case, seed):
    """q of the new tokens; per sequence the keys and values its heads hold,
    [hkv][longest][d] with every head's own length.  The first tokens of a
    sequence draw attention from every query, as in trained models, and one
    token in twenty has larger keys."""
    new, held = _ints(case["new"]), _ints(case["held"])
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    dt = _dtype(case)
    g = _gen(seed)
    lean = torch.randn(hkv, 1, d, generator=g, device="cuda")
    lean = lean / lean.norm(dim=-1, keepdim=True) * 4.0
    q = torch.randn(sum(new), hq, d, generator=g, device="cuda")
    q = (q + lean.repeat_interleave(hq // hkv, 0).squeeze(1)).to(dt)
    cut = _budgets(case)
    window = 32
    seqs = []
    for n, h in zip(new, held):
        k = torch.randn(hkv, h + n, d, generator=g, device="cuda")
        k = k * (1.0 + 2.0 * (torch.rand(hkv, h + n, 1, generator=g, device="cuda") < 0.05))
        k[:, :SINK] += 2.0 * lean
        k = k.to(dt)
        v = _randn(g, hkv, h + n, d, dtype=dt)
        lens = [h + n] * hkv
        full = (k, v)
        if cut:
            # a cut of tokens that no query has scored keeps the earliest ones
            # and the recent window
            lens = [min(h, c) + n for c in cut]
            kk, vv = torch.zeros_like(k)[:, :max(lens)], torch.zeros_like(v)[:, :max(lens)]
            for i, c in enumerate(cut):
                keep = torch.arange(h + n, device="cuda")
                if h > c:
                    keep = torch.cat([keep[:c - window], keep[h - window:]])
                kk[i, :lens[i]], vv[i, :lens[i]] = k[i, keep], v[i, keep]
            k, v = kk, vv
        seqs.append(dict(k=k, v=v, lens=lens, full=full))
    return dict(new=new, held=held, q=q, seqs=seqs, window=window)


def prepare(case, seed):
    new, held = _ints(case["new"]), _ints(case["held"])
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    dt = _dtype(case)
    batch = len(new)
    need = max(h + n for h, n in zip(held, new))
    cap = -(-max(1, need) // PAGE) * PAGE
    if own:
        import importance_aware_kv_gb300 as hk
        cut = _budgets(case)
        cfg = dict(num_layers=1, batch=batch, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, dtype=case["dtype"],
                   num_sink=SINK, recent_window=32, max_tokens=cap, page_tokens=PAGE)
    if case["op"] == "append":
        s = _append_inputs(case, seed)
        s.update(case=case, q_out=torch.empty(sum(new), hq, d, device="cuda", dtype=dt))
        if own:
            cache = hk.Cache(hk.CacheConfig(budgets=[max(36, cap)] * hkv, **cfg))
            s["view"] = cache.device_view()
            s["view"]["pages"].zero_()
            # what the sequences held, then room that the measured call fills
            for lens in (held, new):
                z = torch.zeros(sum(lens), hkv, d, device="cuda", dtype=dt)
                cache.append_packed(z, z, lens)
            s["rope"] = hk.Rope(s["cos"], s["sin"], interleaved=case["interleaved"])
            s["cache"] = cache
        else:
            units, pages = batch * hkv, cap // PAGE
            s["pages"] = torch.zeros(units * pages, 2, PAGE, d, device="cuda", dtype=dt)
            # where every new token's rows go: its page and its row in the page
            seq = torch.repeat_interleave(torch.arange(batch), torch.tensor(new))
            pos = torch.cat([torch.arange(h, h + n) for h, n in zip(held, new)])
            unit = seq[:, None] * hkv + torch.arange(hkv)
            s["page"] = (unit * pages + (pos // PAGE)[:, None]).cuda()
            s["row"] = (pos % PAGE)[:, None].expand(-1, hkv).cuda()
            s["pos"] = pos.cuda()
            s["lengths"] = torch.repeat_interleave(torch.tensor([h + n for h, n in zip(held, new)]), hkv).int().cuda()
        return s
    s = _attend_inputs(case, seed)
    s["case"] = case
    s["out"] = torch.empty(sum(new), hq, d, device="cuda", dtype=dt)
    if own:
        cache = hk.Cache(hk.CacheConfig(budgets=cut or [max(36, cap)] * hkv, **cfg))
        for part in (0, 1):
            lens = held if part == 0 else new
            if sum(lens) == 0:
                continue
            rows = [[t.transpose(0, 1)[:h] if part == 0 else t.transpose(0, 1)[h:] for t in q["full"]]
                    for q, h in zip(s["seqs"], held)]
            cache.append_packed(torch.cat([r[0] for r in rows]), torch.cat([r[1] for r in rows]), lens)
            if part == 0 and cut:
                cache.evict()
        s["cache"] = cache
        s["seqs"] = None
    else:
        for q in s["seqs"]:
            q["full"] = None
            q["n"] = torch.tensor(q["lens"], device="cuda")
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def _rotate(x, cos, sin, interleaved):
    """x [tokens][heads][d] in 32 bits, cos and sin [tokens][rot / 2]."""
    half = cos.shape[1]
    c, s = cos[:, None], sin[:, None]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * c - b * s, b * c + a * s
    return y


def _attend(q, k, v, lens, scale):
    """q [T][hq][d] of the newest T positions over k, v [hkv][n][d], of which
    head g holds lens[g]."""
    t, hq, d = q.shape
    hkv, n, _ = k.shape
    qg = q.view(t, hkv, hq // hkv, d).permute(1, 2, 0, 3)
    out = torch.empty_like(qg)
    kt = k.transpose(1, 2)[:, None]
    step = max(1, (1 << 29) // (hq * n))
    col = torch.arange(n, device=q.device)
    for i in range(0, t, step):
        qi = qg[:, :, i:i + step]
        s = torch.matmul(qi, kt) * scale
        last = lens[:, None] - t + torch.arange(i, i + qi.shape[2], device=q.device)
        s = torch.where((col <= last[:, :, None])[:, None], s, float("-inf"))
        e = torch.exp(s - s.amax(-1, keepdim=True))
        out[:, :, i:i + step] = torch.matmul(e, v[:, None]) / e.sum(-1, keepdim=True)
    return out.permute(2, 0, 1, 3).reshape(t, hq, d)


def run(state):
    case = state["case"]
    if case["op"] == "append":
        if own:
            # the cache takes the next batch in the place of the last one
            state["cache"].drop(state["new"])
            state["cache"].append_packed(state["k"], state["v"], state["new"], q=state["q"], q_out=state["q_out"],
                                         rope=state["rope"])
            view = state["view"]
            return state["q_out"], view["pages"], view["lengths"]
        cos, sin = state["cos"][state["pos"]], state["sin"][state["pos"]]
        dt = state["q"].dtype
        q_out = _rotate(state["q"].float(), cos, sin, case["interleaved"]).to(dt)
        k = _rotate(state["k"].float(), cos, sin, case["interleaved"]).to(dt)
        state["pages"][state["page"], 0, state["row"]] = k
        state["pages"][state["page"], 1, state["row"]] = state["v"]
        return q_out, state["pages"], state["lengths"]
    if own:
        state["cache"].attend_packed(state["q"], state["out"], state["new"])
        return state["out"]
    r = 0
    for n, s in zip(state["new"], state["seqs"]):
        if n:
            state["out"][r:r + n] = _attend(state["q"][r:r + n].float(), s["k"].float(), s["v"].float(), s["n"],
                                            1.0 / math.sqrt(case["d"])).to(state["out"].dtype)
        r += n
    return state["out"]


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "append":
        s = _append_inputs(case, seed)
        half = case["rot"] // 2
        cap = -(-max(1, max(h + n for h, n in zip(s["held"], s["new"]))) // PAGE) * PAGE
        batch = len(s["new"])
        pages = torch.zeros(batch, hkv, cap // PAGE, 2, PAGE, d, device="cuda", dtype=torch.float64)
        slots = pages.permute(0, 1, 3, 2, 4, 5)   # [batch][hkv][k or v][page][row][d]
        first = torch.arange(half, device="cuda")
        a, b = (2 * first, 2 * first + 1) if case["interleaved"] else (first, first + half)
        # the rotated pair (x_a, x_b) is the complex number (x_a + i x_b) e^(i angle)
        turned, r = {"q": s["q"].double(), "k": s["k"].double()}, 0
        for n, h in zip(s["new"], s["held"]):
            turn = torch.complex(s["cos"][h:h + n].double(), s["sin"][h:h + n].double())[:, None]
            for x in turned.values():
                z = torch.complex(x[r:r + n][..., a], x[r:r + n][..., b]) * turn
                x[r:r + n][..., a], x[r:r + n][..., b] = z.real, z.imag
            r += n
        r = 0
        for i, (n, h) in enumerate(zip(s["new"], s["held"])):
            for j, x in enumerate((turned["k"], s["v"].double())):
                flat = torch.zeros(hkv, cap, d, device="cuda", dtype=torch.float64)
                flat[:, h:h + n] = x[r:r + n].transpose(0, 1)
                slots[i, :, j] = flat.view(hkv, cap // PAGE, PAGE, d)
            r += n
        lengths = torch.tensor([h + n for h, n in zip(s["held"], s["new"]) for _ in range(hkv)], dtype=torch.int32,
                               device="cuda")
        return turned["q"], pages.reshape(-1, 2, PAGE, d), lengths
    if work(case)["flops"] > 3e12:
        return None
    s = _attend_inputs(case, seed)
    out = torch.empty(sum(s["new"]), hq, d, device="cuda", dtype=torch.float64)
    group = hq // hkv
    r = 0
    for n, seq in zip(s["new"], s["seqs"]):
        for g in range(hkv if n else 0):
            m = seq["lens"][g]
            k, v = seq["k"][g, :m].double(), seq["v"][g, :m].double()
            step = max(1, (1 << 27) // (m * group))
            for i in range(0, n, step):
                rows = min(step, n - i)
                x = s["q"][r + i:r + i + rows, g * group:(g + 1) * group].double().reshape(rows * group, d)
                z = x @ k.T / math.sqrt(d)
                seen = m - n + i + torch.arange(rows, device="cuda").repeat_interleave(group)
                z.masked_fill_(torch.arange(m, device="cuda")[None] > seen[:, None], float("-inf"))
                out[r + i:r + i + rows, g * group:(g + 1) * group] = (torch.softmax(z, -1) @ v).view(rows, group, d)
        r += n
    return out
