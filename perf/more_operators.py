"""What is measured of the operators around drafted trees, sliding windows and
copied sequences: attention of trees of drafted tokens over the paged cache,
the append of such trees (rotated by depth) and the acceptance of a path of
each, attention over a sliding window and the first tokens, a window for
every KV head, and copies of whole sequences of the cache.

Every case is a dict of plain values; lists are comma-separated texts.  "new"
holds the tokens (or tree nodes) each sequence adds, "held" those it already
has in the cache; for attention the new tokens are in the cache as well.
"""
import math

import torch

own = False

PAGE = 64
SINK = 4


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _text(xs):
    return ",".join(map(str, xs))


def _case(op, hq=32, hkv=8, d=128, dtype="bf16", **kw):
    c = {"op": op, "hq": hq, "hkv": hkv, "d": d, "dtype": dtype}
    c.update({k: _text(v) if isinstance(v, list) else v for k, v in kw.items()})
    return c


def listed():
    return [
        # a small model's drafts of four sequences: latency
        dict(_case("tree", new=[26] * 4, held=[97 + 13 * i for i in range(4)], deep=5, hq=4, hkv=2, d=64),
             name="tree-26-nodes-small"),
        # 64 drafted nodes of each of eight sequences over long contexts
        # (Llama-3-8B's heads): bound by reading the cache
        dict(_case("tree", new=[64] * 8, held=[32763, 8187, 16384, 30001, 24571, 12345, 32000, 20480], deep=7),
             name="tree-64-nodes-over-32k"),
        # 16 sequences with Llama-3-70B's heads, trees that end inside a word of
        # the mask and a sequence without a tree
        dict(_case("tree", new=[60, 61, 33, 0] * 4, held=[2100 - 37 * i for i in range(16)], deep=6, hq=64),
             name="tree-60-nodes-70b-heads"),
        # fp32 cache: ragged trees, one of a single node, one without a context
        dict(_case("tree", new=[40, 1, 63, 17], held=[300, 1025, 0, 64], deep=4, hq=4, hkv=2, d=64, dtype="f32"),
             name="tree-fp32"),
        # one layer's cache work of a verified step of 64 sequences: the trees'
        # masks and depths, 32 nodes in, four of them accepted
        dict(_case("step", new=[32] * 64, held=[97 + 13 * i for i in range(64)], deep=4, rot=128, interleaved=False),
             name="step-64-trees"),
        # the same in fp32 with interleaved pairs and half of a row turned
        dict(_case("step", new=[25, 1, 60, 7, 0], held=[5, 0, 300, 64, 31], deep=3, hq=4, hkv=2, d=64, dtype="f32",
                   rot=32, interleaved=True), name="step-fp32-interleaved"),
        # one 16K prompt in windows of 1024 (a layer of Llama-3-8B)
        dict(_case("window", new=[16384], held=[0], windows=[1024] * 8, sink=SINK), name="window-16k-prompt"),
        # prompts of a model with retrieval heads that see everything and
        # streaming heads that see the first four and the newest 252 tokens
        dict(_case("window", new=[4000, 1, 333, 2047, 640], held=[0, 700, 0, 64, 0],
                   windows=[0, 252, 252, 252, 0, 252, 252, 252], sink=SINK), name="window-retrieval-and-streaming-heads"),
        # a decode step of 64 sequences over 8K contexts, windows of 2044
        dict(_case("window", new=[1] * 64, held=[8191 - 61 * i for i in range(64)], windows=[2044] * 8, sink=SINK),
             name="window-step-64-sequences"),
        # fp32 cache, a window shorter than a page
        dict(_case("window", new=[256, 100, 511, 1], held=[0, 31, 0, 200], windows=[33, 100], sink=1, hq=4, hkv=2, d=64,
                   dtype="f32"), name="window-fp32-prompts"),
        # eight samples of one 8K prompt, two layers of Llama-3-8B
        dict(_case("fork", held=[8187] + [0] * 7, src=[0] * 8, same=[0] * 8, layers=2), name="fork-8k-prompt-to-8"),
        # a step of four beam searches of four beams, eight layers: the beams
        # of a search share its prompt, a few go on from another beam
        dict(_case("fork", held=[613, 613, 613, 613, 541, 541, 541, 541, 130, 130, 130, 130, 700, 700, 700, 700],
                   src=[0, 0, 2, 0, 4, 5, 4, 5, 8, 9, 10, 11, 12, 12, 12, 12],
                   same=[512] * 4 + [500] * 4 + [64] * 4 + [640] * 4, layers=8), name="fork-beams"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8, 8])
    hq = hkv * rng.choice([1, 2, 4, 4, 8])
    shape = dict(hq=hq, hkv=hkv, d=d, dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]))
    op = rng.choice(["tree", "tree", "step", "window", "window", "fork"])
    if op in ("tree", "step"):
        b = _log_int(rng, 1, 16 if op == "tree" else 64)
        most = 32768 if op == "tree" else max(64, 65536 // b)
        new = [_log_int(rng, 1, 96) - (rng.random() < 0.1) for _ in range(b)]
        if sum(new) == 0:
            new[0] = 1
        held = [rng.choice([0, _log_int(rng, 1, most), _log_int(rng, 64, most)]) for _ in range(b)]
        c = _case(op, new=new, held=held, deep=rng.randint(1, 9), **shape)
        if op == "step":
            c.update(rot=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.3)
        return c
    if op == "window":
        kind = rng.choice(["prompts", "chunk", "step"])
        b = _log_int(rng, 1, {"prompts": 8, "chunk": 4, "step": 64}[kind])
        if kind == "prompts":
            new, held = [_log_int(rng, 1, 16384) for _ in range(b)], [0] * b
        elif kind == "chunk":
            new, held = [_log_int(rng, 8, 2048) for _ in range(b)], [_log_int(rng, 64, 24576) for _ in range(b)]
        else:
            new, held = [rng.randint(1, 3) for _ in range(b)], [_log_int(rng, 64, 16384) for _ in range(b)]
        w = _log_int(rng, 16, 4096)
        windows = [rng.choice([w, w, 0, max(1, w // 3)]) for _ in range(hkv)] if rng.random() < 0.3 else [w] * hkv
        return _case(op, new=new, held=held, windows=windows, sink=rng.choice([0, 1, 4, 4, 70]), **shape)
    b = rng.randint(2, 24)
    layers = rng.randint(1, 8)
    held = [_log_int(rng, 1, max(64, 8192 * 8 * 128 * 4 // (b * layers * hkv * d))) for _ in range(b)]
    roots = [i for i in range(b) if i == 0 or rng.random() < 0.4]
    src = [i if i in roots else rng.choice(roots + [i]) for i in range(b)]
    src = [s if src[s] == s else i for i, s in enumerate(src)]
    if all(s == i for i, s in enumerate(src)):
        src[-1] = 0
    same = [rng.choice([0, min(held[i], held[s]) // 2]) for i, s in enumerate(src)]
    return _case(op, held=held, src=src, same=same, layers=layers, **shape)


def draw(rng):
    """One more case, no dearer than the dearest listed one of its operator."""
    c = _draw(rng)
    of = [x for x in listed() if x["op"] == c["op"]]
    dearest = {k: max(work(x)[k] for x in of) for k in ("bytes", "flops")}
    if c["dtype"] == "f32":
        dearest["flops"] /= 16
    while any(work(c)[k] > dearest[k] for k in dearest):
        for name in ("new", "held", "same"):
            if name in c and (name != "new" or c["op"] == "window"):
                c[name] = _text([(x + 1) // 2 if name != "same" else x // 2 for x in _ints(c[name])])
        if c["op"] in ("tree", "step") and max(_ints(c["held"])) <= 1:
            c["new"] = _text([(x + 1) // 2 for x in _ints(c["new"])])
    return c


def _ints(text):
    return [int(x) for x in text.split(",")]


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _visible(lim, window, sink):
    """Tokens that a query at position lim sees."""
    return lim + 1 if window == 0 else min(lim + 1, window + min(sink, max(0, lim + 1 - window)))


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    e = 2 if case["dtype"] == "bf16" else 4
    held = _ints(case["held"])
    if case["op"] == "fork":
        # every source's rows from the first slot that a copy lacks on, read
        # once; every copy written; 8 bytes a slot of scores and positions
        src, same = _ints(case["src"]), _ints(case["same"])
        slots = meta = 0
        for s in set(src):
            copies = [b for b in range(len(src)) if src[b] == s and b != s]
            if copies:
                slots += held[s] - min(same[b] for b in copies) + sum(held[s] - same[b] for b in copies)
                meta += held[s] * (1 + len(copies))
        return {"bytes": (slots * 2 * d * e + meta * 8) * hkv * case["layers"], "flops": 0}
    new = _ints(case["new"])
    total = sum(new)
    if case["op"] == "step":
        spans = sorted((h, h + min(n, case["deep"])) for h, n in zip(held, new) if n)
        rows, end = 0, 0
        for lo, hi in spans:
            rows += max(0, hi - max(lo, end))
            end = max(end, hi)
        accepted = sum(min(n, case["deep"]) for n in new)
        return {"bytes": (2 * total * (hq + 2 * hkv) + 2 * accepted * 2 * hkv) * d * e + rows * case["rot"] * 4,
                "flops": total * (hq + hkv) * case["rot"] * 3}
    pairs, slots = 0, 0
    for n, h in zip(new, held):
        if n == 0:
            continue
        if case["op"] == "tree":
            pairs += hkv * n * (h + (case["deep"] + 1) / 2)
            slots += hkv * (h + n)
        else:
            for w in _ints(case["windows"]):
                pairs += sum(_visible(h + i, w, case["sink"]) for i in range(n))
                slots += h + n if w == 0 else min(h + n, n + w - 1 + case["sink"])
    return {"bytes": (2 * total * hq + 2 * slots) * d * e, "flops": int(4 * d * pairs * (hq // hkv))}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(0x7EE5 + seed)
    return g


def _randn(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _trees(case, seed):
    """Parents of every node (-1: the sequence's last token) and the accepted
    path of each tree: min(nodes, deep) nodes, the first of them node 0.  The
    other nodes hang on random earlier ones."""
    g = _gen(seed, "cpu")
    parents, paths = [], []
    for n in _ints(case["new"]):
        deep = min(n, case["deep"])
        if n == 0:
            paths.append([])
            continue
        spine = [0] + sorted((torch.randperm(n - 1, generator=g)[:deep - 1] + 1).tolist())
        u = torch.rand(n, generator=g).tolist()
        parent = [min(i - 1, int(u[i] * (i + 1)) - 1) for i in range(n)]
        parent[0] = -1
        for a, b in zip(spine, spine[1:]):
            parent[b] = a
        parents += parent
        paths.append(spine)
    return parents, paths


def _sees(parent):
    """[n][n]: whether node i's path to the root passes node j."""
    m = torch.zeros(len(parent), len(parent), dtype=torch.bool)
    for i, p in enumerate(parent):
        if p >= 0:
            m[i] = m[p]
        m[i, i] = True
    return m


def _tables(positions, rot):
    """cos and sin of position x frequency, the angles in 64 bits."""
    inv = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    ang = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * inv
    return ang.cos().float(), ang.sin().float()


def _cap(new, held):
    return -(-max(1, max(h + n for h, n in zip(held, new))) // PAGE) * PAGE


def _step_inputs(case, seed):
    new, held = _ints(case["new"]), _ints(case["held"])
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g = _gen(seed)
    qkv = _randn(g, sum(new), (hq + 2 * hkv) * d, dtype=_dtype(case))
    q, k, v = qkv.split([hq * d, hkv * d, hkv * d], dim=1)   # slices of one projection's output
    cos, sin = _tables(max(h + n for h, n in zip(held, new)), case["rot"])
    parents, paths = _trees(case, seed)
    return dict(new=new, held=held, q=q.unflatten(1, (hq, d)), k=k.unflatten(1, (hkv, d)), v=v.unflatten(1, (hkv, d)),
                cos=cos, sin=sin, parents=parents, paths=paths)


def _attend_inputs(case, seed):
    """q of the new tokens; per sequence the keys and values its heads hold,
    [hkv][tokens][d].  The first tokens of a sequence draw attention from
    every query, as in trained models, and one token in twenty has larger
    keys."""
    new, held = _ints(case["new"]), _ints(case["held"])
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    dt = _dtype(case)
    g = _gen(seed)
    lean = torch.randn(hkv, 1, d, generator=g, device="cuda")
    lean = lean / lean.norm(dim=-1, keepdim=True) * 4.0
    q = torch.randn(sum(new), hq, d, generator=g, device="cuda")
    q = (q + lean.repeat_interleave(hq // hkv, 0).squeeze(1)).to(dt)
    seqs = []
    for n, h in zip(new, held):
        k = torch.randn(hkv, h + n, d, generator=g, device="cuda")
        k = k * (1.0 + 2.0 * (torch.rand(hkv, h + n, 1, generator=g, device="cuda") < 0.05))
        k[:, :SINK] += 2.0 * lean
        seqs.append(dict(k=k.to(dt), v=_randn(g, hkv, h + n, d, dtype=dt)))
    return dict(new=new, held=held, q=q, seqs=seqs)


def _fork_inputs(case, seed):
    """Pages [units][pages][K, V][row][d], scores and positions [units][slots]
    of every (layer, sequence, KV head)."""
    held, src, same = _ints(case["held"]), _ints(case["src"]), _ints(case["same"])
    layers, hkv, d = case["layers"], case["hkv"], case["d"]
    batch, cap = len(held), -(-max(held) // PAGE) * PAGE
    g = _gen(seed)
    pages = _randn(g, layers, batch, hkv, cap // PAGE, 2, PAGE, d, dtype=_dtype(case))
    scores = torch.rand(layers, batch, hkv, cap, generator=g, device="cuda")
    positions = torch.full((layers, batch, hkv, cap), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(cap, dtype=torch.int32, device="cuda")
    for b, (h, s, m) in enumerate(zip(held, src, same)):
        positions[:, b, :, :h] = at[:h]
        if m:   # a beam's tokens up to here are those of the beam it goes on from
            old, row = (pages[:, x].transpose(2, 3).reshape(layers, hkv, 2, cap, d) for x in (s, b))
            row[:, :, :, :m] = old[:, :, :, :m]
            pages[:, b] = row.view(layers, hkv, 2, cap // PAGE, PAGE, d).transpose(2, 3)
    return dict(held=held, src=src, same=same, pages=pages, scores=scores, positions=positions)


def prepare(case, seed):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    dt = _dtype(case)
    held = _ints(case["held"])
    batch = len(held)
    new = _ints(case["new"]) if "new" in case else [0] * batch
    cap = _cap(new, held)
    if own:
        import importance_aware_kv_gb300 as hk
        layers = case.get("layers", 1)
        cache = hk.Cache(hk.CacheConfig(
            num_layers=layers, batch=batch, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, dtype=case["dtype"],
            num_sink=SINK, recent_window=32, max_tokens=cap, page_tokens=PAGE, budgets=[max(36, cap)] * (layers * hkv)))
    if case["op"] == "fork":
        s = _fork_inputs(case, seed)
        s["case"] = case
        units = case["layers"] * batch * hkv
        if own:
            z = torch.zeros(1, 1, d, device="cuda", dtype=dt).expand(sum(held), hkv, d)
            for layer in range(case["layers"]):
                cache.append_packed(z, z, held, layer=layer)
            view = cache.device_view()
            view["pages"].copy_(s["pages"].view(units * cap // PAGE, 2, PAGE, d))
            view["importance"].copy_(s["scores"].view(units, cap))
            s.update(cache=cache, view=view, pages=None, scores=None, positions=None)
        else:
            s["lengths"] = torch.tensor(held, dtype=torch.int32, device="cuda")[None, :, None].expand(
                case["layers"], batch, hkv).contiguous()
        return s
    if case["op"] == "step":
        s = _step_inputs(case, seed)
        s.update(case=case, q_out=torch.empty(sum(new), hq, d, device="cuda", dtype=dt),
                 parent=torch.tensor(s["parents"], dtype=torch.int32, device="cuda"),
                 taken=[len(p) for p in s["paths"]])
        if own:
            s["view"] = cache.device_view()
            s["view"]["pages"].zero_()
            # what the sequences held, then the last step's accepted tokens
            for lens in (held, s["taken"]):
                z = torch.zeros(sum(lens), hkv, d, device="cuda", dtype=dt)
                cache.append_packed(z, z, lens)
            s.update(rope=hk.Rope(s["cos"], s["sin"], interleaved=case["interleaved"]), cache=cache)
        else:
            units, pages = batch * hkv, cap // PAGE
            s["pages"] = torch.zeros(units * pages, 2, PAGE, d, device="cuda", dtype=dt)
            seq = torch.repeat_interleave(torch.arange(batch), torch.tensor(new))
            slot = torch.cat([torch.arange(h, h + n) for h, n in zip(held, new)])
            unit = seq[:, None] * hkv + torch.arange(hkv)
            s["page"] = (unit * pages + (slot // PAGE)[:, None]).cuda()
            s["row"] = (slot % PAGE)[:, None].expand(-1, hkv).cuda()
            s["seq"], s["nth"] = seq.cuda(), torch.cat([torch.arange(n) for n in new]).cuda()
            s["start"] = torch.tensor(held)[seq].cuda()
            # where the accepted nodes' rows are and go
            first = [sum(new[:b]) for b in range(batch)]
            at = [(first[b] + i, first[b] + j) for b, p in enumerate(s["paths"]) for j, i in enumerate(p)]
            s["from"], s["to"] = (torch.tensor(x, device="cuda") for x in zip(*at))
            s["lengths"] = torch.tensor([h + t for h, t in zip(held, s["taken"])], dtype=torch.int32,
                                        device="cuda").repeat_interleave(hkv)
        return s
    s = _attend_inputs(case, seed)
    s["case"] = case
    s["out"] = torch.empty(sum(new), hq, d, device="cuda", dtype=dt)
    if case["op"] == "tree":
        parents, _ = _trees(case, seed)
    else:
        s["windows"] = _ints(case["windows"])
    if own:
        for part in (0, 1):
            lens = held if part == 0 else new
            if sum(lens) == 0:
                continue
            rows = [[x.transpose(0, 1)[:h] if part == 0 else x.transpose(0, 1)[h:] for x in (q["k"], q["v"])]
                    for q, h in zip(s["seqs"], held)]
            cache.append_packed(torch.cat([r[0] for r in rows]), torch.cat([r[1] for r in rows]), lens)
        s.update(cache=cache, seqs=None)
        if case["op"] == "tree":
            s["tree"] = cache.tree(torch.tensor(parents, dtype=torch.int32, device="cuda"), new)
    elif case["op"] == "tree":
        r = 0
        for n, q in zip(new, s["seqs"]):
            q["sees"] = _sees(parents[r:r + n]).cuda()
            r += n
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


def _masked(q, k, v, seen, scale):
    """q [t][heads][d] over k, v [hkv][n][d]; seen [t][n] or [hkv][t][n]."""
    t, hq, d = q.shape
    hkv = k.shape[0]
    qg = q.view(t, hkv, hq // hkv, d).permute(1, 2, 0, 3)
    s = torch.matmul(qg, k.transpose(1, 2)[:, None]) * scale
    s = torch.where(seen[:, None] if seen.dim() == 3 else seen, s, float("-inf"))
    e = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul(e, v[:, None]) / e.sum(-1, keepdim=True)
    return o.permute(2, 0, 1, 3).reshape(t, hq, d)


def _attend_window(q, k, v, windows, sink, scale, out):
    """Chunks of queries over the keys that any of them sees."""
    t, hq, d = q.shape
    hkv, n, _ = k.shape
    group = hq // hkv
    kinds = sorted(set(windows))
    for w in kinds:
        heads = [g for g in range(hkv) if windows[g] == w]
        qh = [h for g in heads for h in range(g * group, (g + 1) * group)]
        all_of = len(kinds) == 1
        qw, kw, vw = (q, k, v) if all_of else (q[:, qh], k[heads], v[heads])
        step = max(64, min(1024, (1 << 28) // (len(qh) * (n if w == 0 else min(n, w + 1024)))))
        for i in range(0, t, step):
            qi = qw[i:i + step].float()
            m = qi.shape[0]
            last = n - t + i + torch.arange(m, device=q.device)[:, None]
            end = n - t + i + m
            lo = 0 if w == 0 else max(0, n - t + i - w + 1)
            col = torch.arange(lo, end, device=q.device)
            if lo > 0 and sink > 0:
                first = torch.arange(min(sink, lo), device=q.device)
                ks = torch.cat([kw[:, :min(sink, lo)], kw[:, lo:end]], 1).float()
                vs = torch.cat([vw[:, :min(sink, lo)], vw[:, lo:end]], 1).float()
                col = torch.cat([first, col])
            else:
                ks, vs = kw[:, lo:end].float(), vw[:, lo:end].float()
            seen = col <= last
            if w:
                seen = seen & ((col > last - w) | (col < sink))
            o = _masked(qi, ks, vs, seen, scale).to(out.dtype)
            if all_of:
                out[i:i + m] = o
            else:
                out[i:i + m, qh] = o


def _plan(parent, seq, nth, batch, words):
    """Depth of every node and the bits of the nodes on its path to the root,
    its own among them, by doubling the steps taken."""
    total, most = parent.shape[0], 32 * words
    root = parent < 0
    up = torch.where(root, 0, parent.long() - nth)   # steps back to the parent's row
    row = torch.arange(total, device=parent.device)
    up = row + up
    depth = (~root).to(torch.int32)
    sees = torch.zeros(total + 1, most, dtype=torch.bool, device=parent.device)   # the last row: past a root
    sees[row, nth] = True
    up = torch.cat([torch.where(root, total, up), torch.tensor([total], device=parent.device)])
    depth = torch.cat([depth, depth.new_zeros(1)])
    for _ in range(max(1, (most - 1).bit_length())):
        sees = sees | sees[up]
        depth = depth + depth[up]
        up = up[up]
    bits = sees[:total].view(total, words, 32).to(torch.int64) << torch.arange(32, device=parent.device)
    bits = bits.sum(-1)
    return torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32), depth[:total]


def run(state):
    case = state["case"]
    if case["op"] == "fork":
        if own:
            state["cache"].fork(state["src"], same=state["same"])
            view = state["view"]
            return view["pages"], view["importance"], view["positions"], view["lengths"]
        pages, cap = state["pages"], state["scores"].shape[-1]
        for b, (s, m) in enumerate(zip(state["src"], state["same"])):
            if s == b:
                continue
            n = state["held"][s]
            lo, hi = m // PAGE, n // PAGE
            if m % PAGE and lo < hi:   # the rest of a page
                pages[:, b, :, lo, :, m % PAGE:] = pages[:, s, :, lo, :, m % PAGE:]
                lo += 1
            if lo < hi:
                pages[:, b, :, lo:hi] = pages[:, s, :, lo:hi]
            first = max(m, hi * PAGE) % PAGE
            if n > max(m, hi * PAGE):
                pages[:, b, :, hi, :, first:n % PAGE] = pages[:, s, :, hi, :, first:n % PAGE]
            state["scores"][:, b, :, :n] = state["scores"][:, s, :, :n]
            state["positions"][:, b, :, :n] = state["positions"][:, s, :, :n]
            state["lengths"][:, b] = state["lengths"][:, s]
        return (pages.view(-1, 2, PAGE, case["d"]), state["scores"].view(-1, cap), state["positions"].view(-1, cap),
                state["lengths"].view(-1))
    if case["op"] == "step":
        words = -(-max(state["new"]) // 32)
        if own:
            cache = state["cache"]
            # the next trees come in the place of the last step's accepted tokens
            cache.drop(state["taken"])
            tree = cache.tree(state["parent"], state["new"])
            cache.append_tree(state["k"], state["v"], tree, q=state["q"], q_out=state["q_out"], rope=state["rope"])
            cache.accept(state["new"], state["paths"])
            view = state["view"]
            return tree.mask, tree.depth, state["q_out"], view["pages"], view["lengths"]
        mask, depth = _plan(state["parent"], state["seq"], state["nth"], len(state["new"]), words)
        pos = state["start"] + depth
        cos, sin = state["cos"][pos], state["sin"][pos]
        dt = state["q"].dtype
        q_out = _rotate(state["q"].float(), cos, sin, case["interleaved"]).to(dt)
        k = _rotate(state["k"].float(), cos, sin, case["interleaved"]).to(dt)
        page, row, pages = state["page"], state["row"], state["pages"]
        pages[page, 0, row] = k
        pages[page, 1, row] = state["v"]
        pages[page[state["to"]], :, row[state["to"]]] = pages[page[state["from"]], :, row[state["from"]]]
        return mask, depth, q_out, pages, state["lengths"]
    scale = 1.0 / math.sqrt(case["d"])
    if own:
        if case["op"] == "tree":
            state["cache"].attend_tree(state["q"], state["out"], state["tree"])
        else:
            state["cache"].attend_window(state["q"], state["out"], state["new"], state["windows"], sink=case["sink"])
        return state["out"]
    r = 0
    for n, h, s in zip(state["new"], state["held"], state["seqs"]):
        q, out = state["q"][r:r + n], state["out"][r:r + n]
        r += n
        if n == 0:
            continue
        if case["op"] == "window":
            _attend_window(q, s["k"], s["v"], state["windows"], case["sink"], scale, out)
            continue
        seen = torch.cat([torch.ones(n, h, dtype=torch.bool, device="cuda"), s["sees"]], 1)
        out.copy_(_masked(q.float(), s["k"].float(), s["v"].float(), seen, scale))
    return state["out"]


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "fork":
        s = _fork_inputs(case, seed)
        layers, batch, _, cap = s["scores"].shape
        pages, scores, positions = s["pages"].double(), s["scores"].double(), s["positions"]
        rows = pages.transpose(3, 4)   # [layer][sequence][head][K, V][page][row][d]
        slot = torch.arange(cap, device="cuda")
        lengths = torch.tensor(s["held"], dtype=torch.int32, device="cuda")[None, :, None].repeat(layers, 1, hkv)
        for b, src in enumerate(s["src"]):
            if src == b:
                continue
            live = slot < s["held"][src]
            scores[:, b] = torch.where(live, scores[:, src], scores[:, b])
            positions[:, b] = torch.where(live, positions[:, src], positions[:, b])
            rows[:, b] = torch.where(live.view(cap // PAGE, PAGE, 1), rows[:, src], rows[:, b])
            lengths[:, b] = s["held"][src]
        return pages.view(-1, 2, PAGE, d), scores.view(-1, cap), positions.view(-1, cap), lengths.view(-1)
    if case["op"] == "step":
        s = _step_inputs(case, seed)
        new, held, half = s["new"], s["held"], case["rot"] // 2
        batch, cap = len(new), _cap(new, held)
        words = -(-max(new) // 32)
        masks, depths, r = [], [], 0
        for n in new:
            for i in range(n):
                bits, steps, at = 0, 0, i
                while at >= 0:
                    bits |= 1 << at
                    steps += 1
                    at = s["parents"][r + at]
                depths.append(steps - 1)
                masks.append([(bits >> 32 * w) & 0xFFFFFFFF for w in range(words)])
            r += n
        masks = [[x - (1 << 32) if x >> 31 else x for x in row] for row in masks]
        pages = torch.zeros(batch, hkv, cap // PAGE, 2, PAGE, d, device="cuda", dtype=torch.float64)
        first = torch.arange(half, device="cuda")
        a, b = (2 * first, 2 * first + 1) if case["interleaved"] else (first, first + half)
        # the rotated pair (x_a, x_b) is the complex number (x_a + i x_b) e^(i angle)
        turned = {"q": s["q"].double(), "k": s["k"].double()}
        start = [h for h, n in zip(held, new) for _ in range(n)]
        at = torch.tensor([h + x for h, x in zip(start, depths)], device="cuda")
        turn = torch.complex(s["cos"].double(), s["sin"].double())[at][:, None]
        for x in turned.values():
            z = torch.complex(x[..., a], x[..., b]) * turn
            x[..., a], x[..., b] = z.real, z.imag
        r = 0
        for i, (n, h, path) in enumerate(zip(new, held, s["paths"])):
            order = list(range(n))
            order[:len(path)] = path   # behind the accepted nodes the tree's rows stay
            for j, x in enumerate((turned["k"], s["v"].double())):
                flat = torch.zeros(hkv, cap, d, device="cuda", dtype=torch.float64)
                if n:
                    flat[:, h:h + n] = x[r:r + n][order].transpose(0, 1)
                pages[i, :, :, j] = flat.view(hkv, cap // PAGE, PAGE, d)
            r += n
        lengths = torch.tensor([h + len(p) for h, p in zip(held, s["paths"]) for _ in range(hkv)], dtype=torch.int32,
                               device="cuda")
        return (torch.tensor(masks, dtype=torch.int32, device="cuda"), torch.tensor(depths, dtype=torch.int32, device="cuda"),
                turned["q"], pages.reshape(-1, 2, PAGE, d), lengths)
    if work(case)["flops"] > 3e12:
        return None
    s = _attend_inputs(case, seed)
    parents = _trees(case, seed)[0] if case["op"] == "tree" else None
    out = torch.empty(sum(s["new"]), hq, d, device="cuda", dtype=torch.float64)
    group = hq // hkv
    r = 0
    for n, h, seq in zip(s["new"], s["held"], s["seqs"]):
        for g in range(hkv if n else 0):
            w = 0 if parents is not None else _ints(case["windows"])[g]
            step = max(1, (1 << 26) // ((h + n if w == 0 else min(h + n, w + 512)) * group))
            step = min(step, 512) if w else step
            for i in range(0, n, step):
                rows = min(step, n - i)
                x = s["q"][r + i:r + i + rows, g * group:(g + 1) * group].double().reshape(rows * group, d)
                last = (h + i + torch.arange(rows, device="cuda"))[:, None]
                if parents is not None:
                    cols = torch.arange(h + n, device="cuda")
                    hidden = torch.ones(rows, h + n, dtype=torch.bool, device="cuda")
                    hidden[:, :h] = False
                    hidden[:, h:] = ~_sees(parents[r:r + n])[i:i + rows].cuda()
                else:
                    cols = torch.arange(h + i + rows, device="cuda")
                    if w:
                        cols = cols[(cols < case["sink"]) | (cols > h + i - w)]
                    hidden = cols > last
                    if w:
                        hidden |= (cols <= last - w) & (cols >= case["sink"])
                k, v = seq["k"][g, cols].double(), seq["v"][g, cols].double()
                z = (x @ k.T / math.sqrt(d)).view(rows, group, -1).masked_fill(hidden[:, None], float("-inf"))
                out[r + i:r + i + rows, g * group:(g + 1) * group] = torch.softmax(z, -1) @ v
        r += n
    return out
