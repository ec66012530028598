"""Cases of the operators around a tree of drafts: what is measured, and their plain forms.

Four operators, as one round of verification uses them over the paged cache:

- ``attend``: attention of the nodes of each request's tree over its pages (``PagedAttention.attend_tree``);
- ``tree``: the round's integer work: ancestor masks, positions and slots of the nodes before it (``tree_layout``), and the
  walk along the target's tokens after it (``tree_accept``);
- ``sample``: the target's token after each row, with temperature, top-k, top-p and min-p, the noise as an input (``sample``);
- ``pages``: the cache's pages: accepted nodes moved behind their context (``PagedAttention.compact``), a prompt shared by
  several requests (``pages_free`` of the last ones, then ``PagedAttention.fork``) and pages copied elsewhere
  (``PagedAttention.copy_pages``).

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits (64 where a value decides between
tokens); with ``own`` true it makes the framework's calls.
"""

import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases


def listed():
    """The sizes are those of the framework's step workloads (64 query and 8 KV heads of 64 over blocks of 16; 32 and 8
    of 128 with 32K contexts; the tiny fp32 layer) and of its verify batches (a vocabulary of 201,088, 8 rows each)."""
    return [
        # one request's tree over a short context: a call where latency counts
        dict(name="attend_b1", op="attend", B=1, n=16, n_hi=16, ctx=2048, ctx_hi=2048, H=64, G=8, hd=64, bs=16, dtype="bf16",
             sinks=False, lens=21),
        # concurrency 64, trees of every size, with attention sinks
        dict(name="attend_b64", op="attend", B=64, n=1, n_hi=64, ctx=512, ctx_hi=8192, H=64, G=8, hd=64, bs=16, dtype="bf16",
             sinks=True, lens=22),
        # long contexts, some 60 nodes each
        dict(name="attend_32k", op="attend", B=16, n=57, n_hi=63, ctx=32768, ctx_hi=32768, H=32, G=8, hd=128, bs=16,
             dtype="bf16", sinks=False, lens=23),
        # the fp32 layer
        dict(name="attend_f32_odd", op="attend", B=5, n=0, n_hi=37, ctx=0, ctx_hi=300, H=4, G=2, hd=16, bs=4, dtype="f32",
             sinks=True, lens=24),
        # the bookkeeping of one request
        dict(name="tree_b1", op="tree", B=1, n=16, n_hi=16, ctx=2048, ctx_hi=2048, bs=16, depth=6, lens=25),
        # many requests with large trees
        dict(name="tree_b256", op="tree", B=256, n=1, n_hi=255, ctx=512, ctx_hi=8192, bs=16, depth=12, lens=26),
        # one request's 8 rows, fp32 logits, top-k and top-p
        dict(name="sample_b1", op="sample", B=1, n=8, n_hi=8, V=201088, dtype="f32", kind="both", lens=27),
        # concurrency 64, bf16 logits, every request with settings of its own, some greedy
        dict(name="sample_b64", op="sample", B=64, n=8, n_hi=8, V=201088, dtype="bf16", kind="mixed", lens=28),
        # ragged requests over a vocabulary whose rows start off the 16-byte grid
        dict(name="sample_ragged", op="sample", B=33, n=0, n_hi=9, V=32003, dtype="f32", kind="mixed", lens=29),
        # the accepted nodes of 64 requests, 16 layers
        dict(name="compact_b64", op="compact", B=64, n=9, n_hi=32, ctx=512, ctx_hi=8192, layers=16, G=8, hd=64, bs=16,
             dtype="bf16", lens=30),
        # 8 prompts of up to 8192 tokens, 8 samples of each: the last pages of 16 layers
        dict(name="fork_b8", op="fork", B=8, each=8, ctx=512, ctx_hi=8192, layers=16, G=8, hd=64, bs=16, dtype="bf16", lens=31),
        # 1001 pages of 16 layers to another part of the pool
        dict(name="copy_1001", op="copy", n=1001, layers=16, G=8, hd=64, bs=16, dtype="bf16", lens=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges: sizes spread over their logarithm, odd ones among them."""
    op = rng.choice(["attend", "attend", "attend", "sample", "sample", "tree", "compact", "fork", "copy"])
    lens = rng.randrange(1 << 30)
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    if op == "attend":
        if dtype == "f32":
            H, G, hd = rng.choice([(4, 2, 16), (8, 2, 64), (6, 3, 40)])
            return dict(op=op, B=_log(rng, 1, 8), n=0, n_hi=_log(rng, 1, 64), ctx=0, ctx_hi=_log(rng, 1, 1000), H=H, G=G,
                        hd=hd, bs=rng.choice([4, 16]), dtype=dtype, sinks=rng.random() < 0.5, lens=lens)
        H, G, hd = rng.choice([(64, 8, 64), (32, 8, 128), (28, 4, 128), (8, 2, 64), (5, 5, 64)])
        B, n_hi = _log(rng, 1, 64), _log(rng, 1, 100)
        return dict(op=op, B=B, n=rng.choice([0, 1, n_hi]), n_hi=n_hi, ctx=0, ctx_hi=_log(rng, 16, 32768 if B <= 8 else 4096),
                    H=H, G=G, hd=hd, bs=rng.choice([16, 32, 64]), dtype=dtype, sinks=rng.random() < 0.3, lens=lens)
    if op == "sample":
        n_hi = rng.choice([1, 4, 8, 9])
        return dict(op=op, B=_log(rng, 1, 64), n=rng.choice([0, 1, n_hi]), n_hi=n_hi, V=_log(rng, 2, 180000), dtype=dtype,
                    kind=rng.choice(["mixed", "mixed", "both", "none"]), lens=lens)
    if op == "tree":
        n_hi = _log(rng, 1, 255)
        return dict(op=op, B=_log(rng, 1, 256), n=rng.choice([0, 1, n_hi]), n_hi=n_hi, ctx=0, ctx_hi=_log(rng, 16, 8192),
                    bs=rng.choice([4, 16, 32]), depth=_log(rng, 1, 12), lens=lens)
    G, hd = rng.choice([(2, 16), (2, 64), (3, 40)] if dtype == "f32" else [(8, 64), (8, 128), (4, 128), (2, 64), (5, 64)])
    bs = rng.choice([4, 16, 32])
    if op == "compact":
        n_hi = _log(rng, 1, 64)
        return dict(op=op, B=_log(rng, 1, 64), n=rng.choice([0, 1, n_hi]), n_hi=n_hi, ctx=0, ctx_hi=_log(rng, 1, 4096),
                    layers=_log(rng, 1, 16), G=G, hd=hd, bs=bs, dtype=dtype, lens=lens)
    if op == "fork":
        return dict(op=op, B=_log(rng, 1, 8), each=_log(rng, 1, 8), ctx=0, ctx_hi=_log(rng, 1, 8192), layers=_log(rng, 1, 8),
                    G=G, hd=hd, bs=bs, dtype=dtype, lens=lens)
    return dict(op=op, n=_log(rng, 1, 500), layers=_log(rng, 1, 16), G=G, hd=hd, bs=bs, dtype=dtype, lens=lens)


def _lengths(c):
    """Rows and prior context of each request, from the case alone (so that work() knows them)."""
    r = random.Random(c["lens"])
    n = [r.randint(c["n"], c["n_hi"]) for _ in range(c["B"])]
    if sum(n) == 0:
        n[0] = 1
    ctx = [r.randint(c["ctx"], c["ctx_hi"]) for _ in range(c["B"])] if "ctx" in c else [0] * c["B"]
    return n, ctx


def _trees(c):
    """Parents of each request's nodes, level by level: the root is the last committed token, the first level its
    candidates for the next one, and so on; -1 is the root's parent."""
    r = random.Random(c["lens"] + 2)
    deep = c.get("depth", 7)
    out = []
    for m in _lengths(c)[0]:
        parents = [-1][:m]
        level = [0]
        d = 1
        while len(parents) < m:
            left = m - len(parents)
            width = left if d >= deep else min(left, r.randint(1, max(1, 2 * m // deep)))
            kids = sorted(r.choice(level) for _ in range(width))
            level = list(range(len(parents), len(parents) + width))
            parents += kids
            d += 1
            if d > deep:
                d = deep
                level = [p for p in range(1, len(parents))] if deep > 1 else [0]
                level = [p for p in level if _depth(parents, p) < deep] or [0]
        out.append(parents)
    return out


def _depth(parents, j):
    d = 0
    while parents[j] >= 0:
        j = parents[j]
        d += 1
    return d


SETTINGS = [  # temperature, top-k (0: off), top-p (1: off), min-p (0: off)
    (0.0, 0, 1.0, 0.0),
    (1.0, 0, 1.0, 0.0),
    (0.8, 50, 0.95, 0.0),
    (1.0, 0, 0.9, 0.0),
    (0.6, 20, 0.95, 0.0),
    (1.3, 0, 1.0, 0.1),
    (0.7, 64, 0.8, 0.02),
    (1.0, 200, 1.0, 0.0),
]


def _settings(c):
    r = random.Random(c["lens"] + 1)
    if c["kind"] == "both":
        return [SETTINGS[2]] * c["B"]
    if c["kind"] == "none":
        return [SETTINGS[1]] * c["B"]
    return [r.choice(SETTINGS) for _ in range(c["B"])]


def _accepted(c):
    """Rows that move, of each request: the accepted path lies behind the slots that it moves to."""
    r = random.Random(c["lens"] + 3)
    return [r.randint(0, min(7, (m - 1) // 2)) if m > 0 else 0 for m in _lengths(c)[0]]


def work(c):
    op = c["op"]
    if op == "tree":
        t = sum(_lengths(c)[0])
        # parents, tokens, targets in; masks, positions, slots, path out
        return {"bytes": t * (12.0 + 4 * _words(c) + 20) + c["B"] * 24, "flops": 4.0 * t}
    if op == "sample":
        n, _ = _lengths(c)
        e = 4 if c["dtype"] == "f32" else 2
        # every logit once; the noise of the rows that keep every token
        noise = sum(m for m, s in zip(n, _settings(c)) if s[0] > 0 and s[1] == 0 and s[2] >= 1 and s[3] == 0)
        return {"bytes": (sum(n) * e + noise * 4.0) * c["V"] + sum(n) * 4, "flops": 4.0 * sum(n) * c["V"]}
    e = 4 if c["dtype"] == "f32" else 2
    if op == "attend":
        n, ctx = _lengths(c)
        kv = sum(2 * (x + m) * c["G"] * c["hd"] * e + (x + m + c["bs"] - 1) // c["bs"] * 4 for x, m in zip(ctx, n) if m)
        pairs = sum(m * x for x, m in zip(ctx, n)) + sum(1 + _depth(p, j) for p in _trees(c) for j in range(len(p)))
        return {"bytes": 2.0 * sum(n) * c["H"] * c["hd"] * e + kv + sum(n) * 4 * _words(c), "flops": 4.0 * pairs * c["H"] * c["hd"]}
    vec = 4.0 * c["layers"] * c["G"] * c["hd"] * e  # of one position: keys and values, read and written
    if op == "compact":
        return {"bytes": max(sum(_accepted(c)), 1) * vec, "flops": float(c["B"])}
    if op == "fork":
        part, pages = _fork_sizes(c)
        return {"bytes": max(part, 1) * vec + pages * 12, "flops": float(c["B"])}
    return {"bytes": c["n"] * c["bs"] * vec, "flops": float(c["n"])}


def _words(c):
    return (c["n_hi"] + 31) // 32


def _contexts(c):
    r = random.Random(c["lens"])
    return [r.randint(c["ctx"], c["ctx_hi"]) for _ in range(c["B"])]


def _fork_sizes(c):
    ctx = _contexts(c)
    return c["each"] * sum(x % c["bs"] for x in ctx), c["each"] * sum((x + c["bs"] - 1) // c["bs"] for x in ctx)


# ------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _dt(c):
    return torch.float32 if c["dtype"] == "f32" else torch.bfloat16


def _randn(g, shape, dt, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dt)


def _offsets(n):
    return torch.tensor([0] + n, device=DEV).cumsum(0).to(torch.int32)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _tables(g, blocks, spare):
    """Pages anywhere in the pool for each request; entries past its last page are -1."""
    B, mb, nb = len(blocks), max(max(blocks), 1), sum(blocks) + spare
    ids = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    at = torch.arange(mb, device=DEV)[None, :]
    first = torch.tensor([0] + blocks, device=DEV).cumsum(0)[:B, None]
    have = at < torch.tensor(blocks, device=DEV)[:, None]
    return torch.where(have, ids[(first + at).clamp(max=nb - 1)], torch.full((), -1, dtype=torch.int32, device=DEV)).contiguous(), nb


def prepare(c, seed):
    return {"attend": _prepare_attend, "tree": _prepare_tree, "sample": _prepare_sample, "compact": _prepare_compact,
            "fork": _prepare_fork, "copy": _prepare_copy}[c["op"]](c, seed)


def _rows(c):
    """Host lists and device tensors of the requests' rows, shared by the operators with rows."""
    n, ctx = _lengths(c)
    return n, ctx, dict(c=c, T=sum(n), nmax=max(n), qsl=_offsets(n))


def _bits(c, trees):
    """The nodes' ancestor masks in words of 32, as tree_layout writes them."""
    w = _words(c)
    rows = []
    for parents in trees:
        sets = []
        for j, p in enumerate(parents):
            sets.append((sets[p] if p >= 0 else 0) | 1 << j)
        rows += [[(x >> 32 * i & 0xffffffff) - ((x >> 32 * i & 0x80000000) << 1) for i in range(w)] for x in sets]
    return _i32(rows)


def _prepare_attend(c, seed):
    g, dt = _gen(seed), _dt(c)
    B, H, G, hd, bs = c["B"], c["H"], c["G"], c["hd"], c["bs"]
    n, ctx, s = _rows(c)
    s["table"], s["nb"] = _tables(g, [(x + m + bs - 1) // bs for x, m in zip(ctx, n)], 2)
    s.update(seq=_i32([x + m for x, m in zip(ctx, n)]), mask=_bits(c, _trees(c)), q=_randn(g, (s["T"], H, hd), dt),
             k=_randn(g, (s["nb"], G, bs, hd), dt), v=_randn(g, (s["nb"], G, bs, hd), dt),
             sink=_randn(g, (H,), torch.float32) if c["sinks"] else None)
    s["out"] = torch.empty(s["T"], H * hd, dtype=dt, device=DEV)
    if own:
        s["plan"] = _plan(c)
        s["ws"] = s["plan"].workspace(B, s["T"])
    return s


def _plan(c):
    from speculative_drafting_gb300 import binding

    return binding.PagedAttention(c.get("H", c["G"]), c["G"], c["hd"], c["bs"], dtype=c["dtype"])


def _prepare_tree(c, seed):
    g = _gen(seed)
    n, ctx, s = _rows(c)
    T = s["T"]
    s["table"], s["nb"] = _tables(g, [(x + m + c["bs"] - 1) // c["bs"] for x, m in zip(ctx, n)], 2)
    trees = _trees(c)
    s.update(seq=_i32([x + m for x, m in zip(ctx, n)]), parent=_i32([p for t in trees for p in t]))
    # few tokens, so that the target's token is often a child's, now and then two children's
    s["tok"] = _i32([j % 7 for t in trees for j in range(len(t))])
    s["tok"] += 7 * torch.randint(0, 2, (T,), generator=g, device=DEV, dtype=torch.int32)
    s["target"] = torch.randint(0, 14, (T,), generator=g, device=DEV, dtype=torch.int32)
    # most nodes: the target agrees with one of the children
    req = torch.searchsorted(s["qsl"], torch.arange(T, device=DEV, dtype=torch.int32), right=True) - 1
    up = torch.where(s["parent"] >= 0, s["parent"].long() + s["qsl"].long()[req], T)
    most = torch.cat([s["target"], s["target"][:1]])
    keep = torch.rand(T, generator=g, device=DEV) < 0.8
    at = torch.arange(T, device=DEV)
    last = torch.full((T + 1,), -1, device=DEV, dtype=torch.int64).scatter_reduce(0, up, torch.where(keep, at, -1), "amax")
    s["target"] = torch.where(last[:T] >= 0, s["tok"][last[:T].clamp(min=0)], most[:T])
    e32 = dict(dtype=torch.int32, device=DEV)
    s.update(mask=torch.empty(T, _words(c), **e32), pos=torch.empty(T, dtype=torch.int64, device=DEV),
             slot=torch.empty(T, dtype=torch.int64, device=DEV), accepted=torch.empty(c["B"], **e32), path=torch.empty(T, **e32),
             bonus=torch.empty(c["B"], **e32))
    if own:
        s["ws"] = torch.zeros(256, dtype=torch.uint8, device=DEV)
    return s


def _prepare_sample(c, seed):
    g, dt = _gen(seed), _dt(c)
    B, V = c["B"], c["V"]
    n, _, s = _rows(c)
    T = s["T"]
    # a broad floor, and some hundred likely tokens whose logits fall off as ranks do; some rows are sharper than others
    logits = torch.randn(T, V, generator=g, device=DEV) * 1.5
    m = min(V, 300)
    likely = (torch.randint(0, V, (T, 1), generator=g, device=DEV) + torch.arange(m, device=DEV) * (V // m)) % V
    rank = torch.arange(1, m + 1, device=DEV, dtype=torch.float32)
    logits.scatter_(1, likely, 17.0 - 1.6 * torch.log(rank) + torch.randn(T, m, generator=g, device=DEV) * 0.5)
    logits *= torch.rand(T, 1, generator=g, device=DEV) * 0.5 + 0.65
    # a few tokens are barred, as by a grammar
    logits[torch.rand(T, V, generator=g, device=DEV) < 0.01] = -math.inf
    logits[:, 0] = logits[:, 0].clamp(min=-5.0)
    st = _settings(c)
    s.update(logits=logits.to(dt), temp=torch.tensor([x[0] for x in st], device=DEV), top_k=_i32([x[1] for x in st]),
             top_p=torch.tensor([x[2] for x in st], device=DEV), min_p=torch.tensor([x[3] for x in st], device=DEV),
             gumbel=-torch.log(torch.empty(T, V, device=DEV).exponential_(generator=g)))
    s["token"] = torch.empty(T, dtype=torch.int32, device=DEV)
    if own:
        from speculative_drafting_gb300 import binding

        s["ws"] = binding.sample_workspace(B, T, V)
    return s


def _caches(c, g, nb):
    shape = (c["layers"], nb, c["G"], c["bs"], c["hd"])
    return dict(nb=nb, k=_randn(g, shape, _dt(c)), v=_randn(g, shape, _dt(c)))


def _prepare_compact(c, seed):
    g = _gen(seed)
    bs = c["bs"]
    n, ctx, s = _rows(c)
    table, nb = _tables(g, [(x + m + bs - 1) // bs for x, m in zip(ctx, n)], 2)
    s.update(table=table, seq=_i32([x + m for x, m in zip(ctx, n)]), accepted=_i32(_accepted(c)), **_caches(c, g, nb))
    # the accepted nodes: any ascending ones behind the slots that they move to
    r = random.Random(seed)
    path = []
    for m, a in zip(n, _accepted(c)):
        path += [0][:m] + sorted(r.sample(range(a + 1, m), a)) + [-1] * (m - 1 - a) if m else []
    s["path"] = _i32(path)
    if own:
        s["plan"] = _plan(c)
        s["ws"] = s["plan"].append_workspace()
    return s


def _prepare_fork(c, seed):
    g = _gen(seed)
    B, each, bs = c["B"], c["each"], c["bs"]
    ctx = _contexts(c)
    table, nb = _tables(g, [(x + bs - 1) // bs for x in ctx], B * each + 3)
    refs = torch.zeros(nb + 1, dtype=torch.int32, device=DEV)
    refs[torch.where(table >= 0, table, nb).long().view(-1)] = 1
    # rows 0 .. B - 1 of the table are the prompts, the rest their samples
    s = dict(c=c, table=torch.cat([table, torch.full((B * each, table.shape[1]), -1, dtype=torch.int32, device=DEV)]),
             refs=refs[:nb].clone(), parent=_i32([i for i in range(B) for _ in range(each)]),
             child=B + torch.randperm(B * each, generator=g, device=DEV).to(torch.int32),
             length=_i32([x for x in ctx for _ in range(each)]), **_caches(c, g, nb))
    if own:
        from speculative_drafting_gb300 import binding

        s["plan"] = _plan(c)
        s["ws"] = binding.pages_workspace(B * each, nb)
    return s


def _prepare_copy(c, seed):
    g = _gen(seed)
    nb = 2 * c["n"] + 3
    ids = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    s = dict(c=c, src=ids[:c["n"]].contiguous(), dst=ids[c["n"]:2 * c["n"]].contiguous(), **_caches(c, g, nb))
    if own:
        s["plan"] = _plan(c)
        s["ws"] = s["plan"].append_workspace()
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    return {"attend": _run_attend, "tree": _run_tree, "sample": _run_sample, "compact": _run_compact, "fork": _run_fork,
            "copy": _run_copy}[s["c"]["op"]](s)


def _side_by_side(s):
    """Rows of the requests side by side: [B, nmax] places in the batch, which are there, and each row's request and place."""
    qsl = s["qsl"].long()
    n = qsl[1:] - qsl[:-1]
    j = torch.arange(s["nmax"], device=DEV)
    t = torch.arange(s["T"], device=DEV)
    req = torch.searchsorted(qsl, t, right=True) - 1
    return (qsl[:-1, None] + j).clamp(max=s["T"] - 1), j < n[:, None], req, t - qsl[req]


def _run_attend(s):
    c = s["c"]
    if own:
        s["plan"].attend_tree(c["B"], s["T"], s["qsl"], s["seq"], s["q"], s["k"], s["v"], s["table"], s["nb"], s["mask"], s["out"],
                              s["ws"], sink=s["sink"])
        return s["out"]
    B, H, G, hd = c["B"], c["H"], c["G"], c["hd"]
    rows, there, req, at = _side_by_side(s)
    q = s["q"][rows].float().view(B, s["nmax"], G, H // G, hd)
    table = s["table"].long().clamp(min=0)
    k, v = (x[table].transpose(2, 3).reshape(B, -1, G, hd).float() for x in (s["k"], s["v"]))
    # key t is node t - ctx of the tree from the context's end on
    seq = s["seq"].long()
    key = torch.arange(k.shape[1], device=DEV)
    node = (key[None] - (seq - there.sum(-1))[:, None])[:, None, :].expand(-1, s["nmax"], -1)
    word = torch.gather(s["mask"][rows].long(), 2, (node >> 5).clamp(0, s["mask"].shape[1] - 1))
    ok = (node < 0) | (word >> (node & 31).clamp(min=0) & 1 == 1)
    ok &= (key < seq[:, None])[:, None, :] & there[:, :, None]
    sc = torch.einsum("bngxd,btgd->bgxnt", q, k) / math.sqrt(hd)
    sc.masked_fill_(~ok[:, None, None], -math.inf)
    sink = torch.full((H,), -math.inf, device=DEV) if s["sink"] is None else s["sink"]
    sink = sink.view(1, G, H // G, 1)
    top = torch.maximum(sc.amax(-1), sink)
    top = torch.where(torch.isinf(top), 0.0, top)
    w = sc.sub_(top[..., None]).exp_()
    den = w.sum(-1) + torch.exp(sink - top)
    o = torch.einsum("bgxnt,btgd->bngxd", w, v)
    o = o / den.clamp(min=1e-30).permute(0, 3, 1, 2)[..., None]
    s["out"].copy_(o[req, at].reshape(s["T"], H * hd))
    return s["out"]


def _run_tree(s):
    c = s["c"]
    out = {x: s[x] for x in ("mask", "pos", "slot", "accepted", "path", "bonus")}
    if own:
        from speculative_drafting_gb300 import binding

        binding.tree_layout(c["B"], s["T"], s["qsl"], s["seq"], s["parent"], s["table"], s["nb"], c["bs"], s["mask"], s["pos"],
                            s["slot"], s["ws"])
        binding.tree_accept(c["B"], s["T"], s["qsl"], s["parent"], s["tok"], s["target"], s["accepted"], s["path"], s["bonus"], s["ws"])
        return out
    T, bs = s["T"], c["bs"]
    rows, there, req, at = _side_by_side(s)
    first = s["qsl"].long()[req]
    n = there.sum(-1)
    up = torch.where(s["parent"] >= 0, first + s["parent"], -1)
    # a node's ancestors, one level a step
    bits = torch.zeros(T, 32 * s["mask"].shape[1], dtype=torch.int64, device=DEV)
    node, depth, t = torch.arange(T, device=DEV), torch.zeros(T, dtype=torch.int64, device=DEV), torch.arange(T, device=DEV)
    for d in range(c["depth"] + 1):
        here = node >= 0
        bits[t, at[node]] |= here.long()
        node = torch.where(here, up[node], -1)
        depth += node >= 0
    bits = (bits.view(T, -1, 32) << torch.arange(32, device=DEV)).sum(-1)
    s["mask"].copy_(torch.where(bits >= 1 << 31, bits - (1 << 32), bits))
    ctx = (s["seq"] - n)[req].long()
    s["pos"].copy_(ctx + depth)
    s["slot"].copy_(s["table"][req, (ctx + at) // bs].long() * bs + (ctx + at) % bs)
    # the walk, all requests at once
    cur = s["qsl"].long()[:-1].clamp(max=T - 1)
    live = n > 0
    b = torch.arange(c["B"], device=DEV)
    path = torch.full((c["B"], s["nmax"]), -1, dtype=torch.int64, device=DEV)
    path[:, 0] = torch.where(live, 0, -1)
    accepted = torch.zeros(c["B"], dtype=torch.int64, device=DEV)
    bonus = torch.where(live, s["target"][cur].long(), -1)
    for d in range(c["depth"]):
        kid = there & (up[rows] == cur[:, None]) & (s["tok"][rows] == s["target"][cur][:, None]) & live[:, None]
        live = kid.any(-1)
        j = kid.long().argmax(-1)
        cur = torch.where(live, rows[b, j], cur)
        accepted += live
        spot = accepted.clamp(max=s["nmax"] - 1)
        path[b, spot] = torch.where(live, j, path[b, spot])
        bonus = torch.where(live, s["target"][cur].long(), bonus)
    s["accepted"].copy_(accepted)
    s["path"].copy_(path[req, at])
    s["bonus"].copy_(bonus)
    return out


def _run_sample(s):
    c = s["c"]
    if own:
        from speculative_drafting_gb300 import binding

        binding.sample(c["B"], s["T"], s["qsl"], s["logits"], c["V"], s["temp"], s["top_k"], s["top_p"], s["min_p"], s["gumbel"],
                       s["token"], s["ws"])
        return s["token"]
    qsl = s["qsl"].long()
    req = torch.searchsorted(qsl, torch.arange(s["T"], device=DEV), right=True) - 1
    temp = s["temp"][req]
    cold = (temp == 0)[:, None]
    l, order = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True)
    # 64 bits: the numbers decide between tokens
    x = (l - l[:, :1]).double() / torch.where(cold, 1.0, temp[:, None]).double()
    w = torch.exp(x)
    rank = torch.arange(c["V"], device=DEV)[None]
    k = s["top_k"][req].long()[:, None]
    keep = (rank < torch.where(k > 0, k, c["V"]))
    before = torch.cumsum(w * keep, -1)
    total = before[:, -1:].clone()
    before -= w * keep
    p = s["top_p"][req].double()[:, None]
    keep &= (before < p * total) | (p >= 1) | (rank == 0)
    keep &= (w >= s["min_p"][req].double()[:, None]) & (w > 0)
    score = torch.where(keep, x + torch.gather(s["gumbel"], 1, order).double(), -math.inf)
    # equal scores: the lowest index
    best = score.amax(-1, keepdim=True)
    pick = torch.where(score == best, order, c["V"]).amin(-1)
    s["token"].copy_(torch.where(cold[:, 0], order[:, 0], pick))
    return s["token"]


def _run_compact(s):
    c = s["c"]
    if own:
        s["plan"].compact(c["layers"], c["B"], s["T"], s["qsl"], s["seq"], s["accepted"], s["path"], s["table"], s["nb"], s["k"], s["v"],
                          s["ws"])
        return {"k_cache": s["k"], "v_cache": s["v"]}
    bs = c["bs"]
    rows, there, req, at = _side_by_side(s)
    ctx = (s["seq"] - there.sum(-1))[req].long()
    moves = torch.nonzero((at > 0) & (at <= s["accepted"][req]))[:, 0]
    req, ctx, frm, to = req[moves], ctx[moves], s["path"][moves].long(), at[moves]
    f, t = ctx + frm, ctx + to
    fb, tb = s["table"][req, f // bs].long(), s["table"][req, t // bs].long()
    for x in (s["k"], s["v"]):
        x[:, tb, :, t % bs] = x[:, fb, :, f % bs]
    return {"k_cache": s["k"], "v_cache": s["v"]}


def _run_fork(s):
    c = s["c"]
    out = {"table": s["table"], "refs": s["refs"], "k_cache": s["k"], "v_cache": s["v"]}
    if own:
        from speculative_drafting_gb300 import binding

        n = c["B"] * c["each"]
        binding.pages_free(n, s["child"], s["table"], s["refs"], s["ws"])
        s["plan"].fork(c["layers"], n, s["parent"], s["child"], s["length"], s["table"], s["refs"], s["k"], s["v"], s["ws"])
        return out
    bs, nb, child = c["bs"], s["nb"], s["child"].long()
    # the samples of the last time give their pages back
    old = s["table"][child].view(-1).long()
    count = torch.zeros(nb + 1, dtype=torch.int32, device=DEV)
    count.index_add_(0, torch.where(old >= 0, old, nb), torch.ones_like(old, dtype=torch.int32))
    s["refs"] -= count[:nb]
    s["table"][child] = -1
    # the lowest free pages, in order, to those whose last page is not full
    part = s["length"] % bs
    free = torch.nonzero(s["refs"] == 0)[:, 0]
    nth = torch.cumsum((part > 0).int(), 0) - 1
    rows = s["table"][s["parent"].long()]
    full = (s["length"] // bs)[:, None]
    at = torch.arange(rows.shape[1], device=DEV)[None]
    new = free[nth.clamp(min=0)].int()[:, None]
    rows_new = torch.where(at < full, rows, torch.where((at == full) & (part > 0)[:, None], new, -1))
    s["table"][child] = rows_new
    ids = rows_new.view(-1).long()
    count = torch.zeros(nb + 1, dtype=torch.int32, device=DEV)
    count.index_add_(0, torch.where(ids >= 0, ids, nb), torch.ones_like(ids, dtype=torch.int32))
    s["refs"] += count[:nb]
    # their first positions
    i, p = torch.nonzero(torch.arange(bs, device=DEV)[None] < part[:, None]).unbind(1)
    src = rows[i, full[i, 0].long()].long()
    dst = new[i, 0].long()
    for x in (s["k"], s["v"]):
        x[:, dst, :, p] = x[:, src, :, p]
    return out


def _run_copy(s):
    c = s["c"]
    if own:
        s["plan"].copy_pages(c["layers"], c["n"], s["src"], s["dst"], s["nb"], s["k"], s["v"], s["ws"])
    else:
        for x in (s["k"], s["v"]):
            x[:, s["dst"].long()] = x[:, s["src"].long()]
    return {"k_cache": s["k"], "v_cache": s["v"]}


# ------------------------------------------------------------------ from the definitions, in 64 bits


def exact(c, seed):
    s = prepare(c, seed)
    return {"attend": _exact_attend, "tree": _exact_tree, "sample": _exact_sample, "compact": _exact_compact, "fork": _exact_fork,
            "copy": _exact_copy}[c["op"]](s)


def _exact_attend(s):
    """Request by request and KV head by KV head, the tree's nodes from their parents."""
    c = s["c"]
    H, G, hd, bs = c["H"], c["G"], c["hd"], c["bs"]
    out = torch.zeros(s["T"], H, hd, dtype=torch.float64, device=DEV)
    qsl, seq = s["qsl"].tolist(), s["seq"].tolist()
    for r, parents in enumerate(_trees(c)):
        n, L = qsl[r + 1] - qsl[r], seq[r]
        if n == 0:
            continue
        line = []  # a node's line of ancestors
        for j, p in enumerate(parents):
            line.append((line[p] if p >= 0 else []) + [j])
        sees = torch.zeros(n, L, dtype=torch.bool)
        sees[:, :L - n] = True
        for j in range(n):
            sees[j, [L - n + i for i in line[j]]] = True
        hide = ~sees.to(DEV)
        pages = s["table"][r, : (L + bs - 1) // bs].long()
        for g in range(G):
            k = s["k"][pages, g].reshape(-1, hd)[:L].double()
            v = s["v"][pages, g].reshape(-1, hd)[:L].double()
            for h in range(g * (H // G), (g + 1) * (H // G)):
                x = (s["q"][qsl[r]:qsl[r + 1], h].double() @ k.T) * hd ** -0.5
                x[hide] = -math.inf
                if s["sink"] is not None:
                    x = torch.cat([x, s["sink"][h].double().expand(n, 1)], 1)
                out[qsl[r]:qsl[r + 1], h] = torch.softmax(x, -1)[:, :L] @ v
    return out.view(s["T"], H * hd)


def _exact_tree(s):
    """Node by node on the host."""
    c = s["c"]
    bs, w = c["bs"], s["mask"].shape[1]
    qsl, seq, tok, target, table = (s[x].tolist() for x in ("qsl", "seq", "tok", "target", "table"))
    mask, pos, slot, acc, path, bonus = [], [], [], [], [], []
    for r, parents in enumerate(_trees(c)):
        lo, n = qsl[r], len(parents)
        ctx = seq[r] - n
        for j in range(n):
            seen, i, d = {j}, j, 0
            while parents[i] >= 0:
                i = parents[i]
                seen.add(i)
                d += 1
            word = [sum(1 << (i - 32 * x) for i in seen if i // 32 == x) for x in range(w)]
            mask.append([x - (1 << 32) if x >= 1 << 31 else x for x in word])
            pos.append(ctx + d)
            slot.append(table[r][(ctx + j) // bs] * bs + (ctx + j) % bs)
        if n == 0:
            acc.append(0)
            bonus.append(-1)
            continue
        walk = [0]
        while True:
            kids = [j for j in range(n) if parents[j] == walk[-1] and tok[lo + j] == target[lo + walk[-1]]]
            if not kids:
                break
            walk.append(kids[0])
        acc.append(len(walk) - 1)
        bonus.append(target[lo + walk[-1]])
        path += walk + [-1] * (n - len(walk))
    return {"mask": _i32(mask), "pos": torch.tensor(pos), "slot": torch.tensor(slot), "accepted": _i32(acc), "path": _i32(path),
            "bonus": _i32(bonus)}


def _exact_sample(s):
    """Row by row: the order of the tokens, then the number of them that each setting leaves."""
    c = s["c"]
    V = c["V"]
    qsl, tokens = s["qsl"].tolist(), []
    place = torch.arange(V, device=DEV)
    for r, (t, k, p, m) in enumerate(zip(*(s[x].tolist() for x in ("temp", "top_k", "top_p", "min_p")))):
        for row in range(qsl[r], qsl[r + 1]):
            y = s["logits"][row].double()
            if t == 0:
                tokens.append((y == y.max()).long().argmax().view(1))
                continue
            order = torch.argsort(-y, stable=True)
            prob = torch.softmax(y / t, -1)[order]
            first = prob[: k if k > 0 else V]
            ahead = torch.cat([prob.new_zeros(1), torch.cumsum(first, 0)[:-1]])
            count = first.numel() if p >= 1 else (ahead < p * first.sum()).sum().clamp(min=1)
            left = (place[: first.numel()] < count) & (first >= m * first[0]) & (first > 0)
            noise = s["gumbel"][row][order[: first.numel()]].double()
            score = torch.where(left, torch.log(first) + noise, -math.inf)
            tokens.append(torch.where(score == score.max(), order[: first.numel()], V).min().view(1))
    return torch.cat(tokens).int()


def _exact_compact(s):
    """Request by request: the path's positions gathered, then put down one after another."""
    c = s["c"]
    bs = c["bs"]
    k, v = s["k"].clone(), s["v"].clone()
    qsl, seq, acc, path, table = (s[x].tolist() for x in ("qsl", "seq", "accepted", "path", "table"))
    for r in range(c["B"]):
        ctx = seq[r] - (qsl[r + 1] - qsl[r])
        for x in (k, v):
            took = [x[:, table[r][f // bs], :, f % bs].clone() for f in (ctx + path[qsl[r] + d] for d in range(1, acc[r] + 1))]
            for d, y in enumerate(took):
                x[:, table[r][(ctx + 1 + d) // bs], :, (ctx + 1 + d) % bs] = y
    return {"k_cache": k, "v_cache": v}


def _exact_fork(s):
    """Sample by sample on the host."""
    c = s["c"]
    bs = c["bs"]
    k, v = s["k"].clone(), s["v"].clone()
    table, refs = s["table"].tolist(), s["refs"].tolist()
    for a, b, n in zip(*(s[x].tolist() for x in ("parent", "child", "length"))):
        full = n // bs
        table[b] = table[a][:full] + [-1] * (len(table[a]) - full)
        if n % bs:
            new = refs.index(0)
            for x in (k, v):
                x[:, new, :, : n % bs] = x[:, table[a][full], :, : n % bs]
            table[b][full] = new
        for page in table[b]:
            if page >= 0:
                refs[page] += 1
    return {"table": _i32(table), "refs": _i32(refs), "k_cache": k, "v_cache": v}


def _exact_copy(s):
    k, v = s["k"].clone(), s["v"].clone()
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        k[:, b], v[:, b] = s["k"][:, a], s["v"][:, a]
    return {"k_cache": k, "v_cache": v}
