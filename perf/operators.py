"""Cases of the paged-cache operators and of verification by sampling: what is measured, and their plain forms.

Three operators, as one round of speculative decoding uses them over the same paged cache:

- ``append``: the RMS norm of each query and key head, their position rotation, and the write of keys and values at
  their cache slots, from the rows of one QKV projection (``PagedAttention.append``);
- ``attend``: attention of each request's new rows over its pages (``PagedAttention.attend``), from one decoded token
  to a whole prompt;
- ``verify``: acceptance of greedy drafts against the target's probabilities, with the random numbers as inputs
  (``verify_sampled``).

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits (64 where a value decides between
tokens or an angle is far); with ``own`` true it makes the framework's calls.
"""

import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases


def listed():
    """The sizes are those of the framework's step workloads (64 query and 8 KV heads of 64 over blocks of 16; 32 and 8
    of 128 with 32K contexts; the tiny fp32 step) and of its verify batches (a vocabulary of 201,088, 8 rows each)."""
    return [
        # the verify rows of one request, K = 7 drafts: a call where latency counts
        dict(name="append_b1_k7", op="append", T=8, H=64, G=8, hd=64, bs=16, dtype="bf16", norm=False, pos=2048, lens=1),
        # a prompt of 8192 tokens through a layer with query and key norms
        dict(name="append_prompt", op="append", T=8192, H=32, G=8, hd=128, bs=16, dtype="bf16", norm=True, pos=0, lens=2),
        # the fp32 layer, odd row count, far positions
        dict(name="append_f32_odd", op="append", T=333, H=4, G=2, hd=16, bs=4, dtype="f32", norm=True, pos=1000003, lens=3),
        # one decoded token for one request
        dict(name="attend_token_b1", op="attend", B=1, n=1, n_hi=1, ctx=2048, ctx_hi=2048, H=64, G=8, hd=64, bs=16,
             dtype="bf16", sinks=False, lens=4),
        # verification of 7 drafts at concurrency 64, with attention sinks
        dict(name="attend_verify_b64", op="attend", B=64, n=8, n_hi=8, ctx=512, ctx_hi=8192, H=64, G=8, hd=64, bs=16,
             dtype="bf16", sinks=True, lens=5),
        # long contexts, 8 drafts, 32 requests
        dict(name="attend_verify_32k", op="attend", B=32, n=9, n_hi=9, ctx=32768, ctx_hi=32768, H=32, G=8, hd=128, bs=16,
             dtype="bf16", sinks=False, lens=6),
        # a whole prompt in one chunk
        dict(name="attend_prompt_8k", op="attend", B=1, n=8192, n_hi=8192, ctx=0, ctx_hi=0, H=64, G=8, hd=64, bs=16,
             dtype="bf16", sinks=False, lens=7),
        # prompt chunks of several requests on top of what they have cached, some requests with no rows in this pass
        dict(name="attend_chunks_mixed", op="attend", B=16, n=0, n_hi=1031, ctx=0, ctx_hi=6007, H=32, G=8, hd=128, bs=32,
             dtype="bf16", sinks=False, lens=8),
        # the fp32 layer
        dict(name="attend_f32_odd", op="attend", B=5, n=1, n_hi=37, ctx=0, ctx_hi=300, H=4, G=2, hd=16, bs=4, dtype="f32",
             sinks=True, lens=9),
        # one request's 8 verify rows, fp32 logits
        dict(name="verify_b1_k7", op="verify", B=1, n=8, n_hi=8, V=201088, dtype="f32", greedy=0.0, lens=10),
        # concurrency 64, bf16 logits, some requests greedy
        dict(name="verify_b64_k7", op="verify", B=64, n=8, n_hi=8, V=201088, dtype="bf16", greedy=0.2, lens=11),
        # ragged requests over a vocabulary whose rows start off the 16-byte grid
        dict(name="verify_ragged", op="verify", B=33, n=1, n_hi=9, V=32003, dtype="f32", greedy=0.1, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges: sizes spread over their logarithm, odd ones among them."""
    op = rng.choice(["append", "attend", "attend", "verify"])
    lens = rng.randrange(1 << 30)
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    if op == "append":
        H, G, hd = rng.choice([(4, 2, 16), (8, 2, 64), (6, 3, 40)] if dtype == "f32" else
                              [(64, 8, 64), (32, 8, 128), (28, 4, 128), (8, 2, 64), (5, 5, 64)])
        return dict(op=op, T=_log(rng, 1, 8192), H=H, G=G, hd=hd, bs=rng.choice([4, 16, 32, 64]), dtype=dtype,
                    norm=rng.random() < 0.5, pos=_log(rng, 1, 1 << 20), lens=lens)
    if op == "attend":
        if dtype == "f32":
            H, G, hd = rng.choice([(4, 2, 16), (8, 2, 64), (6, 3, 40)])
            return dict(op=op, B=_log(rng, 1, 8), n=0, n_hi=_log(rng, 1, 64), ctx=0, ctx_hi=_log(rng, 1, 1000), H=H, G=G,
                        hd=hd, bs=rng.choice([4, 16]), dtype=dtype, sinks=rng.random() < 0.5, lens=lens)
        H, G, hd = rng.choice([(64, 8, 64), (32, 8, 128), (28, 4, 128), (8, 2, 64), (5, 5, 64)])
        if rng.random() < 0.6:  # decoding and verification: few rows each
            B, n_hi = _log(rng, 1, 64), rng.choice([1, 1, 4, 8, 9])
            n, ctx_hi = rng.choice([1, n_hi]), _log(rng, 16, 32768 if B <= 24 else 8192)
        else:  # chunks of prompts
            B = _log(rng, 1, 12)
            n_hi = _log(rng, 32, 4096 // B + 64)
            n, ctx_hi = rng.choice([0, n_hi]), _log(rng, 1, 8192)
        return dict(op=op, B=B, n=n, n_hi=n_hi, ctx=rng.choice([0, ctx_hi]), ctx_hi=ctx_hi, H=H, G=G, hd=hd,
                    bs=rng.choice([16, 32, 64]), dtype=dtype, sinks=rng.random() < 0.3, lens=lens)
    n_hi = rng.choice([1, 4, 8, 9])
    return dict(op=op, B=_log(rng, 1, 64), n=rng.choice([0, 1, n_hi]), n_hi=n_hi, V=_log(rng, 2, 180000), dtype=dtype,
                greedy=rng.choice([0.0, 0.3]), lens=lens)


def _lengths(c):
    """Rows and prior context of each request, from the case alone (so that work() knows them)."""
    r = random.Random(c["lens"])
    n = [r.randint(c["n"], c["n_hi"]) for _ in range(c["B"])]
    if sum(n) == 0:
        n[0] = 1
    ctx = [r.randint(c["ctx"], c["ctx_hi"]) for _ in range(c["B"])] if "ctx" in c else [0] * c["B"]
    return n, ctx


def work(c):
    if c["op"] == "verify":
        n, _ = _lengths(c)
        e = 4 if c["dtype"] == "f32" else 2
        t = sum(n)
        # every logit once, the noise of one row a request, the row tokens and numbers, the results
        b = t * c["V"] * e + _sampled(c) * c["V"] * 4 + t * 12 + c["B"] * 16
        return {"bytes": b, "flops": 4.0 * t * c["V"]}
    e = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "append":
        v = c["T"] * (c["H"] + 2 * c["G"]) * c["hd"]
        return {"bytes": 2.0 * v * e + c["T"] * 16 + 2 * c["hd"] * e, "flops": 8.0 * v}
    n, ctx = _lengths(c)
    rows = sum(n)
    kv = sum(2 * (x + m) * c["G"] * c["hd"] * e + (x + m + c["bs"] - 1) // c["bs"] * 4 for x, m in zip(ctx, n) if m)
    pairs = sum(m * x + m * (m + 1) // 2 for x, m in zip(ctx, n))
    return {"bytes": 2.0 * rows * c["H"] * c["hd"] * e + kv, "flops": 4.0 * pairs * c["H"] * c["hd"]}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _dt(c):
    return torch.float32 if c["dtype"] == "f32" else torch.bfloat16


def _randn(g, shape, dt, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dt)


def _plan(c):
    from speculative_drafting_gb300 import binding

    return binding.PagedAttention(c["H"], c["G"], c["hd"], c["bs"], dtype=c["dtype"])


def _offsets(n):
    return torch.tensor([0] + n, device=DEV).cumsum(0).to(torch.int32)


def prepare(c, seed):
    return {"append": _prepare_append, "attend": _prepare_attend, "verify": _prepare_verify}[c["op"]](c, seed)


def _prepare_append(c, seed):
    g, dt = _gen(seed), _dt(c)
    T, H, G, hd, bs = c["T"], c["H"], c["G"], c["hd"], c["bs"]
    nb = (T + bs - 1) // bs + 3
    s = dict(c=c, qkv=_randn(g, (T, (H + 2 * G) * hd), dt, 1.5),
             gq=_randn(g, (hd,), dt, 0.1) + 1 if c["norm"] else None, gk=_randn(g, (hd,), dt, 0.1) + 1 if c["norm"] else None,
             pos=c["pos"] + torch.arange(T, device=DEV, dtype=torch.int64),
             slot=torch.randperm(nb * bs, generator=g, device=DEV)[:T].to(torch.int64),
             k=_randn(g, (nb, G, bs, hd), dt), v=_randn(g, (nb, G, bs, hd), dt), nb=nb)
    # rejected rows have slot -1: their keys and values are not written
    s["slot"][torch.rand(T, generator=g, device=DEV) < 0.1] = -1
    s["q"] = torch.empty(T, H, hd, dtype=dt, device=DEV)
    if own:
        s["plan"] = _plan(c)
        s["ws"] = s["plan"].append_workspace()
    return s


def _prepare_attend(c, seed):
    g, dt = _gen(seed), _dt(c)
    B, H, G, hd, bs = c["B"], c["H"], c["G"], c["hd"], c["bs"]
    n, ctx = _lengths(c)
    blocks = [(x + m + bs - 1) // bs for x, m in zip(ctx, n)]
    mb, nb = max(max(blocks), 1), sum(blocks) + 2
    # the pages of a request lie anywhere in the pool; entries past its last page are never read
    ids = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    at = torch.arange(mb, device=DEV)[None, :]
    first = torch.tensor([0] + blocks, device=DEV).cumsum(0)[:B, None]
    have = at < torch.tensor(blocks, device=DEV)[:, None]
    table = torch.where(have, ids[(first + at).clamp(max=nb - 1)], torch.full((), -1, dtype=torch.int32, device=DEV))
    T = sum(n)
    s = dict(c=c, T=T, nmax=max(n), qsl=_offsets(n), seq=torch.tensor([x + m for x, m in zip(ctx, n)], device=DEV, dtype=torch.int32),
             table=table.contiguous(), nb=nb, q=_randn(g, (T, H, hd), dt), k=_randn(g, (nb, G, bs, hd), dt),
             v=_randn(g, (nb, G, bs, hd), dt), sink=_randn(g, (H,), torch.float32) if c["sinks"] else None)
    s["out"] = torch.empty(T, H * hd, dtype=dt, device=DEV)
    if own:
        s["plan"] = _plan(c)
        s["ws"] = s["plan"].workspace(B, T)
    return s


def _sampled(c):
    r = random.Random(c["lens"] + 1)
    return sum(r.random() >= c["greedy"] for _ in range(c["B"]))


def _prepare_verify(c, seed):
    g, dt = _gen(seed), _dt(c)
    B, V = c["B"], c["V"]
    n, _ = _lengths(c)
    T, qsl = sum(n), _offsets(n)
    r = random.Random(c["lens"] + 1)
    temp = [0.0 if r.random() < c["greedy"] else r.choice([0.6, 0.8, 1.0, 1.3]) for _ in range(B)]
    logits = torch.randn(T, V, generator=g, device=DEV) * 2
    # a few tokens are barred, as by a grammar or a nucleus cut
    logits[torch.rand(T, V, generator=g, device=DEV) < 0.01] = -math.inf
    tok = torch.randint(0, V, (T,), generator=g, device=DEV, dtype=torch.int64)
    # the target gives most drafts a large share: row i - 1 scores the token of row i
    share = torch.rand(T, generator=g, device=DEV) * 0.75 + 0.2
    lift = torch.logsumexp(logits, -1) + torch.log(share / (1 - share))
    rows = torch.arange(T - 1, device=DEV)
    logits[rows, tok[1:]] = lift[:-1]
    s = dict(c=c, T=T, nmax=max(n), qsl=qsl, tok=tok.to(torch.int32), logits=logits.to(dt),
             temp=torch.tensor(temp, device=DEV, dtype=torch.float32), u=torch.rand(T, generator=g, device=DEV),
             gumbel=-torch.log(torch.empty(B, V, device=DEV).exponential_(generator=g)))
    s["accepted"] = torch.empty(B, dtype=torch.int32, device=DEV)
    s["bonus"] = torch.empty(B, dtype=torch.int32, device=DEV)
    s["p"] = torch.empty(T, dtype=torch.float32, device=DEV)
    if own:
        from speculative_drafting_gb300 import binding

        s["ws"] = binding.verify_sampled_workspace(B, T, V)
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    return {"append": _run_append, "attend": _run_attend, "verify": _run_verify}[s["c"]["op"]](s)


def _run_append(s):
    c = s["c"]
    if own:
        s["plan"].append(c["T"], s["qkv"], s["gq"], s["gk"], s["pos"], s["slot"], s["nb"], s["q"], s["k"], s["v"], s["ws"])
        return {"q": s["q"], "k_cache": s["k"], "v_cache": s["v"]}
    T, H, G, hd, bs = c["T"], c["H"], c["G"], c["hd"], c["bs"]
    x = s["qkv"].view(T, H + 2 * G, hd)
    # angles of far positions: 64 bits, reduced to one turn before cos and sin
    freq = torch.pow(10000.0, -torch.arange(0, hd, 2, device=DEV, dtype=torch.float64) / hd)
    a = torch.remainder(s["pos"].double()[:, None] * freq, 2 * math.pi)
    cs, sn = torch.cos(a).float()[:, None, :], torch.sin(a).float()[:, None, :]
    q = _norm_rotate(x[:, :H], s["gq"], cs, sn)
    k = _norm_rotate(x[:, H:H + G], s["gk"], cs, sn)
    s["q"].copy_(q)
    keep = torch.nonzero(s["slot"] >= 0)[:, 0]
    blk, at = s["slot"][keep] // bs, s["slot"][keep] % bs
    s["k"][blk, :, at] = k[keep].to(s["k"].dtype)
    s["v"][blk, :, at] = x[keep, H + G:]
    return {"q": s["q"], "k_cache": s["k"], "v_cache": s["v"]}


def _norm_rotate(x, gain, cs, sn):
    x = x.float()
    if gain is not None:
        x = x * gain.float() / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    lo, hi = x.chunk(2, -1)
    return torch.cat([lo * cs - hi * sn, hi * cs + lo * sn], -1)


def _run_attend(s):
    c = s["c"]
    if own:
        s["plan"].attend(c["B"], s["T"], s["qsl"], s["seq"], s["q"], s["k"], s["v"], s["table"], s["nb"], s["out"], s["ws"],
                         sink=s["sink"])
        return s["out"]
    B, H, G, hd = c["B"], c["H"], c["G"], c["hd"]
    q, k, v, ok, row, req = _gathered(s, torch.float32)
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
    s["out"].copy_(o[req, row].reshape(s["T"], H * hd))
    return s["out"]


def _gathered(s, dt):
    """The requests side by side: queries [B, n, G, H/G, hd], keys and values [B, t, G, hd], which key each row sees, and
    where each of the T rows lies."""
    c = s["c"]
    B, H, G, hd = c["B"], c["H"], c["G"], c["hd"]
    qsl = s["qsl"].long()
    n = qsl[1:] - qsl[:-1]
    j = torch.arange(s["nmax"], device=DEV)
    q = s["q"][(qsl[:-1, None] + j).clamp(max=s["T"] - 1)].to(dt).view(B, s["nmax"], G, H // G, hd)
    table = s["table"].long().clamp(min=0)
    k, v = (x[table].transpose(2, 3).reshape(B, -1, G, hd).to(dt) for x in (s["k"], s["v"]))
    seq = s["seq"].long()
    ok = torch.arange(k.shape[1], device=DEV)[None, None, :] <= (seq - n)[:, None, None] + j[None, :, None]
    ok &= torch.arange(k.shape[1], device=DEV)[None, None, :] < seq[:, None, None]
    t = torch.arange(s["T"], device=DEV)
    req = torch.searchsorted(qsl, t, right=True) - 1
    return q, k, v, ok, t - qsl[req], req


def _run_verify(s):
    c = s["c"]
    if own:
        from speculative_drafting_gb300 import binding

        binding.verify_sampled(c["B"], s["T"], s["qsl"], s["tok"], s["logits"], c["V"], _code(binding, c), s["temp"], s["u"],
                               s["gumbel"], s["accepted"], s["bonus"], s["p"], s["ws"])
        return {"accepted": s["accepted"], "bonus": s["bonus"], "p": s["p"]}
    qsl = s["qsl"].long()
    n = qsl[1:] - qsl[:-1]
    t = torch.arange(s["T"], device=DEV)
    req = torch.searchsorted(qsl, t, right=True) - 1
    cold = s["temp"][req] == 0
    # 64 bits: the numbers decide between tokens
    x = s["logits"].double() / torch.where(cold, 1.0, s["temp"][req]).double()[:, None]
    top = x.amax(-1)
    lse = top + torch.log(torch.exp(x - top[:, None]).sum(-1))
    pick = x.argmax(-1)
    before = (t - 1).clamp(min=0)
    tok = s["tok"].long()
    p = torch.where(cold, (pick[before] == tok).double(), torch.exp(x[before, tok] - lse[before]))
    p[t == qsl[req]] = 1.0
    # the longest run of accepted drafts of each request
    j = torch.arange(s["nmax"], device=DEV)[None, :] + 1
    at = (qsl[:-1, None] + j).clamp(max=s["T"] - 1)
    ok = (s["u"][at].double() < p[at]) & (j < n[:, None])
    a = torch.where(n > 0, ok.long().cumprod(-1).sum(-1), 0)
    # the token after it: the target's, without the rejected draft
    row = (qsl[:-1] + a).clamp(max=s["T"] - 1)
    cold_r = (s["temp"] == 0)[:, None]
    score = x[row] + torch.where(cold_r, 0.0, s["gumbel"].double())
    nxt = tok[(row + 1).clamp(max=s["T"] - 1)]
    out = (a + 1 < n) & ~cold_r[:, 0]
    r = torch.arange(c["B"], device=DEV)
    score[r, nxt] = torch.where(out, -math.inf, score[r, nxt])
    bonus = torch.where(n > 0, score.argmax(-1), -1)
    s["accepted"].copy_(a)
    s["bonus"].copy_(bonus)
    s["p"].copy_(p)
    return {"accepted": s["accepted"], "bonus": s["bonus"], "p": s["p"]}


def _code(binding, c):
    return binding.PE_DTYPE_F32 if c["dtype"] == "f32" else binding.PE_DTYPE_BF16


# ------------------------------------------------------------------ from the definitions, in 64 bits


def exact(c, seed):
    s = prepare(c, seed)
    return {"append": _exact_append, "attend": _exact_attend, "verify": _exact_verify}[c["op"]](s)


def _exact_append(s):
    """The pair (i, i + hd/2) of a head as a complex number, turned by e^(i pos theta^(-2i/hd))."""
    c = s["c"]
    H, G, hd, bs = c["H"], c["G"], c["hd"], c["bs"]
    x = s["qkv"].double().view(c["T"], H + 2 * G, hd)
    half = hd // 2
    rate = torch.tensor([10000.0 ** (-2.0 * i / hd) for i in range(half)], dtype=torch.float64, device=DEV)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), s["pos"].double()[:, None, None] * rate)

    def head(y, gain):
        if gain is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * gain.double()
        z = torch.complex(y[..., :half], y[..., half:]) * turn
        return torch.cat([z.real, z.imag], -1)

    k, v = s["k"].double(), s["v"].double()
    kk = head(x[:, H:H + G], s["gk"])
    rows = [i for i, m in enumerate(s["slot"].tolist()) if m >= 0]
    slots = s["slot"][rows]
    k[slots // bs, :, slots % bs] = kk[rows]
    v[slots // bs, :, slots % bs] = x[rows, H + G:]
    return {"q": head(x[:, :H], s["gq"]), "k_cache": k, "v_cache": v}


def _exact_attend(s):
    """Request by request and KV head by KV head."""
    c = s["c"]
    H, G, hd, bs = c["H"], c["G"], c["hd"], c["bs"]
    out = torch.zeros(s["T"], H, hd, dtype=torch.float64, device=DEV)
    qsl, seq = s["qsl"].tolist(), s["seq"].tolist()
    for r in range(c["B"]):
        n, L = qsl[r + 1] - qsl[r], seq[r]
        if n == 0 or L == 0:
            continue
        pages = s["table"][r, : (L + bs - 1) // bs].long()
        sees = torch.ones(n, L, dtype=torch.bool, device=DEV).tril(L - n)
        for g in range(G):
            k = s["k"][pages, g].reshape(-1, hd)[:L].double()
            v = s["v"][pages, g].reshape(-1, hd)[:L].double()
            for h in range(g * (H // G), (g + 1) * (H // G)):
                x = (s["q"][qsl[r]:qsl[r + 1], h].double() @ k.T) * hd ** -0.5
                x[~sees] = -math.inf
                if s["sink"] is not None:
                    x = torch.cat([x, s["sink"][h].double().expand(n, 1)], 1)
                out[qsl[r]:qsl[r + 1], h] = torch.softmax(x, -1)[:, :L] @ v
    return out.view(s["T"], H * hd)


def _exact_verify(s):
    """Request by request, draft by draft."""
    c = s["c"]
    qsl, tok, u = s["qsl"].tolist(), s["tok"].tolist(), s["u"].tolist()
    acc, bon, p = [], [], [1.0] * s["T"]
    for r, t in enumerate(s["temp"].tolist()):
        lo, hi = qsl[r], qsl[r + 1]
        if lo == hi:
            acc.append(0)
            bon.append(-1)
            continue
        y = s["logits"][lo:hi].double()
        if t == 0:
            prob = torch.zeros_like(y)
            prob[torch.arange(hi - lo, device=DEV), torch.max(y, -1).indices] = 1.0
        else:
            prob = torch.softmax(y / t, -1)
        took = prob[torch.arange(hi - lo - 1, device=DEV), s["tok"][lo + 1:hi].long()].tolist()
        p[lo + 1:hi] = took
        a = 0
        while a < hi - lo - 1 and u[lo + a + 1] < took[a]:
            a += 1
        if t == 0:
            bon.append(int(prob[a].argmax()))
        else:
            score = torch.log(prob[a]) + s["gumbel"][r].double()
            if a < hi - lo - 1:
                score[tok[lo + a + 1]] = -math.inf
            bon.append(int(score.argmax()))
        acc.append(a)
    return {"accepted": torch.tensor(acc, dtype=torch.int32), "bonus": torch.tensor(bon, dtype=torch.int32),
            "p": torch.tensor(p, dtype=torch.float64)}
