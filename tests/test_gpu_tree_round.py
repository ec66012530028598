"""The tree, sampling and page calls together, as a serving engine runs them."""

import numpy as np
import pytest

from oracle import pe_oracle as O
from oracle import pe_paged as P
from oracle import pe_tree as X
from parity import built, cuda_or_skip, host, setup
from speculative_drafting_gb300 import binding, runner
from test_gpu_tree import tree

pytestmark = pytest.mark.gpu

H, G, HD, BS, D, V, LAYERS = 8, 2, 64, 16, 128, 997, 3


class Engine:
    """A target of LAYERS layers (the same weights in each) over a pool of pages; requests by row of the table."""

    def __init__(self, rows=8, max_blocks=12, num_blocks=90, seed=0):
        self.torch = torch = cuda_or_skip()
        built()
        torch.manual_seed(seed)
        bf = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
        self.w_qkv, self.w_o, self.w_lm = bf((H + 2 * G) * HD, D) * D ** -0.5, bf(D, H * HD) * 0.05, bf(V, D) * 0.2
        self.emb = bf(V, D)
        self.plan = binding.PagedAttention(H, G, HD, BS)
        self.k, self.v = (torch.full((LAYERS, num_blocks, G, BS, HD), float("nan"), dtype=torch.bfloat16, device="cuda")
                          for _ in range(2))
        self.nb = num_blocks
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table, self.refs = torch.full((rows, max_blocks), -1, **i32), torch.zeros(num_blocks, **i32)
        self.wp = binding.pages_workspace(rows, num_blocks)
        self.wa, self.wt = self.plan.append_workspace(), torch.zeros(256, dtype=torch.uint8, device="cuda")

    def i32(self, x):
        return self.torch.tensor(np.asarray(x), dtype=self.torch.int32, device="cuda")

    def layers(self, x, pos, slot, attend):
        """x after the layers; every row's keys and values are written first."""
        torch, T = self.torch, len(x)
        for i in range(LAYERS):
            q, att = torch.empty(T, H, HD, dtype=x.dtype, device="cuda"), torch.empty(T, H * HD, dtype=x.dtype, device="cuda")
            self.plan.append(T, x @ self.w_qkv.T, None, None, pos, slot, self.nb, q, self.k[i], self.v[i], self.wa)
            attend(q, self.k[i], self.v[i], att)
            x = (x.float() + (att @ self.w_o.T).float()).bfloat16()
        return (x @ self.w_lm.T).float()

    def prefill(self, rows, prompts):
        """Prompts into rows of the table; logits of every position."""
        torch = self.torch
        n = [len(p) for p in prompts]
        binding.pages_reserve(len(rows), self.i32(rows), self.i32(n), self.table, self.refs, BS, self.wp)
        qsl = self.i32(np.concatenate([[0], np.cumsum(n)]))
        table = self.table[torch.tensor(rows, device="cuda")].contiguous()
        ws = self.plan.workspace(len(rows), sum(n))
        pos = torch.cat([torch.arange(x, device="cuda") for x in n])
        req = torch.repeat_interleave(torch.arange(len(rows), device="cuda"), torch.tensor(n, device="cuda"))
        slot = table[req, pos // BS].long() * BS + pos % BS
        tok = torch.tensor(np.concatenate(prompts), device="cuda")
        out = self.layers(self.emb[tok], pos, slot, lambda q, k, v, o: self.plan.attend(
            len(rows), sum(n), qsl, self.i32(n), q, k, v, table, self.nb, o, ws))
        assert binding.read_status_ws(ws)[0] == 0
        return out


def test_verification_of_a_tree_leaves_what_its_accepted_line_would():
    """Prompts, then one round over trees: the logits of the accepted nodes, and the cache of every layer after it,
    are those of a prefill of prompt and accepted line; sampled tokens decide the walk."""
    e = Engine()
    torch = e.torch
    rng = np.random.default_rng(1)
    rows, ctx = [5, 0, 3], [37, 16, 3]
    prompts = [rng.integers(0, V, n) for n in ctx]
    e.prefill(rows, prompts)
    ns = [33, 9, 40]
    B, T = 3, sum(ns)
    parent = [p for n in ns for p in tree(rng, n, chain=0.4)]
    tok = rng.integers(0, V, T).astype(np.int32)
    qsl, seq = e.i32(np.concatenate([[0], np.cumsum(ns)])), e.i32([c + n for c, n in zip(ctx, ns)])
    binding.pages_reserve(B, e.i32(rows), seq, e.table, e.refs, BS, e.wp)
    table = e.table[torch.tensor(rows, device="cuda")].contiguous()
    mask = torch.empty(T, 2, dtype=torch.int32, device="cuda")
    pos, slot = (torch.empty(T, dtype=torch.int64, device="cuda") for _ in range(2))
    d_parent, d_tok = e.i32(parent), e.i32(tok)
    binding.tree_layout(B, T, qsl, seq, d_parent, table, e.nb, BS, mask, pos, slot, e.wt)
    ws = e.plan.workspace(B, T)
    attend = lambda q, k, v, o: e.plan.attend_tree(B, T, qsl, seq, q, k, v, table, e.nb, mask, o, ws)  # noqa: E731
    logits = e.layers(e.emb[d_tok.long()], pos, slot, attend)
    # the target's tokens, some of them the tree's: a child's token is favoured
    boost = logits.clone()
    for j, p in enumerate(parent):
        if p >= 0 and rng.random() < 0.7:
            r = int(np.searchsorted(np.cumsum(ns), j, side="right"))
            boost[int(qsl[r]) + p, tok[j]] += 25.0
    gumbel = -torch.log(torch.empty(T, V, device="cuda").exponential_())
    target, path = (torch.empty(T, dtype=torch.int32, device="cuda") for _ in range(2))
    accepted, bonus = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    temp, k, p = torch.tensor([0.8, 0.0, 1.0], device="cuda"), e.i32([20, 0, 0]), torch.tensor([0.9, 1.0, 0.8], device="cuda")
    wss = binding.sample_workspace(B, T, V)
    binding.sample(B, T, qsl, boost, V, temp, k, p, None, gumbel, target, wss)
    binding.tree_accept(B, T, qsl, d_parent, d_tok, target, accepted, path, bonus, e.wt)
    before = e.k.clone(), e.v.clone()
    e.plan.compact(LAYERS, B, T, qsl, seq, accepted, path, table, e.nb, e.k, e.v, e.wa)
    torch.cuda.synchronize()
    assert [binding.read_status_ws(w)[0] for w in (e.wp, e.wt, e.wa, ws, wss)] == [0] * 5
    # each call against the oracle on what it was given
    want, clear = X.sample(host(qsl), host(boost), host(temp), host(k), host(p), None, host(gumbel))
    assert clear.mean() > 0.9 and (host(target)[clear] == want[clear]).all()
    acc, way, bon = X.tree_accept(host(qsl), parent, tok, host(target))
    np.testing.assert_array_equal(host(accepted), acc)
    np.testing.assert_array_equal(host(path), way)
    np.testing.assert_array_equal(host(bonus), bon)
    assert acc.max() >= 3
    nodes = [way[int(qsl[r]):int(qsl[r]) + acc[r] + 1] for r in range(B)]
    # a request that has the prompt and the accepted line as its prompt
    other = Engine()
    lines = [np.concatenate([prompts[r], tok[int(qsl[r]) + nodes[r]]]) for r in range(B)]
    again = other.prefill(rows, lines)
    at = 0
    for r in range(B):
        n, c = len(lines[r]), ctx[r]
        a = logits[int(qsl[r]) + torch.tensor(nodes[r], device="cuda")].cpu().numpy()
        b = again[at + c:at + n].cpu().numpy()
        # two computations of the same rows in bf16 through three layers: each layer rounds weights and rows to
        # 2^-8 of their size, |x| is about 11 = sqrt(D), and a logit weighs D of its entries by 0.2
        assert np.abs(a - b).max() <= 6 * 2.0 ** -8 * 0.2 * np.sqrt(D) * 11, r
        at += n
        for mine, his in ((e.k, other.k), (e.v, other.v)):
            t = np.arange(n)
            x = O.decode(host(mine), "bf16")[:, host(e.table)[rows[r]][t // BS], :, t % BS]
            y = O.decode(host(his), "bf16")[:, host(other.table)[rows[r]][t // BS], :, t % BS]
            np.testing.assert_allclose(x, y, atol=6 * 2.0 ** -8 * 4)
    # nothing but the accepted nodes' slots has moved
    slots = {(int(host(table)[r][(ctx[r] + d) // BS]), (ctx[r] + d) % BS) for r in range(B) for d in range(1, acc[r] + 1)}
    for now, was in ((e.k, before[0]), (e.v, before[1])):
        now, was = host(now).copy(), host(was).copy()
        for blk, off in slots:
            now[:, blk, :, off] = was[:, blk, :, off] = 0
        np.testing.assert_array_equal(now, was)


def test_samples_of_one_prompt_decode_on_shared_pages():
    """A prompt forked into three rows that decode different tokens: each row's attention is that of a prompt of its
    own, and freeing all but one leaves its pages."""
    e = Engine()
    torch = e.torch
    rng = np.random.default_rng(2)
    prompt = rng.integers(0, V, 37)
    e.prefill([2], [prompt])
    e.plan.fork(LAYERS, 2, e.i32([2, 2]), e.i32([6, 1]), e.i32([37, 37]), e.table, e.refs, e.k, e.v, e.wp)
    rows, more = [2, 6, 1], rng.integers(0, V, (3, 12))
    for step in range(12):
        seq = e.i32([38 + step] * 3)
        binding.pages_reserve(3, e.i32(rows), seq, e.table, e.refs, BS, e.wp)
        table = e.table[torch.tensor(rows, device="cuda")].contiguous()
        pos = torch.full((3,), 37 + step, device="cuda")
        slot = table[torch.arange(3, device="cuda"), pos // BS].long() * BS + pos % BS
        ws = e.plan.workspace(3, 3)
        x = e.emb[torch.tensor(more[:, step], device="cuda")]
        logits = e.layers(x, pos, slot, lambda q, k, v, o: e.plan.attend(3, 3, e.i32([0, 1, 2, 3]), seq, q, k, v, table, e.nb, o, ws))
    assert binding.read_status_ws(e.wp)[0] == 0
    refs, table = host(e.refs), host(e.table)
    assert (refs[table[2][:2]] == 3).all() and len({int(table[r][2]) for r in rows}) == 3
    other = Engine()
    again = other.prefill([0, 1, 2], [np.concatenate([prompt, more[i]]) for i in range(3)])
    a, b = logits.cpu().numpy(), again[[48, 97, 146]].cpu().numpy()
    assert np.abs(a - b).max() <= 6 * 2.0 ** -8 * 0.2 * np.sqrt(D) * 11
    binding.pages_free(2, e.i32([2, 6]), e.table, e.refs, e.wp)
    refs, table = host(e.refs), host(e.table)
    assert refs.sum() == 4 and (refs[table[1][:4]] == 1).all() and (table[2] == -1).all()
    # its pages elsewhere, contents and all
    src = table[1][:4].copy()
    dst = [x for x in range(e.nb) if refs[x] == 0][-4:]
    was = host(e.k)[:, src].copy()
    e.plan.copy_pages(LAYERS, 4, e.i32(src), e.i32(dst), e.nb, e.k, e.v, e.wa)
    np.testing.assert_array_equal(host(e.k)[:, dst], was)


def test_a_round_in_a_graph_follows_its_inputs():
    """The round captured once and replayed on other trees, lengths and noise equals the calls one by one."""
    torch = cuda_or_skip()
    built()
    rng = np.random.default_rng(3)
    B, N, nb = 4, 24, 80
    T = B * N
    plan = binding.PagedAttention(H, G, HD, BS)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731

    def inputs(seed):
        r = np.random.default_rng(seed)
        ns = [int(x) for x in r.integers(0, N + 1, B)]
        g = torch.Generator(device="cuda").manual_seed(seed)
        parent = [p for n in ns for p in tree(r, n)]
        return dict(qsl=i32(np.concatenate([[0], np.cumsum(ns)])), seq=i32([n + int(r.integers(0, 150)) for n in ns]),
                    parent=i32(parent + [0] * (T - len(parent))), tok=i32(r.integers(0, 5, T)),
                    table=i32(r.permutation(nb)[:B * 14].reshape(B, 14)),
                    q=torch.randn(T, H, HD, generator=g, device="cuda").bfloat16(),
                    k=torch.randn(nb, G, BS, HD, generator=g, device="cuda").bfloat16(),
                    v=torch.randn(nb, G, BS, HD, generator=g, device="cuda").bfloat16(),
                    logits=torch.randn(T, 5, generator=g, device="cuda") * 3,
                    gumbel=-torch.log(torch.empty(T, 5, device="cuda").exponential_(generator=g)))

    def outputs():
        return dict(mask=torch.zeros(T, 1, dtype=torch.int32, device="cuda"), pos=torch.zeros(T, dtype=torch.int64, device="cuda"),
                    slot=torch.zeros(T, dtype=torch.int64, device="cuda"), out=torch.zeros(T, H * HD, device="cuda").bfloat16(),
                    target=i32([0] * T), accepted=i32([0] * B), path=i32([0] * T), bonus=i32([0] * B))

    temp, top_k, top_p = torch.full((B,), 0.7, device="cuda"), i32([3, 0, 2, 4]), torch.tensor([1.0, 0.8, 0.9, 1.0], device="cuda")

    def work():
        return plan.workspace(B, T), binding.sample_workspace(B, T, 5), torch.zeros(256, dtype=torch.uint8, device="cuda")

    def round_(x, y, w, st=None):
        binding.tree_layout(B, T, x["qsl"], x["seq"], x["parent"], x["table"], nb, BS, y["mask"], y["pos"], y["slot"], w[2], stream=st)
        plan.attend_tree(B, T, x["qsl"], x["seq"], x["q"], x["k"], x["v"], x["table"], nb, y["mask"], y["out"], w[0], stream=st)
        binding.sample(B, T, x["qsl"], x["logits"], 5, temp, top_k, top_p, None, x["gumbel"], y["target"], w[1], stream=st)
        binding.tree_accept(B, T, x["qsl"], x["parent"], x["tok"], y["target"], y["accepted"], y["path"], y["bonus"], w[2], stream=st)
        plan.compact(1, B, T, x["qsl"], x["seq"], y["accepted"], y["path"], x["table"], nb, x["k"], x["v"], w[2], stream=st)

    x, y, w = inputs(0), outputs(), work()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    round_(inputs(9), outputs(), work(), s)  # (a launch of every kernel before the capture)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        round_(x, y, w, s)
    for seed in (1, 2, 3, 4):
        fresh = inputs(seed)
        for k, t in fresh.items():
            x[k].copy_(t)
        for t in y.values():
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        z = outputs()
        round_(fresh, z, work())
        torch.cuda.synchronize()
        for k in y:
            assert torch.equal(y[k], z[k]), (seed, k)
        assert torch.equal(x["k"], fresh["k"]) and torch.equal(x["v"], fresh["v"])
        assert [binding.read_status_ws(t)[0] for t in w] == [0, 0, 0]


def test_the_accepted_line_feeds_the_next_draft_step():
    """pe_prepare_inputs takes the accepted line as its verify rows: rows picked by path, counts and bonus tokens as the
    walk left them; its metadata is the oracle's for that line."""
    torch = cuda_or_skip()
    wl, b, w, kc, vc, r = setup("small_prenorm")
    dm = wl.dims
    B, T = b["B"], b["T_in"]
    ns = np.diff(b["qsl"])
    rng = np.random.default_rng(5)
    parent = np.array([p for n in ns for p in tree(rng, int(n), chain=0.5)], np.int32)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    target = rng.integers(0, dm.vocab, T).astype(np.int32)
    tok = b["prev_tok"].copy()
    for rr in range(B):  # most nodes agree with what the target says after their parent
        lo = int(b["qsl"][rr])
        for j in range(1, int(ns[rr])):
            if rng.random() < 0.8 and parent[lo + j] >= 0:
                tok[lo + j] = target[lo + parent[lo + j]]
    acc, bon = i32([0] * B), i32([0] * B)
    path, ws = i32([0] * T), torch.zeros(256, dtype=torch.uint8, device="cuda")
    binding.tree_accept(B, T, i32(b["qsl"]), i32(parent), i32(tok), i32(target), acc, path, bon, ws)
    a = host(acc)
    assert a.max() > 0
    # the line's rows first, then the others, which the draft step treats as rejected
    order = np.concatenate([lo + np.concatenate([(p := host(path)[lo:hi])[:a[rr] + 1],
                                                 np.setdiff1d(np.arange(hi - lo), p[:a[rr] + 1])]).astype(int)
                            for rr, (lo, hi) in enumerate(zip(b["qsl"][:-1], b["qsl"][1:]))])
    pos = np.concatenate([int(c) + np.arange(n) for c, n in zip(b["ctx"], ns)])
    batch = dict(b, prev_tok=tok[order], prev_pos=pos.astype(np.int64), H_tgt=b["H_tgt"][order])
    step = runner.StepRunner(wl, batch, w, kc, vc)
    step.inp["accepted"], step.inp["bonus"] = acc, bon
    step.run()
    torch.cuda.synchronize()
    assert step.status()[0] == 0
    meta = O.prepare_metadata(b["qsl"], tok[order], pos, a, host(bon), b["block_table"], dm.K, dm.mask_id, dm.block_size)
    for k in ("tok", "pos", "slot", "seq_len", "hidden_src"):
        np.testing.assert_array_equal(host(step.meta[k]), meta[k])


def test_chunk_and_tree_attention_share_a_workspace():
    """One workspace, calls of both kinds in turn on a stream."""
    torch = cuda_or_skip()
    built()
    plan = binding.PagedAttention(H, G, HD, BS)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn(40, G, BS, HD, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(60, H, HD, generator=g, device="cuda").bfloat16()
    qsl, seq, table = i32([0, 20, 60]), i32([300, 200]), i32(np.arange(40).reshape(2, 20))
    mask = i32(np.tril(np.ones((60, 32)))[:, :1] * 0 - 1).repeat(1, 2)
    ws = plan.workspace(2, 60)
    outs = [torch.zeros(60, H * HD, device="cuda").bfloat16() for _ in range(4)]
    for i in range(2):
        plan.attend(2, 60, qsl, seq, q, k, v, table, 40, outs[2 * i], ws)
        plan.attend_tree(2, 60, qsl, seq, q, k, v, table, 40, mask, outs[2 * i + 1], ws)
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    ref = P.chunk_attention(host(qsl), host(seq), O.decode(host(q), "bf16"), O.decode(host(k), "bf16"), O.decode(host(v), "bf16"),
                            host(table))
    assert (np.abs(O.decode(host(outs[0]), "bf16").reshape(ref[0].shape) - ref[0])
            <= 2.0 ** -8 * np.abs(ref[0]) + (2.0 ** -8 + 1e-4) * ref[1]).all()
    ref = X.tree_attention(host(qsl), host(seq), O.decode(host(q), "bf16"), O.decode(host(k), "bf16"),
                           O.decode(host(v), "bf16"), host(table), host(mask))
    assert (np.abs(O.decode(host(outs[1]), "bf16").reshape(ref[0].shape) - ref[0])
            <= 2.0 ** -8 * np.abs(ref[0]) + (2.0 ** -8 + 1e-4) * ref[1]).all()
