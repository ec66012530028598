"""Trees of drafts against the fp64 oracle: layout, attention, the walk.

Layout and walk are integers: equal.  Attention as in test_gpu_paged: bf16 weights may be
rounded to bf16 before their product with the value (relative 2^-8 each), scores carry fp32
rounding (below 1e-4 of a weight), then one rounding of the result: |got - ref| <= h |ref| +
(h + 1e-4) sum p |v| with h = 2^-8; in fp32 h = 2^-24 and 2e-5 for the scores.
"""

import numpy as np
import pytest

from oracle import pe_oracle as O
from oracle import pe_tree as X
from parity import built, cuda_or_skip, host
from speculative_drafting_gb300 import binding, runner, workloads as W

pytestmark = pytest.mark.gpu


def _store(x, dtype):
    return W.f32_to_bf16_bits(x.astype(np.float32)) if dtype == "bf16" else x.astype(np.float32)


def _dev(x, dtype="f32"):
    return runner.to_device(x, dtype)


def tree(rng, n, chain=0.3):
    """Parents of a random tree of n nodes, some stretches of it a chain."""
    return [-1 if j == 0 else j - 1 if rng.random() < chain else int(rng.integers(0, j)) for j in range(n)]


def case(dtype, H, G, hd, bs, ns, Ls, words=None, seed=0, sinks=False, pad=0, extra=0, poison=False, scale=1.0,
         table_edit=None, bits=None, spare=2):
    """Random pages and trees; poison: whatever no row sees is NaN or infinite."""
    rng = np.random.default_rng(seed)
    B, T = len(ns), sum(ns)
    qsl = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    blocks = [(max(L, 0) + bs - 1) // bs for L in Ls]
    mb, nb = max(max(blocks), 1) + 1, sum(blocks) + spare
    ids, table, o = rng.permutation(nb), np.full((B, mb), -1, np.int32), 0
    for r in range(B):
        table[r, :blocks[r]] = ids[o:o + blocks[r]]
        o += blocks[r]
    words = words or max((max(ns) + 31) // 32, 1)
    parent = np.array([p for n in ns for p in tree(rng, n)] + [0] * extra, np.int32)
    mask = X.tree_layout(qsl, Ls, parent, table, nb, bs, words)[0]
    if bits is not None:
        mask[:T] = bits(rng, mask[:T])
    kc, vc = (rng.standard_normal((nb, G, bs, hd)) for _ in range(2))
    if poison:
        seen = np.zeros((nb, bs), bool)
        for r in range(B):
            n = ns[r]
            t = np.arange(max(Ls[r], 0))
            if n:
                any_row = X.unpack(mask[qsl[r]:qsl[r + 1]]).any(0)
                node = t - (Ls[r] - n)
                t = t[(node < 0) | any_row[np.clip(node, 0, len(any_row) - 1)]]
                seen[table[r, t // bs], t % bs] = True
        for c in (kc, vc):
            c.transpose(0, 2, 1, 3)[~seen] = rng.choice([np.nan, np.inf, -np.inf], ((~seen).sum(), G, hd))
    if table_edit:
        table_edit(table, nb)
    q = rng.standard_normal((T + extra, H * hd + pad)) * scale
    sink = rng.standard_normal(H).astype(np.float32) if sinks else None
    return dict(dtype=dtype, H=H, G=G, hd=hd, bs=bs, qsl=qsl, seq=np.array(Ls, np.int32), q=_store(q, dtype),
                kc=_store(kc, dtype), vc=_store(vc, dtype), table=table, nb=nb, sink=sink, T=T + extra, mask=mask,
                parent=parent)


def attend(c, stream=None):
    torch = cuda_or_skip()
    built()
    plan = binding.PagedAttention(c["H"], c["G"], c["hd"], c["bs"], dtype=c["dtype"])
    d = {k: _dev(c[k], c["dtype"]) for k in ("q", "kc", "vc")}
    d |= {k: _dev(c[k]) for k in ("qsl", "seq", "table", "mask")}
    sink = None if c["sink"] is None else _dev(c["sink"])
    ws = plan.workspace(len(c["seq"]), c["T"])
    w = c["H"] * c["hd"]
    out = torch.full((c["T"], w + 8), 3.0, dtype=d["q"].dtype, device="cuda")[:, :w]
    torch.cuda.synchronize()
    plan.attend_tree(len(c["seq"]), c["T"], d["qsl"], d["seq"], d["q"], d["kc"], d["vc"], d["table"], c["nb"],
                     d["mask"], out, ws, sink=sink, stream=stream)
    torch.cuda.synchronize()
    return out, binding.read_status_ws(ws)[0]


def check(c, status=0):
    got, st = attend(c)
    assert st == status
    dtype, H, hd = c["dtype"], c["H"], c["hd"]
    q = O.decode(c["q"], dtype)[:, :H * hd].reshape(c["T"], H, hd)
    ref, spread = X.tree_attention(c["qsl"], c["seq"], q, O.decode(c["kc"], dtype), O.decode(c["vc"], dtype),
                                   c["table"], c["mask"], c["sink"])
    val = O.decode(host(got), dtype).reshape(c["T"], H, hd)
    rows = int(c["qsl"][-1])
    half, w = (2.0 ** -8, 2.0 ** -8 + 1e-4) if dtype == "bf16" else (2.0 ** -24, 2e-5)
    bad = ~(np.abs(val[:rows] - ref[:rows]) <= half * np.abs(ref[:rows]) + w * spread[:rows] + 1e-30)
    assert not bad.any(), (np.argwhere(bad)[:4], val[:rows][bad][:4], ref[:rows][bad][:4], bad.mean())
    assert (val[rows:] == 3.0).all()  # rows behind the last request
    return got


# ------------------------------------------------------------------ layout and walk


def run_layout(qsl, seq, parent, table, nb, bs, words, T, want=True):
    torch = cuda_or_skip()
    built()
    mask = torch.full((T, words), -7, dtype=torch.int32, device="cuda")
    pos, slot = (torch.full((T,), -7, dtype=torch.int64, device="cuda") for _ in range(2))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    binding.tree_layout(len(seq), T, _dev(qsl), _dev(np.asarray(seq, np.int32)), _dev(parent), _dev(table), nb, bs, mask,
                        pos if want else None, slot if want else None, ws)
    return host(mask), host(pos), host(slot), binding.read_status_ws(ws)[0]


@pytest.mark.parametrize("ns,words", [((1,), 1), ((0, 3, 33, 1, 64, 0, 31), 2), ((1024, 7), 32), ((200,) * 5, 7), ((40, 90), 2)])
def test_layout(ns, words):
    rng = np.random.default_rng(len(ns))
    Ls = [n + int(rng.integers(0, 50)) for n in ns]
    c = case("f32", 2, 2, 8, 4, ns, Ls, words=words, extra=3, seed=words)
    if sum(ns) > 1000:
        c["parent"][:1024] = np.arange(1024) - 1  # one line of 1024 nodes
    got = run_layout(c["qsl"], c["seq"], c["parent"], c["table"], c["nb"], 4, words, c["T"])
    want = X.tree_layout(c["qsl"], c["seq"], c["parent"], c["table"], c["nb"], 4, words)
    for a, b in zip(got, want):
        np.testing.assert_array_equal(a, b)
    assert got[3] == (binding.PE_ST_TREE if max(ns) > 32 * words else 0)
    assert (run_layout(c["qsl"], c["seq"], c["parent"], c["table"], c["nb"], 4, words, c["T"], want=False)[0] == want[0]).all()


def test_layout_reports_what_is_wrong():
    qsl, table = np.array([0, 4, 6], np.int32), np.array([[1, 9], [0, -1]], np.int32)
    parent = np.array([-1, 3, -5, 2, 0, 0], np.int32)  # row 1 names a later one, row 2 none, row 4 itself
    seq = [7, 6]
    m, pos, slot, st = run_layout(qsl, seq, parent, table, 3, 4, 1, 6)
    want = X.tree_layout(qsl, seq, parent, table, 3, 4, 1)
    for a, b in zip((m, pos, slot), want):
        np.testing.assert_array_equal(a, b)
    assert st == binding.PE_ST_TREE | binding.PE_ST_BLOCK_RANGE
    good = np.array([-1, 0, 1, 2, -1, 0], np.int32)
    for seq in ([3, 2], [-9, 2], [2 ** 31 - 1, 2], [-2 ** 31, 2]):  # nodes before position 0, past the table
        m, pos, slot, st = run_layout(qsl, seq, good, np.abs(table) % 3, 3, 4, 1, 6)
        want = X.tree_layout(qsl, seq, good, np.abs(table) % 3, 3, 4, 1)
        for a, b in zip((m, pos, slot), want):
            np.testing.assert_array_equal(a, b)
        assert st == binding.PE_ST_BLOCK_RANGE
    for bad in ([0, 5, 4], [1, 2, 6], [0, -3, 6], [0, 4, 99]):
        assert run_layout(np.array(bad, np.int32), [4, 2], good, np.abs(table) % 3, 3, 4, 1, 6)[3] & binding.PE_ST_ROWS_RANGE


def run_accept(qsl, parent, tok, target):
    torch = cuda_or_skip()
    built()
    B, T = len(qsl) - 1, len(tok)
    acc, bonus = (torch.full((B,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    path = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    i32 = lambda x: _dev(np.asarray(x, np.int32))  # noqa: E731
    binding.tree_accept(B, T, i32(qsl), i32(parent), i32(tok), i32(target), acc, path, bonus, ws)
    return host(acc), host(path), host(bonus), binding.read_status_ws(ws)[0]


@pytest.mark.parametrize("ns", [(1,), (0, 5, 1, 33, 0, 2), (64, 300, 17, 1024), (3,) * 200])
@pytest.mark.parametrize("tokens", [1, 2, 5])
def test_walk(ns, tokens):
    rng = np.random.default_rng(sum(ns) + tokens)
    qsl = np.concatenate([[0], np.cumsum(ns)])
    parent = [p for n in ns for p in tree(rng, n)] + [0, 0]
    tok, target = (rng.integers(0, tokens, len(parent)) for _ in range(2))
    target[rng.random(len(target)) < 0.05] = -1
    tok[rng.random(len(tok)) < 0.05] = -1
    got = run_accept(qsl, parent, tok, target)
    for a, b in zip(got, X.tree_accept(qsl, parent, tok, target)):
        np.testing.assert_array_equal(a, b)
    assert got[3] == 0
    if tokens == 1 and max(ns) > 30:
        assert got[0].max() > 2


def test_walk_edges():
    line = np.arange(1024) - 1
    acc, path, bonus, st = run_accept([0, 1024], line, np.full(1024, 5), np.full(1024, 5))
    assert acc.tolist() == [1023] and bonus.tolist() == [5] and (path == np.arange(1024)).all() and st == 0
    # a node past the most is not walked to; two roots: the walk begins at row 0; a child named twice
    line = np.arange(1030) - 1
    acc, path, bonus, st = run_accept([0, 1030], line, np.full(1030, 5), np.full(1030, 5))
    assert acc.tolist() == [1023] and (path[1024:] == -1).all() and st == binding.PE_ST_TREE
    acc, path, _, st = run_accept([0, 5], [-1, -1, 1, 0, 0], [9, 4, 4, 4, 4], [4, 4, 4, 4, 4])
    assert acc.tolist() == [1] and path.tolist() == [0, 3, -1, -1, -1] and st == 0
    acc, _, _, st = run_accept([0, 3], [-1, 2, 0], [4, 4, 4], [4, 4, 4])
    assert acc.tolist() == [1] and st == binding.PE_ST_TREE
    acc, _, bonus, st = run_accept([0, 0, 0], np.zeros(0), np.zeros(0), np.zeros(0))
    assert acc.tolist() == [0, 0] and bonus.tolist() == [-1, -1] and st == 0


# ------------------------------------------------------------------ attention


SHAPES = [("bf16", 64, 8, 64, 16), ("bf16", 32, 8, 128, 16), ("bf16", 8, 2, 64, 8), ("bf16", 7, 1, 128, 64),
          ("bf16", 5, 5, 64, 24), ("bf16", 6, 2, 64, 5), ("bf16", 4, 2, 128, 256), ("f32", 4, 2, 16, 4),
          ("f32", 6, 3, 40, 5), ("f32", 8, 2, 128, 16)]


@pytest.mark.parametrize("dtype,H,G,hd,bs", SHAPES)
@pytest.mark.parametrize("sinks", [False, True])
def test_attend_small_ragged(dtype, H, G, hd, bs, sinks):
    """One node, no rows, no context, more nodes than positions, lengths around a block and a tile."""
    ns = (1, 0, 3, 2, 9, 4, 1, 5, 1, 40, 0, 33)
    Ls = (1, 5, 3, 0, 4, 127, 128, 129, 16, 60, 0, 160)
    check(case(dtype, H, G, hd, bs, ns, Ls, sinks=sinks, extra=3, poison=True, pad=16))


@pytest.mark.parametrize("dtype,H,G,hd,bs", SHAPES[:4] + [("bf16", 128, 1, 64, 16), ("f32", 4, 2, 16, 4)])
@pytest.mark.parametrize("n,L", [(1, 700), (16, 1500), (33, 33), (64, 900), (129, 600), (300, 301), (257, 2000)])
def test_attend_one_request(dtype, H, G, hd, bs, n, L):
    check(case(dtype, H, G, hd, bs, (n,), (L,), poison=True, seed=n))


@pytest.mark.parametrize("ctx", [0, 1, 31, 32, 33, 63, 64, 65, 95, 127, 128, 129, 160])
@pytest.mark.parametrize("hd", [64, 128])
def test_attend_masks_at_every_offset_in_a_tile(ctx, hd):
    """The nodes' bits against the tile's keys: any shift, several words, a tile's end inside."""
    check(case("bf16", 8, 2, hd, 8, (70, 3, 100), (70 + ctx, 3 + ctx, 100 + ctx), poison=True, seed=ctx))


def test_attend_any_masks():
    """Bits that are no tree's: rows that see nothing, not themselves, nodes behind them, bits behind the last node."""
    def bits(rng, m):
        m = rng.integers(-2 ** 31, 2 ** 31, m.shape).astype(np.int32)
        m[::5] = 0
        m[1::5] = -1
        return m

    for dtype, hd, bs in (("bf16", 64, 16), ("bf16", 128, 8), ("f32", 16, 4), ("bf16", 64, 5)):
        check(case(dtype, 4, 2, hd, bs, (40, 1, 70, 6, 5), (40, 1, 300, 6, 5), words=4, bits=bits, seed=hd, sinks=hd == 64))


def test_attend_values_that_only_some_nodes_see_may_be_infinite():
    """A node with NaN or infinities in its keys and values reaches its descendants alone."""
    for dtype, hd, bs in (("bf16", 64, 16), ("bf16", 128, 16), ("f32", 16, 4)):
        c = case(dtype, 4, 2, hd, bs, (30, 9), (200, 9), seed=hd)
        k, v = O.decode(c["kc"], dtype).copy(), O.decode(c["vc"], dtype).copy()
        hurt = {0: [3, 17], 1: [4]}
        for r, nodes in hurt.items():
            for j in nodes:
                t = c["seq"][r] - (c["qsl"][r + 1] - c["qsl"][r]) + j
                v[c["table"][r, t // bs], :, t % bs] = np.nan
                k[c["table"][r, t // bs], :, t % bs, 0] = np.inf if j == 17 else k[c["table"][r, t // bs], :, t % bs, 0]
        clean = host(attend(c)[0])
        got, st = attend(dict(c, kc=_store(k, dtype), vc=_store(v, dtype)))
        got = host(got)
        assert st == 0
        sees = X.unpack(c["mask"])
        for r, nodes in hurt.items():
            for row in range(c["qsl"][r], c["qsl"][r + 1]):
                if sees[row][nodes].any():
                    assert np.isnan(O.decode(got[row], dtype)).all()
                else:
                    a, b = O.decode(got[row], dtype), O.decode(clean[row], dtype)
                    # (computed again in fp32, without the rounding of the weights)
                    np.testing.assert_allclose(a, b, rtol=2.0 ** -7, atol=0.05 if dtype == "bf16" else 1e-5)


def test_attend_a_chain_is_chunk_attention():
    torch = cuda_or_skip()
    for dtype, H, G, hd, bs in SHAPES:
        ns, Ls = (8, 1, 33, 5), (1000, 5, 33, 129)
        c = case(dtype, H, G, hd, bs, ns, Ls, seed=3, sinks=True)
        parent = np.concatenate([np.arange(n) - 1 for n in ns]).astype(np.int32)
        c["mask"] = X.tree_layout(c["qsl"], Ls, parent, c["table"], c["nb"], bs, 2)[0]
        got = check(c)
        plan = binding.PagedAttention(H, G, hd, bs, dtype=dtype)
        d = {k: _dev(c[k], dtype) for k in ("q", "kc", "vc")} | {k: _dev(c[k]) for k in ("qsl", "seq", "table", "sink")}
        out = torch.empty(c["T"], H * hd, dtype=d["q"].dtype, device="cuda")
        plan.attend(4, c["T"], d["qsl"], d["seq"], d["q"], d["kc"], d["vc"], d["table"], c["nb"], out, plan.workspace(4, c["T"]),
                    sink=d["sink"])
        a, b = O.decode(host(got), dtype), O.decode(host(out), dtype)
        # two roundings of the weights and of the result
        np.testing.assert_allclose(a, b, rtol=2.0 ** -7, atol=0.05 if dtype == "bf16" else 1e-5)


def test_attend_bad_input_is_reported():
    def edit(table, nb):
        table[0, 1] = -1
        table[1, 0] = nb
        table[2, :] = -7

    for dtype, hd, bs in (("bf16", 64, 16), ("bf16", 64, 5), ("f32", 16, 4)):
        check(case(dtype, 4, 2, hd, bs, (3, 50, 2), (90, 260, 30), table_edit=edit, seed=5), status=binding.PE_ST_BLOCK_RANGE)
        c = case(dtype, 4, 2, hd, bs, (40, 3), (90, 60), words=1, seed=5)  # 40 nodes, 32 bits
        check(c, status=binding.PE_ST_TREE)
        for qsl in ((0, 50, 43), (1, 2, 43), (0, -3, 43), (0, 40, 99)):
            _, st = attend(dict(c, qsl=np.array(qsl, np.int32)))
            assert st & binding.PE_ST_ROWS_RANGE
        over = dict(c, seq=np.array([c["table"].shape[1] * bs + 9, 60], np.int32))
        assert attend(over)[1] & binding.PE_ST_BLOCK_RANGE


def test_attend_far_blocks_of_a_large_cache():
    """Offsets past 2^31 elements."""
    torch = cuda_or_skip()
    built()
    G, hd, bs = 8, 128, 16
    nb = (1 << 31) // (G * hd * bs) + 40
    plan = binding.PagedAttention(16, G, hd, bs)
    k, v = (torch.zeros(nb, G, bs, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c = case("bf16", 16, G, hd, bs, (20,), (150,), seed=9)
    far = nb - c["nb"]
    k[far:], v[far:] = _dev(c["kc"], "bf16"), _dev(c["vc"], "bf16")
    out = torch.empty(20, 16 * hd, dtype=torch.bfloat16, device="cuda")
    ws = plan.workspace(1, 20)
    table = _dev(np.where(c["table"] >= 0, c["table"] + far, -1).astype(np.int32))
    plan.attend_tree(1, 20, _dev(c["qsl"]), _dev(c["seq"]), _dev(c["q"], "bf16"), k, v, table, nb, _dev(c["mask"]), out, ws)
    assert binding.read_status_ws(ws)[0] == 0
    np.testing.assert_array_equal(host(out), host(attend(c)[0]))


def test_attend_many_requests_and_streams():
    torch = cuda_or_skip()
    rng = np.random.default_rng(8)
    ns = rng.integers(0, 20, 700).tolist()
    Ls = [int(n + rng.integers(0, 60)) for n in ns]
    want = check(case("bf16", 8, 2, 64, 16, ns, Ls, seed=9))
    for _ in range(5):
        got, _ = attend(case("bf16", 8, 2, 64, 16, ns, Ls, seed=9), stream=torch.cuda.Stream())
        assert torch.equal(got, want)
    check(case("f32", 4, 2, 16, 4, ns, Ls, seed=9))
