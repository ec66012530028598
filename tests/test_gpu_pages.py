"""The cache's pages against the oracle: bytes and counts, so everything is equal."""

import numpy as np
import pytest

from oracle import pe_tree as X
from parity import built, cuda_or_skip, host
from speculative_drafting_gb300 import binding, runner
from test_gpu_tree import tree

pytestmark = pytest.mark.gpu

PLANS = [("bf16", 8, 64, 16, 3), ("bf16", 2, 128, 8, 1), ("bf16", 3, 64, 5, 2), ("f32", 2, 16, 4, 2), ("f32", 3, 40, 7, 1)]


def caches(rng, dtype, layers, nb, G, bs, hd):
    shape = (layers, nb, G, bs, hd)
    return [rng.integers(0, 65536, shape).astype(np.uint16) if dtype == "bf16" else
            rng.integers(0, 2 ** 32, shape, dtype=np.uint64).astype(np.uint32).view(np.float32) for _ in range(2)]


def up(x, dtype="f32"):
    return runner.to_device(x, dtype)


def same(a, b):
    np.testing.assert_array_equal(np.ascontiguousarray(a).view(np.uint8), np.ascontiguousarray(b).view(np.uint8))


def i32(x):
    return up(np.asarray(x, np.int32))


# ------------------------------------------------------------------ copy and compact


@pytest.mark.parametrize("dtype,G,hd,bs,layers", PLANS)
@pytest.mark.parametrize("n", [0, 1, 37])
def test_copy(dtype, G, hd, bs, layers, n):
    torch = cuda_or_skip()
    built()
    rng = np.random.default_rng(n)
    nb = 2 * n + 5
    k, v = caches(rng, dtype, layers, nb, G, bs, hd)
    ids = rng.permutation(nb)
    src, dst = ids[:n].copy(), ids[n:2 * n].copy()
    if n > 3:
        dst[1] = src[1]                       # stays
        src[2] = src[0]                       # one page to two
    plan = binding.PagedAttention(G, G, hd, bs, dtype=dtype)
    dk, dv, ws = up(k, dtype), up(v, dtype), plan.append_workspace()
    plan.copy_pages(layers, n, i32(src), i32(dst), nb, dk, dv, ws)
    k[:, dst], v[:, dst] = k[:, src], v[:, src]
    same(host(dk), k)
    same(host(dv), v)
    assert binding.read_status_ws(ws)[0] == 0
    if n:  # pages outside the pool are left out
        plan.copy_pages(layers, 4, i32([-1, nb, ids[0], ids[1]]), i32([ids[2], ids[3], nb, -7]), nb, dk, dv, ws)
        same(host(dk), k)
        same(host(dv), v)
        assert binding.read_status_ws(ws)[0] == binding.PE_ST_BLOCK_RANGE


def run_compact(dtype, G, hd, bs, layers, ns, ctx, accepted, path, table, nb, seed=0, status=0, qsl=None):
    torch = cuda_or_skip()
    built()
    rng = np.random.default_rng(seed)
    qsl = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32) if qsl is None else np.array(qsl, np.int32)
    seq = np.array([n + c for n, c in zip(ns, ctx)], np.int32)
    k, v = caches(rng, dtype, layers, nb, G, bs, hd)
    plan = binding.PagedAttention(G, G, hd, bs, dtype=dtype)
    dk, dv, ws = up(k, dtype), up(v, dtype), plan.append_workspace()
    plan.compact(layers, len(ns), len(path), i32(qsl), i32(seq), i32(accepted), i32(path), i32(table), nb, dk, dv, ws)
    wk, wv = X.compact(qsl, seq, accepted, path, np.asarray(table), k, v)
    same(host(dk), wk)
    same(host(dv), wv)
    assert binding.read_status_ws(ws)[0] == status
    return (wk != k).any()


def tables(rng, lengths, bs, spare=2):
    blocks = [(x + bs - 1) // bs for x in lengths]
    nb = sum(blocks) + spare
    ids, out, o = rng.permutation(nb), np.full((len(lengths), max(max(blocks), 1)), -1, np.int32), 0
    for r, b in enumerate(blocks):
        out[r, :b] = ids[o:o + b]
        o += b
    return out, nb


@pytest.mark.parametrize("dtype,G,hd,bs,layers", PLANS)
def test_compact_paths_of_walks(dtype, G, hd, bs, layers):
    """Accepted lines of random trees: rows whose slots another row of the path moves to."""
    rng = np.random.default_rng(hd)
    ns = [1, 0, 30, 7, 64, 2, 300, 5]
    ctx = [int(x) for x in rng.integers(0, 40, len(ns))]
    table, nb = tables(rng, [n + c for n, c in zip(ns, ctx)], bs)
    acc, path = [], []
    for n in ns:
        line = X.lines(tree(rng, n, chain=0.95))[-1] if n else []
        acc.append(max(len(line) - 1, 0))
        path += line + [-1] * (n - len(line))
    assert max(acc) > 10
    assert run_compact(dtype, G, hd, bs, layers, ns, ctx, acc, path, table, nb)


def test_compact_long_and_idle_paths():
    rng = np.random.default_rng(1)
    n = 1024
    table, nb = tables(rng, [n + 9] * 3, 16)
    line = [0] + sorted(rng.choice(np.arange(1, n), 600, replace=False).tolist())
    ident = list(range(n))          # nothing moves
    shift = [0] + list(range(2, n)) + [-1]   # each row to the slot of the one before
    path = line + [-1] * (n - len(line)) + ident + shift
    assert run_compact("bf16", 2, 64, 16, 2, [n] * 3, [9] * 3, [600, n - 1, n - 2], path, table, nb)


def test_compact_reports_what_is_wrong():
    rng = np.random.default_rng(2)
    table, nb = tables(rng, [12, 12], 4)
    good = [0, 2, 3, 5, -1, -1]
    a = ("f32", 2, 16, 4, 1, [6, 6], [6, 6])
    st = binding
    run_compact(*a, [9, -2], good + good, table, nb, status=st.PE_ST_ACCEPTED_RANGE | st.PE_ST_TREE)
    for bad in ([0, 2, 2, 5], [0, 3, 2, 5], [0, 2, 3, 6], [0, 0, 3, 5], [0, -1, 3, 5], [0, 2, 3, 2 ** 31 - 1]):
        run_compact(*a, [3, 3], bad + [-1, -1] + good, table, nb, status=st.PE_ST_TREE)
    holes = table.copy()
    holes[0, 1], holes[1, 2] = -1, nb
    run_compact(*a, [3, 3], good + good, holes, nb, status=st.PE_ST_BLOCK_RANGE)
    run_compact("f32", 2, 16, 4, 1, [6, 6], [-8, 400], [3, 3], good + good, table, nb, status=st.PE_ST_BLOCK_RANGE)
    run_compact(*a, [3, 3], good + good, table, nb)


# ------------------------------------------------------------------ the pool


class Device:
    """The pool on the device beside the oracle's."""

    def __init__(self, rows, mb, nb, dtype="bf16", G=2, hd=64, bs=4, layers=2, seed=0):
        cuda_or_skip()
        built()
        rng = np.random.default_rng(seed)
        self.pool = X.Pool(np.full((rows, mb), -1, np.int32), np.zeros(nb, np.int32), bs)
        self.k, self.v = caches(rng, dtype, layers, nb, G, bs, hd)
        self.plan = binding.PagedAttention(G, G, hd, bs, dtype=dtype)
        self.dk, self.dv, self.layers = up(self.k, dtype), up(self.v, dtype), layers
        self.table, self.refs = i32(self.pool.table), i32(self.pool.refs)
        self.ws = binding.pages_workspace(rows, nb)

    def check(self):
        same(host(self.table), self.pool.table)
        same(host(self.refs), self.pool.refs)
        same(host(self.dk), self.k)
        same(host(self.dv), self.v)
        st = binding.read_status_ws(self.ws)[0]
        assert (st & binding.PE_ST_PAGES != 0) == self.pool.refused
        refused, self.pool.refused = self.pool.refused, False
        return refused

    def reserve(self, rows, lengths):
        binding.pages_reserve(len(rows), i32(rows), i32(lengths), self.table, self.refs, self.pool.bs, self.ws)
        self.pool.reserve(rows, lengths)
        return self.check()

    def fork(self, parents, children, lengths):
        self.plan.fork(self.layers, len(parents), i32(parents), i32(children), i32(lengths), self.table, self.refs,
                       self.dk, self.dv, self.ws)
        self.pool.fork(parents, children, lengths, (self.k, self.v))
        return self.check()

    def free(self, rows):
        binding.pages_free(len(rows), i32(rows), self.table, self.refs, self.ws)
        self.pool.free(rows)
        return self.check()


def test_pool_by_turns():
    """Requests that come, grow, are sampled several times and go, at random."""
    for dtype, G, hd, bs, layers in PLANS:
        rng = np.random.default_rng(hd)
        d = Device(12, 6, 40, dtype, G, hd, bs, layers)
        for _ in range(25):
            what = rng.integers(0, 3)
            rows = rng.choice(12, int(rng.integers(1, 5)), replace=False)
            if what == 0:
                d.reserve(rows, rng.integers(0, 6 * bs + 1, len(rows)))
            elif what == 1:
                par = rng.integers(0, 12, len(rows))
                d.fork(par, rows, [int(rng.integers(0, max((d.pool.table[p] >= 0).sum() * bs, 1) + 1)) for p in par])
            else:
                d.free(rows)


def test_pool_shares_full_pages_and_copies_the_last():
    d = Device(9, 5, 30)
    assert not d.reserve([0, 1], [10, 8])
    assert not d.fork([0, 0, 1, 0], [5, 3, 4, 8], [10, 10, 8, 7])
    assert d.pool.refs[d.pool.table[0, 0]] == 4 and d.pool.table[5, 2] != d.pool.table[0, 2]
    assert not d.free([0])
    assert not d.reserve([5], [20])
    assert not d.free([5, 3, 4, 8, 1, 1, 5])  # (twice: once)
    assert (d.pool.refs == 0).all()
    assert not d.fork([2], [3], [0])  # nothing of nothing


def test_pool_refuses():
    d = Device(6, 4, 9)
    assert not d.reserve([0], [13])
    for rows, lengths in (([-1], [3]), ([6], [3]), ([1], [-1]), ([1], [17]), ([1, 1], [3, 3]), ([1, 2, 1], [3, 3, 9])):
        assert d.reserve(rows, lengths)
    assert not d.free([1, 2])
    for p, c, n in (([0], [0], [4]), ([0], [6], [4]), ([-1], [1], [4]), ([0], [1], [-3]), ([0], [1], [17]), ([1], [2], [4]),
                    ([0, 0], [1, 1], [4, 4]), ([0, 1], [1, 2], [4, 4]), ([0], [1], [2 ** 31 - 1])):
        assert d.fork(p, c, n)
        d.free([1, 2])
    assert not d.fork([0], [1], [16])   # (13 positions fill four pages)
    assert d.fork([0], [1], [4])        # its row is not empty
    assert d.free([6, -1])
    # an empty pool: the first that fit, in order
    assert d.reserve([2, 3, 4], [8, 16, 4])
    assert not d.free([2, 3, 4])
    assert not d.reserve([2, 3], [12, 7])
    assert d.fork([0, 0, 0], [4, 5, 1], [13, 12, 13])
    # entries that no page has, and counts that are 0 already
    bad = d.pool.table.copy()
    d.free(range(6))
    bad[:] = -1
    bad[0, :3] = [9, 2, 3]
    d.pool.table = bad
    d.table.copy_(i32(bad))
    binding.pages_free(1, i32([0]), d.table, d.refs, d.ws)
    st = binding.read_status_ws(d.ws)[0]
    assert st == binding.PE_ST_PAGES | binding.PE_ST_BLOCK_RANGE
    assert (host(d.table)[0] == -1).all() and (host(d.refs) == 0).all()
    # every negative entry is none
    d.table[0, :3] = i32([-5, -(1 << 31), -2])
    binding.pages_free(1, i32([0]), d.table, d.refs, d.ws)
    assert binding.read_status_ws(d.ws)[0] == 0 and (host(d.table)[0] == -1).all() and (host(d.refs) == 0).all()


def test_pool_large():
    """More entries than a CTA has threads, rows of many pages, a pool that takes several scans."""
    d = Device(1500, 700, 9000, "f32", 1, 8, 2, 1)
    rng = np.random.default_rng(3)
    assert not d.reserve(np.arange(700), rng.integers(0, 12, 700))
    assert not d.reserve([700, 701], [1400, 1399])
    # holes in the pool
    assert not d.free(rng.choice(700, 300, replace=False))
    rows = np.arange(702, 1302)
    par = rng.integers(0, 702, 600)
    n = [int((d.pool.table[p] >= 0).sum()) * 2 - int(rng.integers(0, 2)) for p in par]
    assert not d.fork(par, rows, [max(x, 0) for x in n])
    assert d.reserve(np.arange(1302, 1500), [1400] * 198)


def test_pool_in_a_graph():
    torch = cuda_or_skip()
    d = Device(8, 6, 30)
    d.reserve([0, 1], [10, 17])
    s = torch.cuda.Stream()
    child, par, n = i32([2, 3, 4]), i32([0, 1, 0]), i32([10, 17, 9])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        binding.pages_free(3, child, d.table, d.refs, d.ws, stream=s)
        d.plan.fork(d.layers, 3, par, child, n, d.table, d.refs, d.dk, d.dv, d.ws, stream=s)
    for lengths in ([10, 17, 9], [9, 20, 0], [3, 4, 11]):
        n.copy_(i32(lengths))
        g.replay()
        torch.cuda.synchronize()
        d.pool.free([2, 3, 4])
        d.pool.fork([0, 1, 0], [2, 3, 4], lengths, (d.k, d.v))
        assert not d.check()
