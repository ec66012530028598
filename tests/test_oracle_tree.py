"""Pins of the oracle of trees, sampling and pages: each against a second way to the answer."""

import numpy as np

from oracle import pe_paged as P
from oracle import pe_tree as X


def test_a_chain_is_chunk_attention():
    rng = np.random.default_rng(0)
    H, G, hd, bs, L, n = 4, 2, 16, 4, 23, 6
    kc, vc = (rng.standard_normal((8, G, bs, hd)) for _ in range(2))
    table = rng.permutation(8)[None, :6].astype(np.int32)
    q = rng.standard_normal((n, H, hd))
    parent = np.arange(n) - 1
    mask, pos, slot = X.tree_layout([0, n], [L], parent, table, 8, bs, 1)
    assert pos.tolist() == list(range(L - n, L))
    assert slot.tolist() == [table[0][t // bs] * bs + t % bs for t in range(L - n, L)]
    sink = rng.standard_normal(H)
    a = P.chunk_attention([0, n], [L], q, kc, vc, table, sink)
    b = X.tree_attention([0, n], [L], q, kc, vc, table, mask, sink)
    np.testing.assert_allclose(a[0], b[0], rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(a[1], b[1], rtol=1e-12, atol=1e-14)


def test_a_node_of_a_tree_is_the_end_of_its_line():
    """Each node's row equals that of a request whose rows are the node's line alone."""
    rng = np.random.default_rng(1)
    H, G, hd, bs, ctx = 2, 1, 8, 4, 9
    parent = np.array([-1, 0, 0, 1, 1, 2, 5])
    n = len(parent)
    L = ctx + n
    kc, vc = (rng.standard_normal((6, G, bs, hd)) for _ in range(2))
    table = np.arange(6, dtype=np.int32)[None]
    q = rng.standard_normal((n, H, hd))
    mask, pos, _ = X.tree_layout([0, n], [L], parent, table, 6, bs, 2)
    got = X.tree_attention([0, n], [L], q, kc, vc, table, mask)[0]
    flat = lambda c: c.transpose(0, 2, 1, 3).reshape(-1, G, hd)  # noqa: E731
    for j, line in enumerate(X.lines(parent)):
        keep = list(range(ctx)) + [ctx + i for i in line]
        k1, v1 = (flat(c)[keep].transpose(1, 0, 2)[None] for c in (kc, vc))
        want = P.chunk_attention([0, 1], [len(keep)], q[j:j + 1], k1, v1, np.zeros((1, 1), np.int32))[0]
        np.testing.assert_allclose(got[j], want[0], rtol=1e-12)
        assert pos[j] == ctx + len(line) - 1
    bits = X.unpack(mask)
    assert [np.flatnonzero(b).tolist() for b in bits] == [sorted(x) for x in X.lines(parent)]


def test_the_walk_of_a_chain_is_greedy_verification():
    from oracle import pe_oracle as O

    rng = np.random.default_rng(2)
    qsl = np.array([0, 5, 5, 9, 10])
    lg = rng.standard_normal((10, 3))
    tok = rng.integers(0, 3, 10)
    tgt, acc, bonus = O.verify_greedy(qsl, tok, lg)
    parent = np.concatenate([np.arange(n) - 1 for n in np.diff(qsl)])
    a, path, b = X.tree_accept(qsl, parent, tok, tgt)
    np.testing.assert_array_equal(a, acc)
    np.testing.assert_array_equal(b, bonus)
    for r in range(4):
        assert path[qsl[r]:qsl[r] + a[r] + 1].tolist() == list(range(a[r] + 1)) or qsl[r] == qsl[r + 1]


def test_sampling_by_counting():
    """Frequencies over many noises against the cut and renormalised probabilities."""
    rng = np.random.default_rng(3)
    x = np.log(np.array([0.4, 0.05, 0.25, 0.2, 0.1]))
    for k, p, m, kept in ((0, 1.0, 0.0, [0, 1, 2, 3, 4]), (3, 1.0, 0.0, [0, 2, 3]), (0, 0.6, 0.0, [0, 2]),
                          (0, 0.66, 0.0, [0, 2, 3]), (0, 1.0, 0.3, [0, 2, 3]), (3, 0.9, 0.6, [0, 2]),
                          (1, 1.0, 0.0, [0]), (0, 0.0, 0.0, [0]), (0, 1.0, 2.0, [0])):
        n = 4000
        g = -np.log(rng.exponential(size=(n, 5)))
        hits = np.bincount([X._sample_row(x, 1.0, k, p, m, gi)[0] for gi in g], minlength=5) / n
        prob = np.exp(x) * np.isin(np.arange(5), kept)
        prob /= prob.sum()
        # five standard deviations of a share of n draws
        assert (np.abs(hits - prob) <= 5 * np.sqrt(prob * (1 - prob) / n)).all(), (k, p, m, hits)


def test_ties_of_the_order_go_to_the_lowest_index():
    x = np.zeros(6)
    g = np.array([0, 1, 2, 3, 4, 5.0])
    assert X._sample_row(x, 1.0, 3, 1.0, 0.0, g)[0] == 2       # the first three are kept
    assert X._sample_row(x, 1.0, 0, 0.5, 0.0, g)[0] == 2       # three of six weigh a half
    assert X._sample_row(x, 1.0, 0, 0.51, 0.0, g)[0] == 3
    assert X._sample_row(x, 1.0, 0, 1.0, 0.0, np.zeros(6))[0] == 0


def test_the_pool_keeps_its_counts():
    rng = np.random.default_rng(4)
    pool = X.Pool(np.full((9, 5), -1, np.int32), np.zeros(20, np.int32), 4)
    for _ in range(60):
        row = int(rng.integers(0, 9))
        what = rng.integers(0, 3)
        if what == 0:
            pool.reserve([row], [int(rng.integers(0, 21))])
        elif what == 1:
            have = int((pool.table[row] >= 0).sum())
            pool.fork([row], [int(rng.integers(0, 9))], [int(rng.integers(0, 4 * have + 1))])
        else:
            pool.free([row])
        used = pool.table[pool.table >= 0]
        np.testing.assert_array_equal(np.bincount(used, minlength=20), pool.refs)
