"""The fp64 oracle of the paged attention calls and of verification by sampling,
against closed forms and brute force (CPU only)."""

import itertools

import numpy as np
import pytest

from oracle import pe_oracle as O
from oracle import pe_paged as P


def test_rotation_agrees_with_the_steps_rope_and_the_norm_with_its_rmsnorm():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 16))
    pos = np.array([0, 1, 7, 1000, 32767])
    gain = rng.standard_normal(16)
    np.testing.assert_allclose(P.norm_rotate(x, None, pos, 10000.0, 1e-6), O.rope(x, pos, 10000.0), atol=1e-10)
    y = O.rmsnorm(x, gain, 1e-6)
    np.testing.assert_allclose(P.norm_rotate(x, gain, np.zeros(5), 10000.0, 1e-6), y, atol=1e-13)


def test_append_writes_named_slots_only():
    rng = np.random.default_rng(1)
    kc, vc = rng.standard_normal((2, 3, 2, 4, 8))
    qkv = rng.standard_normal((4, (4 + 2 * 2) * 8))
    slot = np.array([5, -1, 0, 12])  # 12 is past the three blocks of four
    q, k2, v2 = P.qkv_append(qkv, 4, 2, None, None, np.zeros(4), slot, kc, vc)
    np.testing.assert_array_equal(q.reshape(4, -1), qkv[:, :32])  # position 0: no rotation
    np.testing.assert_array_equal(k2[1, :, 1].ravel(), qkv[0, 32:48])
    np.testing.assert_array_equal(v2[0, :, 0].ravel(), qkv[2, 48:])
    same = np.ones((3, 4), bool)
    same[1, 1] = same[0, 0] = False
    assert (k2 == kc).all((1, 3))[same].all() and (v2 == vc).all((1, 3))[same].all()


def test_attention_closed_forms():
    rng = np.random.default_rng(2)
    kc, vc = rng.standard_normal((2, 4, 1, 4, 8))
    table = np.array([[2, 0, 3, 1]])
    q = rng.standard_normal((1, 2, 8))
    one, _ = P.chunk_attention([0, 1], [1], q, kc, vc, table)
    np.testing.assert_allclose(one[0, 1], vc[2, 0, 0])             # one key: its value
    zero, _ = P.chunk_attention([0, 1], [9], np.zeros_like(q), kc, vc, table)
    seq = np.concatenate([vc[2, 0], vc[0, 0], vc[3, 0, :1]])
    np.testing.assert_allclose(zero[0, 0], seq.mean(0))             # equal scores: the mean
    sink, _ = P.chunk_attention([0, 1], [1], np.zeros_like(q), kc, vc, table, sink=[0.0, np.log(3)])
    np.testing.assert_allclose(sink[0, 0], vc[2, 0, 0] / 2)
    np.testing.assert_allclose(sink[0, 1], vc[2, 0, 0] / 4)
    # the step's own attention of one row over the same keys
    full, _ = P.chunk_attention([0, 1], [9], q, kc, vc, table)
    K = np.concatenate([kc[2, 0], kc[0, 0], kc[3, 0, :1]])
    np.testing.assert_allclose(full[0, 0], O.attend(q[0, 0], K, seq), atol=1e-12)


def test_attention_rows_are_causal_and_empty_rows_zero():
    rng = np.random.default_rng(3)
    kc, vc = rng.standard_normal((2, 3, 2, 4, 8))
    table = np.array([[1, 2, 0]])
    q = rng.standard_normal((6, 4, 8))
    whole, _ = P.chunk_attention([0, 6], [10], q, kc, vc, table)
    for j in range(6):  # a row alone sees what it sees in the chunk
        alone, _ = P.chunk_attention([0, 1], [10 - 6 + j + 1], q[j:j + 1], kc, vc, table)
        np.testing.assert_allclose(whole[j], alone[0], atol=1e-12)
    short, _ = P.chunk_attention([0, 6], [2], q, kc, vc, table)     # four rows before position 0
    assert (short[:4] == 0).all() and (short[4:] != 0).all()
    bad, _ = P.chunk_attention([0, 6], [10], q, kc, vc, np.array([[-1, 7, 5]]))
    assert (bad == 0).all()


@pytest.mark.parametrize("V,n", [(3, 1), (3, 2), (4, 3)])
def test_verification_is_rejection_sampling(V, n):
    """Over many draws the first token out (draft 1 if accepted, else the bonus)
    has the target's distribution, whatever the draft."""
    rng = np.random.default_rng(4 + V + n)
    logits = rng.standard_normal((n, V))
    temp = 0.7
    p0 = np.exp(logits[0] / temp)
    p0 /= p0.sum()
    N = 6000
    for draft in itertools.islice(itertools.product(range(V), repeat=n - 1), 3):
        tok = np.array([0, *draft])
        got = np.zeros(V)
        for _ in range(N):
            a, b, p, _ = P.verify_sampled([0, n], tok, logits, [temp], rng.random(n),
                                          -np.log(rng.exponential(size=(1, V))))
            first = tok[1] if a[0] > 0 else b[0]
            got[first] += 1
            if n > 1 and a[0] < n - 1:
                assert b[0] != tok[a[0] + 1]
        np.testing.assert_allclose(got / N, p0, atol=5 * np.sqrt(0.25 / N))
        if n > 1:
            np.testing.assert_allclose(p[1], p0[draft[0]])


def test_verification_at_temperature_zero_is_greedy():
    rng = np.random.default_rng(9)
    qsl = np.array([0, 4, 4, 7, 8])
    logits = rng.integers(-1, 2, (8, 5)).astype(np.float64)
    for _ in range(200):
        tok = rng.integers(0, 5, 8)
        tgt, acc, bon = O.verify_greedy(qsl, tok, logits)
        a, b, _, _ = P.verify_sampled(qsl, tok, logits, np.zeros(4), rng.random(8), np.zeros((4, 5)))
        np.testing.assert_array_equal(a, acc)
        np.testing.assert_array_equal(b, bon)


def test_verification_edges():
    inf = np.inf
    lg = np.array([[0.0, 1.0, -inf], [-inf, -inf, -inf], [0.0, np.nan, 1.0]])
    # a barred draft is rejected whatever the number; the race skips it
    a, b, p, _ = P.verify_sampled([0, 2], [0, 2], lg[:2], [1.0], np.zeros(2), np.zeros((1, 3)))
    assert a[0] == 0 and b[0] == 1 and p[1] == 0
    # no distribution after the accepted draft: no token
    a, b, p, _ = P.verify_sampled([0, 2], [0, 1], lg[:2], [1.0], np.zeros(2), np.zeros((1, 3)))
    assert a[0] == 1 and b[0] == -1
    a, b, p, _ = P.verify_sampled([0, 2], [0, 2], lg[[2, 0]], [1.0], np.zeros(2), np.zeros((1, 3)))
    assert a[0] == 0 and b[0] == -1 and p[1] == 0
    # a draft that holds all the probability is always taken
    a, b, p, _ = P.verify_sampled([0, 2], [0, 1], np.array([[-inf, 3.0, -inf], [0.0, 0, 0]]), [0.5],
                                  np.full(2, 1 - 2.0 ** -24), np.zeros((1, 3)))
    assert a[0] == 1 and p[1] == 1
