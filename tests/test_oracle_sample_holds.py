"""Pins of the oracle's answer to which tokens may stand (sample_holds), against sampling itself and by hand."""

import numpy as np

from oracle import pe_tree as X


def allowed(x, temp, k, p, m, g):
    return [t for t in range(-1, len(x)) if X._sample_holds(x, temp, k, p, m, g, t)]


def test_where_the_answer_is_clear_it_alone_holds():
    rng = np.random.default_rng(0)
    for _ in range(300):
        V = int(rng.integers(1, 30))
        x = rng.standard_normal(V) * 2
        x[rng.random(V) < 0.2] = -np.inf
        g = -np.log(rng.exponential(size=V))
        a = (x, float(rng.choice([0.0, 0.5, 1.0])), int(rng.integers(0, V + 1)), float(rng.choice([1.0, 0.7, 0.2])),
             float(rng.choice([0.0, 0.1, 2.0])), g)
        tok, clear = X.sample([0, 1], x[None], [a[1]], [a[2]], [a[3]], [a[4]], g[None])
        assert tok[0] in allowed(*a)
        if clear[0]:
            assert allowed(*a) == [tok[0]]


def test_what_hangs_on_a_rounding():
    g = np.array([0.0, 1.0, 2.0, 3.0])
    x = np.zeros(4)
    assert allowed(x, 1.0, 0, 0.5, 0.0, g) == [1, 2]        # two weigh a half: the third stands at the bound
    assert allowed(x, 1.0, 2, 1.0, 0.0, g) == [1]           # a count is exact
    assert allowed(x, 1.0, 0, 1.0, 1.0, g) == [0, 1, 2, 3]  # so far as their weights are 1
    assert allowed(x, 1.0, 0, 1.0, 1.1, g) == [0]
    near = np.array([1.0, 1.0 + 1e-7, 0.9, 1.0 - 1e-3])
    assert allowed(x, 1.0, 0, 1.0, 0.0, near) == [0, 1]     # scores within fp32's roundings
    assert allowed(x, 1.0, 3, 1.0, 0.0, np.full(4, -np.inf)) == [-1]
    assert allowed(np.array([0.0, np.nan]), 1.0, 0, 0.9, 0.0, g[:2]) == [-1]
    inf = np.array([0.0, np.inf, 1.0, np.nan])
    assert allowed(x, 1.0, 0, 1.0, 0.0, inf) == [1]


def test_rows_of_no_request_stay():
    x = np.zeros((3, 2))
    ok = X.sample_holds([0, 1], x, None, None, None, None, np.zeros((3, 2)), np.array([0, -7, 1]))
    assert ok.tolist() == [True, True, False]
