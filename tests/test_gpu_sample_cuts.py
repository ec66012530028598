"""pe_sample: cuts that more than one kernel of it can decide, each against the rule itself."""

import numpy as np
import pytest

from oracle import pe_oracle as O
from oracle import pe_tree as X
from speculative_drafting_gb300 import binding
from test_gpu_sample import _bits, case, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("min_p", [1.0000002, 1.5, 2.0, float("inf")])
def test_min_p_above_one_keeps_the_first_token(dtype, min_p):
    """No token weighs as much: the first of the order, which is always kept, is the answer whatever the noise,
    with the largest logit once, in a few places and in more than are put in order, alone and with the other cuts."""
    cuts = [(0, 1.0), (600, 1.0), (0, 0.9), (5000, 0.5), (3, 0.9)]
    for V, kind in ((1, "flat"), (1000, "equal"), (1000, "ties"), (9001, "flat"), (201088, "flat"), (201088, "equal")):
        c = case((1,) * len(cuts), V, dtype, kind, seed=V, settings=[(1.0, k, p, min_p) for k, p in cuts])
        x = O.decode(c["logits"], dtype).copy()
        if kind == "flat" and V > 1:
            x[:, [V // 3, V // 2, V - 1]] = 9.0 if V < 10000 else x.max()
            c["logits"] = _bits(x, dtype)
            c["g"][:, V - 1] = 50.0
        got, st = run(c)
        assert st == 0
        assert got.tolist() == O.target_argmax(O.decode(c["logits"], dtype)).tolist(), (V, kind)
    c = case((2,), 3000, dtype, "equal", settings=(1.0, 0, 1.0, min_p))
    c["g"][0, 0] = -np.inf    # nothing else is kept
    got, st = run(c)
    assert got.tolist() == [-1, 0] and st == binding.PE_ST_SAMPLING
    want = X.sample(c["qsl"], O.decode(c["logits"], dtype), c["temp"], c["k"], c["p"], c["m"], c["g"])[0]
    assert got.tolist() == want.tolist()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_more_than_top_k_where_top_p_is_almost_one(dtype):
    """One token and 199,999 of 1.9 * 2^-40 of its weight, the first 100,000 kept by top_k, 65,000 or so of them by
    top_p = 1 - 2^-24.  The noise lets tokens that top_p rejects win one after another, and is largest where top_k
    has cut."""
    V, k = 200000, 100000
    x = np.full((3, V), np.float32(np.log(1.9) - 40 * np.log(2.0)))
    x[:, 0] = 0.0
    c = case((1, 1, 1), V, dtype, settings=[(1.0, k, float(np.float32(1 - 2.0 ** -24)), 0.0)] * 3)
    c["logits"] = _bits(x, dtype)
    c["g"][:] = 0.0
    for row, n in enumerate((7, 8, 12)):        # as many winners that are rejected, the last ranks first
        c["g"][row, k - 1 - np.arange(n)] = 200.0 - np.arange(n)
        c["g"][row, 10] = 100.0
        c["g"][row, k:] = 1000.0
    got, st = run(c)
    # The sum before any of the first k is in 1 + [0, 1e5 * 1.9 * 2^-40 = 1.73e-7], p of all is 1 + 1.73e-7 - 2^-24
    # = 1 + 1.13e-7: all of them are within 1e-5 of the bound, so each may be kept.  Not those behind the k-th, and
    # where as many winners as are raced for have been rejected, not those either.
    assert st == 0 and (got < k).all()
    assert got[0] == 10 and all(t == 10 or t < k - 7 for t in got)


@pytest.mark.parametrize("qsl,status", [((0, 2, 1, 4), True), ((0, 3, 3, 2, 5), True), ((1, 2), True), ((0, 0, 5), True),
                                        ((0, 2, 2, 4), False), ((0, 0, 0, 0), False)])
def test_bad_offsets_of_any_request_are_reported(qsl, status):
    """Those of requests that no row is looked up in too."""
    qsl = np.array(qsl, np.int32)
    c = dict(case((1,) * (len(qsl) - 1), 300, "f32", settings=(1.0, 5, 0.9, 0.0)), qsl=qsl)
    g = case((4,), 300, "f32")
    c.update(logits=g["logits"], g=g["g"])
    _, st = run(c)
    assert st == (binding.PE_ST_ROWS_RANGE if status else 0)


def test_bad_offsets_among_many_requests_are_reported():
    B = 3000
    qsl = np.concatenate([np.arange(B), [B]]).astype(np.int32)
    c = dict(case((1,) * B, 40, "f32", settings=(1.0, 5, 0.9, 0.0)), qsl=qsl)
    assert run(c)[1] == 0
    qsl[1777] = B
    assert run(c)[1] == binding.PE_ST_ROWS_RANGE


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 3000, 201088])
def test_logits_of_the_lowest_value(dtype, V):
    """Tokens masked by the type's lowest value: quotients by temperatures below 1 are past fp32's range."""
    low = {"f32": np.finfo(np.float32).max, "bf16": np.float32(2.0 ** 127 * (2 - 2.0 ** -7))}[dtype]
    cuts = [(0, 1.0), (V - 1, 1.0), (5, 1.0), (0, 0.9)]
    some = np.unique(np.array([1, 2, V // 3, V // 2, V - 2]))
    for temp in (0.7, 1.0, 1e-30, 3.0):
        c = case((1,) * len(cuts), V, dtype, "equal", seed=V, settings=[(temp, k, p, 0.0) for k, p in cuts])
        x = np.full((len(cuts), V), -low, np.float64)
        x[:, some] = np.arange(len(some)) * 1e-3
        c["logits"] = _bits(x, dtype)
        x = O.decode(c["logits"], dtype)
        got, st = run(c)
        assert st == 0 and X.sample_holds(c["qsl"], x, c["temp"], c["k"], c["p"], c["m"], c["g"], got).all()
        assert np.isin(got, some).all()
        # infinite noise wins where the token is kept: at the lowest index
        c["g"][:, [0, 7, V - 1]] = np.inf
        got, st = run(c)
        assert st == 0 and got[:2].tolist() == [0, 0]
        assert X.sample_holds(c["qsl"], x, c["temp"], c["k"], c["p"], c["m"], c["g"], got).all()
        # nothing but lowest values can win
        c["g"][:, [0, 7, V - 1]] = 0.0
        c["g"][:, some] = -np.inf
        got, st = run(c)
        if temp < 1.0:
            assert got[:2].tolist() == [-1, -1] and st == binding.PE_ST_SAMPLING
        else:
            assert got[:2].tolist() == [0, 0]   # (scores of the same 64-bit number)
        assert X.sample_holds(c["qsl"], x, c["temp"], c["k"], c["p"], c["m"], c["g"], got).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [400, 3000, 201088])
def test_infinite_noise_among_logits_of_the_lowest_value(dtype, V):
    """A masked token that its noise lets win, away from the tokens that are not masked: no thread that holds it has
    another logit, and its distance to the largest is past fp32's range."""
    low = {"f32": np.finfo(np.float32).max, "bf16": np.float32(2.0 ** 127 * (2 - 2.0 ** -7))}[dtype]
    at = V // 5
    for temp in (0.7, 1e-30, 1.0):
        c = case((1, 1, 1), V, dtype, "equal", seed=V, settings=[(temp, 0, 1.0, 0.0), (temp, V - 1, 1.0, 0.0), (temp, 5, 1.0, 0.0)])
        x = np.full((3, V), -low, np.float64)
        x[:, [V - 9, V - 1]] = 1.0
        c["logits"] = _bits(x, dtype)
        c["g"][:, at] = np.inf
        got, st = run(c)
        # (five tokens: the two and the first three masked ones)
        assert st == 0 and got[:2].tolist() == [at, at] and got[2] in (V - 9, V - 1, 0, 1, 2)


@pytest.mark.parametrize("V,T", [(40, 1), (40, 3), (9001, 3)])
def test_bad_offsets_among_more_requests_than_rows_are_reported(V, T):
    B = 65535
    qsl = np.minimum(np.arange(B + 1), T).astype(np.int32)
    g = case((T,), V, "f32")
    one = lambda v, ty: np.full(B, v, ty)  # noqa: E731
    c = dict(qsl=qsl, dtype="f32", V=V, logits=g["logits"], g=g["g"], temp=one(1.0, np.float32), k=one(5, np.int32),
             p=one(0.9, np.float32), m=one(0.0, np.float32))
    assert run(c)[1] == 0
    for at in (5, 300, 40000, B - 1):
        c["qsl"] = qsl.copy()
        c["qsl"][at] = T + 1
        assert run(c)[1] == binding.PE_ST_ROWS_RANGE, at
