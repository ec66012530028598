"""pe_sample, every row: its token has to be one that the formulas allow (oracle.pe_tree.sample_holds), in rows too
whose answer hangs on a rounding: a token that may be kept if the bounds of the weights move by 2e-5 of their size,
and whose score is not behind another's by more than the two's fp32 forms are off.  Rows behind the last request
stay as they were."""

import numpy as np
import pytest

from oracle import pe_oracle as O
from oracle import pe_tree as X
from test_gpu_sample import SETTINGS, _bits, case, run

pytestmark = pytest.mark.gpu


def check(c, **kw):
    got, st = run(c, **kw)
    ok = X.sample_holds(c["qsl"], O.decode(c["logits"], c["dtype"]), c["temp"], c["k"], c["p"], c["m"], c["g"], got)
    assert st == 0 and ok.all(), (np.flatnonzero(~ok), got[~ok])
    assert (got[c["qsl"][-1]:] == -7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["peaked", "flat", "ties", "equal"])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 64, 1000, 4099])
def test_small_vocabularies(dtype, kind, V):
    for seed in range(3):
        check(case((2, 0, 1, 3, 1, 1, 2, 1, 1, 1, 1, 1, 1, 1, 1, 1), V, dtype, kind, seed=V + seed, extra=2),
              pad=(V % 5, V % 3))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["peaked", "flat", "ties", "equal"])
def test_large_vocabularies(dtype, kind):
    check(case((1,) * len(SETTINGS), 201088, dtype, kind, seed=21, extra=1))
    ks = [(1.0, 0, 0.9, 0.0), (1.0, 0, 0.5, 0.02), (0.7, 5000, 0.9, 0.0), (1.0, 0, 0.01, 0.0), (1.5, 60000, 0.99, 0.0)]
    for V in (209001, 300001) if dtype == "f32" else (278001, 600001):
        check(case((1,) * 5, V, dtype, kind, settings=ks, seed=22), pad=(1, 3))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["peaked", "flat", "ties"])
def test_cuts_around_the_most_that_are_put_in_order(dtype, kind):
    ks = [(1.0, k, p, 0.0) for k, p in ((500, 1.0), (512, 0.99), (513, 1.0), (300, 0.9), (0, 0.97))]
    check(case((64,) * 5, 1500, dtype, kind, seed=23, settings=ks, extra=3), pad=(3, 2))
    ks = [(1.0, 3000, 1.0, 0.0), (1.0, 2500, 0.7, 0.0), (1.0, 0, 0.8, 0.0), (5.0, 8999, 0.999, 1e-9), (0.01, 4000, 1.0, 0.0)]
    c = case((9,) * 5, 9001, dtype, kind, settings=ks, seed=24)
    check(c)
    # all tokens within a few roundings of one another, and one far ahead
    x = 1.0 + O.decode(c["logits"], dtype) * 1e-6
    x[:, 50] = 2e4
    check(dict(c, logits=_bits(np.nan_to_num(x, neginf=-np.inf), dtype)))


def test_many_rows_in_two_launch_shapes():
    """The same rows alone and among 640: what hangs on a rounding may differ, each answer has to hold."""
    for dtype in ("f32", "bf16"):
        c = case((9, 1, 8, 0, 14) * 20, 3001, dtype, "flat", seed=25, extra=2)
        check(c)
        few = {k: v[:9] if k in ("logits", "g") else v[:1] if k in ("temp", "k", "p", "m") else v for k, v in c.items()}
        check(dict(few, qsl=c["qsl"][:2]))
