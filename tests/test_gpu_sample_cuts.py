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
