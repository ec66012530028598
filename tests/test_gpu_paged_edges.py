"""The paged calls and sampled verification at edges that their first tests leave out: units
cut into many parts, long chunks, requests without rows, a wait that runs out."""

import numpy as np
import pytest

from oracle import pe_oracle as O
from oracle import pe_paged as P
from parity import built, cuda_or_skip, host
from speculative_drafting_gb300 import binding, runner, workloads as W
from test_gpu_paged import _append, _attend, _check, _chunk, _store

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,bs", [("bf16", 16), ("bf16", 5), ("f32", 4)])
@pytest.mark.parametrize("bad", [-4, 10 ** 6])
def test_bad_lengths_of_requests_without_rows_are_reported(dtype, bs, bad):
    c = _chunk(dtype, 4, 2, 64 if dtype == "bf16" else 16, bs, (3, 0, 2), (30, 20, 12), seed=41)
    want = _check(c)
    c["seq"] = np.array([30, bad, 12], np.int32)
    got, st = _attend(c)
    assert st == binding.PE_ST_BLOCK_RANGE
    np.testing.assert_array_equal(host(got), host(want))
