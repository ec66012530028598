"""The page calls on a workspace that other calls use too, in turn."""

import numpy as np
import pytest

from parity import cuda_or_skip
from speculative_drafting_gb300 import binding, runner
from test_gpu_pages import Device
from test_gpu_sample import case

pytestmark = pytest.mark.gpu


def test_one_workspace_for_sampling_and_pages():
    """What pe_sample leaves in it (of rows that none but its last kernel decides) is nothing to the page calls."""
    torch = cuda_or_skip()
    d = Device(24, 6, 80)
    T, V = 19, 9001
    c = case((1,) * T, V, "bf16", "flat", settings=(1.0, 0, 0.9, 0.0))
    size = max(binding.sample_workspace(T, T, V).numel(), d.ws.numel())
    d.ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    up = [runner.to_device(c[k], "f32") for k in ("qsl", "temp", "k", "p", "m", "g")]
    logits = runner.to_device(c["logits"], "bf16")
    token = torch.zeros(T, dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(0)
    for _ in range(6):
        for call in (lambda: d.reserve(np.arange(12), rng.integers(0, 25, 12)),
                     lambda: d.fork(np.arange(8), np.arange(12, 20), [3] * 8),
                     lambda: d.free(np.arange(24))):
            binding.sample(T, T, up[0], logits, V, *up[1:], token, d.ws)
            call()    # (checks the table, the counts and the caches)
