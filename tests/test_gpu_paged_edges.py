"""The paged calls and sampled verification at edges that their first tests leave out: units
cut into many parts, long chunks, requests without rows, a wait that runs out."""

import time

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


# ------------------------------------------------------------------ a wait that runs out


# (by the split's arithmetic some CTA's part has at least four tiles in each of these)
@pytest.mark.parametrize("H,G,hd,ns,Ls", [(8, 2, 64, (8,), (20000,)), (8, 2, 64, (1000, 5), (9000, 700)),
                                          (7, 1, 128, (9, 700), (2500, 8000))])
@pytest.mark.parametrize("slot", [2, 4])
def test_attend_wait_runs_out_and_the_context_survives(H, G, hd, ns, Ls, slot):
    """A slot of the key ring (0..3) or the value ring (4..7) whose tile never counts as
    there: every warp gives up within the limit, the status says so, and the next call with
    the same workspace matches the oracle."""
    torch = cuda_or_skip()
    built()
    c = _chunk("bf16", H, G, hd, 16, ns, Ls, sinks=True, seed=50 + slot)
    plan = binding.PagedAttention(H, G, hd, 16)
    d = {k: runner.to_device(c[k], "bf16") for k in ("q", "kc", "vc")}
    d |= {k: runner.to_device(c[k], "f32") for k in ("qsl", "seq", "table", "sink")}
    ws = plan.workspace(len(ns), c["T"])
    out = torch.zeros(c["T"], H * hd, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    rc = plan.lib.pe_test_chunk_attention_stall(
        plan.addr, slot, len(ns), c["T"], d["qsl"].data_ptr(), d["seq"].data_ptr(), d["q"].data_ptr(), H * hd,
        d["kc"].data_ptr(), d["vc"].data_ptr(), d["table"].data_ptr(), c["table"].shape[1], c["nb"],
        d["sink"].data_ptr(), out.data_ptr(), H * hd, ws.data_ptr(), ws.numel(),
        torch.cuda.current_stream().cuda_stream)
    assert rc == binding.PE_OK
    torch.cuda.synchronize()
    waited = time.perf_counter() - t0
    st, code = binding.read_status_ws(ws)
    assert st == binding.PE_ST_TIMEOUT and code == binding.PE_ERR_TIMEOUT
    assert 1.5 < waited < 30.0  # limits of 2 s, not a hang
    got, st = _attend(c, plan=plan, ws=ws)
    assert st == 0
    _check(c, got=got)
