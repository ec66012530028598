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
from test_gpu_verify_sampled import _run as _verify

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


# ------------------------------------------------------------------ long contexts and chunks


@pytest.mark.parametrize("H,G,hd", [(8, 2, 64), (7, 1, 128), (4, 4, 64)])
@pytest.mark.parametrize("n", [1, 8])
@pytest.mark.parametrize("sinks", [False, True])
def test_attend_units_cut_into_more_parts_than_a_warp_has_lanes(H, G, hd, n, sinks):
    """One request over 32K keys with few KV heads: 38 to 53 parts a unit by the split's
    arithmetic, joined 32 at a time."""
    _check(_chunk("bf16", H, G, hd, 16, (n,), (32768 + 5,), sinks=sinks, seed=60 + n, wide=2))


@pytest.mark.parametrize("H,G,hd", [(8, 2, 64), (7, 1, 128)])
@pytest.mark.parametrize("sinks", [False, True])
def test_attend_first_parts_without_keys(H, G, hd, sinks):
    """The blocks of the first 24,000 of 32,768 keys are invalid: the first window of 32 parts
    sees nothing, and its maximum stays at -inf."""

    def edit(table, nb):
        table[0, :1500] = -1

    c = _chunk("bf16", H, G, hd, 16, (8,), (32768,), sinks=sinks, table_edit=edit, seed=62)
    _check(c, expect_status=binding.PE_ST_BLOCK_RANGE)
    # and nothing at all is there
    c["table"][:] = -1
    got, st = _attend(c)
    assert st == binding.PE_ST_BLOCK_RANGE and (got == 0).all()


@pytest.mark.parametrize("H,G,hd", [(8, 2, 64), (7, 1, 128)])
def test_attend_infinities_over_many_parts(H, G, hd):
    """A NaN value that only the last rows see, in a unit of many parts: the rows before it are
    computed again over all their keys."""
    n, L = 8, 32768
    c = _chunk("bf16", H, G, hd, 16, (n,), (L,), seed=63)
    clean = O.decode(c["vc"], "bf16")
    vc = clean.copy()
    vc[c["table"][0][(L - 2) // 16], :, (L - 2) % 16, 3] = np.nan  # seen by the last two rows
    ref, spread = P.chunk_attention(c["qsl"], c["seq"], O.decode(c["q"], "bf16").reshape(n, H, hd),
                                    O.decode(c["kc"], "bf16"), clean, c["table"])
    c["vc"] = _store(vc, "bf16")
    got, st = _attend(c)
    assert st == 0
    val = O.decode(host(got), "bf16").reshape(n, H, hd)
    want = ref.copy()
    want[n - 2:, :, 3] = np.nan
    fin = np.isfinite(want)
    np.testing.assert_array_equal(val[~fin], want[~fin])
    assert (np.abs(val - ref)[fin] <= (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 1e-4) * spread)[fin] + 1e-30).all()


@pytest.mark.parametrize("dtype,H,G,hd,bs", [("bf16", 8, 2, 64, 16), ("bf16", 7, 1, 128, 32), ("bf16", 4, 2, 64, 5),
                                             ("f32", 4, 2, 16, 4)])
def test_attend_long_chunks_over_long_contexts(dtype, H, G, hd, bs):
    _check(_chunk(dtype, H, G, hd, bs, (1100, 0, 601), (6000, 17, 5003), sinks=True, extra=3, seed=64))


CALLS = [("bf16", 8, 2, 64, 16), ("bf16", 7, 1, 128, 16), ("bf16", 4, 2, 64, 5), ("f32", 4, 2, 16, 4)]


@pytest.mark.parametrize("dtype,H,G,hd,bs", CALLS)
def test_attend_large_values(dtype, H, G, hd, bs):
    """Values up to the size that the header allows, 3.4e38 / (2^8 * keys), and scores that
    climb by nearly 2^8 in weight before the running maximum follows."""
    L = 700
    c = _chunk(dtype, H, G, hd, bs, (5, 1), (L, 40), seed=66)
    q, k, v = (O.decode(c[x], dtype) for x in ("q", "kc", "vc"))
    q[:] = 1.0
    t = np.arange(L)
    at = c["table"][0][t // bs], slice(None), t % bs
    k[at] = (np.minimum(t / 256.0, 1.0) * 5.4 / np.sqrt(hd))[:, None, None]  # s from 0 to 5.4 = 7.8 in log2
    v *= 0.9 * 3.4e38 / (2.0 ** 8 * L) / np.abs(v).max()
    c["q"], c["kc"], c["vc"] = _store(q, dtype), _store(k, dtype), _store(v, dtype)
    assert np.abs(O.decode(c["vc"], dtype)).max() > 1e33
    _check(c)


@pytest.mark.parametrize("dtype,H,G,hd,bs", CALLS)
def test_attend_sinks_that_are_not_finite(dtype, H, G, hd, bs):
    """-inf: no sink for that head; +inf and NaN: NaN where a row sees a key, zeros where it
    sees none.  A request in one part and one in several."""
    ns, Ls = (3, 6, 8), (1, 90, 3000)  # the first two rows see nothing
    c = _chunk(dtype, H, G, hd, bs, ns, Ls, sinks=True, seed=67)
    c["sink"][0], c["sink"][1], c["sink"][2] = -np.inf, np.inf, np.nan
    got, st = _attend(c)
    assert st == 0
    val = O.decode(host(got), dtype).reshape(c["T"], H, hd)
    assert (val[:2] == 0).all() and np.isnan(val[2:, 1:3]).all()
    q = O.decode(c["q"], dtype)[:, :H * hd].reshape(c["T"], H, hd)
    sink = np.where(np.arange(H) < 3, -np.inf, c["sink"])
    ref, spread = P.chunk_attention(c["qsl"], c["seq"], q, O.decode(c["kc"], dtype), O.decode(c["vc"], dtype),
                                    c["table"], sink)
    half, w = (2.0 ** -8, 2.0 ** -8 + 1e-4) if dtype == "bf16" else (2.0 ** -24, 2e-5)
    ok = np.abs(val - ref) <= half * np.abs(ref) + w * spread + 1e-30
    assert ok[:, 0].all() and ok[:, 3:].all()


@pytest.mark.parametrize("dtype,H,G,hd,bs,T,norm", [("bf16", 64, 8, 64, 16, 2500, True), ("bf16", 32, 8, 128, 16, 1300, False),
                                                    ("f32", 4, 2, 16, 4, 3001, True), ("f32", 6, 3, 40, 5, 2000, True)])
def test_append_many_rows_without_q_out(dtype, H, G, hd, bs, T, norm):
    """Rows past one walk of the CTAs, with the cache alone written."""
    _append(T, H, G, hd, bs, dtype, norm, pos0=10 ** 5, want_q=False, seed=65)


# ------------------------------------------------------------------ sampled verification


@pytest.mark.parametrize("V,apart", [(5000, 1), (5000, 2048), (20000, 4096), (5003, 256), (5003, 1)])
@pytest.mark.parametrize("lead", [2e-5, -2e-5, 0.0])
def test_close_scores_of_one_thread_beside_a_rejected_largest_logit(V, apart, lead):
    """The row's largest logit is the rejected draft's, and the two best of the others are read
    by the same thread, `apart` tokens from each other, with scores 2e-5 apart or equal.  The
    scores' terms are below 16: three fp32 roundings of 2^-24 * 16 each, 3e-6 at most."""
    cuda_or_skip()
    built()
    lg = np.full((2, V), -np.inf, np.float32)
    temp, draft, at = 0.05, 9, 1024
    lg[0, draft] = 3.0
    lg[0, at] = lg[0, at + apart] = 3.0 - 0.0625  # scores -1.25 beside the draft's 0: p(draft) = 0.64
    gumbel = np.full((1, V), -50.0, np.float32)
    gumbel[0, at], gumbel[0, at + apart], gumbel[0, draft] = 5.0, 5.0 + lead, 40.0
    c = dict(qsl=np.array([0, 2], np.int32), tok=np.array([1, draft], np.int32), dtype="f32", V=V, logits=lg,
             temp=np.array([temp], np.float32), u=np.array([0.0, 0.9], np.float32), gumbel=gumbel)
    acc, bon, p, st = _verify(c)
    assert st == 0 and acc.tolist() == [0] and abs(p[1] - 1 / (1 + 2 * np.exp(-1.25))) < 1e-6
    assert bon.tolist() == [at + apart if lead > 0 else at]


def test_infinite_noise_on_a_token_masked_with_the_types_lowest_value():
    """Only a logit of -inf keeps a token with infinite noise from winning: a mask of the
    type's lowest value does not, although (logit - max) / T is below fp32's range (the sum is
    rounded once)."""
    cuda_or_skip()
    built()
    for V in (64, 63):  # rows on and off the 16-byte grid
        lg = np.zeros((1, V), np.float32)
        lg[0, 7] = np.finfo(np.float32).min
        gumbel = np.zeros((1, V), np.float32)
        gumbel[0, 7], gumbel[0, 30] = np.inf, 1.0
        c = dict(qsl=np.array([0, 1], np.int32), tok=np.array([0], np.int32), dtype="f32", V=V, logits=lg,
                 temp=np.array([0.5], np.float32), u=np.zeros(1, np.float32), gumbel=gumbel)
        assert _verify(c)[1].tolist() == [7]
        gumbel[0, 7] = 100.0  # the largest finite noise does not lift it
        assert _verify(c)[1].tolist() == [30]
