"""pe_verify_sampled against the fp64 oracle on the same logits and numbers.

Counts and tokens have to be equal wherever the oracle's decisions are clear: a
draft's number at least 1e-5 from its probability and the winning score ahead by
1e-4 (fp32 scores of size up to 40 carry roundings of 4e-6).  p_draft: the row's
normaliser is a sum of fp32 exponentials whose arguments (below 60 in size) carry a
few roundings, under 60 * 3 * 2^-24 = 1.1e-5 relative for the smallest weights and
far less for those that count: 1e-5 relative and 1e-7 absolute.
"""

import numpy as np
import pytest

from oracle import pe_oracle as O
from oracle import pe_paged as P
from parity import built, cuda_or_skip, host
from speculative_drafting_gb300 import binding, runner, workloads as W

pytestmark = pytest.mark.gpu


def _case(ns, V, dtype, temps=None, seed=0, barred=0.02, spread=2.0, extra=0):
    rng = np.random.default_rng(seed)
    B, T = len(ns), sum(ns)
    qsl = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    lg = rng.standard_normal((T + extra, V)) * spread
    tok = rng.integers(0, V, T + extra).astype(np.int32)
    if V > 4:
        lg[rng.random(lg.shape) < barred] = -np.inf
    for i in range(1, T):  # drafts that are often accepted
        top = lg[i - 1].max()
        share = rng.uniform(0.2, 0.95)
        lg[i - 1, tok[i]] = top + np.log(np.exp(lg[i - 1] - top).sum() * share / (1 - share))
    temps = rng.choice([0.0, 0.5, 1.0, 1.7], B) if temps is None else np.full(B, temps)
    return dict(qsl=qsl, tok=tok, dtype=dtype, temp=temps.astype(np.float32), V=V,
                logits=W.f32_to_bf16_bits(lg.astype(np.float32)) if dtype == "bf16" else lg.astype(np.float32),
                u=rng.random(T + extra).astype(np.float32), gumbel=-np.log(rng.exponential(size=(B, V))).astype(np.float32))


def _run(c, offset=0, with_p=True, stream=None):
    torch = cuda_or_skip()
    built()
    B, T, V = len(c["qsl"]) - 1, len(c["tok"]), c["V"]
    flat = c["logits"].reshape(-1)
    buf = np.zeros(flat.size + offset + 8, flat.dtype)
    buf[offset:offset + flat.size] = flat
    d = {k: runner.to_device(c[k], "f32") for k in ("qsl", "tok", "u", "gumbel")}
    temp = None if c["temp"] is None else runner.to_device(c["temp"], "f32")
    lg = runner.to_device(buf, c["dtype"])[offset:]
    acc, bon = (torch.full((B,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    p = torch.full((max(T, 1),), -7.0, device="cuda") if with_p else None
    ws = binding.verify_sampled_workspace(B, T, V)
    torch.cuda.synchronize()
    code = binding.PE_DTYPE_BF16 if c["dtype"] == "bf16" else binding.PE_DTYPE_F32
    binding.verify_sampled(B, T, d["qsl"], d["tok"], lg, V, code, temp, d["u"], d["gumbel"], acc, bon, p, ws,
                           stream=stream)
    torch.cuda.synchronize()
    return host(acc), host(bon), host(p) if with_p else None, binding.read_status_ws(ws)[0]


def _check(c, status=0, least_clear=0.9, **kw):
    acc, bon, p, st = _run(c, **kw)
    assert st == status
    temp = np.ones(len(acc)) if c["temp"] is None else c["temp"]
    ra, rb, rp, margin = P.verify_sampled(c["qsl"], c["tok"], O.decode(c["logits"], c["dtype"]), temp, c["u"], c["gumbel"])
    clear = margin > 1e-4
    assert clear.mean() >= least_clear
    np.testing.assert_array_equal(acc[clear], ra[clear])
    np.testing.assert_array_equal(bon[clear], rb[clear])
    if p is not None:
        rows = int(c["qsl"][-1])
        np.testing.assert_allclose(p[:rows], rp[:rows], rtol=1e-5, atol=1e-7)
        assert (p[rows:] == -7).all()
    return acc, bon


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [2, 3, 7, 64, 1000, 4099, 32003])
def test_ragged_batches(dtype, V):
    c = _case((1, 8, 0, 3, 9, 2, 1, 5, 0), V, dtype, seed=V, extra=2)
    for offset in (0, 1, 3):
        _check(c, offset=offset, least_clear=0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,n", [(1, 8), (24, 8)])
def test_full_vocabulary(dtype, B, n):
    acc, _ = _check(_case((n,) * B, 201088, dtype, seed=B))
    if B > 1:
        assert 0 < acc.mean() < n - 1


@pytest.mark.parametrize("temp", [None, 0.0, 1.0, 0.01, 1e-30, 50.0])
def test_temperatures(temp):
    c = _case((4, 4, 1, 7), 1500, "f32", temps=temp, seed=5)
    if temp is None:
        c["temp"] = None
    _check(c, least_clear=0.5)


def test_temperature_zero_is_greedy_verification():
    rng = np.random.default_rng(3)
    c = _case((3, 8, 1, 5), 999, "f32", temps=0.0, seed=3)
    lg = rng.integers(-3, 4, c["logits"].shape).astype(np.float32)  # many ties
    lg[2, 17] = np.nan
    c["logits"] = lg
    tgt = O.target_argmax(lg)
    for i in range(1, len(c["tok"])):
        if rng.random() < 0.7:
            c["tok"][i] = tgt[i - 1]
    acc, bon, _, st = _run(c)
    _, ra, rb = O.verify_greedy(c["qsl"], c["tok"], lg)
    np.testing.assert_array_equal(acc, ra)
    np.testing.assert_array_equal(bon, rb)
    assert st == 0


def test_no_temperature_array_no_probabilities():
    _check(dict(_case((3, 8, 1), 777, "bf16", temps=1.0, seed=6), temp=None), with_p=False, least_clear=0.6)


def test_one_token_vocabulary():
    c = dict(_case((3, 1), 2, "f32", temps=1.0), V=1)
    c["logits"], c["gumbel"] = c["logits"][:, :1].copy(), c["gumbel"][:, :1].copy()
    c["logits"][:], c["tok"][:] = 0.25, 0
    acc, bon, p, st = _run(c)  # the one token holds all the probability
    assert acc.tolist() == [2, 0] and bon.tolist() == [0, 0] and (p == 1).all() and st == 0


def test_rows_without_a_distribution():
    V = 300
    inf = np.inf
    c = _case((2, 2, 2, 2, 1), V, "f32", temps=1.0, seed=8, barred=0.0)
    c["u"][:] = 0.0
    lg = c["logits"]
    lg[0, 5] = np.nan            # request 0: the first row: rejected, no token
    lg[3] = -inf                 # request 1: accepted, then nothing to draw from
    lg[4, 7] = inf               # request 2
    lg[6] = -inf                 # request 3: all the mass on the draft itself, with u past it
    lg[6, c["tok"][7]] = 1.0
    c["u"][7] = 2.0
    acc, bon, p, st = _run(c)
    assert acc.tolist() == [0, 1, 0, 0, 0]
    assert bon.tolist()[:4] == [-1, -1, -1, -1] and bon[4] >= 0
    assert p[1] == 0 and p[5] == 0 and p[7] == 1
    assert st == binding.PE_ST_SAMPLING


def test_bad_tokens_and_temperatures_are_reported():
    c = _case((3, 3), 50, "f32", temps=1.0, seed=9)
    c["u"][:] = 0.0
    c["tok"][1], c["tok"][5] = 50, -1
    acc, bon, p, st = _run(c)
    assert st == binding.PE_ST_TOKEN_RANGE and acc.tolist() == [0, 1] and p[1] == 0 and p[5] == 0
    assert 0 <= bon[0] < 50 and 0 <= bon[1] < 50
    c = _case((3, 3), 50, "f32", temps=1.0, seed=9)
    c["temp"][:] = [-1.0, np.nan]
    acc, bon, _, st = _run(c)
    assert st == binding.PE_ST_SAMPLING
    zero = _run(dict(c, temp=np.zeros(2, np.float32)))
    np.testing.assert_array_equal(acc, zero[0])
    np.testing.assert_array_equal(bon, zero[1])


def test_long_and_empty_requests():
    c = _case((1500, 1, 700), 60, "f32", temps=1.0, seed=12, barred=0.0)
    c["u"][:1200] = 0.0  # a long accepted prefix
    acc, _ = _check(c, least_clear=0.3)
    assert acc[0] >= 1199
    acc, bon, _, st = _run(dict(_case((1,), 9, "f32"), qsl=np.zeros(4, np.int32), tok=np.zeros(0, np.int32),
                                logits=np.zeros((0, 9), np.float32), u=np.zeros(0, np.float32),
                                gumbel=np.zeros((3, 9), np.float32), temp=np.ones(3, np.float32)))
    assert acc.tolist() == [0, 0, 0] and bon.tolist() == [-1, -1, -1] and st == 0


@pytest.mark.parametrize("qsl", [(0, 5, 3, 40), (2, 4, 6, 8), (0, -1, 4, 12)])
def test_bad_offsets_are_reported(qsl):
    c = _case((4, 4, 4), 100, "f32", temps=1.0)
    assert _run(dict(c, qsl=np.array(qsl, np.int32)))[3] & binding.PE_ST_ROWS_RANGE


def test_replays_in_a_graph_and_shares_a_workspace():
    torch = cuda_or_skip()
    built()
    cs = [_case((8, 3, 1, 8), 5001, "f32", seed=s) for s in (1, 2)]
    want = [_run(c) for c in cs]
    ws = binding.verify_sampled_workspace(4, 20, 5001)
    s = torch.cuda.Stream()
    held = []
    for c in cs:
        d = {k: runner.to_device(c[k], "f32") for k in ("qsl", "tok", "logits", "temp", "u", "gumbel")}
        o = [torch.zeros(4, dtype=torch.int32, device="cuda") for _ in range(2)] + [torch.zeros(20, device="cuda")]

        def call(d=d, o=o):
            binding.verify_sampled(4, 20, d["qsl"], d["tok"], d["logits"], 5001, binding.PE_DTYPE_F32, d["temp"],
                                   d["u"], d["gumbel"], *o, ws, stream=s)

        with torch.cuda.stream(s):
            call()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
        held.append((g, o))
    for _ in range(3):
        for (g, o), w in zip(held, want):
            for t in o:
                t.fill_(-9)
            g.replay()
            torch.cuda.synchronize()
            for t, x in zip(o, w):
                np.testing.assert_array_equal(host(t), x)


@pytest.mark.parametrize("temp", [1e30, 3e38, np.inf])
def test_high_temperatures_draw_from_the_allowed_tokens_alike(temp):
    c = _case((4, 1, 7), 1500, "f32", temps=temp, seed=15)
    acc, bon = _check(c, least_clear=0.6)
    # every score is the noise alone, of the tokens with a logit above -inf
    row = c["qsl"][1]
    assert bon[1] == np.argmax(np.where(np.isneginf(c["logits"][row]), -np.inf, c["gumbel"][1]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 5003])
def test_infinite_noise(dtype, V):
    """-log(0) among the noise: that token wins, unless it has no probability or is the
    rejected draft."""
    c = _case((1, 1, 2), V, dtype, temps=1.0, seed=16, barred=0.0)
    c["u"][:] = 0.999999  # the draft of request 2 is rejected
    c["gumbel"][0, 11] = np.inf
    lg = O.decode(c["logits"], dtype).astype(np.float32)
    lg[1, 7] = -np.inf
    c["logits"] = W.f32_to_bf16_bits(lg) if dtype == "bf16" else lg
    c["gumbel"][1, 7] = c["gumbel"][1, 23] = np.inf
    draft = int(c["tok"][3])
    c["gumbel"][2, draft] = c["gumbel"][2, (draft + 5) % V] = np.inf
    c["gumbel"][2, (draft + 9) % V] = -np.inf
    acc, bon, _, st = _run(c)
    assert st == 0 and acc.tolist() == [0, 0, 0] and bon.tolist() == [11, 23, (draft + 5) % V]


def test_large_logits_at_low_temperatures():
    """Quotients far past fp32's range: the largest logit wins, wherever it stands."""
    c = _case((1, 1, 1), 3000, "f32", temps=1e-6, seed=17, barred=0.0)
    c["logits"] *= np.float32(1e36)
    acc, bon, _, st = _run(c)
    assert st == 0 and bon.tolist() == c["logits"].argmax(1).tolist()
    c["logits"] -= np.float32(2e37)  # all below zero
    assert _run(c)[1].tolist() == c["logits"].argmax(1).tolist()


def test_inputs_written_right_before_the_call():
    """Calls in a row on one stream whose inputs an earlier kernel of the stream has just
    written, without a host wait in between: each sees its own."""
    torch = cuda_or_skip()
    cases = [_case((8, 1, 4, 8), 5000, "f32", temps=t, seed=40 + i) for i, t in enumerate((1.0, 0.7, 1.3))]
    want = [P.verify_sampled(c["qsl"], c["tok"], c["logits"], c["temp"], c["u"], c["gumbel"]) for c in cases]
    names = ("tok", "logits", "temp", "u", "gumbel")
    src = [{k: runner.to_device(c[k], "f32") for k in names} for c in cases]
    buf = {k: torch.empty_like(src[0][k]) for k in names}
    qsl = runner.to_device(cases[0]["qsl"], "f32")
    T, V = cases[0]["logits"].shape
    acc, bon = (torch.empty(24, 4, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = binding.verify_sampled_workspace(4, T, V)
    for i in range(24):
        for k in names:
            buf[k].copy_(src[i % 3][k])
        binding.verify_sampled(4, T, qsl, buf["tok"], buf["logits"], V, binding.PE_DTYPE_F32, buf["temp"], buf["u"],
                               buf["gumbel"], acc[i], bon[i], None, ws)
    acc, bon = host(acc), host(bon)
    for i in range(24):
        ra, rb, _, margin = want[i % 3]
        clear = margin > 1e-4
        assert clear.mean() >= 0.5
        np.testing.assert_array_equal(acc[i][clear], ra[clear])
        np.testing.assert_array_equal(bon[i][clear], rb[clear])
