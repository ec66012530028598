"""The paged attention calls against the fp64 oracle on the same stored inputs.

Tolerances, from the arithmetic (bf16: half a step is 2^-8 of the value):
  append   the result is rounded once; before that, fp32 products and the angle's
           fp32 rounding move it by at most 2e-6 of the pair's length (a dozen
           roundings of 2^-24).  |got - ref| <= h |ref| + 2e-6 |pair|, h = 2^-8 in
           bf16 and 2^-24 in fp32.  v is a copy: bit-exact.
  attend   in bf16 the weights may be rounded to bf16 before the product with v
           (relative 2^-8 each, the sum of the weights is not rounded), and the
           scores carry fp32 rounding (below 1e-4 of a weight): the error is at
           most (2^-8 + 1e-4) sum_t p_t |v_t|, then one rounding of the result.
           In fp32 the scores' rounding alone: 2e-5 sum_t p_t |v_t|.  A weight below
           fp32's normal range 2^-126 (a sink far above every score) may flush to 0:
           at most L * 2^-126 * max |v| < 4096 * 1.2e-38 * 8 < 1e-30 absolute.
"""

import numpy as np
import pytest

from oracle import pe_oracle as O
from oracle import pe_paged as P
from parity import built, cuda_or_skip, host
from speculative_drafting_gb300 import binding, runner, workloads as W

pytestmark = pytest.mark.gpu


def _store(x, dtype):
    return W.f32_to_bf16_bits(x.astype(np.float32)) if dtype == "bf16" else x.astype(np.float32)


def _dev(x, dtype="f32"):
    return runner.to_device(x, dtype)


def _value(t, dtype):
    return O.decode(host(t), dtype)


# ------------------------------------------------------------------ append


def _append(T, H, G, hd, bs, dtype, norm, pos0=0, pad=0, want_q=True, seed=0):
    torch = cuda_or_skip()
    built()
    rng = np.random.default_rng(seed)
    nb = (T + bs - 1) // bs + 2
    width = (H + 2 * G) * hd
    qkv = _store(rng.standard_normal((T, width + pad)) * 2, dtype)
    gq, gk = ((_store(1 + 0.2 * rng.standard_normal(hd), dtype) for _ in range(2)) if norm else (None, None))
    kc, vc = (_store(rng.standard_normal((nb, G, bs, hd)), dtype) for _ in range(2))
    pos = pos0 + rng.integers(0, 50, T).cumsum()
    slot = rng.permutation(nb * bs)[:T].astype(np.int64)
    slot[rng.random(T) < 0.2] = -1
    plan = binding.PagedAttention(H, G, hd, bs, dtype=dtype)
    ws = plan.append_workspace()
    dk, dv = _dev(kc, dtype), _dev(vc, dtype)
    q = torch.full((T, H, hd), 7.0, dtype=dk.dtype, device="cuda") if want_q else None
    d_qkv = _dev(qkv, dtype)[:, :width]
    args = (T, d_qkv, _dev(gq, dtype) if norm else None, _dev(gk, dtype) if norm else None,
            _dev(pos.astype(np.int64)), _dev(slot), nb, q, dk, dv, ws)
    plan.append(*args)
    torch.cuda.synchronize()
    assert binding.read_status_ws(ws)[0] == 0
    dec = lambda a: None if a is None else O.decode(a, dtype)  # noqa: E731
    ref = P.qkv_append(dec(qkv[:, :width]), H, G, dec(gq), dec(gk), pos, slot, dec(kc), dec(vc))
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24

    def close(got, want):
        a, b = np.split(want, 2, -1)
        pair = np.sqrt(a * a + b * b)
        tol = half * np.abs(want) + 2e-6 * np.concatenate([pair, pair], -1)
        bad = np.abs(got - want) > tol
        assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])

    if want_q:
        close(_value(q, dtype), ref[0])
    close(_value(dk, dtype), ref[1])
    np.testing.assert_array_equal(_value(dv, dtype), ref[2])
    # slots that no row names keep their bytes
    left = np.ones(nb * bs, bool)
    left[slot[slot >= 0]] = False
    for got, was in ((dk, kc), (dv, vc)):
        g = host(got).transpose(0, 2, 1, 3).reshape(nb * bs, G, hd)
        w = was.transpose(0, 2, 1, 3).reshape(nb * bs, G, hd)
        np.testing.assert_array_equal(g[left], w[left])
    return plan, args


@pytest.mark.parametrize("dtype,H,G,hd,bs", [
    ("bf16", 64, 8, 64, 16), ("bf16", 32, 8, 128, 16), ("bf16", 28, 4, 128, 32), ("bf16", 5, 5, 64, 3),
    ("bf16", 3, 1, 128, 1), ("f32", 4, 2, 16, 4), ("f32", 6, 3, 40, 5), ("f32", 8, 2, 128, 16), ("f32", 1, 1, 8, 7)])
@pytest.mark.parametrize("T", [1, 3, 130])
@pytest.mark.parametrize("norm", [False, True])
def test_append(dtype, H, G, hd, bs, T, norm):
    _append(T, H, G, hd, bs, dtype, norm, seed=T)


def test_append_many_rows_far_positions_and_strided_rows():
    _append(2111, 32, 8, 128, 16, "bf16", True, pos0=10 ** 6, pad=64)
    _append(777, 4, 2, 16, 4, "f32", True, pos0=1 << 40, pad=8, seed=1)
    _append(65, 64, 8, 64, 16, "bf16", False, pad=8, want_q=False, seed=2)


def test_append_rows_of_zeros_and_odd_values():
    """A zero row has norm 0 / sqrt(eps); infinities and NaN stay in their head."""
    torch = cuda_or_skip()
    built()
    H, G, hd, T = 4, 2, 64, 3
    x = torch.randn(T, (H + 2 * G) * hd, device="cuda").bfloat16()
    x[0] = 0
    x[1, :hd] = float("inf")
    x[2, 5 * hd + 3] = float("nan")  # the second k head
    plan = binding.PagedAttention(H, G, hd, 16)
    gain = torch.ones(hd, device="cuda").bfloat16()
    q = torch.empty(T, H, hd, device="cuda").bfloat16()
    k, v = torch.zeros(2, 1, G, 16, hd, device="cuda").bfloat16()
    pos, slot = torch.arange(T, device="cuda"), torch.arange(T, device="cuda")
    plan.append(T, x, gain, gain, pos, slot, 1, q, k, v, plan.append_workspace())
    assert (q[0] == 0).all() and (k[0, :, 0] == 0).all()
    assert torch.isnan(q[1, 0]).all() and torch.isfinite(q[1, 1:]).all() and torch.isfinite(q[2]).all()
    assert torch.isnan(k[0, 1, 2]).all() and torch.isfinite(k[0, 0]).all()
    assert torch.isfinite(v).all()


def test_append_reports_slots_past_the_pool_and_keeps_its_status():
    torch = cuda_or_skip()
    plan, args = _append(9, 8, 2, 64, 16, "bf16", False)
    nb, k, v, ws = args[6], args[8], args[9], args[10]
    before = k.clone(), v.clone()
    slot = torch.full((9,), -5, dtype=torch.int64, device="cuda")
    slot[4] = nb * 16
    slot[5] = 1 << 40
    plan.append(*args[:5], slot, *args[6:])
    assert binding.read_status_ws(ws, clear=False)[0] == binding.PE_ST_BLOCK_RANGE
    assert torch.equal(k, before[0]) and torch.equal(v, before[1])
    plan.append(*args)  # a call without a fault does not clear the word
    assert binding.read_status_ws(ws)[0] == binding.PE_ST_BLOCK_RANGE
    assert binding.read_status_ws(ws)[0] == 0


# ------------------------------------------------------------------ attention


def _chunk(dtype, H, G, hd, bs, ns, Ls, sinks=False, pad=0, extra=0, seed=0, poison=False, table_edit=None,
           spare=2, wide=0, scale=1.0):
    """Random pages for the requests (rows ns, lengths Ls); returns what the call needs, on
    the host.  poison: everything outside the visible positions is NaN or infinite."""
    rng = np.random.default_rng(seed)
    B, T = len(ns), sum(ns)
    qsl = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    blocks = [(max(L, 0) + bs - 1) // bs for L in Ls]
    mb, nb = max(max(blocks), 1) + wide, sum(blocks) + spare
    ids, table, o = rng.permutation(nb), np.full((B, mb), -1, np.int32), 0
    for r in range(B):
        table[r, :blocks[r]] = ids[o:o + blocks[r]]
        o += blocks[r]
    kc, vc = (rng.standard_normal((nb, G, bs, hd)) for _ in range(2))
    if poison:
        seen = np.zeros((nb, bs), bool)
        for r in range(B):
            t = np.arange(max(Ls[r], 0))
            seen[table[r, t // bs], t % bs] = True
        for c in (kc, vc):
            c.transpose(0, 2, 1, 3)[~seen] = rng.choice([np.nan, np.inf, -np.inf], ((~seen).sum(), G, hd))
    if table_edit:
        table_edit(table, nb)
    q = rng.standard_normal((T + extra, H * hd + pad)) * scale
    sink = rng.standard_normal(H).astype(np.float32) if sinks else None
    return dict(dtype=dtype, H=H, G=G, hd=hd, bs=bs, qsl=qsl, seq=np.array(Ls, np.int32), q=_store(q, dtype),
                kc=_store(kc, dtype), vc=_store(vc, dtype), table=table, nb=nb, sink=sink, T=T + extra)


def _attend(c, out=None, stream=None, plan=None, ws=None):
    torch = cuda_or_skip()
    built()
    plan = plan or binding.PagedAttention(c["H"], c["G"], c["hd"], c["bs"], dtype=c["dtype"])
    d = {k: _dev(c[k], c["dtype"]) for k in ("q", "kc", "vc")}
    d |= {k: _dev(c[k]) for k in ("qsl", "seq", "table")}
    d["sink"] = None if c["sink"] is None else _dev(c["sink"])
    ws = plan.workspace(len(c["seq"]), c["T"]) if ws is None else ws
    if out is None:
        out = torch.full((c["T"], c["H"] * c["hd"] + 8), 3.0, dtype=d["q"].dtype, device="cuda")[:, :c["H"] * c["hd"]]
    torch.cuda.synchronize()
    plan.attend(len(c["seq"]), c["T"], d["qsl"], d["seq"], d["q"], d["kc"], d["vc"], d["table"], c["nb"], out, ws,
                sink=d["sink"], stream=stream)
    torch.cuda.synchronize()
    return out, binding.read_status_ws(ws)[0]


def _check(c, expect_status=0, got=None):
    if got is None:
        got, st = _attend(c)
        assert st == expect_status
    dtype, H, hd = c["dtype"], c["H"], c["hd"]
    q = O.decode(c["q"], dtype)[:, :H * hd].reshape(c["T"], H, hd)
    ref, spread = P.chunk_attention(c["qsl"], c["seq"], q, O.decode(c["kc"], dtype), O.decode(c["vc"], dtype),
                                    c["table"], c["sink"])
    val = _value(got, dtype).reshape(c["T"], H, hd)
    rows = int(c["qsl"][-1])
    half, w = (2.0 ** -8, 2.0 ** -8 + 1e-4) if dtype == "bf16" else (2.0 ** -24, 2e-5)
    bad = ~(np.abs(val[:rows] - ref[:rows]) <= half * np.abs(ref[:rows]) + w * spread[:rows] + 1e-30)
    assert not bad.any(), (np.argwhere(bad)[:4], val[:rows][bad][:4], ref[:rows][bad][:4], bad.mean())
    assert (val[rows:] == 3.0).all()  # rows behind the last request
    return got


SHAPES = [("bf16", 64, 8, 64, 16), ("bf16", 32, 8, 128, 16), ("bf16", 8, 2, 64, 8), ("bf16", 7, 1, 128, 64),
          ("bf16", 5, 5, 64, 24), ("bf16", 6, 2, 64, 5), ("bf16", 4, 2, 128, 256), ("f32", 4, 2, 16, 4),
          ("f32", 6, 3, 40, 5), ("f32", 8, 2, 128, 16)]


@pytest.mark.parametrize("dtype,H,G,hd,bs", SHAPES)
@pytest.mark.parametrize("sinks", [False, True])
def test_attend_small_ragged(dtype, H, G, hd, bs, sinks):
    """Rows and lengths around every edge: one token, no rows, no keys, more rows than
    positions (rows that see nothing), lengths around a block and a 128-key tile."""
    ns = (1, 0, 3, 2, 9, 4, 1, 5, 1, 17, 0)
    Ls = (1, 5, 3, 0, 4, 127, 128, 129, 16, 40, 0)
    _check(_chunk(dtype, H, G, hd, bs, ns, Ls, sinks=sinks, extra=3, poison=True, pad=16, wide=3))


@pytest.mark.parametrize("dtype,H,G,hd,bs", SHAPES[:4] + [("bf16", 128, 1, 64, 16), ("f32", 4, 2, 16, 4)])
@pytest.mark.parametrize("n,L", [(1, 700), (8, 1500), (33, 33), (40, 900), (129, 600), (300, 301), (257, 257)])
def test_attend_one_request(dtype, H, G, hd, bs, n, L):
    _check(_chunk(dtype, H, G, hd, bs, (n,), (L,), poison=True, seed=n))


@pytest.mark.parametrize("dtype,H,G,hd,bs", [("bf16", 64, 8, 64, 16), ("bf16", 32, 8, 128, 16)])
def test_attend_mixed_batch(dtype, H, G, hd, bs):
    """Prompts, chunks on a cache, verify rows and single tokens in one call."""
    ns = (1, 8, 200, 1, 0, 64, 8, 9, 1, 31)
    Ls = (2300, 1030, 200, 77, 500, 900, 8, 3001, 1, 640)
    _check(_chunk(dtype, H, G, hd, bs, ns, Ls, sinks=True, extra=5, poison=True, seed=3))


def test_attend_many_requests():
    rng = np.random.default_rng(8)
    ns = rng.integers(0, 4, 300).tolist()
    Ls = [int(n + rng.integers(0, 60)) for n in ns]
    _check(_chunk("bf16", 8, 2, 64, 16, ns, Ls, seed=9))
    _check(_chunk("f32", 4, 2, 16, 4, ns, Ls, seed=9))


def test_attend_more_requests_than_a_block_has_threads():
    rng = np.random.default_rng(18)
    ns = rng.integers(0, 2, 5000).tolist()
    Ls = [int(n + rng.integers(0, 9)) for n in ns]
    _check(_chunk("bf16", 2, 2, 64, 16, ns, Ls, seed=19))


def test_attend_extreme_scores():
    """Scores of some hundreds in either direction: one key takes all the weight, and the
    running maximum climbs by far more than any lazy rescaling may skip."""
    c = _chunk("bf16", 8, 2, 64, 16, (40, 8, 1), (900, 700, 513), scale=40.0, seed=21)
    _check(c)
    c["sink"] = np.array([np.inf, -np.inf, 500.0, -500.0, 0, 1, 2, 3], np.float32)
    c["sink"][0] = 3e4
    _check(c)


def test_attend_growing_scores_over_a_long_context():
    """Keys whose scores climb by a little in each tile."""
    c = _chunk("bf16", 4, 2, 64, 16, (8,), (4000,), seed=22)
    k = O.decode(c["kc"], "bf16")
    q = O.decode(c["q"], "bf16")
    q[:] = 1.0
    t = np.arange(4000)
    k[c["table"][0][t // 16], :, t % 16] = (t / 400.0)[:, None, None] + 0.1 * np.random.default_rng(1).standard_normal((4000, 2, 64))
    c["kc"], c["q"] = _store(k, "bf16"), _store(q, "bf16")
    _check(c)


@pytest.mark.parametrize("dtype,bs", [("bf16", 16), ("bf16", 5), ("f32", 4)])
def test_attend_bad_blocks_are_skipped_and_reported(dtype, bs):
    def edit(table, nb):
        table[0, 1] = -1
        table[1, 0] = nb
        table[2, :] = -7

    hd = 64 if dtype == "bf16" else 16
    c = _chunk(dtype, 4, 2, hd, bs, (3, 150, 2), (90, 260, 30), table_edit=edit, poison=False, seed=5)
    _check(c, expect_status=binding.PE_ST_BLOCK_RANGE)
    # a length past the table is clamped to it
    c = _chunk(dtype, 4, 2, hd, bs, (3, 1), (60, 33), seed=6)
    want, _ = _attend(c)
    over = dict(c, seq=c["seq"].copy())
    over["seq"][0] = c["table"].shape[1] * bs + 17
    got, st = _attend(over)
    assert st & binding.PE_ST_BLOCK_RANGE
    np.testing.assert_array_equal(host(got)[3:], host(want)[3:])
    neg = dict(c, seq=np.array([-4, 33], np.int32))
    got, st = _attend(neg)
    assert st == binding.PE_ST_BLOCK_RANGE and (host(got)[:3] == 0).all()


@pytest.mark.parametrize("qsl", [(0, 5, 3, 9), (0, 4, 40, 9), (1, 2, 3, 9), (0, -3, 4, 9)])
def test_attend_bad_offsets_are_reported(qsl):
    c = _chunk("bf16", 4, 2, 64, 16, (3, 3, 3), (30, 30, 30), seed=7)
    c["qsl"] = np.array(qsl, np.int32)
    _, st = _attend(c)
    assert st & binding.PE_ST_ROWS_RANGE


def test_attend_repeats_bit_for_bit_on_streams_and_in_graphs():
    torch = cuda_or_skip()
    c = _chunk("bf16", 64, 8, 64, 16, (8, 1, 150, 9), (1800, 900, 2000, 333), sinks=True, seed=11)
    want = _check(c)
    for _ in range(20):
        got, _ = _attend(c)
        assert torch.equal(got, want)
    s = torch.cuda.Stream()
    got, _ = _attend(c, stream=s)
    assert torch.equal(got, want)
    plan = binding.PagedAttention(64, 8, 64, 16)
    d = {k: _dev(c[k], "bf16") for k in ("q", "kc", "vc")}
    d |= {k: _dev(c[k]) for k in ("qsl", "seq", "table", "sink")}
    ws = plan.workspace(4, c["T"])
    out = torch.empty(c["T"], 64 * 64, dtype=torch.bfloat16, device="cuda")

    def call(st):
        plan.attend(4, c["T"], d["qsl"], d["seq"], d["q"], d["kc"], d["vc"], d["table"], c["nb"], out, ws,
                    sink=d["sink"], stream=st)

    with torch.cuda.stream(s):
        call(s)
    s.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]  # both use the one workspace
    for g in graphs:
        with torch.cuda.graph(g, stream=s):
            call(s)
    for g in (*graphs, *graphs):
        out.fill_(5.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    # the captured call follows its device arrays: other lengths, the same graph
    d["seq"].copy_(torch.tensor([700, 900, 151, 10], dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    _check(dict(c, seq=np.array([700, 900, 151, 10], np.int32)), got=out)


def test_two_calls_at_once():
    """Two streams, a workspace each."""
    torch = cuda_or_skip()
    cases = [_chunk("bf16", 64, 8, 64, 16, (8,) * 16, (1500,) * 16, seed=s) for s in (1, 2)]
    want = [_attend(c)[0] for c in cases]
    plan = binding.PagedAttention(64, 8, 64, 16)
    held = []
    for c in cases:
        d = {k: _dev(c[k], "bf16") for k in ("q", "kc", "vc")}
        d |= {k: _dev(c[k]) for k in ("qsl", "seq", "table")}
        held.append((c, d, plan.workspace(16, 128), torch.empty(128, 4096, dtype=torch.bfloat16, device="cuda"),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for c, d, ws, out, s in held:
            plan.attend(16, 128, d["qsl"], d["seq"], d["q"], d["kc"], d["vc"], d["table"], c["nb"], out, ws, stream=s)
    torch.cuda.synchronize()
    for (c, d, ws, out, s), w in zip(held, want):
        assert binding.read_status_ws(ws)[0] == 0 and torch.equal(out, w)


def test_attend_zero_rows():
    torch = cuda_or_skip()
    c = _chunk("bf16", 4, 2, 64, 16, (0, 0), (20, 30), extra=2, seed=12)
    out, st = _attend(c)
    assert st == 0 and (out == 3).all()
    plan = binding.PagedAttention(4, 2, 64, 16)
    ws = plan.workspace(2, 2)
    z = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    plan.attend(2, 0, t, t, z, z, z, t, 0, z, ws)
    assert binding.read_status_ws(ws)[0] == 0


@pytest.mark.parametrize("dtype,H,G,hd,bs", [("bf16", 64, 8, 64, 16), ("bf16", 28, 4, 128, 16),
                                             ("bf16", 6, 2, 64, 5), ("f32", 4, 2, 16, 4)])
@pytest.mark.parametrize("ns,Ls", [((9,), (9,)), ((300,), (300,)), ((8,), (3000,)), ((100, 5), (2100, 3)),
                                   ((40, 1, 8, 33), (41, 70, 500, 33))])
@pytest.mark.parametrize("sinks", [False, True])
def test_attend_infinities_and_nan_at_later_positions(dtype, H, G, hd, bs, ns, Ls, sinks):
    """What a row does not see does not enter it, be it infinite or NaN in the value or the
    key, although later rows of the same request do see it: those follow the formula."""
    c = _chunk(dtype, H, G, hd, bs, ns, Ls, sinks=sinks, extra=2, seed=31)
    rng = np.random.default_rng(5)
    kc, vc = O.decode(c["kc"], dtype), O.decode(c["vc"], dtype)
    for r, (n, L) in enumerate(zip(ns, Ls)):
        for t in range(max(L - n, 0) + 1, L, max(n // 5, 2)):  # visible from its own row on
            at = c["table"][r][t // bs], slice(None), t % bs
            vc[at][:, rng.integers(hd)] = rng.choice([np.nan, np.inf, -np.inf])
            if t > L - 2:
                kc[at][0] = np.nan
    c["kc"], c["vc"] = _store(kc, dtype), _store(vc, dtype)
    kc, vc = O.decode(c["kc"], dtype), O.decode(c["vc"], dtype)
    got, st = _attend(c)
    assert st == 0
    val = _value(got, dtype).reshape(c["T"], H, hd)
    assert (val[sum(ns):] == 3.0).all()
    q = O.decode(c["q"], dtype)[:, :H * hd].reshape(c["T"], H, hd)
    half, w = (2.0 ** -8, 2.0 ** -8 + 1e-4) if dtype == "bf16" else (2.0 ** -24, 2e-5)
    for r, (n, L) in enumerate(zip(ns, Ls)):
        for j in range(n):
            # one row as a request of its own, over the positions up to its own
            row = c["qsl"][r] + j
            with np.errstate(invalid="ignore"):
                ref, spread = P.chunk_attention([0, 1], [L - n + j + 1], q[row:row + 1], kc, vc,
                                                c["table"][r:r + 1], c["sink"])
            fin = np.isfinite(ref[0])
            np.testing.assert_array_equal(val[row][~fin], ref[0][~fin])
            err = np.abs(val[row] - np.where(fin, ref[0], 0))[fin]
            assert (err <= (half * np.abs(ref[0]) + w * spread[0])[fin] + 1e-30).all(), (r, j)


@pytest.mark.parametrize("H,G,hd", [(64, 8, 64), (28, 4, 128)])
@pytest.mark.parametrize("n,L", [(300, 300), (70, 2500), (8, 90)])
@pytest.mark.parametrize("late", [False, True])
def test_attend_infinities_and_nan_that_all_rows_see(H, G, hd, n, L, late):
    """A value that every row sees reaches every row, in its column and KV head alone; with
    one more that only the last row sees, beside it."""
    c = _chunk("bf16", H, G, hd, 16, (n,), (L,), seed=33)
    vc = O.decode(c["vc"], "bf16")
    clean = vc.copy()
    vc[c["table"][0][0], 0, 0, 5] = np.nan
    vc[c["table"][0][0], 1, 0, 9] = -np.inf
    if late:
        vc[c["table"][0][(L - 1) // 16], 0, (L - 1) % 16, 11] = np.inf
    c["vc"] = _store(vc, "bf16")
    got, st = _attend(c)
    assert st == 0
    val = _value(got, "bf16").reshape(n, H, hd)
    c["vc"] = _store(clean, "bf16")
    ref, spread = P.chunk_attention(c["qsl"], c["seq"], O.decode(c["q"], "bf16").reshape(n, H, hd),
                                    O.decode(c["kc"], "bf16"), clean, c["table"])
    want = ref.copy()
    hg = H // G
    want[:, :hg, 5] = np.nan
    want[:, hg:2 * hg, 9] = -np.inf
    if late:
        want[n - 1, :hg, 11] = np.inf
    fin = np.isfinite(want)
    np.testing.assert_array_equal(val[~fin], want[~fin])
    assert (np.abs(val - ref)[fin] <= (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 1e-4) * spread)[fin] + 1e-30).all()
