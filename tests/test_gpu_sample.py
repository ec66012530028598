"""pe_sample against the fp64 oracle on the same logits and noise.

Tokens have to be equal wherever the oracle's decision is clear: the winning score ahead by
1e-4 (scores of up to 40 are formed in fp32 with roundings of 4e-6), and no change if the
bounds of the weights (top_p, min_p) move by 2e-5 of their size (a weight is off by its
argument's roundings, 30 * 3 * 2^-24 = 5e-6 relative, plus the exponential's 2^-22; their sums by less).
"""

import numpy as np
import pytest

from oracle import pe_oracle as O
from oracle import pe_tree as X
from parity import built, cuda_or_skip, host
from speculative_drafting_gb300 import binding, runner, workloads as W

pytestmark = pytest.mark.gpu

SETTINGS = [(0.0, 0, 1.0, 0.0), (1.0, 0, 1.0, 0.0), (0.8, 50, 0.95, 0.0), (1.0, 0, 0.9, 0.0), (0.6, 20, 0.95, 0.0),
            (1.3, 0, 1.0, 0.1), (0.7, 64, 0.8, 0.02), (1.0, 200, 1.0, 0.0), (2.0, 5000, 1.0, 0.0), (1.0, 3000, 0.7, 0.0),
            (1.0, 0, 0.999, 0.0), (0.9, 1, 1.0, 0.0), (1.0, 0, 0.0, 0.0), (1.0, 0, 1.0, 1.0), (1.5, 0, 1.0, 1e-6)]


def logits(rng, T, V, kind):
    if kind == "flat":
        x = rng.standard_normal((T, V)) * 0.5
    elif kind == "ties":
        x = rng.integers(-3, 4, (T, V)).astype(float)
    elif kind == "equal":
        x = np.full((T, V), 1.25)
    else:  # some likely tokens over a floor
        x = rng.standard_normal((T, V)) * 1.5
        m = min(V, 200)
        for row in x:
            row[rng.choice(V, m, replace=False)] = 12.0 - 1.5 * np.log(np.arange(1, m + 1))
        x[rng.random(x.shape) < 0.02] = -np.inf
        x[:, 0] = 0.0
    return x


def case(ns, V, dtype, kind="peaked", seed=0, settings=None, extra=0):
    rng = np.random.default_rng(seed)
    B, T = len(ns), sum(ns) + extra
    st = [settings or SETTINGS[(seed + i) % len(SETTINGS)] for i in range(B)] if not isinstance(settings, list) else settings
    x = logits(rng, T, V, kind).astype(np.float32)
    f = lambda i, ty: np.array([s[i] for s in st], ty)  # noqa: E731
    return dict(qsl=np.concatenate([[0], np.cumsum(ns)]).astype(np.int32), dtype=dtype, V=V,
                logits=W.f32_to_bf16_bits(x) if dtype == "bf16" else x, temp=f(0, np.float32), k=f(1, np.int32),
                p=f(2, np.float32), m=f(3, np.float32), g=-np.log(rng.exponential(size=(T, V))).astype(np.float32))


def run(c, pad=(0, 0), stream=None, out=None):
    torch = cuda_or_skip()
    built()
    B, (T, V) = len(c["qsl"]) - 1, c["g"].shape

    def strided(x, dtype, by):
        buf = np.zeros((T, V + by), x.dtype)
        buf[:, :V] = x
        return runner.to_device(buf, dtype)[:, :V]

    o = lambda k: None if c[k] is None else runner.to_device(c[k], "f32")  # noqa: E731
    tok = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    ws = binding.sample_workspace(B, T, V)
    args = (B, T, o("qsl"), strided(c["logits"], c["dtype"], pad[0]), V, o("temp"), o("k"), o("p"), o("m"),
            strided(c["g"], "f32", pad[1]), tok, ws)
    torch.cuda.synchronize()
    binding.sample(*args, stream=stream)
    torch.cuda.synchronize()
    return host(tok), binding.read_status_ws(ws)[0]


def check(c, status=0, least_clear=0.9, **kw):
    got, st = run(c, **kw)
    want, clear = X.sample(c["qsl"], O.decode(c["logits"], c["dtype"]), c["temp"], c["k"], c["p"], c["m"], c["g"])
    assert st == status
    assert clear.mean() >= least_clear
    np.testing.assert_array_equal(got[clear], want[clear])
    return got, want


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 64, 1000, 4099])
def test_every_setting(dtype, V):
    """Each setting on rows of each kind, ragged requests, rows off the 16-byte grid."""
    for kind in ("peaked", "flat", "ties", "equal"):
        # (few tokens weigh a bound's share of the whole each, and equal ones meet it exactly)
        c = case((2, 0, 1, 3, 1, 1, 2, 1, 1, 1, 1, 1, 1, 1, 1, 1), V, dtype, kind, seed=V, extra=2)
        check(c, least_clear=0.6, pad=(V % 5, V % 3))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["peaked", "flat", "equal"])
def test_full_vocabulary(dtype, kind):
    check(case((1,) * len(SETTINGS), 201088, dtype, kind, seed=1), least_clear=0.8)


def test_odd_vocabulary_and_many_rows():
    check(case((9, 1, 8, 4, 3) * 5, 32003, "bf16", seed=2), least_clear=0.9)
    check(case((9, 1, 4) * 3, 50257, "f32", seed=3, extra=1), least_clear=0.9)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["peaked", "flat", "ties"])
def test_more_rows_than_fit_at_once(dtype, kind):
    """640 rows: every setting in a batch of that size, candidates up to the most that are put in order."""
    check(case((9, 1, 8, 0, 14) * 20, 3001, dtype, kind, seed=12, extra=1), least_clear=0.8, pad=(3, 2))
    ks = [(1.0, k, p, 0.0) for k, p in ((500, 1.0), (512, 0.99), (513, 1.0), (300, 0.9), (0, 0.97))]
    check(case((64,) * 5, 1500, dtype, kind, seed=13, settings=ks), least_clear=0.5)


def test_large_vocabulary():
    """Slices that no shared memory holds: the rows are read again where they lie."""
    check(case((1,) * 3, 1_000_003, "f32", settings=[SETTINGS[i] for i in (2, 3, 9)], seed=4), least_clear=0.6)
    check(case((1,) * 2, 1_000_003, "bf16", "flat", settings=[SETTINGS[i] for i in (1, 9)], seed=5), least_clear=0.5)


@pytest.mark.parametrize("dtype,V", [("f32", 209001), ("f32", 300001), ("bf16", 278001), ("bf16", 600001)])
def test_slices_with_and_without_their_noise(dtype, V):
    """Vocabularies around the sizes up to which a slice and its noise, or the slice alone, fit in shared memory."""
    ks = [(1.0, 0, 0.9, 0.0), (1.0, 0, 0.5, 0.02), (1.0, 5000, 0.9, 0.0), (1.0, 0, 0.01, 0.0)]
    for kind in ("flat", "ties"):
        check(case((1,) * 4, V, dtype, kind, settings=ks, seed=14), least_clear=0.5, pad=(1, 3))


def test_ties_at_the_cut_go_to_the_lowest_index():
    """Many equal logits, noise that makes the last kept one win: the token shows the cut."""
    for V, k in ((1000, 700), (1000, 10), (60000, 30000), (201088, 7), (201088, 100003), (300, 299)):
        for dtype in ("f32", "bf16"):
            c = case((1, 1), V, dtype, "equal", settings=[(1.0, k, 1.0, 0.0), (1.0, 0, k / V, 0.0)])
            c["g"][:] = np.arange(V, dtype=np.float32)
            c["p"][1] = np.float32(np.ceil(k - 0.5) / V - 0.4 / V)  # k - 1 < p V < k: the first k
            got, st = run(c)
            assert st == 0 and got.tolist() == [k - 1, k - 1], (V, k, dtype)
    # a few above the equal ones
    c = case((1,), 5000, "f32", "equal", settings=(1.0, 2000, 1.0, 0.0))
    c["logits"][0, 4000:4005] = 3.0
    c["g"][:] = np.arange(5000)
    c["g"][0, 4000:4005] = -50
    assert run(c)[0].tolist() == [1994]


def test_the_largest_vocabulary_of_equal_logits():
    """2^20 of them: every slice's sum of weights is 2^17 times the largest one's."""
    V, k = 1 << 20, 5000
    for dtype in ("f32", "bf16"):
        c = case((1, 1), V, dtype, "equal", settings=[(1.0, k, 1.0, 0.0), (1.0, 0, (k - 0.5) / V, 0.0)])
        c["g"][:] = np.arange(V, dtype=np.float32)
        got, st = run(c)
        assert st == 0 and got.tolist() == [k - 1, k - 1]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_tokens_of_little_weight(dtype):
    """One token and 201,087 of 7.6e-10 of its weight: 1.5e-4 together.  0.9999 of all are the first and 69,240 of
    those."""
    V = 201088
    c = case((1, 1, 1), V, dtype, settings=[(1.0, 0, 0.9999, 0.0)] * 3)
    x = np.full((3, V), -21.0)
    x[:, 0] = 0.0
    c["logits"] = _bits(x, dtype)
    c["g"][:] = 0.0
    for row, t in enumerate((30000, 120000, V - 1)):
        c["g"][row, t] = 60.0
    got, _ = check(c, least_clear=1.0)
    assert got.tolist() == [30000, 0, 0]


def test_no_settings_is_a_draw_from_the_softmax():
    c = dict(case((3, 4), 700, "f32", seed=6), temp=None, k=None, p=None, m=None)
    check(c)


def test_temperature_zero_is_the_greedy_token():
    rng = np.random.default_rng(7)
    for dtype in ("f32", "bf16"):
        c = case((5, 3), 3001, dtype, "ties", settings=(0.0, 5, 0.5, 0.1))
        x = O.decode(c["logits"], dtype).copy()
        x[1, [7, 2000]] = np.nan
        x[2] = -np.inf
        x[3, [9, 8]] = np.inf
        x[4] = 0.0
        x[4, ::2] = -0.0
        x[5] = -np.abs(x[5]) - 1
        c["logits"] = W.f32_to_bf16_bits(x.astype(np.float32)) if dtype == "bf16" else x.astype(np.float32)
        got, st = run(c)
        np.testing.assert_array_equal(got, O.target_argmax(x))
        assert st == 0


def test_rows_without_a_distribution():
    V, inf = 900, np.inf
    for s in ((1.0, 0, 1.0, 0.0), (1.0, 20, 0.9, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.1)):
        c = case((6,), V, "f32", settings=s)
        c["logits"][0, 5] = np.nan
        c["logits"][1] = -inf
        c["logits"][2, 7] = inf
        c["g"][3] = -inf                      # nothing can win
        c["logits"][4] = -inf
        c["logits"][4, 33] = -700.0           # one token
        got, st = run(c)
        assert got[:5].tolist() == [-1, -1, -1, -1, 33] and st == binding.PE_ST_SAMPLING
        assert got[5] == check(dict(c, logits=c["logits"][5:], g=c["g"][5:], qsl=np.array([0, 1], np.int32)))[0][0]
    # infinite noise wins where the token is kept, at the lowest index; NaN never does
    c = case((3,), V, "f32", settings=(1.0, 3, 1.0, 0.0))
    order = np.argsort(-c["logits"], axis=1, kind="stable")
    c["g"][0, order[0, [5, 2, 1]]] = inf
    c["g"][1, order[1, 0]] = np.nan
    c["g"][2, order[2, 3:]] = np.nan
    got, st = run(c)
    want = X.sample(c["qsl"], c["logits"], c["temp"], c["k"], c["p"], c["m"], c["g"])[0]
    assert st == 0 and got[0] == min(order[0, [1, 2]]) and got.tolist() == want.tolist()


def test_odd_settings():
    c = case((1,) * 8, 1200, "f32", settings=[(-1.0, 0, 1.0, 0.0), (float("nan"), 0, 1.0, 0.0), (1.0, -5, 2.0, -3.0),
                                             (1.0, 1200, 1.0, 0.0), (1.0, 0, float("nan"), 0.0), (1.0, 0, 1.0, float("nan")),
                                             (1e-38, 0, 0.9, 0.0), (1e38, 4, 1.0, 0.0)], seed=9)
    got, _ = check(c, status=binding.PE_ST_SAMPLING, least_clear=0.7)
    big = O.target_argmax(c["logits"])
    assert got[0] == big[0] and got[1] == big[1] and got[6] == big[6]
    c = case((4,), 5000, "f32", settings=(1.0, 30, 0.9, 0.0))
    c["logits"][0, 77] = 3e38   # a span that overflows, and one that is nothing
    c["logits"][1] = 1e-42 * np.arange(5000)
    c["logits"][2, 99] = 1e6
    check(c, least_clear=0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_cuts_behind_many_tokens(dtype):
    """Cuts that thousands come before: in ranges that bins split badly (one far logit, a span that overflows, all
    tokens within a few roundings), with ties around them, with both settings."""
    V = 9001
    ks = [(1.0, 3000, 1.0, 0.0), (1.0, 2500, 0.7, 0.0), (1.0, 0, 0.8, 0.0), (5.0, 8999, 0.999, 1e-9), (0.01, 4000, 1.0, 0.0)]
    for i, kind in enumerate(("flat", "ties", "peaked", "flat", "equal")):
        c = case((1,) * 5, V, dtype, kind, settings=ks, seed=i)
        x = O.decode(c["logits"], dtype).copy()
        if i == 1:
            x[:, 100] = 3e38
            x[:, 200] = -3e38
        if i == 3:
            x = 1.0 + x * 1e-6
            x[:, 50] = 2e4
        c["logits"] = _bits(x, dtype)
        check(c, least_clear=0.5)


def _bits(x, dtype):
    return W.f32_to_bf16_bits(x.astype(np.float32)) if dtype == "bf16" else x.astype(np.float32)


@pytest.mark.parametrize("qsl", [(0, 5, 3), (0, -2, 4), (1, 2, 3), (0, 3, 60)])
def test_bad_offsets_are_reported(qsl):
    c = dict(case((2, 2), 300, "f32"), qsl=np.array(qsl, np.int32))
    _, st = run(c)
    assert st & binding.PE_ST_ROWS_RANGE


def test_repeats_in_graphs_and_on_streams():
    torch = cuda_or_skip()
    c = case((8, 1, 3) * 5, 20011, "bf16", seed=10)
    want, _ = check(c)
    s = torch.cuda.Stream()
    for _ in range(5):
        assert (run(c, stream=s)[0] == want).all()
    T, V = c["g"].shape
    B = len(c["qsl"]) - 1
    d = [runner.to_device(c[k], "f32") for k in ("qsl", "temp", "k", "p", "m", "g")]
    lg = runner.to_device(c["logits"], "bf16")
    toks = [torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(2)]
    ws = binding.sample_workspace(B, T, V)
    torch.cuda.synchronize()
    graphs = []
    for t in toks:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            binding.sample(B, T, d[0], lg, V, *d[1:5], d[5], t, ws, stream=s)
        graphs.append(g)
    # new inputs in the same place, both graphs in turn
    c2 = case((8, 1, 3) * 5, 20011, "bf16", seed=11)
    lg.copy_(runner.to_device(c2["logits"], "bf16"))
    d[5].copy_(runner.to_device(c2["g"], "f32"))
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    now = run(dict(c, logits=c2["logits"], g=c2["g"]))[0]
    assert all((host(t) == now).all() for t in toks) and (now != want).any()
