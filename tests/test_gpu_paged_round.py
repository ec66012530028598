"""The operators together, as a serving engine runs them around the draft step."""

import numpy as np
import pytest

from oracle import pe_oracle as O
from oracle import pe_paged as P
from parity import LOGIT_TOL, built, cuda_or_skip, host, setup
from speculative_drafting_gb300 import binding, runner, workloads as W

pytestmark = pytest.mark.gpu


def test_target_layer_verifies_drafts_and_feeds_the_next_step():
    """One target layer over a ragged batch of verify rows on paged contexts: append ->
    attend -> output and LM head -> verify_sampled, whose counts and tokens go into
    pe_prepare_inputs as they are.  Each call is checked in 64 bits on what it was given;
    the step's metadata, bit for bit."""
    torch = cuda_or_skip()
    built()
    torch.manual_seed(0)
    wl = W.get("small_prenorm")
    dm = wl.dims
    b = W.make_batch(wl)
    H, G, hd, bs, d, V = 8, 2, 64, dm.block_size, dm.d, dm.vocab
    B, T, nb = b["B"], b["T_in"], b["num_blocks"]
    dev = {k: runner.to_device(b[k], "f32") for k in ("qsl", "prev_tok", "prev_pos", "block_table")}
    bf = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    x, w_qkv, w_o, w_lm = bf(T, d), bf((H + 2 * G) * hd, d) * d ** -0.5, bf(d, H * hd) * 0.05, bf(V, d) * 0.1
    gq, gk = (1 + 0.1 * torch.randn(2, hd, device="cuda")).bfloat16()
    kc, vc = bf(nb, G, bs, hd), bf(nb, G, bs, hd)
    kc0, vc0 = (O.decode(host(t), "bf16") for t in (kc, vc))
    plan = binding.PagedAttention(H, G, hd, bs)
    wa, wt, wv = plan.append_workspace(), plan.workspace(B, T), binding.verify_sampled_workspace(B, T, V)
    # every verify row writes the slot of its position
    req = np.repeat(np.arange(B), np.diff(b["qsl"]))
    slot = np.array([O.slot_of(b["block_table"], r, int(p), bs) for r, p in zip(req, b["prev_pos"])])
    seq = torch.from_numpy((b["ctx"] + np.diff(b["qsl"])).astype(np.int32)).cuda()
    qkv = x @ w_qkv.T
    q, att = torch.empty(T, H, hd, device="cuda").bfloat16(), torch.empty(T, H * hd, device="cuda").bfloat16()
    plan.append(T, qkv, gq, gk, dev["prev_pos"], torch.from_numpy(slot).cuda(), nb, q, kc, vc, wa)
    plan.attend(B, T, dev["qsl"], seq, q, kc, vc, dev["block_table"], nb, att, wt)
    logits = ((x.float() + (att @ w_o.T).float()).bfloat16() @ w_lm.T).float()
    tok = dev["prev_tok"].clone()
    # half the drafts are the target's own pick, so some are accepted
    pick = logits.argmax(-1).int()
    half = torch.rand(T - 1, device="cuda") < 0.7
    tok[1:] = torch.where(half, pick[:-1], tok[1:])
    u, temp = torch.rand(T, device="cuda"), torch.tensor([0.3, 0.0, 0.5], device="cuda")
    gumbel = -torch.log(torch.empty(B, V, device="cuda").exponential_())
    acc, bon = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    p = torch.empty(T, device="cuda")
    binding.verify_sampled(B, T, dev["qsl"], tok, logits, V, binding.PE_DTYPE_F32, temp, u, gumbel, acc, bon, p, wv)
    # the next draft step takes the counts and tokens as they are
    batch = dict(b, prev_tok=host(tok))
    r = runner.StepRunner(wl, batch, W.make_weights(wl), *W.make_kv_cache(wl, nb))
    r.inp["accepted"], r.inp["bonus"] = acc, bon
    r.run()
    torch.cuda.synchronize()
    assert r.status()[0] == 0
    assert [binding.read_status_ws(w)[0] for w in (wa, wt, wv)] == [0, 0, 0]

    val = lambda t: O.decode(host(t), "bf16")  # noqa: E731
    rq, rk, rv = P.qkv_append(val(qkv), H, G, val(gq), val(gk), b["prev_pos"], slot, kc0, vc0)
    for got, want in ((q, rq), (kc, rk), (vc, rv)):
        a, c = np.split(np.abs(want), 2, -1)
        pair = np.hypot(a, c)
        assert (np.abs(val(got) - want) <= 2.0 ** -8 * np.abs(want) + 2e-6 * np.concatenate([pair, pair], -1)).all()
    ro, spread = P.chunk_attention(b["qsl"], host(seq), val(q), val(kc), val(vc), b["block_table"])
    assert (np.abs(val(att).reshape(ro.shape) - ro) <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 1e-4) * spread).all()
    ra, rb, rp, margin = P.verify_sampled(b["qsl"], host(tok), host(logits), host(temp), host(u), host(gumbel))
    clear = margin > 1e-4
    assert clear.sum() >= 2
    np.testing.assert_array_equal(host(acc)[clear], ra[clear])
    np.testing.assert_array_equal(host(bon)[clear], rb[clear])
    np.testing.assert_allclose(host(p), rp, rtol=1e-5, atol=1e-7)
    meta = O.prepare_metadata(b["qsl"], host(tok), b["prev_pos"], host(acc), host(bon), b["block_table"], dm.K,
                              dm.mask_id, bs)
    for k in ("tok", "pos", "slot", "seq_len"):
        np.testing.assert_array_equal(host(r.meta[k]), meta[k])


def test_a_prompt_appended_to_the_drafters_cache_serves_the_draft_step():
    """The drafter's context keys and values written by append (the prompt rows a draft
    step does not take), then a draft step over them: its logits match the oracle's on
    the cache that append left."""
    torch = cuda_or_skip()
    wl, b, w, kc, vc, r = setup("small_prenorm")
    dm, bs = wl.dims, wl.dims.block_size
    H, G, hd = dm.n_heads, dm.n_kv_heads, dm.head_dim
    plan = binding.PagedAttention(H, G, hd, bs)
    rows = [(q, t) for q in range(b["B"]) for t in range(int(b["ctx"][q]))]
    T = len(rows)
    slot = np.array([O.slot_of(b["block_table"], q, t, bs) for q, t in rows])
    pos = np.array([t for _, t in rows])
    u = torch.randn(T, dm.d, device="cuda").bfloat16()
    qkv = u @ r.w["w_qkv"].T
    r.k_cache.fill_(float("nan"))
    r.v_cache.fill_(float("nan"))
    ws = plan.append_workspace()
    plan.append(T, qkv, None, None, torch.from_numpy(pos).cuda(), torch.from_numpy(slot).cuda(), b["num_blocks"],
                None, r.k_cache, r.v_cache, ws)
    # what append did not write, the step may pad with: finite
    r.k_cache.nan_to_num_(0.0)
    r.v_cache.nan_to_num_(0.0)
    k0, v0 = host(r.k_cache).copy(), host(r.v_cache).copy()
    ref_k = P.qkv_append(O.decode(host(qkv), "bf16"), H, G, None, None, pos, slot, np.zeros(k0.shape),
                         np.zeros(k0.shape))[1]
    assert (np.abs(O.decode(k0, "bf16") - ref_k) <= 2.0 ** -8 * np.abs(ref_k) + 2e-6 * 8).all()
    r.run()
    torch.cuda.synchronize()
    assert r.status()[0] == 0 and binding.read_status_ws(ws)[0] == 0
    ref = O.draft_step(dm, w, b, k0, v0)
    logits = host(r.logits)
    for q, out in ref["req"].items():
        assert np.abs(logits[q * dm.K:(q + 1) * dm.K] - out["logits"]).max() <= LOGIT_TOL["bf16"]
