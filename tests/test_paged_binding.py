"""What the binding of the paged calls and of sampled verification hands to the library:
tensors of another type, size or device than the call reads are refused before it (no GPU
needed: the library's calls are stand-ins that note their arguments)."""

import os
import shutil

import pytest

from speculative_drafting_gb300 import binding, build

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists(
    "/usr/local/cuda/bin/nvcc"), reason="needs nvcc to build libpe.so")

H, G, HD, BS, T, NB = 4, 2, 64, 16, 5, 3
BF = torch.bfloat16


class Calls:
    """The library's compute calls, noted instead of made; host-only calls go through."""

    def __init__(self, lib):
        self.lib, self.made = lib, []

    def __getattr__(self, name):
        if name in ("pe_qkv_append", "pe_chunk_attention", "pe_verify_sampled"):
            return lambda *a: self.made.append((name, a)) or binding.PE_OK
        return getattr(self.lib, name)


@pytest.fixture
def calls(monkeypatch):
    build.build()
    c = Calls(binding.load())
    monkeypatch.setattr(binding, "_lib", c)
    # CPU tensors are on device -1
    monkeypatch.setattr(binding, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(binding, "_current_device", lambda: -1)
    return c


def plan():
    return binding.PagedAttention(H, G, HD, BS)


def append(**kw):
    a = dict(T=T, qkv=torch.zeros(T, (H + 2 * G) * HD, dtype=BF), gamma_q=torch.ones(HD, dtype=BF),
             gamma_k=torch.ones(HD, dtype=BF), pos=torch.arange(T), slot=torch.arange(T), num_blocks=NB,
             q_out=torch.zeros(T, H, HD, dtype=BF), k_cache=torch.zeros(NB, G, BS, HD, dtype=BF),
             v_cache=torch.zeros(NB, G, BS, HD, dtype=BF), ws=torch.zeros(256, dtype=torch.uint8))
    a.update(kw)
    plan().append(**a)


def attend(**kw):
    i32 = dict(dtype=torch.int32)
    a = dict(B=1, T=T, qsl=torch.tensor([0, T], **i32), seq_len=torch.tensor([T], **i32),
             q=torch.zeros(T, H, HD, dtype=BF), k_cache=torch.zeros(NB, G, BS, HD, dtype=BF),
             v_cache=torch.zeros(NB, G, BS, HD, dtype=BF), block_table=torch.zeros(1, 2, **i32), num_blocks=NB,
             out=torch.zeros(T, H * HD, dtype=BF), ws=None, sink=torch.zeros(H))
    a.update(kw)
    p = plan()
    a["ws"] = p.workspace(1, T, device="cpu") if a["ws"] is None else a["ws"]
    p.attend(**a)


V = 40


def verify(**kw):
    i32 = dict(dtype=torch.int32)
    a = dict(B=2, T_in=T, qsl=torch.tensor([0, 3, T], **i32), tok=torch.zeros(T, **i32), logits=torch.zeros(T, V),
             vocab=V, dtype=binding.PE_DTYPE_F32, temperature=torch.ones(2), u=torch.zeros(T),
             gumbel=torch.zeros(2, V), accepted=torch.zeros(2, **i32), bonus=torch.zeros(2, **i32),
             p_draft=torch.zeros(T), ws=binding.verify_sampled_workspace(2, T, V, device="cpu"))
    a.update(kw)
    binding.verify_sampled(**a)


def refused(calls, make, *cases):
    """The call as it should be goes through, once; each of the others is refused."""
    make()
    assert len(calls.made) == 1
    for kw in cases:
        with pytest.raises(ValueError):
            make(**kw)
        assert len(calls.made) == 1, {k: getattr(v, "dtype", v) for k, v in kw.items()}


def test_gains_of_another_type_or_size_are_refused(calls):
    append(gamma_q=None, gamma_k=None)
    calls.made.clear()
    refused(calls, append, dict(gamma_q=torch.ones(HD)), dict(gamma_k=torch.ones(HD)),
            dict(gamma_k=torch.ones(HD, dtype=torch.half)), dict(gamma_q=torch.ones(HD // 2, dtype=BF)),
            dict(gamma_q=torch.ones(H, HD, dtype=BF)), dict(gamma_k=torch.ones(2 * HD, dtype=BF)[::2]))


def test_append_indexes_of_another_type_are_refused(calls):
    i = torch.arange(T)
    refused(calls, append, dict(pos=i.int()), dict(slot=i.int()), dict(pos=i.double()),
            dict(slot=torch.arange(2 * T)[::2]), dict(pos=torch.arange(2 * T)[::2]))


def test_attend_indexes_and_sinks_of_another_type_are_refused(calls):
    attend(sink=None)
    calls.made.clear()
    refused(calls, attend, dict(qsl=torch.tensor([0, T])), dict(seq_len=torch.tensor([T])),
            dict(block_table=torch.zeros(1, 2, dtype=torch.int64)), dict(sink=torch.zeros(H, dtype=BF)),
            dict(sink=torch.zeros(H, dtype=torch.float64)), dict(sink=torch.zeros(2 * H)[::2]),
            dict(qsl=torch.tensor([0, 9, T, 9], dtype=torch.int32)[::2]))


def test_verify_sampled_tensors_of_another_type_are_refused(calls):
    verify(temperature=None, p_draft=None)
    verify(logits=torch.zeros(T, V, dtype=BF), dtype=binding.PE_DTYPE_BF16)
    calls.made.clear()
    every = [torch.zeros(2 * T)[::2], torch.zeros(T, dtype=torch.float64), torch.zeros(T, dtype=BF)]
    refused(calls, verify, dict(logits=torch.zeros(T, V, dtype=BF)), dict(dtype=binding.PE_DTYPE_BF16),
            dict(logits=torch.zeros(T, V, dtype=torch.half)), dict(logits=torch.zeros(T, 2 * V)[:, :V]),
            dict(tok=torch.zeros(T, dtype=torch.int64)), dict(tok=torch.zeros(2 * T, dtype=torch.int32)[::2]),
            dict(qsl=torch.tensor([0, 3, T])), dict(accepted=torch.zeros(2, dtype=torch.int64)),
            dict(bonus=torch.zeros(2, dtype=torch.int64)), dict(gumbel=torch.zeros(2, V, dtype=torch.float64)),
            dict(gumbel=torch.zeros(2, 2 * V)[:, :V]),
            *(dict([(k, t)]) for k in ("temperature", "u", "p_draft") for t in every))


def test_append_tensors_too_small_for_the_call_are_refused(calls):
    bf = dict(dtype=BF)
    append(qkv=torch.zeros(T, H + 2 * G, HD, **bf))
    append(qkv=torch.zeros(T + 2, (H + 2 * G) * HD + 64, **bf), pos=torch.arange(9), slot=torch.arange(9), q_out=None)
    append(T=0, qkv=torch.zeros(0, (H + 2 * G) * HD, **bf))
    append(qkv=torch.zeros(T, 1, (H + 2 * G) * HD, **bf))
    calls.made.clear()
    refused(calls, append, dict(T=T + 1), dict(pos=torch.arange(T - 1)), dict(slot=torch.arange(T - 1)),
            dict(qkv=torch.zeros(T - 1, (H + 2 * G) * HD, **bf)), dict(qkv=torch.zeros(T, (H + 2 * G) * HD - 8, **bf)),
            dict(qkv=torch.zeros(T, H + G, HD, **bf)), dict(qkv=torch.zeros((H + 2 * G) * HD, **bf)),
            dict(q_out=torch.zeros(T - 1, H, HD, **bf)), dict(q_out=torch.zeros(T, H - 1, HD, **bf)),
            dict(num_blocks=NB + 1), dict(k_cache=torch.zeros(NB, G, BS - 1, HD, **bf)),
            dict(v_cache=torch.zeros(NB - 1, G, BS, HD, **bf)))


def test_attend_tensors_too_small_for_the_call_are_refused(calls):
    bf, i32 = dict(dtype=BF), dict(dtype=torch.int32)
    attend(q=torch.zeros(T + 1, H * HD + 64, **bf), out=torch.zeros(T, H, HD, **bf))
    none, two = torch.zeros(0, H * HD, **bf), torch.zeros(2, 1, **i32)
    attend(B=2, T=0, q=none, out=none, qsl=two, seq_len=two, block_table=two)  # nothing to do: nothing is read
    calls.made.clear()
    refused(calls, attend, dict(T=T + 1), dict(B=2), dict(qsl=torch.zeros(1, **i32)), dict(seq_len=torch.zeros(0, **i32)),
            dict(block_table=torch.zeros(0, 2, **i32)), dict(sink=torch.zeros(H - 1)),
            dict(q=torch.zeros(T - 1, H, HD, **bf)), dict(q=torch.zeros(T, H * HD - 8, **bf)),
            dict(out=torch.zeros(T - 1, H * HD, **bf)), dict(out=torch.zeros(T, H - 1, HD, **bf)),
            dict(out=torch.zeros(H * HD, **bf)), dict(num_blocks=NB + 1),
            dict(k_cache=torch.zeros(NB, G, BS - 1, HD, **bf)), dict(v_cache=torch.zeros(NB - 1, G, BS, HD, **bf)))


def test_verify_sampled_tensors_too_small_for_the_call_are_refused(calls):
    i32 = dict(dtype=torch.int32)
    verify(logits=torch.zeros(T * V + 7), p_draft=torch.zeros(T + 1), temperature=torch.ones(5))
    verify(T_in=0, logits=torch.zeros(0, V), tok=torch.zeros(0, **i32), u=torch.zeros(0))
    verify(T_in=0, logits=None, tok=None, u=None, gumbel=None, p_draft=None)
    verify(B=0, T_in=0, qsl=None, logits=None, tok=None, u=None, gumbel=None, accepted=None, bonus=None, p_draft=None)
    calls.made.clear()
    refused(calls, verify, dict(B=3), dict(T_in=T + 1), dict(vocab=V + 1), dict(qsl=torch.zeros(2, **i32)),
            dict(tok=torch.zeros(T - 1, **i32)), dict(u=torch.zeros(T - 1)), dict(logits=torch.zeros(T - 1, V)),
            dict(gumbel=torch.zeros(1, V)), dict(gumbel=torch.zeros(2, V - 1)), dict(temperature=torch.ones(1)),
            dict(accepted=torch.zeros(1, **i32)), dict(bonus=torch.zeros(1, **i32)), dict(p_draft=torch.zeros(T - 1)))


class Elsewhere(torch.Tensor):
    def get_device(self):
        return 1


@pytest.mark.parametrize("make", [append, attend, verify])
def test_tensors_of_another_device_than_the_workspace_are_refused(calls, monkeypatch, make):
    """Each tensor in turn: the launch goes to the current device, where its address is
    another's or nobody's."""
    sent = {}
    name = {append: "append", attend: "attend"}.get(make, "verify_sampled")
    owner = binding if make is verify else binding.PagedAttention
    real = getattr(owner, name)
    monkeypatch.setattr(owner, name, lambda *a, **kw: (sent.update(kw), real(*a, **kw))[1])
    make()
    given = dict(sent)
    tensors = [k for k, t in given.items() if isinstance(t, torch.Tensor)]
    assert len(tensors) >= 9
    refused(calls, lambda **kw: make(**{**given, **kw}) if kw else None,
            *(dict([(k, given[k].as_subclass(Elsewhere))]) for k in tensors))


def test_rows_of_more_dimensions_are_taken_where_they_are_dense(calls):
    """Heads by KV head, as a model may hold them: [T][G][H/G][hd]."""
    bf = dict(dtype=BF)
    attend(q=torch.zeros(T, G, H // G, HD, **bf), out=torch.zeros(T + 1, G, H // G, HD, **bf)[:T])
    append(qkv=torch.zeros(T, (H + 2 * G) // 2, 2, HD, **bf), q_out=torch.zeros(T, G, H // G, HD, **bf))
    assert [a[1][6] for a in calls.made[:1]] == [H * HD] and calls.made[1][1][3] == (H + 2 * G) * HD
    calls.made.clear()
    wide = torch.zeros(T, G, H // G, 2 * HD, **bf)
    refused(calls, attend, dict(q=wide[..., :HD]), dict(q=wide[..., ::2]), dict(out=wide[..., :HD]),
            dict(q=torch.zeros(T, H // G, G, HD, **bf).transpose(1, 2)), dict(q=torch.zeros(T, 1, G, HD, **bf)),
            dict(q=torch.zeros(T - 1, G, H // G, HD, **bf)))
