"""Host-side checks of the paged attention calls and of pe_verify_sampled: every
refusal is answered before a device call (no GPU needed; the addresses are fake
and never dereferenced)."""

import ctypes
import os
import shutil
import subprocess

import pytest

from speculative_drafting_gb300 import binding, build

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists(
    "/usr/local/cuda/bin/nvcc"), reason="needs nvcc to build libpe.so")

F32, BF16 = binding.PE_DTYPE_F32, binding.PE_DTYPE_BF16
ARG, UNSUP, OK = binding.PE_ERR_ARG, binding.PE_ERR_UNSUPPORTED, binding.PE_OK
P = 1 << 21          # an aligned address
WS = 1 << 22
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _plan(lib, H=64, G=8, hd=64, bs=16, dtype=BF16, eps=1e-6, theta=1e4):
    p = binding.PeAttnPlan()
    return lib.pe_attn_plan_init(ctypes.addressof(p), H, G, hd, bs, dtype, eps, theta), p


def test_plan_refusals(lib):
    assert _plan(lib)[0] == OK and _plan(lib, H=4, G=2, hd=40, dtype=F32)[0] == OK
    assert lib.pe_attn_plan_init(None, 4, 2, 64, 16, BF16, 1e-6, 1e4) == ARG
    for bad in (dict(H=0), dict(G=0), dict(H=6, G=4), dict(H=258, G=2), dict(hd=0), dict(hd=12), dict(hd=136),
                dict(hd=96), dict(bs=0), dict(dtype=7), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(theta=0.0), dict(theta=float("nan")),
                dict(theta=float("inf")), dict(H=-8, G=-1)):
        rc, p = _plan(lib, **bad)
        assert rc == UNSUP, bad
        assert bytes(p) == bytes(ctypes.sizeof(p)), bad
        assert lib.pe_chunk_attention_workspace_bytes(ctypes.addressof(p), 1, 1) == 0


def test_plan_layout_matches_the_header(lib, tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs a host C++ compiler")
    src = tmp_path / "size.cc"
    src.write_text('#include <cstdio>\n#include <cstddef>\n#include "pe.h"\nint main(){std::printf("%zu %zu",'
                   ' sizeof(pe_attn_plan), offsetof(pe_attn_plan, rope_turn));}\n')
    subprocess.run([gxx, "-I", build.INCLUDE, str(src), "-o", str(tmp_path / "size")], check=True)
    got = subprocess.run([str(tmp_path / "size")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in got] == [ctypes.sizeof(binding.PeAttnPlan), binding.PeAttnPlan.rope_turn.offset]


APPEND = dict(plan=None, T=4, qkv=P, ld=80 * 64, gq=P, gk=P, pos=P, slot=P, nb=8, q=P, k=P, v=P, ws=WS, wsb=256,
              stream=None)


def test_append_refusals(lib):
    _, plan = _plan(lib)

    def call(**kw):
        a = dict(APPEND, plan=ctypes.addressof(plan), **kw)
        return lib.pe_qkv_append(*a.values())

    assert call(T=0, qkv=None, pos=None) == OK
    for kw in (dict(plan=None), dict(T=-1), dict(nb=-1), dict(ld=80 * 64 - 8), dict(ld=80 * 64 + 4), dict(qkv=None),
               dict(pos=None), dict(slot=None), dict(k=None), dict(v=None), dict(ws=None), dict(qkv=P + 2),
               dict(gq=P + 8), dict(q=P + 4), dict(k=P + 8), dict(pos=P + 4), dict(slot=P + 4),
               dict(ws=WS + 128), dict(wsb=255)):
        args = dict(APPEND, plan=ctypes.addressof(plan))
        args.update(kw)
        assert lib.pe_qkv_append(*args.values()) == ARG, kw
    empty = binding.PeAttnPlan()
    assert lib.pe_qkv_append(*dict(APPEND, plan=ctypes.addressof(empty)).values()) == ARG


ATTEND = dict(plan=None, B=2, T=4, qsl=P, seq=P, q=P, ldq=64 * 64, k=P, v=P, table=P, mb=4, nb=8, sink=None, out=P,
              ldo=64 * 64, ws=WS, wsb=BIG, stream=None)


def test_attention_refusals(lib):
    _, plan = _plan(lib)

    def call(**kw):
        a = dict(ATTEND, plan=ctypes.addressof(plan))
        a.update(kw)
        return lib.pe_chunk_attention(*a.values())

    for kw in (dict(plan=None), dict(B=-1), dict(T=-1), dict(mb=0), dict(nb=-1), dict(ldq=64 * 64 - 8),
               dict(ldq=64 * 64 + 2), dict(ldo=64), dict(ldo=64 * 64 + 4), dict(qsl=None), dict(seq=None),
               dict(q=None), dict(k=None), dict(v=None), dict(table=None), dict(out=None), dict(q=P + 2),
               dict(k=P + 8), dict(v=P + 8), dict(out=P + 8), dict(qsl=P + 2), dict(seq=P + 1), dict(table=P + 2),
               dict(sink=P + 2), dict(ws=None), dict(ws=WS + 64), dict(wsb=64)):
        assert call(**kw) == ARG, kw
    assert call(B=65536) == UNSUP
    assert call(nb=1 << 24) == UNSUP  # 2^31 cache rows
    ws = lib.pe_chunk_attention_workspace_bytes
    assert ws(ctypes.addressof(plan), -1, 1) == 0 and ws(ctypes.addressof(plan), 1, -1) == 0
    assert ws(None, 1, 1) == 0 and ws(ctypes.addressof(plan), 0, 0) >= 256
    # larger batches and row counts never need less
    sizes = [ws(ctypes.addressof(plan), b, t) for b, t in ((1, 1), (1, 8192), (64, 8192), (64, 65536))]
    assert sizes == sorted(sizes)


VERIFY = dict(B=2, T=4, qsl=P, tok=P, logits=P, V=100, dtype=F32, temp=None, u=P, gumbel=P, acc=P, bonus=P, p=None,
              ws=WS, wsb=BIG, stream=None)


def test_verify_sampled_refusals(lib):
    def call(**kw):
        return lib.pe_verify_sampled(*dict(VERIFY, **kw).values())

    assert call(B=0, T=0, qsl=None) == OK
    for kw in (dict(B=-1), dict(T=-1), dict(V=0), dict(B=0), dict(qsl=None), dict(tok=None), dict(logits=None),
               dict(u=None), dict(gumbel=None), dict(acc=None), dict(bonus=None), dict(ws=None), dict(ws=WS + 8),
               dict(wsb=100), dict(logits=P + 2), dict(logits=P + 1, dtype=BF16), dict(u=P + 2), dict(gumbel=P + 1),
               dict(temp=P + 2), dict(qsl=P + 2), dict(tok=P + 1), dict(p=P + 2)):
        assert call(**kw) == ARG, kw
    assert call(dtype=5) == UNSUP and call(B=65536) == UNSUP
    ws = lib.pe_verify_sampled_workspace_bytes
    assert ws(1, 8, 0) == 0 and ws(-1, 8, 10) == 0 and ws(1, -8, 10) == 0 and ws(0, 0, 1) >= 256
    sizes = [ws(b, t, v) for b, t, v in ((1, 8, 1000), (1, 64, 1000), (64, 64, 1000), (64, 64, 200000))]
    assert sizes == sorted(sizes)


def test_sizes_past_the_indexes_are_refused(lib):
    assert lib.pe_verify_sampled(*dict(VERIFY, V=(1 << 30) + 1).values()) == UNSUP
    rc, plan = _plan(lib, H=64, G=8)
    at = dict(ATTEND, plan=ctypes.addressof(plan))
    assert lib.pe_chunk_attention(*dict(at, T=(1 << 25) - 2).values()) == UNSUP  # T * H past 2^31 - 256
    assert lib.pe_chunk_attention(*dict(at, mb=1 << 27).values()) == UNSUP
    assert _plan(lib, H=65536, G=1024)[0] == UNSUP and _plan(lib, H=65535, G=65535)[0] == OK


def test_unknown_dtypes_are_refused(lib):
    for name in ("fp16", "BF16", None, "bfloat16"):
        with pytest.raises(binding.PeError):
            binding.PagedAttention(8, 2, 64, 16, dtype=name)


def test_workspaces_of_another_device_are_refused(lib, monkeypatch):
    """The launch goes to the current device: tensors of another one are not for it."""
    import torch

    class Other:
        def get_device(self):
            return 1

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 64 + d, raising=False)
    monkeypatch.setattr(binding, "_raw_stream", None)
    monkeypatch.setattr(binding, "_current_device", None)
    with pytest.raises(ValueError, match="device"):
        binding._stream_handle(None, Other())
    monkeypatch.setattr(Other, "get_device", lambda self: 0)
    assert binding._stream_handle(None, Other()) == 64
    # what the test's stand-ins left is not kept
    binding._raw_stream = binding._current_device = None


def test_views_that_are_not_dense_are_refused(lib):
    """Only rows may be strided: other views would be read as if they were dense."""
    import torch

    plan = binding.PagedAttention(4, 2, 64, 16)
    bf = dict(dtype=torch.bfloat16)
    pair = torch.zeros(3, 2, 2, 16, 64, **bf)  # keys and values of a block side by side
    k, v = torch.zeros(2, 3, 2, 16, 64, **bf)
    q, out = torch.zeros(2, 5, 4, 64, **bf)
    table, ints, ws = torch.zeros(1, 8, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), torch.zeros(256)

    def attend(q=q, k=k, v=v, table=table, out=out):
        plan.attend(1, 5, ints, ints, q, k, v, table, 3, out, ws)

    def append(qkv, k=k, v=v, q_out=q):
        plan.append(5, qkv, None, None, ints, ints, 3, q_out, k, v, ws)

    qkv = torch.zeros(5, 8 * 64, **bf)
    wide = torch.zeros(2, 16, dtype=torch.int32)
    for call in (lambda: attend(k=pair[:, 0]), lambda: attend(v=pair[:, 1]), lambda: attend(table=wide[:, :8]),
                 lambda: attend(q=q.transpose(1, 2).contiguous().transpose(1, 2)),
                 lambda: attend(out=torch.zeros(5, 4, 128, **bf)[:, :, ::2]),
                 lambda: attend(out=torch.zeros(5, 4, 128, **bf)[:, :, :64]),
                 lambda: attend(q=q.float()), lambda: attend(out=out.half()), lambda: attend(k=k.float()),
                 lambda: append(qkv, k=pair[:, 0]), lambda: append(qkv, v=pair[:, 0]),
                 lambda: append(qkv, q_out=torch.zeros(5, 8, 64, **bf)[:, :4]), lambda: append(qkv[:, ::2]),
                 lambda: append(qkv.float()), lambda: append(qkv, q_out=q.float()),
                 lambda: binding.verify_sampled(1, 4, ints, ints, torch.zeros(4, 32)[:, :16], 16, F32, None, ints,
                                                torch.zeros(1, 16), ints, ints, None, ws)):
        with pytest.raises(ValueError, match="dense|type"):
            call()
