"""Host-side checks of the tree, sampling and page calls: every refusal is answered before a
device call (no GPU needed; the addresses are fake and never dereferenced)."""

import ctypes
import os
import shutil

import pytest

from speculative_drafting_gb300 import binding, build

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists(
    "/usr/local/cuda/bin/nvcc"), reason="needs nvcc to build libpe.so")

F32, BF16 = binding.PE_DTYPE_F32, binding.PE_DTYPE_BF16
ARG, UNSUP, OK = binding.PE_ERR_ARG, binding.PE_ERR_UNSUPPORTED, binding.PE_OK
P, WS = 1 << 21, 1 << 22
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


@pytest.fixture(scope="module")
def plan(lib):
    p = binding.PeAttnPlan()
    assert lib.pe_attn_plan_init(ctypes.addressof(p), 64, 8, 64, 16, BF16, 1e-6, 1e4) == OK
    return p


def layout(**kw):
    a = dict(B=2, T=4, qsl=P, seq=P, parent=P, table=P, mb=3, nb=8, bs=16, mask=P, words=1, pos=P, slot=P, ws=WS, wsb=256,
             st=None)
    a.update(kw)
    return tuple(a.values())


def accept(**kw):
    a = dict(B=2, T=4, qsl=P, parent=P, tok=P, target=P, accepted=P, path=P, bonus=P, ws=WS, wsb=256, st=None)
    a.update(kw)
    return tuple(a.values())


def attend(p, **kw):
    a = dict(plan=ctypes.addressof(p), B=2, T=4, qsl=P, seq=P, q=P, ldq=4096, k=P, v=P, table=P, mb=3, nb=8, mask=P, words=1,
             sink=None, out=P, ldo=4096, ws=WS, wsb=BIG, st=None)
    a.update(kw)
    return tuple(a.values())


def sample(**kw):
    a = dict(B=2, T=4, qsl=P, logits=P, ld=50, V=50, dtype=F32, temp=P, k=P, p=P, m=P, g=P, ldg=50, token=P, ws=WS, wsb=BIG,
             st=None)
    a.update(kw)
    return tuple(a.values())


def compact(p, **kw):
    a = dict(plan=ctypes.addressof(p), layers=2, B=2, T=4, qsl=P, seq=P, acc=P, path=P, table=P, mb=3, nb=8, k=P, v=P, ws=WS,
             wsb=256, st=None)
    a.update(kw)
    return tuple(a.values())


def copy(p, **kw):
    a = dict(plan=ctypes.addressof(p), layers=2, n=3, src=P, dst=P, nb=8, k=P, v=P, ws=WS, wsb=256, st=None)
    a.update(kw)
    return tuple(a.values())


def fork(p, **kw):
    a = dict(plan=ctypes.addressof(p), layers=2, n=3, parent=P, child=P, length=P, table=P, rows=4, mb=3, nb=8, refs=P, k=P,
             v=P, ws=WS, wsb=BIG, st=None)
    a.update(kw)
    return tuple(a.values())


def reserve(**kw):
    a = dict(n=3, row=P, length=P, table=P, rows=4, mb=3, nb=8, bs=16, refs=P, ws=WS, wsb=BIG, st=None)
    a.update(kw)
    return tuple(a.values())


def free(**kw):
    a = dict(n=3, row=P, table=P, rows=4, mb=3, nb=8, refs=P, ws=WS, wsb=256, st=None)
    a.update(kw)
    return tuple(a.values())


def check(call, make, bad, code=ARG):
    for kw in bad:
        assert call(*make(**kw)) == code, kw


def pointers(*names, align=4):
    return [{n: None} for n in names] + [{n: P + align // 2} for n in names]


def test_layout_and_walk(lib):
    assert lib.pe_tree_layout(*layout(B=0, T=0, qsl=None)) == OK and lib.pe_tree_layout(*layout(T=0, parent=None)) == OK
    check(lib.pe_tree_layout, layout, [dict(B=-1), dict(T=-1), dict(B=0), dict(words=0), dict(words=33), dict(mb=0), dict(nb=-1),
                                       dict(bs=0), dict(wsb=255), dict(ws=WS + 128), dict(ws=None), dict(pos=P + 4),
                                       dict(slot=P + 4), *pointers("qsl", "seq", "parent", "table", "mask")])
    assert lib.pe_tree_layout(*layout(B=65536)) == UNSUP
    assert lib.pe_tree_accept(*accept(B=0, T=0)) == OK
    check(lib.pe_tree_accept, accept, [dict(B=-1), dict(T=-1), dict(B=0), dict(wsb=255), dict(ws=WS + 128), dict(ws=None),
                                       *pointers("qsl", "parent", "tok", "target", "accepted", "path", "bonus")])
    assert lib.pe_tree_accept(*accept(B=65536)) == UNSUP


def test_attention(lib, plan):
    make = lambda **kw: attend(plan, **kw)  # noqa: E731
    assert lib.pe_tree_attention(*make(B=0)) == OK and lib.pe_tree_attention(*make(T=0)) == OK
    check(lib.pe_tree_attention, make, [dict(B=-1), dict(T=-1), dict(words=0), dict(words=33), dict(mask=None), dict(mask=P + 2),
                                        dict(ldq=4088), dict(ldo=4100), dict(mb=0), dict(nb=-1), dict(plan=None), dict(wsb=256),
                                        dict(ws=WS + 8), *pointers("qsl", "seq", "table"),
                                        *pointers("q", "k", "v", "out", align=16)])
    check(lib.pe_tree_attention, make, [dict(B=65536), dict(T=1 << 26), dict(nb=1 << 25), dict(mb=1 << 28)], UNSUP)


def test_sampling(lib):
    assert lib.pe_sample(*sample(B=0, T=0)) == OK and lib.pe_sample(*sample(T=0)) == OK
    check(lib.pe_sample, sample, [dict(B=-1), dict(T=-1), dict(B=0), dict(V=0), dict(ld=49), dict(ldg=49), dict(ws=WS + 128),
                                  dict(ws=None), dict(wsb=lib.pe_sample_workspace_bytes(2, 4, 50) - 1),
                                  dict(temp=P + 2), dict(k=P + 2), dict(p=P + 2), dict(m=P + 1),
                                  *pointers("qsl", "logits", "g", "token")])
    assert lib.pe_sample(*sample(dtype=BF16, logits=P + 1)) == ARG
    check(lib.pe_sample, sample, [dict(dtype=3), dict(B=65536), dict(V=(1 << 20) + 1, ld=1 << 21, ldg=1 << 21)], UNSUP)
    size = lib.pe_sample_workspace_bytes
    assert size(1, 1, 0) == 0 and size(-1, 1, 5) == 0 and size(1, -1, 5) == 0 and size(1, 1, (1 << 20) + 1) == 0
    assert size(1, 0, 5) >= 256 and size(4, 9, 1 << 20) > size(4, 8, 1 << 20) > size(4, 8, 1000)


def test_pages(lib, plan):
    both = lambda make: (lambda **kw: make(plan, **kw))  # noqa: E731
    assert lib.pe_cache_compact(*compact(plan, B=0)) == OK and lib.pe_cache_compact(*compact(plan, T=0)) == OK
    check(lib.pe_cache_compact, both(compact), [dict(plan=None), dict(layers=0), dict(B=-1), dict(T=-1), dict(mb=0), dict(nb=-1),
                                                dict(wsb=255), dict(ws=WS + 4), *pointers("qsl", "seq", "acc", "path", "table"),
                                                *pointers("k", "v", align=16)])
    assert lib.pe_cache_compact(*compact(plan, B=65536)) == UNSUP
    assert lib.pe_cache_copy(*copy(plan, n=0)) == OK
    check(lib.pe_cache_copy, both(copy), [dict(plan=None), dict(layers=0), dict(n=-1), dict(nb=-1), dict(wsb=255), dict(ws=None),
                                          *pointers("src", "dst"), *pointers("k", "v", align=16)])
    need = lib.pe_pages_workspace_bytes(3, 8)
    assert lib.pe_pages_workspace_bytes(-1, 1) == 0 and lib.pe_pages_workspace_bytes(1, -1) == 0
    assert lib.pe_pages_fork(*fork(plan, n=0)) == OK
    check(lib.pe_pages_fork, both(fork), [dict(plan=None), dict(layers=0), dict(n=-1), dict(rows=-1), dict(mb=0), dict(nb=-1),
                                          dict(wsb=need - 1), dict(ws=WS + 128),
                                          *pointers("parent", "child", "length", "table", "refs"),
                                          *pointers("k", "v", align=16)])
    assert lib.pe_pages_fork(*fork(plan, n=65536)) == UNSUP
    assert lib.pe_pages_reserve(*reserve(n=0)) == OK and lib.pe_pages_reserve(*reserve(n=65536)) == UNSUP
    check(lib.pe_pages_reserve, reserve, [dict(n=-1), dict(rows=-1), dict(mb=0), dict(nb=-1), dict(bs=0), dict(wsb=need - 1),
                                          dict(ws=None), *pointers("row", "length", "table", "refs")])
    assert lib.pe_pages_free(*free(n=0)) == OK
    check(lib.pe_pages_free, free, [dict(n=-1), dict(rows=-1), dict(mb=0), dict(nb=-1), dict(wsb=255), dict(ws=WS + 64),
                                    *pointers("row", "table", "refs")])
    for mb, code in (((1 << 22) - 1, OK), (1 << 22, UNSUP)):
        assert lib.pe_pages_free(*free(n=0, mb=mb)) == code and lib.pe_pages_reserve(*reserve(n=0, mb=mb)) == code
        assert lib.pe_pages_fork(*fork(plan, n=0, mb=mb)) == code


def test_status_bits_match_the_header():
    src = open(binding.HEADER).read()
    for name in ("PE_ST_TREE", "PE_ST_PAGES"):
        value = int(src.split(f"#define {name} ")[1].split("u")[0], 16)
        assert getattr(binding, name) == value
    assert f"#define PE_TREE_MAX_NODES {binding.PE_TREE_MAX_NODES}" in src
