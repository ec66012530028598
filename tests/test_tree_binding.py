"""What the binding of the tree, sampling and page calls hands to the library: tensors of another
type, size, layout or device than the call reads are refused before it (no GPU needed: the
library's calls are stand-ins that note their arguments)."""

import os
import shutil

import pytest

from speculative_drafting_gb300 import binding, build

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists(
    "/usr/local/cuda/bin/nvcc"), reason="needs nvcc to build libpe.so")

H, G, HD, BS, T, B, NB, V, LAYERS, ROWS = 4, 2, 64, 16, 5, 2, 3, 40, 2, 4
BF, I32, I64 = torch.bfloat16, torch.int32, torch.int64
NAMES = ("pe_tree_layout", "pe_tree_attention", "pe_tree_accept", "pe_sample", "pe_cache_compact", "pe_cache_copy",
         "pe_pages_reserve", "pe_pages_fork", "pe_pages_free")


class Calls:
    def __init__(self, lib):
        self.lib, self.made = lib, []

    def __getattr__(self, name):
        if name in NAMES:
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


def ints(*shape):
    return torch.zeros(*shape, dtype=I32)


def ws():
    return torch.zeros(256, dtype=torch.uint8)


def caches():
    return dict(k_cache=torch.zeros(LAYERS, NB, G, BS, HD, dtype=BF), v_cache=torch.zeros(LAYERS, NB, G, BS, HD, dtype=BF))


def plan():
    return binding.PagedAttention(H, G, HD, BS)


def given():
    """Each call: the function, and its arguments as they should be."""
    p = plan()
    qsl, seq, table = torch.tensor([0, 3, T], dtype=I32), ints(B), ints(B, 2)
    one = dict(k_cache=torch.zeros(NB, G, BS, HD, dtype=BF), v_cache=torch.zeros(NB, G, BS, HD, dtype=BF))
    pages = dict(block_table=ints(ROWS, 2), refs=ints(NB), ws=binding.pages_workspace(4, NB, device="cpu"))
    return {
        "layout": (binding.tree_layout, dict(B=B, T=T, qsl=qsl, seq_len=seq, parent=ints(T), block_table=table, num_blocks=NB,
                                             block_size=BS, mask=ints(T, 2), pos=torch.zeros(T, dtype=I64),
                                             slot=torch.zeros(T, dtype=I64), ws=ws())),
        "accept": (binding.tree_accept, dict(B=B, T=T, qsl=qsl, parent=ints(T), tok=ints(T), target=ints(T), accepted=ints(B),
                                             path=ints(T), bonus=ints(B), ws=ws())),
        "attend": (p.attend_tree, dict(B=B, T=T, qsl=qsl, seq_len=seq, q=torch.zeros(T, H, HD, dtype=BF), block_table=table,
                                       num_blocks=NB, mask=ints(T, 2), out=torch.zeros(T, H * HD, dtype=BF),
                                       ws=p.workspace(B, T, device="cpu"), sink=torch.zeros(H), **one)),
        "sample": (binding.sample, dict(B=B, T=T, qsl=qsl, logits=torch.zeros(T, V), vocab=V, temperature=torch.ones(B),
                                        top_k=ints(B), top_p=torch.ones(B), min_p=torch.zeros(B), gumbel=torch.zeros(T, V),
                                        token=ints(T), ws=binding.sample_workspace(B, T, V, device="cpu"))),
        "compact": (p.compact, dict(n_layers=LAYERS, B=B, T=T, qsl=qsl, seq_len=seq, accepted=ints(B), path=ints(T),
                                    block_table=table, num_blocks=NB, ws=ws(), **caches())),
        "copy": (p.copy_pages, dict(n_layers=LAYERS, n=2, src=ints(2), dst=ints(2), num_blocks=NB, ws=ws(), **caches())),
        "fork": (p.fork, dict(n_layers=LAYERS, n=2, parent=ints(2), child=ints(2), length=ints(2), **pages, **caches())),
        "reserve": (binding.pages_reserve, dict(n=2, row=ints(2), length=ints(2), block_size=BS, **pages)),
        "free": (binding.pages_free, dict(n=2, row=ints(2), **pages)),
    }


def refused(calls, call, args, *cases):
    call(**args)
    assert len(calls.made) == 1
    for kw in cases:
        with pytest.raises((ValueError, binding.PeError)):
            call(**{**args, **kw})
        assert len(calls.made) == 1, {k: getattr(v, "dtype", v) for k, v in kw.items()}
    calls.made.clear()


CALLS = ("layout", "accept", "attend", "sample", "compact", "copy", "fork", "reserve", "free")


@pytest.mark.parametrize("name", CALLS)
def test_every_tensor_of_another_type_layout_or_size_is_refused(calls, name):
    call, args = given()[name]
    for k, t in args.items():
        if not isinstance(t, torch.Tensor) or k == "ws":
            continue
        other = {I32: I64, I64: I32, torch.float32: torch.float64, BF: torch.float32}[t.dtype]
        cases = [{k: t.to(other)}, {k: t.to(torch.half)}]
        if t.dtype == torch.float32 and k != "logits":
            cases.append({k: t.to(BF)})
        wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2]
        cases.append({k: wide})
        if k not in ("block_table", "refs", "mask"):
            cases.append({k: t[:-1] if k not in ("k_cache", "v_cache") else t[..., :-1].contiguous()})
        if k == "mask":
            cases.append({k: t[:-1]})
        if k == "block_table" and name in ("layout", "attend", "compact"):
            cases.append({k: t[:-1]})
        if k in ("block_table", "mask"):
            cases.append({k: t.view(-1)})
        refused(calls, call, args, *cases)


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_are_refused(calls, name):
    class Elsewhere(torch.Tensor):
        def get_device(self):
            return 1

    call, args = given()[name]
    tensors = [k for k, t in args.items() if isinstance(t, torch.Tensor)]
    assert len(tensors) >= 3
    refused(calls, call, args, *({k: args[k].as_subclass(Elsewhere)} for k in tensors))


@pytest.mark.parametrize("name", CALLS)
def test_more_rows_than_the_tensors_have_are_refused(calls, name):
    call, args = given()[name]
    if "n" in args:
        refused(calls, call, args, dict(n=3))
    else:
        refused(calls, call, args, dict(T=T + 1), dict(B=B + 1))
    if "n_layers" in args:
        refused(calls, call, args, dict(n_layers=LAYERS + 1))
    if name in ("compact", "copy", "attend"):
        refused(calls, call, args, dict(num_blocks=NB + 1))
    if name == "sample":
        refused(calls, call, args, dict(vocab=V + 1))


def test_optional_tensors_and_strided_rows(calls):
    g = given()
    call, args = g["layout"]
    call(**{**args, "pos": None, "slot": None})
    call, args = g["attend"]
    call(**{**args, "sink": None, "q": torch.zeros(T, H * HD + 8, dtype=BF)})
    call, args = g["sample"]
    call(**{**args, "temperature": None, "top_k": None, "top_p": None, "min_p": None,
            "logits": torch.zeros(T, V + 3, dtype=BF)[:, :V], "gumbel": torch.zeros(2 * T, V)[::2]})
    (_, layout), (_, attend), (_, sample) = calls.made
    assert layout[11] is None and layout[12] is None
    assert attend[6] == H * HD + 8 and attend[14] is None
    assert sample[4] == V + 3 and sample[6] == binding.PE_DTYPE_BF16 and sample[12] == 2 * V and sample[7:11] == (None,) * 4
    # nothing to do
    call, args = g["accept"]
    call(**{**args, "B": 0, "T": 0, "qsl": ints(0)})
    call, args = g["free"]
    call(**{**args, "n": 0})
