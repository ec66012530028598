"""ctypes binding of ``libpe.so`` (include/pe.h), with the same call names.

Argument marshalling only: every step of the draft path runs in the library's
CUDA kernels.  PyTorch supplies device memory (tensor data pointers) and
streams; the helpers below allocate the caller-owned buffers the C-ABI expects.
There is no fallback: loading fails loudly when the library is missing.
"""

from __future__ import annotations

import ctypes
import os
import re

from . import build as _build

PE_OK = 0
PE_ERR_ARG = 1
PE_ERR_UNSUPPORTED = 2
PE_ERR_CUDA = 3
PE_ERR_DEVICE_INPUT = 4
PE_ERR_TIMEOUT = 5
PE_ST_ACCEPTED_RANGE = 0x1
PE_ST_BLOCK_RANGE = 0x2
PE_ST_TOKEN_RANGE = 0x4
PE_ST_ROWS_RANGE = 0x8
PE_ST_TIMEOUT = 0x10
PE_ST_CAPACITY = 0x20
PE_ST_SAMPLING = 0x40
PE_COD_MAX_DEPTH = 16
PE_DTYPE_F32 = 0
PE_DTYPE_BF16 = 1

HEADER = os.path.join(_build.ROOT, "include", "pe.h")
TESTING_HEADER = os.path.join(_build.ROOT, "include", "pe_testing.h")


class PeError(RuntimeError):
    def __init__(self, code, what):
        super().__init__(f"{what}: {status_string(code)} (code {code})")
        self.code = code


class PeDims(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("n_streams", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("K", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("mask_id", ctypes.c_int32), ("post_norm", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("eps", ctypes.c_float), ("rope_theta", ctypes.c_float), ("n_layers", ctypes.c_int32)]


WEIGHT_FIELDS = ["emb", "emb_mask", "h_shared", "gamma_stream", "w_fc", "gamma_in", "w_qkv", "w_o",
                 "gamma_post", "w_gate", "w_up", "w_down", "gamma_final", "w_lm", "attn_sink"]
LAYER_FIELDS = ["gamma_in", "w_qkv", "w_o", "gamma_post", "w_gate", "w_up", "w_down", "gamma_final",
                "attn_sink"]


class PeLayerWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in LAYER_FIELDS]


class PeWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in WEIGHT_FIELDS] + \
        [("more_layers", ctypes.POINTER(PeLayerWeights)), ("packed", ctypes.c_void_p),
         ("packed_bytes", ctypes.c_size_t)]


META_FIELDS = ["out_qsl", "tok", "pos", "is_rejected", "is_masked", "hidden_src", "slot",
               "valid_qsl", "valid_rows", "n_valid", "sample_idx", "seq_len"]


class PeMeta(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in META_FIELDS]


class PeAttnPlan(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("rope_turn", ctypes.c_uint64 * 64)]


_lib = None
_vp, _i32, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t


def lib_path() -> str:
    return _build.LIB_PATH


def load(path: str | None = None):
    """Load libpe.so (built by ``build.build()``); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built: run speculative_drafting_gb300.build.build()")
    lib = ctypes.CDLL(path)
    lib.pe_create.argtypes = [ctypes.POINTER(PeDims), ctypes.POINTER(PeWeights), ctypes.POINTER(_vp)]
    lib.pe_create.restype = _i32
    lib.pe_destroy.argtypes = [_vp]
    lib.pe_destroy.restype = None
    lib.pe_packed_weights_bytes.argtypes = [ctypes.POINTER(PeDims)]
    lib.pe_packed_weights_bytes.restype = _sz
    lib.pe_pack_weights.argtypes = [ctypes.POINTER(PeDims), ctypes.POINTER(PeWeights), _vp, _sz, _vp]
    lib.pe_pack_weights.restype = _i32
    lib.pe_workspace_bytes.argtypes = [_vp, _i32, _i32, _i32]
    lib.pe_workspace_bytes.restype = _sz
    lib.pe_prepare_inputs.argtypes = [_vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _vp,
                                      ctypes.POINTER(PeMeta), _vp, _vp, _vp, _vp, _sz, _vp]
    lib.pe_prepare_inputs.restype = _i32
    lib.pe_draft_step.argtypes = [_vp, _i32, _i32, ctypes.POINTER(PeMeta), _vp, _vp, _i32, _i32, _vp,
                                  _vp, _vp, _vp, _sz, _vp]
    lib.pe_draft_step.restype = _i32
    lib.pe_argmax.argtypes = [_vp, _vp, _i32, _vp, _vp, _vp, _sz, _vp]
    lib.pe_argmax.restype = _i32
    lib.pe_read_status.argtypes = [_vp, _vp, ctypes.POINTER(ctypes.c_uint32), _i32, _vp]
    lib.pe_read_status.restype = _i32
    lib.pe_status_string.argtypes = [_i32]
    lib.pe_status_string.restype = ctypes.c_char_p
    lib.pe_autoregressive_workspace_bytes.argtypes = [_vp, _i32, _i32, _i32]
    lib.pe_autoregressive_workspace_bytes.restype = _sz
    lib.pe_draft_autoregressive.argtypes = [_vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                            _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
    lib.pe_draft_autoregressive.restype = _i32
    lib.pe_argmax_noalloc.argtypes = [_vp, _vp, _i32, _vp, _vp, _vp]
    lib.pe_argmax_noalloc.restype = _i32
    lib.pe_test_projection_workspace.argtypes = [_vp, _i32, _i32]
    lib.pe_test_projection_workspace.restype = _sz
    lib.pe_test_projection.argtypes = [_vp, _i32, _vp, _i32, _vp, _vp, _sz, _vp]
    lib.pe_test_projection.restype = _i32
    lib.pe_test_bounded_wait.argtypes = [_vp, _sz, _vp]
    lib.pe_test_bounded_wait.restype = _i32
    lib.pe_verify_workspace_bytes.argtypes = [_i32, _i32]
    lib.pe_verify_workspace_bytes.restype = _sz
    lib.pe_verify_greedy.argtypes = [_i32, _i32, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _vp,
                                     _sz, _vp]
    lib.pe_verify_greedy.restype = _i32
    lib.pe_cod_workspace_bytes.argtypes = [_i32, _i32, _i32]
    lib.pe_cod_workspace_bytes.restype = _sz
    lib.pe_cod_sample_indices.argtypes = [_i32, _i32, _vp, _vp, _i32, ctypes.c_float, _i32, _vp,
                                          _vp, _vp, _vp, _vp, _sz, _vp]
    lib.pe_cod_sample_indices.restype = _i32
    lib.pe_cod_mask.argtypes = [_i32, _i32, _vp, _i32, _vp, _vp, _vp, ctypes.c_int64,
                                ctypes.c_int64, ctypes.c_int64, _vp, _sz, _vp]
    lib.pe_cod_mask.restype = _i32
    lib.pe_verify_sampled_workspace_bytes.argtypes = [_i32, _i32, _i32]
    lib.pe_verify_sampled_workspace_bytes.restype = _sz
    lib.pe_verify_sampled.argtypes = [_i32, _i32, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _vp,
                                      _vp, _vp, _vp, _sz, _vp]
    lib.pe_verify_sampled.restype = _i32
    lib.pe_attn_plan_init.argtypes = [_vp, _i32, _i32, _i32, _i32, _i32, ctypes.c_float,
                                      ctypes.c_float]
    lib.pe_attn_plan_init.restype = _i32
    lib.pe_qkv_append.argtypes = [_vp, _i32, _vp, ctypes.c_int64, _vp, _vp, _vp, _vp, _i32, _vp,
                                  _vp, _vp, _vp, _sz, _vp]
    lib.pe_qkv_append.restype = _i32
    lib.pe_chunk_attention_workspace_bytes.argtypes = [_vp, _i32, _i32]
    lib.pe_chunk_attention_workspace_bytes.restype = _sz
    lib.pe_chunk_attention.argtypes = [_vp, _i32, _i32, _vp, _vp, _vp, ctypes.c_int64, _vp, _vp,
                                       _vp, _i32, _i32, _vp, _vp, ctypes.c_int64, _vp, _sz, _vp]
    lib.pe_chunk_attention.restype = _i32
    args = lib.pe_chunk_attention.argtypes
    lib.pe_test_chunk_attention_stall.argtypes = [args[0], _i32, *args[1:]]
    lib.pe_test_chunk_attention_stall.restype = _i32
    _lib = lib
    return lib


def declared_functions(header: str = HEADER):
    """Names of the functions include/pe.h declares."""
    src = open(header).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(pe_[a-z_]+)\s*\(", src)))


def status_string(code: int) -> str:
    return load().pe_status_string(int(code)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _addr(t):
    # a plain integer: ctypes converts it to the void* argument without an object
    return None if t is None else t.data_ptr()


_raw_stream = None
_current_device = None


def _stream_handle(stream, t):
    """The cudaStream_t of `stream`, or the current one; a tensor t of another device than
    the current one is refused (the launch would go to the current one)."""
    global _raw_stream, _current_device
    if _raw_stream is None:
        import torch

        # what torch.cuda.current_stream and current_device wrap, 3 us a call
        _raw_stream = torch._C._cuda_getCurrentRawStream
        _current_device = torch._C._cuda_getDevice
    dev = t.get_device()
    if dev != _current_device():
        raise ValueError(f"tensors on device {dev}, the current device is {_current_device()}")
    return _raw_stream(dev) if stream is None else stream.cuda_stream


def _row_stride(t, T, heads, hd):
    """Elements from one row of [T][heads][hd] (or [T][heads hd]) to the next; the rows
    themselves have to be dense, and there."""
    n, s = t.shape, t.stride()
    if len(s) == 3:
        dense, width = s[2] == 1 and (s[1] == hd or n[1] == 1), n[1] * n[2]
    elif len(s) == 2:
        dense, width = s[1] == 1, n[1]
    else:  # [T][G][H/G][hd] and the like
        dense, width = True, 1
        for size, stride in zip(reversed(n[1:]), reversed(s[1:])):
            dense = dense and (stride == width or size == 1)
            width *= size
    if not dense:
        raise ValueError(f"rows of shape {tuple(n[1:])} with strides {s}: a row has to be dense")
    if n[0] < T or width < heads * hd:
        raise ValueError(f"{T} rows of {heads} heads of {hd} do not fit the shape {tuple(n)}")
    return s[0]


def _check(rc, what):
    if rc != PE_OK:
        raise PeError(rc, what)


def make_dims(dm) -> PeDims:
    """PeDims from any object with the Dims attributes (workloads.Dims)."""
    return PeDims(d=dm.d, n_streams=3, n_heads=dm.n_heads, n_kv_heads=dm.n_kv_heads,
                  head_dim=dm.head_dim, inter=dm.inter, vocab=dm.vocab, K=dm.K,
                  block_size=dm.block_size, mask_id=dm.mask_id, post_norm=int(bool(dm.post_norm)),
                  dtype=PE_DTYPE_BF16 if dm.dtype == "bf16" else PE_DTYPE_F32,
                  eps=dm.eps, rope_theta=dm.rope_theta, n_layers=getattr(dm, "n_layers", 1))


class Meta:
    """Caller-owned metadata buffers for a batch of B requests and T_in rows."""

    def __init__(self, B: int, T_in: int, K: int, device="cuda"):
        import torch

        T_out = T_in + B * (K - 1)
        i32, i64, u8 = torch.int32, torch.int64, torch.uint8
        self.B, self.T_in, self.T_out, self.K = B, T_in, T_out, K
        self.t = {
            "out_qsl": torch.empty(B + 1, dtype=i32, device=device),
            "tok": torch.empty(T_out, dtype=i32, device=device),
            "pos": torch.empty(T_out, dtype=i64, device=device),
            "is_rejected": torch.empty(T_out, dtype=u8, device=device),
            "is_masked": torch.empty(T_out, dtype=u8, device=device),
            "hidden_src": torch.empty(T_out, dtype=i32, device=device),
            "slot": torch.empty(T_out, dtype=i64, device=device),
            "valid_qsl": torch.empty(B + 1, dtype=i32, device=device),
            "valid_rows": torch.empty(T_out, dtype=i32, device=device),
            "n_valid": torch.empty(1, dtype=i32, device=device),
            "sample_idx": torch.empty(B * K, dtype=i32, device=device),
            "seq_len": torch.empty(B, dtype=i32, device=device),
        }
        self.c = PeMeta(**{k: v.data_ptr() for k, v in self.t.items()})

    def __getitem__(self, k):
        return self.t[k]


class Drafter:
    """One drafter handle: ``pe_create`` over device weight tensors (borrowed).
    A bf16 drafter's projection matrices are first tile-packed (pe_pack_weights)
    into a buffer this object owns and the handle borrows."""

    def __init__(self, dims, weights: dict, stream=None):
        import torch

        self.lib = load()
        self.dims = dims
        self.weights = weights  # keep the tensors alive for the handle's lifetime
        cw = PeWeights(**{k: (weights[k].data_ptr() if weights.get(k) is not None else None)
                          for k in WEIGHT_FIELDS})
        more = weights.get("layers") or []
        if more:
            # host array of the later layers' device pointers (read by pe_create)
            arr = (PeLayerWeights * len(more))()
            for i, lw in enumerate(more):
                for k in LAYER_FIELDS:
                    setattr(arr[i], k, lw[k].data_ptr() if lw.get(k) is not None else None)
            cw.more_layers = arr
        self.cw = cw
        h = ctypes.c_void_p()
        self.cdims = make_dims(dims)
        self.packed = None
        n = int(self.lib.pe_packed_weights_bytes(ctypes.byref(self.cdims)))
        if n and weights.get("w_fc") is not None:
            dev = weights["w_fc"].device
            self.packed = torch.empty(n, dtype=torch.uint8, device=dev)
            self.pack(stream)
            # the handle may be used on any stream: let the packing finish first
            (stream or torch.cuda.current_stream()).synchronize()
            cw.packed = self.packed.data_ptr()
            cw.packed_bytes = n
        _check(self.lib.pe_create(ctypes.byref(self.cdims), ctypes.byref(cw), ctypes.byref(h)), "pe_create")
        self.h = h

    def pack(self, stream=None, weights=None):
        """pe_pack_weights into this drafter's packed buffer (from `weights`, a
        PeWeights, when given: the tests pack other matrices into it)."""
        _check(self.lib.pe_pack_weights(ctypes.byref(self.cdims), ctypes.byref(weights or self.cw),
                                        _ptr(self.packed), self.packed.numel(), _stream(stream)),
               "pe_pack_weights")

    def close(self):
        if self.h:
            self.lib.pe_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def workspace_bytes(self, max_batch: int, max_rows_in: int, max_blocks: int) -> int:
        return int(self.lib.pe_workspace_bytes(self.h, max_batch, max_rows_in, max_blocks))

    def workspace(self, max_batch: int, max_rows_in: int, max_blocks: int, device="cuda"):
        import torch

        n = self.workspace_bytes(max_batch, max_rows_in, max_blocks)
        if n == 0:
            raise PeError(PE_ERR_ARG, "pe_workspace_bytes")
        return torch.zeros(n, dtype=torch.uint8, device=device)

    def prepare_inputs(self, B, T_in, qsl, prev_tok, prev_pos, accepted, bonus, block_table,
                       num_blocks, H_tgt, meta: Meta, ws, G=None, E=None, A=None, stream=None):
        rc = self.lib.pe_prepare_inputs(
            self.h, B, T_in, _ptr(qsl), _ptr(prev_tok), _ptr(prev_pos), _ptr(accepted), _ptr(bonus),
            _ptr(block_table), block_table.shape[1], num_blocks, _ptr(H_tgt), ctypes.byref(meta.c),
            _ptr(G), _ptr(E), _ptr(A), _ptr(ws), ws.numel(), _stream(stream))
        _check(rc, "pe_prepare_inputs")

    def draft_step(self, B, T_in, meta: Meta, A, block_table, num_blocks, k_cache, v_cache, z_out,
                   ws, stream=None):
        rc = self.lib.pe_draft_step(self.h, B, T_in, ctypes.byref(meta.c), _ptr(A), _ptr(block_table),
                                    block_table.shape[1], num_blocks, _ptr(k_cache), _ptr(v_cache),
                                    _ptr(z_out), _ptr(ws), ws.numel(), _stream(stream))
        _check(rc, "pe_draft_step")

    def argmax(self, z, n_rows, draft_tokens, ws, logits=None, stream=None):
        rc = self.lib.pe_argmax(self.h, _ptr(z), n_rows, _ptr(draft_tokens), _ptr(logits), _ptr(ws),
                                ws.numel(), _stream(stream))
        _check(rc, "pe_argmax")

    def autoregressive_workspace(self, max_batch: int, max_rows_in: int, max_blocks: int,
                                 device="cuda"):
        import torch

        n = int(self.lib.pe_autoregressive_workspace_bytes(self.h, max_batch, max_rows_in,
                                                           max_blocks))
        if n == 0:
            raise PeError(PE_ERR_ARG, "pe_autoregressive_workspace_bytes")
        return torch.zeros(n, dtype=torch.uint8, device=device)

    def draft_autoregressive(self, B, T_in, qsl, prev_tok, prev_pos, accepted, bonus, block_table,
                             num_blocks, H_tgt, k_cache, v_cache, draft_tokens, ws, logits=None,
                             hidden=None, stream=None):
        """pe_draft_autoregressive: K sequential one-token passes (the baseline)."""
        rc = self.lib.pe_draft_autoregressive(
            self.h, B, T_in, _ptr(qsl), _ptr(prev_tok), _ptr(prev_pos), _ptr(accepted), _ptr(bonus),
            _ptr(block_table), block_table.shape[1], num_blocks, _ptr(H_tgt), _ptr(k_cache),
            _ptr(v_cache), _ptr(draft_tokens), _ptr(logits), _ptr(hidden), _ptr(ws), ws.numel(),
            _stream(stream))
        _check(rc, "pe_draft_autoregressive")

    def argmax_noalloc(self, z, n_rows, draft_tokens, logits=None, stream=None):
        """pe_argmax without a workspace (its scratch is a static device array)."""
        rc = self.lib.pe_argmax_noalloc(self.h, _ptr(z), n_rows, _ptr(draft_tokens), _ptr(logits),
                                        _stream(stream))
        _check(rc, "pe_argmax_noalloc")

    def test_projection(self, which, X, n_rows, out, stream=None):
        """One drafter projection through the step's GEMM kernel (pe_testing.h)."""
        import torch

        n = int(self.lib.pe_test_projection_workspace(self.h, which, n_rows))
        if n == 0:
            raise PeError(PE_ERR_ARG, "pe_test_projection_workspace")
        ws = torch.zeros(n, dtype=torch.uint8, device=X.device)
        rc = self.lib.pe_test_projection(self.h, which, _ptr(X), n_rows, _ptr(out), _ptr(ws), n,
                                         _stream(stream))
        _check(rc, "pe_test_projection")
        return ws

    def read_status(self, ws, clear=True, stream=None):
        v = ctypes.c_uint32(0)
        rc = self.lib.pe_read_status(self.h, _ptr(ws), ctypes.byref(v), int(clear), _stream(stream))
        if rc not in (PE_OK, PE_ERR_DEVICE_INPUT, PE_ERR_TIMEOUT):
            raise PeError(rc, "pe_read_status")
        return int(v.value), rc


# ----------------------------------------------------------------------------- verification


def verify_workspace_bytes(max_rows_in: int, vocab: int) -> int:
    n = int(load().pe_verify_workspace_bytes(int(max_rows_in), int(vocab)))
    if n == 0:
        raise PeError(PE_ERR_ARG, "pe_verify_workspace_bytes")
    return n


def verify_workspace(max_rows_in: int, vocab: int, device="cuda"):
    """A device workspace for pe_verify_greedy (torch allocates it 256-byte aligned)."""
    import torch

    return torch.zeros(verify_workspace_bytes(max_rows_in, vocab), dtype=torch.uint8,
                       device=device)


def verify_greedy(B, T_in, qsl, tok, logits, vocab, dtype, target_tok, accepted, bonus, ws,
                  stream=None):
    """pe_verify_greedy on device tensors; dtype is PE_DTYPE_F32 or PE_DTYPE_BF16."""
    rc = load().pe_verify_greedy(int(B), int(T_in), _ptr(qsl), _ptr(tok), _ptr(logits),
                                 int(vocab), int(dtype), _ptr(target_tok), _ptr(accepted),
                                 _ptr(bonus), _ptr(ws), int(ws.numel()), _stream(stream))
    _check(rc, "pe_verify_greedy")


def read_status_ws(ws, clear=True, stream=None):
    """pe_read_status without a handle (the verification call has none)."""
    v = ctypes.c_uint32(0)
    rc = load().pe_read_status(None, _ptr(ws), ctypes.byref(v), int(clear), _stream(stream))
    if rc not in (PE_OK, PE_ERR_DEVICE_INPUT, PE_ERR_TIMEOUT):
        raise PeError(rc, "pe_read_status")
    return int(v.value), rc


_torch_types = None


def _types():
    global _torch_types
    if _torch_types is None:
        import torch

        _torch_types = torch.float32, torch.bfloat16, torch.int32
    return _torch_types


def verify_sampled_workspace(max_batch: int, max_rows_in: int, vocab: int, device="cuda"):
    """A device workspace for pe_verify_sampled (torch allocates it 256-byte aligned)."""
    import torch

    n = int(load().pe_verify_sampled_workspace_bytes(int(max_batch), int(max_rows_in), int(vocab)))
    if n == 0:
        raise PeError(PE_ERR_ARG, "pe_verify_sampled_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def verify_sampled(B, T_in, qsl, tok, logits, vocab, dtype, temperature, u, gumbel, accepted, bonus,
                   p_draft, ws, stream=None):
    """pe_verify_sampled on device tensors, dense ones; dtype is PE_DTYPE_F32 or
    PE_DTYPE_BF16 and the type of logits; qsl, tok, accepted and bonus are int32, the other
    tensors float32; temperature and p_draft may be None."""
    f32, bf16, i32 = _types()
    dev = ws.get_device()
    for name, t, ty, n in (("logits", logits, bf16 if dtype == PE_DTYPE_BF16 else f32, T_in * vocab),
                           ("qsl", qsl, i32, B and B + 1), ("tok", tok, i32, T_in), ("u", u, f32, T_in),
                           ("temperature", temperature, f32, B), ("gumbel", gumbel, f32, B * vocab),
                           ("accepted", accepted, i32, B), ("bonus", bonus, i32, B),
                           ("p_draft", p_draft, f32, T_in)):
        if t is None:
            continue
        if t.get_device() != dev:
            raise ValueError(f"{name} is on device {t.get_device()}, ws on {dev}")
        if not (t.dtype is ty and t.numel() >= n and t.is_contiguous()):
            raise ValueError(f"{name}: {n} dense elements of the type {ty} are read or written, "
                             f"got {t.dtype} {tuple(t.shape)} strides {t.stride()}")
    rc = load().pe_verify_sampled(B, T_in, _addr(qsl), _addr(tok), _addr(logits), vocab, dtype,
                                  _addr(temperature), _addr(u), _addr(gumbel), _addr(accepted),
                                  _addr(bonus), _addr(p_draft), _addr(ws), ws.numel(),
                                  _stream_handle(stream, ws))
    _check(rc, "pe_verify_sampled")


# ----------------------------------------------------------------------------- paged attention calls


class PagedAttention:
    """The paged cache write and attention of one layer shape (a pe_attn_plan): rows
    outside a draft step, such as prompts, chunks of prompts and verify rows.
    dtype is "bf16" or "f32"; caches are [num_blocks][G][block_size][hd]."""

    def __init__(self, n_heads, n_kv_heads, head_dim, block_size, dtype="bf16", eps=1e-6,
                 rope_theta=10000.0):
        import torch

        self.lib = load()
        self.c = PeAttnPlan()
        self.addr = ctypes.addressof(self.c)
        self.hd = head_dim
        self.i32, self.i64, self.f32 = torch.int32, torch.int64, torch.float32
        self.dtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.heads, self.qkv_heads = n_heads, n_heads + 2 * n_kv_heads
        self.width = n_heads * head_dim
        self.block = n_kv_heads * block_size * head_dim  # elements of a cache's block
        code = {"bf16": PE_DTYPE_BF16, "f32": PE_DTYPE_F32}.get(dtype, -1)
        _check(self.lib.pe_attn_plan_init(self.addr, n_heads, n_kv_heads, head_dim, block_size,
                                          code, eps, rope_theta), "pe_attn_plan_init")

    def _refuse(self, *tensors):
        got = ", ".join(f"{t.dtype} {tuple(t.shape)} strides {t.stride()}" for t in tensors if t is not None)
        raise ValueError(f"the plan's type is {self.dtype}; caches, q_out, gains (of head_dim elements) and "
                         f"block_table are dense: got {got}")

    def _refuse_ints(self, what, *tensors):
        got = ", ".join(f"{t.dtype} strides {t.stride()}" for t in tensors)
        raise ValueError(f"{what}, all dense: got {got}")

    def _too_small(self, what, *tensors):
        raise ValueError(f"{what} of {self.heads} heads do not fit the shapes "
                         f"{[tuple(t.shape) for t in tensors if t is not None]}")

    def _apart(self, *tensors):
        raise ValueError(f"tensors on devices {[t.get_device() for t in tensors if t is not None]}: "
                         "all have to be on the workspace's")

    def _gain(self, t):
        # of the plan's type: other bytes would be read as if they were
        if not (t.dtype is self.dtype and t.numel() == self.hd and t.is_contiguous()):
            self._refuse(t)
        return t.data_ptr()

    def append_workspace(self, device="cuda"):
        """The status word of ``append`` (zeroed)."""
        import torch

        return torch.zeros(256, dtype=torch.uint8, device=device)

    def workspace(self, max_batch: int, max_rows: int, device="cuda"):
        """A device workspace for ``attend`` with at most max_batch requests and max_rows rows."""
        import torch

        n = int(self.lib.pe_chunk_attention_workspace_bytes(self.addr, int(max_batch),
                                                            int(max_rows)))
        if n == 0:
            raise PeError(PE_ERR_ARG, "pe_chunk_attention_workspace_bytes")
        return torch.zeros(n, dtype=torch.uint8, device=device)

    def append(self, T, qkv, gamma_q, gamma_k, pos, slot, num_blocks, q_out, k_cache, v_cache, ws,
               stream=None):
        """pe_qkv_append: qkv [T][H + 2G][hd] (or [T][(H + 2G) hd]; its rows may be
        strided), gains and q_out may be None; the gains have the plan's type."""
        # (a call of a few rows is bound by its host time: the checks stand in line and cost
        # 1.1 us of 6.5)
        d, i64, n = self.dtype, self.i64, num_blocks * self.block
        if not (qkv.dtype is d and k_cache.dtype is d and v_cache.dtype is d
                and k_cache.is_contiguous() and v_cache.is_contiguous()
                and (q_out is None or (q_out.dtype is d and q_out.is_contiguous()))):
            self._refuse(qkv, k_cache, v_cache, q_out)
        if not (pos.dtype is i64 and slot.dtype is i64 and pos.is_contiguous() and slot.is_contiguous()):
            self._refuse_ints("pos and slot have the type int64", pos, slot)
        if (pos.numel() < T or slot.numel() < T or (q_out is not None and q_out.numel() < T * self.width)
                or k_cache.numel() < n or v_cache.numel() < n):
            self._too_small(f"{T} rows, {num_blocks} blocks", pos, slot, q_out, k_cache, v_cache)
        dev = ws.get_device()
        if not (dev == qkv.get_device() == pos.get_device() == slot.get_device()
                == k_cache.get_device() == v_cache.get_device() and (q_out is None or q_out.get_device() == dev)
                and (gamma_q is None or gamma_q.get_device() == dev)
                and (gamma_k is None or gamma_k.get_device() == dev)):
            self._apart(ws, qkv, pos, slot, k_cache, v_cache, q_out, gamma_q, gamma_k)
        rc = self.lib.pe_qkv_append(self.addr, T, qkv.data_ptr(), _row_stride(qkv, T, self.qkv_heads, self.hd),
                                    None if gamma_q is None else self._gain(gamma_q),
                                    None if gamma_k is None else self._gain(gamma_k),
                                    pos.data_ptr(), slot.data_ptr(), num_blocks,
                                    None if q_out is None else q_out.data_ptr(),
                                    k_cache.data_ptr(), v_cache.data_ptr(), ws.data_ptr(),
                                    ws.numel(), _stream_handle(stream, ws))
        _check(rc, "pe_qkv_append")

    def attend(self, B, T, qsl, seq_len, q, k_cache, v_cache, block_table, num_blocks, out, ws,
               sink=None, stream=None):
        """pe_chunk_attention: q and out [T][H][hd] (or [T][H hd]; their rows may be
        strided)."""
        d = self.dtype
        if not (q.dtype is d and k_cache.dtype is d and v_cache.dtype is d and out.dtype is d
                and k_cache.is_contiguous() and v_cache.is_contiguous() and block_table.is_contiguous()):
            self._refuse(q, k_cache, v_cache, out, block_table)
        i32 = self.i32
        if not (qsl.dtype is i32 and seq_len.dtype is i32 and block_table.dtype is i32
                and qsl.is_contiguous() and seq_len.is_contiguous()):
            self._refuse_ints("qsl, seq_len and block_table have the type int32", qsl, seq_len, block_table)
        if sink is not None and not (sink.dtype is self.f32 and sink.is_contiguous()):
            self._refuse_ints("sink has the type float32", sink)
        if T > 0 and B > 0 and (
                qsl.numel() <= B or seq_len.numel() < B or block_table.shape[0] < B
                or (sink is not None and sink.numel() < self.heads)
                or k_cache.numel() < num_blocks * self.block or v_cache.numel() < num_blocks * self.block):
            self._too_small(f"{B} requests, {num_blocks} blocks", qsl, seq_len, block_table, sink, k_cache, v_cache)
        if not (ws.get_device() == qsl.get_device() == seq_len.get_device() == q.get_device() == k_cache.get_device()
                == v_cache.get_device() == block_table.get_device() == out.get_device()
                == (ws if sink is None else sink).get_device()):
            self._apart(ws, qsl, seq_len, q, k_cache, v_cache, block_table, out, sink)
        rc = self.lib.pe_chunk_attention(self.addr, B, T, qsl.data_ptr(), seq_len.data_ptr(), q.data_ptr(),
                                         _row_stride(q, T, self.heads, self.hd), k_cache.data_ptr(), v_cache.data_ptr(),
                                         block_table.data_ptr(), block_table.shape[1], num_blocks,
                                         _addr(sink), out.data_ptr(), _row_stride(out, T, self.heads, self.hd), ws.data_ptr(),
                                         ws.numel(), _stream_handle(stream, ws))
        _check(rc, "pe_chunk_attention")


# ----------------------------------------------------------------------------- COD training indices


def cod_workspace_bytes(B: int, S_max: int, n_depth: int) -> int:
    n = int(load().pe_cod_workspace_bytes(int(B), int(S_max), int(n_depth)))
    if n == 0:
        raise PeError(PE_ERR_ARG, "pe_cod_workspace_bytes")
    return n


def cod_workspace(B: int, S_max: int, n_depth: int, device="cuda"):
    """A device workspace for the two COD calls (torch allocates it 256-byte aligned)."""
    import torch

    return torch.zeros(cod_workspace_bytes(B, S_max, n_depth), dtype=torch.uint8, device=device)


def cod_sample_indices(B, S_max, seq_len, loss_mask, n_depth, retain, max_anchors, u_anchor, u_keep,
                       idx, counts, ws, stream=None):
    """pe_cod_sample_indices on device tensors."""
    rc = load().pe_cod_sample_indices(int(B), int(S_max), _ptr(seq_len), _ptr(loss_mask),
                                      int(n_depth), float(retain), int(max_anchors), _ptr(u_anchor),
                                      _ptr(u_keep), _ptr(idx), _ptr(counts), _ptr(ws),
                                      int(ws.numel()), _stream(stream))
    _check(rc, "pe_cod_sample_indices")


def cod_mask(B, S_max, seq_len, n_depth, idx, counts, mask, q_cap, ld, mask_stride, ws, stream=None):
    """pe_cod_mask on device tensors; mask is a uint8 buffer of B * mask_stride bytes."""
    rc = load().pe_cod_mask(int(B), int(S_max), _ptr(seq_len), int(n_depth), _ptr(idx), _ptr(counts),
                            _ptr(mask), int(q_cap), int(ld), int(mask_stride), _ptr(ws),
                            int(ws.numel()), _stream(stream))
    _check(rc, "pe_cod_mask")
