"""Engram n-gram hash + fp8 row lookup on GB300 (sm_103a): thin Python binding.

The work is done by ``libengram.so`` (CUDA kernels behind the C ABI declared in
``include/engram.h``). This module only marshals torch tensors into pointers,
sizes and the current CUDA stream; it has no compute path of its own and no
fallback: if the library is missing, every call raises.

Functions carry the C names: :func:`engram_state_create`,
:func:`engram_state_destroy`, :func:`engram_cache_reset`,
:func:`engram_state_status`, :func:`engram_hash`, :func:`engram_lookup`,
:func:`engram_hash_lookup` (and their packed forms), the Engram block after
the lookup (:func:`engram_project`, :func:`engram_gate`,
:func:`engram_project_gate`, and with the lookup inside the projection
:func:`engram_lookup_project`, :func:`engram_lookup_project_gate`), and the
row-sharded lookup's two ends (:func:`engram_shard_pack`,
:func:`engram_shard_unpack`). :class:`EngramHash` bundles a state with them.
Training the front end: :func:`engram_embed` (trainable rows) with its gradient
:func:`engram_embed_grad` / :func:`engram_embed_grad_dense`,
:func:`engram_gate_grad`, :func:`engram_grad_norm` and :func:`engram_grad_clip`.

Method: the "DeepSeek V4.1" pages -- blocks/stack-hashes page (the n-gram hash
``forward``, ``Engram.forward``) and engram-first/lookup page
(``ParallelEngramEmbedding.forward``).
"""
from __future__ import annotations

import array
import ctypes
import os

import torch

from ._build import LIB as _LIB_PATH
from ._build import build

__all__ = [
    "EngramError", "EngramHash", "build", "engram_state_create", "engram_state_destroy", "engram_cache_reset",
    "engram_state_status", "engram_hash", "engram_lookup", "engram_hash_lookup", "engram_hash_varlen",
    "engram_hash_lookup_varlen", "engram_gate", "PreparedHashLookup", "engram_strerror", "STATUS_BAD_START",
    "STATUS_BAD_ID", "STATUS_BAD_LENGTH", "STATUS_BAD_ROW", "STATUS_CHECK", "SCALE_F32", "SCALE_BF16", "SCALE_E8M0", "SCALE_E4M3",
    "library_path", "set_l2_fetch_granularity", "engram_project", "engram_project_gate",
    "engram_project_gate_workspace", "engram_device_status", "STATUS_TIMEOUT", "engram_shard_pack",
    "engram_shard_unpack", "shard_part", "sharded_lookup", "dist_exchange", "engram_lookup_project",
    "engram_lookup_project_workspace", "engram_lookup_project_gate", "engram_lookup_project_gate_workspace",
    "engram_embed", "engram_embed_grad", "engram_embed_grad_dense", "engram_embed_grad_workspace", "engram_gate_grad",
    "engram_gate_grad_workspace", "engram_grad_norm", "engram_grad_clip", "engram_grad_norm_workspace",
    "PreparedGradClip",
    "TYPE_F32", "TYPE_BF16", "TYPE_F16", "NORM_L2", "NORM_MAX",
]

OK, ERR_INVALID, ERR_RANGE, ERR_CUDA, ERR_NOMEM, ERR_UNSUPPORTED = 0, -1, -2, -3, -4, -5
STATUS_BAD_START = 1
STATUS_BAD_ID = 2
STATUS_BAD_LENGTH = 4
STATUS_BAD_ROW = 8
STATUS_CHECK = 16  # checked builds only: a kernel skipped an access outside the call's buffers
STATUS_TIMEOUT = 32  # a tensor-core kernel gave up a wait (engram_device_status)
# storage types of the scale tensors (ENGRAM_SCALE_*)
SCALE_F32, SCALE_BF16, SCALE_E8M0, SCALE_E4M3 = 0, 1, 2, 3
_SCALE_BYTES = {SCALE_F32: 4, SCALE_BF16: 2, SCALE_E8M0: 1, SCALE_E4M3: 1}
_SCALE_OF_DTYPE = {torch.float32: SCALE_F32, torch.bfloat16: SCALE_BF16, torch.float8_e4m3fn: SCALE_E4M3}
if hasattr(torch, "float8_e8m0fnu"):
    _SCALE_OF_DTYPE[torch.float8_e8m0fnu] = SCALE_E8M0
# value types of the training operators' tensors (ENGRAM_TYPE_*) and their norms (ENGRAM_NORM_*)
TYPE_F32, TYPE_BF16, TYPE_F16 = 0, 1, 2
_TYPE_OF_DTYPE = {torch.float32: TYPE_F32, torch.bfloat16: TYPE_BF16, torch.float16: TYPE_F16}
NORM_L2, NORM_MAX = 2, 0
MAX_LAYERS = 8


class EngramError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {engram_strerror(code)} ({code})")


class _Layout(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("max_ngram", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("block", ctypes.c_int32), ("max_batch", ctypes.c_int32),
                ("max_seq_len", ctypes.c_int64), ("raw_vocab", ctypes.c_int64), ("dead", ctypes.c_int64),
                ("pad_id", ctypes.c_int64), ("scale_dtype", ctypes.c_int32)]


class _Table(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("S", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("head_dim", ctypes.c_int32), ("block", ctypes.c_int32), ("scale_dtype", ctypes.c_int32)]


class _Tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("out", ctypes.c_void_p), ("rows_used", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("row_len", ctypes.c_int32), ("type", ctypes.c_int32),
                ("out_type", ctypes.c_int32)]


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_lib_handle = None


def library_path() -> str:
    return _LIB_PATH


def _lib():
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"libengram.so is not built ({_LIB_PATH}); run gram_hash_embedding_gb300.build()")
        L = ctypes.CDLL(_LIB_PATH)
        L.engram_state_create.argtypes = [ctypes.POINTER(_Layout), _P, _P, _P, _P, _P, ctypes.POINTER(_P)]
        L.engram_state_destroy.argtypes = [_P]
        L.engram_cache_reset.argtypes = [_P, _P]
        L.engram_state_status.argtypes = [_P, _P, ctypes.POINTER(ctypes.c_uint32), ctypes.c_int]
        L.engram_hash.argtypes = [_P, _P, _P, _P, _P, _I32, _I64, _P, _P]
        L.engram_lookup.argtypes = [_P, _I64, _P, _P, _I64, _I32, _I32, _I32, _P, _P]
        L.engram_hash_lookup.argtypes = [_P, _P, _P, _P, _P, _I32, _I64, _P, _P, _P, _P, _P, _P]
        L.engram_hash_varlen.argtypes = [_P, _P, _P, _P, _P, _P, _I32, _I64, _I64, _P, _P]
        L.engram_hash_lookup_varlen.argtypes = [_P, _P, _P, _P, _P, _P, _I32, _I64, _I64, _P, _P, _P, _P, _P, _P]
        L.engram_state_layout.argtypes = [_P, ctypes.POINTER(_Layout)]
        L.engram_gate.argtypes = [_P, _P, _P, _P, _P, _I64, _I32, _I32, ctypes.c_float, _P, _P]
        L.engram_project.argtypes = [_P, _P, _I64, _I32, _I32, _P, _P]
        L.engram_project_gate_workspace.argtypes = [_I64, _I32, _I32]
        L.engram_project_gate_workspace.restype = ctypes.c_uint64
        L.engram_project_gate.argtypes = [_P, _P, _P, _P, _P, _P, _I64, _I32, _I32, _I32, ctypes.c_float, _P,
                                          ctypes.c_uint64, _P, _P]
        L.engram_device_status.argtypes = [_P, ctypes.POINTER(ctypes.c_uint32), ctypes.c_int]
        L.engram_lookup_project_workspace.argtypes = [_I64, _I32, _I32]
        L.engram_lookup_project_workspace.restype = ctypes.c_uint64
        L.engram_lookup_project.argtypes = [_P, _I64, _I64, _I32, ctypes.POINTER(_Table), _P, _I32, _P,
                                            ctypes.c_uint64, _P, _P]
        L.engram_lookup_project_gate_workspace.argtypes = [_I64, _I32, _I32, _I32, _I32]
        L.engram_lookup_project_gate_workspace.restype = ctypes.c_uint64
        L.engram_lookup_project_gate.argtypes = [_P, _P, _I64, _I64, _I32, ctypes.POINTER(_Table), _P, _P, _P, _P,
                                                 _I32, _I32, ctypes.c_float, _P, ctypes.c_uint64, _P, _P]
        L.engram_shard_pack_workspace.argtypes = [_I64, _I32]
        L.engram_shard_pack_workspace.restype = ctypes.c_uint64
        L.engram_shard_pack.argtypes = [_P, _I64, _I64, _I32, _P, _P, _P, _P, ctypes.c_uint64, _P]
        L.engram_shard_unpack.argtypes = [_P, _P, _I64, _I64, _I32, _P, _P]
        _F = ctypes.c_float
        L.engram_embed.argtypes = [_P, _I64, _I64, _I32, _P, _I64, _I32, _I64, _I32, _F, _P, _I32, _P]
        L.engram_embed_grad_workspace.argtypes = [_I64, _I64, _I32]
        L.engram_embed_grad_workspace.restype = ctypes.c_uint64
        L.engram_embed_grad.argtypes = [_P, _I64, _I64, _I32, _P, _I64, _I32, _I64, _I32, _F, _P, _P, _I32, _P, _P,
                                        ctypes.c_uint64, _P]
        L.engram_embed_grad_dense.argtypes = [_P, _I64, _I64, _I32, _P, _I64, _I32, _I64, _I32, _F, _P, _I64, _I32,
                                              _I32, _P, ctypes.c_uint64, _P]
        L.engram_gate_grad_workspace.argtypes = [_I64, _I32, _I32]
        L.engram_gate_grad_workspace.restype = ctypes.c_uint64
        L.engram_gate_grad.argtypes = [_P, _P, _P, _P, _P, _P, _I64, _I32, _I32, _F, _P, _P, _P, _P, _P,
                                       ctypes.c_uint64, _P]
        L.engram_grad_norm_workspace.argtypes = [_I32]
        L.engram_grad_norm_workspace.restype = ctypes.c_uint64
        L.engram_grad_norm.argtypes = [_P, _I32, _I32, _P, _P, ctypes.c_uint64, _P]
        L.engram_grad_clip.argtypes = [_P, _I32, _I32, _F, _P, _P, ctypes.c_uint64, _P]
        L.engram_strerror.argtypes = [ctypes.c_int]
        L.engram_set_l2_fetch_granularity.argtypes = [_I32, ctypes.POINTER(_I32)]
        L.engram_strerror.restype = ctypes.c_char_p
        for name in ("engram_state_create", "engram_state_destroy", "engram_cache_reset", "engram_state_status",
                     "engram_hash", "engram_lookup", "engram_hash_lookup", "engram_state_layout",
                     "engram_hash_varlen", "engram_hash_lookup_varlen", "engram_gate", "engram_project",
                     "engram_project_gate", "engram_device_status", "engram_shard_pack", "engram_shard_unpack",
                     "engram_lookup_project", "engram_lookup_project_gate", "engram_embed", "engram_embed_grad",
                     "engram_embed_grad_dense", "engram_gate_grad", "engram_grad_norm", "engram_grad_clip"):
            getattr(L, name).restype = ctypes.c_int
        _lib_handle = L
    return _lib_handle


def engram_strerror(code: int) -> str:
    return _lib().engram_strerror(int(code)).decode()


def _check(rc: int, where: str):
    if rc != OK:
        raise EngramError(rc, where)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# the current stream's handle without a Stream object around it (0.4 us a call instead of 2.9)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current_stream_handle() -> int:
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def _launch_stream(stream, temps=()) -> int:
    """The stream handle a call launches on. The wrapper's own temporaries (a start_pos array built
    from an int, outputs it allocates) are made on the current stream; when the caller names another
    stream, that stream first waits for the current one, and each temporary is marked as in use on it
    so the caching allocator does not hand its memory out again before the library's kernel is done."""
    if stream is None:
        return _current_stream_handle()
    cur = torch.cuda.current_stream()
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        if handle == cur.cuda_stream:
            return handle
        stream = torch.cuda.ExternalStream(handle)
    if stream.cuda_stream != cur.cuda_stream:
        stream.wait_stream(cur)
        for t in temps:
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
    return stream.cuda_stream


def _dev(t: torch.Tensor, dtype, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _host_i64(a, n: int, name: str):
    t = torch.as_tensor(a, dtype=torch.int64).reshape(-1).contiguous()
    if t.numel() != n:
        raise ValueError(f"{name}: expected {n} values, got {t.numel()}")
    return t


# ----------------------------------------------------------------------------- C-named functions
def engram_state_create(*, n_layers, max_ngram, n_heads, head_dim, block, max_batch, max_seq_len, token_map,
                        multipliers, primes, offsets, dead=-1, pad_id=2, stream=None, scale_dtype=SCALE_F32) -> int:
    """Create a state; returns the opaque handle (an int). Host arrays: token_map [raw_vocab],
    multipliers [n_layers, max_ngram], primes [n_layers, max_ngram-1, n_heads], offsets [n_layers, C].
    scale_dtype: storage type of the tables' scales (SCALE_*)."""
    tm = torch.as_tensor(token_map, dtype=torch.int64).reshape(-1).contiguous()
    C = (max_ngram - 1) * n_heads
    mu = _host_i64(multipliers, n_layers * max_ngram, "multipliers")
    pr = _host_i64(primes, n_layers * C, "primes")
    of = _host_i64(offsets, n_layers * C, "offsets")
    lay = _Layout(n_layers, max_ngram, n_heads, head_dim, block, max_batch, max_seq_len, tm.numel(), dead, pad_id,
                  int(scale_dtype))
    h = _P()
    _check(_lib().engram_state_create(ctypes.byref(lay), tm.data_ptr(), mu.data_ptr(), pr.data_ptr(), of.data_ptr(),
                                      _stream(stream), ctypes.byref(h)), "engram_state_create")
    return h.value


def engram_state_destroy(state: int) -> None:
    _check(_lib().engram_state_destroy(state), "engram_state_destroy")


def engram_cache_reset(state: int, stream=None) -> None:
    _check(_lib().engram_cache_reset(state, _stream(stream)), "engram_cache_reset")


def engram_state_status(state: int, clear: bool = True, stream=None) -> int:
    v = ctypes.c_uint32(0)
    _check(_lib().engram_state_status(state, _stream(stream), ctypes.byref(v), int(bool(clear))),
           "engram_state_status")
    return v.value


def engram_state_layout(state: int) -> dict:
    lay = _Layout()
    _check(_lib().engram_state_layout(state, ctypes.byref(lay)), "engram_state_layout")
    return {f: getattr(lay, f) for f, _ in _Layout._fields_}


def _scale_dtype_of(S: torch.Tensor, scale_dtype=None) -> int:
    """The storage type of a scale tensor: given explicitly (then S may hold the raw bits in any
    dtype of that width), or read from S's dtype (float32, bfloat16, float8_e8m0fnu, float8_e4m3fn)."""
    if scale_dtype is not None:
        return int(scale_dtype)
    if S.dtype not in _SCALE_OF_DTYPE:
        raise TypeError(f"cannot tell the scale storage type of a {S.dtype} tensor; pass scale_dtype")
    return _SCALE_OF_DTYPE[S.dtype]


def _dev_scales(S: torch.Tensor, scale_dtype: int, name: str = "S") -> int:
    if not isinstance(S, torch.Tensor) or not S.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if scale_dtype not in _SCALE_BYTES or S.element_size() != _SCALE_BYTES[scale_dtype]:
        raise TypeError(f"{name}: {S.dtype} does not hold scales of storage type {scale_dtype}")
    if S.dtype in _SCALE_OF_DTYPE and _SCALE_OF_DTYPE[S.dtype] != scale_dtype:
        raise TypeError(f"{name} is {S.dtype} but the scales are stored as type {scale_dtype}")
    if not S.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return S.data_ptr()


def _start_tensor(start_pos, B: int, device) -> torch.Tensor:
    if isinstance(start_pos, torch.Tensor):
        return start_pos
    return torch.full((B,), int(start_pos), dtype=torch.int32, device=device)


def set_l2_fetch_granularity(nbytes: int) -> int:
    """Set the current device context's L2 fetch granularity limit (0, 32, 64 or 128 bytes; a hint)
    and return the previous value. Process-wide and not stream-ordered: call it at set-up. At 32 a
    random 4-byte scale read costs one 32-byte DRAM sector instead of a 128-byte line."""
    prev = _I32(0)
    _check(_lib().engram_set_l2_fetch_granularity(int(nbytes), ctypes.byref(prev)), "engram_set_l2_fetch_granularity")
    return prev.value


def _size(t, n: int, name: str) -> None:
    """Sizes are checked here, before any pointer reaches the library: the C calls take raw pointers
    and would read or write past a buffer that is too small."""
    if t is not None and isinstance(t, torch.Tensor) and t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} elements, expected {n}")


def _tables(lay: dict, W: list, S: list, out: list | None, n_rows_out: int) -> None:
    """Per-layer tables of a fused call: one W, S (and out) per engram layer of the state, W [rows, D],
    S holding rows * D / block scales, out holding n_rows_out * C rows of D values."""
    n = lay["n_layers"]
    if len(W) != n or len(S) != n or (out is not None and len(out) != n):
        raise ValueError(f"W, S and out need one entry per engram layer ({n})")
    D, C = lay["head_dim"], (lay["max_ngram"] - 1) * lay["n_heads"]
    for l in range(n):
        if W[l].dim() != 2 or W[l].shape[1] != D:
            raise ValueError(f"W[{l}] must be [rows, {D}], got {tuple(W[l].shape)}")
        _size(S[l], W[l].shape[0] * (D // lay["block"]), f"S[{l}]")
        if out is not None:
            _size(out[l], n_rows_out * C * D, f"out[{l}]")


def _rows_ptr(cache_rows):
    return None if cache_rows is None else _dev(cache_rows, torch.int32, "cache_rows")


def engram_hash(state: int, ids: torch.Tensor, start_pos, mask: torch.Tensor | None = None,
                hashes: torch.Tensor | None = None, n_layers: int | None = None, n_cols: int | None = None,
                stream=None, cache_rows: torch.Tensor | None = None) -> torch.Tensor:
    """ids int64 [B, L] (CUDA); start_pos int or int32 [B]; mask bool/uint8 [B, L] or None;
    cache_rows int32 [B] or None (row b uses cache row cache_rows[b], else b).
    Returns (or fills) int64 hash ids [B, L, n_layers, C]."""
    B, L = ids.shape
    lay = engram_state_layout(state)
    NC = lay["n_layers"] * (lay["max_ngram"] - 1) * lay["n_heads"]
    temps = []
    if hashes is None:
        hashes = torch.empty((B, L, lay["n_layers"], (lay["max_ngram"] - 1) * lay["n_heads"]), dtype=torch.int64,
                             device=ids.device)
        temps.append(hashes)
    _size(hashes, B * L * NC, "hashes")
    _size(mask, B * L, "mask")
    _size(cache_rows, B, "cache_rows")
    _size(start_pos, B, "start_pos")
    sp = _start_tensor(start_pos, B, ids.device)
    if sp is not start_pos:
        temps.append(sp)
    m = None if mask is None else _dev(_as_u8(mask), torch.uint8, "mask")
    _check(_lib().engram_hash(state, _dev(ids, torch.int64, "ids"), m, _dev(sp, torch.int32, "start_pos"),
                              _rows_ptr(cache_rows), B, L, _dev(hashes, torch.int64, "hashes"),
                              _launch_stream(stream, temps)), "engram_hash")
    return hashes


def _as_u8(mask: torch.Tensor) -> torch.Tensor:
    return mask.view(torch.uint8) if mask.dtype == torch.bool else mask


def engram_lookup(idx: torch.Tensor, W: torch.Tensor, S: torch.Tensor, block: int, out: torch.Tensor | None = None,
                  stream=None, scale_dtype: int | None = None) -> torch.Tensor:
    """idx int64 [...]; W fp8 (float8_e4m3fn or uint8) [rows, D]; S [rows, D/block] scales (float32,
    bfloat16, float8_e8m0fnu or float8_e4m3fn; or raw bits with scale_dtype). Returns (or fills) bf16 [..., D]."""
    sdt = _scale_dtype_of(S, scale_dtype)
    rows, D = W.shape
    temps = []
    if out is None:
        out = torch.empty(tuple(idx.shape) + (D,), dtype=torch.bfloat16, device=idx.device)
        temps.append(out)
    _size(out, idx.numel() * D, "out")
    if int(block) > 0 and D % int(block) == 0:
        _size(S, rows * (D // int(block)), "S")
    Wu = W.view(torch.uint8)
    _check(_lib().engram_lookup(_dev(idx, torch.int64, "idx"), idx.numel(), _dev(Wu, torch.uint8, "W"),
                                _dev_scales(S, sdt), rows, D, int(block), sdt, _dev(out, torch.bfloat16, "out"),
                                _launch_stream(stream, temps)), "engram_lookup")
    return out


def engram_hash_lookup(state: int, ids: torch.Tensor, start_pos, W: list, S: list, mask: torch.Tensor | None = None,
                       out: list | None = None, hashes: torch.Tensor | None = None, stream=None,
                       cache_rows: torch.Tensor | None = None) -> list:
    """Hash + per-layer lookup in one launch. W/S: per-layer tables. Returns (or fills) the
    per-layer bf16 outputs [B, L, C, D]. An int start_pos costs a small fill kernel before the call;
    in a loop of calls pass a device int32 [B] tensor (or use PreparedHashLookup): consecutive calls of
    this library overlap their launches only when no other kernel or copy runs between them."""
    B, L = ids.shape
    lay = engram_state_layout(state)
    n = len(W)
    D, C = lay["head_dim"], (lay["max_ngram"] - 1) * lay["n_heads"]
    temps = []
    if out is None and len(W) == lay["n_layers"]:
        out = [torch.empty((B, L, C, D), dtype=torch.bfloat16, device=ids.device) for _ in range(n)]
        temps.extend(out)
    _tables(lay, W, S, out, B * L)
    _size(hashes, B * L * lay["n_layers"] * C, "hashes")
    _size(mask, B * L, "mask")
    _size(cache_rows, B, "cache_rows")
    _size(start_pos, B, "start_pos")
    sp = _start_tensor(start_pos, B, ids.device)
    if sp is not start_pos:
        temps.append(sp)
    m = None if mask is None else _dev(_as_u8(mask), torch.uint8, "mask")
    Wp = (_P * n)(*[_dev(w.view(torch.uint8), torch.uint8, "W") for w in W])
    sdt = lay["scale_dtype"]
    Sp = (_P * n)(*[_dev_scales(s, sdt) for s in S])
    Rp = (_I64 * n)(*[w.shape[0] for w in W])
    Op = (_P * n)(*[_dev(o, torch.bfloat16, "out") for o in out])
    hp = None if hashes is None else _dev(hashes, torch.int64, "hashes")
    _check(_lib().engram_hash_lookup(state, _dev(ids, torch.int64, "ids"), m, _dev(sp, torch.int32, "start_pos"),
                                     _rows_ptr(cache_rows), B, L, Wp, Sp, Rp, Op, hp, _launch_stream(stream, temps)),
           "engram_hash_lookup")
    return out


def _max_len(cu_seqlens: torch.Tensor, max_len) -> int:
    if max_len is not None:
        return int(max_len)
    # convenience only: reads the extents back (a device-to-host copy); pass max_len to avoid it
    return int((cu_seqlens[1:] - cu_seqlens[:-1]).max().item()) if cu_seqlens.numel() > 1 else 0


def engram_hash_varlen(state: int, ids: torch.Tensor, cu_seqlens: torch.Tensor, start_pos: torch.Tensor,
                       mask: torch.Tensor | None = None, hashes: torch.Tensor | None = None, max_len: int | None = None,
                       stream=None, cache_rows: torch.Tensor | None = None) -> torch.Tensor:
    """Packed sequences: ids int64 [T]; cu_seqlens int32 [B+1]; start_pos int32 [B]; mask [T] or None.
    Returns (or fills) int64 hash ids [T, n_layers, C]."""
    T = ids.numel()
    B = cu_seqlens.numel() - 1
    lay = engram_state_layout(state)
    temps = []
    if hashes is None:
        hashes = torch.empty((T, lay["n_layers"], (lay["max_ngram"] - 1) * lay["n_heads"]), dtype=torch.int64,
                             device=ids.device)
        temps.append(hashes)
    _size(hashes, T * lay["n_layers"] * (lay["max_ngram"] - 1) * lay["n_heads"], "hashes")
    _size(mask, T, "mask")
    _size(start_pos, B, "start_pos")
    _size(cache_rows, B, "cache_rows")
    m = None if mask is None else _dev(_as_u8(mask), torch.uint8, "mask")
    _check(_lib().engram_hash_varlen(state, _dev(ids, torch.int64, "ids"), m, _dev(cu_seqlens, torch.int32, "cu_seqlens"),
                                     _dev(start_pos, torch.int32, "start_pos"), _rows_ptr(cache_rows), B, T,
                                     _max_len(cu_seqlens, max_len), _dev(hashes, torch.int64, "hashes"),
                                     _launch_stream(stream, temps)), "engram_hash_varlen")
    return hashes


def engram_hash_lookup_varlen(state: int, ids: torch.Tensor, cu_seqlens: torch.Tensor, start_pos: torch.Tensor,
                              W: list, S: list, mask: torch.Tensor | None = None, out: list | None = None,
                              hashes: torch.Tensor | None = None, max_len: int | None = None, stream=None,
                              cache_rows: torch.Tensor | None = None) -> list:
    """Packed sequences, hash + per-layer lookup in one launch. Returns (or fills) per-layer bf16
    outputs [T, C, D]."""
    T = ids.numel()
    B = cu_seqlens.numel() - 1
    lay = engram_state_layout(state)
    n = len(W)
    D, C = lay["head_dim"], (lay["max_ngram"] - 1) * lay["n_heads"]
    temps = []
    if out is None and len(W) == lay["n_layers"]:
        out = [torch.empty((T, C, D), dtype=torch.bfloat16, device=ids.device) for _ in range(n)]
        temps.extend(out)
    _tables(lay, W, S, out, T)
    _size(hashes, T * lay["n_layers"] * C, "hashes")
    _size(mask, T, "mask")
    _size(start_pos, B, "start_pos")
    _size(cache_rows, B, "cache_rows")
    m = None if mask is None else _dev(_as_u8(mask), torch.uint8, "mask")
    Wp = (_P * n)(*[_dev(w.view(torch.uint8), torch.uint8, "W") for w in W])
    sdt = lay["scale_dtype"]
    Sp = (_P * n)(*[_dev_scales(x, sdt) for x in S])
    Rp = (_I64 * n)(*[w.shape[0] for w in W])
    Op = (_P * n)(*[_dev(o, torch.bfloat16, "out") for o in out])
    hp = None if hashes is None else _dev(hashes, torch.int64, "hashes")
    _check(_lib().engram_hash_lookup_varlen(state, _dev(ids, torch.int64, "ids"), m,
                                            _dev(cu_seqlens, torch.int32, "cu_seqlens"),
                                            _dev(start_pos, torch.int32, "start_pos"), _rows_ptr(cache_rows), B, T,
                                            _max_len(cu_seqlens, max_len), Wp, Sp, Rp, Op, hp,
                                            _launch_stream(stream, temps)),
           "engram_hash_lookup_varlen")
    return out


def engram_gate(x: torch.Tensor, kv: torch.Tensor, q_weight: torch.Tensor, k_weight: torch.Tensor,
                mask: torch.Tensor | None = None, eps: float = 1e-20, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """The Engram gate on bf16 tensors: x [T, hc, dim] (or [..., hc, dim]), kv [..., (hc+1)*dim],
    q_weight / k_weight [hc, dim], mask [...] bool or None. Returns (or fills; may be x) bf16 [..., hc, dim]."""
    hc, dim = x.shape[-2], x.shape[-1]
    T = x.numel() // (hc * dim)
    temps = []
    if out is None:
        out = torch.empty_like(x)
        temps.append(out)
    _size(kv, T * (hc + 1) * dim, "kv")
    _size(q_weight, hc * dim, "q_weight")
    _size(k_weight, hc * dim, "k_weight")
    _size(mask, T, "mask")
    _size(out, T * hc * dim, "out")
    m = None if mask is None else _dev(_as_u8(mask), torch.uint8, "mask")
    _check(_lib().engram_gate(_dev(x, torch.bfloat16, "x"), _dev(kv, torch.bfloat16, "kv"),
                              _dev(q_weight, torch.bfloat16, "q_weight"), _dev(k_weight, torch.bfloat16, "k_weight"),
                              m, T, hc, dim, float(eps), _dev(out, torch.bfloat16, "out"),
                              _launch_stream(stream, temps)), "engram_gate")
    return out


def engram_project(emb: torch.Tensor, w: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The `wkv` projection on the tensor cores: emb bf16 [..., K] (T rows), w bf16 [N, K].
    Returns (or fills) bf16 [..., N] = bf16(emb @ w^T), fp32 accumulation."""
    K = emb.shape[-1]
    T = emb.numel() // K if K else 0
    N = w.shape[0]
    if w.dim() != 2 or w.shape[1] != K:
        raise ValueError(f"w must be [N, {K}], got {tuple(w.shape)}")
    temps = []
    if out is None:
        out = torch.empty(tuple(emb.shape[:-1]) + (N,), dtype=torch.bfloat16, device=emb.device)
        temps.append(out)
    _size(out, T * N, "out")
    _check(_lib().engram_project(_dev(emb, torch.bfloat16, "emb"), _dev(w, torch.bfloat16, "w"), T, K, N,
                                 _dev(out, torch.bfloat16, "out"), _launch_stream(stream, temps)), "engram_project")
    return out


def engram_project_gate_workspace(T: int, hc: int, dim: int) -> int:
    """Bytes of workspace engram_project_gate needs (0 for T == 0 or an unsupported hc / dim)."""
    return int(_lib().engram_project_gate_workspace(int(T), int(hc), int(dim)))


def engram_project_gate(x: torch.Tensor, emb: torch.Tensor, wkv: torch.Tensor, q_weight: torch.Tensor,
                        k_weight: torch.Tensor, mask: torch.Tensor | None = None, eps: float = 1e-20,
                        workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """The Engram block after the lookup, fused: the `wkv` projection with the gate's sums in its
    epilogue (keys never written), then the gate. x bf16 [T, hc, dim]; emb bf16 [T, K];
    wkv bf16 [(hc+1)*dim, K]; q_weight / k_weight bf16 [hc, dim]; mask [T] bool or None;
    workspace: a uint8 CUDA tensor of at least engram_project_gate_workspace(T, hc, dim) bytes
    (allocated here when None). Returns (or fills; may be x) bf16 [T, hc, dim]."""
    hc, dim = x.shape[-2], x.shape[-1]
    T = x.numel() // (hc * dim)
    K = emb.shape[-1]
    temps = []
    if out is None:
        out = torch.empty_like(x)
        temps.append(out)
    _size(emb, T * K, "emb")
    _size(wkv, (hc + 1) * dim * K, "wkv")
    _size(q_weight, hc * dim, "q_weight")
    _size(k_weight, hc * dim, "k_weight")
    _size(mask, T, "mask")
    _size(out, T * hc * dim, "out")
    need = engram_project_gate_workspace(T, hc, dim)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
        temps.append(workspace)
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace holds {workspace.numel() * workspace.element_size()} bytes, need {need}")
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    m = None if mask is None else _dev(_as_u8(mask), torch.uint8, "mask")
    _check(_lib().engram_project_gate(_dev(x, torch.bfloat16, "x"), _dev(emb, torch.bfloat16, "emb"),
                                      _dev(wkv, torch.bfloat16, "wkv"), _dev(q_weight, torch.bfloat16, "q_weight"),
                                      _dev(k_weight, torch.bfloat16, "k_weight"), m, T, K, hc, dim, float(eps),
                                      workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                      _dev(out, torch.bfloat16, "out"), _launch_stream(stream, temps)),
           "engram_project_gate")
    return out


def _table(W: torch.Tensor, S: torch.Tensor, block: int, scale_dtype=None) -> _Table:
    sdt = _scale_dtype_of(S, scale_dtype)
    rows, D = W.shape
    if int(block) > 0 and D % int(block) == 0:
        _size(S, rows * (D // int(block)), "S")
    return _Table(_dev(W.view(torch.uint8), torch.uint8, "W"), _dev_scales(S, sdt), rows, D, int(block), sdt)


def _hash_ids(idx: torch.Tensor):
    """idx int64 [T, C] with unit stride along C (e.g. one layer of an engram_hash output viewed as
    [T, n_layers, C][:, layer]): returns (pointer, row stride, T, C)."""
    if not isinstance(idx, torch.Tensor) or not idx.is_cuda or idx.dtype != torch.int64:
        raise TypeError("idx must be an int64 CUDA tensor")
    if idx.dim() != 2 or (idx.shape[1] > 1 and idx.stride(1) != 1):
        raise ValueError(f"idx must be [T, C] with unit stride along C, got shape {tuple(idx.shape)} "
                         f"strides {idx.stride()}")
    T, C = idx.shape
    stride = idx.stride(0) if T > 1 else C
    if stride < C:
        raise ValueError("idx rows overlap")
    return idx.data_ptr(), stride, T, C


def _workspace(workspace, need: int, device, temps: list) -> tuple:
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
        temps.append(workspace)
    nbytes = workspace.numel() * workspace.element_size()
    if nbytes < need:
        raise ValueError(f"workspace holds {nbytes} bytes, need {need}")
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace.data_ptr(), nbytes


def engram_lookup_project_workspace(T: int, n_cols: int, head_dim: int) -> int:
    """Bytes of workspace engram_lookup_project needs."""
    return int(_lib().engram_lookup_project_workspace(int(T), int(n_cols), int(head_dim)))


def engram_lookup_project(idx: torch.Tensor, W: torch.Tensor, S: torch.Tensor, wkv: torch.Tensor, block: int,
                          out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None,
                          scale_dtype: int | None = None) -> torch.Tensor:
    """The lookup and the `wkv` projection in one kernel: idx int64 [T, C] hash ids of one layer (unit
    stride along C); W, S that layer's table (as engram_lookup); wkv bf16 [N, C * head_dim].
    Returns (or fills) bf16 [T, N], bit-identical to engram_project(engram_lookup(idx, W, S), wkv).
    workspace: uint8 CUDA tensor of engram_lookup_project_workspace(T, C, head_dim) bytes (allocated
    here when None)."""
    ptr, stride, T, C = _hash_ids(idx)
    tb = _table(W, S, block, scale_dtype)
    N = wkv.shape[0]
    _size(wkv, N * C * tb.head_dim, "wkv")
    temps = []
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=idx.device)
        temps.append(out)
    _size(out, T * N, "out")
    ws, nbytes = _workspace(workspace, engram_lookup_project_workspace(T, C, tb.head_dim), idx.device, temps)
    _check(_lib().engram_lookup_project(ptr, stride, T, C, ctypes.byref(tb), _dev(wkv, torch.bfloat16, "wkv"), N,
                                        ws, nbytes, _dev(out, torch.bfloat16, "out"), _launch_stream(stream, temps)),
           "engram_lookup_project")
    return out


def engram_lookup_project_gate_workspace(T: int, n_cols: int, head_dim: int, hc: int, dim: int) -> int:
    """Bytes of workspace engram_lookup_project_gate needs (0 for T == 0 or an unsupported shape)."""
    return int(_lib().engram_lookup_project_gate_workspace(int(T), int(n_cols), int(head_dim), int(hc), int(dim)))


def engram_lookup_project_gate(x: torch.Tensor, idx: torch.Tensor, W: torch.Tensor, S: torch.Tensor,
                               wkv: torch.Tensor, q_weight: torch.Tensor, k_weight: torch.Tensor, block: int,
                               mask: torch.Tensor | None = None, eps: float = 1e-20,
                               workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                               stream=None, scale_dtype: int | None = None) -> torch.Tensor:
    """The whole Engram block of one layer from its hash ids: the lookup inside the `wkv` projection,
    the gate's sums in its epilogue, then the gate. x bf16 [T, hc, dim]; idx int64 [T, C]; W, S the
    layer's table; wkv bf16 [(hc+1)*dim, C * head_dim]; q_weight / k_weight bf16 [hc, dim]; mask [T]
    bool or None. Returns (or fills; may be x) bf16 [T, hc, dim], bit-identical to
    engram_project_gate(x, engram_lookup(idx, W, S).view(T, -1), wkv, ...)."""
    ptr, stride, T, C = _hash_ids(idx)
    tb = _table(W, S, block, scale_dtype)
    hc, dim = x.shape[-2], x.shape[-1]
    if x.numel() != T * hc * dim:
        raise ValueError(f"x holds {x.numel()} values, expected T * hc * dim = {T * hc * dim}")
    temps = []
    if out is None:
        out = torch.empty_like(x)
        temps.append(out)
    _size(wkv, (hc + 1) * dim * C * tb.head_dim, "wkv")
    _size(q_weight, hc * dim, "q_weight")
    _size(k_weight, hc * dim, "k_weight")
    _size(mask, T, "mask")
    _size(out, T * hc * dim, "out")
    need = engram_lookup_project_gate_workspace(T, C, tb.head_dim, hc, dim)
    ws, nbytes = _workspace(workspace, need, x.device, temps)
    m = None if mask is None else _dev(_as_u8(mask), torch.uint8, "mask")
    _check(_lib().engram_lookup_project_gate(_dev(x, torch.bfloat16, "x"), ptr, stride, T, C, ctypes.byref(tb),
                                             _dev(wkv, torch.bfloat16, "wkv"),
                                             _dev(q_weight, torch.bfloat16, "q_weight"),
                                             _dev(k_weight, torch.bfloat16, "k_weight"), m, hc, dim, float(eps), ws,
                                             nbytes, _dev(out, torch.bfloat16, "out"), _launch_stream(stream, temps)),
           "engram_lookup_project_gate")
    return out


def engram_device_status(clear: bool = True, stream=None) -> int:
    """Status flags of the kernels that have no state object (STATUS_TIMEOUT) on the current device;
    synchronises the stream."""
    v = ctypes.c_uint32(0)
    _check(_lib().engram_device_status(_stream(stream), ctypes.byref(v), int(bool(clear))), "engram_device_status")
    return v.value


def shard_part(rows: int, world: int) -> int:
    """Rows per rank of a table split over `world` ranks, as `ParallelEngramEmbedding` splits it:
    rank r holds rows [r * part, (r + 1) * part)."""
    return -(-int(rows) // int(world))


def engram_shard_pack(idx: torch.Tensor, rows: int, world: int, stream=None):
    """Group the indices of one lookup by the rank that owns their row. Returns (counts int64
    [world + 1], local_rows int64 [n], positions int64 [n]): bucket r = rank r's rows as rows of its
    shard, then the indices no rank owns; each bucket in index order; positions index into idx."""
    n = idx.numel()
    dev = idx.device
    counts = torch.zeros(world + 1, dtype=torch.int64, device=dev)
    local_rows = torch.empty(n, dtype=torch.int64, device=dev)
    positions = torch.empty(n, dtype=torch.int64, device=dev)
    ws = torch.empty(max(int(_lib().engram_shard_pack_workspace(n, int(world))), 16), dtype=torch.uint8, device=dev)
    _check(_lib().engram_shard_pack(_dev(idx, torch.int64, "idx"), n, int(rows), int(world), counts.data_ptr(),
                                    local_rows.data_ptr(), positions.data_ptr(), ws.data_ptr(), ws.numel(),
                                    _launch_stream(stream, (counts, local_rows, positions, ws))), "engram_shard_pack")
    return counts, local_rows, positions


def engram_shard_unpack(rows: torch.Tensor, positions: torch.Tensor, m: int, head_dim: int,
                        out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[positions[i]] = rows[i] for i < m, +0 rows at positions[m:] (the unowned indices).
    rows bf16 [m, head_dim]; returns (or fills) bf16 [n, head_dim]."""
    n = positions.numel()
    temps = []
    if out is None:
        out = torch.empty((n, head_dim), dtype=torch.bfloat16, device=positions.device)
        temps.append(out)
    _size(out, n * head_dim, "out")
    _size(rows, int(m) * head_dim, "rows")
    rp = _dev(rows, torch.bfloat16, "rows") if int(m) > 0 else None
    _check(_lib().engram_shard_unpack(rp, _dev(positions, torch.int64, "positions"), int(m), n, int(head_dim),
                                      _dev(out, torch.bfloat16, "out"), _launch_stream(stream, temps)),
           "engram_shard_unpack")
    return out


def dist_exchange(group=None):
    """The all-to-all of sharded_lookup over a torch.distributed process group (NCCL on GPUs):
    exchange(t, send_splits, recv_splits) sends t's first send_splits[0] rows to rank 0, the next
    send_splits[1] to rank 1, ..., and returns the rows received, rank 0's first."""
    import torch.distributed as dist

    def exchange(t: torch.Tensor, send_splits, recv_splits) -> torch.Tensor:
        # moved as raw bytes (row = dim 0): any element type travels, on every backend
        rest = tuple(t.shape[1:])
        row_bytes = t.element_size() * int(torch.tensor(rest).prod()) if rest else t.element_size()
        if t.numel() == 0:
            b = torch.empty((t.shape[0], row_bytes), dtype=torch.uint8, device=t.device)
        else:
            b = t.contiguous().view(torch.uint8).reshape(t.shape[0], row_bytes)
        out = torch.empty((int(sum(recv_splits)), row_bytes), dtype=torch.uint8, device=t.device)
        dist.all_to_all_single(out, b, [int(c) for c in recv_splits], [int(c) for c in send_splits], group=group)
        return out.view(t.dtype).reshape((out.shape[0],) + rest)

    return exchange


def sharded_lookup(idx: torch.Tensor, W_shard: torch.Tensor, S_shard: torch.Tensor, rows: int, block: int,
                   world: int, exchange, scale_dtype: int | None = None, ops=None) -> torch.Tensor:
    """One rank's part of a row-sharded lookup (engram-first/lookup page, `ParallelEngramEmbedding`,
    world > 1): this rank holds rows [rank * part, ...) of a table of `rows` rows (W_shard, S_shard:
    its shard_part(rows, world) rows, fewer for the last rank) and looks up its own indices idx [n].
    Instead of looking every index up locally, zeroing foreign rows and all-reducing, each request
    goes to the rank that owns its row and only that row comes back:
      pack by owner -> exchange the counts -> exchange the row ids -> look them up in the shard ->
      exchange the rows back -> unpack (+0 rows where no rank owns the index).
    `exchange(t, send_splits, recv_splits)` is the all-to-all (dist_exchange(group) over NCCL).
    `ops` replaces the device steps (pack, lookup, unpack) with others of the same contract; the
    library's kernels when None. Returns bf16 [n, head_dim], equal to engram_lookup on the whole table."""
    if ops is None:
        ops = (engram_shard_pack,
               lambda r, W, S: engram_lookup(r, W, S, block, scale_dtype=scale_dtype),
               engram_shard_unpack)
    pack, lookup, unpack = ops
    D = W_shard.shape[1]
    n = idx.numel()
    counts, local_rows, positions = pack(idx.reshape(-1), rows, world)
    send = [int(c) for c in counts[:world].cpu()]  # split sizes are host values for the exchange
    m = sum(send)
    recv = [int(c) for c in exchange(counts[:world].reshape(world, 1), [1] * world, [1] * world).reshape(-1).cpu()]
    wanted = exchange(local_rows[:m], send, recv)          # row ids other ranks want from this shard
    found = lookup(wanted, W_shard, S_shard).reshape(-1, D)  # this shard's rows for them
    back = exchange(found, recv, send)                      # this rank's rows, in packed order
    return unpack(back, positions, m, D).reshape(tuple(idx.shape) + (D,))


# ----------------------------------------------------------------------------- training operators
# A training step makes many small calls, so these wrappers check a call's tensors in one pass each and
# allocate no more than the call returns: Python's share of a small call is what it costs. They record nothing for
# torch.autograd; the caller wires the backward pass.
def _float_type(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in _TYPE_OF_DTYPE:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return _TYPE_OF_DTYPE[t.dtype]


def _pointers(specs) -> list:
    """The device pointers of (tensor, dtype, elements, name) specifications, all of them contiguous CUDA
    tensors of that type and size; otherwise the error that _size or _dev raises."""
    try:
        ptrs = [t.data_ptr() for t, dtype, n, _ in specs
                if t.dtype is dtype and t.is_cuda and t.numel() == n and t.is_contiguous()]
    except AttributeError:
        ptrs = ()
    if len(ptrs) != len(specs):
        for t, _, n, name in specs:
            _size(t, n, name)
        for t, dtype, _, name in specs:
            _dev(t, dtype, name)
    return ptrs


def _scratch(workspace, need: int, device) -> tuple:
    """(the tensor to keep alive, pointer, bytes) of a caller's workspace, or of one made for this call."""
    if workspace is not None:
        return (workspace, *_workspace(workspace, need, device, []))
    ws = torch.empty(need if need > 256 else 256, dtype=torch.uint8, device=device)
    return ws, ws.data_ptr(), ws.numel()


def _narrow(size: int, name: str) -> int:
    """A size that the library takes as 32 bits (ctypes would pass on its low bits)."""
    if size > 0x7fffffff:
        raise ValueError(f"{name} is {size}, beyond 2^31 - 1")
    return size


def _embed_ids(idx: torch.Tensor):
    """Row ids of a lookup: int64 [T, C] with unit stride along C, or any contiguous shape (then one
    column): (pointer, row stride, T, C)."""
    if not isinstance(idx, torch.Tensor) or not idx.is_cuda or idx.dtype is not torch.int64:
        raise TypeError("idx must be an int64 CUDA tensor")
    shape = idx.shape
    if len(shape) == 2 and shape[1] > 0:
        _narrow(shape[1], "the ids per token")
        return (idx.data_ptr(), shape[1], shape[0], shape[1]) if idx.is_contiguous() else _hash_ids(idx)
    if not idx.is_contiguous():
        raise ValueError(f"idx must be contiguous, or [T, C] with unit stride along C, got strides {idx.stride()}")
    return idx.data_ptr(), 1, idx.numel(), 1


def _rows_of(t: torch.Tensor, name: str):
    """A table [rows, dim] with unit stride along dim: (pointer, rows, dim, row stride)."""
    shape = t.shape
    if len(shape) != 2 or (shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be [rows, dim] with unit stride along dim, got shape {tuple(shape)} "
                         f"strides {t.stride()}")
    rows, dim = shape
    stride = t.stride(0) if rows > 1 else dim
    if stride < dim:
        raise ValueError(f"{name}: rows overlap")
    return t.data_ptr(), rows, _narrow(dim, f"the width of {name}"), stride


def engram_embed(idx: torch.Tensor, W: torch.Tensor, scale: float = 1.0, out: torch.Tensor | None = None,
                 out_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """Rows of a trainable table: out[..., k] = scale * W[idx[...], k], +0 rows where idx is outside the
    table. idx int64 [T, C] (unit stride along C, e.g. one layer of an engram_hash output) or any
    contiguous shape; W float32, bfloat16 or float16 [rows, dim] (rows may be a stride apart).
    Returns (or fills) idx.shape + (dim,) of out_dtype (W's dtype when neither out nor out_dtype is given)."""
    wt = _float_type(W, "W")
    wp, rows, dim, stride = _rows_of(W, "W")
    ip, istride, T, C = _embed_ids(idx)
    if out is None:
        out = torch.empty((*idx.shape, dim), dtype=out_dtype or W.dtype, device=idx.device)
        ot, op = _float_type(out, "out"), out.data_ptr()
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError(f"out is {out.dtype}, not {out_dtype}")
        _size(out, T * C * dim, "out")
        ot, op = _float_type(out, "out"), _dev(out, out.dtype, "out")
    _check(_lib().engram_embed(ip, istride, T, C, wp, rows, dim, stride, wt, float(scale), op, ot,
                               _launch_stream(stream, (out,))), "engram_embed")
    return out


def engram_embed_grad_workspace(n: int, rows: int, dim: int) -> int:
    """Bytes of workspace that engram_embed_grad and engram_embed_grad_dense need for n ids (never fewer for more ids)."""
    return int(_lib().engram_embed_grad_workspace(int(n), int(rows), int(dim)))


def _row_width(values: torch.Size, ids: torch.Size) -> int:
    """Values per id of a gradient of that shape (0: it does not hold one row for each id). In an empty batch the
    zeros of both shapes cancel, so that its rows are as wide as those of a full one."""
    n, m = ids.numel(), values.numel()
    if n == 0:
        if sum(s == 0 for s in values) != sum(s == 0 for s in ids):
            return 0
        n, m = (torch.Size([s or 1 for s in shape]).numel() for shape in (ids, values))
    return 0 if m % n else m // n


def _embed_dout(dout: torch.Tensor, ids: torch.Size, T: int, C: int):
    """The gradient of a lookup's output: contiguous, or [T, C * dim] / [T, C, dim] whose tokens are a
    stride apart: (pointer, token stride, dim)."""
    dim = _narrow(_row_width(dout.shape, ids), "the width of dout")
    if dim == 0:
        raise ValueError(f"dout {tuple(dout.shape)} does not hold one row for each of {T * C} ids")
    if dout.is_contiguous():
        return dout.data_ptr(), C * dim, dim
    inner = dout.dim() == 2 and dout.shape == (T, C * dim) and (dout.shape[1] == 1 or dout.stride(1) == 1)
    inner = inner or (dout.dim() == 3 and dout.shape == (T, C, dim) and (dim == 1 or dout.stride(2) == 1)
                      and (C == 1 or dout.stride(1) == dim))
    if not inner or (T > 1 and dout.stride(0) < C * dim):
        raise ValueError(f"dout must be contiguous, or [T, C, dim] with only its tokens a stride apart, got shape "
                         f"{tuple(dout.shape)} strides {dout.stride()}")
    return dout.data_ptr(), dout.stride(0) if T > 1 else C * dim, dim


def engram_embed_grad(idx: torch.Tensor, dout: torch.Tensor, rows: int, scale: float = 1.0,
                      grad_dtype: torch.dtype | None = None, grad_rows: torch.Tensor | None = None,
                      grad: torch.Tensor | None = None, count: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None):
    """The gradient of engram_embed for a table of `rows` rows, as the rows that occur. idx as in
    engram_embed; dout: the gradient of its output, float32, bfloat16 or float16 (tokens may be a stride
    apart). Returns (or fills) grad_rows int64 [n] (the distinct ids ascending, then -1), grad [n, dim]
    (grad[u] belongs to grad_rows[u]; float32 unless given; rows from count on are not written) and count
    int64 [1], n = idx.numel(). The sums are fp32 in an order fixed by the ids, their number and dim."""
    ip, istride, T, C = _embed_ids(idx)
    dt = _float_type(dout, "dout")
    dp, dstride, dim = _embed_dout(dout, idx.shape, T, C)
    n, dev = T * C, idx.device
    temps = []
    if grad_rows is None:
        grad_rows = torch.empty(n, dtype=torch.int64, device=dev)
        temps.append(grad_rows)
    if count is None:
        count = torch.empty(1, dtype=torch.int64, device=dev)
        temps.append(count)
    rp, cp = _pointers(((grad_rows, torch.int64, n, "grad_rows"), (count, torch.int64, 1, "count")))
    if grad is None:
        grad = torch.empty((n, dim), dtype=grad_dtype or torch.float32, device=dev)
        temps.append(grad)
    elif grad_dtype is not None and grad.dtype != grad_dtype:
        raise TypeError(f"grad is {grad.dtype}, not {grad_dtype}")
    gt = _float_type(grad, "grad")
    _size(grad, n * dim, "grad")
    keep, ws, nbytes = _scratch(workspace, _lib().engram_embed_grad_workspace(n, int(rows), dim), dev)
    temps.append(keep)
    _check(_lib().engram_embed_grad(ip, istride, T, C, dp, dstride, dt, int(rows), dim, float(scale), rp,
                                    _dev(grad, grad.dtype, "grad"), gt, cp, ws, nbytes,
                                    _launch_stream(stream, temps)), "engram_embed_grad")
    return grad_rows, grad, count


def engram_embed_grad_dense(idx: torch.Tensor, dout: torch.Tensor, grad: torch.Tensor, scale: float = 1.0,
                            accumulate: bool = False, workspace: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """The gradient of engram_embed as a whole table: grad [rows, dim] (float32, bfloat16 or float16; rows
    may be a stride apart) is written, zeros where no id named the row; with accumulate the gradient is
    added to what grad holds. Other arguments as engram_embed_grad. Returns grad."""
    ip, istride, T, C = _embed_ids(idx)
    dt, gt = _float_type(dout, "dout"), _float_type(grad, "grad")
    gp, rows, dim, gstride = _rows_of(grad, "grad")
    dp, dstride, ddim = _embed_dout(dout, idx.shape, T, C)
    if ddim != dim:
        raise ValueError(f"dout has rows of {ddim} values, grad of {dim}")
    keep, ws, nbytes = _scratch(workspace, _lib().engram_embed_grad_workspace(T * C, rows, dim), idx.device)
    _check(_lib().engram_embed_grad_dense(ip, istride, T, C, dp, dstride, dt, rows, dim, float(scale), gp, gstride, gt,
                                          int(bool(accumulate)), ws, nbytes, _launch_stream(stream, (keep,))),
           "engram_embed_grad_dense")
    return grad


def engram_gate_grad_workspace(T: int, hc: int, dim: int) -> int:
    """Bytes of workspace engram_gate_grad needs (0 for T == 0 or an unsupported hc / dim)."""
    return int(_lib().engram_gate_grad_workspace(int(T), int(hc), int(dim)))


def engram_gate_grad(x: torch.Tensor, kv: torch.Tensor, q_weight: torch.Tensor, k_weight: torch.Tensor,
                     dout: torch.Tensor, mask: torch.Tensor | None = None, eps: float = 1e-20,
                     dx: torch.Tensor | None = None, dkv: torch.Tensor | None = None,
                     dq_weight: torch.Tensor | None = None, dk_weight: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None):
    """The gradient of engram_gate (same x, kv, weights, mask, eps) for dout, the gradient of its output.
    Returns (or fills) dx bf16 like x (may be dout), dkv bf16 like kv, and dq_weight, dk_weight float32
    [hc, dim], summed over the tokens in a fixed order. A masked token passes dout through."""
    hc, dim = x.shape[-2:]
    _narrow(max(hc, dim), "hc or dim")
    T = x.numel() // (hc * dim)
    bf, f32, dev = torch.bfloat16, torch.float32, x.device
    temps = []
    if dx is None:
        dx = torch.empty_like(x)
        temps.append(dx)
    if dkv is None:
        dkv = torch.empty_like(kv)
        temps.append(dkv)
    if dq_weight is None:
        dq_weight = torch.empty((hc, dim), dtype=f32, device=dev)
        temps.append(dq_weight)
    if dk_weight is None:
        dk_weight = torch.empty((hc, dim), dtype=f32, device=dev)
        temps.append(dk_weight)
    specs = [(x, bf, T * hc * dim, "x"), (kv, bf, T * (hc + 1) * dim, "kv"), (q_weight, bf, hc * dim, "q_weight"),
             (k_weight, bf, hc * dim, "k_weight"), (dout, bf, T * hc * dim, "dout"), (dx, bf, T * hc * dim, "dx"),
             (dkv, bf, T * (hc + 1) * dim, "dkv"), (dq_weight, f32, hc * dim, "dq_weight"),
             (dk_weight, f32, hc * dim, "dk_weight")]
    if mask is not None:  # a bool tensor's bytes, without a view of it
        specs.append((mask, torch.bool if mask.dtype is torch.bool else torch.uint8, T, "mask"))
    p = _pointers(specs)
    keep, ws, nbytes = _scratch(workspace, _lib().engram_gate_grad_workspace(T, hc, dim), dev)
    temps.append(keep)
    _check(_lib().engram_gate_grad(*p[:5], p[9] if mask is not None else None, T, hc, dim, float(eps), *p[5:9], ws,
                                   nbytes, _launch_stream(stream, temps)), "engram_gate_grad")
    return dx, dkv, dq_weight, dk_weight


def engram_grad_norm_workspace(n_tensors: int) -> int:
    """Bytes of workspace engram_grad_norm and engram_grad_clip need."""
    return int(_lib().engram_grad_norm_workspace(int(n_tensors)))


_NORM_OF = {2: NORM_L2, 2.0: NORM_L2, float("inf"): NORM_MAX}


def _list_part(ts, name: str):
    """(types, pointers, sizes) of a list of tensors; checked in passes over the whole list, since a model
    has hundreds of gradients and a Python call for each check of each would outlast the kernels."""
    try:
        types = [_TYPE_OF_DTYPE[t.dtype] for t in ts]
        fine = all([t.is_cuda for t in ts])
    except (AttributeError, KeyError):
        fine = False
    if not fine:
        for t in ts:
            _float_type(t, name)
    if not all(map(torch.Tensor.is_contiguous, ts)):
        raise ValueError(f"{name} must be contiguous")
    return types, map(torch.Tensor.data_ptr, ts), list(map(torch.Tensor.numel, ts))


def _tensor_list(grads, out, counts):
    """A list's engram_tensor array, packed as 64-bit words: data, out, rows_used, n, row_len | type << 32,
    out_type."""
    n = len(grads)
    if (out is not None and len(out) != n) or (counts is not None and len(counts) != n):
        raise ValueError(f"out and counts need one entry per gradient ({n})")
    words = [0] * (6 * n)
    types, words[0::6], sizes = _list_part(grads, "grads")
    words[3::6] = sizes
    words[4::6] = [t << 32 for t in types]
    if out is not None:
        at = range(n) if all([o is not None for o in out]) else [i for i in range(n) if out[i] is not None]
        types, ptrs, osizes = _list_part(out if len(at) == n else [out[i] for i in at], "out")
        if osizes != (sizes if len(at) == n else [sizes[i] for i in at]):
            i = next(i for i, m in zip(at, osizes) if m != sizes[i])
            raise ValueError(f"out[{i}] has {out[i].numel()} elements, expected {sizes[i]}")
        if len(at) == n:
            words[1::6], words[5::6] = ptrs, types
        else:
            for i, p, t in zip(at, ptrs, types):
                words[6 * i + 1], words[6 * i + 5] = p, t
    if counts is not None:
        for i in [i for i, c in enumerate(counts) if c is not None]:
            c = counts[i]
            _size(c, 1, "counts")
            if grads[i].dim() < 2:
                raise ValueError("a gradient with a count must be [n, dim]")
            words[6 * i + 2] = _dev(c, torch.int64, "counts")
            # no values: any length will do
            words[6 * i + 4] |= _narrow(grads[i].shape[1:].numel() or 1, "the length of rows of a gradient with a count")
    return array.array("q", words), n


def _norm_call(grads, norm_type, counts, norm, workspace, stream, out=None, max_norm=None):
    if norm_type not in _NORM_OF:
        raise ValueError(f"norm_type must be 2 or inf, got {norm_type}")
    grads = list(grads)
    arr, n = _tensor_list(grads, out, counts)
    ap = arr.buffer_info()[0]
    dev = grads[0].device if n else (norm.device if norm is not None else torch.device("cuda"))
    need = _lib().engram_grad_norm_workspace(n)
    if norm is None and workspace is None:  # one allocation: the norm, then the workspace
        keep = torch.empty(64 + (need + 3) // 4, dtype=torch.float32, device=dev)
        norm, p = keep[0], keep.data_ptr()
        args = (p, p + 256, need)
    else:
        if norm is None:
            norm = torch.empty((), dtype=torch.float32, device=dev)
        keep, ws, nbytes = _scratch(workspace, need, dev)
        args = (*_pointers(((norm, torch.float32, 1, "norm"),)), ws, nbytes)
    args += (_launch_stream(stream, (keep, norm)),)
    if max_norm is None:
        _check(_lib().engram_grad_norm(ap, n, _NORM_OF[norm_type], *args), "engram_grad_norm")
    else:
        _check(_lib().engram_grad_clip(ap, n, _NORM_OF[norm_type], float(max_norm), *args), "engram_grad_clip")
    return norm


def engram_grad_norm(grads, norm_type: float = 2.0, counts=None, norm: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The norm over all values of a list of contiguous float32, bfloat16 or float16 CUDA tensors
    (norm_type 2 or inf), as a float32 scalar tensor on the device. counts: None, or per tensor None or an
    int64 [1] CUDA tensor saying how many of its leading rows count (engram_embed_grad's count)."""
    return _norm_call(grads, norm_type, counts, norm, workspace, stream)


def engram_grad_clip(grads, max_norm: float, norm_type: float = 2.0, out=None, counts=None,
                     norm: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Multiply the gradients by min(1, max_norm / (norm + 1e-6)), norm as engram_grad_norm (returned, as
    it was before clipping). In place, or into `out`: per gradient a tensor of the same size in any of the
    three types, or None for in place. Rows past a gradient's count are neither read nor written."""
    if max_norm is None:
        raise TypeError("max_norm must be a number (engram_grad_norm computes the norm alone)")
    return _norm_call(grads, norm_type, counts, norm, workspace, stream, out, max_norm)


class PreparedGradClip:
    """A call of engram_grad_norm (max_norm None) or engram_grad_clip whose tensors are checked and marshalled once,
    for training loops that refill the same gradient buffers: the look at every tensor is most of an
    unprepared call's time where a model has hundreds. Calling it only enqueues the kernels and returns the norm (one
    device scalar, written by every call). It runs on the stream given here, or else on the stream current
    at each call (so it also works inside a CUDA-graph capture). The object keeps the tensors alive.

    Its calls share one norm and one workspace, so they must not overlap on the GPU: a caller who uses several
    streams orders them, and orders the work that fills the gradients before a call on another stream. A
    graph that captured a call needs the object for as long as it is replayed."""

    def __init__(self, grads, max_norm: float | None = None, norm_type: float = 2.0, out=None, counts=None,
                 norm: torch.Tensor | None = None, stream=None):
        if norm_type not in _NORM_OF:
            raise ValueError(f"norm_type must be 2 or inf, got {norm_type}")
        # copies: what the caller does with its lists later frees none of the tensors
        grads = list(grads)
        out, counts = None if out is None else list(out), None if counts is None else list(counts)
        self._arr, n = _tensor_list(grads, out if max_norm is not None else None, counts)
        dev = grads[0].device if n else torch.device("cuda")
        self.norm = torch.empty((), dtype=torch.float32, device=dev) if norm is None else norm
        _size(self.norm, 1, "norm")
        L = _lib()
        ws, wp, nbytes = _scratch(None, L.engram_grad_norm_workspace(n), dev)
        self._keep = (grads, out, counts, ws)
        head = (self._arr.buffer_info()[0], n, _NORM_OF[norm_type])
        tail = (_dev(self.norm, torch.float32, "norm"), wp, nbytes)
        self._fn = L.engram_grad_norm if max_norm is None else L.engram_grad_clip
        self._args = head + tail if max_norm is None else head + (float(max_norm),) + tail
        # The memory made here belongs to the current stream, whose earlier work may still use it
        self._own = (ws,) if norm is not None else (ws, self.norm)
        self._ordered = {_current_stream_handle()}  # streams on which a call may use it
        self._made = None
        if not torch.cuda.is_current_stream_capturing():
            self._made = torch.cuda.Event()
            self._made.record()
        self._given, self._stream = stream, None if stream is None else _stream(stream)

    def _order(self) -> None:
        """The first call on a stream other than the constructing one: what that stream had in hand when this
        object was made ends first, and the memory made here is not handed out again before the calls
        on the new stream have ended. A capture cannot wait for work outside it (torch.cuda.graph waits
        for the device before it captures)."""
        if self._made is None or torch.cuda.is_current_stream_capturing():
            return
        stream = self._given
        if stream is None:
            stream = torch.cuda.current_stream()
        elif not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(self._stream)
        stream.wait_event(self._made)
        for t in self._own:
            t.record_stream(stream)
        self._ordered.add(stream.cuda_stream)

    def __call__(self) -> torch.Tensor:
        handle = self._stream if self._stream is not None else _current_stream_handle()
        if handle not in self._ordered:
            self._order()
        rc = self._fn(*self._args, handle)
        if rc != OK:
            raise EngramError(rc, "prepared engram_grad_clip")
        return self.norm


class PreparedHashLookup:
    """A fused hash + lookup call whose arguments are checked and marshalled once, for serving loops
    that call it many times on the same buffers (refill `ids` / `start_pos` / `mask` in place between
    calls). Calling it only enqueues the kernel, without rebuilding pointer arrays or re-checking
    tensors. It runs on the stream given here, or else on the stream current at each call (so it
    also works inside a CUDA-graph capture)."""

    def __init__(self, state: int, ids: torch.Tensor, start_pos: torch.Tensor, W: list, S: list,
                 out: list, mask: torch.Tensor | None = None, hashes: torch.Tensor | None = None,
                 cu_seqlens: torch.Tensor | None = None, max_len: int | None = None, stream=None,
                 cache_rows: torch.Tensor | None = None):
        n = len(W)
        lay = engram_state_layout(state)
        NC = lay["n_layers"] * (lay["max_ngram"] - 1) * lay["n_heads"]
        if cu_seqlens is None:
            B, T = ids.shape
            rows_out = B * T
        else:
            B, T = cu_seqlens.numel() - 1, ids.numel()
            rows_out = T
        _tables(lay, W, S, out, rows_out)
        _size(hashes, rows_out * NC, "hashes")
        _size(mask, rows_out, "mask")
        _size(start_pos, B, "start_pos")
        _size(cache_rows, B, "cache_rows")
        # the buffers stay alive, whatever the caller does with its lists
        self._keep = (ids, start_pos, list(W), list(S), list(out), mask, hashes, cu_seqlens, cache_rows)
        self._W = (_P * n)(*[_dev(w.view(torch.uint8), torch.uint8, "W") for w in W])
        sdt = lay["scale_dtype"]
        self._S = (_P * n)(*[_dev_scales(x, sdt) for x in S])
        self._R = (_I64 * n)(*[w.shape[0] for w in W])
        self._O = (_P * n)(*[_dev(o, torch.bfloat16, "out") for o in out])
        m = None if mask is None else _dev(_as_u8(mask), torch.uint8, "mask")
        h = None if hashes is None else _dev(hashes, torch.int64, "hashes")
        sp = _dev(start_pos, torch.int32, "start_pos")
        cr = _rows_ptr(cache_rows)
        self._stream = None if stream is None else _stream(stream)
        L = _lib()
        if cu_seqlens is None:
            self._fn = L.engram_hash_lookup
            self._args = (state, _dev(ids, torch.int64, "ids"), m, sp, cr, B, T, self._W, self._S, self._R, self._O, h)
        else:
            self._fn = L.engram_hash_lookup_varlen
            self._args = (state, _dev(ids, torch.int64, "ids"), m, _dev(cu_seqlens, torch.int32, "cu_seqlens"), sp, cr,
                          B, ids.numel(), _max_len(cu_seqlens, max_len), self._W, self._S, self._R, self._O, h)

    def __call__(self) -> None:
        st = self._stream if self._stream is not None else torch.cuda.current_stream().cuda_stream
        rc = self._fn(*self._args, st)
        if rc != OK:
            raise EngramError(rc, "prepared engram_hash_lookup")


# ----------------------------------------------------------------------------- convenience object
class EngramHash:
    """A state plus the calls that use it (the hash module of the model, with its cache)."""

    def __init__(self, *, n_layers, max_ngram, n_heads, head_dim, block, max_batch, max_seq_len, token_map,
                 multipliers, primes, offsets, dead=-1, pad_id=2, scale_dtype=SCALE_F32):
        self.n_layers, self.max_ngram, self.n_heads = n_layers, max_ngram, n_heads
        self.n_cols = (max_ngram - 1) * n_heads
        self.head_dim, self.block, self.scale_dtype = head_dim, block, int(scale_dtype)
        self.handle = engram_state_create(n_layers=n_layers, max_ngram=max_ngram, n_heads=n_heads, head_dim=head_dim,
                                          block=block, max_batch=max_batch, max_seq_len=max_seq_len,
                                          token_map=token_map, multipliers=multipliers, primes=primes,
                                          offsets=offsets, dead=dead, pad_id=pad_id, scale_dtype=scale_dtype)

    def close(self):
        if self.handle:
            engram_state_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def reset(self):
        engram_cache_reset(self.handle)

    def status(self, clear=True) -> int:
        return engram_state_status(self.handle, clear)

    def hash(self, ids, start_pos=0, mask=None, hashes=None, cache_rows=None):
        if hashes is None:
            B, L = ids.shape
            hashes = torch.empty((B, L, self.n_layers, self.n_cols), dtype=torch.int64, device=ids.device)
        return engram_hash(self.handle, ids, start_pos, mask, hashes, cache_rows=cache_rows)

    def hash_lookup(self, ids, W, S, start_pos=0, mask=None, out=None, hashes=None, cache_rows=None):
        if out is None:
            B, L = ids.shape
            out = [torch.empty((B, L, self.n_cols, self.head_dim), dtype=torch.bfloat16, device=ids.device)
                   for _ in range(len(W))]
        return engram_hash_lookup(self.handle, ids, start_pos, W, S, mask, out, hashes, cache_rows=cache_rows)

    def hash_varlen(self, ids, cu_seqlens, start_pos, mask=None, hashes=None, max_len=None, cache_rows=None):
        return engram_hash_varlen(self.handle, ids, cu_seqlens, start_pos, mask, hashes, max_len,
                                  cache_rows=cache_rows)

    def hash_lookup_varlen(self, ids, cu_seqlens, start_pos, W, S, mask=None, out=None, hashes=None, max_len=None,
                           cache_rows=None):
        return engram_hash_lookup_varlen(self.handle, ids, cu_seqlens, start_pos, W, S, mask, out, hashes, max_len,
                                         cache_rows=cache_rows)

    def prepare_hash_lookup(self, ids, start_pos, W, S, out, mask=None, hashes=None, cu_seqlens=None, max_len=None,
                            stream=None, cache_rows=None) -> PreparedHashLookup:
        return PreparedHashLookup(self.handle, ids, start_pos, W, S, out, mask, hashes, cu_seqlens, max_len, stream,
                                  cache_rows)

    def lookup(self, idx, W, S, out=None):
        return engram_lookup(idx, W, S, self.block, out, scale_dtype=self.scale_dtype)
