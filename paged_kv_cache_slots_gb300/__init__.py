"""Paged KV cache and decode attention for one GB300 GPU (sm_103a).

Thin ctypes binding of libpkv.so (include/pkv.h): it only turns torch
tensors into pointers and sizes and raises on a non-zero status.  Every step
of the path runs in the library's CUDA kernels; there is no fallback.  If
the library is missing it is built in-tree with nvcc, and if that fails the
import of the first call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple

import torch

from . import build as _build

__all__ = [
    "KVError", "KVPool", "Rope", "BlockAllocator", "PrefixCachePool", "kv_pool_bytes", "slot_mapping", "workspace_bytes",
    "paged_decode_attention", "device_status", "library_path", "load_library", "workspace_init",
    "make_workspace", "paged_decode_append_attention", "paged_prefill_attention", "slot_mapping_varlen",
    "paged_shared_prefix_attention", "shared_prefix_workspace_bytes", "make_shared_prefix_workspace",
    "paged_window_decode_attention", "paged_window_prefill_attention", "window_prefill_workspace_bytes",
    "make_window_prefill_workspace", "StepTables", "make_step_tables", "make_free_queue", "extend_tables", "release_tables",
]

KV_F32, KV_F16, KV_BF16, KV_FP8_E4M3 = 0, 1, 2, 3
DTYPE_CODE = {torch.float32: KV_F32, torch.float16: KV_F16, torch.bfloat16: KV_BF16,
              torch.float8_e4m3fn: KV_FP8_E4M3}
CODE_DTYPE = {v: k for k, v in DTYPE_CODE.items()}
DTYPE_NAMES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
               "e4m3": torch.float8_e4m3fn, "fp8": torch.float8_e4m3fn}
FP8 = torch.float8_e4m3fn
_ROW_DTYPES = (torch.float32, torch.float16, torch.bfloat16)
KERNELS = {"auto": 0, "ffma": 1, "mma": 2}
FLAG_BAD_BLOCK_ID, FLAG_BAD_SLOT, FLAG_BAD_CONTEXT, FLAG_TIMEOUT = 0x1, 0x2, 0x4, 0x8
FLAG_BAD_GROUP, FLAG_BAD_QUEUE = 0x20, 0x40

_lock = threading.Lock()
_lib = None


class KVError(RuntimeError):
    """A libpkv call returned a non-zero kv_status_t."""

    def __init__(self, status: int, name: str, detail: str):
        super().__init__(f"{name}: {detail}" if detail else name)
        self.status = status
        self.name = name


class _PoolConfig(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int), ("num_blocks", ctypes.c_int),
                ("block_size", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int), ("device", ctypes.c_int)]


class _RopeConfig(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("num_axes", ctypes.c_int),
                ("amplitude", ctypes.c_float), ("inv_freq", ctypes.POINTER(ctypes.c_double)),
                ("axis", ctypes.POINTER(ctypes.c_int32))]


class _DecodeOptions(ctypes.Structure):
    _fields_ = [("num_ctas", ctypes.c_int), ("ctas_per_sm", ctypes.c_int),
                ("consumer_warps", ctypes.c_int), ("kernel", ctypes.c_int),
                ("heads_per_stage", ctypes.c_int), ("separate_reduce", ctypes.c_int),
                ("no_pdl", ctypes.c_int), ("early_reads", ctypes.c_int), ("test_stall", ctypes.c_int)]


def library_path() -> str:
    return _build.LIBRARY


def _declare(lib):
    P, I, I64, U32P, SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                           ctypes.POINTER(ctypes.c_uint32), ctypes.c_size_t)
    sig = {
        "kv_status_string": (ctypes.c_char_p, [I]),
        "kv_last_error": (ctypes.c_char_p, []),
        "kv_pool_bytes": (SZ, [ctypes.POINTER(_PoolConfig)]),
        "kv_pool_create": (I, [ctypes.POINTER(_PoolConfig), P, SZ, ctypes.POINTER(P)]),
        "kv_pool_destroy": (None, [P]),
        "kv_pool_layer": (I, [P, I, ctypes.POINTER(P), ctypes.POINTER(P)]),
        "kv_pool_config": (I, [P, ctypes.POINTER(_PoolConfig)]),
        "kv_slot_mapping": (I, [P, I, P, I, I, I, P, P]),
        "kv_append": (I, [P, I, P, I, P, P, P, P]),
        "kv_rope_create": (I, [ctypes.POINTER(_RopeConfig), ctypes.POINTER(P)]),
        "kv_rope_destroy": (None, [P]),
        "kv_append_rope": (I, [P, I, P, P, I, P, I64, P, I64, I, P, P, I64, P, I64, P, I64, I, ctypes.c_float,
                               ctypes.c_float, P]),
        "kv_append_norm_rope": (I, [P, I, P, P, I, P, I64, P, I64, I, P, P, I64, P, I64, P, I64, I, P, I64, P, I64, I,
                                    ctypes.c_float, ctypes.c_float, ctypes.c_float, P]),
        "kv_tables_extend": (I, [P, I, P, P, I, I, I, P, P, I, P, P, P, P, P, P, P]),
        "kv_tables_release": (I, [P, I, P, I, I, I, P, I, I, P, P, P]),
        "paged_decode_workspace_bytes": (I, [I, I, I, I, I, ctypes.POINTER(_DecodeOptions),
                                             ctypes.POINTER(SZ)]),
        "paged_decode_attention": (I, [P, P, P, I, P, I, P, I, I, I, I, I, I, ctypes.c_float, P,
                                       I, P, SZ, ctypes.POINTER(_DecodeOptions), P]),
        "paged_decode_workspace_init": (I, [P, SZ, I, I, P]),
        "paged_decode_append_attention": (I, [P, P, P, P, P, P, I, P, I, P, I, I, I, I, I, I,
                                              ctypes.c_float, P, I, P, P, SZ,
                                              ctypes.POINTER(_DecodeOptions), P]),
        "paged_decode_attention_static": (I, [P, P, P, I, P, I, P, I, I, I, I, I, I, ctypes.c_float,
                                              P, I, ctypes.POINTER(_DecodeOptions), P]),
        "kv_device_status": (I, [I, P, U32P]),
        "kv_allocator_create": (I, [I, I, I, ctypes.POINTER(P)]),
        "kv_allocator_destroy": (None, [P]),
        "kv_allocator_extend": (I, [P, I64, I]),
        "kv_seq_extend": (I, [P, I, I, P, I, ctypes.POINTER(I), P]),
        "kv_seq_free": (I, [P, I]),
        "kv_allocator_release": (I, [P, I64]),
        "kv_allocator_table": (I, [P, I64, ctypes.POINTER(ctypes.c_int32), I,
                                   ctypes.POINTER(I), ctypes.POINTER(I)]),
        "kv_allocator_slot": (I, [P, I64, I, ctypes.POINTER(ctypes.c_int32)]),
        "kv_allocator_free_queue": (I, [P, ctypes.POINTER(ctypes.c_int32), I, ctypes.POINTER(I)]),
        "kv_append_fp8": (I, [P, I, P, I, P, P, I, P, ctypes.c_float, ctypes.c_float, P]),
        "paged_decode_attention_fp8": (I, [P, I, P, P, ctypes.c_float, ctypes.c_float, I, P, I, P, I,
                                           I, I, I, I, ctypes.c_float, P, I, P, SZ,
                                           ctypes.POINTER(_DecodeOptions), P]),
        "paged_decode_append_attention_fp8": (I, [P, P, P, P, I, P, P, ctypes.c_float, ctypes.c_float,
                                                  I, P, I, P, I, I, I, I, I, ctypes.c_float, P, I, P,
                                                  P, SZ, ctypes.POINTER(_DecodeOptions), P]),
        "paged_prefill_workspace_bytes": (SZ, [I]),
        "kv_slot_mapping_varlen": (I, [P, I, P, P, I, I, I, I, P, P]),
        "paged_prefill_attention": (I, [P, P, P, I, P, I, P, P, I, I, I, I, I, I, I, ctypes.c_float, P, I,
                                        P, SZ, P]),
        "paged_prefill_attention_fp8": (I, [P, I, P, P, ctypes.c_float, ctypes.c_float, I, P, I, P, P, I, I, I,
                                            I, I, I, ctypes.c_float, P, I, P, SZ, P]),
        "paged_shared_prefix_workspace_bytes": (I, [I, I, I, I, I, I, ctypes.POINTER(SZ)]),
        "paged_shared_prefix_attention": (I, [P, P, P, I, P, I, P, I, P, P, I, I, I, I, I, I, ctypes.c_float, P, I, P,
                                              SZ, P]),
        "paged_shared_prefix_attention_fp8": (I, [P, I, P, P, ctypes.c_float, ctypes.c_float, I, P, I, P, I, P, P, I,
                                                  I, I, I, I, ctypes.c_float, P, I, P, SZ, P]),
        "paged_window_decode_attention": (I, [P, P, P, I, P, I, P, I, I, I, I, I, I, ctypes.c_float, I, I, P, I, P, SZ,
                                              ctypes.POINTER(_DecodeOptions), P]),
        "paged_window_decode_attention_fp8": (I, [P, I, P, P, ctypes.c_float, ctypes.c_float, I, P, I, P, I, I, I, I, I,
                                                  ctypes.c_float, I, I, P, I, P, SZ, ctypes.POINTER(_DecodeOptions), P]),
        "paged_window_prefill_workspace_bytes": (I, [I, I, I, I, I, I, ctypes.POINTER(SZ)]),
        "paged_window_prefill_attention": (I, [P, P, P, I, P, I, P, P, I, I, I, I, I, I, I, ctypes.c_float, I, I, P, I, P,
                                               SZ, P]),
        "paged_window_prefill_attention_fp8": (I, [P, I, P, P, ctypes.c_float, ctypes.c_float, I, P, I, P, P, I, I, I, I,
                                                   I, I, ctypes.c_float, I, I, P, I, P, SZ, P]),
        "kv_swap_bytes": (SZ, [P, I]),
        "kv_swap_out": (I, [P, P, I, P, SZ, P]),
        "kv_swap_in": (I, [P, P, I, P, SZ, P]),
        "kv_prefix_pool_create": (I, [I, I, ctypes.POINTER(P)]),
        "kv_prefix_pool_destroy": (None, [P]),
        "kv_prefix_pool_allocate": (I, [P, ctypes.POINTER(ctypes.c_int32), I,
                                        ctypes.POINTER(ctypes.c_int32), I, ctypes.POINTER(I),
                                        ctypes.POINTER(I), ctypes.POINTER(ctypes.c_int32), I,
                                        ctypes.POINTER(I)]),
        "kv_prefix_pool_free": (I, [P, ctypes.POINTER(ctypes.c_int32), I]),
        "kv_prefix_pool_free_queue": (I, [P, ctypes.POINTER(ctypes.c_int32), I, ctypes.POINTER(I)]),
        "kv_prefix_pool_cache_size": (I, [P, ctypes.POINTER(I), ctypes.POINTER(I)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def load_library(path: str | None = None):
    """Load libpkv.so (building it in-tree first if it is missing or stale)."""
    global _lib
    with _lock:
        if path is None and _lib is not None:
            return _lib
        lib = _declare(ctypes.CDLL(path or _build.build()))
        if path is None:
            _lib = lib
        return lib


def _check(status: int, lib=None):
    if status != 0:
        lib = lib or load_library()
        raise KVError(status, lib.kv_status_string(status).decode(), lib.kv_last_error().decode())


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream(t: torch.Tensor, stream) -> int:
    if stream is None:
        index = t.get_device()
        if _raw_stream is not None and index >= 0:
            return _raw_stream(index)
        stream = torch.cuda.current_stream(t.device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _made(t: torch.Tensor, stream, make) -> torch.Tensor:
    """make(), a tensor of a call's own on t's device, on the stream that the call is given.

    On a stream other than torch's current one this puts the fill or copy that make() does, and whatever held the
    memory before, in order with the call's kernels.  The current stream, where the caller may read what is returned,
    has to reach the point of its release too before the memory is used again."""
    if stream is None:
        return make()
    handle, current = _stream(t, stream), torch.cuda.current_stream(t.device)
    if handle == current.cuda_stream:
        return make()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle, device=t.device) if handle else torch.cuda.default_stream(t.device)
    with torch.cuda.stream(stream):
        made = make()
    made.record_stream(current)
    return made


def _call_on(t: torch.Tensor, lib, fn, *args):
    """Call a library entry point with t's device current: the library takes
    the SM count, the status word and the static scratch of the current
    device, and the stream passed is t's."""
    index = t.get_device()
    # (A host tensor has index -1.  The library does not see what an address is: tensors are the caller's to check.)
    if index < 0 or index == torch.cuda.current_device():
        status = fn(*args)
        if status:
            _check(status, lib)
        return
    with torch.cuda.device(index):
        _check(fn(*args), lib)


def _call(index: int, lib, fn, *args):
    """_call_on for an index that is known to be a GPU's."""
    if index == _current_device():
        status = fn(*args)
        if status:
            _check(status, lib)
        return
    with torch.cuda.device(index):
        _check(fn(*args), lib)


def _need(cond: bool, msg: str):
    if not cond:
        raise ValueError(msg)


def kv_pool_bytes(num_layers, num_blocks, block_size, num_kv_heads, head_dim, dtype) -> int:
    cfg = _PoolConfig(num_layers, num_blocks, block_size, num_kv_heads, head_dim,
                      DTYPE_CODE[dtype], 0)
    return int(load_library().kv_pool_bytes(ctypes.byref(cfg)))


class KVPool:
    """A pool of KV blocks for every layer, in one device buffer owned by torch.

    Layout per layer: K [num_blocks, num_kv_heads, block_size, head_dim], then V.
    """

    def __init__(self, num_layers, num_blocks, block_size, num_kv_heads, head_dim, dtype,
                 device=None, buffer: torch.Tensor | None = None):
        lib = load_library()
        device = torch.device(device if device is not None else "cuda")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        if isinstance(dtype, str):
            _need(dtype in DTYPE_NAMES, f"dtype must be one of {sorted(DTYPE_NAMES)}")
            dtype = DTYPE_NAMES[dtype]
        self.cfg = _PoolConfig(num_layers, num_blocks, block_size, num_kv_heads, head_dim,
                               DTYPE_CODE[dtype], device.index)
        self.nbytes = int(lib.kv_pool_bytes(ctypes.byref(self.cfg)))
        _need(self.nbytes > 0, "invalid pool configuration")
        if buffer is None:
            buffer = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        _need(buffer.dtype == torch.uint8 and buffer.is_contiguous() and buffer.numel() >= self.nbytes,
              "buffer must be a contiguous uint8 tensor of at least kv_pool_bytes bytes")
        self.buffer = buffer
        self.dtype = dtype
        self.device = device
        self.shape = (num_blocks, num_kv_heads, block_size, head_dim)
        self._kv_heads, self._head_dim, self._index = num_kv_heads, head_dim, device.index
        handle = ctypes.c_void_p()
        _check(lib.kv_pool_create(ctypes.byref(self.cfg), _ptr(buffer), buffer.numel(),
                                  ctypes.byref(handle)), lib)
        self._handle = handle
        self._lib = lib

    @property
    def num_layers(self):
        return self.cfg.num_layers

    def seq_extend(self, seq_id: int, new_tokens: int, ctx_len: int, max_blocks: int):
        """kv_seq_extend: grow sequence seq_id (currently ctx_len tokens) by
        new_tokens on the pool's own allocator.  Returns (table row [max_blocks]
        padded with -1, new length, slots of the new tokens), host int32 tensors."""
        row = torch.full((max_blocks,), -1, dtype=torch.int32)
        slots = torch.zeros(max(new_tokens, 1), dtype=torch.int32)
        n = ctypes.c_int(ctx_len)
        _check(self._lib.kv_seq_extend(self._handle, seq_id, new_tokens, ctypes.c_void_p(row.data_ptr()),
                                       max_blocks, ctypes.byref(n), ctypes.c_void_p(slots.data_ptr())),
               self._lib)
        return row, n.value, slots[:new_tokens]

    def seq_free(self, seq_id: int):
        """kv_seq_free: return the sequence's blocks to the pool's free queue."""
        _check(self._lib.kv_seq_free(self._handle, seq_id), self._lib)

    def layer(self, layer: int):
        """(K, V) torch views of one layer, addresses taken from kv_pool_layer."""
        k = ctypes.c_void_p()
        v = ctypes.c_void_p()
        _check(self._lib.kv_pool_layer(self._handle, layer, ctypes.byref(k), ctypes.byref(v)),
               self._lib)
        base = self.buffer.data_ptr()
        n = self.nbytes // (2 * self.cfg.num_layers)
        views = []
        for addr in (k.value, v.value):
            off = addr - base
            views.append(self.buffer[off:off + n].view(self.dtype).view(self.shape))
        return views[0], views[1]

    def swap_bytes(self, num_blocks: int) -> int:
        """Bytes of host memory that num_blocks swapped blocks occupy."""
        return int(self._lib.kv_swap_bytes(self._handle, num_blocks))

    def _swap_ids(self, block_ids) -> torch.Tensor:
        if not isinstance(block_ids, torch.Tensor):
            block_ids = torch.tensor(list(block_ids), dtype=torch.int32)
        _need(block_ids.dtype == torch.int32 and block_ids.dim() == 1, "block_ids must be int32 [n]")
        return block_ids.to(self.device).contiguous()

    def swap_out(self, block_ids, host: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Copy the listed blocks (all layers, K and V) into page-locked host memory.

        Returns the host buffer (uint8, kv_swap_bytes(n) bytes; a new pinned
        tensor unless `host` is given).  Asynchronous on `stream`."""
        ids = _made(self.buffer, stream, lambda: self._swap_ids(block_ids))
        n = ids.numel()
        need = self.swap_bytes(n)
        if host is None:
            host = torch.empty(max(need, 16), dtype=torch.uint8, pin_memory=True)
        _need(host.dtype == torch.uint8 and host.is_contiguous() and host.numel() >= need,
              "host must be a contiguous uint8 tensor of at least swap_bytes(n) bytes")
        _check(self._lib.kv_swap_out(self._handle, _ptr(ids), n, _ptr(host), host.numel(),
                                     _stream(self.buffer, stream)), self._lib)
        self._swap_keep = ids  # alive until the next swap call on this pool
        return host

    def swap_in(self, block_ids, host: torch.Tensor, stream=None):
        """Copy swapped records from host memory into the listed blocks."""
        ids = _made(self.buffer, stream, lambda: self._swap_ids(block_ids))
        n = ids.numel()
        _need(host.dtype == torch.uint8 and host.is_contiguous() and host.numel() >= self.swap_bytes(n),
              "host must be a contiguous uint8 tensor of at least swap_bytes(n) bytes")
        _check(self._lib.kv_swap_in(self._handle, _ptr(ids), n, _ptr(host), host.numel(),
                                    _stream(self.buffer, stream)), self._lib)
        self._swap_keep = ids

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
               seq_ids: torch.Tensor | None = None, stream=None, k_scale=None, v_scale=None):
        """Write k, v ([n, Hkv, D]) into this layer at slot_mapping ([n] int32).

        An E4M3 pool quantizes on the way and needs this layer's k_scale and
        v_scale; k and v are then f32, f16 or bf16."""
        n = slot_mapping.shape[0]
        if self.dtype == FP8:
            _need(k_scale is not None and v_scale is not None, "an E4M3 pool needs k_scale and v_scale")
            _need(k.dtype == v.dtype and k.dtype in (torch.float32, torch.float16, torch.bfloat16),
                  "k/v must be f32, f16 or bf16")
            _need(tuple(k.shape) == (n, self.cfg.num_kv_heads, self.cfg.head_dim) and k.shape == v.shape,
                  "k and v must be [n_tokens, num_kv_heads, head_dim]")
            _need(k.is_contiguous() and v.is_contiguous() and slot_mapping.is_contiguous(), "contiguous inputs")
            _need(slot_mapping.dtype == torch.int32, "slot_mapping must be int32")
            _need(seq_ids is None or (seq_ids.dtype == torch.int32 and seq_ids.shape[0] == n),
                  "seq_ids must be int32 [n_tokens]")
            _check(self._lib.kv_append_fp8(self._handle, layer, _ptr(seq_ids), n, _ptr(k), _ptr(v),
                                           DTYPE_CODE[k.dtype], _ptr(slot_mapping), float(k_scale),
                                           float(v_scale), _stream(k, stream)), self._lib)
            return
        _need(k.dtype == self.dtype and v.dtype == self.dtype, "k/v dtype must match the pool")
        _need(tuple(k.shape) == (n, self.cfg.num_kv_heads, self.cfg.head_dim) and k.shape == v.shape,
              "k and v must be [n_tokens, num_kv_heads, head_dim]")
        _need(k.is_contiguous() and v.is_contiguous() and slot_mapping.is_contiguous(), "contiguous inputs")
        _need(slot_mapping.dtype == torch.int32, "slot_mapping must be int32")
        _need(seq_ids is None or (seq_ids.dtype == torch.int32 and seq_ids.shape[0] == n),
              "seq_ids must be int32 [n_tokens]")
        _check(self._lib.kv_append(self._handle, layer, _ptr(seq_ids), n, _ptr(k), _ptr(v),
                                   _ptr(slot_mapping), _stream(k, stream)), self._lib)

    def append_rope(self, layer: int, k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                    positions: torch.Tensor, rope: "Rope", q: torch.Tensor | None = None,
                    q_out: torch.Tensor | None = None, seq_ids: torch.Tensor | None = None, stream=None,
                    k_scale=None, v_scale=None) -> torch.Tensor | None:
        """append() with the K rows rotated by `rope` at each token's position, and the query
        rows q ([n, Hq, D]) rotated into q_out (a new tensor unless given; may be q itself).

        k, v and q may be slices of a packed projection (any stride between tokens, heads
        contiguous).  positions: int32 [n], or [axes, n] for a rope with several axes (text tokens:
        one row expanded to all axes).  A negative slot writes no K and V; a token with a negative
        seq_id writes nothing, q_out neither (a new q_out holds zeros there).  Returns q_out, or None
        without q.

        Everything runs on `stream` (torch's current one unless given), a new q_out's zeros and the
        copy of positions that are not contiguous too: order the inputs before it, and what reads
        the outputs behind it."""
        head, tail, q_out, _keep = self._rope_call(k, v, slot_mapping, positions, rope, q, q_out, seq_ids, stream, k_scale, v_scale)
        status = self._lib.kv_append_rope(self._handle, layer, rope._handle, *head, *tail)
        if status:
            _check(status, self._lib)
        return q_out

    def append_norm_rope(self, layer: int, k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                         positions: torch.Tensor, rope: "Rope", k_weight: torch.Tensor | None, q: torch.Tensor | None = None,
                         q_weight: torch.Tensor | None = None, eps: float = 1e-6, q_out: torch.Tensor | None = None,
                         seq_ids: torch.Tensor | None = None, stream=None, k_scale=None, v_scale=None) -> torch.Tensor | None:
        """append_rope() with each head's K and q rows normalised first: x / sqrt(mean(x^2) + eps) times the
        weights, then rotated, rounded once.

        k_weight, q_weight: [head_dim], or [heads, head_dim] with a row for each head, of k's dtype or float32
        (both the same; None: all 1).  The other arguments and the result are append_rope's."""
        head, tail, q_out, _keep = self._rope_call(k, v, slot_mapping, positions, rope, q, q_out, seq_ids, stream, k_scale, v_scale)
        wt = k.dtype if k_weight is None and q_weight is None else (q_weight if k_weight is None else k_weight).dtype
        if wt != k.dtype:
            _need(wt == torch.float32, "weights must be of k's dtype or float32")
        kw, ks = self._weights(k_weight, self._kv_heads, wt)
        if q is not None:
            qw, qs = self._weights(q_weight, q.shape[1], wt)
        else:
            _need(q_weight is None, "q_weight without q")
            qw, qs = None, 0
        status = self._lib.kv_append_norm_rope(self._handle, layer, rope._handle, *head, qw, qs, kw, ks, DTYPE_CODE[wt], float(eps), *tail)
        if status:
            _check(status, self._lib)
        return q_out

    def _weights(self, w, heads, dtype):
        """Address and stride of a head's norm weights."""
        if w is None:
            return None, 0
        D = self._head_dim
        flat = w.dim() == 1
        _need(w.dtype == dtype and w.shape == ((D,) if flat else (heads, D)) and w.stride(-1) == 1 and w.get_device() == self._index,
              "weights must be [head_dim] or [heads, head_dim], both of one dtype, contiguous along head_dim, on the pool's device")
        if flat:
            return w.data_ptr(), 0
        step = w.stride(0)
        _need(heads == 1 or step == 0 or step >= D, "rows of weights overlap")
        return w.data_ptr(), step

    def _rope_call(self, k, v, slot_mapping, positions, rope, q, q_out, seq_ids, stream, k_scale, v_scale):
        """Checks of append_rope and append_norm_rope; their arguments from seq_ids to num_q_heads, those from
        k_scale on, q_out, and positions (a copy made here has to live until the call)."""
        n, dt, D, index = slot_mapping.shape[0], k.dtype, self._head_dim, self._index
        ks, vs = k.stride(), v.stride()
        flat = rope.num_axes == 1
        # The usual call in one expression; _check_append_rope says what is wrong with any other.
        if not (k.shape == v.shape == (n, self._kv_heads, D) and ks[1:] == vs[1:] == (D, 1) and v.dtype == dt
                and slot_mapping.dtype == positions.dtype == torch.int32 and slot_mapping.is_contiguous()
                and positions.shape == ((n,) if flat else (rope.num_axes, n)) and positions.stride(-1) == 1
                and (dt == self.dtype and dt != FP8 or self.dtype == FP8 and dt in _ROW_DTYPES
                     and k_scale is not None and v_scale is not None)
                and k.get_device() == v.get_device() == slot_mapping.get_device() == positions.get_device() == index):
            positions = self._check_append_rope(k, v, slot_mapping, positions, rope, k_scale, v_scale, stream)
            ks, vs = k.stride(), v.stride()
        ids = None
        if seq_ids is not None:
            _need(seq_ids.dtype == torch.int32 and seq_ids.shape == (n,) and seq_ids.is_contiguous()
                  and seq_ids.get_device() == index, "seq_ids must be int32 [n_tokens] on the pool's device")
            ids = seq_ids.data_ptr()
        if q is not None:
            if q_out is None:
                make = torch.empty if seq_ids is None else torch.zeros
                q_out = _made(self.buffer, stream, lambda: make(q.shape, dtype=q.dtype, device=q.device))
            shape, qs, os = q.shape, q.stride(), q_out.stride()
            if not (q.dtype == dt == q_out.dtype and q_out.shape == shape and len(shape) == 3 and shape[0] == n and shape[2] == D
                    and qs[1:] == os[1:] == (D, 1) and q.get_device() == index == q_out.get_device()):
                _need(q.dtype == dt and q.dim() == 3 and q.shape[0] == n and q.shape[2] == D and _rows_whole(q)
                      and q.get_device() == index,
                      "q must be [n_tokens, num_q_heads, head_dim] of k's dtype on the pool's device, a token's rows contiguous")
                _need(q_out.dtype == dt and q_out.shape == q.shape and _rows_whole(q_out) and q_out.get_device() == index,
                      "q_out must be like q")
            query = (q.data_ptr(), qs[0], q_out.data_ptr(), os[0], shape[1])
        else:
            _need(q_out is None, "q_out without q")
            query = (None, 0, None, 0, 0)
        if self.dtype != FP8:
            k_scale = v_scale = 1.0
        return ((ids, n, k.data_ptr(), ks[0], v.data_ptr(), vs[0], DTYPE_CODE[dt], slot_mapping.data_ptr(),
                 positions.data_ptr(), n if flat else positions.stride(0), *query),
                (float(k_scale), float(v_scale), _raw_stream(index) if stream is None and _raw_stream else _stream(self.buffer, stream)),
                q_out, positions)

    def _check_append_rope(self, k, v, slot_mapping, positions, rope, k_scale, v_scale, stream):
        """append_rope's checks one by one; returns positions, contiguous along tokens."""
        n, dt, rows = slot_mapping.shape[0], k.dtype, (slot_mapping.shape[0], self._kv_heads, self._head_dim)
        if self.dtype == FP8:
            _need(k_scale is not None and v_scale is not None, "an E4M3 pool needs k_scale and v_scale")
            _need(dt in _ROW_DTYPES, "k/v must be f32, f16 or bf16")
        else:
            _need(dt == self.dtype, "k/v dtype must match the pool")
        _need(v.dtype == dt, "k, v and q share a dtype")
        _need(k.shape == rows and v.shape == rows, "k and v must be [n_tokens, num_kv_heads, head_dim]")
        _need(_rows_whole(k) and _rows_whole(v), "a token's k and v rows must be contiguous")
        _need(slot_mapping.dtype == torch.int32 and slot_mapping.dim() == 1 and slot_mapping.is_contiguous(),
              "slot_mapping must be int32 [n_tokens]")
        _need(positions.dtype == torch.int32, "positions must be int32")
        _need(positions.shape == (rope.num_axes, n) or (rope.num_axes == 1 and positions.shape == (n,)),
              "positions must be [n_tokens], or [axes, n_tokens]")
        _need(all(t.get_device() == self._index for t in (k, v, slot_mapping, positions)),
              "every tensor must be on the pool's device")
        return positions if n < 2 or positions.stride(-1) == 1 else _made(self.buffer, stream, positions.contiguous)

    def close(self):
        if getattr(self, "_handle", None):
            self._lib.kv_pool_destroy(self._handle)
            self._handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _rows_whole(t: torch.Tensor) -> bool:
    """[n, heads, D] whose heads lie one after the other (any stride between tokens)."""
    if t.dim() != 3:
        return False
    st, sh = t.stride(), t.shape
    return (st[1] == sh[2] and st[2] == 1) or t.is_contiguous() or (
        (sh[2] == 1 or st[2] == 1) and (sh[1] == 1 or st[1] == sh[2]))


class Rope:
    """Rotation of positions into query and key rows, for KVPool.append_rope.

    inv_freq: the rot_dim / 2 frequencies (radians a position; a sequence or a 1-D tensor).
    Pairs are elements (i, i + rot_dim / 2) of a head, or (2i, 2i + 1) when interleaved.
    axes: the axis of each frequency (0 for all unless given), for tokens with several
    positions (time, height, width).  amplitude: factor on the rotated elements.
    """

    def __init__(self, inv_freq, interleaved: bool = False, axes=None, amplitude: float = 1.0):
        lib = load_library()
        if isinstance(inv_freq, torch.Tensor):
            _need(inv_freq.dim() == 1, "inv_freq must be 1-D")
            inv_freq = inv_freq.detach().double().tolist()
        freq = [float(f) for f in inv_freq]
        axes = None if axes is None else [int(x) for x in axes]
        _need(axes is None or len(axes) == len(freq), "one axis per frequency")
        _need(len(freq) > 0, "inv_freq is empty")
        self.rot_dim = 2 * len(freq)
        self.num_axes = 1 if axes is None else max(axes) + 1
        self.interleaved = bool(interleaved)
        cfg = _RopeConfig(self.rot_dim, int(self.interleaved), self.num_axes, float(amplitude),
                          (ctypes.c_double * len(freq))(*freq),
                          None if axes is None else (ctypes.c_int32 * len(axes))(*axes))
        handle = ctypes.c_void_p()
        _check(lib.kv_rope_create(ctypes.byref(cfg), ctypes.byref(handle)), lib)
        self._handle = handle
        self._lib = lib

    def __del__(self):
        try:
            if getattr(self, "_handle", None):
                self._lib.kv_rope_destroy(self._handle)
                self._handle = None
        except Exception:
            pass


def slot_mapping(block_tables: torch.Tensor, context_lens: torch.Tensor, block_size: int,
                 num_blocks: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Device slot of every sequence's newest token (position context_lens - 1)."""
    lib = load_library()
    B = context_lens.shape[0]
    _need(block_tables.dtype == torch.int32 and context_lens.dtype == torch.int32, "int32 inputs")
    _need(block_tables.is_contiguous() and block_tables.shape[0] == B, "block_tables [B, max_blocks]")
    if out is None:
        out = _made(context_lens, stream, lambda: torch.empty(B, dtype=torch.int32, device=context_lens.device))
    _call_on(context_lens, lib, lib.kv_slot_mapping,
             _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), B,
             block_size, num_blocks, _ptr(out), _stream(out, stream))
    return out


class StepTables(NamedTuple):
    """What extend_tables makes of a step: int32 tensors on the GPU."""

    context_lens: torch.Tensor  # [sequences] cached and granted tokens
    query_start: torch.Tensor   # [sequences + 1] where each sequence's new tokens start
    slot_mapping: torch.Tensor  # [tokens] slot of each new token; -1 behind the last
    positions: torch.Tensor     # [tokens] its position; 0 behind the last
    seq_ids: torch.Tensor       # [tokens] its sequence; -1 behind the last
    queue_state: torch.Tensor   # [2] front of the free queue and number of free blocks


def make_step_tables(num_seqs: int, num_tokens: int, device=None) -> StepTables:
    """Buffers for extend_tables' results with room for num_tokens new tokens."""
    dev = torch.device(device if device is not None else "cuda")
    return StepTables(*(torch.empty(n, dtype=torch.int32, device=dev)
                        for n in (num_seqs, num_seqs + 1, num_tokens, num_tokens, num_tokens, 2)))


def make_free_queue(num_blocks: int, reserve_null_block: bool = False, device=None):
    """(free_queue, queue_state) with every block free, in increasing order (block 0 held back as the null
    block if asked for), as a new BlockAllocator has them."""
    dev = torch.device(device if device is not None else "cuda")
    first = int(bool(reserve_null_block))
    _need(num_blocks > first, "no block is left")
    queue = torch.full((num_blocks,), -1, dtype=torch.int32, device=dev)
    queue[:num_blocks - first] = torch.arange(first, num_blocks, dtype=torch.int32, device=dev)
    return queue, torch.tensor([0, num_blocks - first], dtype=torch.int32, device=dev)


def _check_tables(block_tables, lens, *rest):
    _need(block_tables.dim() == 2 and lens.shape == (block_tables.shape[0],), "block_tables [B, max_blocks], lengths [B]")
    index, i32 = block_tables.get_device(), torch.int32
    good = index >= 0 and block_tables.dtype == i32 and block_tables.is_contiguous()
    for t in (lens, *rest):
        good = good and (t is None or (t.dtype == i32 and t.get_device() == index and t.is_contiguous()))
    _need(good, "every tensor must be contiguous int32 on block_tables' GPU")


def extend_tables(block_tables: torch.Tensor, cached_lens: torch.Tensor, new_lens: torch.Tensor, free_queue: torch.Tensor,
                  queue_state: torch.Tensor, block_size: int, num_tokens: int, out: StepTables | None = None,
                  stream=None) -> StepTables:
    """Blocks from the free queue for each sequence's new tokens, into block_tables, and the step's lists.

    Sequence s ([B], int32) has cached_lens[s] tokens and brings new_lens[s]; blocks go out in the sequences'
    order, and a sequence that needs more than are left, or whose tokens do not fit num_tokens, is refused (an
    empty run in query_start; see kv_tables_extend).  The lists have num_tokens entries, those behind the last
    token padding (slot -1, position 0, sequence -1), so they go as they are to KVPool.append_rope,
    append_norm_rope and paged_window_prefill_attention, in a captured graph too.  out: buffers to write to
    (make_step_tables); out.context_lens may be cached_lens itself and out.queue_state queue_state itself.
    Everything runs on `stream` (torch's current one unless given)."""
    lib = _lib or load_library()
    if out is None:
        out = _made(block_tables, stream, lambda: make_step_tables(block_tables.shape[0], num_tokens, block_tables.device))
    _check_tables(block_tables, cached_lens, new_lens, free_queue, queue_state, *out)
    lens, start, slots, positions, seqs, state = out
    B, width = block_tables.shape
    if not (new_lens.shape == lens.shape == (B,) and start.shape == (B + 1,)
            and slots.shape == positions.shape == seqs.shape == (num_tokens,)
            and queue_state.shape == state.shape == (2,) and free_queue.dim() == 1):
        raise ValueError("shapes of the lists (see make_step_tables)")
    _call(block_tables.get_device(), lib, lib.kv_tables_extend, block_tables.data_ptr(), width, cached_lens.data_ptr(),
          new_lens.data_ptr(), B, block_size, free_queue.shape[0], free_queue.data_ptr(), queue_state.data_ptr(), num_tokens,
          lens.data_ptr(), start.data_ptr(), slots.data_ptr(), positions.data_ptr(), seqs.data_ptr(), state.data_ptr(),
          _stream(block_tables, stream))
    return out


def release_tables(block_tables: torch.Tensor, context_lens: torch.Tensor, free_queue: torch.Tensor, queue_state: torch.Tensor,
                   block_size: int, finished: torch.Tensor | None = None, window: int = 0, sinks: int = 0, stream=None):
    """Give blocks back to the free queue, in place: all blocks of sequences whose `finished` entry (int32 [B])
    is not 0, their lengths becoming 0; and with window > 0, of the others the blocks that no later query of a
    layer with this window and these first tokens sees (see kv_tables_release)."""
    lib = _lib or load_library()
    _check_tables(block_tables, context_lens, free_queue, queue_state, finished)
    _need(queue_state.shape == (2,) and free_queue.dim() == 1 and (finished is None or finished.shape == context_lens.shape),
          "queue_state [2], free_queue [blocks], finished [B]")
    _need(window >= 0 and sinks >= 0, "window and sinks from 0 on")
    _call_on(block_tables, lib, lib.kv_tables_release, block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(),
             context_lens.shape[0], block_size, free_queue.shape[0], _ptr(finished), min(int(window), 0x7FFFFFFF),
             min(int(sinks), 0x7FFFFFFF), free_queue.data_ptr(), queue_state.data_ptr(), _stream(block_tables, stream))


def _options(num_ctas=0, ctas_per_sm=0, consumer_warps=0, kernel="auto", heads_per_stage=0,
             separate_reduce=False, pdl=True, early_reads=False, test_stall=False) -> _DecodeOptions:
    return _DecodeOptions(num_ctas, ctas_per_sm, consumer_warps, KERNELS[kernel], heads_per_stage,
                          int(separate_reduce), int(not pdl), int(early_reads), int(test_stall))


def workspace_init(workspace: torch.Tensor, num_seqs: int, num_kv_heads: int, stream=None):
    """Zero the merge counters at the start of a workspace (once after allocation)."""
    lib = load_library()
    _call_on(workspace, lib, lib.paged_decode_workspace_init,
             _ptr(workspace), workspace.numel(), num_seqs, num_kv_heads,
                                           _stream(workspace, stream))


def make_workspace(num_seqs, num_q_heads, num_kv_heads, head_dim, device=None, **opts) -> torch.Tensor:
    """A zero-filled workspace for paged_decode_attention with these sizes and options."""
    dev = torch.device(device if device is not None else "cuda")
    n = workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, dev, **opts)
    return torch.zeros(n, dtype=torch.uint8, device=dev)


def workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, device=None, **opts) -> int:
    lib = load_library()
    dev = torch.device(device if device is not None else "cuda")
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    o = _options(**opts)
    n = ctypes.c_size_t()
    _check(lib.paged_decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, idx,
                                            ctypes.byref(o), ctypes.byref(n)), lib)
    return int(n.value)


def paged_decode_attention(q, k_cache, v_cache, block_tables, context_lens, scale: float,
                           out=None, out_dtype=None, workspace=None, stream=None, k_scale=None,
                           v_scale=None, **opts):
    """out[s, g] = softmax(scale q[s, g] . K_s^T) V_s over the paged cache (one layer).

    q [B, Hq, D]; k_cache/v_cache [NB, Hkv, bs, D]; block_tables int32 [B, max_blocks];
    context_lens int32 [B].  opts: num_ctas, ctas_per_sm, consumer_warps, kernel.
    E4M3 (torch.float8_e4m3fn) caches stand for k_scale (v_scale) times their codes.
    """
    lib = load_library()
    B, Hq, D = q.shape
    NB, Hkv, bs, D2 = k_cache.shape
    _need(D == D2 and tuple(v_cache.shape) == tuple(k_cache.shape), "cache shapes")
    fp8 = k_cache.dtype == FP8
    if fp8:
        _need(v_cache.dtype == FP8 and k_scale is not None and v_scale is not None,
              "an E4M3 cache needs both caches E4M3 and k_scale, v_scale")
    else:
        _need(q.dtype == k_cache.dtype == v_cache.dtype, "q and the caches share a dtype")
    _need(all(t.is_contiguous() for t in (q, k_cache, v_cache, block_tables, context_lens)),
          "contiguous inputs")
    _need(block_tables.dtype == torch.int32 and context_lens.dtype == torch.int32, "int32 tables")
    _need(block_tables.shape[0] == B and context_lens.shape[0] == B, "one table row and length per sequence")
    out_dtype = out_dtype or q.dtype
    if out is None:
        out = _made(q, stream, lambda: torch.empty((B, Hq, D), dtype=out_dtype, device=q.device))
    _need(out.dtype == out_dtype and tuple(out.shape) == (B, Hq, D) and out.is_contiguous(), "out")
    o = _options(**opts)
    if workspace is None:
        workspace = _made(q, stream, lambda: make_workspace(B, Hq, Hkv, D, q.device, **opts))
    if fp8:
        _call_on(q, lib, lib.paged_decode_attention_fp8,
            _ptr(q), DTYPE_CODE[q.dtype], _ptr(k_cache), _ptr(v_cache), float(k_scale), float(v_scale),
            NB, _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), B, Hq, Hkv, D, bs,
            float(scale), _ptr(out), DTYPE_CODE[out_dtype], _ptr(workspace), workspace.numel(),
            ctypes.byref(o), _stream(q, stream))
        return out
    _call_on(q, lib, lib.paged_decode_attention,
        _ptr(q), _ptr(k_cache), _ptr(v_cache), NB, _ptr(block_tables), block_tables.shape[1],
        _ptr(context_lens), B, Hq, Hkv, D, bs, DTYPE_CODE[q.dtype], float(scale), _ptr(out),
        DTYPE_CODE[out_dtype], _ptr(workspace), workspace.numel(), ctypes.byref(o),
        _stream(q, stream))
    return out


def paged_decode_append_attention(q, k_new, v_new, k_cache, v_cache, block_tables, context_lens,
                                  scale: float, seq_ids=None, out=None, out_dtype=None,
                                  slot_mapping=None, workspace=None, stream=None, k_scale=None,
                                  v_scale=None, **opts):
    """One layer of a decode step in one kernel: append k_new/v_new ([B, Hkv, D]) at
    position context_lens - 1 of every sequence, then attend (see paged_decode_attention).

    seq_ids: optional int32 [B]; a negative entry skips the append of that sequence.
    slot_mapping: optional int32 [B] output receiving the newest-token slots.
    """
    lib = load_library()
    B, Hq, D = q.shape
    NB, Hkv, bs, D2 = k_cache.shape
    _need(D == D2 and tuple(v_cache.shape) == tuple(k_cache.shape), "cache shapes")
    fp8 = k_cache.dtype == FP8
    if fp8:
        _need(v_cache.dtype == FP8 and k_scale is not None and v_scale is not None,
              "an E4M3 cache needs both caches E4M3 and k_scale, v_scale")
        _need(q.dtype == k_new.dtype == v_new.dtype, "q, k_new and v_new share a dtype")
    else:
        _need(q.dtype == k_cache.dtype == v_cache.dtype == k_new.dtype == v_new.dtype, "one dtype")
    _need(tuple(k_new.shape) == (B, Hkv, D) and k_new.shape == v_new.shape, "k_new/v_new [B, Hkv, D]")
    _need(all(t.is_contiguous() for t in (q, k_new, v_new, k_cache, v_cache, block_tables, context_lens)),
          "contiguous inputs")
    _need(block_tables.dtype == torch.int32 and context_lens.dtype == torch.int32, "int32 tables")
    _need(block_tables.shape[0] == B and context_lens.shape[0] == B, "one table row and length per sequence")
    _need(seq_ids is None or (seq_ids.dtype == torch.int32 and seq_ids.shape[0] == B), "seq_ids int32 [B]")
    _need(slot_mapping is None or (slot_mapping.dtype == torch.int32 and slot_mapping.shape[0] == B),
          "slot_mapping int32 [B]")
    out_dtype = out_dtype or q.dtype
    if out is None:
        out = _made(q, stream, lambda: torch.empty((B, Hq, D), dtype=out_dtype, device=q.device))
    _need(out.dtype == out_dtype and tuple(out.shape) == (B, Hq, D) and out.is_contiguous(), "out")
    o = _options(**opts)
    if workspace is None:
        workspace = _made(q, stream, lambda: make_workspace(B, Hq, Hkv, D, q.device, **opts))
    if fp8:
        _call_on(q, lib, lib.paged_decode_append_attention_fp8,
            _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(seq_ids), DTYPE_CODE[q.dtype], _ptr(k_cache),
            _ptr(v_cache), float(k_scale), float(v_scale), NB, _ptr(block_tables), block_tables.shape[1],
            _ptr(context_lens), B, Hq, Hkv, D, bs, float(scale), _ptr(out), DTYPE_CODE[out_dtype],
            _ptr(slot_mapping), _ptr(workspace), workspace.numel(), ctypes.byref(o),
            _stream(q, stream))
        return out
    _call_on(q, lib, lib.paged_decode_append_attention,
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(seq_ids), _ptr(k_cache), _ptr(v_cache), NB,
        _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), B, Hq, Hkv, D, bs,
        DTYPE_CODE[q.dtype], float(scale), _ptr(out), DTYPE_CODE[out_dtype], _ptr(slot_mapping),
        _ptr(workspace), workspace.numel(), ctypes.byref(o), _stream(q, stream))
    return out


def slot_mapping_varlen(block_tables: torch.Tensor, query_start: torch.Tensor, context_lens: torch.Tensor,
                        block_size: int, num_blocks: int, num_tokens: int | None = None,
                        out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Device slot of every new token of a multi-token step (int32 [num_tokens])."""
    lib = load_library()
    B = context_lens.shape[0]
    _need(block_tables.dtype == torch.int32 and context_lens.dtype == torch.int32 and
          query_start.dtype == torch.int32, "int32 inputs")
    _need(query_start.shape[0] == B + 1 and block_tables.shape[0] == B and block_tables.is_contiguous(),
          "query_start [B + 1], block_tables [B, max_blocks]")
    if num_tokens is None:
        num_tokens = int(query_start[-1].item())
    if out is None:
        out = _made(context_lens, stream, lambda: torch.empty(max(num_tokens, 1), dtype=torch.int32,
                                                              device=context_lens.device))[:num_tokens]
    _call_on(context_lens, lib, lib.kv_slot_mapping_varlen,
             _ptr(block_tables), block_tables.shape[1], _ptr(query_start),
             _ptr(context_lens), B, num_tokens, block_size, num_blocks, _ptr(out),
             _stream(context_lens, stream))
    return out


def paged_prefill_attention(q, k_cache, v_cache, block_tables, query_start, context_lens, scale: float,
                            out=None, out_dtype=None, workspace=None, stream=None, k_scale=None, v_scale=None):
    """Causal attention of a step's new tokens (q [T, Hq, D], rows grouped by
    sequence as query_start says) over the paged cache they were appended to.
    E4M3 (torch.float8_e4m3fn) caches stand for k_scale (v_scale) times their codes."""
    lib = load_library()
    T, Hq, D = q.shape
    NB, Hkv, bs, D2 = k_cache.shape
    B = context_lens.shape[0]
    _need(D == D2 and tuple(v_cache.shape) == tuple(k_cache.shape), "cache shapes")
    fp8 = k_cache.dtype == FP8
    if fp8:
        _need(v_cache.dtype == FP8 and k_scale is not None and v_scale is not None,
              "an E4M3 cache needs both caches E4M3 and k_scale, v_scale")
    else:
        _need(q.dtype == k_cache.dtype == v_cache.dtype, "q and the caches share a dtype")
    _need(all(t.is_contiguous() for t in (q, k_cache, v_cache, block_tables, query_start, context_lens)),
          "contiguous inputs")
    _need(block_tables.dtype == torch.int32 and context_lens.dtype == torch.int32 and
          query_start.dtype == torch.int32, "int32 tables")
    _need(block_tables.shape[0] == B and query_start.shape[0] == B + 1, "table rows / query_start")
    out_dtype = out_dtype or q.dtype
    if out is None:
        out = _made(q, stream, lambda: torch.empty((T, Hq, D), dtype=out_dtype, device=q.device))
    _need(out.dtype == out_dtype and tuple(out.shape) == (T, Hq, D) and out.is_contiguous(), "out")
    if workspace is None:
        workspace = _made(q, stream, lambda: torch.empty(max(16, int(lib.paged_prefill_workspace_bytes(B))),
                                                         dtype=torch.uint8, device=q.device))
    if fp8:
        _call_on(q, lib, lib.paged_prefill_attention_fp8,
                 _ptr(q), DTYPE_CODE[q.dtype], _ptr(k_cache), _ptr(v_cache), float(k_scale), float(v_scale), NB,
                 _ptr(block_tables), block_tables.shape[1], _ptr(query_start), _ptr(context_lens), B, T, Hq, Hkv,
                 D, bs, float(scale), _ptr(out), DTYPE_CODE[out_dtype], _ptr(workspace), workspace.numel(),
                 _stream(q, stream))
        return out
    _call_on(q, lib, lib.paged_prefill_attention,
        _ptr(q), _ptr(k_cache), _ptr(v_cache), NB, _ptr(block_tables), block_tables.shape[1],
        _ptr(query_start), _ptr(context_lens), B, T, Hq, Hkv, D, bs, DTYPE_CODE[q.dtype], float(scale),
        _ptr(out), DTYPE_CODE[out_dtype], _ptr(workspace), workspace.numel(), _stream(q, stream))
    return out


def shared_prefix_workspace_bytes(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, device=None) -> int:
    lib = load_library()
    dev = torch.device(device if device is not None else "cuda")
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    n = ctypes.c_size_t()
    _check(lib.paged_shared_prefix_workspace_bytes(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, idx,
                                                   ctypes.byref(n)), lib)
    return int(n.value)


def make_shared_prefix_workspace(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, device=None) -> torch.Tensor:
    """A workspace for paged_shared_prefix_attention with these sizes (or smaller ones)."""
    dev = torch.device(device if device is not None else "cuda")
    n = shared_prefix_workspace_bytes(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, dev)
    return torch.empty(n, dtype=torch.uint8, device=dev)


def paged_shared_prefix_attention(q, k_cache, v_cache, block_tables, context_lens, group_start, prefix_lens,
                                  scale: float, out=None, out_dtype=None, workspace=None, stream=None, k_scale=None,
                                  v_scale=None):
    """paged_decode_attention of a batch whose sequences share prefixes, each read once for its group.

    Sequences group_start[g] .. group_start[g + 1] - 1 (int32 [groups + 1]) hold the same blocks in their
    first prefix_lens[g] / block_size table entries (int32 [groups]); a sequence shorter than that, or in
    no group, is read through its own table throughout.  The other arguments are those of
    paged_decode_attention; q f16 or bf16, block_size a multiple of 16.  Everything runs on `stream`
    (torch's current one unless given): order the inputs before it, and what reads out behind it.
    """
    lib = _lib or load_library()
    B, Hq, D = q.shape
    NB, Hkv, bs, D2 = k_cache.shape
    fp8 = k_cache.dtype == FP8
    i32, index = torch.int32, q.get_device()
    groups = prefix_lens.shape[0] if prefix_lens.dim() == 1 else -1
    out_dtype = out_dtype or q.dtype
    # (The library cannot tell a host address from a device one.)
    _need(0 <= index == k_cache.get_device() == v_cache.get_device() == block_tables.get_device()
          == context_lens.get_device() == group_start.get_device() == prefix_lens.get_device()
          and (out is None or out.get_device() == index) and (workspace is None or workspace.get_device() == index),
          "every tensor must be on q's GPU")
    if out is None:
        out = _made(q, stream, lambda: torch.empty((B, Hq, D), dtype=out_dtype, device=q.device))
    if workspace is None:
        workspace = _made(q, stream, lambda: make_shared_prefix_workspace(B, max(groups, 0), Hq, Hkv, D, q.device))
    _need(D == D2 and v_cache.shape == k_cache.shape, "cache shapes")
    _need((v_cache.dtype == FP8 and k_scale is not None and v_scale is not None) if fp8
          else q.dtype == k_cache.dtype == v_cache.dtype,
          "q and the caches share a dtype, or both caches are E4M3 with k_scale and v_scale")
    _need(block_tables.dtype == context_lens.dtype == group_start.dtype == prefix_lens.dtype == i32, "int32 tables")
    _need(q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous() and block_tables.is_contiguous()
          and context_lens.is_contiguous() and group_start.is_contiguous() and prefix_lens.is_contiguous(),
          "contiguous inputs")
    _need(block_tables.dim() == 2 and block_tables.shape[0] == B and context_lens.shape == (B,),
          "one table row and length per sequence")
    _need(groups >= 0 and group_start.shape == (groups + 1,), "group_start [groups + 1], prefix_lens [groups]")
    _need(out.dtype == out_dtype and out.shape == q.shape and out.is_contiguous(), "out")
    _need(workspace.is_contiguous(), "a contiguous workspace")
    sizes = (NB, block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(), B, group_start.data_ptr(),
             prefix_lens.data_ptr(), groups, Hq, Hkv, D, bs)
    rest = (float(scale), out.data_ptr(), DTYPE_CODE[out_dtype], workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _stream(q, stream))
    if fp8:
        _call_on(q, lib, lib.paged_shared_prefix_attention_fp8, q.data_ptr(), DTYPE_CODE[q.dtype], k_cache.data_ptr(),
                 v_cache.data_ptr(), float(k_scale), float(v_scale), *sizes, *rest)
    else:
        _call_on(q, lib, lib.paged_shared_prefix_attention, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                 *sizes, DTYPE_CODE[q.dtype], *rest)
    return out


def _check_window(q, k_cache, v_cache, block_tables, context_lens, query_start, window, sinks, k_scale, v_scale):
    """The checks of the windowed attention calls one by one; returns window and sinks within 32 bits."""
    index = q.get_device()
    lists = (block_tables, context_lens) if query_start is None else (block_tables, context_lens, query_start)
    # (The library cannot tell a host address from a device one.)
    _need(index >= 0 and all(t.get_device() == index for t in (k_cache, v_cache, *lists)), "every tensor must be on q's GPU")
    _need(k_cache.dim() == 4 and k_cache.shape[3] == q.shape[2] and v_cache.shape == k_cache.shape,
          "q [n, Hq, D], caches [NB, Hkv, bs, D]")
    _need((q.dtype in _ROW_DTYPES and v_cache.dtype == FP8 and k_scale is not None and v_scale is not None)
          if k_cache.dtype == FP8 else (q.dtype in _ROW_DTYPES and q.dtype == k_cache.dtype == v_cache.dtype),
          "q and the caches share a dtype, or both caches are E4M3 with k_scale and v_scale")
    _need(all(t.is_contiguous() for t in (q, k_cache, v_cache, *lists)), "contiguous inputs")
    _need(all(t.dtype == torch.int32 for t in lists), "int32 tables and lengths")
    B = context_lens.shape[0] if query_start is not None else q.shape[0]
    _need(block_tables.dim() == 2 and block_tables.shape[0] == B and context_lens.shape == (B,)
          and (query_start is None or query_start.shape == (B + 1,)),
          "one table row and length per sequence, query_start [sequences + 1]")
    _need(0 < window and 0 <= sinks, "window from 1 on, sinks from 0 on")
    return min(int(window), 0x7FFFFFFF), min(int(sinks), 0x7FFFFFFF)


def _check_out(index, shape, out, out_dtype, workspace):
    if not (out.dtype == out_dtype and out_dtype in _ROW_DTYPES and out.shape == shape and out.is_contiguous()
            and workspace.is_contiguous() and out.get_device() == index == workspace.get_device()):
        raise ValueError("out must be contiguous, of q's shape and of out_dtype, the workspace contiguous, both on q's GPU")


def paged_window_decode_attention(q, k_cache, v_cache, block_tables, context_lens, scale: float, window: int,
                                  sinks: int = 0, out=None, out_dtype=None, workspace=None, stream=None, k_scale=None,
                                  v_scale=None, **opts):
    """paged_decode_attention over the last `window` cached tokens of each sequence (the newest
    among them) and its first `sinks` ones.

    Table entries of blocks out of sight are not read and may be anything.  The other arguments are
    those of paged_decode_attention, the workspace too (make_workspace).  Everything runs on
    `stream` (torch's current one unless given)."""
    lib = _lib or load_library()
    B, Hq, D = shape = q.shape
    cache = k_cache.shape
    index, dt, kdt, i32 = q.get_device(), q.dtype, k_cache.dtype, torch.int32
    # The usual call in one expression; _check_window says what is wrong with any other.
    if not (kdt == v_cache.dtype and dt in _ROW_DTYPES and (dt == kdt or kdt == FP8 and k_scale is not None and v_scale is not None)
            and len(cache) == 4 and cache[3] == D and v_cache.shape == cache
            and block_tables.dtype == i32 and context_lens.dtype == i32 and block_tables.dim() == 2
            and block_tables.shape[0] == B and context_lens.shape == (B,) and 0 < window <= 0x7FFFFFFF
            and 0 <= sinks <= 0x7FFFFFFF and q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()
            and block_tables.is_contiguous() and context_lens.is_contiguous()
            and 0 <= index == k_cache.get_device() == v_cache.get_device() == block_tables.get_device()
            == context_lens.get_device()):
        window, sinks = _check_window(q, k_cache, v_cache, block_tables, context_lens, None, window, sinks, k_scale, v_scale)
    if out_dtype is None:
        out_dtype = dt
    if out is None:
        out = _made(q, stream, lambda: torch.empty(shape, dtype=out_dtype, device=q.device))
    if workspace is None:
        workspace = _made(q, stream, lambda: make_workspace(B, Hq, cache[1], D, q.device, **opts))
    _check_out(index, shape, out, out_dtype, workspace)
    sizes = (cache[0], block_tables.data_ptr(), block_tables.shape[1], context_lens.data_ptr(), B, Hq, cache[1], D, cache[2])
    rest = (float(scale), window, sinks, out.data_ptr(), DTYPE_CODE[out_dtype], workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), ctypes.byref(_options(**opts)) if opts else None, _stream(q, stream))
    if kdt == FP8:
        _call(index, lib, lib.paged_window_decode_attention_fp8, q.data_ptr(), DTYPE_CODE[dt], k_cache.data_ptr(),
              v_cache.data_ptr(), float(k_scale), float(v_scale), *sizes, *rest)
    else:
        _call(index, lib, lib.paged_window_decode_attention, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), *sizes,
              DTYPE_CODE[dt], *rest)
    return out


def window_prefill_workspace_bytes(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, device=None) -> int:
    lib = load_library()
    dev = torch.device(device if device is not None else "cuda")
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    n = ctypes.c_size_t()
    _check(lib.paged_window_prefill_workspace_bytes(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, idx,
                                                    ctypes.byref(n)), lib)
    return int(n.value)


def make_window_prefill_workspace(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, device=None) -> torch.Tensor:
    """A workspace for paged_window_prefill_attention with these sizes (or smaller ones)."""
    dev = torch.device(device if device is not None else "cuda")
    n = window_prefill_workspace_bytes(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, dev)
    return torch.empty(n, dtype=torch.uint8, device=dev)


def paged_window_prefill_attention(q, k_cache, v_cache, block_tables, query_start, context_lens, scale: float, window: int,
                                   sinks: int = 0, out=None, out_dtype=None, workspace=None, stream=None, k_scale=None,
                                   v_scale=None):
    """paged_prefill_attention in which each new token sees the last `window` tokens up to itself and
    the first `sinks` ones of its sequence.

    Table entries of blocks that none of a sequence's new tokens sees are not read.  Rows of q behind
    the last sequence (query_start[-1]) are padding and may hold anything: those rows of out stay as they
    are (a new out holds zeros there).  With a 16-bit out_dtype weights are rounded to it before they meet V;
    out_dtype=torch.float32 keeps twice as many bits of them.  Everything runs on `stream` (torch's current one unless given)."""
    lib = _lib or load_library()
    T, Hq, D = shape = q.shape
    cache = k_cache.shape
    B = context_lens.shape[0]
    index, dt, kdt, i32 = q.get_device(), q.dtype, k_cache.dtype, torch.int32
    if not (kdt == v_cache.dtype and dt in _ROW_DTYPES and (dt == kdt or kdt == FP8 and k_scale is not None and v_scale is not None)
            and len(cache) == 4 and cache[3] == D and v_cache.shape == cache
            and block_tables.dtype == i32 and context_lens.dtype == i32 and query_start.dtype == i32
            and block_tables.dim() == 2 and block_tables.shape[0] == B and context_lens.shape == (B,)
            and query_start.shape == (B + 1,) and 0 < window <= 0x7FFFFFFF and 0 <= sinks <= 0x7FFFFFFF
            and q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous() and block_tables.is_contiguous()
            and context_lens.is_contiguous() and query_start.is_contiguous()
            and 0 <= index == k_cache.get_device() == v_cache.get_device() == block_tables.get_device()
            == context_lens.get_device() == query_start.get_device()):
        window, sinks = _check_window(q, k_cache, v_cache, block_tables, context_lens, query_start, window, sinks, k_scale, v_scale)
    if out_dtype is None:
        out_dtype = dt
    if out is None:
        out = _made(q, stream, lambda: torch.zeros(shape, dtype=out_dtype, device=q.device))
    if workspace is None:
        workspace = _made(q, stream, lambda: make_window_prefill_workspace(B, T, Hq, cache[1], D, q.device))
    _check_out(index, shape, out, out_dtype, workspace)
    sizes = (cache[0], block_tables.data_ptr(), block_tables.shape[1], query_start.data_ptr(), context_lens.data_ptr(), B, T,
             Hq, cache[1], D, cache[2])
    rest = (float(scale), window, sinks, out.data_ptr(), DTYPE_CODE[out_dtype], workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _stream(q, stream))
    if kdt == FP8:
        _call(index, lib, lib.paged_window_prefill_attention_fp8, q.data_ptr(), DTYPE_CODE[dt], k_cache.data_ptr(),
              v_cache.data_ptr(), float(k_scale), float(v_scale), *sizes, *rest)
    else:
        _call(index, lib, lib.paged_window_prefill_attention, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), *sizes,
              DTYPE_CODE[dt], *rest)
    return out


def paged_decode_attention_static(q, k_cache, v_cache, block_tables, context_lens, scale: float,
                                  out=None, out_dtype=None, stream=None, **opts):
    """paged_decode_attention with the library's fixed device scratch instead of a
    workspace: the call allocates nothing (see include/pkv.h)."""
    lib = load_library()
    B, Hq, D = q.shape
    NB, Hkv, bs, D2 = k_cache.shape
    _need(D == D2 and tuple(v_cache.shape) == tuple(k_cache.shape), "cache shapes")
    _need(q.dtype == k_cache.dtype == v_cache.dtype, "q and the caches share a dtype")
    _need(all(t.is_contiguous() for t in (q, k_cache, v_cache, block_tables, context_lens)),
          "contiguous inputs")
    _need(block_tables.dtype == torch.int32 and context_lens.dtype == torch.int32, "int32 tables")
    out_dtype = out_dtype or q.dtype
    _need(out is not None, "out must be given (the call allocates nothing)")
    _need(out.dtype == out_dtype and tuple(out.shape) == (B, Hq, D) and out.is_contiguous(), "out")
    o = _options(**opts)
    _call_on(q, lib, lib.paged_decode_attention_static,
        _ptr(q), _ptr(k_cache), _ptr(v_cache), NB, _ptr(block_tables), block_tables.shape[1],
        _ptr(context_lens), B, Hq, Hkv, D, bs, DTYPE_CODE[q.dtype], float(scale), _ptr(out),
        DTYPE_CODE[out_dtype], ctypes.byref(o), _stream(q, stream))
    return out


def device_status(device=None, stream=None):
    """Synchronise, then read and clear the device status word: (status, flags)."""
    lib = load_library()
    dev = torch.device(device if device is not None else "cuda")
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    s = stream if stream is not None else torch.cuda.current_stream(idx)
    flags = ctypes.c_uint32()
    st = lib.kv_device_status(idx, ctypes.c_void_p(s.cuda_stream), ctypes.byref(flags))
    return int(st), int(flags.value)


class BlockAllocator:
    """Host block allocator (FIFO free queue, optional null block 0)."""

    def __init__(self, num_blocks: int, block_size: int, reserve_null_block: bool = True):
        self._lib = load_library()
        h = ctypes.c_void_p()
        _check(self._lib.kv_allocator_create(num_blocks, block_size, int(reserve_null_block),
                                             ctypes.byref(h)), self._lib)
        self._h = h
        self.num_blocks = num_blocks
        self.block_size = block_size

    def extend(self, seq_id: int, new_tokens: int) -> bool:
        """Room for new_tokens more tokens; False (nothing changed) when blocks run out."""
        st = self._lib.kv_allocator_extend(self._h, seq_id, new_tokens)
        if st == 4:  # KV_ERR_OUT_OF_BLOCKS
            return False
        _check(st, self._lib)
        return True

    def release(self, seq_id: int):
        _check(self._lib.kv_allocator_release(self._h, seq_id), self._lib)

    def table(self, seq_id: int):
        nb, nt = ctypes.c_int(), ctypes.c_int()
        _check(self._lib.kv_allocator_table(self._h, seq_id, None, 0, ctypes.byref(nb),
                                            ctypes.byref(nt)), self._lib)
        buf = (ctypes.c_int32 * max(1, nb.value))()
        _check(self._lib.kv_allocator_table(self._h, seq_id, buf, nb.value, None, None), self._lib)
        return list(buf[:nb.value]), nt.value

    def slot(self, seq_id: int, position: int) -> int:
        out = ctypes.c_int32()
        _check(self._lib.kv_allocator_slot(self._h, seq_id, position, ctypes.byref(out)), self._lib)
        return int(out.value)

    def free_queue(self):
        n = ctypes.c_int()
        _check(self._lib.kv_allocator_free_queue(self._h, None, 0, ctypes.byref(n)), self._lib)
        buf = (ctypes.c_int32 * max(1, n.value))()
        _check(self._lib.kv_allocator_free_queue(self._h, buf, n.value, None), self._lib)
        return list(buf[:n.value])

    def __del__(self):
        try:
            if getattr(self, "_h", None):
                self._lib.kv_allocator_destroy(self._h)
                self._h = None
        except Exception:
            pass


class PrefixCachePool:
    """Host block pool with prefix caching (chained block hashes, LRU free queue)."""

    def __init__(self, num_blocks: int, block_size: int):
        self._lib = load_library()
        h = ctypes.c_void_p()
        _check(self._lib.kv_prefix_pool_create(num_blocks, block_size, ctypes.byref(h)), self._lib)
        self._h = h
        self.num_blocks = num_blocks
        self.block_size = block_size

    def allocate(self, tokens):
        """Blocks for a request with these token ids: (blocks, cached_tokens, evicted).

        Returns None (nothing changed) when too few blocks are free."""
        tokens = [int(t) for t in tokens]
        n = len(tokens)
        cap = max(1, -(-n // self.block_size))
        tok = (ctypes.c_int32 * max(1, n))(*tokens)
        blocks = (ctypes.c_int32 * cap)()
        evicted = (ctypes.c_int32 * cap)()
        nb, cached, ne = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
        st = self._lib.kv_prefix_pool_allocate(self._h, tok, n, blocks, cap, ctypes.byref(nb),
                                               ctypes.byref(cached), evicted, cap, ctypes.byref(ne))
        if st == 4:  # KV_ERR_OUT_OF_BLOCKS
            return None
        _check(st, self._lib)
        return list(blocks[:nb.value]), int(cached.value), list(evicted[:ne.value])

    def free(self, blocks):
        blocks = [int(b) for b in blocks]
        buf = (ctypes.c_int32 * max(1, len(blocks)))(*blocks)
        _check(self._lib.kv_prefix_pool_free(self._h, buf, len(blocks)), self._lib)

    def free_queue(self):
        n = ctypes.c_int()
        _check(self._lib.kv_prefix_pool_free_queue(self._h, None, 0, ctypes.byref(n)), self._lib)
        buf = (ctypes.c_int32 * max(1, n.value))()
        _check(self._lib.kv_prefix_pool_free_queue(self._h, buf, n.value, None), self._lib)
        return list(buf[:n.value])

    def cache_size(self):
        h, b = ctypes.c_int(), ctypes.c_int()
        _check(self._lib.kv_prefix_pool_cache_size(self._h, ctypes.byref(h), ctypes.byref(b)),
               self._lib)
        return int(h.value), int(b.value)

    def __del__(self):
        try:
            if getattr(self, "_h", None):
                self._lib.kv_prefix_pool_destroy(self._h)
                self._h = None
        except Exception:
            pass
