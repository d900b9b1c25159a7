"""Thin ctypes binding of libhsa (``include/hsa.h``), same names as the C ABI.

Arguments are marshalled only: torch tensors become raw pointers, the current torch
stream becomes the ``void* stream`` argument, and a nonzero status raises ``HsaError``.
Every step of the decode path runs in the CUDA library; nothing here computes. When the
library is missing or fails to load, every call raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libhsa.so")

HSA_OK = 0
HSA_ERR_INVALID_ARG = 1
HSA_ERR_UNSUPPORTED = 2
HSA_ERR_CUDA = 3
HSA_ERR_TIMEOUT = 4
HSA_ERR_WORKSPACE_TOO_SMALL = 5
HSA_ERR_DEVICE_CHECK = 6

HSA_OP_QUANTIZE = 0
HSA_OP_SELECT = 1
HSA_OP_ATTEND = 2
HSA_OP_DENSE = 3
HSA_OP_STEP = 4
HSA_OP_CACHED = 5
HSA_OP_KV8_DECODE = 6
HSA_OP_KV8_PREFILL = 7

# Every entry point declared in include/hsa.h.
EXPORTS = (
    "hsa_workspace_bytes", "hsa_status_string", "hsa_quantize_keys", "hsa_append_kv",
    "hsa_score_blocks", "hsa_prune", "hsa_select", "hsa_attend", "dense_decode",
    "hsa_decode_step", "hsa_decode_step_reuse", "hsa_read_device_error", "hsa_select_noalloc",
    "hsa_decode_step_kernels",
    "hsa_block_cache_bytes", "hsa_block_cache_mass", "hsa_attend_cached",
    "hsa_decode_step_cached",
    "hsa_kv8_write", "hsa_kv8_read", "hsa_kv8_decode", "hsa_kv8_attend",
    "hsa_kv8_prefill",
)


class HsaError(RuntimeError):
    def __init__(self, name: str, code: int, text: str):
        super().__init__(f"{name} failed: {text} (status {code})")
        self.code = code


class hsa_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "hq", "hkv", "head_dim", "page_size", "max_pages_per_seq", "num_pages",
        "chunk", "block", "k1", "k2", "sink", "window")] + [
        ("sm_scale", ctypes.c_float), ("kv_on_host", ctypes.c_int32),
        ("chunk0", ctypes.c_int32), ("k0", ctypes.c_int32), ("key_bits", ctypes.c_int32),
        ("per_head", ctypes.c_int32), ("key_fp8", ctypes.c_int32),
        ("cache_policy", ctypes.c_int32)]


class hsa_step_io(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("io_on_host", ctypes.c_int32)]


class hsa_kv8(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("format", ctypes.c_int32)]


_DIMS_CACHE: dict = {}  # field values -> their C struct (read-only to the library)


@dataclasses.dataclass
class Dims:
    batch: int
    hq: int
    hkv: int
    max_pages_per_seq: int
    num_pages: int
    chunk: int = 64
    k1: int = 16
    k2: int = 16
    sink: int = 64
    window: int = 256
    head_dim: int = 128
    page_size: int = 16
    block: int = 16
    sm_scale: float = 0.0
    kv_on_host: bool = False
    chunk0: int = 0  # k0 > 0: module 0 keeps the top-k0 chunks of chunk0 tokens
    k0: int = 0
    key_bits: int = 0  # 4: 4-bit key codes, two per byte; 0 or 8: 8-bit
    per_head: int = 0  # 1: every query head selects its own blocks (rows = hq)
    key_fp8: int = 0  # 1: FP8 E4M3 key codes (8-bit layout), fp32 scores
    cache_policy: int = 0  # block cache victims: 0 least recently used, 1 least cumulative mass

    def c(self) -> hsa_dims:
        """The C struct, built once per set of field values (every call of a step passes it)."""
        key = (self.batch, self.hq, self.hkv, self.head_dim, self.page_size,
               self.max_pages_per_seq, self.num_pages, self.chunk, self.block, self.k1,
               self.k2, self.sink, self.window, float(self.sm_scale),
               1 if self.kv_on_host else 0, self.chunk0, self.k0, self.key_bits, self.per_head,
               self.key_fp8, self.cache_policy)
        c = _DIMS_CACHE.get(key)
        if c is None:
            if len(_DIMS_CACHE) > 256:
                _DIMS_CACHE.clear()
            c = _DIMS_CACHE[key] = hsa_dims(*key)
        return c


_LIB = None


def load(path: Optional[str] = None):
    """Load libhsa.so (once). Raises if it has not been built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"libhsa.so is not built ({path}); run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    C = ctypes.POINTER(hsa_kv8)
    D = ctypes.POINTER(hsa_dims)
    sig = {
        "hsa_workspace_bytes": (SZ, [D, I32]),
        "hsa_status_string": (ctypes.c_char_p, [I32]),
        "hsa_quantize_keys": (I32, [D, P, P, P, I32, I32, P, P, P, SZ, P]),
        "hsa_append_kv": (I32, [D, P, P, P, P, P, P, P, P, P]),
        "hsa_score_blocks": (I32, [D, P, P, P, P, P, P, P, P]),
        "hsa_prune": (I32, [D, P, P, P, P, P, P, P, P]),
        "hsa_select": (I32, [D, P, P, P, P, P, P, P, P, P, P, SZ, P]),
        "hsa_attend": (I32, [D, P, P, P, P, P, P, P, P, P, P, SZ, P]),
        "dense_decode": (I32, [D, P, P, P, P, P, P, P, P, SZ, P]),
        "hsa_decode_step": (I32, [D, ctypes.POINTER(hsa_step_io), P, P, P, P, P, P, P, P, P,
                                  SZ, P]),
        "hsa_decode_step_reuse": (I32, [D, ctypes.POINTER(hsa_step_io), P, P, P, P, P, P, P, P,
                                        P, SZ, P]),
        "hsa_block_cache_bytes": (SZ, [D, I32]),
        "hsa_block_cache_mass": (P, [D, P, I32]),
        "hsa_attend_cached": (I32, [D, P, P, P, P, P, P, P, P, I32, P, P, P, SZ, P]),
        "hsa_decode_step_cached": (I32, [D, ctypes.POINTER(hsa_step_io), P, P, P, P, P, P, P, P,
                                         P, I32, P, SZ, P]),
        "hsa_read_device_error": (I32, [P, P, ctypes.POINTER(I32)]),
        "hsa_select_noalloc": (I32, [D, P, P, P, P, P, P, P, P, P, P]),
        "hsa_decode_step_kernels": (I32, [D]),
        "hsa_kv8_write": (I32, [D, C, P, I64, P, I64, P, I32, P, P, P, SZ, P]),
        "hsa_kv8_read": (I32, [D, C, P, I64, P, I64, P, I32, P, P, P, SZ, P]),
        "hsa_kv8_decode": (I32, [D, C, P, P, P, P, P, P, SZ, P]),
        "hsa_kv8_attend": (I32, [D, C, P, P, P, P, P, P, P, P, SZ, P]),
        "hsa_kv8_prefill": (I32, [D, C, P, I64, P, I32, P, P, P, P, P, SZ, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _LIB = lib
    return lib


def _p(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None) -> int:
    if stream is None:
        if _RAW_STREAM is not None:  # the current stream's handle without a Stream object
            return _RAW_STREAM(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(name: str, rc: int) -> None:
    if rc != HSA_OK:
        raise HsaError(name, rc, load().hsa_status_string(rc).decode())


def hsa_status_string(code: int) -> str:
    return load().hsa_status_string(code).decode()


def hsa_workspace_bytes(d: Dims, op: int) -> int:
    cd = d.c()
    return int(load().hsa_workspace_bytes(ctypes.byref(cd), op))


def workspace(d: Dims, op: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace tensor of the size `op` needs (256-byte aligned storage)."""
    n = hsa_workspace_bytes(d, op)
    if n == 0:
        raise HsaError("hsa_workspace_bytes", HSA_ERR_INVALID_ARG, "invalid descriptor")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def hsa_quantize_keys(d: Dims, k_cache, page_table, seq_lens, mode: int, append_from: int, kq,
                      k_scale, ws=None, stream=None) -> None:
    cd = d.c()
    _check("hsa_quantize_keys", load().hsa_quantize_keys(
        ctypes.byref(cd), _p(k_cache), _p(page_table), _p(seq_lens), mode, append_from, _p(kq),
        _p(k_scale), _p(ws), 0 if ws is None else ws.numel(), _stream(stream)))


def hsa_append_kv(d: Dims, k_new, v_new, k_cache, v_cache, kq, k_scale, page_table, seq_lens,
                  stream=None) -> None:
    cd = d.c()
    _check("hsa_append_kv", load().hsa_append_kv(
        ctypes.byref(cd), _p(k_new), _p(v_new), _p(k_cache), _p(v_cache), _p(kq), _p(k_scale),
        _p(page_table), _p(seq_lens), _stream(stream)))


def hsa_score_blocks(d: Dims, q, kq, k_scale, page_table, seq_lens, block_max, tile_max=None,
                     stream=None) -> None:
    cd = d.c()
    _check("hsa_score_blocks", load().hsa_score_blocks(
        ctypes.byref(cd), _p(q), _p(kq), _p(k_scale), _p(page_table), _p(seq_lens),
        _p(block_max), _p(tile_max), _stream(stream)))


def hsa_prune(d: Dims, seq_lens, block_max, tile_max, chunk_idx, n_chunks, block_idx, n_blocks,
              stream=None) -> None:
    cd = d.c()
    _check("hsa_prune", load().hsa_prune(
        ctypes.byref(cd), _p(seq_lens), _p(block_max), _p(tile_max), _p(chunk_idx),
        _p(n_chunks), _p(block_idx), _p(n_blocks), _stream(stream)))


def hsa_select(d: Dims, q, kq, k_scale, page_table, seq_lens, chunk_idx, n_chunks, block_idx,
               n_blocks, ws, stream=None) -> None:
    cd = d.c()
    _check("hsa_select", load().hsa_select(
        ctypes.byref(cd), _p(q), _p(kq), _p(k_scale), _p(page_table), _p(seq_lens),
        _p(chunk_idx), _p(n_chunks), _p(block_idx), _p(n_blocks), _p(ws), ws.numel(),
        _stream(stream)))


def hsa_select_noalloc(d: Dims, q, kq, k_scale, page_table, seq_lens, chunk_idx, n_chunks,
                       block_idx, n_blocks, stream=None) -> None:
    """hsa_select for callers that cannot allocate device memory: the scratch is a fixed
    4 MiB array inside the library (see include/hsa.h for the size limit and the sharing
    rules)."""
    cd = d.c()
    _check("hsa_select_noalloc", load().hsa_select_noalloc(
        ctypes.byref(cd), _p(q), _p(kq), _p(k_scale), _p(page_table), _p(seq_lens),
        _p(chunk_idx), _p(n_chunks), _p(block_idx), _p(n_blocks), _stream(stream)))


def hsa_attend(d: Dims, q, k_cache, v_cache, page_table, seq_lens, block_idx, n_blocks, out,
               lse, ws, stream=None) -> None:
    cd = d.c()
    _check("hsa_attend", load().hsa_attend(
        ctypes.byref(cd), _p(q), _p(k_cache), _p(v_cache), _p(page_table), _p(seq_lens),
        _p(block_idx), _p(n_blocks), _p(out), _p(lse), _p(ws), ws.numel(), _stream(stream)))


def dense_decode(d: Dims, q, k_cache, v_cache, page_table, seq_lens, out, lse, ws,
                 stream=None) -> None:
    cd = d.c()
    _check("dense_decode", load().dense_decode(
        ctypes.byref(cd), _p(q), _p(k_cache), _p(v_cache), _p(page_table), _p(seq_lens),
        _p(out), _p(lse), _p(ws), ws.numel(), _stream(stream)))


def hsa_decode_step(d: Dims, q, k_new, v_new, out, lse, k_cache, v_cache, kq, k_scale,
                    page_table, seq_lens, block_idx, n_blocks, ws, io_on_host: bool = False,
                    stream=None) -> None:
    cd = d.c()
    io = hsa_step_io(_p(q), _p(k_new), _p(v_new), _p(out), _p(lse), 1 if io_on_host else 0)
    _check("hsa_decode_step", load().hsa_decode_step(
        ctypes.byref(cd), ctypes.byref(io), _p(k_cache), _p(v_cache), _p(kq), _p(k_scale),
        _p(page_table), _p(seq_lens), _p(block_idx), _p(n_blocks), _p(ws), ws.numel(),
        _stream(stream)))


class DecodeStep:
    """hsa_decode_step over a fixed set of buffers, for a decode loop that calls it every
    step: the C arguments are marshalled once, so a call costs the C call alone. The
    buffers' contents may change between calls (new q / k_new / v_new, longer seq_lens);
    the buffers themselves must stay alive and in place.

    graph=True: the first call runs the step and then records it into a CUDA graph; every
    later call replays the graph on the current stream (one launch instead of one per
    kernel). The kernels read every input from its buffer, so replays see new contents; the
    descriptor and the buffers are those of the recording."""

    def __init__(self, d: Dims, q, k_new, v_new, out, lse, k_cache, v_cache, kq, k_scale,
                 page_table, seq_lens, block_idx, n_blocks, ws, io_on_host: bool = False,
                 stream=None, graph: bool = False):
        self._keep = (q, k_new, v_new, out, lse, k_cache, v_cache, kq, k_scale, page_table,
                      seq_lens, block_idx, n_blocks, ws)
        self._cd = d.c()
        self._io = hsa_step_io(_p(q), _p(k_new), _p(v_new), _p(out), _p(lse),
                               1 if io_on_host else 0)
        self._fn = load().hsa_decode_step
        self._head = (ctypes.byref(self._cd), ctypes.byref(self._io), _p(k_cache), _p(v_cache),
                      _p(kq), _p(k_scale), _p(page_table), _p(seq_lens), _p(block_idx),
                      _p(n_blocks), _p(ws), ws.numel())
        self._args = self._head + (_stream(stream),)
        self._use_graph = graph
        self._graph = None

    def _run(self, args) -> None:
        rc = self._fn(*args)
        if rc != HSA_OK:
            _check("hsa_decode_step", rc)

    def __call__(self) -> None:
        if self._graph is not None:
            self._graph.replay()
            return
        self._run(self._args)
        if self._use_graph:
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):  # the step's launches, on the recording stream
                self._run(self._head + (_stream(None),))
            self._graph = g


def hsa_decode_step_reuse(d: Dims, q, k_new, v_new, out, lse, k_cache, v_cache, kq, k_scale,
                          page_table, seq_lens, block_idx, n_blocks, ws, io_on_host: bool = False,
                          stream=None) -> None:
    """Append + attend with the selection block_idx / n_blocks of an earlier step."""
    cd = d.c()
    io = hsa_step_io(_p(q), _p(k_new), _p(v_new), _p(out), _p(lse), 1 if io_on_host else 0)
    _check("hsa_decode_step_reuse", load().hsa_decode_step_reuse(
        ctypes.byref(cd), ctypes.byref(io), _p(k_cache), _p(v_cache), _p(kq), _p(k_scale),
        _p(page_table), _p(seq_lens), _p(block_idx), _p(n_blocks), _p(ws), ws.numel(),
        _stream(stream)))


def block_cache(d: Dims, capacity: int):
    """A zeroed device buffer for the GPU block cache (see hsa_block_cache_bytes)."""
    n = load().hsa_block_cache_bytes(ctypes.byref(d.c()), capacity)
    if n == 0:
        raise HsaError("hsa_block_cache_bytes", HSA_ERR_INVALID_ARG, "capacity or shape rejected")
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def block_cache_mass(d: Dims, cache, capacity: int):
    """The block cache's cumulative attention masses: a float32 [num_pages][hkv] view into
    `cache` (see hsa_block_cache_mass)."""
    ptr = load().hsa_block_cache_mass(ctypes.byref(d.c()), _p(cache), capacity)
    if not ptr:
        raise HsaError("hsa_block_cache_mass", HSA_ERR_INVALID_ARG, "shape or capacity rejected")
    off = ptr - cache.data_ptr()
    n = d.num_pages * d.hkv
    return cache[off: off + 4 * n].view(torch.float32).view(d.num_pages, d.hkv)


def hsa_attend_cached(d: Dims, q, k_cache, v_cache, page_table, seq_lens, block_idx, n_blocks,
                      cache, capacity: int, out, lse, ws, stream=None) -> None:
    cd = d.c()
    _check("hsa_attend_cached", load().hsa_attend_cached(
        ctypes.byref(cd), _p(q), _p(k_cache), _p(v_cache), _p(page_table), _p(seq_lens),
        _p(block_idx), _p(n_blocks), _p(cache), capacity, _p(out), _p(lse), _p(ws), ws.numel(),
        _stream(stream)))


def hsa_decode_step_cached(d: Dims, q, k_new, v_new, out, lse, k_cache, v_cache, kq, k_scale,
                           page_table, seq_lens, block_idx, n_blocks, cache, capacity: int, ws,
                           io_on_host: bool = False, stream=None) -> None:
    cd = d.c()
    io = hsa_step_io(_p(q), _p(k_new), _p(v_new), _p(out), _p(lse), 1 if io_on_host else 0)
    _check("hsa_decode_step_cached", load().hsa_decode_step_cached(
        ctypes.byref(cd), ctypes.byref(io), _p(k_cache), _p(v_cache), _p(kq), _p(k_scale),
        _p(page_table), _p(seq_lens), _p(block_idx), _p(n_blocks), _p(cache), capacity, _p(ws),
        ws.numel(), _stream(stream)))


def hsa_decode_step_kernels(d: Dims) -> int:
    """Kernels that hsa_decode_step launches for d (device I/O)."""
    return int(load().hsa_decode_step_kernels(ctypes.byref(d.c())))


class KV8:
    """The 8-bit K/V cache of include/hsa.h: code tensors k and v [num_pages][hkv][16][128],
    both torch.int8 or both torch.float8_e4m3fn (the format follows), and float32 scales
    [num_pages][hkv]. Keeps the tensors; the C struct is built once."""

    def __init__(self, k, v, k_scale, v_scale):
        formats = {torch.int8: 0, torch.float8_e4m3fn: 1}
        for codes, scale in ((k, k_scale), (v, v_scale)):
            if (codes.dtype not in formats or codes.dtype != k.dtype or codes.dim() != 4 or
                    codes.shape != k.shape or scale.shape != k.shape[:2] or
                    scale.dtype != torch.float32 or not codes.is_contiguous() or
                    not scale.is_contiguous()):
                raise HsaError("KV8", HSA_ERR_INVALID_ARG, "shapes, types or layout rejected")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.hkv = k.shape[:2]
        self._c = hsa_kv8(_p(k), _p(v), _p(k_scale), _p(v_scale), formats[k.dtype])
        self._ref = ctypes.byref(self._c)

    @classmethod
    def zeros(cls, d: Dims, fp8: bool = False, device="cuda"):
        """An empty cache for d's pages: int8 codes, or FP8 E4M3 ones."""
        codes = [torch.zeros((d.num_pages, d.hkv, 16, 128), dtype=torch.int8, device=device)
                 for _ in range(2)]
        if fp8:
            codes = [c.view(torch.float8_e4m3fn) for c in codes]
        return cls(*codes, *(torch.zeros((d.num_pages, d.hkv), dtype=torch.float32, device=device)
                             for _ in range(2)))


def _cache(name: str, d: Dims, cache: KV8):
    """The cache's C struct, for a descriptor of its heads and of no more pages than it has (the
    library sees only addresses: it would follow page numbers past the arrays)."""
    if cache.num_pages < d.num_pages or cache.hkv != d.hkv:
        raise HsaError(name, HSA_ERR_INVALID_ARG,
                       f"a cache of {cache.num_pages} pages x {cache.hkv} kv heads, a descriptor "
                       f"of {d.num_pages} x {d.hkv}")
    return cache._ref


def _list(name: str, t) -> Optional[int]:
    """The address of a page table, of lengths, blocks or their numbers."""
    if t is None or type(t) is int:
        return t
    if t.dtype is not torch.int32:
        raise HsaError(name, HSA_ERR_INVALID_ARG, "page tables, lengths and blocks are torch.int32")
    return t.data_ptr()


def _offsets(name: str, d: Dims, cu) -> Optional[int]:
    """The address of the new tokens' offsets: contiguous int32, batch + 1 of them at least."""
    if cu is None or type(cu) is int:
        return cu
    if cu.dtype is not torch.int32 or cu.numel() <= d.batch or not cu.is_contiguous():
        raise HsaError(name, HSA_ERR_INVALID_ARG,
                       "cu_tokens must be contiguous torch.int32, batch + 1 offsets")
    return cu.data_ptr()


def _lists(name: str, d: Dims, cu, page_table, seq_lens):
    """The addresses of new tokens' offsets, page table and lengths."""
    try:  # the lists as they should be, without a call for each
        if (page_table.dtype is torch.int32 and seq_lens.dtype is torch.int32 and
                (cu is None or (cu.dtype is torch.int32 and cu.numel() > d.batch and
                                cu.is_contiguous()))):
            return (cu if cu is None else cu.data_ptr(), page_table.data_ptr(),
                    seq_lens.data_ptr())
    except AttributeError:  # addresses
        pass
    return _offsets(name, d, cu), _list(name, page_table), _list(name, seq_lens)


def _dense(name: str, what: str, t, dtype, n: int) -> Optional[int]:
    """The address of a contiguous tensor of n values (None stays None, an address itself)."""
    if t is None or type(t) is int:
        return t
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        raise HsaError(name, HSA_ERR_INVALID_ARG, f"{what} must be contiguous {dtype}, {n} values")
    return t.data_ptr()


def _heads(name: str, d: Dims, q, out, lse):
    """The addresses of a decode attention's q, out and lse."""
    n = d.batch * d.hq
    f32 = torch.float32
    try:  # the arrays as they should be, without a call for each
        if (q.dtype is torch.bfloat16 and out.dtype is f32 and q.numel() == n * 128 == out.numel()
                and q.is_contiguous() and out.is_contiguous()):
            if lse is None:
                return q.data_ptr(), out.data_ptr(), None
            if lse.dtype is f32 and lse.numel() == n and lse.is_contiguous():
                return q.data_ptr(), out.data_ptr(), lse.data_ptr()
    except AttributeError:  # addresses
        pass
    return (_dense(name, "q", q, torch.bfloat16, n * 128),
            _dense(name, "out", out, f32, n * 128), _dense(name, "lse", lse, f32, n))


def _rows(name: str, t, heads: int):
    """(rows, row stride) of a bf16 tensor [tokens][heads][128] whose rows are contiguous. A
    single row's stride means nothing and may be any: it is given the row's length."""
    shape, stride = t.shape, t.stride()
    if (t.dtype is not torch.bfloat16 or len(stride) != 3 or shape[1] != heads or
            shape[2] != 128 or stride[2] != 1 or (stride[1] != 128 and heads > 1)):
        raise HsaError(name, HSA_ERR_INVALID_ARG, "rows must be bf16 [tokens][heads][128]")
    return shape[0], stride[0] if shape[0] > 1 else heads * 128


def _row_pair(name: str, k, v, heads: int):
    """(rows, k's row stride, v's) of two such tensors of as many rows."""
    shape, ks, vs = k.shape, k.stride(), v.stride()
    if (k.dtype is not torch.bfloat16 or v.dtype is not torch.bfloat16 or shape != v.shape or
            len(ks) != 3 or shape[1] != heads or shape[2] != 128 or ks[2] != 1 or vs[2] != 1 or
            (heads > 1 and (ks[1] != 128 or vs[1] != 128))):
        raise HsaError(name, HSA_ERR_INVALID_ARG,
                       "k and v must be bf16 [tokens][heads][128], of as many rows")
    if shape[0] < 2:
        return shape[0], heads * 128, heads * 128
    return shape[0], ks[0], vs[0]


def hsa_kv8_write(d: Dims, cache: KV8, k_new, v_new, cu_tokens, page_table, seq_lens, ws=None,
                  stream=None) -> None:
    """k_new / v_new: bf16 [total_tokens][hkv][128], rows contiguous (any row stride)."""
    name = "hsa_kv8_write"
    rows, k_stride, v_stride = _row_pair(name, k_new, v_new, d.hkv)
    cu, table, lens = _lists(name, d, cu_tokens, page_table, seq_lens)
    rc = load().hsa_kv8_write(
        ctypes.byref(d.c()), _cache(name, d, cache), k_new.data_ptr(), k_stride, v_new.data_ptr(),
        v_stride, cu, rows, table, lens, _p(ws), 0 if ws is None else ws.numel(), _stream(stream))
    if rc != HSA_OK:
        _check(name, rc)


def hsa_kv8_read(d: Dims, cache: KV8, k_out, v_out, cu_tokens, page_table, seq_lens, ws=None,
                 stream=None) -> None:
    """k_out / v_out: bf16 [total_tokens][hkv][128], rows contiguous (any row stride)."""
    name = "hsa_kv8_read"
    rows, k_stride, v_stride = _row_pair(name, k_out, v_out, d.hkv)
    cu, table, lens = _lists(name, d, cu_tokens, page_table, seq_lens)
    rc = load().hsa_kv8_read(
        ctypes.byref(d.c()), _cache(name, d, cache), k_out.data_ptr(), k_stride, v_out.data_ptr(),
        v_stride, cu, rows, table, lens, _p(ws), 0 if ws is None else ws.numel(), _stream(stream))
    if rc != HSA_OK:
        _check(name, rc)


def hsa_kv8_decode(d: Dims, cache: KV8, q, page_table, seq_lens, out, lse, ws,
                   stream=None) -> None:
    """q: bf16 [batch][hq][128]; out: float32, as q; lse: float32 [batch][hq] or None; all
    contiguous."""
    name = "hsa_kv8_decode"
    q, out, lse = _heads(name, d, q, out, lse)
    _, table, lens = _lists(name, d, None, page_table, seq_lens)
    rc = load().hsa_kv8_decode(ctypes.byref(d.c()), _cache(name, d, cache), q, table, lens, out,
                               lse, _p(ws), ws.numel(), _stream(stream))
    if rc != HSA_OK:
        _check(name, rc)


def hsa_kv8_attend(d: Dims, cache: KV8, q, page_table, seq_lens, block_idx, n_blocks, out, lse,
                   ws, stream=None) -> None:
    """q, out, lse: as hsa_kv8_decode."""
    name = "hsa_kv8_attend"
    q, out, lse = _heads(name, d, q, out, lse)
    _, table, lens = _lists(name, d, None, page_table, seq_lens)
    rc = load().hsa_kv8_attend(ctypes.byref(d.c()), _cache(name, d, cache), q, table, lens,
                               _list(name, block_idx), _list(name, n_blocks), out, lse, _p(ws),
                               ws.numel(), _stream(stream))
    if rc != HSA_OK:
        _check(name, rc)


def hsa_kv8_prefill(d: Dims, cache: KV8, q, cu_tokens, page_table, seq_lens, out, lse, ws,
                    stream=None) -> None:
    """q: bf16 [total_tokens][hq][128], rows contiguous (any row stride); out: bf16, contiguous;
    lse: float32 [total_tokens][hq], contiguous, or None."""
    name = "hsa_kv8_prefill"
    rows, q_stride = _rows(name, q, d.hq)
    if not out.is_contiguous() or out.shape != q.shape or out.dtype is not torch.bfloat16:
        raise HsaError(name, HSA_ERR_INVALID_ARG, "out must be contiguous, as q")
    lse = _dense(name, "lse", lse, torch.float32, rows * d.hq)
    cu, table, lens = _lists(name, d, cu_tokens, page_table, seq_lens)
    rc = load().hsa_kv8_prefill(
        ctypes.byref(d.c()), _cache(name, d, cache), q.data_ptr(), q_stride, cu, rows, table, lens,
        out.data_ptr(), lse, _p(ws), ws.numel(), _stream(stream))
    if rc != HSA_OK:
        _check(name, rc)


def hsa_read_device_error(ws, stream=None) -> int:
    """Reads and clears a workspace's device error word (ws None: the error word of
    hsa_select_noalloc's fixed scratch array)."""
    code = ctypes.c_int32(0)
    _check("hsa_read_device_error", load().hsa_read_device_error(
        _p(ws), _stream(stream), ctypes.byref(code)))
    return int(code.value)
