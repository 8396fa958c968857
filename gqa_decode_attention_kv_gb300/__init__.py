"""Python binding of the GB300 grouped-query decode-attention library.

Argument marshalling only: tensors are passed to the C ABI in
``include/gqa_decode.h`` as raw device pointers with the current CUDA stream;
every step of the computation runs in the library's CUDA kernels. PyTorch
provides device memory and streams. There is no fallback: if the compiled
library is missing, loading raises.

Entry points (same names as the C ABI, without the ``gqa_`` prefix where it
would repeat the module name):

* ``kv_append``            -- write the new token(s) of every sequence into the paged cache
* ``gqa_decode``           -- grouped-query decode attention over the paged cache
                              (one or T causal new tokens per sequence, optional
                              sliding window)
* ``kv_append_varlen``     -- the same for a different number of new tokens per sequence
* ``rope_table``           -- (cos, sin) of every position and pair, for the two calls below
* ``qk_norm_rope``         -- per-head norm of queries and keys and their rotation, one pass
* ``qk_norm_rope_append``  -- the same with K and V written into the paged cache
* ``kv_pages_reserve``, ``kv_pages_fork``, ``kv_pages_free``, ``kv_pages_trim``,
  ``kv_pages_compact``     -- the pages of a pool: counts and block tables kept in step on the device
* ``kv_copy_pages``        -- the page copies a fork or compaction asks for, in every layer's cache
* ``gqa_prefill``          -- causal attention of prompts (any length) over the paged cache
* ``decode_workspace_size``-- workspace bytes ``gqa_decode`` needs
* ``kv_pool_elements``     -- elements a pool of ``num_blocks`` blocks holds (K and V)
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import os
import threading
from typing import Optional

import torch

from . import build as _build

BLOCK_SIZE = 16
DTYPE_CODE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.int8: 3,
              torch.float8_e4m3fn: 4}

_DEV_DTYPES = frozenset(DTYPE_CODE) | {torch.uint8}

GQA_DEVERR_BLOCK_INDEX = 1
GQA_DEVERR_CONTEXT_LEN = 2
GQA_DEVERR_POSITION = 4
GQA_DEVERR_TIMEOUT = 8
GQA_DEVERR_ROW = 16
GQA_DEVERR_NO_PAGES = 32
GQA_DEVERR_REF_COUNT = 64

KERNEL_AUTO, KERNEL_MMA, KERNEL_FMA = 0, 1, 2
GQA_DTYPE_I4 = 5
GQA_DTYPE_I4_KC = 6


class GqaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class KVCacheDesc(ctypes.Structure):
    """Mirror of gqa_kv_cache_t."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("num_blocks", ctypes.c_int64), ("num_kv_heads", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("stride_block", ctypes.c_int64),
                ("stride_head", ctypes.c_int64), ("stride_token", ctypes.c_int64),
                ("k_residual", ctypes.c_void_p), ("residual_rows", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class DecodeOpts(ctypes.Structure):
    """Mirror of gqa_decode_opts_t."""
    _fields_ = [("tokens_per_seq", ctypes.c_int32), ("sliding_window", ctypes.c_int32),
                ("kernel", ctypes.c_int32), ("max_warps", ctypes.c_int32),
                ("min_blocks_per_warp", ctypes.c_int32), ("row_layout", ctypes.c_int32),
                ("event_main_begin", ctypes.c_void_p), ("event_main_end", ctypes.c_void_p)]


class NormRopeDesc(ctypes.Structure):
    """Mirror of gqa_norm_rope_t."""
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("rope", ctypes.c_void_p),
                ("weight_dtype", ctypes.c_int32), ("eps", ctypes.c_float), ("rope_rows", ctypes.c_int32),
                ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return _build.LIB_PATH


def load() -> ctypes.CDLL:
    """Load the compiled library (build it first with ``build.build()``)."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB_PATH
            if not os.path.exists(path):
                raise RuntimeError(f"CUDA library not built: {path} is missing "
                                   "(run gqa_decode_attention_kv_gb300.build.build())")
            lib = ctypes.CDLL(path)
            vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
            lib.gqa_status_string.argtypes = [ctypes.c_int]
            lib.gqa_status_string.restype = ctypes.c_char_p
            lib.gqa_version.argtypes = []
            lib.gqa_version.restype = ctypes.c_int
            lib.gqa_kv_pool_elements.argtypes = [i64, i32, i32]
            lib.gqa_kv_pool_elements.restype = i64
            lib.gqa_kv_append.argtypes = [ctypes.POINTER(KVCacheDesc), vp, vp, i32, vp, i32, vp,
                                          i32, i32, vp, vp]
            lib.gqa_kv_append.restype = ctypes.c_int
            lib.gqa_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
            lib.gqa_decode_workspace_size.restype = ctypes.c_size_t
            lib.gqa_decode.argtypes = [ctypes.POINTER(KVCacheDesc), vp, i32, i32, vp, i32, vp, i32,
                                       ctypes.c_float, vp, i32, vp, ctypes.c_size_t,
                                       ctypes.POINTER(DecodeOpts), vp, vp]
            lib.gqa_decode.restype = ctypes.c_int
            lib.gqa_decode_sinks.argtypes = [*lib.gqa_decode.argtypes[:-2], i32, vp, vp]
            lib.gqa_decode_sinks.restype = ctypes.c_int
            lib.gqa_decode_noalloc.argtypes = [ctypes.POINTER(KVCacheDesc), vp, i32, i32, vp, i32,
                                               vp, i32, ctypes.c_float, vp, i32,
                                               ctypes.POINTER(DecodeOpts), vp, vp]
            lib.gqa_decode_noalloc.restype = ctypes.c_int
            lib.gqa_decode_noalloc_sinks.argtypes = [*lib.gqa_decode_noalloc.argtypes[:-2], i32, vp, vp]
            lib.gqa_decode_noalloc_sinks.restype = ctypes.c_int
            lib.gqa_kv_append_varlen.argtypes = [ctypes.POINTER(KVCacheDesc), vp, vp, i32, vp, i32, vp,
                                                 i32, vp, i32, vp, vp]
            lib.gqa_kv_append_varlen.restype = ctypes.c_int
            lib.gqa_prefill.argtypes = [ctypes.POINTER(KVCacheDesc), vp, i32, i32, vp, i32, vp, i32, vp,
                                        i32, ctypes.c_float, i32, vp, i32, i32, vp, vp]
            lib.gqa_prefill.restype = ctypes.c_int
            lib.gqa_prefill_sinks.argtypes = [*lib.gqa_prefill.argtypes[:12], i32, i64, *lib.gqa_prefill.argtypes[12:]]
            lib.gqa_prefill_sinks.restype = ctypes.c_int
            lib.gqa_kv_pages_workspace_size.argtypes = [i64, i32]
            lib.gqa_kv_pages_workspace_size.restype = ctypes.c_size_t
            lib.gqa_kv_pages_reserve.argtypes = [vp, i64, vp, i32, vp, vp, i32, i32, vp, ctypes.c_size_t, vp, vp]
            lib.gqa_kv_pages_fork.argtypes = [vp, i64, vp, i32, i32, vp, vp, vp, i32, vp, vp, vp, vp, ctypes.c_size_t,
                                              vp, vp]
            lib.gqa_kv_pages_free.argtypes = [vp, i64, vp, i32, i32, vp, vp, i32, vp, vp]
            lib.gqa_kv_pages_trim.argtypes = [vp, i64, vp, i32, vp, i32, i32, i32, vp, vp]
            lib.gqa_kv_pages_compact.argtypes = [vp, i64, vp, i32, i32, vp, i32, vp, vp, ctypes.c_size_t, vp, vp]
            lib.gqa_kv_copy_pages.argtypes = [ctypes.POINTER(KVCacheDesc), i32, vp, vp, i32, vp, i32, vp, vp]
            for f in (lib.gqa_kv_pages_reserve, lib.gqa_kv_pages_fork, lib.gqa_kv_pages_free, lib.gqa_kv_pages_trim,
                      lib.gqa_kv_pages_compact, lib.gqa_kv_copy_pages):
                f.restype = ctypes.c_int
            lib.gqa_rope_table.argtypes = [vp, i32, i32, ctypes.c_double, vp]
            lib.gqa_rope_table.restype = ctypes.c_int
            lib.gqa_qk_norm_rope.argtypes = [ctypes.POINTER(NormRopeDesc), vp, i64, vp, i32, vp, i64, vp, i32, i32,
                                             i32, i64, vp, vp, vp]
            lib.gqa_qk_norm_rope.restype = ctypes.c_int
            lib.gqa_qk_norm_rope_append.argtypes = [ctypes.POINTER(KVCacheDesc), ctypes.POINTER(NormRopeDesc), vp, i64,
                                                    vp, i32, vp, i64, vp, i64, i32, i64, vp, i32, vp, i32, vp, vp, i32,
                                                    vp, vp]
            lib.gqa_qk_norm_rope_append.restype = ctypes.c_int
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().gqa_status_string(int(status)).decode()


def version() -> int:
    return int(load().gqa_version())


def kv_pool_elements(num_blocks: int, num_kv_heads: int, head_dim: int) -> int:
    return int(load().gqa_kv_pool_elements(num_blocks, num_kv_heads, head_dim))


@dataclasses.dataclass
class PagedKVCache:
    """Device tensors of one paged KV cache plus their element strides.

    Default layout is the pool ``[num_blocks, K, 16, d]``; any layout whose
    element of (block p, kv-head g, slot s, dim i) is at
    ``p*stride_block + g*stride_head + s*stride_token + i`` works."""
    k: torch.Tensor
    v: torch.Tensor
    num_blocks: int
    num_kv_heads: int
    head_dim: int
    stride_block: int
    stride_head: int
    stride_token: int
    k_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None
    dtype_code: Optional[int] = None   # set for storage the tensor dtype does not name (int4)
    k_residual: Optional[torch.Tensor] = None   # KIVI-style cache: fp32 [rows, K, 16, d]

    @staticmethod
    def allocate(num_blocks: int, num_kv_heads: int, head_dim: int, dtype,
                 device="cuda", residual_rows: int = 0) -> "PagedKVCache":
        """dtype: a torch dtype; "int4" for two 4-bit codes per byte (uint8
        storage [num_blocks, K, 16, d/2]; strides still count 4-bit elements);
        "int4kc" for the same codes with K scaled per (block, kv-head, channel)
        (k_scale [num_blocks, K, d]) and a zeroed fp32 residual of
        ``residual_rows`` sequences."""
        int4 = dtype in ("int4", "int4kc")
        kc = dtype == "int4kc"
        shape = (num_blocks, num_kv_heads, BLOCK_SIZE, head_dim // 2 if int4 else head_dim)
        k = torch.empty(shape, dtype=torch.uint8 if int4 else dtype, device=device)
        v = torch.empty_like(k)
        ks = vs = res = None
        if int4 or dtype in (torch.int8, torch.float8_e4m3fn):
            vs = torch.empty((num_blocks, num_kv_heads, BLOCK_SIZE), dtype=torch.float16, device=device)
            ks = torch.empty((num_blocks, num_kv_heads, head_dim), dtype=torch.float16,
                             device=device) if kc else torch.empty_like(vs)
        if kc:
            res = torch.zeros((residual_rows, num_kv_heads, BLOCK_SIZE, head_dim), dtype=torch.float32,
                              device=device)
        code = GQA_DTYPE_I4_KC if kc else GQA_DTYPE_I4 if int4 else None
        return PagedKVCache(k, v, num_blocks, num_kv_heads, head_dim,
                            num_kv_heads * BLOCK_SIZE * head_dim, BLOCK_SIZE * head_dim, head_dim,
                            ks, vs, code, res)

    @property
    def dtype(self) -> torch.dtype:
        return self.k.dtype

    def desc(self) -> KVCacheDesc:
        return KVCacheDesc(
            self.k.data_ptr(), self.v.data_ptr(),
            self.k_scale.data_ptr() if self.k_scale is not None else None,
            self.v_scale.data_ptr() if self.v_scale is not None else None,
            self.num_blocks, self.num_kv_heads, BLOCK_SIZE, self.head_dim,
            self.dtype_code if self.dtype_code is not None else DTYPE_CODE[self.k.dtype],
            self.stride_block, self.stride_head, self.stride_token,
            self.k_residual.data_ptr() if self.k_residual is not None else None,
            int(self.k_residual.shape[0]) if self.k_residual is not None else 0, 0)


# The current stream's handle without a Stream object around it: building one takes
# 2.9 us a call on the Grace cores, the handle alone 0.1 us.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_ptr(stream) -> Optional[int]:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A result of a call on ``stream``, allocated there: memory another stream just
    freed may still be in use on that one."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _dev(t: Optional[torch.Tensor], name: str, index: bool = False, optional: bool = False):
    """Device pointer of a tensor the library reads or writes as a packed array.

    The C ABI sees a bare pointer, so what it cannot check is checked here:
    the tensor must be contiguous, an index array must be int32, and the memory
    must be on a CUDA device."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if t.is_cuda and t.is_contiguous() and (t.dtype is torch.int32 if index else t.dtype in _DEV_DTYPES):
        return t.data_ptr()
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (the library reads it as a packed array)")
    if index and t.dtype != torch.int32:
        raise ValueError(f"{name} must be int32, not {t.dtype}")
    if not index and t.dtype not in DTYPE_CODE and t.dtype != torch.uint8:
        raise ValueError(f"{name} has unsupported dtype {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.data_ptr()


def _on_cache_device(cache: "PagedKVCache", **tensors):
    """Every array must sit on the cache's device, and that device must be the
    current one: the library launches on the current device and reads the
    pointers it is given there."""
    dev = cache.k.device
    if dev.type == "cuda" and dev.index != torch.cuda.current_device():
        raise ValueError(f"the cache is on {dev} but the current device is cuda:{torch.cuda.current_device()}")
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the cache on {dev}")


def _check_table_and_lens(block_tables: torch.Tensor, lens: torch.Tensor, batch: int, lens_name: str,
                          lens_min: int):
    if block_tables.dim() != 2 or block_tables.shape[0] < batch:
        raise ValueError(f"block_tables must be [>= {batch}, max_blocks], not {tuple(block_tables.shape)}")
    if lens.dim() != 1 or lens.numel() < lens_min:
        raise ValueError(f"{lens_name} must be 1-D with >= {lens_min} entries, not {tuple(lens.shape)}")


def _check_query(cache: "PagedKVCache", q: torch.Tensor, dims: tuple):
    if q.dim() not in dims:
        raise ValueError(f"q must have {' or '.join(str(x) for x in dims)} dims, not {q.dim()}")
    H, d = int(q.shape[-2]), int(q.shape[-1])
    if d != cache.head_dim:
        raise ValueError(f"q's head_dim {d} differs from the cache's {cache.head_dim}")
    if H % cache.num_kv_heads:
        raise ValueError(f"{H} query heads are not a multiple of {cache.num_kv_heads} kv-heads")


def _check_out(q: torch.Tensor, out: Optional[torch.Tensor]):
    if out is not None and tuple(out.shape) != tuple(q.shape):
        raise ValueError(f"out must have q's shape {tuple(q.shape)}, not {tuple(out.shape)}")


def _check_new_rows(cache: "PagedKVCache", k_new: torch.Tensor, v_new: torch.Tensor, dims: tuple):
    if k_new.dim() not in dims or tuple(v_new.shape) != tuple(k_new.shape):
        raise ValueError(f"k_new and v_new must share one shape with {dims} dims, "
                         f"not {tuple(k_new.shape)} and {tuple(v_new.shape)}")
    if tuple(k_new.shape[-2:]) != (cache.num_kv_heads, cache.head_dim):
        raise ValueError(f"new rows end in {tuple(k_new.shape[-2:])}, the cache's heads and "
                         f"head_dim are {(cache.num_kv_heads, cache.head_dim)}")


def _check(status: int, where: str):
    if status != 0:
        raise GqaError(status, where)


def kv_append(cache: PagedKVCache, k_new: torch.Tensor, v_new: torch.Tensor,
              block_tables: torch.Tensor, positions: torch.Tensor,
              err: Optional[torch.Tensor] = None, stream=None) -> None:
    """Write k_new/v_new [B, K, d] (one token) or [B, T, K, d] (T tokens) at
    positions positions[b] .. positions[b]+T-1 of each sequence's paged cache."""
    T = 1 if k_new.dim() == 3 else int(k_new.shape[1])
    args = (_dev(k_new, "k_new"), _dev(v_new, "v_new"), _dev(block_tables, "block_tables", True),
            _dev(positions, "positions", True), _dev(err, "err", True, True))
    _check_new_rows(cache, k_new, v_new, (3, 4))
    B = int(positions.shape[0]) if positions.dim() == 1 else -1
    if B < 0 or int(k_new.shape[0]) != B:
        raise ValueError(f"positions must be [B] with B = k_new.shape[0] = {int(k_new.shape[0])}")
    _check_table_and_lens(block_tables, positions, B, "positions", B)
    _on_cache_device(cache, k_new=k_new, v_new=v_new, block_tables=block_tables,
                     positions=positions, err=err)
    desc = cache.desc()
    st = load().gqa_kv_append(ctypes.byref(desc), args[0], args[1], DTYPE_CODE[k_new.dtype], args[2],
                              int(block_tables.shape[1]), args[3], int(positions.shape[0]),
                              T, args[4], _stream_ptr(stream))
    _check(st, "gqa_kv_append")


def decode_workspace_size(batch: int, num_heads: int, num_kv_heads: int, head_dim: int,
                          device: int = -1, tokens_per_seq: int = 1) -> int:
    return int(load().gqa_decode_workspace_size(batch, num_heads, num_kv_heads, head_dim,
                                                tokens_per_seq, device))


_workspace_size_of = functools.lru_cache(maxsize=256)(decode_workspace_size)   # a shape's size does not change


class _ThreadScratch(threading.local):
    """Workspaces of the calls of one host thread, per (device, stream). A call queues
    kernels that hand their results on through its workspace, and the interpreter may
    change threads between two of them: threads on one stream must not share it."""

    def __init__(self):
        self.decode: dict = {}
        self.pages: dict = {}


_thread_scratch = _ThreadScratch()


def _capturing(stream) -> bool:
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _scratch(cache: dict, need: int, idx: int, stream, zero: bool) -> torch.Tensor:
    """``need`` bytes of device scratch: kept in the thread's ``cache`` per (device,
    stream), or a captured call's own."""
    capturing = _capturing(stream)
    key = (idx, stream.cuda_stream if stream is not None else
           _raw_stream(idx) if _raw_stream is not None else
           torch.cuda.current_stream(torch.device("cuda", idx)).cuda_stream)
    buf = None if capturing else cache.get(key)
    if buf is None or buf.numel() < need:
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(torch.device("cuda", idx))):
            buf = torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", idx))
            if zero:                           # a captured call zeroes at every replay: the counter's header alone
                (buf[:256] if capturing else buf).zero_()
        if not capturing:
            cache[key] = buf
    return buf


def workspace_for(batch: int, num_heads: int, num_kv_heads: int, head_dim: int,
                  device: torch.device, tokens_per_seq: int = 1, stream=None) -> torch.Tensor:
    """A cached, zero-initialised device workspace large enough for this shape,
    one per (host thread, device, stream): a thread's calls on one stream run in
    order, so they may share it; calls of other threads or on other streams get
    others. The buffer is allocated on that stream, so a larger one replacing it
    is ordered after the calls already queued there. A call that is being captured
    gets one of its own from the graph's memory, zeroed by the graph: graphs
    captured on one stream may be replayed on several, in any order. (The zeroing
    is a node of the graph: 16 decodes in a row take 0.4 to 0.9 us more each than
    with a workspace of the caller's.)"""
    dev = torch.device(device)
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    need = _workspace_size_of(batch, num_heads, num_kv_heads, head_dim, idx, tokens_per_seq)
    if need == 0:
        raise ValueError("no workspace size for this shape")
    # zero-filled once: the library keeps its run-time work counter at zero between calls
    return _scratch(_thread_scratch.decode, need, idx, stream, zero=True)


def gqa_decode(cache: PagedKVCache, q: torch.Tensor, block_tables: torch.Tensor,
               context_lens: torch.Tensor, scale: float, out: Optional[torch.Tensor] = None,
               out_dtype: torch.dtype = torch.float32, workspace: Optional[torch.Tensor] = None,
               kernel: int = KERNEL_AUTO, max_warps: int = 0, min_blocks_per_warp: int = 0,
               events: Optional[tuple] = None, err: Optional[torch.Tensor] = None,
               stream=None, window: int = 0, row_layout: int = 0, sinks: int = 0) -> torch.Tensor:
    """out[b,h] = softmax(scale * q[b,h] . K_g^T) V_g over context_lens[b] cached tokens.

    q is [B, H, d] (one new token per sequence) or [B, T, H, d] (T new tokens,
    causal among themselves); ``window`` > 0 keeps each query's last ``window``
    positions, and with ``sinks`` > 0 the sequence's first ``sinks`` as well
    (without a window, ``sinks`` changes nothing). ``out`` has q's shape."""
    T = 1 if q.dim() == 3 else int(q.shape[1])
    B, H, d = q.shape[0], q.shape[-2], q.shape[-1]
    qp, tp, lp = _dev(q, "q"), _dev(block_tables, "block_tables", True), _dev(context_lens, "context_lens", True)
    ep = _dev(err, "err", True, True)
    _check_query(cache, q, (3, 4))
    _check_table_and_lens(block_tables, context_lens, B, "context_lens", B)
    _check_out(q, out)
    _on_cache_device(cache, q=q, block_tables=block_tables, context_lens=context_lens, out=out,
                     workspace=workspace, err=err)
    if out is None:
        out = _empty(q.shape, out_dtype, q.device, stream)
    if workspace is None:
        workspace = workspace_for(B, H, cache.num_kv_heads, d, q.device, T, stream)
    op, wp = _dev(out, "out"), _dev(workspace, "workspace")
    opts = DecodeOpts(T, window, kernel, max_warps, min_blocks_per_warp, row_layout, None, None)
    if events is not None:
        opts.event_main_begin = events[0].cuda_event
        opts.event_main_end = events[1].cuda_event
    desc = cache.desc()
    st = load().gqa_decode_sinks(ctypes.byref(desc), qp, DTYPE_CODE[q.dtype], H, tp,
                                 int(block_tables.shape[1]), lp, B, float(scale),
                                 op, DTYPE_CODE[out.dtype], wp, workspace.numel() * workspace.element_size(),
                                 ctypes.byref(opts), int(sinks), ep, _stream_ptr(stream))
    _check(st, "gqa_decode")
    return out


def gqa_decode_noalloc(cache: PagedKVCache, q: torch.Tensor, block_tables: torch.Tensor,
                       context_lens: torch.Tensor, scale: float, out: Optional[torch.Tensor] = None,
                       out_dtype: torch.dtype = torch.float32, kernel: int = KERNEL_AUTO,
                       err: Optional[torch.Tensor] = None, stream=None,
                       window: int = 0, sinks: int = 0) -> torch.Tensor:
    """gqa_decode with the library's built-in scratch instead of a workspace.

    For callers that may not allocate device memory; the output tensor is still
    the caller's (pass ``out`` to avoid even that allocation here). Calls on
    different streams or of different host threads share one scratch array and race:
    serialise them."""
    T = 1 if q.dim() == 3 else int(q.shape[1])
    B, H, d = q.shape[0], q.shape[-2], q.shape[-1]
    qp, tp, lp = _dev(q, "q"), _dev(block_tables, "block_tables", True), _dev(context_lens, "context_lens", True)
    ep = _dev(err, "err", True, True)
    _check_query(cache, q, (3, 4))
    _check_table_and_lens(block_tables, context_lens, B, "context_lens", B)
    _check_out(q, out)
    _on_cache_device(cache, q=q, block_tables=block_tables, context_lens=context_lens, out=out, err=err)
    if out is None:
        out = _empty(q.shape, out_dtype, q.device, stream)
    op = _dev(out, "out")
    opts = DecodeOpts(T, window, kernel, 0, 0, 0, None, None)
    desc = cache.desc()
    st = load().gqa_decode_noalloc_sinks(ctypes.byref(desc), qp, DTYPE_CODE[q.dtype], H,
                                         tp, int(block_tables.shape[1]),
                                         lp, B, float(scale), op,
                                         DTYPE_CODE[out.dtype], ctypes.byref(opts), int(sinks), ep,
                                         _stream_ptr(stream))
    _check(st, "gqa_decode_noalloc")
    return out


def kv_append_varlen(cache: PagedKVCache, k_new: torch.Tensor, v_new: torch.Tensor,
                     token_start: torch.Tensor, max_new_tokens: int, block_tables: torch.Tensor,
                     positions: torch.Tensor, err: Optional[torch.Tensor] = None, stream=None) -> None:
    """Write rows token_start[b] .. token_start[b+1]-1 of k_new/v_new [total, K, d] at
    positions positions[b], positions[b]+1, ... of sequence b."""
    args = (_dev(k_new, "k_new"), _dev(v_new, "v_new"), _dev(token_start, "token_start", True),
            _dev(block_tables, "block_tables", True), _dev(positions, "positions", True),
            _dev(err, "err", True, True))
    _check_new_rows(cache, k_new, v_new, (3,))
    B = int(positions.shape[0]) if positions.dim() == 1 else -1
    if B < 0:
        raise ValueError("positions must be 1-D")
    _check_table_and_lens(block_tables, positions, B, "positions", B)
    if token_start.dim() != 1 or token_start.numel() < B + 1:
        raise ValueError(f"token_start must be 1-D with >= {B + 1} entries")
    _on_cache_device(cache, k_new=k_new, v_new=v_new, token_start=token_start,
                     block_tables=block_tables, positions=positions, err=err)
    desc = cache.desc()
    st = load().gqa_kv_append_varlen(ctypes.byref(desc), args[0], args[1],
                                     DTYPE_CODE[k_new.dtype], args[2], int(max_new_tokens),
                                     args[3], int(block_tables.shape[1]), args[4],
                                     int(positions.shape[0]), args[5], _stream_ptr(stream))
    _check(st, "gqa_kv_append_varlen")


def rope_table(positions: int, rotary_dim: int, base: float = 10000.0, device="cuda", stream=None) -> torch.Tensor:
    """fp32 [positions, rotary_dim/2, 2]: cos and sin of p * base^(-2i/rotary_dim),
    the angles in fp64. Made once and kept; for another rule of angles pass a
    table of your own to the calls below."""
    if positions < 0 or rotary_dim <= 0 or rotary_dim % 2:
        raise ValueError(f"no table of {positions} positions and rotary_dim {rotary_dim}")
    s = stream if stream is not None else torch.cuda.current_stream(torch.device(device))
    with torch.cuda.stream(s):
        table = torch.empty((positions, rotary_dim // 2, 2), dtype=torch.float32, device=device)
        _check(load().gqa_rope_table(table.data_ptr(), int(positions), int(rotary_dim), float(base), s.cuda_stream),
               "gqa_rope_table")
    return table


_ROW_DTYPES = frozenset((torch.float32, torch.float16, torch.bfloat16))


def _token_rows(t: torch.Tensor, name: str, like: torch.Tensor, heads: Optional[int] = None):
    """(pointer, elements between tokens) of rows [..., heads, d] whose heads are
    contiguous and whose tokens are evenly spaced (a view into a fused projection)."""
    if t.dim() == 3 and like.dim() == 3:               # the usual case: [tokens, heads, d]
        n, H, d = t.shape
        sn, sh, sd = t.stride()
        if (n == like.shape[0] and d == like.shape[2] and t.dtype is like.dtype and t.dtype in _ROW_DTYPES and sd == 1
                and sh == d and sn >= H * d and (heads is None or H == heads) and t.is_cuda):
            return t.data_ptr(), sn if n > 1 else H * d          # one token has no next one
    if t.dim() not in (3, 4) or tuple(t.shape[:-2]) != tuple(like.shape[:-2]) or t.shape[-1] != like.shape[-1]:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, which does not go with q's {tuple(like.shape)}")
    if heads is not None and t.shape[-2] != heads:
        raise ValueError(f"{name} has {t.shape[-2]} heads, not {heads}")
    if t.dtype not in _ROW_DTYPES or t.dtype != like.dtype:
        raise ValueError(f"{name} must have q's dtype, one of float32, float16, bfloat16, not {t.dtype}")
    H, d = int(t.shape[-2]), int(t.shape[-1])
    st = t.stride()
    if t.numel() and (st[-1] != 1 or (H > 1 and st[-2] != d)):
        raise ValueError(f"{name}'s heads must be contiguous, not strided by {st}")
    if t.dim() == 4 and t.shape[0] > 1 and t.shape[1] > 1 and st[0] != t.shape[1] * st[1]:
        raise ValueError(f"{name}'s tokens must be evenly spaced, not strided by {st}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    tokens = 1
    for n in t.shape[:-2]:
        tokens *= int(n)
    if tokens <= 1:
        stride = H * d
    else:
        stride = st[-3] if t.shape[-3] > 1 else st[0]
    if tokens and stride < H * d:
        raise ValueError(f"{name}'s tokens overlap (strides {st})")
    return t.data_ptr(), int(stride)


def _norm_rope_desc(q, rope, q_weight, k_weight, eps, interleaved) -> NormRopeDesc:
    d = q.shape[-1]
    pointers, code = [None, None], 0
    for i, w in enumerate((q_weight, k_weight)):
        if w is None:
            continue
        name = ("q_weight", "k_weight")[i]
        if w.dim() != 1 or w.shape[0] != d:
            raise ValueError(f"{name} must be [{d}], not {tuple(w.shape)}")
        if w.dtype not in _ROW_DTYPES:
            raise ValueError(f"{name} has unsupported dtype {w.dtype}")
        pointers[i], code = _dev(w, name), DTYPE_CODE[w.dtype]
    if q_weight is not None and k_weight is not None and q_weight.dtype != k_weight.dtype:
        raise ValueError("q_weight and k_weight must have one dtype")
    table, rows, rotary = None, 0, 0
    if rope is not None:
        if rope.dim() != 3 or rope.shape[2] != 2 or rope.dtype != torch.float32:
            raise ValueError(f"rope must be float32 [positions, rotary_dim/2, 2], not {rope.dtype} {tuple(rope.shape)}")
        table, rows, rotary = _dev(rope, "rope"), rope.shape[0], 2 * rope.shape[1]
    return NormRopeDesc(pointers[0], pointers[1], table, code, eps, rows, rotary, 1 if interleaved else 0, 0)


def _same_or_apart(out: torch.Tensor, src: torch.Tensor, name: str, same: bool = True):
    """out may be memory that src does not touch or, with ``same``, src itself (dense)."""
    if out.untyped_storage().data_ptr() != src.untyped_storage().data_ptr() or not out.numel() or not src.numel():
        return
    if same and out.data_ptr() == src.data_ptr() and src.is_contiguous():
        return
    end = lambda t: t.data_ptr() + (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()  # noqa: E731
    if out.data_ptr() < end(src) and src.data_ptr() < end(out):
        raise ValueError(f"{name} overlaps an input without being its own")


def _q_out(q: torch.Tensor, q_out: Optional[torch.Tensor], name: str, stream, *others: torch.Tensor) -> torch.Tensor:
    if q_out is None:
        return _empty(q.shape, q.dtype, q.device, stream)
    if tuple(q_out.shape) != tuple(q.shape) or q_out.dtype != q.dtype:
        raise ValueError(f"{name} must have the input's shape and dtype, not {tuple(q_out.shape)} {q_out.dtype}")
    _dev(q_out, name)
    _same_or_apart(q_out, q, name)
    for t in others:
        _same_or_apart(q_out, t, name, False)
    return q_out


def _on_one_device(**tensors):
    """Every array on the current CUDA device."""
    cur = torch.device("cuda", torch.cuda.current_device())
    for name, t in tensors.items():
        if t is not None and t.device != cur:
            raise ValueError(f"{name} is on {t.device}, the current device is {cur}")


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: Optional[torch.Tensor] = None,
                 rope: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, interleaved: bool = False,
                 q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                 err: Optional[torch.Tensor] = None, stream=None):
    """Norm of every head of q [..., H, d] and k [..., K, d] (x / sqrt(mean(x^2) + eps)
    * weight; no weight, no norm), then the rotation by each token's position.

    ``rope`` is a table as ``rope_table`` makes it, ``positions`` int32 with one
    entry per token. q and k may be views into one fused projection; the dense
    results (q_out, k_out) may be q and k themselves where those are dense."""
    qp, qs = _token_rows(q, "q", q)
    kp, ks = _token_rows(k, "k", q)
    desc = _norm_rope_desc(q, rope, q_weight, k_weight, eps, interleaved)
    tokens = q.numel() // max(1, int(q.shape[-2]) * int(q.shape[-1]))
    pp = _dev(positions, "positions", True, rope is None)
    if positions is not None and positions.numel() != tokens:
        raise ValueError(f"positions must have {tokens} entries, not {positions.numel()}")
    ep = _dev(err, "err", True, True)
    _on_one_device(q=q, k=k, positions=positions, rope=rope, q_weight=q_weight, k_weight=k_weight, q_out=q_out,
                   k_out=k_out, err=err)
    q_out, k_out = _q_out(q, q_out, "q_out", stream, k), _q_out(k, k_out, "k_out", stream, q)
    _same_or_apart(k_out, q_out, "k_out", False)
    st = load().gqa_qk_norm_rope(ctypes.byref(desc), qp, qs, q_out.data_ptr(), int(q.shape[-2]), kp, ks,
                                 k_out.data_ptr(), int(k.shape[-2]), int(q.shape[-1]), DTYPE_CODE[q.dtype], tokens, pp,
                                 ep, _stream_ptr(stream))
    _check(st, "gqa_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_append(cache: PagedKVCache, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                        block_tables: torch.Tensor, positions: torch.Tensor, rope: Optional[torch.Tensor] = None,
                        q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                        eps: float = 1e-6, interleaved: bool = False, token_start: Optional[torch.Tensor] = None,
                        max_new_tokens: Optional[int] = None, rope_positions: Optional[torch.Tensor] = None,
                        q_out: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """``qk_norm_rope`` with the append in the same pass: returns q_out, and K and V
    are in the cache. Tokens as in ``kv_append`` (q [B, H, d] or [B, T, H, d], new
    tokens at positions[b], ...) or, with ``token_start`` [B+1] and
    ``max_new_tokens``, as in ``kv_append_varlen`` (q [total, H, d]). A token is
    turned by its position in the cache, or by ``rope_positions`` [tokens].
    A KIVI-style cache takes ``qk_norm_rope`` and ``kv_append`` instead."""
    _check_query(cache, q, (3,) if token_start is not None else (3, 4))
    qp, qs = _token_rows(q, "q", q)
    kp, ks = _token_rows(k, "k", q, cache.num_kv_heads)
    vp, vs = _token_rows(v, "v", q, cache.num_kv_heads)
    desc = _norm_rope_desc(q, rope, q_weight, k_weight, eps, interleaved)
    tp, pp = _dev(block_tables, "block_tables", True), _dev(positions, "positions", True)
    sp, rp = _dev(token_start, "token_start", True, True), _dev(rope_positions, "rope_positions", True, True)
    ep = _dev(err, "err", True, True)
    B = int(positions.shape[0]) if positions.dim() == 1 else -1
    tokens = int(q.shape[0]) * (int(q.shape[1]) if q.dim() == 4 else 1)
    if token_start is not None:
        if B < 0 or token_start.dim() != 1 or token_start.numel() != B + 1:
            raise ValueError("token_start must be [B + 1] and positions [B]")
        if max_new_tokens is None:
            raise ValueError("max_new_tokens is required with token_start")
        T = int(max_new_tokens)
    else:
        T = 1 if q.dim() == 3 else int(q.shape[1])
        if B != int(q.shape[0]):
            raise ValueError(f"positions must be [B] with B = q.shape[0] = {int(q.shape[0])}")
        if max_new_tokens is not None and int(max_new_tokens) != T:
            raise ValueError(f"q holds {T} tokens per sequence, max_new_tokens is {max_new_tokens}")
    _check_table_and_lens(block_tables, positions, B, "positions", B)
    if rope_positions is not None and rope_positions.numel() != tokens:
        raise ValueError(f"rope_positions must have {tokens} entries, not {rope_positions.numel()}")
    _on_cache_device(cache, q=q, k=k, v=v, block_tables=block_tables, positions=positions, rope=rope,
                     q_weight=q_weight, k_weight=k_weight, token_start=token_start, rope_positions=rope_positions,
                     q_out=q_out, err=err)
    q_out = _q_out(q, q_out, "q_out", stream, k, v)
    if tokens == 0 or T == 0:
        return q_out
    cdesc = cache.desc()
    st = load().gqa_qk_norm_rope_append(ctypes.byref(cdesc), ctypes.byref(desc), qp, qs, q_out.data_ptr(),
                                        int(q.shape[-2]), kp, ks, vp, vs, DTYPE_CODE[q.dtype], tokens, sp, T, tp,
                                        int(block_tables.shape[1]), pp, rp, B, ep, _stream_ptr(stream))
    _check(st, "gqa_qk_norm_rope_append")
    return q_out


@dataclasses.dataclass
class PageCopies:
    """What a fork or a compaction moves: ``pairs`` int32 [capacity, 2] (from, to),
    ``count`` int32 (copies; for a compaction also the live pages), and for a fork
    ``rows`` int32 [n, 2], the table rows of every fork that was done."""
    pairs: torch.Tensor
    count: torch.Tensor
    rows: Optional[torch.Tensor] = None


@functools.lru_cache(maxsize=256)
def _pages_workspace_size(num_blocks: int, rows: int) -> int:
    return int(load().gqa_kv_pages_workspace_size(num_blocks, rows))


def _pages_workspace(num_blocks: int, rows: int, device: torch.device, workspace, stream) -> torch.Tensor:
    """The caller's workspace, or one per (host thread, device, stream) as ``workspace_for`` keeps."""
    if workspace is not None:
        _dev(workspace, "workspace")
        return workspace
    need = _pages_workspace_size(num_blocks, rows)
    if need == 0:
        raise ValueError(f"no workspace size for {num_blocks} pages and {rows} rows")
    return _scratch(_thread_scratch.pages, need, device.index, stream, zero=False)


def _check_pool(ref_counts: torch.Tensor, block_tables: torch.Tensor, lens: Optional[torch.Tensor], **more):
    """The pool's arrays: shapes, types, and one device, which must be the current one."""
    _dev(ref_counts, "ref_counts", True)
    _dev(block_tables, "block_tables", True)
    if ref_counts.dim() != 1 or block_tables.dim() != 2:
        raise ValueError(f"ref_counts must be [num_blocks] and block_tables [rows, max_blocks], not "
                         f"{tuple(ref_counts.shape)} and {tuple(block_tables.shape)}")
    if lens is not None:
        _dev(lens, "context_lens", True)
        if lens.dim() != 1 or lens.shape[0] != block_tables.shape[0]:
            raise ValueError(f"context_lens must be [{int(block_tables.shape[0])}], not {tuple(lens.shape)}")
    dev = ref_counts.device
    cur = torch.cuda.current_device()
    if dev.index != cur:
        raise ValueError(f"the pool is on {dev} but the current device is cuda:{cur}")
    for name, t in (("block_tables", block_tables), ("context_lens", lens), *more.items()):
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the pool on {dev}")


def _row_list(rows: torch.Tensor, name: str) -> int:
    p = _dev(rows, name, True)
    if rows.dim() != 1:
        raise ValueError(f"{name} must be 1-D, not {tuple(rows.shape)}")
    return p


def kv_pages_reserve(ref_counts: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor, new_tokens,
                     err: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """Pages for the next ``new_tokens`` (a number, or int32 [rows]) of every sequence:
    the table entries they need that are still empty get the lowest free pages.
    Entries that hold one keep it. Lengths stay as they are."""
    many = isinstance(new_tokens, torch.Tensor)
    np_ = _dev(new_tokens, "new_tokens", True) if many else None
    ep = _dev(err, "err", True, True)
    _check_pool(ref_counts, block_tables, context_lens, new_tokens=new_tokens if many else None, err=err,
                workspace=workspace)
    B = int(block_tables.shape[0])
    if many and tuple(new_tokens.shape) != (B,):
        raise ValueError(f"new_tokens must be a number or [{B}], not {tuple(new_tokens.shape)}")
    nb = int(ref_counts.shape[0])
    ws = _pages_workspace(nb, B, ref_counts.device, workspace, stream)
    st = load().gqa_kv_pages_reserve(ref_counts.data_ptr(), nb, block_tables.data_ptr(), int(block_tables.shape[1]),
                                     context_lens.data_ptr(), np_, 0 if many else int(new_tokens), B, ws.data_ptr(),
                                     ws.numel() * ws.element_size(), ep, _stream_ptr(stream))
    _check(st, "gqa_kv_pages_reserve")


def kv_pages_fork(ref_counts: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                  src_rows: torch.Tensor, dst_rows: torch.Tensor, copies: Optional[PageCopies] = None,
                  err: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None) -> PageCopies:
    """Sequences ``dst_rows[i]`` (empty rows) continue ``src_rows[i]``: full pages are
    shared, an unfinished last page gets a fresh one, to be filled by
    ``kv_copy_pages`` with the list returned, in every layer's cache, before the
    sequences are read or written. A sequence taken back into a shared page may not
    append there."""
    sp, dp = _row_list(src_rows, "src_rows"), _row_list(dst_rows, "dst_rows")
    if src_rows.shape != dst_rows.shape:
        raise ValueError(f"src_rows and dst_rows differ in length: {tuple(src_rows.shape)}, {tuple(dst_rows.shape)}")
    n = int(src_rows.shape[0])
    ep = _dev(err, "err", True, True)
    _check_pool(ref_counts, block_tables, context_lens, src_rows=src_rows, dst_rows=dst_rows, err=err,
                workspace=workspace)
    if copies is None:
        dev = ref_counts.device
        copies = PageCopies(*(_empty(shape, torch.int32, dev, stream) for shape in ((n, 2), (1,), (n, 2))))
    elif copies.rows is None or copies.pairs.shape[0] < n or copies.rows.shape[0] != n:
        raise ValueError(f"copies must have room for {n} pairs and exactly {n} rows")
    else:
        _check_copies(copies, ref_counts.device)
    nb = int(ref_counts.shape[0])
    ws = _pages_workspace(nb, n, ref_counts.device, workspace, stream)
    st = load().gqa_kv_pages_fork(ref_counts.data_ptr(), nb, block_tables.data_ptr(), int(block_tables.shape[0]),
                                  int(block_tables.shape[1]), context_lens.data_ptr(), sp, dp, n,
                                  copies.pairs.data_ptr(), copies.count.data_ptr(), copies.rows.data_ptr(),
                                  ws.data_ptr(), ws.numel() * ws.element_size(), ep, _stream_ptr(stream))
    _check(st, "gqa_kv_pages_fork")
    return copies


def _check_copies(copies: PageCopies, device):
    for name, t in (("pairs", copies.pairs), ("count", copies.count), ("rows", copies.rows)):
        if t is None and name == "rows":
            continue
        _dev(t, f"copies.{name}", True)
        if t.device != device:
            raise ValueError(f"copies.{name} is on {t.device}, not {device}")
        if name != "count" and (t.dim() != 2 or t.shape[1] != 2):
            raise ValueError(f"copies.{name} must be [n, 2], not {tuple(t.shape)}")
    if copies.count.numel() < 1:
        raise ValueError("copies.count is empty")


def kv_pages_free(ref_counts: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                  rows: torch.Tensor, err: Optional[torch.Tensor] = None, stream=None) -> None:
    """The sequences in ``rows`` ended: their pages' counts fall, their entries become
    -1 and their lengths 0."""
    rp = _row_list(rows, "rows")
    ep = _dev(err, "err", True, True)
    _check_pool(ref_counts, block_tables, context_lens, rows=rows, err=err)
    st = load().gqa_kv_pages_free(ref_counts.data_ptr(), int(ref_counts.shape[0]), block_tables.data_ptr(),
                                  int(block_tables.shape[0]), int(block_tables.shape[1]), context_lens.data_ptr(), rp,
                                  int(rows.shape[0]), ep, _stream_ptr(stream))
    _check(st, "gqa_kv_pages_free")


def kv_pages_trim(ref_counts: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor, window: int,
                  sinks: int = 0, err: Optional[torch.Tensor] = None, stream=None) -> None:
    """Releases the pages that no later token of ``gqa_decode`` or ``gqa_prefill`` with
    this ``window`` and ``sinks`` sees; their entries become -1."""
    ep = _dev(err, "err", True, True)
    _check_pool(ref_counts, block_tables, context_lens, err=err)
    st = load().gqa_kv_pages_trim(ref_counts.data_ptr(), int(ref_counts.shape[0]), block_tables.data_ptr(),
                                  int(block_tables.shape[1]), context_lens.data_ptr(), int(block_tables.shape[0]),
                                  int(window), int(sinks), ep, _stream_ptr(stream))
    _check(st, "gqa_kv_pages_trim")


def kv_pages_compact(ref_counts: torch.Tensor, block_tables: torch.Tensor, max_copies: Optional[int] = None,
                     copies: Optional[PageCopies] = None, err: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> PageCopies:
    """Moves the highest live pages into the lowest holes until the live pages are the
    pool's first ones, ``max_copies`` of them at most (default: as many as it takes).
    ``kv_copy_pages`` applies the list returned; its count[1] is the number of live
    pages. ``block_tables`` must hold every entry that names a page of the pool.
    ``rows`` that an earlier fork left in a list given as ``copies`` become (-1, -1):
    a compaction moves no table rows."""
    ep = _dev(err, "err", True, True)
    _check_pool(ref_counts, block_tables, None, err=err, workspace=workspace)
    nb = int(ref_counts.shape[0])
    if copies is None:
        n = nb // 2 if max_copies is None else int(max_copies)
        if n < 0:
            raise ValueError(f"max_copies must not be negative: {n}")
        copies = PageCopies(*(_empty(shape, torch.int32, ref_counts.device, stream) for shape in ((n, 2), (2,))))
    else:
        _check_copies(copies, ref_counts.device)
        n = int(copies.pairs.shape[0]) if max_copies is None else int(max_copies)
        if not 0 <= n <= copies.pairs.shape[0] or copies.count.numel() < 2:
            raise ValueError(f"copies must have room for {n} pairs and two counts")
        if copies.rows is not None:
            with torch.cuda.stream(stream):              # (None: the current one)
                copies.rows.fill_(-1)
    ws = _pages_workspace(nb, 0, ref_counts.device, workspace, stream)
    st = load().gqa_kv_pages_compact(ref_counts.data_ptr(), nb, block_tables.data_ptr(), int(block_tables.shape[0]),
                                     int(block_tables.shape[1]), copies.pairs.data_ptr(), n, copies.count.data_ptr(),
                                     ws.data_ptr(), ws.numel() * ws.element_size(), ep, _stream_ptr(stream))
    _check(st, "gqa_kv_pages_compact")
    return copies


def kv_copy_pages(caches, copies: PageCopies, err: Optional[torch.Tensor] = None, stream=None) -> None:
    """Copies the pages of ``copies`` (K, V and scales, and for a fork of KIVI-style
    caches the residual rows) in ``caches``: one cache, or those of all layers, which
    must be alike in shape, layout and type."""
    caches = [caches] if isinstance(caches, PagedKVCache) else list(caches)
    if not caches:
        return
    dev = caches[0].k.device
    _on_cache_device(caches[0], err=err)
    _check_copies(copies, dev)
    for c in caches[1:]:
        if c.k.device != dev:
            raise ValueError(f"a cache is on {c.k.device}, the first on {dev}")
    descs = (KVCacheDesc * len(caches))(*[c.desc() for c in caches])
    st = load().gqa_kv_copy_pages(descs, len(caches), copies.pairs.data_ptr(), copies.count.data_ptr(),
                                  int(copies.pairs.shape[0]), copies.rows.data_ptr() if copies.rows is not None else None,
                                  int(copies.rows.shape[0]) if copies.rows is not None else 0,
                                  _dev(err, "err", True, True), _stream_ptr(stream))
    _check(st, "gqa_kv_copy_pages")


def gqa_prefill(cache: PagedKVCache, q: torch.Tensor, q_start: torch.Tensor, max_new_tokens: int,
                block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.float32,
                window: int = 0, err: Optional[torch.Tensor] = None, stream=None,
                kernel: int = 0, sinks: int = 0) -> torch.Tensor:
    """Causal attention of each sequence's new tokens (rows q_start[b] .. of q
    [total, H, d]) over its paged cache, new tokens included; ``window`` and
    ``sinks`` as in ``gqa_decode``. kernel: 0 auto,
    1 tcgen05 one-tile (32-token chunks), 2 warp-level mma.sync, 3 tcgen05
    two-tile (64-token chunks, head_dim 128), 4 tcgen05 one-tile with 64-token
    chunks and two CTAs per SM (head_dim 128)."""
    args = (_dev(q, "q"), _dev(q_start, "q_start", True), _dev(block_tables, "block_tables", True),
            _dev(context_lens, "context_lens", True), _dev(err, "err", True, True))
    _check_query(cache, q, (3,))
    B = int(context_lens.shape[0]) if context_lens.dim() == 1 else -1
    if B < 0:
        raise ValueError("context_lens must be 1-D")
    _check_table_and_lens(block_tables, context_lens, B, "context_lens", B)
    if q_start.dim() != 1 or q_start.numel() < B + 1:
        raise ValueError(f"q_start must be 1-D with >= {B + 1} entries")
    _check_out(q, out)
    _on_cache_device(cache, q=q, q_start=q_start, block_tables=block_tables,
                     context_lens=context_lens, out=out, err=err)
    if out is None:
        out = _empty(q.shape, out_dtype, q.device, stream)
    op = _dev(out, "out")
    desc = cache.desc()
    st = load().gqa_prefill_sinks(ctypes.byref(desc), args[0], DTYPE_CODE[q.dtype], int(q.shape[1]),
                                  args[1], int(max_new_tokens), args[2],
                                  int(block_tables.shape[1]), args[3], B, float(scale), int(window),
                                  int(sinks), int(q.shape[0]), op, DTYPE_CODE[out.dtype], int(kernel), args[4],
                                  _stream_ptr(stream))
    _check(st, "gqa_prefill")
    return out


def cache_from_case(case) -> PagedKVCache:
    """Wrap the device tensors of a generated decode case (gqa_inputs.DecodeCase)."""
    return PagedKVCache(case.k_cache, case.v_cache, case.num_blocks, case.num_kv_heads,
                        case.head_dim, case.stride_block, case.stride_head, case.stride_token,
                        case.k_scale, case.v_scale,
                        {"i4": GQA_DTYPE_I4, "i4kc": GQA_DTYPE_I4_KC}.get(case.cache_dtype),
                        getattr(case, "k_residual", None))
