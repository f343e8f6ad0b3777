"""Paged grouped-query decode attention for GB300 (sm_103a).

A thin binding over the C ABIs of libpgd (include/pgd.h) and libpgd_ext
(include/pgd_ext.h): it turns torch tensors into device pointers, sizes and
the current CUDA stream, and nothing else.  Every step of the computation runs
in the libraries' CUDA kernels; there is no CPU or PyTorch fallback, and every
call fails loudly if a library is missing or the tensors are not on a CUDA
device.

Entry points (same names as the C ABI, without the ``pgd_`` / ``pgdx_`` prefix):

- ``kv_append_paged``: write each row's new key and value at its page slot.
- ``paged_decode_attention``: grouped-query decode attention of each row over
  its pages, with optional per-head sink logits and sliding window.
- ``rope_append_paged``: rope_rows on q and k fused into the append.
- ``page_slots``, ``kv_write_slots``, ``paged_prefill_attention``: packed
  prompt tokens (prefill) and prompts plus decode steps in one pass.
- ``kv_append_rows``, ``decode_rows_attention``: the same step over dense
  per-row caches [Batch, KvHeads, MaxSeq, D] (decode_rows).
- ``assign_pages``: block-table entries, slots, rows and positions of a pass
  from the requests' lengths.
- ``rotary_append_paged``: rotary positions (``Rotary``: half or interleaved
  pairs, part of the head, scaled frequencies) fused with the append.
- decode, prefill and their steps take ``softcap`` (tanh score cap),
  ``alibi_slopes`` (distance bias), ``first_key`` (documents) and, for prefill,
  ``prefix_len`` (bidirectional prefixes); without them they are libpgd's.
- ``fork_rows``: table rows forked, reordered (beam search), cut back and
  released over reference-counted pages; ``copy_pages``: the copies it leaves to
  make, in all layers' pools; ``compact_pages``: held pages moved to the pool's
  lower end.
- decode and its step take ``group_starts`` and ``group_pages``: rows that share
  their first pages, which are read once for all of them.
- ``paged_decode_workspace_bytes``, ``shared_decode_workspace_bytes``,
  ``get_device_error``.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import math
import os
import threading
from typing import NamedTuple

import torch

PAGE_SIZE = 64
PAGE_MAJOR = 0
HEAD_MAJOR = 1
ROW_MAJOR = 2

OK, EINVAL, EUNSUPPORTED, ECUDA, EDEVICE_BOUNDS, EDEVICE_TIMEOUT, EWORKSPACE = range(7)

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libpgd.so")
EXT_PATH = os.path.join(_PKG, "_build", "libpgd_ext.so")

_lock = threading.Lock()
_lib = None
_ext = None


class PgdError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


class Dims(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int32) for name in (
        "rows", "num_q_heads", "num_kv_heads", "head_dim", "page_size", "num_pages",
        "max_pages_per_row", "layout")]


(KERNEL_AUTO, KERNEL_TENSOR_CORE, KERNEL_CUDA_CORE, KERNEL_PREFILL_TILED, KERNEL_PREFILL_UMMA,
 KERNEL_PREFILL_PAIR) = range(6)


class DecodeOptions(ctypes.Structure):
    _fields_ = [("pages_per_split", ctypes.c_int32), ("kernel", ctypes.c_int32)]


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Loads libpgd.so (built by ``paged_gqa_decode_gb300.build``); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = path or LIB_PATH
            if not os.path.exists(path):
                raise RuntimeError(
                    f"libpgd is not built ({path} missing): run "
                    "`python -c 'import __graft_entry__ as g; g.build()'`")
            lib = ctypes.CDLL(path)
            vp, i32 = ctypes.c_void_p, ctypes.c_int32
            dims_p = ctypes.POINTER(Dims)
            opts_p = ctypes.POINTER(DecodeOptions)
            lib.pgd_kv_append_paged.argtypes = [dims_p, vp, vp, vp, vp, vp, vp, vp]
            lib.pgd_kv_append_paged.restype = ctypes.c_int
            lib.pgd_rope_append_paged.argtypes = [dims_p, ctypes.c_float, vp, vp, vp, vp, vp,
                                                  vp, vp, vp, vp]
            lib.pgd_rope_append_paged.restype = ctypes.c_int
            lib.pgd_selftest_bounded_wait.argtypes = [vp, vp]
            lib.pgd_selftest_bounded_wait.restype = ctypes.c_int
            lib.pgd_page_slots.argtypes = [dims_p, i32, vp, vp, vp, vp, vp]
            lib.pgd_page_slots.restype = ctypes.c_int
            lib.pgd_kv_write_slots.argtypes = [dims_p, vp, vp, vp, vp, vp, vp]
            lib.pgd_kv_write_slots.restype = ctypes.c_int
            lib.pgd_paged_prefill_attention.argtypes = [dims_p, i32, vp, vp, vp, vp, vp, vp, vp,
                                                       i32, ctypes.c_float, vp, vp,
                                                       ctypes.c_size_t, opts_p, vp]
            lib.pgd_paged_prefill_attention.restype = ctypes.c_int
            lib.pgd_paged_prefill_step.argtypes = [dims_p, i32, vp, vp, vp, vp, vp, vp, vp, vp,
                                                   vp, i32, ctypes.c_float, vp, vp,
                                                   ctypes.c_size_t, opts_p, vp]
            lib.pgd_paged_prefill_step.restype = ctypes.c_int
            lib.pgd_prefill_step_kernel_count.argtypes = [dims_p, i32, i32, opts_p, vp]
            lib.pgd_prefill_step_kernel_count.restype = ctypes.c_int
            lib.pgd_paged_decode_workspace_bytes.argtypes = [dims_p, opts_p]
            lib.pgd_paged_decode_workspace_bytes.restype = ctypes.c_size_t
            lib.pgd_attention_kernel_count.argtypes = [dims_p, i32, i32, opts_p, vp]
            lib.pgd_attention_kernel_count.restype = ctypes.c_int
            lib.pgd_paged_decode_attention.argtypes = [dims_p, vp, vp, vp, vp, vp, vp, i32,
                                                      ctypes.c_float, vp, vp, ctypes.c_size_t,
                                                      opts_p, vp]
            lib.pgd_paged_decode_attention.restype = ctypes.c_int
            lib.pgd_paged_decode_step.argtypes = [dims_p, vp, vp, vp, vp, vp, vp, vp, vp, i32,
                                                  ctypes.c_float, vp, vp, ctypes.c_size_t,
                                                  opts_p, vp]
            lib.pgd_paged_decode_step.restype = ctypes.c_int
            lib.pgd_get_device_error.argtypes = [vp]
            lib.pgd_get_device_error.restype = ctypes.c_int
            lib.pgd_status_string.argtypes = [ctypes.c_int]
            lib.pgd_status_string.restype = ctypes.c_char_p
            lib.pgd_version.argtypes = []
            lib.pgd_version.restype = ctypes.c_int
            _lib = lib
    return _lib


class RotaryConfig(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int32) for name in (
        "rotary_dim", "interleaved", "scaling", "exact_bounds")] + [
        (name, ctypes.c_double) for name in (
            "theta", "factor", "original_positions", "beta_fast", "beta_slow", "low_band",
            "high_band", "attention_factor")]


class RotaryPlan(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("factor", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("turns", ctypes.c_uint64 * 64)]


class Score(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("alibi_slopes", ctypes.c_void_p),
                ("first_key", ctypes.c_void_p), ("prefix_len", ctypes.c_void_p)]


def load_extension(path: str | None = None) -> ctypes.CDLL:
    """Loads libpgd_ext.so (built beside libpgd.so); raises if absent."""
    global _ext
    if _ext is None:
        with _lock:
            if _ext is None:
                path = path or EXT_PATH
                if not os.path.exists(path):
                    raise RuntimeError(
                        f"libpgd_ext is not built ({path} missing): run "
                        "`python -c 'import __graft_entry__ as g; g.build()'`")
                lib = ctypes.CDLL(path)
                vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
                dims_p = ctypes.POINTER(Dims)
                plan_p = ctypes.POINTER(RotaryPlan)
                lib.pgdx_assign_pages.argtypes = [i32] * 4 + [vp] * 4 + [i32] + [vp] * 8
                lib.pgdx_rotary_init.argtypes = [ctypes.POINTER(RotaryConfig), plan_p]
                lib.pgdx_rotary_append.argtypes = [dims_p, plan_p, vp, i64, vp, vp, i64, vp, i64,
                                                   vp, i32, vp, vp, vp, vp, vp, vp]
                score_p, opts_p = ctypes.POINTER(Score), ctypes.POINTER(DecodeOptions)
                tail = [i32, ctypes.c_float, vp, vp, ctypes.c_size_t, opts_p, vp]
                lib.pgdx_paged_decode.argtypes = [dims_p, score_p] + [vp] * 8 + tail
                lib.pgdx_paged_prefill.argtypes = [dims_p, i32, score_p] + [vp] * 9 + tail
                size = ctypes.c_size_t
                lib.pgdx_fork_rows.argtypes = [i32] * 3 + [vp] * 6 + [i32] + [vp] * 7
                lib.pgdx_copy_pages.argtypes = [dims_p, i32, vp, vp, i32, vp, vp, vp, vp]
                lib.pgdx_compact_workspace_bytes.argtypes = [i32]
                lib.pgdx_compact_pages.argtypes = [i32] * 3 + [vp] * 4 + [i32, vp, i32] + \
                    [vp] * 7 + [size, vp]
                lib.pgdx_shared_decode_workspace_bytes.argtypes = [dims_p, i32]
                lib.pgdx_shared_decode.argtypes = [dims_p, i32] + [vp] * 10 + \
                    [ctypes.c_float, vp, vp, size, opts_p, vp]
                lib.pgdx_get_device_error.argtypes = [vp]
                for name in ("assign_pages", "rotary_init", "rotary_append", "paged_decode",
                             "paged_prefill", "fork_rows", "copy_pages", "compact_pages",
                             "shared_decode", "get_device_error"):
                    getattr(lib, "pgdx_" + name).restype = ctypes.c_int
                for name in ("compact", "shared_decode"):
                    getattr(lib, f"pgdx_{name}_workspace_bytes").restype = size
                _ext = lib
    return _ext


def status_string(status: int) -> str:
    return load_library().pgd_status_string(status).decode()


# A small call's kernel runs for a few microseconds, and its checks here cost as
# much: these go straight to what torch.cuda's functions call (CUDA tensors
# exist by then, so CUDA is initialised).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_BF16, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32


def _stream_handle(stream: torch.cuda.Stream | None, device: int | None = None) -> int:
    """`device`: the current one, where the caller knows it."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:  # the current stream's handle, without a Stream object for it
        return _raw_stream(torch.cuda.current_device() if device is None else device)
    return torch.cuda.current_stream().cuda_stream


_no_switch = contextlib.nullcontext()


def _on_device(index: int):
    """Makes a device the current one; most calls find it so (and the guard of
    torch.cuda.device costs as much as a small call's kernel runs)."""
    return _no_switch if torch.cuda.current_device() == index else torch.cuda.device(index)


def _scratch(size: tuple, dtype: torch.dtype, device: int,
             stream: torch.cuda.Stream | None) -> torch.Tensor:
    """Memory for a call on `stream`: out of that stream's own pool, so that nothing that
    runs elsewhere still uses it and nothing gets it before the call is done with it."""
    if stream is None:
        return torch.empty(size, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(size, dtype=dtype, device=device)


def _result(size: tuple, dtype: torch.dtype, device: int,
            stream: torch.cuda.Stream | None) -> torch.Tensor:
    """_scratch that the caller gets: it may be used on the current stream later on."""
    t = _scratch(size, dtype, device, stream)
    if stream is not None:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _check_cuda(*tensors: torch.Tensor | None) -> int | None:
    """The index of the device all tensors given are on, checking that it is one
    and that they are contiguous (None: no tensor)."""
    device = None
    for t in tensors:
        if t is not None:
            index = t.get_device()
            if index != device:
                if not t.is_cuda:
                    raise ValueError("paged_gqa_decode_gb300 runs on CUDA tensors only")
                if device is not None:
                    raise ValueError("all tensors must be on one device")
                device = index
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")
    return device


def _dtype(t: torch.Tensor, dtype: torch.dtype, name: str) -> None:
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def make_dims(*, rows: int, num_q_heads: int, num_kv_heads: int, head_dim: int, num_pages: int,
              max_pages_per_row: int, layout: int = PAGE_MAJOR) -> Dims:
    return Dims(rows, num_q_heads, num_kv_heads, head_dim, PAGE_SIZE, num_pages,
                max_pages_per_row, layout)


_dims_kept: dict[tuple, Dims] = {}
_opts_kept: dict[tuple, DecodeOptions] = {}


def _dims_of(*sizes: int) -> Dims:
    """make_dims of (rows, q heads, kv heads, head_dim, pages, max pages per row, layout), the
    struct kept for the next call of these sizes (it is only read)."""
    dims = _dims_kept.get(sizes)
    if dims is None:
        if len(_dims_kept) >= 1024:
            _dims_kept.clear()
        dims = _dims_kept[sizes] = Dims(*sizes[:4], PAGE_SIZE, *sizes[4:])
    return dims


def _opts_of(pages_per_split: int, kernel: int) -> DecodeOptions:
    key = (pages_per_split, kernel)
    opts = _opts_kept.get(key)
    if opts is None:
        if len(_opts_kept) >= 64:
            _opts_kept.clear()
        opts = _opts_kept[key] = DecodeOptions(pages_per_split, kernel)
    return opts


def _pool_pages(pool: torch.Tensor, kv_heads: int, head_dim: int) -> int:
    per_page = kv_heads * PAGE_SIZE * head_dim
    if pool.numel() % per_page:
        raise ValueError(f"pool of {pool.numel()} values is not a whole number of pages")
    return pool.numel() // per_page


def kv_append_paged(k_new: torch.Tensor, v_new: torch.Tensor, table: torch.Tensor,
                    positions: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, *,
                    layout: int = PAGE_MAJOR, stream: torch.cuda.Stream | None = None) -> None:
    """Writes k_new/v_new (bf16 [R, Hkv, D]) into the pools at each row's slot:
    position positions[b] % 64 of page table[b][positions[b] // 64]."""
    dev = _check_cuda(k_new, v_new, table, positions, k_pool, v_pool)
    for t, n in ((k_new, "k_new"), (v_new, "v_new"), (k_pool, "k_pool"), (v_pool, "v_pool")):
        _dtype(t, torch.bfloat16, n)
    _dtype(table, torch.int32, "table")
    _dtype(positions, torch.int32, "positions")
    rows, hkv, d = k_new.shape
    if v_new.shape != k_new.shape or positions.shape != (rows,) or table.dim() != 2 \
            or table.shape[0] != rows or k_pool.shape != v_pool.shape:
        raise ValueError("inconsistent shapes")
    dims = make_dims(rows=rows, num_q_heads=hkv, num_kv_heads=hkv, head_dim=d,
                     num_pages=_pool_pages(k_pool, hkv, d), max_pages_per_row=table.shape[1],
                     layout=layout)
    with _on_device(dev):
        rc = load_library().pgd_kv_append_paged(
            ctypes.byref(dims), _ptr(k_new), _ptr(v_new), _ptr(table), _ptr(positions),
            _ptr(k_pool), _ptr(v_pool), _stream_handle(stream))
    if rc != OK:
        raise PgdError(rc, "kv_append_paged")


def paged_decode_workspace_bytes(dims: Dims, pages_per_split: int = 0) -> int:
    opts = DecodeOptions(pages_per_split, KERNEL_AUTO)
    return load_library().pgd_paged_decode_workspace_bytes(ctypes.byref(dims), ctypes.byref(opts))


def attention_kernel_count(dims: Dims, table_rows: int = 0, window: int = 0,
                           pages_per_split: int = 0, kernel: int = KERNEL_AUTO) -> int:
    """Kernels one paged_decode_attention (table_rows 0) or
    paged_prefill_attention (table_rows > 0) call with these arguments (and
    none of softcap, alibi_slopes, first_key, prefix_len) launches on the
    current device."""
    opts = DecodeOptions(pages_per_split, kernel)
    count = ctypes.c_int32(0)
    rc = load_library().pgd_attention_kernel_count(ctypes.byref(dims), int(table_rows),
                                                   int(window), ctypes.byref(opts),
                                                   ctypes.byref(count))
    if rc != OK:
        raise PgdError(rc, "attention_kernel_count")
    return count.value


def paged_decode_attention(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                           table: torch.Tensor, positions: torch.Tensor,
                           sinks: torch.Tensor | None = None, window: int = 0,
                           scale: float | None = None, *, num_kv_heads: int,
                           layout: int = PAGE_MAJOR, out: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None, pages_per_split: int = 0,
                           kernel: int = KERNEL_AUTO, softcap: float = 0.0,
                           alibi_slopes: torch.Tensor | None = None,
                           first_key: torch.Tensor | None = None,
                           group_starts: torch.Tensor | None = None,
                           group_pages: torch.Tensor | None = None,
                           stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Grouped-query decode attention of each row over its pages.

    q: bf16 [R, Hq, D]; pools: bf16 with num_kv_heads kv heads in ``layout``;
    table: int32 [R, max_pages]; positions: int32 [R]; sinks: fp32 [Hq] or
    None; window <= 0 for full attention.  softcap > 0: scores softcap *
    tanh(scale q.k / softcap); alibi_slopes (fp32 [Hq]): less slope * distance;
    first_key (int32 [R]): row b sees positions from first_key[b] on.
    group_starts (int32 [S + 1]) and group_pages (int32 [S]): rows group_starts[g] ..
    group_starts[g + 1] - 1 hold the same first group_pages[g] pages, which are read
    once for all of them (full attention, none of the above; a workspace of
    shared_decode_workspace_bytes; kernel KERNEL_PREFILL_UMMA does so always, KERNEL_TENSOR_CORE
    never, AUTO where the rows' tables, at their full width, come to more than 128 MB of
    pages).  Returns bf16 [R, Hq, D]."""
    if group_starts is not None or group_pages is not None:
        return _shared_decode(q, None, None, k_pool, v_pool, table, positions, sinks, window,
                              scale, num_kv_heads, layout, out, workspace, pages_per_split, kernel,
                              stream, _score(softcap, alibi_slopes, first_key), group_starts,
                              group_pages)
    return _decode(q, None, None, k_pool, v_pool, table, positions, sinks, window, scale,
                   num_kv_heads, layout, out, workspace, pages_per_split, kernel, stream,
                   _score(softcap, alibi_slopes, first_key))


def paged_decode_step(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                      k_pool: torch.Tensor, v_pool: torch.Tensor, table: torch.Tensor,
                      positions: torch.Tensor, sinks: torch.Tensor | None = None,
                      window: int = 0, scale: float | None = None, *, num_kv_heads: int,
                      layout: int = PAGE_MAJOR, out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, pages_per_split: int = 0,
                      kernel: int = KERNEL_AUTO, softcap: float = 0.0,
                      alibi_slopes: torch.Tensor | None = None,
                      first_key: torch.Tensor | None = None,
                      group_starts: torch.Tensor | None = None,
                      group_pages: torch.Tensor | None = None,
                      stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """kv_append_paged then paged_decode_attention in one launch: each row's
    new K/V (bf16 [R, Hkv, D]) goes to its slot in the pools and the row
    attends over its pages, the new token included.  (With groups that are read once for
    all of their rows, the two calls take less time than this one.)"""
    if group_starts is not None or group_pages is not None:
        return _shared_decode(q, k_new, v_new, k_pool, v_pool, table, positions, sinks, window,
                              scale, num_kv_heads, layout, out, workspace, pages_per_split, kernel,
                              stream, _score(softcap, alibi_slopes, first_key), group_starts,
                              group_pages)
    return _decode(q, k_new, v_new, k_pool, v_pool, table, positions, sinks, window, scale,
                   num_kv_heads, layout, out, workspace, pages_per_split, kernel, stream,
                   _score(softcap, alibi_slopes, first_key))


def _score(softcap, alibi_slopes, first_key, prefix_len=None):
    """What changes the scores, or None where nothing does."""
    if softcap == 0.0 and alibi_slopes is None and first_key is None and prefix_len is None:
        return None
    return float(softcap), alibi_slopes, first_key, prefix_len


def _check_score(score, dev, rows, hq, table_rows) -> Score:
    softcap, slopes, first_key, prefix_len = score
    if not math.isfinite(softcap) or softcap < 0.0:
        raise ValueError("softcap must be finite and >= 0 (0: none)")
    for t, n, dtype, size in ((slopes, "alibi_slopes", _F32, hq),
                              (first_key, "first_key", _I32, rows),
                              (prefix_len, "prefix_len", _I32, table_rows)):
        if t is not None:
            if _check_cuda(t) != dev:
                raise ValueError("all tensors must be on one device")
            _dtype(t, dtype, n)
            if t.shape != (size,):
                raise ValueError(f"{n} must have {size} entries")
    return Score(softcap, _ptr(slopes), _ptr(first_key), _ptr(prefix_len))


def _decode(q, k_new, v_new, k_pool, v_pool, table, positions, sinks, window, scale,
            num_kv_heads, layout, out, workspace, pages_per_split, kernel, stream, score=None):
    dev = _check_cuda(q, k_new, v_new, k_pool, v_pool, table, positions, sinks, out, workspace)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return _decode(q, k_new, v_new, k_pool, v_pool, table, positions, sinks, window, scale,
                           num_kv_heads, layout, out, workspace, pages_per_split, kernel, stream,
                           score)
    if not (q.dtype is k_pool.dtype is v_pool.dtype is _BF16
            and table.dtype is positions.dtype is _I32):
        _dtype(q, torch.bfloat16, "q")
        _dtype(k_pool, torch.bfloat16, "k_pool")
        _dtype(v_pool, torch.bfloat16, "v_pool")
        _dtype(table, torch.int32, "table")
        _dtype(positions, torch.int32, "positions")
    if sinks is not None:
        _dtype(sinks, torch.float32, "sinks")
    rows, hq, d = q.shape
    if positions.shape != (rows,) or table.dim() != 2 or table.shape[0] != rows \
            or k_pool.shape != v_pool.shape or (sinks is not None and sinks.shape != (hq,)):
        raise ValueError("inconsistent shapes")
    if k_new is not None:
        _dtype(k_new, torch.bfloat16, "k_new")
        _dtype(v_new, torch.bfloat16, "v_new")
        if k_new.shape != (rows, num_kv_heads, d) or v_new.shape != k_new.shape:
            raise ValueError("k_new and v_new must be [R, Hkv, D]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dims = ctypes.byref(_dims_of(rows, hq, num_kv_heads, d, _pool_pages(k_pool, num_kv_heads, d),
                                 table.shape[1], layout))
    opts = ctypes.byref(_opts_of(pages_per_split, kernel))
    lib = load_library()
    if out is None:
        out = torch.empty_like(q) if stream is None else _result(q.shape, _BF16, dev, stream)
    elif out.shape != q.shape or out.dtype != torch.bfloat16:
        raise ValueError("out must be bf16 shaped like q")
    if workspace is None:  # (one that is given is checked by the call)
        need = lib.pgd_paged_decode_workspace_bytes(dims, opts)
        workspace = _scratch((max(need, 16),), torch.uint8, dev, stream)
    tail = (table.data_ptr(), positions.data_ptr(), _ptr(sinks), int(window), float(scale),
            out.data_ptr(), workspace.data_ptr(), workspace.nbytes, opts,
            _stream_handle(stream, dev))
    if score is not None:
        mod = _check_score(score, dev, rows, hq, rows)
        rc = load_extension().pgdx_paged_decode(
            dims, ctypes.byref(mod), q.data_ptr(), _ptr(k_new), _ptr(v_new), k_pool.data_ptr(),
            v_pool.data_ptr(), *tail)
        what = "paged_decode_attention" if k_new is None else "paged_decode_step"
    elif k_new is None:
        rc = lib.pgd_paged_decode_attention(dims, q.data_ptr(), k_pool.data_ptr(),
                                            v_pool.data_ptr(), *tail)
        what = "paged_decode_attention"
    else:
        rc = lib.pgd_paged_decode_step(dims, q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
                                       k_pool.data_ptr(), v_pool.data_ptr(), *tail)
        what = "paged_decode_step"
    if rc != OK:
        raise PgdError(rc, what)
    return out


def shared_decode_workspace_bytes(dims: Dims, groups: int) -> int:
    """Workspace of a decode call of these dims with group_starts of groups + 1 entries."""
    return load_extension().pgdx_shared_decode_workspace_bytes(ctypes.byref(dims), groups)


def _shared_decode(q, k_new, v_new, k_pool, v_pool, table, positions, sinks, window, scale,
                   num_kv_heads, layout, out, workspace, pages_per_split, kernel, stream, score,
                   group_starts, group_pages):
    if group_starts is None or group_pages is None:
        raise ValueError("group_starts and group_pages go together")
    if window > 0 or score is not None:
        raise ValueError("group_starts: full attention, without softcap, alibi_slopes or first_key")
    if pages_per_split > 0:
        raise ValueError("group_starts: the split is the library's")
    dev = _check_cuda(q, k_new, v_new, k_pool, v_pool, table, positions, sinks, out, workspace,
                      group_starts, group_pages)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return _shared_decode(q, k_new, v_new, k_pool, v_pool, table, positions, sinks, window,
                                  scale, num_kv_heads, layout, out, workspace, pages_per_split,
                                  kernel, stream, score, group_starts, group_pages)
    if not (q.dtype is k_pool.dtype is v_pool.dtype is _BF16 and table.dtype is positions.dtype
            is group_starts.dtype is group_pages.dtype is _I32):
        for t, n in ((q, "q"), (k_pool, "k_pool"), (v_pool, "v_pool")):
            _dtype(t, torch.bfloat16, n)
        for t, n in ((table, "table"), (positions, "positions"), (group_starts, "group_starts"),
                     (group_pages, "group_pages")):
            _dtype(t, torch.int32, n)
    if sinks is not None:
        _dtype(sinks, torch.float32, "sinks")
    rows, hq, d = q.shape
    if positions.shape != (rows,) or table.dim() != 2 or table.shape[0] != rows \
            or k_pool.shape != v_pool.shape or (sinks is not None and sinks.shape != (hq,)):
        raise ValueError("inconsistent shapes")
    groups = group_pages.shape[0] if group_pages.dim() == 1 else -1
    if groups < 0 or group_starts.shape != (groups + 1,):
        raise ValueError("group_pages must be [S] and group_starts [S + 1]")
    what = "paged_decode_attention" if k_new is None else "paged_decode_step"
    if k_new is not None:
        _dtype(k_new, torch.bfloat16, "k_new")
        _dtype(v_new, torch.bfloat16, "v_new")
        if k_new.shape != (rows, num_kv_heads, d) or v_new.shape != k_new.shape:
            raise ValueError("k_new and v_new must be [R, Hkv, D]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dims = ctypes.byref(_dims_of(rows, hq, num_kv_heads, d, _pool_pages(k_pool, num_kv_heads, d),
                                 table.shape[1], layout))
    lib = load_extension()
    if out is None:
        out = torch.empty_like(q) if stream is None else _result(q.shape, _BF16, dev, stream)
    elif out.shape != q.shape or out.dtype != torch.bfloat16:
        raise ValueError("out must be bf16 shaped like q")
    if workspace is None:  # (one that is given is checked by the call)
        need = lib.pgdx_shared_decode_workspace_bytes(dims, groups)
        workspace = _scratch((max(need, 16),), torch.uint8, dev, stream)
    rc = lib.pgdx_shared_decode(
        dims, groups, group_starts.data_ptr(), group_pages.data_ptr(), q.data_ptr(), _ptr(k_new),
        _ptr(v_new), k_pool.data_ptr(), v_pool.data_ptr(), table.data_ptr(), positions.data_ptr(),
        _ptr(sinks), float(scale), out.data_ptr(), workspace.data_ptr(), workspace.nbytes,
        ctypes.byref(_opts_of(0, kernel)), _stream_handle(stream, dev))
    if rc != OK:
        raise PgdError(rc, what)
    return out


def rope_append_paged(q: torch.Tensor | None, k_new: torch.Tensor, v_new: torch.Tensor,
                      table: torch.Tensor | None, positions: torch.Tensor, k_pool: torch.Tensor,
                      v_pool: torch.Tensor, *, theta: float, slots: torch.Tensor | None = None,
                      layout: int = PAGE_MAJOR, max_pages_per_row: int | None = None,
                      stream: torch.cuda.Stream | None = None) -> None:
    """rope_rows + append: rotates q (bf16 [R, Hq, D], in place) and k_new at
    positions[b] (base theta), writes rotated k and v into the pools at each
    row's slot (from the table, or the explicit slots).  With ROW_MAJOR pools and
    no table, max_pages_per_row says how many pages a row has (None: one)."""
    dev = _check_cuda(q, k_new, v_new, table, positions, slots, k_pool, v_pool)
    for t, n in ((k_new, "k_new"), (v_new, "v_new"), (k_pool, "k_pool"), (v_pool, "v_pool")):
        _dtype(t, torch.bfloat16, n)
    if q is not None:
        _dtype(q, torch.bfloat16, "q")
    _dtype(positions, torch.int32, "positions")
    rows, hkv, d = k_new.shape
    if v_new.shape != k_new.shape or positions.shape != (rows,) or k_pool.shape != v_pool.shape \
            or (q is not None and (q.shape[0] != rows or q.shape[2] != d)):
        raise ValueError("inconsistent shapes")
    width = table.shape[1] if table is not None else (max_pages_per_row or 1)
    dims = make_dims(rows=rows, num_q_heads=q.shape[1] if q is not None else hkv,
                     num_kv_heads=hkv, head_dim=d, num_pages=_pool_pages(k_pool, hkv, d),
                     max_pages_per_row=width, layout=layout)
    with _on_device(dev):
        rc = load_library().pgd_rope_append_paged(
            ctypes.byref(dims), float(theta), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(table),
            _ptr(positions), _ptr(slots), _ptr(k_pool), _ptr(v_pool), _stream_handle(stream))
    if rc != OK:
        raise PgdError(rc, "rope_append_paged")


def page_slots(table: torch.Tensor, positions: torch.Tensor, rows: torch.Tensor | None = None, *,
               num_pages: int, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Pool position of each token: table[r][n // 64] * 64 + n % 64 with
    n = positions[p], r = rows[p] (rows None: r = p); -1 for n < 0."""
    dev = _check_cuda(table, positions, rows)
    _dtype(table, torch.int32, "table")
    _dtype(positions, torch.int32, "positions")
    if rows is not None:
        _dtype(rows, torch.int32, "rows")
        if rows.shape != positions.shape:
            raise ValueError("rows and positions must have one entry per token")
    elif table.shape[0] != positions.shape[0]:
        raise ValueError("without rows, the table needs one row per token")
    tokens = positions.shape[0]
    dims = make_dims(rows=tokens, num_q_heads=1, num_kv_heads=1, head_dim=64,
                     num_pages=num_pages, max_pages_per_row=table.shape[1])
    with _on_device(dev):
        slots = _result((tokens,), _I32, dev, stream)
        rc = load_library().pgd_page_slots(ctypes.byref(dims), table.shape[0], _ptr(table),
                                           _ptr(rows), _ptr(positions), _ptr(slots),
                                           _stream_handle(stream))
    if rc != OK:
        raise PgdError(rc, "page_slots")
    return slots


def kv_write_slots(k_new: torch.Tensor, v_new: torch.Tensor, slots: torch.Tensor,
                   k_pool: torch.Tensor, v_pool: torch.Tensor, *, layout: int = PAGE_MAJOR,
                   max_pages_per_row: int = 1,
                   stream: torch.cuda.Stream | None = None) -> None:
    """Writes token p's key and value (bf16 [P, Hkv, D]) at pool position slots[p].
    With ROW_MAJOR pools slots do not say how many pages a row has:
    max_pages_per_row does (MaxSeq / 64)."""
    dev = _check_cuda(k_new, v_new, slots, k_pool, v_pool)
    for t, n in ((k_new, "k_new"), (v_new, "v_new"), (k_pool, "k_pool"), (v_pool, "v_pool")):
        _dtype(t, torch.bfloat16, n)
    _dtype(slots, torch.int32, "slots")
    tokens, hkv, d = k_new.shape
    if v_new.shape != k_new.shape or slots.shape != (tokens,) or k_pool.shape != v_pool.shape:
        raise ValueError("inconsistent shapes")
    dims = make_dims(rows=tokens, num_q_heads=hkv, num_kv_heads=hkv, head_dim=d,
                     num_pages=_pool_pages(k_pool, hkv, d), max_pages_per_row=max_pages_per_row,
                     layout=layout)
    with _on_device(dev):
        rc = load_library().pgd_kv_write_slots(ctypes.byref(dims), _ptr(k_new), _ptr(v_new),
                                               _ptr(slots), _ptr(k_pool), _ptr(v_pool),
                                               _stream_handle(stream))
    if rc != OK:
        raise PgdError(rc, "kv_write_slots")


def paged_prefill_attention(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                            table: torch.Tensor, rows: torch.Tensor, positions: torch.Tensor,
                            sinks: torch.Tensor | None = None, window: int = 0,
                            scale: float | None = None, *, num_kv_heads: int,
                            layout: int = PAGE_MAJOR, out: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None, pages_per_split: int = 0,
                            kernel: int = KERNEL_AUTO, softcap: float = 0.0,
                            alibi_slopes: torch.Tensor | None = None,
                            first_key: torch.Tensor | None = None,
                            prefix_len: torch.Tensor | None = None,
                            stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Packed prompt tokens: token p (q bf16 [P, Hq, D]) attends over table row
    rows[p]'s pages up to positions[p].  Prompts and decode steps can share one
    call (a step of row b is a token with rows[p] = b).  softcap, alibi_slopes
    and first_key (int32 [P]: the first position of each token's document) as
    for paged_decode_attention; prefix_len (int32 [table rows]): positions of
    each row that all of its tokens see.  Returns bf16 [P, Hq, D]."""
    return _prefill(q, None, None, k_pool, v_pool, table, rows, positions, sinks, window, scale,
                    num_kv_heads, layout, out, workspace, pages_per_split, kernel, stream,
                    _score(softcap, alibi_slopes, first_key, prefix_len))


def paged_prefill_step(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                       k_pool: torch.Tensor, v_pool: torch.Tensor, table: torch.Tensor,
                       rows: torch.Tensor, positions: torch.Tensor,
                       sinks: torch.Tensor | None = None, window: int = 0,
                       scale: float | None = None, *, num_kv_heads: int,
                       layout: int = PAGE_MAJOR, out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, pages_per_split: int = 0,
                       kernel: int = KERNEL_AUTO, softcap: float = 0.0,
                       alibi_slopes: torch.Tensor | None = None,
                       first_key: torch.Tensor | None = None,
                       prefix_len: torch.Tensor | None = None,
                       stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The prefill call with the tokens' writes in it: token p's k_new / v_new
    (bf16 [P, Hkv, D]) go to its slot of table row rows[p] at positions[p],
    then every token attends as in paged_prefill_attention -- the same as
    page_slots + kv_write_slots + paged_prefill_attention.  Returns bf16
    [P, Hq, D]."""
    return _prefill(q, k_new, v_new, k_pool, v_pool, table, rows, positions, sinks, window,
                    scale, num_kv_heads, layout, out, workspace, pages_per_split, kernel, stream,
                    _score(softcap, alibi_slopes, first_key, prefix_len))


def _prefill(q, k_new, v_new, k_pool, v_pool, table, rows, positions, sinks, window, scale,
             num_kv_heads, layout, out, workspace, pages_per_split, kernel, stream, score=None):
    step = k_new is not None
    dev = _check_cuda(q, k_new, v_new, k_pool, v_pool, table, rows, positions, sinks, out,
                      workspace)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return _prefill(q, k_new, v_new, k_pool, v_pool, table, rows, positions, sinks, window,
                            scale, num_kv_heads, layout, out, workspace, pages_per_split, kernel,
                            stream, score)
    if not (q.dtype is k_pool.dtype is v_pool.dtype is _BF16
            and table.dtype is rows.dtype is positions.dtype is _I32):
        _dtype(q, torch.bfloat16, "q")
        _dtype(k_pool, torch.bfloat16, "k_pool")
        _dtype(v_pool, torch.bfloat16, "v_pool")
        _dtype(table, torch.int32, "table")
        _dtype(rows, torch.int32, "rows")
        _dtype(positions, torch.int32, "positions")
    if sinks is not None:
        _dtype(sinks, torch.float32, "sinks")
    tokens, hq, d = q.shape
    if positions.shape != (tokens,) or rows.shape != (tokens,) or table.dim() != 2 \
            or k_pool.shape != v_pool.shape or (sinks is not None and sinks.shape != (hq,)):
        raise ValueError("inconsistent shapes")
    if step:
        if v_new is None:
            raise ValueError("k_new and v_new go together")
        _dtype(k_new, torch.bfloat16, "k_new")
        _dtype(v_new, torch.bfloat16, "v_new")
        if k_new.shape != (tokens, num_kv_heads, d) or v_new.shape != k_new.shape:
            raise ValueError("k_new and v_new are bf16 [P, Hkv, D]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    table_rows = table.shape[0]
    dims = ctypes.byref(_dims_of(tokens, hq, num_kv_heads, d,
                                 _pool_pages(k_pool, num_kv_heads, d), table.shape[1], layout))
    opts = ctypes.byref(_opts_of(pages_per_split, kernel))
    lib = load_library()
    if out is None:
        out = torch.empty_like(q) if stream is None else _result(q.shape, _BF16, dev, stream)
    elif out.shape != q.shape or out.dtype != torch.bfloat16:
        raise ValueError("out must be bf16 shaped like q")
    if workspace is None:  # (one that is given is checked by the call)
        need = lib.pgd_paged_decode_workspace_bytes(dims, opts)
        workspace = _scratch((max(need, 16),), torch.uint8, dev, stream)
    tail = (table.data_ptr(), rows.data_ptr(), positions.data_ptr(), _ptr(sinks), int(window),
            float(scale), out.data_ptr(), workspace.data_ptr(), workspace.nbytes, opts,
            _stream_handle(stream, dev))
    if score is not None:
        mod = _check_score(score, dev, tokens, hq, table_rows)
        rc = load_extension().pgdx_paged_prefill(
            dims, table_rows, ctypes.byref(mod), q.data_ptr(), _ptr(k_new), _ptr(v_new),
            k_pool.data_ptr(), v_pool.data_ptr(), *tail)
    elif step:
        rc = lib.pgd_paged_prefill_step(dims, table_rows, q.data_ptr(), k_new.data_ptr(),
                                        v_new.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(),
                                        *tail)
    else:
        rc = lib.pgd_paged_prefill_attention(dims, table_rows, q.data_ptr(), k_pool.data_ptr(),
                                             v_pool.data_ptr(), *tail)
    if rc != OK:
        raise PgdError(rc, "paged_prefill_step" if step else "paged_prefill_attention")
    return out


def prefill_step_kernel_count(dims: Dims, table_rows: int, window: int = 0,
                              pages_per_split: int = 0, kernel: int = KERNEL_AUTO) -> int:
    """Kernels one paged_prefill_step call with these arguments launches on
    the current device."""
    opts = DecodeOptions(pages_per_split, kernel)
    count = ctypes.c_int32(0)
    rc = load_library().pgd_prefill_step_kernel_count(ctypes.byref(dims), int(table_rows),
                                                      int(window), ctypes.byref(opts),
                                                      ctypes.byref(count))
    if rc != OK:
        raise PgdError(rc, "prefill_step_kernel_count")
    return count.value


def _dense_dims(cache: torch.Tensor, rows: int, num_q_heads: int) -> Dims:
    if cache.dim() != 4 or cache.shape[2] % PAGE_SIZE:
        raise ValueError("dense caches are [Batch, KvHeads, MaxSeq, D] with MaxSeq % 64 == 0")
    batch, hkv, max_seq, d = cache.shape
    if rows > batch:
        raise ValueError("more rows than cache rows")
    per_row = max_seq // PAGE_SIZE
    return make_dims(rows=rows, num_q_heads=num_q_heads, num_kv_heads=hkv, head_dim=d,
                     num_pages=batch * per_row, max_pages_per_row=per_row, layout=ROW_MAJOR)


def kv_append_rows(k_new: torch.Tensor, v_new: torch.Tensor, positions: torch.Tensor,
                   cache_k: torch.Tensor, cache_v: torch.Tensor, *,
                   stream: torch.cuda.Stream | None = None) -> None:
    """write_rows: row b's new key and value (bf16 [R, Hkv, D]) go to position
    positions[b] of row b of the dense caches (bf16 [Batch, Hkv, MaxSeq, D])."""
    dev = _check_cuda(k_new, v_new, positions, cache_k, cache_v)
    for t, n in ((k_new, "k_new"), (v_new, "v_new"), (cache_k, "cache_k"), (cache_v, "cache_v")):
        _dtype(t, torch.bfloat16, n)
    _dtype(positions, torch.int32, "positions")
    if v_new.shape != k_new.shape or cache_k.shape != cache_v.shape \
            or positions.shape != (k_new.shape[0],):
        raise ValueError("inconsistent shapes")
    dims = _dense_dims(cache_k, k_new.shape[0], k_new.shape[1])
    with _on_device(dev):
        rc = load_library().pgd_kv_append_paged(
            ctypes.byref(dims), _ptr(k_new), _ptr(v_new), None, _ptr(positions), _ptr(cache_k),
            _ptr(cache_v), _stream_handle(stream))
    if rc != OK:
        raise PgdError(rc, "kv_append_rows")


def decode_rows_attention(q: torch.Tensor, cache_k: torch.Tensor, cache_v: torch.Tensor,
                          positions: torch.Tensor, sinks: torch.Tensor | None = None,
                          window: int = 0, scale: float | None = None, *,
                          out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                          pages_per_split: int = 0, kernel: int = KERNEL_AUTO,
                          softcap: float = 0.0, alibi_slopes: torch.Tensor | None = None,
                          first_key: torch.Tensor | None = None,
                          stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """decode_rows: row b's queries (q bf16 [R, Hq, D]) attend over row b of the
    dense caches (bf16 [Batch, Hkv, MaxSeq, D]) up to positions[b]; softcap,
    alibi_slopes and first_key as for paged_decode_attention."""
    return _decode_rows(q, None, None, cache_k, cache_v, positions, sinks, window, scale, out,
                        workspace, pages_per_split, kernel, stream,
                        _score(softcap, alibi_slopes, first_key))


def decode_rows_step(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                     cache_k: torch.Tensor, cache_v: torch.Tensor, positions: torch.Tensor,
                     sinks: torch.Tensor | None = None, window: int = 0,
                     scale: float | None = None, *, out: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, pages_per_split: int = 0,
                     kernel: int = KERNEL_AUTO, softcap: float = 0.0,
                     alibi_slopes: torch.Tensor | None = None,
                     first_key: torch.Tensor | None = None,
                     stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """kv_append_rows then decode_rows_attention in one launch."""
    return _decode_rows(q, k_new, v_new, cache_k, cache_v, positions, sinks, window, scale, out,
                        workspace, pages_per_split, kernel, stream,
                        _score(softcap, alibi_slopes, first_key))


def _decode_rows(q, k_new, v_new, cache_k, cache_v, positions, sinks, window, scale, out,
                 workspace, pages_per_split, kernel, stream, score=None):
    dev = _check_cuda(q, k_new, v_new, cache_k, cache_v, positions, sinks, out, workspace)
    _dtype(q, torch.bfloat16, "q")
    _dtype(cache_k, torch.bfloat16, "cache_k")
    _dtype(cache_v, torch.bfloat16, "cache_v")
    _dtype(positions, torch.int32, "positions")
    if sinks is not None:
        _dtype(sinks, torch.float32, "sinks")
    rows, hq, d = q.shape
    if cache_k.shape != cache_v.shape or positions.shape != (rows,) or cache_k.shape[3] != d \
            or (sinks is not None and sinks.shape != (hq,)):
        raise ValueError("inconsistent shapes")
    if k_new is not None:
        _dtype(k_new, torch.bfloat16, "k_new")
        _dtype(v_new, torch.bfloat16, "v_new")
        if k_new.shape != (rows, cache_k.shape[1], d) or v_new.shape != k_new.shape:
            raise ValueError("k_new and v_new must be [R, Hkv, D]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dims = _dense_dims(cache_k, rows, hq)
    opts = DecodeOptions(pages_per_split, kernel)
    lib = load_library()
    with _on_device(dev):
        if out is None:
            out = torch.empty_like(q) if stream is None else _result(q.shape, _BF16, dev, stream)
        elif out.shape != q.shape or out.dtype != torch.bfloat16:
            raise ValueError("out must be bf16 shaped like q")
        if workspace is None:  # (one that is given is checked by the call)
            need = lib.pgd_paged_decode_workspace_bytes(ctypes.byref(dims), ctypes.byref(opts))
            workspace = _scratch((max(need, 16),), torch.uint8, dev, stream)
        tail = (None, _ptr(positions), _ptr(sinks), int(window), float(scale), _ptr(out),
                _ptr(workspace), workspace.numel() * workspace.element_size(),
                ctypes.byref(opts), _stream_handle(stream))
        if score is not None:
            mod = _check_score(score, dev, rows, hq, rows)
            rc = load_extension().pgdx_paged_decode(
                ctypes.byref(dims), ctypes.byref(mod), _ptr(q), _ptr(k_new), _ptr(v_new),
                _ptr(cache_k), _ptr(cache_v), *tail)
            what = "decode_rows_attention" if k_new is None else "decode_rows_step"
        elif k_new is None:
            rc = lib.pgd_paged_decode_attention(ctypes.byref(dims), _ptr(q), _ptr(cache_k),
                                                _ptr(cache_v), *tail)
            what = "decode_rows_attention"
        else:
            rc = lib.pgd_paged_decode_step(ctypes.byref(dims), _ptr(q), _ptr(k_new), _ptr(v_new),
                                           _ptr(cache_k), _ptr(cache_v), *tail)
            what = "decode_rows_step"
    if rc != OK:
        raise PgdError(rc, what)
    return out


def selftest_bounded_wait(stream: torch.cuda.Stream | None = None) -> tuple[int, int, int]:
    """Runs the bounded-wait self-test (about 4 s): returns (device status,
    wait bits, abandoned-split bits); a correct run gives
    (EDEVICE_TIMEOUT, 0, 0)."""
    outcome = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    rc = load_library().pgd_selftest_bounded_wait(_ptr(outcome), _stream_handle(stream))
    if rc != OK:
        raise PgdError(rc, "selftest_bounded_wait")
    status = get_device_error(stream)
    waits, abandoned = outcome.tolist()
    return status, int(waits), int(abandoned)


def get_device_error(stream: torch.cuda.Stream | None = None) -> int:
    """Synchronises the stream and returns (and clears) the device error words
    of libpgd and, where it is in use, libpgd_ext (the first that is set)."""
    handle = _stream_handle(stream)
    status = load_library().pgd_get_device_error(handle)
    if _ext is not None:
        ext = _ext.pgdx_get_device_error(handle)
        status = status if status != OK else ext
    return status


# ---------------------------------------------------------------------------
# A step's set-up on the GPU (libpgd_ext).

class PagePlan(NamedTuple):
    """What assign_pages makes, int32 on the GPU: per token of the packed pass
    its table row, position and pool slot (padding: 0, -1, -1); per request its
    first token (and the tokens' count) and its length after the pass; the index
    of the next free page."""
    rows: torch.Tensor
    positions: torch.Tensor
    slots: torch.Tensor
    starts: torch.Tensor
    lengths: torch.Tensor
    free_head: torch.Tensor


def assign_pages(table: torch.Tensor, cached: torch.Tensor, new_tokens: torch.Tensor,
                 free_pages: torch.Tensor, *, num_tokens: int, num_pages: int,
                 free_head: torch.Tensor | None = None, out: PagePlan | None = None,
                 stream: torch.cuda.Stream | None = None) -> PagePlan:
    """Gives each request the pages of its new tokens and lays out the pass.

    table: int32 [R, W], its new entries written in place; cached, new_tokens:
    int32 [R], positions in the cache and positions of this pass; free_pages:
    int32 [F], handed out in order from free_head (int32 [1] or None for 0);
    num_tokens: the packed pass's fixed token count (the rest is padding);
    num_pages: the pool's pages.  Requests that do not fit are left out and
    reported (get_device_error: EDEVICE_BOUNDS).  ``out`` reuses a plan."""
    dev = _check_cuda(table, cached, new_tokens, free_pages, free_head)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return assign_pages(table, cached, new_tokens, free_pages, num_tokens=num_tokens,
                                num_pages=num_pages, free_head=free_head, out=out, stream=stream)
    if not (table.dtype is cached.dtype is new_tokens.dtype is free_pages.dtype is _I32
            and (free_head is None or free_head.dtype is _I32)):
        for t, n in ((table, "table"), (cached, "cached"), (new_tokens, "new_tokens"),
                     (free_pages, "free_pages"), (free_head, "free_head")):
            if t is not None:
                _dtype(t, torch.int32, n)
    requests, width = table.shape if table.dim() == 2 else (-1, 0)
    if cached.shape != (requests,) or new_tokens.shape != (requests,) or free_pages.dim() != 1 \
            or (free_head is not None and free_head.numel() != 1):
        raise ValueError("inconsistent shapes")
    sizes = (num_tokens, num_tokens, num_tokens, requests + 1, requests, 1)
    whole = None
    if out is None:  # one allocation, cut into the plan's arrays after the launch
        if num_tokens < 0:
            raise ValueError("num_tokens must be >= 0")
        whole = _result((3 * num_tokens + 2 * requests + 2,), _I32, dev, stream)
        at = whole.data_ptr()
        starts = at + 12 * num_tokens
        lengths = starts + 4 * (requests + 1)
        ptrs = (at, at + 4 * num_tokens, at + 8 * num_tokens, starts, lengths,
                lengths + 4 * requests)
    else:
        if _check_cuda(*out) != dev:
            raise ValueError("all tensors must be on one device")
        for t, n, size in zip(out, PagePlan._fields, sizes):
            _dtype(t, torch.int32, n)
            if t.shape != (size,):
                raise ValueError(f"out.{n} must have {size} entries")
        ptrs = [t.data_ptr() for t in out]
    rc = load_extension().pgdx_assign_pages(
        requests, width, num_pages, num_tokens, table.data_ptr(), cached.data_ptr(),
        new_tokens.data_ptr(), free_pages.data_ptr(), free_pages.shape[0], _ptr(free_head),
        *ptrs, _stream_handle(stream, dev))
    if rc != OK:
        raise PgdError(rc, "assign_pages")
    if whole is not None:
        out = PagePlan(*torch.unsafe_split_with_sizes(whole, sizes))
    return out


_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "banded": 4}


class Rotary:
    """Rotary frequencies, computed once and passed to rotary_append_paged.

    rotary_dim: leading dims of each head that are rotated (a multiple of 16);
    interleaved: dims 2i and 2i + 1 pair up (else i and i + rotary_dim / 2);
    scaling: "none", "linear", "ntk", "yarn" or "banded", with their factor,
    original_positions, beta_fast / beta_slow (yarn; exact_bounds leaves its
    ramp's ends unrounded) and low_band / high_band (banded), as
    include/pgd_ext.h defines them; attention_factor: factor of cos and sin
    (None: the scaling's own)."""

    def __init__(self, rotary_dim: int, theta: float, *, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, original_positions: float = 0.0,
                 beta_fast: float = 32.0, beta_slow: float = 1.0, exact_bounds: bool = False,
                 low_band: float = 1.0, high_band: float = 4.0,
                 attention_factor: float | None = None):
        if scaling not in _SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
        if attention_factor is not None and not attention_factor > 0:
            raise ValueError("attention_factor must be positive")
        config = RotaryConfig(rotary_dim, int(interleaved), _SCALINGS[scaling], int(exact_bounds),
                              theta, factor, original_positions, beta_fast, beta_slow, low_band,
                              high_band, attention_factor or 0.0)
        self.plan = RotaryPlan()
        rc = load_extension().pgdx_rotary_init(ctypes.byref(config), ctypes.byref(self.plan))
        if rc != OK:
            raise PgdError(rc, "rotary_init")


def _token_stride(t: torch.Tensor, name: str) -> int:
    """Values from token to token of a [P, heads, D] tensor whose tokens are
    contiguous (a view of a fused projection, say)."""
    tokens, heads, d = t.shape
    if t.is_contiguous():
        return heads * d
    token, head, value = t.stride()
    if value != 1 or (heads > 1 and head != d):
        raise ValueError(f"{name}: each token's heads must be contiguous")
    return token if tokens > 1 else heads * d


def rotary_append_paged(q: torch.Tensor | None, k_new: torch.Tensor, v_new: torch.Tensor,
                        positions: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, *,
                        rotary: Rotary, slots: torch.Tensor | None = None,
                        table: torch.Tensor | None = None, rows: torch.Tensor | None = None,
                        table_rows: int | None = None, layout: int = PAGE_MAJOR,
                        max_pages_per_row: int | None = None, q_out: torch.Tensor | None = None,
                        stream: torch.cuda.Stream | None = None) -> torch.Tensor | None:
    """Rotates q and k_new at positions[p] and writes rotated k and v into the
    pools, at slots[p] or, without slots, at position positions[p] of table row
    rows[p] (None: row p).

    q (bf16 [P, Hq, D]), k_new and v_new (bf16 [P, Hkv, D]) may be views with a
    token stride of their own (a multiple of 8 values).  Returns the rotated q:
    q_out if given (q itself for in place), else a new contiguous tensor.
    Tokens with a negative position or slot are left alone, their q_out rows
    too.  With ROW_MAJOR pools the table may be None: max_pages_per_row then
    says how many pages a row has (with slots too), and with rows table_rows
    how many rows there are."""
    dev = _check_cuda(positions, k_pool, v_pool, slots, table, rows, q_out)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return rotary_append_paged(
                q, k_new, v_new, positions, k_pool, v_pool, rotary=rotary, slots=slots, table=table,
                rows=rows, table_rows=table_rows, layout=layout,
                max_pages_per_row=max_pages_per_row, q_out=q_out, stream=stream)
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new")):
        if t is not None:
            if t.get_device() != dev:
                raise ValueError("all tensors must be on one CUDA device")
            if t.dim() != 3:
                raise ValueError(f"{n} must be [P, heads, D]")
            if t.dtype is not _BF16:
                _dtype(t, torch.bfloat16, n)
    if not k_pool.dtype is v_pool.dtype is _BF16:
        _dtype(k_pool, torch.bfloat16, "k_pool")
        _dtype(v_pool, torch.bfloat16, "v_pool")
    for t, n in ((positions, "positions"), (slots, "slots"), (table, "table"), (rows, "rows")):
        if t is not None and t.dtype is not _I32:
            _dtype(t, torch.int32, n)
    tokens, hkv, d = k_new.shape
    if v_new.shape != k_new.shape or positions.shape != (tokens,) or k_pool.shape != v_pool.shape \
            or (q is not None and (q.shape[0] != tokens or q.shape[2] != d)) \
            or (slots is not None and slots.shape != (tokens,)) \
            or (rows is not None and rows.shape != (tokens,)) \
            or (table is not None and table.dim() != 2):
        raise ValueError("inconsistent shapes")
    if slots is None and rows is None and table is not None and table.shape[0] != tokens:
        raise ValueError("without rows, the table needs one row per token")
    if q is None and q_out is not None:
        raise ValueError("q_out without q")
    if q_out is not None:
        _dtype(q_out, torch.bfloat16, "q_out")
        if q_out.shape != q.shape:
            raise ValueError("q_out must be shaped like q")
    if layout == ROW_MAJOR and table is None and max_pages_per_row is None:
        raise ValueError("ROW_MAJOR pools without a table need max_pages_per_row")
    width = table.shape[1] if table is not None else \
        1 if max_pages_per_row is None else max_pages_per_row
    count = table.shape[0] if table is not None else (table_rows or 0)
    dims = _dims_of(tokens, q.shape[1] if q is not None else hkv, hkv, d,
                    _pool_pages(k_pool, hkv, d), width, layout)
    if q is not None and q_out is None:
        q_out = _result(q.shape, _BF16, dev, stream)
    rc = load_extension().pgdx_rotary_append(
        ctypes.byref(dims), ctypes.byref(rotary.plan), _ptr(q),
        0 if q is None else _token_stride(q, "q"), _ptr(q_out), k_new.data_ptr(),
        _token_stride(k_new, "k_new"), v_new.data_ptr(), _token_stride(v_new, "v_new"),
        _ptr(table), count, _ptr(rows), positions.data_ptr(), _ptr(slots), k_pool.data_ptr(),
        v_pool.data_ptr(), _stream_handle(stream, dev))
    if rc != OK:
        raise PgdError(rc, "rotary_append_paged")
    return q_out


# ---------------------------------------------------------------------------
# Pages that several rows hold (libpgd_ext).

class ForkPlan(NamedTuple):
    """What fork_rows makes, int32 on the GPU: the rows' lengths; per row the page
    to copy from, the page to copy to and the positions to copy (-1, -1, 0: none),
    as copy_pages takes them; the index of the next free page."""
    lengths: torch.Tensor
    sources: torch.Tensor
    targets: torch.Tensor
    counts: torch.Tensor
    free_head: torch.Tensor


class CompactPlan(NamedTuple):
    """What compact_pages makes, int32 on the GPU: the table, shares and free pages
    under the pages' new names; the copies (-1 past the last) as copy_pages takes them;
    1 + the highest page held."""
    table: torch.Tensor
    shares: torch.Tensor
    free_pages: torch.Tensor
    sources: torch.Tensor
    targets: torch.Tensor
    end: torch.Tensor


def _int32(*tensors) -> None:
    for t, name in tensors:
        if t is not None and t.dtype is not _I32:
            _dtype(t, torch.int32, name)


def _plan_ptrs(out, sizes, dev) -> list[int]:
    if _check_cuda(*out) != dev:
        raise ValueError("all tensors must be on one device")
    for t, n, size in zip(out, out._fields, sizes):
        _dtype(t, torch.int32, n)
        if t.shape != size:
            raise ValueError(f"out.{n} must be {list(size)}")
    return [t.data_ptr() for t in out]


def fork_rows(table: torch.Tensor, lengths: torch.Tensor, parents: torch.Tensor,
              shares: torch.Tensor, free_pages: torch.Tensor, *,
              free_head: torch.Tensor | None = None, keep: torch.Tensor | None = None,
              out: ForkPlan | None = None, stream: torch.cuda.Stream | None = None) -> ForkPlan:
    """Makes each row a copy of an old row, over pages that rows share.

    table: int32 [R, W], rewritten in place; lengths: int32 [R], positions in the
    cache; parents: int32 [R], the old row that each row continues (itself: as it
    was; -1: none, its pages are given back); shares: int32 [pages], how many rows hold
    each page beyond the first, kept up to date in place; free_pages: int32 [F] with
    the next page at free_head (int32 [1] or None for 0), as for assign_pages, in
    place: pages that no row holds any more come back below it, copies of last
    pages in part use are taken from it.  keep (int32 [R]): row r keeps at most its
    parent's first keep[r] positions.  The copies themselves are copy_pages'.  ``out``
    reuses a plan (its tensors must be none of the inputs)."""
    dev = _check_cuda(table, lengths, parents, shares, free_pages, free_head, keep)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return fork_rows(table, lengths, parents, shares, free_pages, free_head=free_head,
                             keep=keep, out=out, stream=stream)
    _int32((table, "table"), (lengths, "lengths"), (parents, "parents"), (shares, "shares"),
           (free_pages, "free_pages"), (free_head, "free_head"), (keep, "keep"))
    rows, width = table.shape if table.dim() == 2 else (-1, 0)
    if lengths.shape != (rows,) or parents.shape != (rows,) or shares.dim() != 1 \
            or free_pages.dim() != 1 or (free_head is not None and free_head.numel() != 1) \
            or (keep is not None and keep.shape != (rows,)):
        raise ValueError("inconsistent shapes")
    whole = None
    if out is None:  # one allocation, cut into the plan's arrays after the launch
        whole = _result((4 * rows + 1,), _I32, dev, stream)
        ptrs = [whole.data_ptr() + 4 * rows * k for k in range(5)]
    else:
        ptrs = _plan_ptrs(out, ((rows,),) * 4 + ((1,),), dev)
    rc = load_extension().pgdx_fork_rows(
        rows, width, shares.shape[0], table.data_ptr(), lengths.data_ptr(), parents.data_ptr(),
        _ptr(keep), shares.data_ptr(), free_pages.data_ptr(), free_pages.shape[0],
        _ptr(free_head), *ptrs, _stream_handle(stream, dev))
    if rc != OK:
        raise PgdError(rc, "fork_rows")
    if whole is not None:
        out = ForkPlan(*torch.unsafe_split_with_sizes(whole, (rows, rows, rows, rows, 1)))
    return out


def copy_pages(k_pools: torch.Tensor | list[torch.Tensor], v_pools: torch.Tensor |
               list[torch.Tensor], sources: torch.Tensor, targets: torch.Tensor,
               counts: torch.Tensor | None = None, *, num_kv_heads: int, head_dim: int,
               layout: int = PAGE_MAJOR, stream: torch.cuda.Stream | None = None) -> None:
    """Copies the first counts[i] positions (None: all) of page sources[i] to page
    targets[i] (int32 [n]; negative: no copy) in the K and V pools, bf16 in ``layout``,
    of one layer or, as lists, of several."""
    if isinstance(k_pools, torch.Tensor):
        k_pools = [k_pools]
    if isinstance(v_pools, torch.Tensor):
        v_pools = [v_pools]
    if len(k_pools) != len(v_pools):
        raise ValueError("k_pools and v_pools must be of the same layers")
    dev = _check_cuda(sources, targets, counts, *k_pools, *v_pools)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return copy_pages(k_pools, v_pools, sources, targets, counts,
                              num_kv_heads=num_kv_heads, head_dim=head_dim, layout=layout,
                              stream=stream)
    _int32((sources, "sources"), (targets, "targets"), (counts, "counts"))
    if sources.dim() != 1 or targets.shape != sources.shape \
            or (counts is not None and counts.shape != sources.shape):
        raise ValueError("sources, targets and counts must be [n]")
    layers = len(k_pools)
    if layers == 0:
        return
    pools, shape = (*k_pools, *v_pools), k_pools[0].shape
    for pool in pools:
        if pool.dtype is not _BF16:
            _dtype(pool, torch.bfloat16, "k_pools and v_pools")
    if list(map(torch.Tensor.size, pools)).count(shape) != len(pools):
        raise ValueError("the pools must have one shape")
    dims = _dims_of(sources.shape[0], num_kv_heads, num_kv_heads, head_dim,
                    _pool_pages(k_pools[0], num_kv_heads, head_dim), 1, layout)
    ptrs = array.array("Q", map(torch.Tensor.data_ptr, pools))
    at = ptrs.buffer_info()[0]
    rc = load_extension().pgdx_copy_pages(
        ctypes.byref(dims), layers, at, at + layers * ptrs.itemsize, sources.shape[0],
        sources.data_ptr(), targets.data_ptr(), _ptr(counts), _stream_handle(stream, dev))
    if rc != OK:
        raise PgdError(rc, "copy_pages")


def compact_pages(table: torch.Tensor, lengths: torch.Tensor, shares: torch.Tensor,
                  free_pages: torch.Tensor, *, free_head: torch.Tensor | None = None,
                  max_moves: int | None = None, out: CompactPlan | None = None,
                  stream: torch.cuda.Stream | None = None) -> CompactPlan:
    """Gives held pages the names of lower free ones: the highest page goes to the
    lowest free one and so on, at most max_moves of them (None: half of the pool, all
    there can be).  The arguments are fork_rows'; nothing is changed in place unless ``out``
    names the inputs as its table, shares and free_pages.  The copies themselves are
    copy_pages'."""
    dev = _check_cuda(table, lengths, shares, free_pages, free_head)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return compact_pages(table, lengths, shares, free_pages, free_head=free_head,
                                 max_moves=max_moves, out=out, stream=stream)
    _int32((table, "table"), (lengths, "lengths"), (shares, "shares"),
           (free_pages, "free_pages"), (free_head, "free_head"))
    rows, width = table.shape if table.dim() == 2 else (-1, 0)
    if lengths.shape != (rows,) or shares.dim() != 1 or free_pages.dim() != 1 \
            or (free_head is not None and free_head.numel() != 1):
        raise ValueError("inconsistent shapes")
    pages, listed = shares.shape[0], free_pages.shape[0]
    if max_moves is None:
        max_moves = pages // 2
    if max_moves < 0:
        raise ValueError("max_moves must be >= 0")
    lib = load_extension()
    sizes = (rows * width, pages, listed, max_moves, max_moves, 1)
    whole = None
    if out is None:  # one allocation, the workspace (16-byte aligned) at its front
        need = (lib.pgdx_compact_workspace_bytes(pages) + 15) // 16 * 4
        whole = _result((need + sum(sizes),), _I32, dev, stream)
        ptrs, at = [], whole.data_ptr() + 4 * need
        for size in sizes:
            ptrs.append(at)
            at += 4 * size
        workspace = whole
    else:
        ptrs = _plan_ptrs(out, ((rows, width),) + tuple((n,) for n in sizes[1:]), dev)
        need = (lib.pgdx_compact_workspace_bytes(pages) + 15) // 16 * 4
        workspace = _scratch((max(need, 4),), _I32, dev, stream)
    rc = lib.pgdx_compact_pages(
        rows, width, pages, table.data_ptr(), lengths.data_ptr(), shares.data_ptr(),
        free_pages.data_ptr(), listed, _ptr(free_head), max_moves, *ptrs, workspace.data_ptr(),
        4 * need, _stream_handle(stream, dev))
    if rc != OK:
        raise PgdError(rc, "compact_pages")
    if whole is not None:
        parts = torch.unsafe_split_with_sizes(whole, (need,) + sizes)
        out = CompactPlan(parts[1].view(rows, width), *parts[2:])
    return out
