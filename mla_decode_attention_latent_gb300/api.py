"""Python binding of the MLA decode C ABI (argument marshalling only).

The two calls mirror the usage page "FlashMLA란 무엇인가?" (section "FlashMLA
설치 및 사용", steps 2 and 3):

    md, ns = mla_get_metadata(cache_seqlens, s_q * h_q // h_kv, h_kv)
    for layer in range(num_layers):
        o, lse = mla_decode_kvcache(q[layer], kcache[layer], block_table, cache_seqlens,
                                    dv, md, ns, causal=True)

``get_mla_metadata`` and ``flash_mla_with_kvcache`` are the same calls under
the page's names.  Every step runs in the CUDA library; this module only
checks tensor properties, allocates outputs with torch on the caller's device
and passes raw pointers and the current stream.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import MLA_METADATA_INTS, MLA_V_DIM, check, load


def _stream_handle(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _need_cuda(name: str, t: torch.Tensor, dtype: torch.dtype) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def mla_num_sm_parts(num_q_rows: int, h_kv: int = 1, device: Optional[torch.device] = None) -> int:
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    out = ctypes.c_int(0)
    check("mla_num_sm_parts", load().mla_num_sm_parts(dev.index or 0, int(num_q_rows), int(h_kv), ctypes.byref(out)))
    return out.value


# the partition's costs (include/mla_decode.h): per segment and for needing
# the combine, in pages of the lengths the partition is computed on
SCHED_FIXED_COST_PAGES = 8
SCHED_COMBINE_COST_PAGES = 4
SCHED_SPARSE_FIXED_COST_CHUNKS = 1
SCHED_SPARSE_COMBINE_COST_CHUNKS = 1


def mla_get_metadata(cache_seqlens: torch.Tensor, num_q_rows: int, h_kv: int = 1,
                     num_parts: Optional[int] = None, fixed_cost: Optional[int] = None,
                     combine_cost: Optional[int] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Split-KV work partition: (tile_scheduler_metadata int32 [P, 8], num_splits int32 [b + 1]).

    ``fixed_cost`` / ``combine_cost`` override the partition's costs
    (``mla_get_metadata_costs``); by default those of a dense decode."""
    _need_cuda("cache_seqlens", cache_seqlens, torch.int32)
    dev = cache_seqlens.device
    if num_parts is None:
        num_parts = mla_num_sm_parts(num_q_rows, h_kv, dev)
    batch = cache_seqlens.numel()
    md = torch.empty((num_parts, MLA_METADATA_INTS), dtype=torch.int32, device=dev)
    ns = torch.empty((batch + 1,), dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        if fixed_cost is None and combine_cost is None:
            st = load().mla_get_metadata(cache_seqlens.data_ptr(), batch, int(num_q_rows), int(h_kv), int(num_parts),
                                         md.data_ptr(), ns.data_ptr(), _stream_handle(dev))
        else:
            fc = SCHED_FIXED_COST_PAGES if fixed_cost is None else int(fixed_cost)
            cc = SCHED_COMBINE_COST_PAGES if combine_cost is None else int(combine_cost)
            st = load().mla_get_metadata_costs(cache_seqlens.data_ptr(), batch, int(num_q_rows), int(h_kv),
                                               int(num_parts), fc, cc, md.data_ptr(), ns.data_ptr(),
                                               _stream_handle(dev))
    check("mla_get_metadata", st)
    return md, ns


def mla_get_metadata_sparse(list_lens: torch.Tensor, num_q_rows: int, h_kv: int = 1,
                            num_parts: Optional[int] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The work partition of a sparse decode: over the index lists' lengths,
    with the sparse decode's costs (a 64-entry list chunk's gathers take about
    four dense pages' time, so its per-segment costs, in list chunks, are a
    quarter of the dense ones or less; the values were measured on GB300)."""
    return mla_get_metadata(list_lens, num_q_rows, h_kv, num_parts, fixed_cost=SCHED_SPARSE_FIXED_COST_CHUNKS,
                            combine_cost=SCHED_SPARSE_COMBINE_COST_CHUNKS)


def mla_workspace_bytes(batch: int, s_q: int, h_q: int, h_kv: int, dv: int, num_parts: int) -> int:
    n = load().mla_workspace_bytes(batch, s_q, h_q, h_kv, dv, num_parts)
    if n == 0:
        raise ValueError("invalid shape for the decode workspace")
    return int(n)


def _dense_decode_args(q, kcache, block_table, cache_seqlens, dv, tile_scheduler_metadata, num_splits, out, lse,
                       allocate):
    """Check the tensors of a decode over a bf16 cache; return (b, s_q, h_q, d, num_blocks, h_kv, num_parts, out,
    lse).  Shapes are checked here, before the library is called, so that a
    wrongly shaped tensor can never make a kernel read or write out of bounds;
    ``allocate`` creates missing outputs (otherwise they are required)."""
    _need_cuda("q", q, torch.bfloat16)
    _need_cuda("kcache", kcache, torch.bfloat16)
    _need_cuda("block_table", block_table, torch.int32)
    _need_cuda("cache_seqlens", cache_seqlens, torch.int32)
    _need_cuda("tile_scheduler_metadata", tile_scheduler_metadata, torch.int32)
    _need_cuda("num_splits", num_splits, torch.int32)
    if q.dim() != 4 or kcache.dim() != 4 or block_table.dim() != 2:
        raise ValueError("q must be [b, s_q, h_q, d], kcache [num_blocks, page, h_kv, d], block_table [b, max_blocks]")
    b, s_q, h_q, d = q.shape
    num_blocks, page, h_kv, dk = kcache.shape
    if dk != d or page != _lib.MLA_PAGE_SIZE:
        raise ValueError("kcache must be [num_blocks, 64, h_kv, d] with the same d as q")
    if block_table.shape[0] != b or cache_seqlens.numel() != b or num_splits.numel() != b + 1:
        raise ValueError("batch size differs between q, block_table, cache_seqlens and num_splits")
    if tile_scheduler_metadata.dim() != 2 or tile_scheduler_metadata.shape[1] != MLA_METADATA_INTS:
        raise ValueError("tile_scheduler_metadata must be [num_parts, 8]")
    dev = q.device
    if out is None and allocate:
        out = torch.empty((b, s_q, h_q, dv), dtype=torch.bfloat16, device=dev)
    if lse is None and allocate:
        lse = torch.empty((b, s_q, h_q), dtype=torch.float32, device=dev)
    _need_cuda("out", out, torch.bfloat16)
    _need_cuda("lse", lse, torch.float32)
    if tuple(out.shape) != (b, s_q, h_q, dv) or tuple(lse.shape) != (b, s_q, h_q):
        raise ValueError("out must be [b, s_q, h_q, dv] and lse [b, s_q, h_q]")
    _same_device(dev, kcache=kcache, block_table=block_table, cache_seqlens=cache_seqlens,
                 tile_scheduler_metadata=tile_scheduler_metadata, num_splits=num_splits, out=out, lse=lse)
    return b, s_q, h_q, d, num_blocks, h_kv, tile_scheduler_metadata.shape[0], out, lse


def _same_device(dev: torch.device, of: str = "q", **tensors) -> None:
    for name, t in tensors.items():
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, but {of} is on {dev}")


def mla_decode_kvcache(q: torch.Tensor, kcache: torch.Tensor, block_table: torch.Tensor,
                       cache_seqlens: torch.Tensor, dv: int, tile_scheduler_metadata: torch.Tensor,
                       num_splits: torch.Tensor, softmax_scale: Optional[float] = None, causal: bool = False,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """MLA decode: returns (o bf16 [b, s_q, h_q, dv], lse fp32 [b, s_q, h_q])."""
    b, s_q, h_q, d, num_blocks, h_kv, num_parts, out, lse = _dense_decode_args(
        q, kcache, block_table, cache_seqlens, dv, tile_scheduler_metadata, num_splits, out, lse, allocate=True)
    dev = q.device
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    ws_need = mla_workspace_bytes(b, s_q, h_q, h_kv, dv, num_parts) if dv == MLA_V_DIM and h_q % h_kv == 0 else 256
    if workspace is None:
        workspace = torch.empty((ws_need,), dtype=torch.uint8, device=dev)
    _need_cuda("workspace", workspace, torch.uint8)
    _same_device(dev, workspace=workspace)
    with torch.cuda.device(dev):
        st = load().mla_decode_kvcache(
            q.data_ptr(), kcache.data_ptr(), num_blocks, block_table.data_ptr(), block_table.shape[1],
            cache_seqlens.data_ptr(), b, s_q, h_q, h_kv, d, dv, tile_scheduler_metadata.data_ptr(),
            num_splits.data_ptr(), num_parts, float(softmax_scale), int(bool(causal)), out.data_ptr(),
            lse.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream_handle(dev))
    check("mla_decode_kvcache", st)
    return out, lse


def mla_decode_kvcache_fp8(q: torch.Tensor, kv_pages: torch.Tensor, block_table: torch.Tensor,
                           cache_seqlens: torch.Tensor, dv: int, tile_scheduler_metadata: torch.Tensor,
                           num_splits: torch.Tensor, softmax_scale: Optional[float] = None, causal: bool = False,
                           out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """MLA decode over packed e4m3 pages with per-token scales.

    ``kv_pages`` is uint8 [num_blocks, MLA_FP8_PAGE_BYTES(d)]: per page, 64 rows
    of d e4m3 codes, then 64 fp32 scales; row j dequantizes to scale_j * code_j
    (layout and precision in ``include/mla_decode.h``).  Returns (o bf16
    [b, s_q, h_q, dv], lse fp32 [b, s_q, h_q]) as ``mla_decode_kvcache``.
    """
    _need_cuda("q", q, torch.bfloat16)
    _need_cuda("kv_pages", kv_pages, torch.uint8)
    _need_cuda("block_table", block_table, torch.int32)
    _need_cuda("cache_seqlens", cache_seqlens, torch.int32)
    _need_cuda("tile_scheduler_metadata", tile_scheduler_metadata, torch.int32)
    _need_cuda("num_splits", num_splits, torch.int32)
    if q.dim() != 4 or block_table.dim() != 2:
        raise ValueError("q must be [b, s_q, h_q, d] and block_table [b, max_blocks]")
    b, s_q, h_q, d = q.shape
    if kv_pages.dim() != 2 or kv_pages.shape[1] != _lib.MLA_FP8_PAGE_BYTES(d):
        raise ValueError(f"kv_pages must be [num_blocks, {_lib.MLA_FP8_PAGE_BYTES(d)}] for d = {d}")
    num_blocks = kv_pages.shape[0]
    if block_table.shape[0] != b or cache_seqlens.numel() != b or num_splits.numel() != b + 1:
        raise ValueError("batch size differs between q, block_table, cache_seqlens and num_splits")
    if tile_scheduler_metadata.dim() != 2 or tile_scheduler_metadata.shape[1] != MLA_METADATA_INTS:
        raise ValueError("tile_scheduler_metadata must be [num_parts, 8]")
    num_parts = tile_scheduler_metadata.shape[0]
    dev = q.device
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((b, s_q, h_q, dv), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((b, s_q, h_q), dtype=torch.float32, device=dev)
    _need_cuda("out", out, torch.bfloat16)
    _need_cuda("lse", lse, torch.float32)
    if tuple(out.shape) != (b, s_q, h_q, dv) or tuple(lse.shape) != (b, s_q, h_q):
        raise ValueError("out must be [b, s_q, h_q, dv] and lse [b, s_q, h_q]")
    ws_need = mla_workspace_bytes(b, s_q, h_q, 1, dv, num_parts) if dv == MLA_V_DIM else 256
    if workspace is None:
        workspace = torch.empty((ws_need,), dtype=torch.uint8, device=dev)
    _need_cuda("workspace", workspace, torch.uint8)
    _same_device(dev, kv_pages=kv_pages, block_table=block_table, cache_seqlens=cache_seqlens,
                 tile_scheduler_metadata=tile_scheduler_metadata, num_splits=num_splits, out=out, lse=lse,
                 workspace=workspace)
    with torch.cuda.device(dev):
        st = load().mla_decode_kvcache_fp8(
            q.data_ptr(), kv_pages.data_ptr(), num_blocks, block_table.data_ptr(), block_table.shape[1],
            cache_seqlens.data_ptr(), b, s_q, h_q, 1, d, dv, tile_scheduler_metadata.data_ptr(),
            num_splits.data_ptr(), num_parts, float(softmax_scale), int(bool(causal)), out.data_ptr(),
            lse.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream_handle(dev))
    check("mla_decode_kvcache_fp8", st)
    return out, lse


def mla_decode_kvcache_sparse(q: torch.Tensor, kcache: torch.Tensor, block_table: torch.Tensor,
                              cache_seqlens: torch.Tensor, indices: torch.Tensor, dv: int,
                              tile_scheduler_metadata: Optional[torch.Tensor] = None,
                              num_splits: Optional[torch.Tensor] = None, list_lens: Optional[torch.Tensor] = None,
                              softmax_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                              lse: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Sparse top-k MLA decode: query token i of sequence b attends to the cache
    positions ``indices[b, i]`` (int32 [b, s_q, topk]; entries outside
    [0, cache_seqlens[b]) are ignored).  The work partition is computed on
    ``list_lens`` (default: topk for every sequence) with the sparse decode's
    costs (``mla_get_metadata_sparse``) unless given.  Returns
    (o bf16 [b, s_q, h_q, dv], lse fp32 [b, s_q, h_q]); see ``include/mla_decode.h``."""
    for name, t, dt in (("q", q, torch.bfloat16), ("kcache", kcache, torch.bfloat16),
                        ("block_table", block_table, torch.int32), ("cache_seqlens", cache_seqlens, torch.int32),
                        ("indices", indices, torch.int32)):
        _need_cuda(name, t, dt)
    if q.dim() != 4 or kcache.dim() != 4 or indices.dim() != 3:
        raise ValueError("q must be [b, s_q, h_q, d], kcache [num_blocks, page, h_kv, d], indices [b, s_q, topk]")
    b, s_q, h_q, d = q.shape
    num_blocks, page, h_kv, dk = kcache.shape
    if dk != d or page != _lib.MLA_PAGE_SIZE or tuple(indices.shape[:2]) != (b, s_q):
        raise ValueError("kcache and indices must match q")
    topk = indices.shape[2]
    dev = q.device
    if list_lens is None:
        list_lens = torch.full((b,), topk, dtype=torch.int32, device=dev)
    _need_cuda("list_lens", list_lens, torch.int32)
    if tile_scheduler_metadata is None or num_splits is None:
        tile_scheduler_metadata, num_splits = mla_get_metadata_sparse(list_lens, s_q * h_q // h_kv, h_kv)
    _need_cuda("tile_scheduler_metadata", tile_scheduler_metadata, torch.int32)
    _need_cuda("num_splits", num_splits, torch.int32)
    if (block_table.dim() != 2 or block_table.shape[0] != b or cache_seqlens.numel() != b or list_lens.numel() != b
            or num_splits.numel() != b + 1):
        raise ValueError("batch size differs between q, block_table, cache_seqlens, list_lens and num_splits")
    if tile_scheduler_metadata.dim() != 2 or tile_scheduler_metadata.shape[1] != MLA_METADATA_INTS:
        raise ValueError("tile_scheduler_metadata must be [num_parts, 8]")
    num_parts = tile_scheduler_metadata.shape[0]
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((b, s_q, h_q, dv), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((b, s_q, h_q), dtype=torch.float32, device=dev)
    _need_cuda("out", out, torch.bfloat16)
    _need_cuda("lse", lse, torch.float32)
    if tuple(out.shape) != (b, s_q, h_q, dv) or tuple(lse.shape) != (b, s_q, h_q):
        raise ValueError("out must be [b, s_q, h_q, dv] and lse [b, s_q, h_q]")
    _same_device(dev, kcache=kcache, block_table=block_table, cache_seqlens=cache_seqlens, indices=indices,
                 list_lens=list_lens, tile_scheduler_metadata=tile_scheduler_metadata, num_splits=num_splits,
                 out=out, lse=lse)
    ws_need = mla_workspace_bytes(b, s_q, h_q, h_kv, dv, num_parts) if dv == MLA_V_DIM and h_q % h_kv == 0 else 256
    if workspace is None:
        workspace = torch.empty((ws_need,), dtype=torch.uint8, device=dev)
    _need_cuda("workspace", workspace, torch.uint8)
    _same_device(dev, workspace=workspace)
    with torch.cuda.device(dev):
        st = load().mla_decode_kvcache_sparse(
            q.data_ptr(), kcache.data_ptr(), num_blocks, block_table.data_ptr(), block_table.shape[1],
            cache_seqlens.data_ptr(), indices.data_ptr(), topk, list_lens.data_ptr(), b, s_q, h_q, h_kv, d, dv,
            tile_scheduler_metadata.data_ptr(), num_splits.data_ptr(), num_parts, float(softmax_scale),
            out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream_handle(dev))
    check("mla_decode_kvcache_sparse", st)
    return out, lse


def mla_decode_kvcache_noalloc(q: torch.Tensor, kcache: torch.Tensor, block_table: torch.Tensor,
                               cache_seqlens: torch.Tensor, dv: int, tile_scheduler_metadata: torch.Tensor,
                               num_splits: torch.Tensor, out: torch.Tensor, lse: torch.Tensor,
                               softmax_scale: Optional[float] = None, causal: bool = False) -> None:
    """Decode into caller-provided ``out`` / ``lse`` without any device allocation.

    For callers that cannot allocate at decode time: the split-KV scratch is
    the library's fixed internal array (``MLA_NOALLOC_SCRATCH_BYTES``), shared
    by every call, so calls must not overlap on the GPU.  Make the first call
    on a device before any stream capture (it looks up the array's address).
    """
    b, s_q, h_q, d, num_blocks, h_kv, num_parts, out, lse = _dense_decode_args(
        q, kcache, block_table, cache_seqlens, dv, tile_scheduler_metadata, num_splits, out, lse, allocate=False)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    dev = q.device
    with torch.cuda.device(dev):
        st = load().mla_decode_kvcache_noalloc(
            q.data_ptr(), kcache.data_ptr(), num_blocks, block_table.data_ptr(), block_table.shape[1],
            cache_seqlens.data_ptr(), b, s_q, h_q, h_kv, d, dv, tile_scheduler_metadata.data_ptr(),
            num_splits.data_ptr(), num_parts, float(softmax_scale), int(bool(causal)),
            out.data_ptr(), lse.data_ptr(), _stream_handle(dev))
    check("mla_decode_kvcache_noalloc", st)


# Serving loops make the calls below once per layer and token, so the host's
# share of a small call counts: what depends on the device or on shapes alone is
# asked of the library once, and the device is switched only when it is not the
# current one.
def _call(name: str, dev: torch.device, *args) -> None:
    """Run a library call on ``dev`` and its current stream; raise on a bad status."""
    fn = getattr(_lib._lib or load(), name)
    index = dev.index
    if index == torch.cuda.current_device():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st != _lib.MLA_OK:
        check(name, st)


def _on(dev: torch.device, of: str, name: str, t: torch.Tensor, dtype: torch.dtype) -> int:
    """Check a contiguous CUDA tensor on ``dev``; returns its address."""
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == dev and t.is_contiguous()):
        _need_cuda(name, t, dtype)
        _same_device(dev, of, **{name: t})
    return t.data_ptr()


@functools.lru_cache(maxsize=None)
def _pairs(index: int) -> int:
    """CTA pairs of a device: the split-KV parts of a decode over row tiles."""
    return mla_num_sm_parts(1, 1, torch.device("cuda", index))


# ---------------------------------------------------------------- cache rows
def _need_rows(name: str, t: torch.Tensor, cols: int, n: int, dev: torch.device, written: bool) -> int:
    """bf16 [n, cols] with unit inner stride, 16-byte aligned rows; returns the row stride in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.device != dev:
        _same_device(dev, "cache", **{name: t})
    if t.dim() != 2 or t.shape[0] != n or t.shape[1] != cols:
        raise ValueError(f"{name} must be [{n}, {cols}]")
    stride, inner = t.stride()
    if n <= 1:
        stride = cols
    if inner != 1 or stride % 8 or (written and stride < cols):
        raise ValueError(f"{name}: rows must be contiguous, the row stride a multiple of 8 elements"
                         + (" and rows must not overlap" if written else ""))
    if t.data_ptr() % 16:
        raise ValueError(f"{name} must be 16-byte aligned")
    return stride


def _row_count(latent) -> int:
    if not isinstance(latent, torch.Tensor):
        raise TypeError("latent must be a torch.Tensor")
    if latent.dim() != 2:
        raise ValueError(f"latent must be [n, {MLA_V_DIM}]")
    return latent.shape[0]


def _paged_args(cache, block_table, fp8):
    """Check a paged cache and its table; returns (num_blocks, d, b, max_blocks, device, address of the table)."""
    if fp8:
        _need_cuda("kv_pages", cache, torch.uint8)
        d = _lib.MLA_HEAD_DIM
        if cache.dim() != 2 or cache.shape[1] != _FP8_PAGE:
            raise ValueError(f"kv_pages must be [num_blocks, {_FP8_PAGE}]")
        num_blocks = cache.shape[0]
    else:
        _need_cuda("kcache", cache, torch.bfloat16)
        if cache.dim() != 4:
            raise ValueError("kcache must be [num_blocks, 64, 1, d]")
        num_blocks, page, h_kv, d = cache.shape
        if page != _lib.MLA_PAGE_SIZE or h_kv != 1:
            raise ValueError("kcache must be [num_blocks, 64, 1, d]")
    dev = cache.device
    table = _on(dev, "cache", "block_table", block_table, torch.int32)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [b, max_blocks]")
    b, max_blocks = block_table.shape
    if b < 1 or max_blocks < 1:
        raise ValueError("block_table must be [b, max_blocks], neither of them 0")
    return num_blocks, d, b, max_blocks, dev, table


_FP8_PAGE = _lib.MLA_FP8_PAGE_BYTES(_lib.MLA_HEAD_DIM)


def _vector(dev: torch.device, of: str, name: str, t: torch.Tensor, n: int) -> int:
    """Check an int32 [n] on ``dev``; returns its address."""
    ptr = _on(dev, of, name, t, torch.int32)
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} must be [{n}]")
    return ptr


def _cache_rows(call, cache, block_table, starts, num_rows, cu_rows, latent, k_rope, fp8, write):
    num_blocks, d, b, max_blocks, dev, table = _paged_args(cache, block_table, fp8)
    st_ptr = _vector(dev, "cache", "starts", starts, b)
    cu_ptr = None
    if cu_rows is not None:
        cu_ptr = _vector(dev, "cache", "cu_rows", cu_rows, b + 1)
    elif num_rows % b:
        raise ValueError("without cu_rows every sequence has the same number of rows: b must divide them")
    ls = _need_rows("latent", latent, MLA_V_DIM, num_rows, dev, not write)
    rs, rope_ptr = 0, None
    if d > MLA_V_DIM:
        rs = _need_rows("k_rope", k_rope, d - MLA_V_DIM, num_rows, dev, not write)
        rope_ptr = k_rope.data_ptr()
    elif k_rope is not None:
        raise ValueError("a cache of 512-wide rows has no RoPE part: k_rope must be None")
    if write:
        _call(call, dev, latent.data_ptr(), ls, rope_ptr, rs, num_rows, cu_ptr, st_ptr, b, cache.data_ptr(), num_blocks,
              table, max_blocks, d)
    else:
        _call(call, dev, cache.data_ptr(), num_blocks, table, max_blocks, st_ptr, cu_ptr, b, num_rows,
              latent.data_ptr(), ls, rope_ptr, rs, d)


def mla_cache_write(latent: torch.Tensor, k_rope: Optional[torch.Tensor], kcache: torch.Tensor,
                    block_table: torch.Tensor, starts: torch.Tensor, cu_rows: Optional[torch.Tensor] = None) -> None:
    """Write new tokens' rows into the bf16 cache, in place.

    Rows ``cu_rows[b] .. cu_rows[b + 1]`` of ``latent`` bf16 [n, 512] and
    ``k_rope`` bf16 [n, 64] (None for a cache of 512-wide rows) go to positions
    ``starts[b], starts[b] + 1, ...`` of sequence b; without ``cu_rows`` every
    sequence has n / b rows.  Rows behind ``cu_rows[b]`` are ignored.  The
    inputs may be slices of wider rows (strides of a multiple of 8 elements)."""
    _cache_rows("mla_cache_write", kcache, block_table, starts, _row_count(latent), cu_rows, latent, k_rope, False, True)


def mla_cache_write_fp8(latent: torch.Tensor, k_rope: torch.Tensor, kv_pages: torch.Tensor,
                        block_table: torch.Tensor, starts: torch.Tensor, cu_rows: Optional[torch.Tensor] = None) -> None:
    """``mla_cache_write`` into packed e4m3 pages (uint8 [num_blocks, MLA_FP8_PAGE_BYTES(576)]): each row is
    quantised as it is written, with its own scale max |x| / 448."""
    _cache_rows("mla_cache_write_fp8", kv_pages, block_table, starts, _row_count(latent), cu_rows, latent, k_rope, True,
                True)


def _cache_read(call, cache, block_table, starts, num_rows, cu_rows, latent, k_rope, fp8):
    num_rows = int(num_rows)
    if num_rows < 0:
        raise ValueError("num_rows must not be negative")
    d = _paged_args(cache, block_table, fp8)[1] if latent is None or k_rope is None else 0
    if latent is None:
        latent = torch.empty((num_rows, MLA_V_DIM), dtype=torch.bfloat16, device=cache.device)
    if k_rope is None and d > MLA_V_DIM:
        k_rope = torch.empty((num_rows, d - MLA_V_DIM), dtype=torch.bfloat16, device=cache.device)
    _cache_rows(call, cache, block_table, starts, num_rows, cu_rows, latent, k_rope, fp8, False)
    return latent, k_rope


def mla_cache_read(kcache: torch.Tensor, block_table: torch.Tensor, starts: torch.Tensor, num_rows: int,
                   cu_rows: Optional[torch.Tensor] = None, latent: Optional[torch.Tensor] = None,
                   k_rope: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Read ranges of the bf16 cache back to contiguous rows: (latent bf16
    [num_rows, 512], k_rope bf16 [num_rows, 64], None for 512-wide rows).

    Output rows ``cu_rows[b] .. cu_rows[b + 1]`` are positions ``starts[b],
    starts[b] + 1, ...`` of sequence b (without ``cu_rows``: num_rows / b each).
    Rows behind ``cu_rows[b]`` are left as they were (unset in outputs that the
    call allocates)."""
    return _cache_read("mla_cache_read", kcache, block_table, starts, num_rows, cu_rows, latent, k_rope, False)


def mla_cache_read_fp8(kv_pages: torch.Tensor, block_table: torch.Tensor, starts: torch.Tensor, num_rows: int,
                       cu_rows: Optional[torch.Tensor] = None, latent: Optional[torch.Tensor] = None,
                       k_rope: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``mla_cache_read`` from packed e4m3 pages: scale * code, rounded to bf16."""
    return _cache_read("mla_cache_read_fp8", kv_pages, block_table, starts, num_rows, cu_rows, latent, k_rope, True)


# ---------------------------------------------------------------- page keys and page selection
def _page_key_args(dev, num_blocks, d, page_keys, page_scales):
    """Check the page keys of a cache; returns their addresses."""
    keys = _on(dev, "cache", "page_keys", page_keys, torch.int8)
    scales = _on(dev, "cache", "page_scales", page_scales, torch.float32)
    if page_keys.shape != (num_blocks, d) or page_scales.shape != (num_blocks,):
        raise ValueError(f"page_keys must be [{num_blocks}, {d}] and page_scales [{num_blocks}]")
    return keys, scales


def _update_page_keys(call, cache, block_table, cache_seqlens, page_keys, page_scales, starts, fp8):
    num_blocks, d, b, max_blocks, dev, table = _paged_args(cache, block_table, fp8)
    lens = _vector(dev, "cache", "cache_seqlens", cache_seqlens, b)
    keys, scales = _page_key_args(dev, num_blocks, d, page_keys, page_scales)
    st_ptr = None if starts is None else _vector(dev, "cache", "starts", starts, b)
    _call(call, dev, cache.data_ptr(), num_blocks, table, max_blocks, lens, st_ptr, b, d, keys, scales)


def mla_update_page_keys(kcache: torch.Tensor, block_table: torch.Tensor, cache_seqlens: torch.Tensor,
                         page_keys: torch.Tensor, page_scales: torch.Tensor,
                         starts: Optional[torch.Tensor] = None) -> None:
    """Recompute the keys of the pages that positions ``starts[b] .. cache_seqlens[b]`` touch (every page
    without ``starts``), in place: ``page_keys`` int8 [num_blocks, d] and ``page_scales`` fp32 [num_blocks] hold
    the mean of each page's rows, quantised per page; see ``include/mla_decode.h``."""
    _update_page_keys("mla_update_page_keys", kcache, block_table, cache_seqlens, page_keys, page_scales, starts,
                      False)


def mla_update_page_keys_fp8(kv_pages: torch.Tensor, block_table: torch.Tensor, cache_seqlens: torch.Tensor,
                             page_keys: torch.Tensor, page_scales: torch.Tensor,
                             starts: Optional[torch.Tensor] = None) -> None:
    """``mla_update_page_keys`` over packed e4m3 pages."""
    _update_page_keys("mla_update_page_keys_fp8", kv_pages, block_table, cache_seqlens, page_keys, page_scales,
                      starts, True)


@functools.lru_cache(maxsize=256)
def mla_blocks_workspace_bytes(batch: int, s_q: int, h_q: int, h_kv: int, dv: int, max_blocks: int, topk_pages: int,
                               num_parts: int) -> int:
    n = load().mla_blocks_workspace_bytes(batch, s_q, h_q, h_kv, dv, max_blocks, topk_pages, num_parts)
    if n == 0:
        raise ValueError("invalid shape for the workspace of a decode over selected pages")
    return int(n)


def _outputs(q, b, s_q, h_q, dv, dev, out, lse):
    """The outputs of a decode, created where missing, and their addresses."""
    if out is None:
        out = q.new_empty((b, s_q, h_q, dv))
    elif out.shape != (b, s_q, h_q, dv):
        raise ValueError("out must be [b, s_q, h_q, dv]")
    if lse is None:
        lse = torch.empty((b, s_q, h_q), dtype=torch.float32, device=dev)
    elif lse.shape != (b, s_q, h_q):
        raise ValueError("lse must be [b, s_q, h_q]")
    return out, lse, _on(dev, "q", "out", out, torch.bfloat16), _on(dev, "q", "lse", lse, torch.float32)


def _query_args(q, cache, block_table, cache_seqlens, fp8):
    """Check the query against a paged cache; returns (b, s_q, h_q, d, num_blocks, max_blocks, device, addresses of
    q, the table and the lengths)."""
    num_blocks, d, b, max_blocks, dev, table = _paged_args(cache, block_table, fp8)
    q_ptr = _on(dev, "the cache", "q", q, torch.bfloat16)
    if q.dim() != 4 or q.shape[0] != b or q.shape[3] != d or q.shape[1] < 1 or q.shape[2] < 1:
        raise ValueError(f"q must be [{b}, s_q, h_q, {d}]")
    lens = _vector(dev, "q", "cache_seqlens", cache_seqlens, b)
    return b, q.shape[1], q.shape[2], d, num_blocks, max_blocks, dev, q_ptr, table, lens


def _decode_blocks(call, q, cache, block_table, cache_seqlens, page_keys, page_scales, topk_pages, dv, sink_pages,
                   local_pages, softmax_scale, causal, out, lse, pages, workspace, fp8):
    b, s_q, h_q, d, num_blocks, max_blocks, dev, q_ptr, table, lens = _query_args(q, cache, block_table, cache_seqlens, fp8)
    keys, scales = _page_key_args(dev, num_blocks, d, page_keys, page_scales)
    topk_pages, sink_pages, local_pages = int(topk_pages), int(sink_pages), int(local_pages)
    if sink_pages < 0 or local_pages < 1 or topk_pages < sink_pages + local_pages:
        raise ValueError("topk_pages must cover sink_pages (>= 0) and local_pages (>= 1)")
    if topk_pages * _lib.MLA_PAGE_SIZE > 0x7fffffff:
        raise ValueError("topk_pages is too large")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    num_parts = _pairs(dev.index)
    out, lse, o_ptr, lse_ptr = _outputs(q, b, s_q, h_q, dv, dev, out, lse)
    if pages is None:
        pages = block_table.new_empty((b, s_q, topk_pages))
    elif pages.shape != (b, s_q, topk_pages):
        raise ValueError("pages must be [b, s_q, topk_pages]")
    pages_ptr = _on(dev, "q", "pages", pages, torch.int32)
    if workspace is None:
        need = mla_blocks_workspace_bytes(b, s_q, h_q, 1, dv, max_blocks, topk_pages, num_parts)
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    ws_ptr = _on(dev, "q", "workspace", workspace, torch.uint8)
    _call(call, dev, q_ptr, cache.data_ptr(), num_blocks, table, max_blocks, lens, keys, scales, topk_pages, sink_pages,
          local_pages, b, s_q, h_q, 1, d, dv, num_parts, float(softmax_scale), int(bool(causal)), o_ptr, lse_ptr, pages_ptr,
          ws_ptr, workspace.numel())
    return out, lse, pages


def mla_decode_kvcache_blocks(q: torch.Tensor, kcache: torch.Tensor, block_table: torch.Tensor,
                              cache_seqlens: torch.Tensor, page_keys: torch.Tensor, page_scales: torch.Tensor,
                              topk_pages: int, dv: int, sink_pages: int = 1, local_pages: int = 1,
                              softmax_scale: Optional[float] = None, causal: bool = False,
                              out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                              pages: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                              ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Decode over the pages that each query token selects: the first ``sink_pages``, the last ``local_pages``
    and, up to ``topk_pages``, those whose key (``mla_update_page_keys``) scores highest against its heads.
    Returns (o bf16 [b, s_q, h_q, dv], lse fp32 [b, s_q, h_q], pages int32 [b, s_q, topk_pages]: the
    selected pages, ascending, -1 behind them); see ``include/mla_decode.h``."""
    return _decode_blocks("mla_decode_kvcache_blocks", q, kcache, block_table, cache_seqlens, page_keys, page_scales,
                          topk_pages, dv, sink_pages, local_pages, softmax_scale, causal, out, lse, pages, workspace,
                          False)


def mla_decode_kvcache_blocks_fp8(q: torch.Tensor, kv_pages: torch.Tensor, block_table: torch.Tensor,
                                  cache_seqlens: torch.Tensor, page_keys: torch.Tensor, page_scales: torch.Tensor,
                                  topk_pages: int, dv: int, sink_pages: int = 1, local_pages: int = 1,
                                  softmax_scale: Optional[float] = None, causal: bool = False,
                                  out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                                  pages: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                                  ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """``mla_decode_kvcache_blocks`` over packed e4m3 pages."""
    return _decode_blocks("mla_decode_kvcache_blocks_fp8", q, kv_pages, block_table, cache_seqlens, page_keys,
                          page_scales, topk_pages, dv, sink_pages, local_pages, softmax_scale, causal, out, lse, pages,
                          workspace, True)


# ---------------------------------------------------------------- draft trees
def mla_tree_mask(parents: torch.Tensor) -> torch.Tensor:
    """The masks of draft trees, int32 [b, s_q, ceil(s_q / 32)], from their parent lists (int32 [b, s_q]: a node
    before it, or -1): bit j of row i is set when node j is node i or one of its ancestors."""
    _need_cuda("parents", parents, torch.int32)
    if parents.dim() != 2:
        raise ValueError("parents must be [b, s_q]")
    b, s_q = parents.shape
    dev = parents.device
    mask = torch.empty((b, s_q, (s_q + 31) // 32), dtype=torch.int32, device=dev)
    _call("mla_tree_mask", dev, parents.data_ptr(), b, s_q, mask.data_ptr())
    return mask


def _row_tiles(s_q: int, h_q: int) -> int:
    return (s_q * h_q + _lib.MLA_TILE_ROWS - 1) // _lib.MLA_TILE_ROWS


def mla_get_metadata_tree(cache_seqlens: torch.Tensor, s_q: int, h_q: int, tree_lens: Optional[torch.Tensor] = None,
                          num_parts: Optional[int] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The work partition of a draft-tree decode, over the 128-row tiles of every sequence:
    (tile_scheduler_metadata int32 [P, 8], num_splits int32 [b * ceil(s_q * h_q / 128) + 1]).  It depends on the
    lengths and shapes only: one call serves every layer of a step."""
    _need_cuda("cache_seqlens", cache_seqlens, torch.int32)
    dev = cache_seqlens.device
    b = cache_seqlens.numel()
    s_q, h_q = int(s_q), int(h_q)
    if b < 1 or s_q < 1 or h_q < 1:
        raise ValueError("cache_seqlens, s_q and h_q must not be empty or 0")
    nodes = None if tree_lens is None else _vector(dev, "cache_seqlens", "tree_lens", tree_lens, b)
    if num_parts is None:
        num_parts = _pairs(dev.index)
    md = torch.empty((num_parts, MLA_METADATA_INTS), dtype=torch.int32, device=dev)
    ns = torch.empty((b * _row_tiles(s_q, h_q) + 1,), dtype=torch.int32, device=dev)
    _call("mla_get_metadata_tree", dev, cache_seqlens.data_ptr(), nodes, b, s_q, h_q, 1, int(num_parts), md.data_ptr(),
          ns.data_ptr())
    return md, ns


@functools.lru_cache(maxsize=256)
def mla_tree_workspace_bytes(batch: int, s_q: int, h_q: int, h_kv: int, dv: int, num_parts: int) -> int:
    n = load().mla_tree_workspace_bytes(batch, s_q, h_q, h_kv, dv, num_parts)
    if n == 0:
        raise ValueError("invalid shape for the workspace of a draft-tree decode")
    return int(n)


def _decode_tree(call, q, cache, block_table, cache_seqlens, tree_mask, dv, tile_scheduler_metadata, num_splits,
                 tree_lens, softmax_scale, out, lse, workspace, fp8):
    b, s_q, h_q, d, num_blocks, max_blocks, dev, q_ptr, table, lens = _query_args(q, cache, block_table, cache_seqlens, fp8)
    mask = _on(dev, "q", "tree_mask", tree_mask, torch.int32)
    if tree_mask.shape != (b, s_q, (s_q + 31) // 32):
        raise ValueError("tree_mask must be [b, s_q, ceil(s_q / 32)]")
    nodes = None if tree_lens is None else _vector(dev, "q", "tree_lens", tree_lens, b)
    md = ns = None
    if (tile_scheduler_metadata is None) != (num_splits is None):
        raise ValueError("tile_scheduler_metadata and num_splits come together")
    if tile_scheduler_metadata is None:
        num_parts = _pairs(dev.index)
    else:
        md = _on(dev, "q", "tile_scheduler_metadata", tile_scheduler_metadata, torch.int32)
        ns = _vector(dev, "q", "num_splits", num_splits, b * _row_tiles(s_q, h_q) + 1)
        if tile_scheduler_metadata.dim() != 2 or tile_scheduler_metadata.shape[1] != MLA_METADATA_INTS:
            raise ValueError("tile_scheduler_metadata must be [num_parts, 8]")
        num_parts = tile_scheduler_metadata.shape[0]
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    out, lse, o_ptr, lse_ptr = _outputs(q, b, s_q, h_q, dv, dev, out, lse)
    if workspace is None:
        need = mla_tree_workspace_bytes(b, s_q, h_q, 1, dv, num_parts)
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    ws_ptr = _on(dev, "q", "workspace", workspace, torch.uint8)
    _call(call, dev, q_ptr, cache.data_ptr(), num_blocks, table, max_blocks, lens, mask, nodes, b, s_q, h_q, 1, d, dv, md, ns,
          num_parts, float(softmax_scale), o_ptr, lse_ptr, ws_ptr, workspace.numel())
    return out, lse


def mla_decode_kvcache_tree(q: torch.Tensor, kcache: torch.Tensor, block_table: torch.Tensor,
                            cache_seqlens: torch.Tensor, tree_mask: torch.Tensor, dv: int,
                            tile_scheduler_metadata: Optional[torch.Tensor] = None,
                            num_splits: Optional[torch.Tensor] = None, tree_lens: Optional[torch.Tensor] = None,
                            softmax_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                            lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                            ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Decode of draft trees: the last ``tree_lens[b]`` (default s_q) cached rows of each sequence are drafted
    nodes, query token i is node i, and it sees every position before the nodes and the nodes of its row of
    ``tree_mask`` (``mla_tree_mask``).  Rows behind a shorter tree get o = 0, lse = -inf.  The work partition
    (``mla_get_metadata_tree``) is computed when not given.  Returns (o, lse) as
    ``mla_decode_kvcache``."""
    return _decode_tree("mla_decode_kvcache_tree", q, kcache, block_table, cache_seqlens, tree_mask, dv,
                        tile_scheduler_metadata, num_splits, tree_lens, softmax_scale, out, lse, workspace, False)


def mla_decode_kvcache_tree_fp8(q: torch.Tensor, kv_pages: torch.Tensor, block_table: torch.Tensor,
                                cache_seqlens: torch.Tensor, tree_mask: torch.Tensor, dv: int,
                                tile_scheduler_metadata: Optional[torch.Tensor] = None,
                                num_splits: Optional[torch.Tensor] = None, tree_lens: Optional[torch.Tensor] = None,
                                softmax_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                                lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                                ) -> Tuple[torch.Tensor, torch.Tensor]:
    """``mla_decode_kvcache_tree`` over packed e4m3 pages."""
    return _decode_tree("mla_decode_kvcache_tree_fp8", q, kv_pages, block_table, cache_seqlens, tree_mask, dv,
                        tile_scheduler_metadata, num_splits, tree_lens, softmax_scale, out, lse, workspace, True)


def mla_device_status(clear: bool = True) -> int:
    """Synchronize and return the OR of the MLA_DEVERR_* bits kernels raised."""
    v = ctypes.c_int(0)
    check("mla_device_status", load().mla_device_status(ctypes.byref(v), int(bool(clear))))
    return v.value


def mla_set_timing_events(split_begin: Optional[torch.cuda.Event], split_end: Optional[torch.cuda.Event]) -> None:
    """Record the two events around the split-KV kernel of every later decode call (None, None: stop)."""
    b = split_begin.cuda_event if split_begin is not None else None
    e = split_end.cuda_event if split_end is not None else None
    check("mla_set_timing_events", load().mla_set_timing_events(b, e))


def mla_set_cluster_multicast(enabled: bool) -> None:
    """Sparse decode: split each list chunk's row gathers between the CTA pair with
    cluster multicast (True, the default) or have each CTA gather its own rows
    (False; processes that run one job across several GPUs use this)."""
    check("mla_set_cluster_multicast", load().mla_set_cluster_multicast(int(bool(enabled))))


# the usage page's names for the same two calls
get_mla_metadata = mla_get_metadata
flash_mla_with_kvcache = mla_decode_kvcache
