"""The serving calls for long and shared contexts: attention with shared prefixes; mean keys
of a cache's pages, the pages each query attends, and attention over those alone.  Prepared
calls (classes) and the functions of the C names, as in serve.py."""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import _ptr, lib
from .serve import _MAX_SEQ_LEN, AttentionResult, NVFP4KVCache, _head_rows, _need, _Prepared


class _Keys(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


def _int32(value: int, name: str, lo: int) -> int:
    """A 32-bit argument: a larger one must not wrap into another."""
    if not lo <= value < 1 << 31:
        raise ValueError(f"{name} must be in [{lo}, 2^31), got {value}")
    return int(value)


def _sequences(block_table: torch.Tensor, seq_lens: torch.Tensor, q_starts: torch.Tensor, dev):
    """Checks them; batch, pages of a row, row stride."""
    _need(block_table, "block_table", (torch.int32,), dev, 2)
    _need(seq_lens, "seq_lens", (torch.int32,), dev, 1)
    _need(q_starts, "q_starts", (torch.int32,), dev, 1)
    batch, pages = block_table.shape
    if seq_lens.shape[0] != batch or q_starts.shape[0] != batch + 1:
        raise ValueError("seq_lens is [batch], q_starts [batch + 1]")
    if not seq_lens.is_contiguous() or not q_starts.is_contiguous() or (block_table.numel() > 0 and pages > 1
                                                                        and block_table.stride(1) != 1):
        raise ValueError("seq_lens, q_starts and the rows of block_table must be contiguous")
    return batch, pages, block_table.stride(0) if batch > 1 else pages


def _outputs(q: torch.Tensor, out: Optional[torch.Tensor], lse: bool, d: int, dev):
    """Attention's out (a fresh one is zeroed once), its token stride, and lse."""
    total, hq = q.shape[0], q.shape[1]
    if out is None:
        out = torch.zeros((total, hq, d), dtype=torch.bfloat16, device=dev)
    ld_out = _head_rows(out, "out", hq, d, dev)
    if out.shape[0] != total:
        raise ValueError("out must hold as many rows as q")
    return out, ld_out, torch.zeros((total, hq), dtype=torch.float32, device=dev) if lse else None


def _workspace(workspace: Optional[torch.Tensor], need: int, dev) -> Optional[torch.Tensor]:
    if workspace is None:
        return torch.empty((need,), dtype=torch.uint8, device=dev) if need > 0 else None
    if not _need(workspace, "workspace", (torch.uint8,), dev, 1).is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace


# ---------------------------------------------------------------------------- shared prefixes
def mxq_attention_prefix_nvfp4_workspace_size(q_heads: int, kv_heads: int, head_dim: int, batch: int, groups: int,
                                              total_q: int, max_q_len: int, max_prefix_len: int, max_own_len: int) -> int:
    return int(lib().mxq_attention_prefix_nvfp4_workspace_size(q_heads, kv_heads, head_dim, batch, groups, total_q, max_q_len,
                                                               max_prefix_len, max_own_len))


class AttentionPrefixNVFP4(_Prepared):
    """A prepared attention call where groups of sequences share prefixes.  group_starts:
    int32 [groups + 1], the first sequence of each group and batch; prefix_lens: int32
    [batch], the tokens of each sequence that are read through the pages of its group's
    first.  max_prefix_len, max_own_len (default: what the table can hold) bound the longest
    prefix and the most tokens behind one, to plan the split for.  Sequences that share
    nothing belong in one group with prefix_lens 0, not in groups of one (the split is planned
    for groups of about the same size).  The rest as AttentionNVFP4, without a window."""

    def __init__(self, q: torch.Tensor, cache: NVFP4KVCache, block_table: torch.Tensor, seq_lens: torch.Tensor,
                 q_starts: torch.Tensor, group_starts: torch.Tensor, prefix_lens: torch.Tensor, max_q_len: int,
                 max_prefix_len: Optional[int] = None, max_own_len: Optional[int] = None, scale: Optional[float] = None,
                 lse: bool = False, out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
        dev, d = cache.device, cache.head_dim
        ld_q = _head_rows(q, "q", None, d, dev)
        total, hq = q.shape[0], q.shape[1]
        out, ld_out, lse_t = _outputs(q, out, lse, d, dev)
        batch, pages, ld_table = _sequences(block_table, seq_lens, q_starts, dev)
        _need(group_starts, "group_starts", (torch.int32,), dev, 1)
        _need(prefix_lens, "prefix_lens", (torch.int32,), dev, 1)
        groups = group_starts.shape[0] - 1
        if groups < 1 or prefix_lens.shape[0] != batch:
            raise ValueError("group_starts is [groups + 1], prefix_lens [batch]")
        if not group_starts.is_contiguous() or not prefix_lens.is_contiguous():
            raise ValueError("group_starts and prefix_lens must be contiguous")
        held = min(pages * cache.page_size, _MAX_SEQ_LEN)
        max_prefix_len = held if max_prefix_len is None else max_prefix_len
        max_own_len = held if max_own_len is None else max_own_len
        need = mxq_attention_prefix_nvfp4_workspace_size(hq, cache.kv_heads, d, batch, groups, total, max_q_len,
                                                         max_prefix_len, max_own_len)
        self.workspace = workspace = _workspace(workspace, need, dev)
        self.out, self._cache = AttentionResult(out, lse_t), cache
        self._bind("mxq_attention_prefix_nvfp4", dev,
                   (q, out, lse_t, block_table, seq_lens, q_starts, group_starts, prefix_lens, workspace, *cache.tensors()),
                   _ptr(q), ld_q, hq, total, _ptr(out), ld_out, _ptr(lse_t), ctypes.byref(cache._c), _ptr(block_table),
                   ld_table, pages, _ptr(seq_lens), _ptr(q_starts), batch, _ptr(group_starts), _ptr(prefix_lens), groups,
                   max_q_len, max_prefix_len, max_own_len, float(scale) if scale is not None else 1.0 / math.sqrt(d),
                   _ptr(workspace), workspace.numel() if workspace is not None else 0)

    def __call__(self, stream=None) -> AttentionResult:
        return self._launch(stream)


def mxq_attention_prefix_nvfp4(q: torch.Tensor, cache: NVFP4KVCache, block_table: torch.Tensor, seq_lens: torch.Tensor,
                               q_starts: torch.Tensor, group_starts: torch.Tensor, prefix_lens: torch.Tensor,
                               max_q_len: int, max_prefix_len: Optional[int] = None, max_own_len: Optional[int] = None,
                               scale: Optional[float] = None, lse: bool = False, out: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None, stream=None) -> AttentionResult:
    """Causal attention of sequences whose groups share prefixes, each attended once."""
    return AttentionPrefixNVFP4(q, cache, block_table, seq_lens, q_starts, group_starts, prefix_lens, max_q_len,
                                max_prefix_len, max_own_len, scale, lse, out, workspace)(stream)


# ---------------------------------------------------------------------------- mean keys
class PageKeys:
    """The mean keys of a cache's pages.  codes: int8 [pages][kv_heads][head_dim]; scales:
    float32 [pages][kv_heads]; page_size: tokens of a page."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, page_size: int):
        dev = codes.device
        pages, heads, d = _need(codes, "codes", (torch.int8,), dev, 3).shape
        _need(scales, "scales", (torch.float32,), dev, 2)
        if tuple(scales.shape) != (pages, heads):
            raise ValueError(f"scales must be [{pages}][{heads}], got {tuple(scales.shape)}")
        if not codes.is_contiguous() or not scales.is_contiguous():
            raise ValueError("codes and scales must be contiguous")
        self.codes, self.scales, self.device = codes, scales, dev
        self.num_pages, self.kv_heads, self.head_dim, self.page_size = pages, heads, d, _int32(page_size, "page_size", 1)
        self._c = _Keys(codes.data_ptr(), scales.data_ptr(), pages, self.page_size, heads, d)

    @classmethod
    def allocate(cls, cache: NVFP4KVCache):
        """Zeroed, for every page of a cache."""
        shape = (cache.num_pages, cache.kv_heads)
        return cls(torch.zeros((*shape, cache.head_dim), dtype=torch.int8, device=cache.device),
                   torch.zeros(shape, dtype=torch.float32, device=cache.device), cache.page_size)


class PageKeysNVFP4(_Prepared):
    """A prepared update of mean keys.  slots: int64 [tokens], those of the append that it
    follows; the pages whose last row is among them get their mean keys."""

    def __init__(self, cache: NVFP4KVCache, slots: torch.Tensor, keys: PageKeys):
        dev = cache.device
        _need(slots, "slots", (torch.int64,), dev, 1)
        if not slots.is_contiguous():
            raise ValueError("slots must be contiguous")
        if keys.device != dev:
            raise ValueError(f"the mean keys are on {keys.device}, expected {dev}")
        self.out, self._cache = keys, cache
        self._bind("mxq_page_keys_nvfp4", dev, (slots, keys.codes, keys.scales, *cache.tensors()),
                   ctypes.byref(cache._c), _ptr(slots), slots.shape[0], ctypes.byref(keys._c))

    def __call__(self, stream=None) -> PageKeys:
        return self._launch(stream)


def mxq_page_keys_nvfp4(cache: NVFP4KVCache, slots: torch.Tensor, keys: PageKeys, stream=None) -> PageKeys:
    """The mean keys of the pages whose last row is among slots."""
    return PageKeysNVFP4(cache, slots, keys)(stream)


# ---------------------------------------------------------------------------- selection
def mxq_select_pages_nvfp4_workspace_size(q_heads: int, kv_heads: int, page_size: int, batch: int, total_q: int,
                                          max_seq_len: int) -> int:
    return int(lib().mxq_select_pages_nvfp4_workspace_size(q_heads, kv_heads, page_size, batch, total_q, max_seq_len))


class SelectPagesNVFP4(_Prepared):
    """A prepared selection of pages.  q: [total_q][q_heads][d] BF16 (rotated); block_table,
    seq_lens, q_starts: as for attention.  Each query and cached head gets at most `top`
    pages of its sequence, ascending and filled up with -1: the first `first`, the last
    `last` with its own, and those of the highest scores.  max_seq_len (default: what the
    table can hold) is the length to hold scores for.  Its result, the int32 tensor
    [total_q][kv_heads][top], leaves rows that belong to no sequence as they were (a fresh
    one holds -1)."""

    def __init__(self, q: torch.Tensor, keys: PageKeys, block_table: torch.Tensor, seq_lens: torch.Tensor,
                 q_starts: torch.Tensor, top: int, first: int = 1, last: int = 2, max_seq_len: Optional[int] = None,
                 out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
        dev, d = keys.device, keys.head_dim
        ld_q = _head_rows(q, "q", None, d, dev)
        total, hq = q.shape[0], q.shape[1]
        batch, pages, ld_table = _sequences(block_table, seq_lens, q_starts, dev)
        top, first, last = _int32(top, "top", 1), _int32(first, "first", 0), _int32(last, "last", 1)
        if max_seq_len is None:
            max_seq_len = min(pages * keys.page_size, _MAX_SEQ_LEN)
        shape = (total, keys.kv_heads, top)
        if out is None:
            out = torch.full(shape, -1, dtype=torch.int32, device=dev)
        _need(out, "out", (torch.int32,), dev, 3)
        if tuple(out.shape) != shape or not out.is_contiguous():
            raise ValueError(f"out must be {list(shape)}, contiguous")
        need = mxq_select_pages_nvfp4_workspace_size(hq, keys.kv_heads, keys.page_size, batch, total, max_seq_len)
        self.workspace = workspace = _workspace(workspace, need, dev)
        self.out, self._keys = out, keys
        self._bind("mxq_select_pages_nvfp4", dev, (q, keys.codes, keys.scales, block_table, seq_lens, q_starts, out, workspace),
                   _ptr(q), ld_q, hq, total, ctypes.byref(keys._c), _ptr(block_table), ld_table, pages, _ptr(seq_lens),
                   _ptr(q_starts), batch, max_seq_len, top, first, last, _ptr(out), _ptr(workspace),
                   workspace.numel() if workspace is not None else 0)

    def __call__(self, stream=None) -> torch.Tensor:
        return self._launch(stream)


def mxq_select_pages_nvfp4(q: torch.Tensor, keys: PageKeys, block_table: torch.Tensor, seq_lens: torch.Tensor,
                           q_starts: torch.Tensor, top: int, first: int = 1, last: int = 2,
                           max_seq_len: Optional[int] = None, out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The pages that each query attends, for each cached head."""
    return SelectPagesNVFP4(q, keys, block_table, seq_lens, q_starts, top, first, last, max_seq_len, out, workspace)(stream)


# ---------------------------------------------------------------------------- attention over them
def mxq_attention_pages_nvfp4_workspace_size(q_heads: int, kv_heads: int, head_dim: int, page_size: int, total_q: int,
                                             top: int) -> int:
    return int(lib().mxq_attention_pages_nvfp4_workspace_size(q_heads, kv_heads, head_dim, page_size, total_q, top))


class AttentionPagesNVFP4(_Prepared):
    """A prepared attention call over listed pages of an NVFP4KVCache.  pages: int32
    [total_q][kv_heads][top], as SelectPagesNVFP4 writes them; the rest as AttentionNVFP4,
    without a window."""

    def __init__(self, q: torch.Tensor, cache: NVFP4KVCache, block_table: torch.Tensor, seq_lens: torch.Tensor,
                 q_starts: torch.Tensor, pages: torch.Tensor, scale: Optional[float] = None, lse: bool = False,
                 out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
        dev, d = cache.device, cache.head_dim
        ld_q = _head_rows(q, "q", None, d, dev)
        total, hq = q.shape[0], q.shape[1]
        out, ld_out, lse_t = _outputs(q, out, lse, d, dev)
        batch, table_pages, ld_table = _sequences(block_table, seq_lens, q_starts, dev)
        _need(pages, "pages", (torch.int32,), dev, 3)
        if tuple(pages.shape[:2]) != (total, cache.kv_heads) or not pages.is_contiguous():
            raise ValueError(f"pages must be [{total}][{cache.kv_heads}][top], contiguous")
        top = pages.shape[2]
        need = mxq_attention_pages_nvfp4_workspace_size(hq, cache.kv_heads, d, cache.page_size, total, top)
        self.workspace = workspace = _workspace(workspace, need, dev)
        self.out, self._cache = AttentionResult(out, lse_t), cache
        self._bind("mxq_attention_pages_nvfp4", dev,
                   (q, out, lse_t, block_table, seq_lens, q_starts, pages, workspace, *cache.tensors()),
                   _ptr(q), ld_q, hq, total, _ptr(out), ld_out, _ptr(lse_t), ctypes.byref(cache._c), _ptr(block_table),
                   ld_table, table_pages, _ptr(seq_lens), _ptr(q_starts), batch, _ptr(pages), top,
                   float(scale) if scale is not None else 1.0 / math.sqrt(d), _ptr(workspace),
                   workspace.numel() if workspace is not None else 0)

    def __call__(self, stream=None) -> AttentionResult:
        return self._launch(stream)


def mxq_attention_pages_nvfp4(q: torch.Tensor, cache: NVFP4KVCache, block_table: torch.Tensor, seq_lens: torch.Tensor,
                              q_starts: torch.Tensor, pages: torch.Tensor, scale: Optional[float] = None,
                              lse: bool = False, out: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None, stream=None) -> AttentionResult:
    """Causal attention of the queries over the pages listed for them."""
    return AttentionPagesNVFP4(q, cache, block_table, seq_lens, q_starts, pages, scale, lse, out, workspace)(stream)
