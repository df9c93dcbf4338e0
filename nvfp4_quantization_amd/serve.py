"""The serving calls: residual + RMS norm -> FP8, rotary append to the paged NVFP4 KV
cache, and attention over it.  Prepared calls (classes) check their tensors and build
their ctypes arguments once, allocate outputs and workspace once, and each `()` runs the
kernels on what the tensors hold then; the functions of the C names prepare and call."""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass
from typing import Optional

import torch

from . import _check, _current_stream, _ptr, _stream, lib

MXQ_ROPE_INTERLEAVED = 1
_MAX_SEQ_LEN = (1 << 31) - 128                    # the longest estimate that the library takes


class _KV(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k_codes", "k_scales", "v_codes", "v_scales", "k_global", "v_global")]
                + [("num_pages", ctypes.c_int64)]
                + [(n, ctypes.c_int32) for n in ("page_size", "kv_heads", "head_dim")]
                + [(n, ctypes.c_int64) for n in ("code_stride_page", "code_stride_head", "code_stride_token",
                                                 "scale_stride_page", "scale_stride_head", "scale_stride_token")])


class _Rope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("factor", ctypes.c_double)]


def _need(t: torch.Tensor, name: str, dtypes, device, dim: Optional[int] = None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: expected {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {t.dim()}")
    return t


_BITS16 = (torch.bfloat16, torch.int16, torch.uint16)
_ByRef = type(ctypes.byref(ctypes.c_int()))


class _Prepared:
    """A call whose ctypes arguments are built once.  It runs on its tensors' device,
    whichever is current."""

    def _bind(self, what: str, device, tensors, *args):
        """The C function (the library's own object keeps the declared types, this one takes
        arguments that were converted to them here once), its arguments but the stream, and
        the tensors behind them."""
        types = getattr(lib(), what).argtypes
        self._fn = lib()[what]
        self._fn.restype = ctypes.c_int
        assert len(args) == len(types) - 1
        self._args = tuple(a if isinstance(a, (ctypes.c_void_p, _ByRef)) else t(a) for a, t in zip(args, types))
        self._what, self._device, self._tensors = what, device, tensors
        self._index = device.index if device.type == "cuda" else None

    def _launch(self, stream):
        index = self._index
        if index is None:
            raise ValueError(f"{self._what}: the tensors are on {self._device}, expected a GPU")
        if index == torch.cuda.current_device():
            self._run(index, stream)
        else:
            with torch.cuda.device(index):
                self._run(index, stream)
        return self.out

    def _run(self, index, stream):
        st = self._fn(*self._args, _current_stream(index) if stream is None else _stream(stream, *self._tensors))
        if st:
            _check(st, self._what)


# ---------------------------------------------------------------------------- RMS norm -> FP8
@dataclass
class RMSNormFP8Result:
    q: torch.Tensor                               # [m][n] uint8 (E4M3)
    scales: torch.Tensor                          # [m][n/128] float32 (or [n/128][m])
    residual: Optional[torch.Tensor] = None       # [m][n] bfloat16: x + residual (None without one)
    y: Optional[torch.Tensor] = None              # [m][n] bfloat16: the norm (when asked for)


class AddRMSNormFP8(_Prepared):
    """A prepared residual addition + RMS norm -> FP8 1x128 call.  x, residual: [m][n]
    BF16 with unit column stride; weight: [n] BF16.  residual_out: where x + residual goes
    (default: a tensor of its own; residual itself updates in place).  options: 0 or
    MXQ_FP8_UE8M0; out_bf16: also the norm in BF16; scale_transposed: scales [n/128][m]."""

    def __init__(self, x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, options: int = 0, out_bf16: bool = False, scale_transposed: bool = False,
                 residual_out: Optional[torch.Tensor] = None):
        dev = x.device
        _need(x, "x", _BITS16, dev, 2)
        m, n = x.shape
        _need(weight, "weight", _BITS16, dev, 1)
        if weight.shape[0] != n or (n > 1 and weight.stride(0) != 1):
            raise ValueError("weight must be [n], contiguous")
        if residual is None and residual_out is not None:
            raise ValueError("residual_out needs a residual")
        if residual is not None and residual_out is None:
            residual_out = torch.empty((m, n), dtype=torch.bfloat16, device=dev)
        for name, t in (("x", x), ("residual", residual), ("residual_out", residual_out)):
            if t is None:
                continue
            _need(t, name, _BITS16, dev, 2)
            if t.shape != (m, n) or (t.numel() > 0 and t.stride(1) != 1):
                raise ValueError(f"{name} must be [m][n] with unit column stride")
        q = torch.empty((m, n), dtype=torch.uint8, device=dev)
        scales = torch.empty((n // 128, m) if scale_transposed else (m, n // 128), dtype=torch.float32, device=dev)
        y = torch.empty((m, n), dtype=torch.bfloat16, device=dev) if out_bf16 else None
        sr, sg = (1, m) if scale_transposed else (n // 128, 1)

        def rows(t):
            """Row stride.  A dimension of one has none to speak of: torch may report any."""
            return 0 if t is None else t.stride(0) if m > 1 else n

        self.out = RMSNormFP8Result(q, scales, residual_out, y)
        self._bind("mxq_add_rmsnorm_quant_fp8", dev, (x, residual, residual_out, weight, y, q, scales),
                   _ptr(x), rows(x), _ptr(residual), rows(residual), _ptr(residual_out), rows(residual_out),
                   _ptr(weight), float(eps), m, n, options, _ptr(y), n, _ptr(q), n, _ptr(scales), sr, sg)

    def __call__(self, stream=None) -> RMSNormFP8Result:
        return self._launch(stream)


def mxq_add_rmsnorm_quant_fp8(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                              eps: float = 1e-6, options: int = 0, out_bf16: bool = False,
                              scale_transposed: bool = False, residual_out: Optional[torch.Tensor] = None,
                              stream=None) -> RMSNormFP8Result:
    """BF16(x + residual) -> RMS norm with weight -> FP8 1x128, one pass."""
    return AddRMSNormFP8(x, weight, residual, eps, options, out_bf16, scale_transposed, residual_out)(stream)


# ---------------------------------------------------------------------------- the cache
class NVFP4KVCache:
    """A paged KV cache in NVFP4.  k_codes, v_codes: uint8 [pages][kv_heads][page_size]
    [head_dim/2]; k_scales, v_scales: uint8 (E4M3) [..][head_dim/16]; k_global, v_global:
    float32 [kv_heads], the tensor scale of each head.  The first three dimensions may be
    strided in any way (a [pages][page_size][kv_heads][...] buffer goes in transposed), the
    same for K and V."""

    def __init__(self, k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor, v_scales: torch.Tensor,
                 k_global: torch.Tensor, v_global: torch.Tensor):
        dev = k_codes.device
        pages, heads, page, half = _need(k_codes, "k_codes", (torch.uint8,), dev, 4).shape
        for name, t, width in (("k_codes", k_codes, half), ("v_codes", v_codes, half),
                               ("k_scales", k_scales, half // 8), ("v_scales", v_scales, half // 8)):
            _need(t, name, (torch.uint8,), dev, 4)
            if tuple(t.shape) != (pages, heads, page, width) or (t.numel() > 0 and t.stride(3) != 1):
                raise ValueError(f"{name} must be [{pages}][{heads}][{page}][{width}] with unit last stride")
        for name, t in (("k_global", k_global), ("v_global", v_global)):
            _need(t, name, (torch.float32,), dev, 1)
            if t.shape[0] != heads or not t.is_contiguous():
                raise ValueError(f"{name} must be [{heads}], contiguous")

        def strides(t):
            """A dimension of one has no stride to speak of: torch may report any."""
            width = t.shape[3]
            tok = t.stride(2) if t.shape[2] > 1 else width
            return (t.stride(0) if t.shape[0] > 1 else 0, t.stride(1) if t.shape[1] > 1 else 0, tok)

        if strides(k_codes) != strides(v_codes) or strides(k_scales) != strides(v_scales):
            raise ValueError("K and V of a cache share their strides")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.k_global, self.v_global = k_global, v_global
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, page, 2 * half
        self.device = dev
        self._c = _KV(*[t.data_ptr() for t in self.tensors()], pages, page, heads, 2 * half, *strides(k_codes),
                      *strides(k_scales))

    @classmethod
    def allocate(cls, num_pages: int, page_size: int, kv_heads: int, head_dim: int, k_amax, v_amax, device="cuda"):
        """A zeroed cache.  k_amax, v_amax: the largest magnitude each head is calibrated
        to hold (a float, or one per head); the tensor scale of a head is
        max(amax, 1e-10) / 2688, and larger values saturate."""
        def codes(width):
            return torch.zeros((num_pages, kv_heads, page_size, width), dtype=torch.uint8, device=device)

        def scale(amax):
            a = torch.as_tensor(amax, dtype=torch.float32).expand(kv_heads).clamp(min=1e-10)
            return (a * torch.tensor(1.0 / 2688.0, dtype=torch.float32)).to(device)

        return cls(codes(head_dim // 2), codes(head_dim // 16), codes(head_dim // 2), codes(head_dim // 16),
                   scale(k_amax), scale(v_amax))

    def tensors(self) -> tuple:
        return (self.k_codes, self.k_scales, self.v_codes, self.v_scales, self.k_global, self.v_global)


# ---------------------------------------------------------------------------- rotary append
class RopePlan:
    """Rotary positions: inv_freq, a float64 tensor of rot_dim / 2 angles per position (on
    the tokens' device), interleaved pairs (2i, 2i + 1) or halves (i, i + rot_dim/2), and
    the factor on cos and sin."""

    def __init__(self, inv_freq: torch.Tensor, interleaved: bool = False, factor: float = 1.0):
        _need(inv_freq, "inv_freq", (torch.float64,), inv_freq.device, 1)
        self.inv_freq, self.interleaved, self.factor = inv_freq.contiguous(), bool(interleaved), float(factor)
        self.rot_dim = 2 * inv_freq.shape[0]
        self._c = _Rope(self.inv_freq.data_ptr() if self.rot_dim else None, self.rot_dim,
                        MXQ_ROPE_INTERLEAVED if interleaved else 0, self.factor)


def rope_plan(rot_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
              scale: float = 1.0, trained_length: int = 0, fast_turns: float = 32.0, slow_turns: float = 1.0,
              device="cuda") -> RopePlan:
    """The plan of base^(-2i / rot_dim) angles per position, scaled for contexts `scale`
    times the trained ones:
      "none"    as they are
      "linear"  every frequency divided by scale (positions interpolated)
      "base"    base multiplied by scale^(rot_dim / (rot_dim - 2)): the slowest pair slows
                by scale, the fastest keeps its frequency
      "ramp"    by parts (Peng, Quesnelle, Fan, Shippole, "YaRN", 2023): pairs that turn
                more than fast_turns times over trained_length positions keep their
                frequency, those under slow_turns are divided by scale, a linear ramp in
                between; cos and sin are multiplied by 0.1 ln(scale) + 1."""
    if rot_dim % 2 or rot_dim < 0:
        raise ValueError("rot_dim must be even")
    if scaling not in ("none", "linear", "base", "ramp"):
        raise ValueError(f"scaling: {scaling!r} is none of none, linear, base, ramp")
    if not scale >= 1.0:
        raise ValueError("scale must be at least 1")
    if scaling == "base" and rot_dim > 2:
        base = base * scale ** (rot_dim / (rot_dim - 2))
    f = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / max(rot_dim, 1))
    factor = 1.0
    if scaling == "linear":
        f = f / scale
    elif scaling == "ramp":
        if trained_length <= 0 or not fast_turns > slow_turns:
            raise ValueError("ramp needs trained_length, and fast_turns above slow_turns")
        turns = f * trained_length / (2.0 * math.pi)
        keep = ((turns - slow_turns) / (fast_turns - slow_turns)).clamp(0.0, 1.0)
        f = f * keep + f / scale * (1.0 - keep)
        factor = 0.1 * math.log(scale) + 1.0
    return RopePlan(f.to(device), interleaved, factor)


@dataclass
class RopeAppendResult:
    q: Optional[torch.Tensor]                     # [tokens][q_heads][head_dim] bfloat16, rotated
    k_values: Optional[torch.Tensor] = None       # [tokens][kv_heads][head_dim] bfloat16 (when asked for)
    v_values: Optional[torch.Tensor] = None


def _head_rows(t: torch.Tensor, name: str, heads: Optional[int], d: int, dev) -> int:
    """Token stride of a [tokens][heads][d] BF16 tensor whose heads lie one after another."""
    _need(t, name, _BITS16, dev, 3)
    if t.shape[2] != d or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [tokens][{heads if heads is not None else 'heads'}][{d}], got {tuple(t.shape)}")
    if t.numel() > 0 and (t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != d)):
        raise ValueError(f"{name}: a token's heads must lie one after another")
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1] * d, 8)


class RopeAppendNVFP4(_Prepared):
    """A prepared rotary append.  q: [tokens][q_heads][d] or None; k, v: [tokens][kv_heads]
    [d] BF16 (views into one QKV buffer work); positions: int32 [tokens]; slots: int64
    [tokens], page * page_size + row, negative for padding.  q_out: where the rotated Q
    goes (default: a tensor of its own; q itself rotates in place).  values: also the BF16
    values that the cache now stands for."""

    def __init__(self, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                 slots: torch.Tensor, rope: RopePlan, cache: NVFP4KVCache, values: bool = False,
                 q_out: Optional[torch.Tensor] = None):
        dev, d, hk = cache.device, cache.head_dim, cache.kv_heads
        tokens = k.shape[0]
        ld_k, ld_v = _head_rows(k, "k", hk, d, dev), _head_rows(v, "v", hk, d, dev)
        hq, ld_q, ld_qo = 0, 0, 0
        if q is not None:
            ld_q = _head_rows(q, "q", None, d, dev)
            hq = q.shape[1]
            if q_out is None:
                q_out = torch.empty((tokens, hq, d), dtype=torch.bfloat16, device=dev)
            ld_qo = _head_rows(q_out, "q_out", hq, d, dev)
        elif q_out is not None:
            raise ValueError("q_out needs q")
        _need(positions, "positions", (torch.int32,), dev, 1)
        _need(slots, "slots", (torch.int64,), dev, 1)
        for name, t in (("q", q), ("q_out", q_out), ("v", v), ("positions", positions), ("slots", slots)):
            if t is not None and t.shape[0] != tokens:
                raise ValueError(f"{name} holds {t.shape[0]} tokens, k {tokens}")
        if not positions.is_contiguous() or not slots.is_contiguous():
            raise ValueError("positions and slots must be contiguous")
        if rope.rot_dim and rope.inv_freq.device != dev:
            raise ValueError(f"the rotary plan is on {rope.inv_freq.device}, expected {dev}")
        kv = [torch.empty((tokens, hk, d), dtype=torch.bfloat16, device=dev) if values else None for _ in range(2)]
        self.out = RopeAppendResult(q_out, *kv)
        self._cache, self._rope = cache, rope
        self._bind("mxq_rope_append_nvfp4", dev, (q, q_out, k, v, positions, slots, rope.inv_freq, *kv, *cache.tensors()),
                   _ptr(q), ld_q, hq, _ptr(q_out), ld_qo, _ptr(k), ld_k, _ptr(v), ld_v, tokens, _ptr(positions),
                   _ptr(slots), ctypes.byref(rope._c), ctypes.byref(cache._c), _ptr(kv[0]), _ptr(kv[1]))

    def __call__(self, stream=None) -> RopeAppendResult:
        return self._launch(stream)


def mxq_rope_append_nvfp4(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                          slots: torch.Tensor, rope: RopePlan, cache: NVFP4KVCache, values: bool = False,
                          q_out: Optional[torch.Tensor] = None, stream=None) -> RopeAppendResult:
    """Rotary positions on q and k; k and v into the cache rows that slots name."""
    return RopeAppendNVFP4(q, k, v, positions, slots, rope, cache, values, q_out)(stream)


# ---------------------------------------------------------------------------- attention
@dataclass
class AttentionResult:
    out: torch.Tensor                             # [total_q][q_heads][head_dim] bfloat16
    lse: Optional[torch.Tensor] = None            # [total_q][q_heads] float32 (when asked for)


def mxq_attention_nvfp4_workspace_size(q_heads: int, kv_heads: int, head_dim: int, batch: int, total_q: int,
                                       max_q_len: int, max_seq_len: int, window: int = 0, sinks: int = 0) -> int:
    return int(lib().mxq_attention_nvfp4_workspace_size(q_heads, kv_heads, head_dim, batch, total_q, max_q_len,
                                                        max_seq_len, window, sinks))


class AttentionNVFP4(_Prepared):
    """A prepared attention call over an NVFP4KVCache.  q: [total_q][q_heads][d] BF16, the
    queries of all sequences one after another; block_table: int32 [batch][pages];
    seq_lens: int32 [batch], cached tokens with the new ones; q_starts: int32 [batch + 1].
    max_q_len bounds the longest query run, max_seq_len (default: what the table can hold)
    is the length to plan the split over the cache for.  window, sinks: each query sees
    the last `window` tokens up to its own (0: all of them) and the first `sinks`.  scale: on
    the scores (default 1/sqrt(d)).  The outputs of rows that belong to no sequence are
    left as they were (a fresh out is zeroed once)."""

    def __init__(self, q: torch.Tensor, cache: NVFP4KVCache, block_table: torch.Tensor, seq_lens: torch.Tensor,
                 q_starts: torch.Tensor, max_q_len: int, max_seq_len: Optional[int] = None,
                 scale: Optional[float] = None, window: int = 0, sinks: int = 0, lse: bool = False,
                 out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
        dev, d = cache.device, cache.head_dim
        ld_q = _head_rows(q, "q", None, d, dev)
        total, hq = q.shape[0], q.shape[1]
        if out is None:
            out = torch.zeros((total, hq, d), dtype=torch.bfloat16, device=dev)
        ld_out = _head_rows(out, "out", hq, d, dev)
        if out.shape[0] != total:
            raise ValueError("out must hold as many rows as q")
        _need(block_table, "block_table", (torch.int32,), dev, 2)
        _need(seq_lens, "seq_lens", (torch.int32,), dev, 1)
        _need(q_starts, "q_starts", (torch.int32,), dev, 1)
        batch, pages = block_table.shape
        if seq_lens.shape[0] != batch or q_starts.shape[0] != batch + 1:
            raise ValueError("seq_lens is [batch], q_starts [batch + 1]")
        if not seq_lens.is_contiguous() or not q_starts.is_contiguous() or (block_table.numel() > 0 and pages > 1
                                                                             and block_table.stride(1) != 1):
            raise ValueError("seq_lens, q_starts and the rows of block_table must be contiguous")
        for name, value in (("window", window), ("sinks", sinks)):
            if not 0 <= value < 1 << 31:
                raise ValueError(f"{name} must be in [0, 2^31), got {value}")
        if max_seq_len is None:
            max_seq_len = min(pages * cache.page_size, _MAX_SEQ_LEN)
        lse_t = torch.zeros((total, hq), dtype=torch.float32, device=dev) if lse else None
        need = mxq_attention_nvfp4_workspace_size(hq, cache.kv_heads, d, batch, total, max_q_len, max_seq_len, window,
                                                  sinks)
        if workspace is None and need > 0:
            workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
        elif workspace is not None:
            if not _need(workspace, "workspace", (torch.uint8,), dev, 1).is_contiguous():
                raise ValueError("workspace must be contiguous")
        self.workspace = workspace
        self.out = AttentionResult(out, lse_t)
        self._cache = cache
        self._bind("mxq_attention_nvfp4", dev,
                   (q, out, lse_t, block_table, seq_lens, q_starts, workspace, *cache.tensors()),
                   _ptr(q), ld_q, hq, total, _ptr(out), ld_out, _ptr(lse_t), ctypes.byref(cache._c),
                   _ptr(block_table), block_table.stride(0) if batch > 1 else pages, pages, _ptr(seq_lens),
                   _ptr(q_starts), batch, max_q_len, max_seq_len,
                   float(scale) if scale is not None else 1.0 / math.sqrt(d), window, sinks, _ptr(workspace),
                   workspace.numel() if workspace is not None else 0)

    def __call__(self, stream=None) -> AttentionResult:
        return self._launch(stream)


def mxq_attention_nvfp4(q: torch.Tensor, cache: NVFP4KVCache, block_table: torch.Tensor, seq_lens: torch.Tensor,
                        q_starts: torch.Tensor, max_q_len: int, max_seq_len: Optional[int] = None,
                        scale: Optional[float] = None, window: int = 0, sinks: int = 0, lse: bool = False,
                        out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        stream=None) -> AttentionResult:
    """Causal attention of the queries over the cached tokens of their sequences."""
    return AttentionNVFP4(q, cache, block_table, seq_lens, q_starts, max_q_len, max_seq_len, scale, window, sinks,
                          lse, out, workspace)(stream)
