"""The operators that a decoder runs beside its 8-bit linear layers, bound to
libi8 (include/i8.h): argument marshalling only, as in binding.py.

One step of a decoder, for requests of any lengths:

    plan = build_block_tables(context_lens, new_lens, tables, free_blocks, cache.block_size, T)
    q, s, h = add_rmsnorm_quant_act_pertoken(x, h, weight)     # feeds the fused GEMM
    kv_cache_append(k, v, plan.slots, cache)
    o = paged_attention(q, cache, tables, plan.seq_lens, plan.cu_new, max_new)

Every call runs on the current stream of its tensors' device, allocates its
outputs with torch unless they are given, never waits for the device, and can
be captured into a CUDA graph.  Lengths, slots and block ids live on the
device: the kernels leave out what is out of range, and ``sync_check`` then
raises I8_ERR_DEVICE_DATA.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from .binding import _FMT, KVCacheInfo, _check, load

_CODES = {torch.int8: 0, torch.float8_e4m3fn: 1}


class BlockPlan(NamedTuple):
    """What one step of build_block_tables gives besides the tables."""
    cu_new: torch.Tensor      # int32 [R + 1]: exclusive sums of the new lengths
    seq_lens: torch.Tensor    # int32 [R]: context + new
    slots: torch.Tensor       # int64 [max_tokens]: block * block_size + offset, or -1
    positions: torch.Tensor   # int32 [max_tokens]
    counts: torch.Tensor      # int32 [3]: tokens, free-list entries in use, tokens without a block

    @classmethod
    def empty(cls, requests: int, max_tokens: int, device="cuda") -> "BlockPlan":
        """Buffers to keep from step to step (``out=`` of build_block_tables)."""
        def t(n, dtype=torch.int32):
            return torch.empty((n,), dtype=dtype, device=device)
        return cls(t(requests + 1), t(requests), t(max_tokens, torch.int64), t(max_tokens), t(3))


class QuantKVCache(NamedTuple):
    """A paged cache of keys and values in 8 bits: value = code * scale of its
    block and head."""
    k: torch.Tensor           # int8 or float8_e4m3fn [blocks, kv_heads, block_size, head_dim]
    v: torch.Tensor
    k_scale: torch.Tensor     # fp32 [blocks, kv_heads]
    v_scale: torch.Tensor

    @classmethod
    def empty(cls, blocks: int, kv_heads: int, block_size: int, head_dim: int, fmt: str = "int8",
              device="cuda") -> "QuantKVCache":
        """A cache of zeros; fmt "int8" or "e4m3"."""
        if fmt not in ("int8", "e4m3"):
            raise ValueError("fmt must be 'int8' or 'e4m3'")
        def codes():
            return torch.zeros((blocks, kv_heads, block_size, head_dim), dtype=torch.uint8,
                               device=device).view(_FMT[fmt][1])
        def scales():
            return torch.zeros((blocks, kv_heads), dtype=torch.float32, device=device)
        return cls(codes(), codes(), scales(), scales())

    @property
    def block_size(self) -> int:
        return self.k.shape[2]


class _on_device:
    """The stream to launch on, with the tensors' device made current for the
    call (nothing to do where it is already)."""
    __slots__ = ("device", "guard")

    def __init__(self, device):
        self.device, self.guard = device, None

    def __enter__(self):
        if self.device.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(self.device)
            self.guard.__enter__()
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)
        return False


def _need(t, dtype, name, ndim, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")


def _vector(t, dtype, name, n, device):
    _need(t, dtype, name, 1, device)
    if t.shape[0] != n:
        raise ValueError(f"{name} must have {n} elements, got {t.shape[0]}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _matrix(t, name, rows, cols, device):
    """Row stride of a bf16 matrix with unit stride along its rows."""
    _need(t, torch.bfloat16, name, 2, device)
    if tuple(t.shape) != (rows, cols):
        raise ValueError(f"{name} must be {(rows, cols)}, got {tuple(t.shape)}")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride along K")
    if rows <= 1:
        return cols
    if t.stride(0) < cols:
        raise ValueError(f"{name} rows overlap")
    return t.stride(0)


def _heads(t, name, device, head_dim=None):
    """(token, head) strides of a bf16 [tokens, heads, head_dim] tensor."""
    _need(t, torch.bfloat16, name, 3, device)
    if head_dim is not None and t.shape[2] != head_dim:
        raise ValueError(f"{name} must have head_dim {head_dim}, got {t.shape[2]}")
    if t.stride(2) != 1 and t.shape[2] > 1:
        raise ValueError(f"{name} must have unit stride along head_dim")
    # a stride along a dimension of one element says nothing
    return (t.stride(0) if t.shape[0] > 1 else 0), (t.stride(1) if t.shape[1] > 1 else 0)


def _cache(cache: QuantKVCache, device) -> KVCacheInfo:
    k, v, ks, vs = cache.k, cache.v, cache.k_scale, cache.v_scale
    fmt = _CODES.get(k.dtype) if isinstance(k, torch.Tensor) else None
    if fmt is None:
        raise TypeError("the cache's codes must be int8 or float8_e4m3fn")
    _need(k, k.dtype, "cache.k", 4, device)
    _need(v, k.dtype, "cache.v", 4, device)
    _need(ks, torch.float32, "cache.k_scale", 2, device)
    _need(vs, torch.float32, "cache.v_scale", 2, device)
    if v.shape != k.shape or ks.shape != k.shape[:2] or vs.shape != k.shape[:2]:
        raise ValueError("the cache's shapes do not agree")
    if not (k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()):
        raise ValueError("the cache must be contiguous")
    return KVCacheInfo(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), k.shape[0],
                       k.shape[2], k.shape[1], k.shape[3], fmt)


def add_rmsnorm_quant_act_pertoken(x: torch.Tensor, residual: torch.Tensor | None = None,
                                   weight: torch.Tensor | None = None, eps: float = 1e-6,
                                   fmt: str = "int8", residual_out: torch.Tensor | None = None):
    """bf16 [M,K] -> codes and per-token scales of the RMS norm of x + residual,
    times ``weight`` [K]; with a residual also the sum, bf16 [M,K], which goes
    to ``residual_out`` (it may be ``residual`` or ``x`` itself: in place).

    Returns (q, s) without a residual and (q, s, h) with one.  fmt as in
    layernorm_quant_act_pertoken; x and residual may be row-strided views."""
    if fmt not in _FMT:
        raise ValueError(f"fmt must be one of {sorted(_FMT)}")
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise TypeError("x must be a 2-D bf16 CUDA tensor")
    M, K = x.shape
    dev = x.device
    ldx = _matrix(x, "x", M, K, None)
    ldr = _matrix(residual, "residual", M, K, dev) if residual is not None else 0
    if weight is not None:
        _vector(weight, torch.bfloat16, "weight", K, dev)
    if residual is None and residual_out is not None:
        raise ValueError("residual_out without a residual")
    code, dtype = _FMT[fmt]
    q = torch.empty((M, K), dtype=dtype, device=dev)
    s = torch.empty((M,), dtype=torch.float32, device=dev)
    h = residual_out
    if residual is not None and h is None:
        h = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    ldh = _matrix(h, "residual_out", M, K, dev) if h is not None else 0
    with _on_device(dev) as stream:
        _check(load().i8_add_rmsnorm_quant_act_pertoken(
            x.data_ptr(), M, K, ldx, residual.data_ptr() if residual is not None else None, ldr,
            weight.data_ptr() if weight is not None else None, eps, code, q.data_ptr(), K,
            s.data_ptr(), h.data_ptr() if h is not None else None, ldh, stream),
            "i8_add_rmsnorm_quant_act_pertoken")
    return (q, s) if h is None else (q, s, h)


def build_block_tables(context_lens: torch.Tensor, new_lens: torch.Tensor, block_tables: torch.Tensor,
                       free_blocks: torch.Tensor, block_size: int, max_tokens: int,
                       taken: torch.Tensor | None = None, out: BlockPlan | None = None) -> BlockPlan:
    """One step's offsets, lengths, slots and positions from the requests'
    lengths (int32 [R] each); ``block_tables`` (int32 [R, width], row-strided
    views allowed) gets the blocks that the new tokens need, from
    ``free_blocks`` (int32) in request order, beginning at entry ``taken``
    (int32 [1]; None: 0).  See i8_build_block_tables for the outputs."""
    dev = context_lens.device
    R = context_lens.shape[0]
    _vector(context_lens, torch.int32, "context_lens", R, None)
    _vector(new_lens, torch.int32, "new_lens", R, dev)
    _need(block_tables, torch.int32, "block_tables", 2, dev)
    width = block_tables.shape[1]
    if block_tables.shape[0] != R:
        raise ValueError("block_tables must have a row for each request")
    if width > 1 and block_tables.stride(1) != 1:
        raise ValueError("block_tables must have unit stride along its rows")
    ld = block_tables.stride(0) if R > 1 else width
    if ld < width:
        raise ValueError("block_tables rows overlap")
    _vector(free_blocks, torch.int32, "free_blocks", free_blocks.shape[0], dev)
    if taken is not None:
        _vector(taken, torch.int32, "taken", 1, dev)
    if max_tokens < 0 or block_size <= 0:
        raise ValueError("max_tokens must be >= 0 and block_size > 0")
    if out is None:
        out = BlockPlan.empty(R, max_tokens, dev)
    else:
        _vector(out.cu_new, torch.int32, "out.cu_new", R + 1, dev)
        _vector(out.seq_lens, torch.int32, "out.seq_lens", R, dev)
        _vector(out.slots, torch.int64, "out.slots", max_tokens, dev)
        _vector(out.positions, torch.int32, "out.positions", max_tokens, dev)
        _vector(out.counts, torch.int32, "out.counts", 3, dev)
    with _on_device(dev) as stream:
        _check(load().i8_build_block_tables(
            context_lens.data_ptr(), new_lens.data_ptr(), R, block_tables.data_ptr(), width, ld,
            free_blocks.data_ptr(), free_blocks.shape[0],
            taken.data_ptr() if taken is not None else None, block_size, max_tokens,
            out.cu_new.data_ptr(), out.seq_lens.data_ptr(), out.slots.data_ptr(),
            out.positions.data_ptr(), out.counts.data_ptr(), stream), "i8_build_block_tables")
    return out


def kv_cache_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                    cache: QuantKVCache) -> QuantKVCache:
    """Quantizes the step's keys and values, bf16 [T, kv_heads, head_dim] each
    (views of the fused projection's output allowed), into their slots
    (int64 [T], as build_block_tables gives them; negative: skipped).  A block
    whose tokens get louder is re-coded with its new scale."""
    dev = k.device
    info = _cache(cache, dev)
    kt, kh = _heads(k, "k", None, info.head_dim)
    vt, vh = _heads(v, "v", dev, info.head_dim)
    T = k.shape[0]
    if k.shape[1] != info.kv_heads or v.shape != k.shape:
        raise ValueError("k and v must be [T, kv_heads, head_dim] of the cache")
    _vector(slots, torch.int64, "slots", T, dev)
    with _on_device(dev) as stream:
        _check(load().i8_kv_cache_append(k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, slots.data_ptr(),
                                         T, ctypes.byref(info), stream), "i8_kv_cache_append")
    return cache


def paged_attention(q: torch.Tensor, cache: QuantKVCache, block_tables: torch.Tensor,
                    seq_lens: torch.Tensor, cu_new: torch.Tensor, max_new: int | None = None,
                    scale: float | None = None, want_lse: bool = False,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Causal attention of the step's tokens q, bf16 [T, q_heads, head_dim],
    over the cache, which holds them already.  Request r's tokens are rows
    cu_new[r]..cu_new[r+1] of q and the last of its seq_lens[r] tokens; its
    blocks are row r of ``block_tables``.  ``max_new`` bounds the new tokens of
    a request (None: T); scale defaults to head_dim ** -0.5.

    Returns out [T, q_heads, head_dim] bf16, and with ``want_lse`` also the
    natural log of the sum of exponentials, fp32 [T, q_heads] (-inf for a row
    that sees nothing, whose output is 0).  Rows of no request are not written."""
    dev = q.device
    info = _cache(cache, dev)
    qt, qh = _heads(q, "q", None, info.head_dim)
    T, Hq, D = q.shape
    R, width = seq_lens.shape[0], block_tables.shape[1]
    _vector(seq_lens, torch.int32, "seq_lens", R, dev)
    _vector(cu_new, torch.int32, "cu_new", R + 1, dev)
    _need(block_tables, torch.int32, "block_tables", 2, dev)
    if block_tables.shape[0] != R:
        raise ValueError("block_tables must have a row for each request")
    if width > 1 and block_tables.stride(1) != 1:
        raise ValueError("block_tables must have unit stride along its rows")
    ld = block_tables.stride(0) if R > 1 else width
    if ld < width:
        raise ValueError("block_tables rows overlap")
    if Hq == 0 or Hq % info.kv_heads:
        raise ValueError("q_heads must be a multiple of kv_heads")
    if max_new is None:
        max_new = T
    if out is None:
        out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
    ot, oh = _heads(out, "out", dev, D)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if (T > 1 and ot < D) or (Hq > 1 and oh < D):
        raise ValueError("out's rows overlap")
    lse = torch.empty((T, Hq), dtype=torch.float32, device=dev) if want_lse else None
    with _on_device(dev) as stream:
        lib = load()
        need = lib.i8_paged_attention_workspace_bytes(Hq, info.kv_heads, D, info.fmt, min(max_new, T))
        if workspace is None and need:
            workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
        _check(lib.i8_paged_attention(
            q.data_ptr(), qt, qh, T, Hq, ctypes.byref(info), block_tables.data_ptr(), width, ld,
            seq_lens.data_ptr(), cu_new.data_ptr(), R, max_new, D ** -0.5 if scale is None else scale,
            out.data_ptr(), ot, oh, lse.data_ptr() if lse is not None else None,
            workspace.data_ptr() if workspace is not None else None,
            workspace.numel() * workspace.element_size() if workspace is not None else 0, stream),
            "i8_paged_attention")
    return (out, lse) if want_lse else out
