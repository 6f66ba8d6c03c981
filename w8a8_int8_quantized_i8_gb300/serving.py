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
import functools
from typing import NamedTuple

import torch

from .binding import _FMT, KVCacheInfo, _check, load

_CODES = {torch.int8: 0, torch.float8_e4m3fn: 1}
_bf16, _i32, _i64, _f32 = torch.bfloat16, torch.int32, torch.int64, torch.float32
_lib = None


def _library():
    global _lib
    if _lib is None:
        _lib = load()
    return _lib


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


def _call(fn: str, index: int, *args) -> None:
    """Calls the library on the current stream of device `index`, made the
    current device for the call where it is not."""
    lib = _library()
    if index == torch.cuda.current_device():
        status = getattr(lib, fn)(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = getattr(lib, fn)(*args, torch._C._cuda_getCurrentRawStream(index))
    if status:
        _check(status, fn)


# The checks below cost the host a microsecond or so each, as much as a launch,
# so each is one expression over cheap attributes; _explain says what was wrong.

def _explain(t, dtype, name, ndim, index=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}")


def _vector(t, dtype, name, n, index):
    """The address of a contiguous vector of n elements."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.dim() == 1
            and t.shape[0] == n and t.is_contiguous() and index >= 0):
        return t.data_ptr()
    _explain(t, dtype, name, 1, index)
    if t.shape[0] != n:
        raise ValueError(f"{name} must have {n} elements, got {t.shape[0]}")
    raise ValueError(f"{name} must be contiguous")


def _rows(t, dtype, name, rows, cols, index):
    """(address, row stride) of a matrix with unit stride along its rows."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.dim() == 2
            and index >= 0):
        _explain(t, dtype, name, 2, index)
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be {(rows, cols)}, got {tuple(t.shape)}")
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    if rows <= 1:
        return t.data_ptr(), cols       # the stride of a single row says nothing
    if ld < cols:
        raise ValueError(f"{name} rows overlap")
    return t.data_ptr(), ld


def _heads(t, name, shape, index):
    """(address, token stride, head stride) of a bf16 [tokens, heads, head_dim]."""
    if not (isinstance(t, torch.Tensor) and t.dtype is _bf16 and t.get_device() == index and t.dim() == 3
            and index >= 0):
        _explain(t, _bf16, name, 3, index)
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    token, head, unit = t.stride()
    if unit != 1 and shape[2] > 1:
        raise ValueError(f"{name} must have unit stride along head_dim")
    # the stride along a dimension of one element says nothing
    return t.data_ptr(), token if shape[0] > 1 else 0, head if shape[1] > 1 else 0


def _cache(cache: QuantKVCache, index: int) -> KVCacheInfo:
    k, v, ks, vs = cache
    fmt = _CODES.get(k.dtype) if isinstance(k, torch.Tensor) else None
    if fmt is None:
        raise TypeError("the cache's codes must be int8 or float8_e4m3fn")
    shape = k.shape
    if not (k.dim() == 4 and isinstance(v, torch.Tensor) and v.dtype is k.dtype and v.shape == shape
            and isinstance(ks, torch.Tensor) and ks.dtype is _f32 and ks.shape == shape[:2]
            and isinstance(vs, torch.Tensor) and vs.dtype is _f32 and vs.shape == shape[:2]
            and index >= 0 and k.get_device() == v.get_device() == ks.get_device() == vs.get_device() == index
            and k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()):
        _explain(k, k.dtype, "cache.k", 4, index)
        _explain(v, k.dtype, "cache.v", 4, index)
        _explain(ks, _f32, "cache.k_scale", 2, index)
        _explain(vs, _f32, "cache.v_scale", 2, index)
        if v.shape != shape or ks.shape != shape[:2] or vs.shape != shape[:2]:
            raise ValueError("the cache's shapes do not agree")
        raise ValueError("the cache must be contiguous")
    blocks, heads, block, dim = shape
    return KVCacheInfo(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), blocks, block, heads, dim, fmt)


def _device_index(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


@functools.lru_cache(maxsize=4096)
def _attention_workspace(q_heads, kv_heads, head_dim, fmt, max_new, index) -> int:
    with torch.cuda.device(index):
        return _library().i8_paged_attention_workspace_bytes(q_heads, kv_heads, head_dim, fmt, max_new)


def paged_attention_workspace_bytes(q_heads: int, cache: QuantKVCache, max_new: int) -> int:
    """Bytes of workspace that paged_attention needs for these sizes."""
    info = _cache(cache, _device_index(cache.k, "cache.k"))
    return _attention_workspace(q_heads, info.kv_heads, info.head_dim, info.fmt, max_new, cache.k.get_device())


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
    index = _device_index(x, "x")
    M, K = x.shape
    dev = x.device
    xp, ldx = _rows(x, _bf16, "x", M, K, index)
    wp = _vector(weight, _bf16, "weight", K, index) if weight is not None else None
    code, dtype = _FMT[fmt]
    q = torch.empty((M, K), dtype=dtype, device=dev)
    s = torch.empty((M,), dtype=_f32, device=dev)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out without a residual")
        _call("i8_add_rmsnorm_quant_act_pertoken", index, xp, M, K, ldx, None, 0, wp, eps, code,
              q.data_ptr(), K, s.data_ptr(), None, 0)
        return q, s
    rp, ldr = _rows(residual, _bf16, "residual", M, K, index)
    if residual_out is None:
        residual_out = torch.empty((M, K), dtype=_bf16, device=dev)
        hp, ldh = residual_out.data_ptr(), K
    else:
        hp, ldh = _rows(residual_out, _bf16, "residual_out", M, K, index)
    _call("i8_add_rmsnorm_quant_act_pertoken", index, xp, M, K, ldx, rp, ldr, wp, eps, code,
          q.data_ptr(), K, s.data_ptr(), hp, ldh)
    return q, s, residual_out


def build_block_tables(context_lens: torch.Tensor, new_lens: torch.Tensor, block_tables: torch.Tensor,
                       free_blocks: torch.Tensor, block_size: int, max_tokens: int,
                       taken: torch.Tensor | None = None, out: BlockPlan | None = None) -> BlockPlan:
    """One step's offsets, lengths, slots and positions from the requests'
    lengths (int32 [R] each); ``block_tables`` (int32 [R, width], row-strided
    views allowed) gets the blocks that the new tokens need, from
    ``free_blocks`` (int32) in request order, beginning at entry ``taken``
    (int32 [1]; None: 0).  See i8_build_block_tables for the outputs; they and
    the tables share no memory with the inputs (lengths that are kept from step
    to step are copied over afterwards, as decoder.Requests does)."""
    index = _device_index(context_lens, "context_lens")
    if context_lens.dim() != 1:
        raise ValueError("context_lens must be 1-D")
    R = context_lens.shape[0]
    ctx = _vector(context_lens, _i32, "context_lens", R, index)
    new = _vector(new_lens, _i32, "new_lens", R, index)
    if not isinstance(block_tables, torch.Tensor) or block_tables.dim() != 2:
        raise TypeError("block_tables must be a 2-D int32 CUDA tensor")
    width = block_tables.shape[1]
    table, ld = _rows(block_tables, _i32, "block_tables", R, width, index)
    if not isinstance(free_blocks, torch.Tensor) or free_blocks.dim() != 1:
        raise TypeError("free_blocks must be a 1-D int32 CUDA tensor")
    free, n_free = _vector(free_blocks, _i32, "free_blocks", free_blocks.shape[0], index), free_blocks.shape[0]
    if max_tokens < 0 or block_size <= 0:
        raise ValueError("max_tokens must be >= 0 and block_size > 0")
    if out is None:
        out = BlockPlan.empty(R, max_tokens, context_lens.device)
    cu, lens, slots, positions, counts = out
    _call("i8_build_block_tables", index, ctx, new, R, table, width, ld, free, n_free,
          _vector(taken, _i32, "taken", 1, index) if taken is not None else None, block_size, max_tokens,
          _vector(cu, _i32, "out.cu_new", R + 1, index), _vector(lens, _i32, "out.seq_lens", R, index),
          _vector(slots, _i64, "out.slots", max_tokens, index),
          _vector(positions, _i32, "out.positions", max_tokens, index),
          _vector(counts, _i32, "out.counts", 3, index))
    return out


def kv_cache_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                    cache: QuantKVCache) -> QuantKVCache:
    """Quantizes the step's keys and values, bf16 [T, kv_heads, head_dim] each
    (views of the fused projection's output allowed), into their slots
    (int64 [T], as build_block_tables gives them; negative: skipped; a block's
    tokens in order and together).  A block whose tokens get louder is re-coded
    with its new scale; a NaN makes the scale of its block and head NaN."""
    index = _device_index(k, "k")
    info = _cache(cache, index)
    T = k.shape[0] if k.dim() else 0
    shape = (T, info.kv_heads, info.head_dim)
    kp, kt, kh = _heads(k, "k", shape, index)
    vp, vt, vh = _heads(v, "v", shape, index)
    _call("i8_kv_cache_append", index, kp, kt, kh, vp, vt, vh, _vector(slots, _i64, "slots", T, index), T,
          ctypes.byref(info))
    return cache


def paged_attention(q: torch.Tensor, cache: QuantKVCache, block_tables: torch.Tensor,
                    seq_lens: torch.Tensor, cu_new: torch.Tensor, max_new: int | None = None,
                    scale: float | None = None, want_lse: bool = False,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Causal attention of the step's tokens q, bf16 [T, q_heads, head_dim],
    over the cache, which holds them already.  Request r's tokens are rows
    cu_new[r]..cu_new[r+1] of q and the last of its seq_lens[r] tokens; its
    blocks are row r of ``block_tables``.  ``max_new`` bounds the new tokens of
    a request and chooses the kernels by it (None: T, which costs a batch of
    single tokens a third more: 90 -> 119 us for 64 requests of 4096 tokens);
    scale defaults to head_dim ** -0.5.

    Returns out [T, q_heads, head_dim] bf16, and with ``want_lse`` also the
    natural log of the sum of exponentials, fp32 [T, q_heads] (-inf for a row
    that sees nothing, whose output is 0).  Rows of no request are not written.
    NaN shows in the rows that see it, and in no others."""
    index = _device_index(q, "q")
    info = _cache(cache, index)
    if q.dim() != 3:
        raise ValueError("q must be 3-D")
    T, Hq, D = shape = q.shape
    if D != info.head_dim or Hq == 0 or Hq % info.kv_heads:
        raise ValueError("q must be [T, q_heads, head_dim] with the cache's head_dim and a multiple of its kv_heads")
    qp, qt, qh = _heads(q, "q", shape, index)
    if not isinstance(seq_lens, torch.Tensor) or seq_lens.dim() != 1:
        raise TypeError("seq_lens must be a 1-D int32 CUDA tensor")
    R = seq_lens.shape[0]
    lens = _vector(seq_lens, _i32, "seq_lens", R, index)
    cu = _vector(cu_new, _i32, "cu_new", R + 1, index)
    if not isinstance(block_tables, torch.Tensor) or block_tables.dim() != 2:
        raise TypeError("block_tables must be a 2-D int32 CUDA tensor")
    width = block_tables.shape[1]
    table, ld = _rows(block_tables, _i32, "block_tables", R, width, index)
    max_new = T if max_new is None else min(max_new, T)
    if out is None:
        out = torch.empty(shape, dtype=_bf16, device=q.device)
        op, ot, oh = out.data_ptr(), Hq * D, D
    else:
        op, ot, oh = _heads(out, "out", shape, index)
        if (T > 1 and ot < D) or (Hq > 1 and oh < D):
            raise ValueError("out's rows overlap")
    lse = torch.empty((T, Hq), dtype=_f32, device=q.device) if want_lse else None
    if workspace is None:
        need = _attention_workspace(Hq, info.kv_heads, D, info.fmt, max_new, index)
        workspace = torch.empty((need,), dtype=torch.uint8, device=q.device)
    elif not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on cuda:{index}")
    _call("i8_paged_attention", index, qp, qt, qh, T, Hq, ctypes.byref(info), table, width, ld, lens, cu, R,
          max_new, D ** -0.5 if scale is None else scale, op, ot, oh,
          lse.data_ptr() if want_lse else None, workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return (out, lse) if want_lse else out
