"""The 4-bit route of the linear layer, bound to libi8 (include/i8.h): argument
marshalling only, as in binding.py.

    w = quant_rows_fp4(weight, "nvfp4")              # offline, bf16 [N, K]
    y = linear_fp4(x, w, bias)                       # bf16 [M, K] -> bf16 [M, N]

    rows, h = add_rmsnorm_quant_fp4(x, h, gain)      # or the steps by themselves
    y = gemm_fp4_bias_bf16(rows, w)

    u = gated_linear_fp4(x, gate, up)                # act(x gate^T) * (x up^T), one product kernel

Formats: "nvfp4" (blocks of 16, E4M3 scales, a power of two for each row) and
"mxfp4" (blocks of 32, power-of-two scales); include/i8.h defines both.  Every
call runs on the current stream of its tensors' device, allocates its outputs
with torch unless they are given, never waits for the device, and can be
captured into a CUDA graph.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from .binding import FP4RowsInfo
from .serving import _bf16, _call, _explain, _f32, _library, _rows, _vector

FORMATS = {"nvfp4": 0, "mxfp4": 1}
ACTIVATIONS = {"silu": 0, "gelu": 1}
_NAMES = ("nvfp4", "mxfp4")
_TILE = (2048, 1024)          # bytes of block scales of 128 rows by 256 elements
_u8 = torch.uint8


class FP4Rows(NamedTuple):
    """Rows in microscaled 4-bit floating point: a layer's tokens or weights."""
    codes: torch.Tensor                    # uint8 [rows, K / 2]: two E2M1 codes a byte, the even element low
    block_scales: torch.Tensor             # uint8 [ceil(rows / 128), ceil(K / 256), 2048 (nvfp4) or 1024 (mxfp4)]
    row_scales: torch.Tensor | None = None  # fp32 [rows]; None: ones

    @classmethod
    def empty(cls, rows: int, K: int, fmt: str = "nvfp4", device="cuda", scaled: bool | None = None) -> "FP4Rows":
        """Buffers to keep from step to step (``out=`` of the quantizers).  scaled:
        with a scale for each row (nvfp4 has one; mxfp4 behind a norm)."""
        code = _format(fmt)
        return cls(torch.empty((rows, K // 2), dtype=_u8, device=device),
                   torch.empty((-(-rows // 128), -(-K // 256), _TILE[code]), dtype=_u8, device=device),
                   torch.empty((rows,), dtype=_f32, device=device) if (code == 0 if scaled is None else scaled) else None)

    @property
    def fmt(self) -> str:
        return _NAMES[_TILE.index(self.block_scales.shape[2])]

    @property
    def shape(self) -> tuple[int, int]:
        return self.codes.shape[0], 2 * self.codes.shape[1]


def _format(fmt) -> int:
    code = FORMATS.get(fmt) if isinstance(fmt, str) else None
    if code is None:
        raise ValueError(f"fmt must be one of {sorted(FORMATS)}")
    return code


def _activation(activation) -> int:
    code = ACTIVATIONS.get(activation) if isinstance(activation, str) else None
    if code is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    return code


# As in serving.py, the checks are one expression over cheap attributes where all is
# well: what the host does between two launches runs with cold caches and is what
# a small call costs.

def _info(rows, name: str, index: int):
    """(struct, rows, K, format's code) of 4-bit rows on a device."""
    if type(rows) is not FP4Rows:
        raise TypeError(f"{name} must be FP4Rows")
    codes, scales, row = rows
    if not (isinstance(codes, torch.Tensor) and codes.dtype is _u8 and codes.get_device() == index and codes.dim() == 2
            and isinstance(scales, torch.Tensor) and scales.dtype is _u8 and scales.get_device() == index
            and scales.dim() == 3 and codes.is_contiguous() and scales.is_contiguous() and index >= 0):
        _explain(codes, _u8, f"{name}.codes", 2, index)
        _explain(scales, _u8, f"{name}.block_scales", 3, index)
        raise ValueError(f"{name} must be contiguous")
    n, half = codes.shape
    tiles, deep, size = scales.shape
    if size not in _TILE or tiles != (n + 127) // 128 or deep != (half + 127) // 128:
        raise ValueError(f"{name}.block_scales must be [ceil(rows / 128), ceil(K / 256), 2048 or 1024]")
    code = 0 if size == 2048 else 1
    rp = None if row is None else _vector(row, _f32, f"{name}.row_scales", n, index)
    return FP4RowsInfo(codes.data_ptr(), scales.data_ptr(), rp, n, 2 * half, code), n, 2 * half, code


def _out_rows(out, rows: int, K: int, code: int, scaled: bool, x, index: int) -> tuple[FP4Rows, FP4RowsInfo]:
    if out is None:
        out = FP4Rows.empty(rows, K, _NAMES[code], x.device, scaled)
        codes, scales, row = out
        return out, FP4RowsInfo(codes.data_ptr(), scales.data_ptr(), row.data_ptr() if scaled else None, rows, K, code)
    info, *sizes = _info(out, "out", index)
    if sizes != [rows, K, code] or scaled != (out.row_scales is not None):
        raise ValueError("out must be FP4Rows.empty of the rows' sizes and format")
    return out, info


def _matrix(x, name: str):
    """(device, rows, K, address, row stride) of bf16 rows to quantize."""
    if not (isinstance(x, torch.Tensor) and x.dtype is _bf16 and x.dim() == 2 and x.get_device() >= 0):
        _explain(x, _bf16, name, 2)
    rows, K = x.shape
    ld, unit = x.stride()
    if K % 32 or not K:
        raise ValueError(f"{name}'s width must be a multiple of 32")
    if unit != 1 or (ld < K and rows > 1):
        raise ValueError(f"{name} must have unit stride along its rows, which do not overlap")
    return x.get_device(), rows, K, x.data_ptr(), ld if rows > 1 else K


def quant_rows_fp4(x: torch.Tensor, fmt: str = "nvfp4", out: FP4Rows | None = None) -> FP4Rows:
    """bf16 [rows, K] -> 4-bit codes and scales, of a layer's tokens or of its
    weights; x may be a row-strided view.  K % 32 == 0."""
    code = _format(fmt)
    index, rows, K, p, ld = _matrix(x, "x")
    out, o = _out_rows(out, rows, K, code, code == 0, x, index)
    _call("i8_quant_rows_fp4", index, p, rows, K, ld, code, o.codes, o.block_scales, o.row_scales)
    return out


def add_rmsnorm_quant_fp4(x: torch.Tensor, residual: torch.Tensor | None = None, weight: torch.Tensor | None = None,
                          eps: float = 1e-6, fmt: str = "nvfp4", residual_out: torch.Tensor | None = None,
                          out: FP4Rows | None = None):
    """add_rmsnorm_quant_act_pertoken with a 4-bit output: the RMS norm of x +
    residual, times ``weight`` [K]; with a residual also the sum, bf16 [M, K], which
    goes to ``residual_out`` (it may be ``residual`` or ``x`` itself: in place).

    Returns rows without a residual and (rows, h) with one."""
    code = _format(fmt)
    index, M, K, xp, ldx = _matrix(x, "x")
    wp = _vector(weight, _bf16, "weight", K, index) if weight is not None else None
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out without a residual")
        rp, ldr, hp, ldh = None, 0, None, 0
    else:
        rp, ldr = _rows(residual, _bf16, "residual", M, K, index)
        if residual_out is None:
            residual_out = torch.empty((M, K), dtype=_bf16, device=x.device)
        hp, ldh = _rows(residual_out, _bf16, "residual_out", M, K, index)
    out, o = _out_rows(out, M, K, code, True, x, index)
    _call("i8_add_rmsnorm_quant_fp4", index, xp, M, K, ldx, rp, ldr, wp, eps, code, o.codes, o.block_scales,
          o.row_scales, hp, ldh)
    return out if residual is None else (out, residual_out)


def _output(out, M: int, N: int, device, index: int):
    if out is None:
        out = torch.empty((M, N), dtype=_bf16, device=device)
        return out, out.data_ptr(), N
    p, ld = _rows(out, _bf16, "out", M, N, index)
    return out, p, ld


def _bias(bias, name: str, N: int, index: int):
    return _vector(bias, _bf16, name, N, index) if bias is not None else None


def _of(a) -> int:
    return a.codes.get_device() if type(a) is FP4Rows and isinstance(a.codes, torch.Tensor) else -1


def gemm_fp4_bias_bf16(a: FP4Rows, w: FP4Rows, bias: torch.Tensor | None = None,
                       out: torch.Tensor | None = None) -> torch.Tensor:
    """bf16(acc * s_a[m] * s_w[n] + bias[n]): tokens a [M, K] by weights w [N, K] of
    the same format, N % 8 == 0."""
    index = _of(a)
    ai, M, *kind = _info(a, "a", index)
    wi, N, *kind_w = _info(w, "w", index)
    if kind != kind_w:
        raise ValueError("a and w must have the same K and format")
    out, p, ld = _output(out, M, N, a.codes.device, index)
    _call("i8_gemm_fp4_bias_bf16", index, ctypes.byref(ai), ctypes.byref(wi), _bias(bias, "bias", N, index), p, ld)
    return out


def gemm_fp4_gated_bf16(a: FP4Rows, gate: FP4Rows, up: FP4Rows, gate_bias: torch.Tensor | None = None,
                        up_bias: torch.Tensor | None = None, activation: str = "silu",
                        out: torch.Tensor | None = None) -> torch.Tensor:
    """bf16(act(g) * u) with g and u the products of a with ``gate`` and ``up``
    [N, K] (biases added), both in fp32: the first half of a gated feed-forward
    block in one kernel.  activation: "silu" or "gelu" (erf form)."""
    code = _activation(activation)
    index = _of(a)
    ai, M, *kind = _info(a, "a", index)
    gi, N, *kind_g = _info(gate, "gate", index)
    ui, *up_sizes = _info(up, "up", index)
    if kind != kind_g or up_sizes != [N, *kind]:
        raise ValueError("a, gate and up must have the same K and format, gate and up the same rows")
    out, p, ld = _output(out, M, N, a.codes.device, index)
    _call("i8_gemm_fp4_gated_bf16", index, ctypes.byref(ai), ctypes.byref(gi), ctypes.byref(ui),
          _bias(gate_bias, "gate_bias", N, index), _bias(up_bias, "up_bias", N, index), code, p, ld)
    return out


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(M: int, K: int, code: int) -> int:
    return _library().i8_linear_fp4_workspace_bytes(M, K, code)


def linear_fp4_workspace_bytes(M: int, w: FP4Rows) -> int:
    """Bytes of workspace that linear_fp4 and gated_linear_fp4 need for M tokens."""
    return _workspace_bytes(M, w.shape[1], _format(w.fmt))


def _workspace(workspace, M: int, K: int, code: int, device, index: int):
    """(workspace, its address, its bytes)"""
    if workspace is None:
        size = _workspace_bytes(M, K, code)
        workspace = torch.empty((size,), dtype=_u8, device=device)
        return workspace, workspace.data_ptr(), size
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on cuda:{index}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def linear_fp4(x: torch.Tensor, w: FP4Rows, bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The whole 4-bit linear layer: quantizes x, bf16 [M, K] (row-strided views
    allowed), in w's format, then the product."""
    index, M, K, xp, ldx = _matrix(x, "x")
    wi, N, Kw, code = _info(w, "w", index)
    if Kw != K:
        raise ValueError("x and w must have the same K")
    out, yp, ldy = _output(out, M, N, x.device, index)
    workspace, wp, size = _workspace(workspace, M, K, code, x.device, index)
    _call("i8_linear_fp4", index, xp, M, K, ldx, ctypes.byref(wi), _bias(bias, "bias", N, index), yp, ldy, wp, size)
    return out


def gated_linear_fp4(x: torch.Tensor, gate: FP4Rows, up: FP4Rows, gate_bias: torch.Tensor | None = None,
                     up_bias: torch.Tensor | None = None, activation: str = "silu",
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Quantizes x in the weights' format, then gemm_fp4_gated_bf16."""
    act = _activation(activation)
    index, M, K, xp, ldx = _matrix(x, "x")
    gi, N, Kw, code = _info(gate, "gate", index)
    ui, *up_sizes = _info(up, "up", index)
    if Kw != K or up_sizes != [N, K, code]:
        raise ValueError("x, gate and up must have the same K, gate and up the same rows and format")
    out, yp, ldy = _output(out, M, N, x.device, index)
    workspace, wp, size = _workspace(workspace, M, K, code, x.device, index)
    _call("i8_gated_linear_fp4", index, xp, M, K, ldx, ctypes.byref(gi), ctypes.byref(ui),
          _bias(gate_bias, "gate_bias", N, index), _bias(up_bias, "up_bias", N, index), act, yp, ldy, wp, size)
    return out
