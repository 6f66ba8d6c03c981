"""The 4-bit route of the linear layer, bound to libi8 (include/i8.h): argument
marshalling only, as in binding.py, in the extension csrc/torch_calls.cpp.

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

from typing import NamedTuple

import torch

from .binding import load, load_calls

FORMATS = {"nvfp4": 0, "mxfp4": 1}
ACTIVATIONS = {"silu": 0, "gelu": 1}
_NAMES = ("nvfp4", "mxfp4")
_TILE = (2048, 1024)          # bytes of block scales of 128 rows by 256 elements
_u8, _f32 = torch.uint8, torch.float32


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


_calls = None


def _ext():
    global _calls
    if _calls is None:
        _calls = load_calls()
    return _calls


def quant_rows_fp4(x: torch.Tensor, fmt: str = "nvfp4", out: FP4Rows | None = None) -> FP4Rows:
    """bf16 [rows, K] -> 4-bit codes and scales, of a layer's tokens or of its
    weights; x may be a row-strided view.  K % 32 == 0."""
    return (_calls or _ext()).quant_rows(x, _format(fmt), out)


def add_rmsnorm_quant_fp4(x: torch.Tensor, residual: torch.Tensor | None = None, weight: torch.Tensor | None = None,
                          eps: float = 1e-6, fmt: str = "nvfp4", residual_out: torch.Tensor | None = None,
                          out: FP4Rows | None = None):
    """add_rmsnorm_quant_act_pertoken with a 4-bit output: the RMS norm of x +
    residual, times ``weight`` [K]; with a residual also the sum, bf16 [M, K], which
    goes to ``residual_out`` (it may be ``residual`` or ``x`` itself: in place).

    Returns rows without a residual and (rows, h) with one."""
    return (_calls or _ext()).norm_rows(x, residual, weight, eps, _format(fmt), residual_out, out)


def gemm_fp4_bias_bf16(a: FP4Rows, w: FP4Rows, bias: torch.Tensor | None = None,
                       out: torch.Tensor | None = None) -> torch.Tensor:
    """bf16(acc * s_a[m] * s_w[n] + bias[n]): tokens a [M, K] by weights w [N, K] of
    the same format, N % 8 == 0."""
    return (_calls or _ext()).gemm(a, w, bias, out)


def gemm_fp4_gated_bf16(a: FP4Rows, gate: FP4Rows, up: FP4Rows, gate_bias: torch.Tensor | None = None,
                        up_bias: torch.Tensor | None = None, activation: str = "silu",
                        out: torch.Tensor | None = None) -> torch.Tensor:
    """bf16(act(g) * u) with g and u the products of a with ``gate`` and ``up``
    [N, K] (biases added), both in fp32: the first half of a gated feed-forward
    block in one kernel.  activation: "silu" or "gelu" (erf form)."""
    return (_calls or _ext()).gemm_gated(a, gate, up, gate_bias, up_bias, _activation(activation), out)


def linear_fp4_workspace_bytes(M: int, w: FP4Rows) -> int:
    """Bytes of workspace that linear_fp4 and gated_linear_fp4 need for M tokens."""
    return load().i8_linear_fp4_workspace_bytes(M, w.shape[1], _format(w.fmt))


def linear_fp4(x: torch.Tensor, w: FP4Rows, bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The whole 4-bit linear layer: quantizes x, bf16 [M, K] (row-strided views
    allowed), in w's format, then the product."""
    return (_calls or _ext()).linear(x, w, bias, out, workspace)


def gated_linear_fp4(x: torch.Tensor, gate: FP4Rows, up: FP4Rows, gate_bias: torch.Tensor | None = None,
                     up_bias: torch.Tensor | None = None, activation: str = "silu",
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Quantizes x in the weights' format, then gemm_fp4_gated_bf16."""
    return (_calls or _ext()).linear_gated(x, gate, up, gate_bias, up_bias, _activation(activation), out, workspace)
