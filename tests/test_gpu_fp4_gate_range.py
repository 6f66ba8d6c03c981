"""The gate far below zero, beside large values: act(g) * u against the formula in 64
bits, down to where fp32's exp(-g) is infinite (g = -88.7)."""
import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from tests.test_gpu_fp4_gemm import FMTS, _gate64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [2, 100, 600])
def test_silu_down_to_the_range_s_end(fmt, M):
    g = torch.tensor([0.0, -1.0, -40.0, -80.0, -84.0, -86.0, -87.0, -87.5, -88.0, -88.5, 30.0, 88.5, 200.0, 1e30], device="cuda")
    u = torch.tensor([1.0, -3.0, 1e20, 1e30, 1e37, -3e38], device="cuda")
    g, u = (t.flatten().bfloat16() for t in torch.meshgrid(g, u, indexing="ij"))
    g, u = (t[: t.numel() // 8 * 8].contiguous() for t in (g, u))
    N = g.numel()
    zero = i8.quant_rows_fp4(torch.zeros(N, 64, device="cuda").bfloat16(), fmt)
    a = i8.quant_rows_fp4(torch.ones(M, 64, device="cuda").bfloat16(), fmt)
    got = i8.gemm_fp4_gated_bf16(a, zero, zero, g, u).double()      # the products are 0: gate and value are the biases
    want = _gate64(g.double(), u.double(), "silu")
    inside = want.abs() < 3.3e38
    # half a step of bf16, and fp32's steps: exp's argument is off by 2^-24 of itself
    tol = (2.0 ** -8 + (16 + 2 * g.double().abs().clamp(max=90)) * 2.0 ** -23) * want.abs()
    assert ((got - want).abs() <= tol)[:, inside].all()
    assert torch.isinf(got[:, ~inside]).all()
