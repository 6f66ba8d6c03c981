"""Both formats over the whole of bf16, against the definition in 64 bits, bit for bit."""
import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from tests.test_gpu_fp4_quant import FMTS, _check, _gen

pytestmark = pytest.mark.gpu


def _every():
    every = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    return every[torch.isfinite(every)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("seed", [0, 1])
def test_every_finite_bf16(fmt, seed):
    """In the order of the bits, so that a row's are alike, and shuffled; both in rows of 256 and of 4096."""
    x = _every()
    x = x[torch.randperm(x.numel(), generator=_gen(seed), device="cuda")] if seed else x
    for K in (256, 4096):
        rows = x[: x.numel() // K * K].view(-1, K)
        _check(i8.quant_rows_fp4(rows, fmt), rows.double(), fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K", [32, 256, 2080, 33024])
def test_rows_of_every_exponent(fmt, K):
    """A row whose largest magnitude has each exponent, from the subnormals to the largest finite number, and
    elements of all sizes below it."""
    g = _gen(K)
    top = 2.0 ** torch.arange(-133, 128, dtype=torch.float64, device="cuda")[:, None]
    rows = top.shape[0]
    x = torch.rand(rows, K, generator=g, device="cuda", dtype=torch.float64) * 2 - 1
    x *= torch.exp2(-torch.randint(0, 14, (rows, K), generator=g, device="cuda").double())
    x = (x * top).bfloat16()
    for mantissa in (1.0, 1.3125, 1.3203125, 1.5, 1.5078125, 1.9921875):      # around the powers' borders
        x[:, K // 2] = (top[:, 0] * mantissa).bfloat16()
        assert torch.isfinite(x).all()
        _check(i8.quant_rows_fp4(x, fmt), x.double(), fmt)
