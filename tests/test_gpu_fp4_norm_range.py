"""The norm with a 4-bit output at the ends of the range, against the definition in 64
bits: codes and block scales bit for bit."""
import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from tests import _fp4
from tests.test_gpu_fp4_quant import FMTS, _check, _gen, _norm_case

pytestmark = pytest.mark.gpu
LARGEST = float(torch.finfo(torch.float32).max)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K", [32, 512, 4096, 33024])
@pytest.mark.parametrize("exponent", [-133, -132, -130, -128, -127])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -149, 1e-38])
def test_the_smallest_rows(fmt, K, exponent, eps):
    g = _gen(K)
    x = torch.randint(-3, 4, (5, K), generator=g, device="cuda").double().mul(2.0 ** exponent).bfloat16()
    x[:, 7] = 2.0 ** exponent
    rows = i8.add_rmsnorm_quant_fp4(x, eps=eps, fmt=fmt)
    t = x.double()
    # a factor beyond fp32's largest number is that number (mxfp4: its block scales end at 2^-127)
    factor = 1 / (t.square().mean(1) + eps).sqrt()
    if fmt == "mxfp4":
        factor = factor.clamp(max=LARGEST)
    # (tolerance: see _norm_check)
    _check(rows, t, fmt, (factor, (K / 512 + 40) * 2.0 ** -24))
    assert torch.isfinite(_fp4.values(rows)).all()
