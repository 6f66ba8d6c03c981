"""The norm with a 4-bit output where h * weight leaves fp32's range and h does not:
the row is taken times 2^-126, which its scale undoes.  Against the definition in 64
bits: codes and block scales bit for bit."""
import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from tests import _fp4
from tests.test_gpu_fp4_quant import FMTS, _check, _gen

pytestmark = pytest.mark.gpu
LARGEST = float(torch.finfo(torch.float32).max)


def _reference(x, r, w, eps):
    """(t as it is quantized, the factor of each row)"""
    h = (x.float() + r.float() if r is not None else x.float()).double()
    over = (h.abs() * w.double().abs()).amax(1) >= LARGEST * (1 + 2.0 ** -25)
    f = torch.where(over, 2.0 ** -126, 1.0).double()[:, None]
    # fp32 steps: h times a power of two, and its product with the gain
    t = ((h * f).float().double() * w.double()).float().double()
    return t, 1 / f[:, 0] / (h.square().mean(1) + eps).sqrt(), over


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K", [32, 512, 4096, 16384, 33024])
@pytest.mark.parametrize("gain,size", [(1.0, 3.3e38), (2.0, 3e38), (2.0, 1e38), (300.0, 2.0 ** 125), (2.0 ** 70, 2.0 ** 60),
                                       (2.0 ** 100, 1e38)])
@pytest.mark.parametrize("residual", [False, True])
def test_rows_whose_products_leave_the_range(fmt, K, gain, size, residual):
    g = _gen(K)
    x = (torch.rand(6, K, generator=g, device="cuda") * 2 - 1).mul(size).bfloat16()
    x[4:] = torch.randn(2, K, generator=g, device="cuda").bfloat16()          # ordinary rows beside them
    x[2, ::3] = 1.0
    r = (torch.rand(6, K, generator=g, device="cuda") * 1e30).bfloat16() if residual else None
    w = (gain * (1 + 0.1 * torch.randn(K, generator=g, device="cuda"))).bfloat16()
    got = i8.add_rmsnorm_quant_fp4(x, r, w, fmt=fmt)
    rows, h = got if residual else (got, None)
    t, factor, over = _reference(x, r, w, 1e-6)
    assert torch.isfinite(t).all()
    # (tolerance: see _norm_check)
    _check(rows, t, fmt, (factor, (K / 512 + 40) * 2.0 ** -24))
    assert torch.isfinite(_fp4.values(rows)).all()
    if residual:
        assert torch.equal(h, (x.float() + r.float()).bfloat16())
    if gain == 2.0 and size == 3e38 and K > 32:
        assert over[:2].all() and not over[4:].any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K", [512, 33024])
def test_in_place_and_what_is_not_finite(fmt, K):
    g = _gen(K + 1)
    x = ((torch.rand(4, K, generator=g, device="cuda") * 2 - 1) * 3e38).bfloat16()
    r = torch.ones(4, K, device="cuda").bfloat16()
    w = torch.full((K,), 2.0, device="cuda").bfloat16()
    x[1, 40] = torch.inf
    x0 = x.clone()
    rows, h = i8.add_rmsnorm_quant_fp4(x, r, w, fmt=fmt, residual_out=x)
    assert h is x and torch.equal(h.isinf(), x0.isinf())
    v = _fp4.values(rows)
    assert torch.isnan(v[1, 32:64]).all()
    keep = torch.tensor([0, 2, 3], device="cuda")
    t, factor, _ = _reference(x0[keep], r[keep], w, 1e-6)
    assert torch.isfinite(v[keep]).all()
    # half a code's step of the blocks' largest, which the formula's values are near
    want = t * factor[:, None]
    assert ((v[keep] - want).abs() <= want.abs().amax(1, keepdim=True) * 0.25).all()
