"""The product kernels where they have been running for a while: many tiles a CTA pair
(every buffer and phase used again), and every split of K with any count of tokens.
Sums that fp32 holds, so the output is the rounded exact one, bit for bit."""
import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from tests import _fp4
from tests.test_gpu_fp4_gemm import FMTS, _exact_rows, _gate64, _gen

pytestmark = pytest.mark.gpu


# tokens, channels, K; 256 x 256 tiles (gated: 256 x 128) on 76 pairs: 5.5, 6.7 and 5.5 (11, 13 and 11) tiles a pair,
# with one, two and three stages of K a tile
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(5000, 5128, 288), (5121, 6144, 256), (4999, 5240, 704), (1500, 17416, 544)])
def test_many_tiles_a_pair(fmt, M, N, K):
    g = _gen(M + N + K)
    a, w, u = _exact_rows(g, M, K, fmt, fmt == "nvfp4"), _exact_rows(g, N, K, fmt, True), _exact_rows(g, N, K, fmt, True)
    b = (torch.randint(-8, 9, (N,), generator=g, device="cuda") / 8).bfloat16()
    va, vw = _fp4.values(a), _fp4.values(w)
    pre = va @ vw.T
    got = i8.gemm_fp4_bias_bf16(a, w)
    assert torch.equal(got, pre.float().bfloat16())
    got = i8.gemm_fp4_bias_bf16(a, w, b)
    assert torch.equal(got, (pre + b.double()).float().bfloat16())
    small = w._replace(row_scales=w.row_scales / 16)
    pre = pre / 16 + b.double()
    up = va @ _fp4.values(u).T
    for activation in ("silu", "gelu"):
        got = i8.gemm_fp4_gated_bf16(a, small, u, b, None, activation=activation).double()
        want = _gate64(pre, up, activation)
        # (tolerance: see test_gated_product)
        tol = (2.0 ** -8 + (16 + 2 * pre.abs()) * 2.0 ** -23) * want.abs() + 1e-30
        assert ((got - want).abs() <= tol).all()
    i8.sync_check()


@pytest.fixture(params=range(1, 9))
def splits(request):
    i8.set_option("force_splits", request.param)
    yield request.param
    i8.set_option("force_splits", 0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 7, 16, 17, 31, 33, 61, 64, 65, 100, 127, 128, 129])
@pytest.mark.parametrize("N,K", [(264, 2080), (128, 4128)])
def test_every_split(fmt, M, N, K, splits):
    g = _gen(M + N + K)
    a, w, u = _exact_rows(g, M, K, fmt, fmt == "nvfp4"), _exact_rows(g, N, K, fmt, True), _exact_rows(g, N, K, fmt, True)
    b = (torch.randint(-8, 9, (N,), generator=g, device="cuda") / 8).bfloat16()
    va = _fp4.values(a)
    pre, up = va @ _fp4.values(w).T, va @ _fp4.values(u).T
    wide = torch.full((M + 2, N + 16), 7.0, device="cuda", dtype=torch.bfloat16)
    got = i8.gemm_fp4_bias_bf16(a, w, b, out=wide[1:-1, 8:-8])
    assert torch.equal(got, (pre + b.double()).float().bfloat16())
    assert (wide[0] == 7).all() and (wide[-1] == 7).all() and (wide[:, :8] == 7).all() and (wide[:, -8:] == 7).all()
    small = w._replace(row_scales=w.row_scales / 16)
    pre = pre / 16 + b.double()
    got = i8.gemm_fp4_gated_bf16(a, small, u, b, None).double()
    want = _gate64(pre, up, "silu")
    tol = (2.0 ** -8 + (16 + 2 * pre.abs()) * 2.0 ** -23) * want.abs() + 1e-30
    assert ((got - want).abs() <= tol).all()
    i8.sync_check()
