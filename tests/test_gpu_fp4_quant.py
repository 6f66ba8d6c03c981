"""Rows to 4 bits, as they are and behind the norm, against the definition in 64
bits: codes and scales bit for bit."""
import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from tests import _fp4

pytestmark = pytest.mark.gpu
FMTS = ("nvfp4", "mxfp4")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows(g, rows, K):
    """Rows of very different loudness, loud channels, zeros, ties."""
    x = torch.randn(rows, K, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g, device="cuda").float())
    x[:, ::37] *= 64
    x[:, 32:64] *= 2.0 ** -12          # a quiet block
    if K > 64:
        x[:, 64:96] = 0
    x[rows // 2:, ::3] = (x[rows // 2:, ::3] * 8).round() / 8
    return x.bfloat16()


def _check(rows, t, fmt, factor=None):
    """rows against the definition for t (fp64); factor: the norm's, with its relative error bound."""
    n, K = t.shape
    codes, scales, s = _fp4.quantize(t, fmt)
    held = _fp4.untile(rows.block_scales, n, K, fmt)
    groups = K // _fp4.BLOCK[fmt]
    assert torch.equal(held[:, :groups], scales)
    assert not held[:, groups:].any(), "scales past K are 0"
    assert torch.equal(rows.codes, codes)
    if factor is not None:
        want = s * factor[0]
        assert ((rows.row_scales.double() - want).abs() <= factor[1] * want).all()
    elif fmt == "nvfp4":
        assert torch.equal(rows.row_scales.double(), s)
    else:
        assert rows.row_scales is None


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (5, 224), (129, 256), (2, 288), (33, 2080), (7, 4096), (3, 8192),
                                    (2, 8224), (2, 16384), (2, 16416), (3, 32768), (1, 131072)])
def test_rows(fmt, rows, K):
    x = _rows(_gen(rows * K), rows, K)
    _check(i8.quant_rows_fp4(x, fmt), x.double(), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_every_bf16_beside_every_loudness(fmt):
    """Each finite bf16 as an element of blocks whose largest magnitude goes through
    the significands."""
    every = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    every = every[torch.isfinite(every)]
    block = _fp4.BLOCK[fmt]
    small = every[(every.abs() <= 2.0 ** -3) & (every.abs() >= 2.0 ** -9)]
    tops = torch.arange(128, 256, device="cuda").float().div(128).bfloat16()
    n = small.numel() // (block - 1)
    body = small[: n * (block - 1)].view(n, block - 1)
    x = torch.cat([torch.cat((body, t.repeat(n, 1)), 1) for t in tops]).reshape(-1, 32 * 8)
    _check(i8.quant_rows_fp4(x, fmt), x.double(), fmt)
    x = every[: every.numel() // 256 * 256].view(-1, 256)[:, torch.randperm(256, generator=_gen(0), device="cuda")].contiguous()
    if fmt == "mxfp4":
        _check(i8.quant_rows_fp4(x, fmt), x.double(), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_strided_rows_and_given_buffers(fmt):
    wide = _rows(_gen(3), 70, 1024)
    x = wide[:, 512:832]
    out = i8.FP4Rows.empty(70, 320, fmt)
    out.block_scales.fill_(0x55)
    got = i8.quant_rows_fp4(x, fmt, out=out)
    assert got is out
    _check(got, x.double(), fmt)
    assert (_fp4.untile(out.block_scales, 128, 320, fmt)[70:] == 0x55).all(), "scales behind the last row stay"


@pytest.mark.parametrize("fmt", FMTS)
def test_zero_rows_and_no_rows(fmt):
    x = torch.zeros(4, 96, device="cuda", dtype=torch.bfloat16)
    x[2, 5] = 1
    got = i8.quant_rows_fp4(x, fmt)
    _check(got, x.double(), fmt)
    assert torch.equal(_fp4.values(got) != 0, x != 0)
    assert i8.quant_rows_fp4(x[:0], fmt).shape == (0, 96)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite_show(fmt, bad):
    x = torch.ones(3, 96, device="cuda", dtype=torch.bfloat16)
    want = _fp4.values(i8.quant_rows_fp4(x, fmt))
    assert torch.isfinite(want).all()
    x[1, 40] = bad
    v = _fp4.values(i8.quant_rows_fp4(x, fmt))
    assert torch.equal(v[0::2], want[0::2])
    assert torch.isnan(v[1, 32:64]).all()
    if fmt == "mxfp4":
        assert torch.equal(v[1, :32], want[1, :32]) and torch.equal(v[1, 64:], want[1, 64:])


def _norm_case(g, M, K, loud=4.0):
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    r = (torch.randn(M, K, generator=g, device="cuda") * loud).bfloat16()
    w = (1 + 0.1 * torch.randn(K, generator=g, device="cuda")).bfloat16()
    return x, r, w


def _norm_check(rows, x, r, w, eps, fmt):
    # t as fp32 holds it: the sum is exact or rounded once, the product rounded once
    h = x.float() + r.float() if r is not None else x.float()
    t = h * w.float() if w is not None else h
    d = x.double() + (r.double() if r is not None else 0)
    factor = 1 / (d.square().mean(1) + eps).sqrt()
    # the sum of squares: each of them and the additions rounded to 2^-24, K / (32 * warps) deep and the
    # tree's; halved by the square root; four more steps
    K = x.shape[1]
    _check(rows, t.double(), fmt, (factor, (K / 512 + 40) * 2.0 ** -24))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K", [(1, 32), (5, 544), (64, 2048), (130, 4096), (3, 16384), (2, 32768), (2, 33024)])
@pytest.mark.parametrize("residual,weight", [(True, True), (False, True), (True, False), (False, False)])
def test_norm(fmt, M, K, residual, weight):
    x, r, w = _norm_case(_gen(M + K), M, K)
    r, w = r if residual else None, w if weight else None
    got = i8.add_rmsnorm_quant_fp4(x, r, w, eps=1e-5, fmt=fmt)
    rows, h = got if residual else (got, None)
    _norm_check(rows, x, r, w, 1e-5, fmt)
    if residual:
        assert torch.equal(h, (x.float() + r.float()).bfloat16())


@pytest.mark.parametrize("K", [512, 40960])
@pytest.mark.parametrize("where", ["residual", "x"])
def test_norm_in_place(K, where):
    x, r, w = _norm_case(_gen(K), 9, K)
    x0, r0 = x.clone(), r.clone()
    rows, h = i8.add_rmsnorm_quant_fp4(x, r, w, residual_out=r if where == "residual" else x)
    assert h is (r if where == "residual" else x)
    assert torch.equal(h, (x0.float() + r0.float()).bfloat16())
    _norm_check(rows, x0, r0, w, 1e-6, "nvfp4")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("exponent", [-120, -70, -34, 40, 63, 70, 100])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norm_of_rows_whose_squares_leave_the_range(fmt, exponent, eps):
    x, _, w = _norm_case(_gen(7), 6, 512)
    x = (x.double() * 2.0 ** exponent).bfloat16()
    rows = i8.add_rmsnorm_quant_fp4(x, None, w, eps=eps, fmt=fmt)
    _norm_check(rows, x, None, w, eps, fmt)


def test_norm_of_zeros():
    x = torch.zeros(3, 64, device="cuda", dtype=torch.bfloat16)
    for fmt in FMTS:
        for eps in (0.0, 1e-6):
            assert not _fp4.values(i8.add_rmsnorm_quant_fp4(x, eps=eps, fmt=fmt)).any()
