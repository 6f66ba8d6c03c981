"""The 4-bit products against the definition in 64 bits.

Exact cases: codes and block scales whose products sum to numbers that fp32 holds,
so the bf16 output is the rounded exact one, bit for bit, whatever the order of
the sum.  Others: within the rounding of the output (half a step of bf16, 2^-8 of
the value) and of the fp32 sum (K additions of 2^-24 of the sum of magnitudes, and
the epilogue's steps)."""
import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from tests import _fp4

pytestmark = pytest.mark.gpu
FMTS = ("nvfp4", "mxfp4")
# tokens, channels, K: one token; odd sizes; the borders of the tiles; several tiles; K that ends inside a tile of 256
SIZES = [(1, 8, 32), (1, 128, 256), (2, 136, 288), (15, 264, 512), (16, 128, 1056), (17, 1000, 2048), (32, 64, 96),
         (33, 256, 4096), (64, 512, 768), (65, 392, 1312), (127, 128, 256), (128, 136, 544), (129, 1288, 1024),
         (255, 256, 512), (256, 512, 256), (257, 520, 2080), (300, 2056, 1024), (513, 768, 4128), (1000, 1304, 320),
         (2600, 2824, 288), (1024, 6400, 768),
         (2049, 2312, 512)]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _exact_rows(g, rows, K, fmt, row_scales):
    """Random codes of 0, +-1, +-2, +-0.5 and block scales of 1/2, 1, 2: a product is at most 16 in units of
    1/16, so sums of 4128 of them stay below 2^24 units."""
    nibbles = torch.tensor([0, 1, 2, 4, 9, 10, 12, 0], dtype=torch.uint8, device="cuda")[
        torch.randint(0, 8, (rows, K), generator=g, device="cuda")]
    codes = nibbles[:, 0::2] | (nibbles[:, 1::2] << 4)
    held = torch.tensor([0x30, 0x38, 0x40] if fmt == "nvfp4" else [126, 127, 128], dtype=torch.uint8, device="cuda")[
        torch.randint(0, 3, (rows, K // _fp4.BLOCK[fmt]), generator=g, device="cuda")]
    s = torch.exp2(torch.randint(-3, 4, (rows,), generator=g, device="cuda").float()) if row_scales else None
    return i8.FP4Rows(codes.contiguous(), _fp4.tile(held, fmt), s)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_exact_product(fmt, M, N, K):
    g = _gen(M * N + K)
    a, w = _exact_rows(g, M, K, fmt, fmt == "nvfp4"), _exact_rows(g, N, K, fmt, True)
    want = _fp4.values(a) @ _fp4.values(w).T
    got = i8.gemm_fp4_bias_bf16(a, w)
    assert torch.equal(got, want.float().bfloat16())
    assert torch.equal(i8.gemm_fp4_bias_bf16(a, w), got), "repeated calls give the same bits"
    i8.sync_check()


def _gate64(g, u, activation):
    # (erfc: 1 + erf cancels where g is far below 0)
    return (torch.nn.functional.silu(g) if activation == "silu" else 0.5 * g * torch.special.erfc(-g * 0.5 ** 0.5)) * u


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("activation", ["silu", "gelu"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gated_product(fmt, activation, M, N, K):
    g = _gen(M * N + K + 1)
    a, gate, up = (_exact_rows(g, n, K, fmt, True) for n in (M, N, N))
    bg, bu = ((torch.randint(-8, 9, (N,), generator=g, device="cuda") / 8).bfloat16() for _ in range(2))
    va, small = _fp4.values(a), 1 / 16.0
    gate = gate._replace(row_scales=gate.row_scales * small)
    pre = va @ _fp4.values(gate).T + bg.double()
    u = va @ _fp4.values(up).T + bu.double()
    want = _gate64(pre, u, activation)
    got = i8.gemm_fp4_gated_bf16(a, gate, up, bg, bu, activation=activation).double()
    # half a step of bf16; exp, erfc and the division to a few units of fp32 beside it, and where |g| is large
    # and negative the factor's relative error grows with |g| (that of exp's argument)
    tol = (2.0 ** -8 + (16 + 2 * pre.abs()) * 2.0 ** -23) * want.abs() + 1e-30
    assert ((got - want).abs() <= tol).all(), float(((got - want).abs() / tol).max())
    i8.sync_check()


def _dense(g, M, N, K, loud=8):
    x = torch.randn(M, K, generator=g, device="cuda")
    x[:, :: max(1, K // 5)] *= loud
    return x.bfloat16(), (torch.randn(N, K, generator=g, device="cuda") * 0.05).bfloat16(), \
        torch.randn(N, generator=g, device="cuda").bfloat16()


def _bound(va, vw, bias):
    """(value in 64 bits, tolerance) of a product."""
    want, size = va @ vw.T, va.abs() @ vw.abs().T
    want = want + bias.double()
    return want, 2.0 ** -8 * want.abs() + (va.shape[1] + 4) * 2.0 ** -24 * (size + bias.double().abs())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear(fmt, M, N, K):
    x, w, b = _dense(_gen(M + N + K), M, N, K)
    rows = i8.quant_rows_fp4(w, fmt)
    got = i8.linear_fp4(x, rows, b).double()
    want, tol = _bound(_fp4.values(i8.quant_rows_fp4(x, fmt)), _fp4.values(rows), b)
    assert ((got - want).abs() <= tol).all()
    i8.sync_check()


@pytest.mark.parametrize("fmt", FMTS)
def test_all_codes_and_scales(fmt):
    """Every code, and every finite block scale that keeps the sums in fp32's range."""
    g = _gen(5)
    M, N, K = 48, 64, 512
    rows = []
    for n in (M, N):
        codes = torch.randint(0, 256, (n, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        low, high = (0, 127) if fmt == "nvfp4" else (127 - 25, 127 + 25)
        held = torch.randint(low, high, (n, K // _fp4.BLOCK[fmt]), generator=g, device="cuda", dtype=torch.uint8)
        rows.append(i8.FP4Rows(codes, _fp4.tile(held, fmt), torch.rand(n, generator=g, device="cuda") + 0.5))
    got = i8.gemm_fp4_bias_bf16(*rows).double()
    want, tol = _bound(_fp4.values(rows[0]), _fp4.values(rows[1]), torch.zeros(N, device="cuda").bfloat16())
    assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [3, 200, 600])
def test_what_is_not_finite_shows_in_its_rows_only(fmt, M):
    x, w, b = _dense(_gen(M), M, 264, 544)
    x[1, 300] = float("nan")
    rows = i8.quant_rows_fp4(w, fmt)
    if fmt == "nvfp4":
        rows.row_scales[7] = float("nan")
    y = i8.linear_fp4(x, rows, b)
    assert torch.isnan(y[1]).all()
    bad = torch.isnan(y)
    bad[1] = False
    if fmt == "nvfp4":
        assert bad[:, 7].sum() == M - 1
        bad[:, 7] = False
    assert not bad.any()


@pytest.mark.parametrize("M", [5, 140, 700])
def test_strided_output_keeps_what_lies_between(M):
    x, w, b = _dense(_gen(M), M, 264, 256)
    rows = i8.quant_rows_fp4(w, "nvfp4")
    want = i8.linear_fp4(x, rows, b)
    wide = torch.full((M + 2, 264 + 24), 7.0, device="cuda", dtype=torch.bfloat16)
    got = i8.linear_fp4(x, rows, b, out=wide[1:-1, 8:-16])
    assert got.data_ptr() == wide[1:-1, 8:-16].data_ptr() and torch.equal(got, want)
    assert (wide[0] == 7).all() and (wide[-1] == 7).all() and (wide[:, :8] == 7).all() and (wide[:, -16:] == 7).all()


def test_no_tokens_and_no_channels():
    x, w, b = _dense(_gen(1), 4, 16, 64)
    rows = i8.quant_rows_fp4(w, "mxfp4")
    assert i8.linear_fp4(x[:0], rows, b).shape == (0, 16)
    assert i8.linear_fp4(x, i8.quant_rows_fp4(w[:0], "mxfp4")).shape == (4, 0)
    i8.sync_check()


@pytest.mark.parametrize("M", [1, 40, 300])
def test_another_stream_and_a_graph(M):
    x, w, b = _dense(_gen(M), M, 512, 768)
    gate, up = i8.quant_rows_fp4(w, "nvfp4"), i8.quant_rows_fp4(w.flip(0).contiguous(), "nvfp4")
    want, want_gated = i8.linear_fp4(x, gate, b), i8.gated_linear_fp4(x, gate, up, b, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = i8.linear_fp4(x, gate, b)
    side.synchronize()
    assert torch.equal(got, want)
    graph, held = torch.cuda.CUDAGraph(), torch.zeros_like(x)
    with torch.cuda.graph(graph):
        y, u = i8.linear_fp4(held, gate, b), i8.gated_linear_fp4(held, gate, up, b, None)
    held.copy_(x)
    for _ in range(2):
        y.zero_(), u.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(u, want_gated)
    i8.sync_check()
