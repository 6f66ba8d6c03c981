"""One to four tokens, which the 4-bit layer quantizes inside its product: the bits
are those of the quantizer and the product called one after the other."""
import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8

pytestmark = pytest.mark.gpu
FMTS = ("nvfp4", "mxfp4")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _layer(g, M, N, K, fmt):
    x = torch.randn(M, K, generator=g, device="cuda")
    x[:, :: max(1, K // 5)] *= 8
    w = (torch.randn(N, K, generator=g, device="cuda") * 0.05).bfloat16()
    return x.bfloat16(), i8.quant_rows_fp4(w, fmt), torch.randn(N, generator=g, device="cuda").bfloat16()


def _same(got, want):
    """Bit for bit, a NaN like any other NaN."""
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(0.0, torch.inf, -torch.inf), want.nan_to_num(0.0, torch.inf, -torch.inf))


@pytest.fixture(params=[0, 1, 2, 3, 4, 8])
def splits(request):
    """How many CTAs share K (0: the library's choice); more than K or the kernel has room for are fewer."""
    i8.set_option("force_splits", request.param)
    yield request.param
    i8.set_option("force_splits", 0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("N,K", [(8, 32), (136, 288), (264, 1056), (128, 2048), (1000, 4128), (64, 20000)])
def test_the_bits_of_the_two_calls(fmt, M, N, K, splits):
    g = _gen(M * N + K)
    x, w, b = _layer(g, M, N, K, fmt)
    _same(i8.linear_fp4(x, w, b), i8.gemm_fp4_bias_bf16(i8.quant_rows_fp4(x, fmt), w, b))
    up = i8.quant_rows_fp4((torch.randn(N, K, generator=g, device="cuda") * 0.05).bfloat16(), fmt)
    for act in ("silu", "gelu"):
        _same(i8.gated_linear_fp4(x, w, up, b, None, activation=act),
              i8.gemm_fp4_gated_bf16(i8.quant_rows_fp4(x, fmt), w, up, b, None, activation=act))
    i8.sync_check()


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_of_all_magnitudes(fmt, splits):
    """Zeros, the smallest and the largest numbers, a NaN and an infinity, each in a row of its own."""
    g = _gen(3)
    N, K = 136, 1312
    _, w, b = _layer(g, 1, N, K, fmt)
    unit = torch.randn(4, K, generator=g, device="cuda").clamp(-3, 3)
    for factors in ([0.0, 1.0, 2.0 ** -133, 2.0 ** 125], [2.0 ** -110, 2.0 ** 110, 2.0 ** -126, 0.0]):
        x = (unit * torch.tensor(factors, device="cuda")[:, None]).bfloat16()
        _same(i8.linear_fp4(x, w, b), i8.gemm_fp4_bias_bf16(i8.quant_rows_fp4(x, fmt), w, b))
        _same(i8.linear_fp4(x, w), i8.gemm_fp4_bias_bf16(i8.quant_rows_fp4(x, fmt), w))
    x = unit.bfloat16()
    x[1, K - 1], x[2, 5] = torch.nan, -torch.inf
    got = i8.linear_fp4(x, w, b)
    _same(got, i8.gemm_fp4_bias_bf16(i8.quant_rows_fp4(x, fmt), w, b))
    assert torch.isnan(got[1:3]).all() and torch.isfinite(got[[0, 3]]).all()
    i8.sync_check()


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_apart_and_an_output_over_the_tokens(fmt):
    x, w, b = _layer(_gen(4), 3, 512, 512, fmt)
    want = i8.linear_fp4(x, w, b)
    wide = torch.full((5, 1024), torch.nan, dtype=torch.bfloat16, device="cuda")
    wide[1:4, 256:768] = x
    assert torch.equal(i8.linear_fp4(wide[1:4, 256:768], w, b), want)
    for first in (0, 1, 2):  # in place, and a row further up or down
        rows = torch.empty(5, 512, dtype=torch.bfloat16, device="cuda")
        rows[1:4] = x
        assert torch.equal(i8.linear_fp4(rows[1:4], w, b, out=rows[first:first + 3]), want)
    # beside the tokens in one matrix
    both = torch.zeros(3, 1024, dtype=torch.bfloat16, device="cuda")
    both[:, :512] = x
    assert torch.equal(i8.linear_fp4(both[:, :512], w, b, out=both[:, 512:]), want)
    assert torch.equal(both[:, :512], x)
    i8.sync_check()


@pytest.mark.parametrize("M", [1, 4])
def test_behind_the_kernel_that_writes_the_tokens(M):
    """In a graph, layer upon layer: each begins while the one before it ends."""
    x, w, b = _layer(_gen(5), M, 2048, 2048, "nvfp4")
    def run(call):
        y = x
        for _ in range(6):
            y = call(y) * 0.25
        return y
    want = run(lambda t: i8.gemm_fp4_bias_bf16(i8.quant_rows_fp4(t, "nvfp4"), w, b))
    run(lambda t: i8.linear_fp4(t, w, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(lambda t: i8.linear_fp4(t, w, b))
    for _ in range(20):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    # without a kernel of torch's between them
    direct = x
    for _ in range(6):
        direct = i8.linear_fp4(direct, w, b)
    again = x
    for _ in range(6):
        again = i8.gemm_fp4_bias_bf16(i8.quant_rows_fp4(again, "nvfp4"), w, b)
    assert torch.equal(direct, again)
    i8.sync_check()
