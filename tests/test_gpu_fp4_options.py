"""The options of the tiled kernels, on the 4-bit route: same bits, other CTAs."""
import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from tests.test_gpu_fp4_gemm import FMTS, _exact_rows, _gen

pytestmark = pytest.mark.gpu


@pytest.fixture
def options():
    yield i8.set_option
    i8.set_option("max_ctas", 0)
    i8.set_option("cta_pair", 0)


def _time(call):
    """The quickest of a few, in ms."""
    best = float("inf")
    for _ in range(5):
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        call()
        end.record()
        end.synchronize()
        best = min(best, begin.elapsed_time(end))
    return best


def _operands(M, N, K, fmt):
    g = _gen(M)
    return [_exact_rows(g, n, K, fmt, True) for n in (M, N, N)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(2048, 4096, 1024), (300, 520, 544)])
def test_a_cap_on_the_grid(fmt, M, N, K, options):
    a, w, u = _operands(M, N, K, fmt)
    want, gated = i8.gemm_fp4_bias_bf16(a, w), i8.gemm_fp4_gated_bf16(a, w, u)
    options("cta_pair", 2)
    for ctas in (1, 2, 3, 10, 151, 100000):
        options("max_ctas", ctas)
        assert torch.equal(i8.gemm_fp4_bias_bf16(a, w), want) and torch.equal(i8.gemm_fp4_gated_bf16(a, w, u), gated)
    i8.sync_check()


def test_the_options_have_an_effect(options):
    """16 x 16 tiles on one pair, one after the other, and on all of them; the kernel without pairs has no cap."""
    a, w, u = _operands(4096, 4096, 4096, "mxfp4")
    for call in (lambda: i8.gemm_fp4_bias_bf16(a, w), lambda: i8.gemm_fp4_gated_bf16(a, w, u)):
        options("max_ctas", 0)
        options("cta_pair", 2)
        free = _time(call)
        options("max_ctas", 2)
        one = _time(call)
        options("cta_pair", 1)
        never = _time(call)
        assert one > 10 * free and one > 5 * never, (free, one, never)
