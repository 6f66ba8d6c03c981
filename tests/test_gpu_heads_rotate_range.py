"""The norm and rotation of heads at the ends of bf16's range, against the formula in
64 bits (tolerances: see test_gpu_heads_rotate.py; fp32 holds the steps between, and
what an element is scaled by on the way is a power of two)."""
import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from tests.test_gpu_heads_rotate import _case, _check, _gen

pytestmark = pytest.mark.gpu
LARGEST = float(torch.finfo(torch.bfloat16).max)


def _both(q, k, positions, inv, sections, w, eps, interleaved=False):
    got = i8.heads_rmsnorm_rotate(q, k, positions, inv, *w, eps=eps, interleaved=interleaved)
    for y, x, g in zip(got, (q, k), w):
        assert torch.isfinite(y).all()
        _check(y, x, g, positions, inv, sections, interleaved, eps)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(64, 64), (96, 48), (128, 128), (256, 256), (8, 0)])
@pytest.mark.parametrize("size", [2.0 ** 120, 2.0 ** 126, 1.7e38, 2.4e38, LARGEST])
def test_elements_up_to_the_largest(size, D, R, interleaved):
    _, q, k, positions, inv, sections, w = _case(int(D + R), 9, 5, 3, D, R)
    g = _gen(1)
    # all of a size, and a pair of loud ones among quiet ones
    q = (torch.rand(q.shape, generator=g, device="cuda") * 2 - 1).mul(size).bfloat16()
    k = (torch.randn(k.shape, generator=g, device="cuda") * 1e30).bfloat16()
    k[:, :, 0], k[:, :, 1] = size, -size
    if R:
        k[:, :, R // 2] = size
    assert torch.isfinite(q).all() and torch.isfinite(k).all()
    for gains in (w, [(2 * v).bfloat16() for v in w], [(v / 3).bfloat16() for v in w]):
        _both(q, k, positions, inv, sections, gains, 1e-6, interleaved)


def test_two_that_form_a_pair():
    q = torch.full((1, 1, 64), 1e30, device="cuda").bfloat16()
    q[0, 0, 0] = q[0, 0, 32] = 3e38
    w = torch.full((64,), 1.1, device="cuda").bfloat16()
    inv = torch.full((32,), 0.7, device="cuda")
    positions = torch.ones(1, dtype=torch.int32, device="cuda")
    _both(q, q.clone(), positions, inv, [32], [w, w], 1e-6)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(64, 64), (96, 48), (128, 128)])
@pytest.mark.parametrize("exponent", [-133, -132, -130, -128, -127, -126])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -149, 1e-38, 1e-6])
def test_elements_down_to_the_smallest(exponent, eps, D, R, interleaved):
    _, q, k, positions, inv, sections, w = _case(int(D + R), 9, 5, 3, D, R)
    g = _gen(2)
    # whole numbers of the smallest, so that each element is a number of bf16's
    step = 2.0 ** exponent
    q, k = (torch.randint(-3, 4, t.shape, generator=g, device="cuda").double().mul(step).bfloat16() for t in (q, k))
    q[:, :, 3] = k[:, :, 5] = step
    _both(q, k, positions, inv, sections, w, eps, interleaved)


@pytest.mark.parametrize("gain", [2.0 ** -120, 2.0 ** 70, 2.0 ** 120])
def test_gains_far_from_one(gain):
    _, q, k, positions, inv, sections, w = _case(4, 9, 5, 3, 64, 64)
    q = (q.float() * 2.0 ** 58).bfloat16()
    _both(q, k, positions, inv, sections, [(v.double() * gain).bfloat16() for v in w], 1e-6)
