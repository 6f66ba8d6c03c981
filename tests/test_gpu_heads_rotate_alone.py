"""A head's bits are its own: they do not depend on what the heads beside it hold."""
import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from tests.test_gpu_heads_rotate import _case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(64, 64), (96, 96), (128, 128), (128, 64), (256, 256), (24, 16)])
@pytest.mark.parametrize("beside", [0.0, 2.0 ** -100, 2.0 ** 100, float("inf"), float("nan")])
def test_what_lies_beside_a_head_does_not_count(beside, D, R, interleaved):
    _, q, k, positions, inv, _, w = _case(D + R, 260, 7, 4, D, R)
    want = i8.heads_rmsnorm_rotate(q, k, positions, inv, *w, interleaved=interleaved)
    qm, km = (torch.rand(t.shape[:2], generator=torch.Generator().manual_seed(n)).cuda() < 0.5 for n, t in enumerate((q, k)))
    qz, kz = q.clone(), k.clone()
    qz[qm], kz[km] = beside, beside
    got = i8.heads_rmsnorm_rotate(qz, kz, positions, inv, *w, interleaved=interleaved)
    assert torch.equal(got[0][~qm], want[0][~qm]) and torch.equal(got[1][~km], want[1][~km])


@pytest.mark.parametrize("D", [64, 96, 128])
def test_a_head_alone_and_among_others(D):
    _, q, k, positions, inv, _, w = _case(D, 50, 8, 2, D, D)
    want = i8.heads_rmsnorm_rotate(q, k, positions, inv, *w)
    for head in (0, 3, 7):
        got = i8.heads_rmsnorm_rotate(q[:, head:head + 1], k[:, :0], positions, inv, *w)
        assert torch.equal(got[0], want[0][:, head:head + 1])
    # the last tokens as a batch of their own
    got = i8.heads_rmsnorm_rotate(q[33:], k[33:], positions[33:].contiguous(), inv, *w)
    assert torch.equal(got[0], want[0][33:]) and torch.equal(got[1], want[1][33:])
