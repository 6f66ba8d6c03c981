"""The norm and rotation of query and key heads against the formula in 64 bits.

The output is within half a step of bf16 (2^-8 of the value) of it, and, because
fp32 holds what comes before, within a few 2^-24 of the pair's size: the angle is
off by up to 2 pi 2^-24, the norm by some 2^-22, products and sums by 2^-24 each."""
import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _reference(x, weight, positions, inv_freq, sections, interleaved, eps):
    x = x.double()
    if weight is not None:
        x = x / (x.square().mean(2, keepdim=True) + eps).sqrt() * weight.double()
    n = inv_freq.shape[0]
    where = positions.reshape(-1, x.shape[0]).double()
    turn = torch.cat([p[:, None] * f for p, f in zip(where, inv_freq.double().split(sections))], 1)[:, None]
    y, size = x.clone(), x.abs()
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    y[:, :, a] = x[:, :, a] * turn.cos() - x[:, :, b] * turn.sin()
    y[:, :, b] = x[:, :, b] * turn.cos() + x[:, :, a] * turn.sin()
    pair = x[:, :, a].abs() + x[:, :, b].abs()
    size[:, :, a] = size[:, :, b] = pair
    return y, size


def _case(seed, T, Hq, Hk, D, R, axes=1, far=131071, norm=True):
    g = _gen(seed)
    qkv = (torch.randn(T, Hq + 2 * Hk, D, generator=g, device="cuda") * 3).bfloat16()
    q, k, _ = qkv.split((Hq, Hk, Hk), dim=1)
    n = R // 2
    sections = [n // axes + (1 if i < n % axes else 0) for i in range(axes)]
    positions = torch.randint(0, far + 1, (axes, T), generator=g, device="cuda", dtype=torch.int32)
    inv = torch.cat([10000.0 ** (-torch.arange(s, device="cuda").double() / max(s, 1)) for s in sections]).float()
    w = [(1 + 0.1 * torch.randn(D, generator=g, device="cuda")).bfloat16() if norm else None for _ in range(2)]
    return qkv, q, k, positions if axes > 1 else positions[0].contiguous(), inv, sections, w


def _check(got, x, weight, positions, inv, sections, interleaved, eps):
    want, size = _reference(x, weight, positions, inv, sections, interleaved, eps)
    tol = 2.0 ** -8 * want.abs() + 40 * 2.0 ** -24 * size + 1e-38
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got.double() - want).abs() / tol).max()))


@pytest.mark.parametrize("T,Hq,Hk,D,R", [(1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (3, 5, 1, 80, 80), (64, 24, 8, 128, 128),
                                         (77, 24, 24, 96, 48), (19, 16, 2, 256, 256), (5, 7, 3, 72, 32), (9, 2, 2, 8, 0),
                                         (4, 3, 2, 512, 512), (6, 4, 2, 120, 16), (5000, 3, 1, 64, 32), (1300, 40, 8, 128, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_heads(T, Hq, Hk, D, R, interleaved, norm):
    _, q, k, positions, inv, sections, w = _case(T + D, T, Hq, Hk, D, R, norm=norm)
    qo, ko = i8.heads_rmsnorm_rotate(q, k, positions, inv, *w, interleaved=interleaved)
    _check(qo, q, w[0], positions, inv, sections, interleaved, 1e-6)
    _check(ko, k, w[1], positions, inv, sections, interleaved, 1e-6)


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("interleaved", [False, True])
def test_axes(axes, interleaved):
    _, q, k, positions, inv, sections, w = _case(axes, 301, 6, 2, 128, 96, axes=axes, far=900)
    got = i8.heads_rmsnorm_rotate(q, k, positions, inv, *w, sections=sections, interleaved=interleaved)
    for y, x, g in zip(got, (q, k), w):
        _check(y, x, g, positions, inv, sections, interleaved, 1e-6)


def test_an_axis_may_turn_nothing():
    _, q, k, positions, inv, _, w = _case(1, 20, 2, 1, 64, 64, axes=3, far=50)
    got = i8.heads_rmsnorm_rotate(q, k, positions, inv, *w, sections=(0, 20, 12))
    _check(got[0], q, w[0], positions, inv, [0, 20, 12], False, 1e-6)


@pytest.mark.parametrize("positions", [(0, 1, 2, 3), (131071, 131072, 1048575, 1048576), (-1, -2, -4096, -131071),
                                       (4095, 4096, 4097, 8191)])
def test_far_and_negative_positions(positions):
    _, q, k, _, inv, sections, w = _case(8, 4, 8, 2, 128, 128, norm=False)
    p = torch.tensor(positions, dtype=torch.int32, device="cuda")
    got = i8.heads_rmsnorm_rotate(q, k, p, inv)
    _check(got[0], q, None, p, inv, sections, False, 1e-6)


@pytest.mark.parametrize("one", [0, 1])
def test_a_norm_of_one_of_them(one):
    _, q, k, positions, inv, sections, w = _case(3, 50, 9, 3, 64, 64)
    w[one] = None
    got = i8.heads_rmsnorm_rotate(q, k, positions, inv, *w)
    for y, x, g in zip(got, (q, k), w):
        _check(y, x, g, positions, inv, sections, False, 1e-6)


@pytest.mark.parametrize("T", [1, 70, 3000])
def test_in_place(T):
    qkv, q, k, positions, inv, sections, w = _case(T, T, 12, 4, 128, 128)
    before = qkv.clone()
    got = i8.heads_rmsnorm_rotate(q, k, positions, inv, *w, out=(q, k))
    assert got[0] is q and got[1] is k
    q0, k0, v0 = before.split((12, 4, 4), dim=1)
    _check(q, q0, w[0], positions, inv, sections, False, 1e-6)
    _check(k, k0, w[1], positions, inv, sections, False, 1e-6)
    assert torch.equal(qkv[:, 16:], v0)


@pytest.mark.parametrize("exponent", [-125, -70, 62, 70, 120])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norm_of_heads_whose_squares_leave_the_range(exponent, eps):
    _, q, k, positions, inv, sections, w = _case(5, 7, 3, 1, 64, 64)
    q = (q.double() * 2.0 ** exponent).bfloat16()     # the keys stay as they are: rows of both kinds in a warp
    got = i8.heads_rmsnorm_rotate(q, k, positions, inv, *w, eps=eps)
    for y, x, g in zip(got, (q, k), w):
        _check(y, x, g, positions, inv, sections, False, eps)


def test_a_nan_shows_in_its_head_only():
    _, q, k, positions, inv, sections, w = _case(6, 9, 4, 2, 64, 64)
    q[3, 2, 5] = float("nan")
    qo, ko = i8.heads_rmsnorm_rotate(q, k, positions, inv, *w)
    bad = torch.isnan(qo)
    assert bad[3, 2].all() and bad.sum() == 64 and not torch.isnan(ko).any()


def test_no_tokens_and_no_keys():
    _, q, k, positions, inv, sections, w = _case(2, 6, 4, 2, 64, 64)
    qo, ko = i8.heads_rmsnorm_rotate(q[:0], k[:0], positions[:0], inv, *w)
    assert qo.shape == (0, 4, 64) and ko.shape == (0, 2, 64)
    qo, ko = i8.heads_rmsnorm_rotate(q, k[:, :0], positions, inv, *w)
    _check(qo, q, w[0], positions, inv, sections, False, 1e-6)
    i8.sync_check()


def test_another_stream_and_a_graph():
    _, q, k, positions, inv, sections, w = _case(4, 40, 8, 2, 128, 128)
    want = i8.heads_rmsnorm_rotate(q, k, positions, inv, *w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = i8.heads_rmsnorm_rotate(q, k, positions, inv, *w)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph, held = torch.cuda.CUDAGraph(), torch.zeros_like(positions)
    with torch.cuda.graph(graph):
        got = i8.heads_rmsnorm_rotate(q, k, held, inv, *w)
    held.copy_(positions)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_without_a_norm_what_is_not_finite_stays_in_its_pair(interleaved, bad):
    _, q, k, positions, inv, sections, _ = _case(6, 9, 4, 2, 128, 64, norm=False)
    q[3, 2, 5], q[3, 2, 70], q[4, 1, 101] = bad, bad, bad     # one that is rotated, two that are not
    qo, ko = i8.heads_rmsnorm_rotate(q, k, positions, inv, interleaved=interleaved)
    where = (~torch.isfinite(qo)).nonzero().tolist()
    assert where == [[3, 2, 4], [3, 2, 5], [3, 2, 70], [4, 1, 101]] if interleaved else \
        where == [[3, 2, 5], [3, 2, 37], [3, 2, 70], [4, 1, 101]]
    assert torch.isfinite(ko).all()
    keep = torch.ones(9, dtype=torch.bool, device="cuda")
    keep[3:5] = False
    _check(qo[keep], q[keep], None, positions[keep], inv, sections, interleaved, 1e-6)
