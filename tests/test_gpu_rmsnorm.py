"""add_rmsnorm_quant_act_pertoken against its definition.

Codes and h bit for bit: t = h * w, max|t| and the quotients are fp32 steps
whose result does not depend on any order.  Scales within 2^-20 relative: the
fp32 sum of K squares in some order (each lane at most 8 V + 25 additions, a
relative 2^-24 each, halved by the square root), four roundings after it.
"""
import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from tests import _serving as ref

pytestmark = pytest.mark.gpu


def _values(q):
    return ref.code_values(q)


def _compare(r, x, residual, weight, eps, fmt):
    codes, scale, h = ref.norm_reference(x, residual, weight, eps, fmt)
    assert torch.equal(_values(r[0]), codes)
    got = r[1].cpu().double()
    assert (got - scale).abs().le(2.0 ** -20 * scale + 1e-44).all()
    if residual is not None:
        assert torch.equal(r[2].cpu().view(torch.int16), h.bfloat16().view(torch.int16))


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "f16codes"])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 3072), (3, 48), (7, 264 * 2), (33, 4096), (5, 10512), (2, 32768), (300, 144)])
def test_matches_definition(M, K, fmt):
    g = torch.Generator().manual_seed(M * 100003 + K)
    x = torch.randn(M, K, generator=g).bfloat16()
    res = (torch.randn(M, K, generator=g) * 3).bfloat16()
    res[:, torch.randperm(K, generator=g)[: max(1, K // 100)]] *= 20
    w = (1 + 0.2 * torch.randn(K, generator=g)).bfloat16()
    for residual, weight in ((res, w), (None, w), (res, None), (None, None)):
        args = [t.cuda() if t is not None else None for t in (x, residual, weight)]
        r = i8.add_rmsnorm_quant_act_pertoken(*args, fmt=fmt)
        i8.sync_check()
        _compare(r, x, residual, weight, 1e-6, fmt)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_near_ties_and_small_values(fmt):
    """Quotients on and next to the ties of the code format, and far below it."""
    K = 4096
    g = torch.Generator().manual_seed(3)
    top = ref.LIMIT[fmt]
    base = torch.randint(-int(top) * 2, int(top) * 2 + 1, (16, K), generator=g).float() / 4
    base[8:] = torch.exp2(torch.randint(-20, 9, (8, K), generator=g).float()) * (1 + torch.randint(0, 16, (8, K), generator=g) / 16)
    base[:, 0] = top
    base = base.clamp(-top, top)
    scale = torch.tensor([1.0, 2.0 ** -10, 3.0, 0.1, 7e-3, 1e10, 1e-10, 1e-30] * 2)[:, None]
    x = (base * scale).bfloat16()
    w = torch.ones(K).bfloat16()
    w[K // 2:] = 1.25
    r = i8.add_rmsnorm_quant_act_pertoken(x.cuda(), None, w.cuda(), eps=1e-6, fmt=fmt)
    i8.sync_check()
    _compare(r, x, None, w, 1e-6, fmt)


def test_zero_rows_and_eps_zero():
    x = torch.zeros(4, 64).bfloat16()
    x[2, 5] = 3.0
    for eps in (0.0, 1e-6, 1.0):
        q, s, h = i8.add_rmsnorm_quant_act_pertoken(x.cuda(), torch.zeros_like(x).cuda(), eps=eps)
        i8.sync_check()
        assert torch.equal(s.cpu()[[0, 1, 3]], torch.zeros(3)) and not q.cpu()[[0, 1, 3]].any()
        assert q.cpu()[2, 5] == 127 and torch.equal(h.cpu(), x)
        _compare((q, s, h), x, torch.zeros_like(x), None, eps, "int8")


def test_views_and_in_place():
    g = torch.Generator().manual_seed(9)
    wide = torch.randn(11, 3 * 256 + 16, generator=g).bfloat16()
    stream = torch.randn(11, 512, generator=g).bfloat16()
    w = torch.randn(256, generator=g).bfloat16()
    x, res = wide[:, 256:512], stream[:, 128:384]
    dw, ds = wide.cuda(), stream.cuda()
    r = i8.add_rmsnorm_quant_act_pertoken(dw[:, 256:512], ds[:, 128:384], w.cuda(), residual_out=ds[:, 128:384])
    i8.sync_check()
    assert r[2].data_ptr() == ds[:, 128:384].data_ptr()
    _compare(r, x, res, w, 1e-6, "int8")
    after = ds.cpu()
    assert torch.equal(after[:, :128], stream[:, :128]) and torch.equal(after[:, 384:], stream[:, 384:])
    dx = dw[:, 256:512].contiguous()                      # in place of x
    r = i8.add_rmsnorm_quant_act_pertoken(dx, res.contiguous().cuda(), w.cuda(), residual_out=dx)
    i8.sync_check()
    _compare(r, x, res, w, 1e-6, "int8")


def test_other_stream_and_graph():
    g = torch.Generator().manual_seed(4)
    x, res = (torch.randn(17, 1024, generator=g).bfloat16() for _ in range(2))
    dx, dr = x.cuda(), res.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r = i8.add_rmsnorm_quant_act_pertoken(dx, dr)
    side.synchronize()
    _compare(r, x, res, None, 1e-6, "int8")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = i8.add_rmsnorm_quant_act_pertoken(dx, dr)
    x2 = torch.randn(17, 1024, generator=g).bfloat16()
    dx.copy_(x2)
    graph.replay()
    i8.sync_check()
    _compare(r, x2, res, None, 1e-6, "int8")


def test_empty():
    q, s, h = i8.add_rmsnorm_quant_act_pertoken(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"),
                                                torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0,) and h.shape == (0, 64)


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "f16codes"])
@pytest.mark.parametrize("K", [64, 3072, 32768])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_squares_outside_of_fp32(K, eps, fmt):
    """Rows whose squares (not the row or its norm) leave fp32: the result is
    the formula's.  Codes within half a step of y / s_a (E4M3: half a step of
    the code, or of the smallest one), s_a within 2^-19 of max|y| / L: the
    reduction's 2^-20 and the fp32 steps after it.  A scale below fp32's normal
    range is off by half its spacing, 2^-150."""
    g = torch.Generator().manual_seed(K)
    mags = torch.tensor([1e25, 3e37, 1.9e19, 1e19, 1e-12, 1e-23, 1e-30, 1e-38, 1e-40])
    x = (torch.randn(len(mags), K, generator=g).clamp(-8, 8) * mags[:, None]).bfloat16()
    x[0, 1:] *= 1e-12                                     # one element far above the others
    res = (torch.randn(len(mags), K, generator=g).clamp(-8, 8) * mags[:, None] * 0.5).bfloat16()
    w = (1 + 0.2 * torch.randn(K, generator=g)).bfloat16()
    q, s, h = i8.add_rmsnorm_quant_act_pertoken(x.cuda(), res.cuda(), w.cuda(), eps=eps, fmt=fmt)
    i8.sync_check()
    hh = x.double() + res.double()
    y = hh * w.double() / (hh.square().mean(1, keepdim=True) + eps).sqrt()
    limit = ref.LIMIT[fmt]
    want = y.abs().amax(1) / limit
    got = s.cpu().double()
    assert ((got - want).abs() <= 2.0 ** -19 * want + 2.0 ** -149).all()
    codes, ratio = _values(q), y / want[:, None]
    step = 0.5 if fmt != "e4m3" else (2.0 ** -4 * ratio.abs()).clamp(min=2.0 ** -10)
    assert ((codes - ratio).abs() <= step + 2.0 ** -18 * limit).all()
    assert torch.equal(h.cpu().view(torch.int16), (x.float() + res.float()).bfloat16().view(torch.int16))


def test_h_between_the_rows_of_the_inputs():
    """h in the columns beside x, in place of the residual, and over a single
    row with another stride: nothing of it lies over another row."""
    g = torch.Generator().manual_seed(12)
    both = torch.randn(9, 2 * 128, generator=g).bfloat16()
    res = torch.randn(9, 128, generator=g).bfloat16()
    d = both.cuda()
    r = i8.add_rmsnorm_quant_act_pertoken(d[:, :128], res.cuda(), residual_out=d[:, 128:])
    i8.sync_check()
    _compare(r, both[:, :128], res, None, 1e-6, "int8")
    assert torch.equal(d[:, :128].cpu(), both[:, :128])
    one = both[:1].cuda()
    r = i8.add_rmsnorm_quant_act_pertoken(one[:, :128], res[:1].cuda(), residual_out=one[:, :128])
    i8.sync_check()
    _compare(r, both[:1, :128], res[:1], None, 1e-6, "int8")
    with pytest.raises(i8.I8Error) as e:
        i8.add_rmsnorm_quant_act_pertoken(d[:8, :128], res[:8].cuda(), residual_out=d[1:, :128])
    assert e.value.status == 1
