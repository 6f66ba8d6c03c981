"""Refusals of the 4-bit route and of the heads' rotation, on the host and without a
GPU: argument, size, alignment and overlap errors come back before anything is
queued (the addresses are no memory)."""
import ctypes

import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from w8a8_int8_quantized_i8_gb300 import binding

P = ctypes.c_void_p
FAR = 1 << 28                       # operands lie this far apart
AT = {name: (i + 1) * FAR for i, name in enumerate(
    ["x", "codes", "scales", "rows", "residual", "weight", "h", "y", "w", "ws", "u", "us", "bias", "q", "k", "qo", "ko",
     "pos", "freq", "work"])}


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def _p(v):
    return None if v is None else P(v)


def test_scale_bytes(lib):
    f = lib.i8_fp4_block_scale_bytes
    assert f(1, 32, 0) == 2048 and f(128, 256, 1) == 1024 and f(129, 288, 0) == 4 * 2048 and f(0, 32, 0) == 0
    for bad in ((-1, 32, 0), (1, 0, 0), (1, 48, 0), (1, 131104, 0), (1, 32, 2), (2 ** 31, 32, 0)):
        assert f(*bad) == 0


def _quant(lib, rows=4, K=64, ldx=64, fmt=0, **at):
    a = {**AT, **at}
    return lib.i8_quant_rows_fp4(_p(a["x"]), rows, K, ldx, fmt, _p(a["codes"]), _p(a["scales"]), _p(a["rows"]), None)


def _norm(lib, M=4, K=64, ldx=64, ldr=64, eps=1e-6, fmt=0, ldh=64, **at):
    a = {**AT, **at}
    return lib.i8_add_rmsnorm_quant_fp4(_p(a["x"]), M, K, ldx, _p(a["residual"]), ldr, _p(a["weight"]), eps, fmt,
                                        _p(a["codes"]), _p(a["scales"]), _p(a["rows"]), _p(a["h"]), ldh, None)


SIZES = [(dict(K=0), 1), (dict(fmt=2), 1), (dict(fmt=-1), 1), (dict(ldx=32), 1), (dict(x=None), 1), (dict(codes=None), 1),
         (dict(scales=None), 1), (dict(rows_=None), 1), (dict(K=48, ldx=48), 3), (dict(K=131104, ldx=131104), 3),
         (dict(x=AT["x"] + 8), 2), (dict(codes=AT["codes"] + 8), 2), (dict(scales=AT["scales"] + 4), 2),
         (dict(rows_=AT["rows"] + 2), 2), (dict(ldx=68), 2)]


@pytest.mark.parametrize("bad,want", SIZES + [(dict(rows=-1), 1), (dict(rows=2 ** 31), 3)])
def test_quant_refusals(lib, bad, want):
    bad = dict(bad)
    if "rows_" in bad:      # the row scales' address
        at = bad.pop("rows_")
        assert lib.i8_quant_rows_fp4(_p(AT["x"]), 4, 64, 64, 0, _p(AT["codes"]), _p(AT["scales"]), _p(at), None) == want
        return
    assert _quant(lib, **bad) == want


def test_quant_of_no_rows(lib):
    assert _quant(lib, rows=0) == 0 and _quant(lib, rows=0, x=None, codes=None, scales=None) == 0


@pytest.mark.parametrize("bad,want", [(b, w) for b, w in SIZES if "rows_" not in b] + [
    (dict(M=-1), 1), (dict(ldr=32), 1), (dict(ldh=32), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1), (dict(rows=None), 1), (dict(rows=None, fmt=1), 1), (dict(M=2 ** 31), 3),
    (dict(residual=AT["residual"] + 8), 2), (dict(weight=AT["weight"] + 8), 2), (dict(h=AT["h"] + 8), 2),
    (dict(ldr=68), 2), (dict(ldh=68), 2), (dict(rows=AT["rows"] + 2), 2)])
def test_norm_refusals(lib, bad, want):
    assert _norm(lib, **bad) == want


# every pair of an output and another operand that would share memory
@pytest.mark.parametrize("a,b", [(a, b) for a in ("codes", "scales", "rows") for b in ("x", "codes", "scales", "rows") if a != b])
def test_quant_overlaps(lib, a, b):
    assert _quant(lib, **{a: AT[b]}) == 1


@pytest.mark.parametrize("a,b", [(a, b) for a in ("codes", "scales", "rows")
                                 for b in ("x", "residual", "weight", "h", "codes", "scales", "rows") if a != b]
                         + [("h", "weight")])
def test_norm_overlaps(lib, a, b):
    assert _norm(lib, **{a: AT[b]}) == 1


@pytest.mark.parametrize("h", [AT["x"] + 2 * 64, AT["residual"] - 2 * 64, AT["x"] + 32, AT["residual"] + 2 * 64 * 3])
def test_norm_h_over_other_rows(lib, h):
    assert _norm(lib, h=h) == 1


def _rows(codes="codes", scales="scales", rows="rows", n=4, K=64, fmt=0):
    at = lambda v: AT[v] if isinstance(v, str) else v  # noqa: E731
    return binding.FP4RowsInfo(at(codes), at(scales), at(rows), n, K, fmt)


W = dict(codes="w", scales="ws", rows=None, n=16)


def _gemm(lib, a=None, w=None, bias=AT["bias"], y=AT["y"], ldy=16):
    return lib.i8_gemm_fp4_bias_bf16(ctypes.byref(a or _rows()), ctypes.byref(w or _rows(**W)), _p(bias), _p(y), ldy, None)


def test_gemm_refusals(lib):
    assert _gemm(lib, a=_rows(n=0)) == 0 and _gemm(lib, w=_rows(**{**W, "n": 0})) == 0
    assert lib.i8_gemm_fp4_bias_bf16(None, ctypes.byref(_rows(**W)), None, _p(AT["y"]), 16, None) == 1
    assert lib.i8_gemm_fp4_bias_bf16(ctypes.byref(_rows()), None, None, _p(AT["y"]), 16, None) == 1
    for a in (_rows(n=-1), _rows(K=0), _rows(fmt=2), _rows(codes=None), _rows(scales=None), _rows(K=96), _rows(fmt=1)):
        assert _gemm(lib, a=a) == 1
    for kw, want in ((dict(y=None), 1), (dict(ldy=8), 1), (dict(y=AT["y"] + 8), 2), (dict(ldy=20), 2),
                     (dict(bias=AT["bias"] + 8), 2), (dict(a=_rows(codes=AT["codes"] + 8)), 2),
                     (dict(a=_rows(scales=AT["scales"] + 8)), 2), (dict(a=_rows(rows=AT["rows"] + 2)), 2),
                     (dict(w=_rows(**{**W, "n": 12})), 3), (dict(a=_rows(K=80)), 3)):
        assert _gemm(lib, **kw) == want, kw


@pytest.mark.parametrize("y", ["codes", "scales", "rows", "w", "ws", "bias"])
def test_gemm_overlaps(lib, y):
    assert _gemm(lib, y=AT[y]) == 1


def test_gated_refusals(lib):
    def call(gate=None, up=None, act=0, y=AT["y"], gb=None, ub=None, none=False):
        gate, up = gate or _rows(**W), up or _rows("u", "us", None, 16)
        return lib.i8_gemm_fp4_gated_bf16(ctypes.byref(_rows()), ctypes.byref(gate), None if none else ctypes.byref(up),
                                          _p(gb), _p(ub), act, _p(y), 16, None)

    assert call(none=True) == 1 and call(act=2) == 1 and call(act=-1) == 1
    for up in (_rows("u", "us", None, 24), _rows("u", "us", None, 16, K=96), _rows("u", "us", None, 16, fmt=1)):
        assert call(up=up) == 1
    for y in ("u", "us", "w", "ws", "codes"):
        assert call(y=AT[y]) == 1
    assert call(gb=AT["bias"], y=AT["bias"]) == 1 and call(ub=AT["bias"], y=AT["bias"]) == 1
    assert call(gb=AT["bias"] + 2) == 2 and call(ub=AT["bias"] + 2) == 2


def test_linear_refusals(lib):
    need = lib.i8_linear_fp4_workspace_bytes(4, 64, 0)
    assert need == 4 * 32 + 2048 + 16 and lib.i8_linear_fp4_workspace_bytes(4, 64, 1) == 4 * 32 + 1024
    assert lib.i8_linear_fp4_workspace_bytes(4, 40, 0) == 0

    def call(M=4, K=64, ldx=64, x=AT["x"], w=None, ws=AT["work"], size=need, y=AT["y"], bias=None):
        return lib.i8_linear_fp4(_p(x), M, K, ldx, ctypes.byref(w or _rows(**W)), _p(bias), _p(y), 16, _p(ws), size, None)

    assert call(M=0, size=0, ws=None) == 0
    for kw, want in ((dict(K=96, ldx=96), 1), (dict(M=-1), 1), (dict(ldx=32), 1), (dict(x=None), 1), (dict(ws=None), 4),
                     (dict(size=need - 1), 4), (dict(ws=AT["work"] + 8), 2), (dict(y=AT["work"]), 1),
                     (dict(ws=AT["w"]), 1), (dict(ws=AT["ws"]), 1), (dict(ws=AT["x"]), 1), (dict(y=AT["y"] + 8), 2),
                     (dict(bias=AT["work"]), 1), (dict(w=_rows(**{**W, "n": 12})), 3)):
        assert call(**kw) == want, kw


def _rotate(lib, T=4, Hq=2, Hk=1, D=64, R=64, axes=1, sections=(32,), eps=1e-6, ldp=4, q=AT["q"], k=AT["k"], qo=AT["qo"],
            ko=AT["ko"], pos=AT["pos"], freq=AT["freq"], qw=None, kw=None, lq=(128, 64), lk=(64, 64), lqo=(128, 64),
            lko=(64, 64)):
    s = (ctypes.c_int32 * 4)(*sections, *([0] * (4 - len(sections)))) if sections is not None else None
    return lib.i8_heads_rmsnorm_rotate(_p(q), *lq, Hq, _p(k), *lk, Hk, T, D, _p(qw), _p(kw), eps, _p(pos), ldp, axes, s,
                                       _p(freq), R, 0, _p(qo), *lqo, _p(ko), *lko, None)


def test_rotate_refusals(lib):
    assert _rotate(lib, T=0) == 0 and _rotate(lib, Hq=0, Hk=0) == 0
    for kw in (dict(T=-1), dict(D=0), dict(Hq=-1), dict(R=-16), dict(R=80, sections=(40,)), dict(axes=0), dict(axes=5),
               dict(sections=None), dict(sections=(31,)), dict(sections=(-1, 33), axes=2), dict(sections=(33,)), dict(eps=-1.0),
               dict(eps=float("nan")), dict(q=None), dict(ko=None), dict(pos=None), dict(freq=None), dict(lq=(-64, 64)),
               dict(axes=2, sections=(16, 16), ldp=3)):
        assert _rotate(lib, **kw) == 1, kw
    for kw in (dict(D=60, R=16, sections=(8,)), dict(D=520), dict(R=40, sections=(20,)), dict(T=2 ** 31), dict(Hq=32767)):
        assert _rotate(lib, **kw) == 3, kw
    for kw in (dict(q=AT["q"] + 8), dict(qo=AT["qo"] + 8), dict(qw=AT["weight"] + 8), dict(pos=AT["pos"] + 2),
               dict(freq=AT["freq"] + 2), dict(lq=(132, 64)), dict(lko=(64, 68))):
        assert _rotate(lib, **kw) == 2, kw


# q, k and v of one projection's output, 4 heads of 64 a token
FUSED = dict(q=AT["q"], lq=(256, 64), k=AT["q"] + 256, lk=(256, 64))


@pytest.mark.parametrize("kw", [
    dict(FUSED, qo=AT["q"], lqo=(256, 64), ko=AT["q"], lko=(256, 64)),                # both outputs in one place
    dict(FUSED, qo=AT["q"] + 128, lqo=(256, 64), ko=AT["ko"]),                        # q's output a head on
    dict(FUSED, qo=AT["q"] + 256, lqo=(256, 64), ko=AT["ko"]),                        # over k
    dict(FUSED, qo=AT["q"], lqo=(128, 64), ko=AT["ko"]),                              # its place, other strides
    dict(FUSED, qo=AT["q"] + 512, lqo=(256, 64), ko=AT["ko"]),                        # a token on
    dict(FUSED, qo=AT["qo"], ko=AT["q"] + 512 - 64, lko=(256, 64)),                   # k's output over the next q
    dict(FUSED, qo=AT["qo"], lqo=(64, 64), ko=AT["ko"]),                              # rows that share elements
    dict(FUSED, qo=AT["qo"], lqo=(128, 32), ko=AT["ko"]),
    dict(FUSED, qo=AT["pos"], ko=AT["ko"]), dict(FUSED, qo=AT["freq"], ko=AT["ko"]),
    dict(FUSED, qo=AT["qo"], ko=AT["weight"], kw=AT["weight"]), dict(FUSED, qo=AT["qo"], ko=AT["weight"] - 64, qw=AT["weight"])])
def test_rotate_overlaps(lib, kw):
    assert _rotate(lib, **kw) == 1, kw


def _cpu_rows(n=8, K=64, fmt="nvfp4"):
    return i8.FP4Rows.empty(n, K, fmt, "cpu")


def test_the_binding_s_refusals():
    x, r = torch.zeros(4, 64).bfloat16(), _cpu_rows()
    assert r.shape == (8, 64) and r.fmt == "nvfp4" and r.row_scales.shape == (8,)
    assert _cpu_rows(fmt="mxfp4").row_scales is None and _cpu_rows(129, 288, "mxfp4").block_scales.shape == (2, 2, 1024)
    assert i8.linear_fp4_workspace_bytes(4, r) == 4 * 32 + 2048 + 16
    for call in (lambda: i8.quant_rows_fp4(x), lambda: i8.add_rmsnorm_quant_fp4(x), lambda: i8.linear_fp4(x, r),
                 lambda: i8.gated_linear_fp4(x, r, r), lambda: i8.gemm_fp4_bias_bf16(r, r),
                 lambda: i8.gemm_fp4_gated_bf16(r, r, r), lambda: i8.heads_rmsnorm_rotate(x, x, x, x),
                 lambda: i8.quant_rows_fp4(x, "fp4"), lambda: i8.FP4Rows.empty(4, 64, "int4"),
                 lambda: i8.gated_linear_fp4(x, r, r, activation="relu"),
                 lambda: i8.gemm_fp4_gated_bf16(r, r, r, activation=None)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: i8.quant_rows_fp4(None), lambda: i8.linear_fp4(3, r), lambda: i8.gemm_fp4_bias_bf16(x, r),
                 lambda: i8.gemm_fp4_bias_bf16(tuple(r), r), lambda: i8.heads_rmsnorm_rotate(None, x, x, x)):
        with pytest.raises(TypeError):
            call()
