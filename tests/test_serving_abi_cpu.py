"""Refusals of the serving operators, on the host and without a GPU: argument,
size and alignment errors come back before anything is queued."""
import ctypes

import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from w8a8_int8_quantized_i8_gb300 import binding

P = ctypes.c_void_p
OK = P(0x10000)


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def test_norm_refusals(lib):
    f = lib.i8_add_rmsnorm_quant_act_pertoken

    def call(x=OK, M=4, K=64, ldx=64, r=OK, ldr=64, w=OK, eps=1e-6, fmt=0, q=OK, ldq=64, s=OK, h=OK, ldh=64):
        return f(x, M, K, ldx, r, ldr, w, eps, fmt, q, ldq, s, h, ldh, None)

    assert call(M=0) == 0 and call(M=0, r=None, w=None, h=None, ldr=0, ldh=0) == 0
    for bad in (dict(M=-1), dict(K=0), dict(ldx=32), dict(ldr=32), dict(ldh=32), dict(ldq=32), dict(fmt=3),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(q=None), dict(s=None)):
        assert call(**bad) == 1, bad
    for bad in (dict(K=40, ldx=40, ldr=40, ldq=48, ldh=40), dict(K=32784, ldx=32784, ldr=32784, ldq=32784, ldh=32784),
                dict(M=2 ** 31)):
        assert call(**bad) == 3, bad
    odd = P(0x10008)
    for bad in (dict(x=odd), dict(r=odd), dict(w=odd), dict(h=odd), dict(q=odd), dict(s=P(0x10002)), dict(ldx=68),
                dict(ldr=68), dict(ldh=68), dict(ldq=72), dict(ldq=68, fmt=2)):
        assert call(**bad) == 2, bad


def test_tables_refusals(lib):
    f = lib.i8_build_block_tables

    def call(c=OK, n=OK, R=2, t=OK, width=4, ld=4, free=OK, n_free=8, taken=None, B=16, T=8, cu=OK, sl=OK, slots=OK,
             pos=OK, counts=OK):
        return f(c, n, R, t, width, ld, free, n_free, taken, B, T, cu, sl, slots, pos, counts, None)

    for bad in (dict(R=-1), dict(width=-1), dict(ld=3), dict(n_free=-1), dict(B=0), dict(T=-1), dict(c=None), dict(n=None),
                dict(t=None), dict(free=None), dict(cu=None), dict(sl=None), dict(slots=None), dict(pos=None),
                dict(counts=None)):
        assert call(**bad) == 1, bad
    for bad in (dict(R=16385), dict(B=1025), dict(T=2 ** 31), dict(width=2 ** 27, ld=2 ** 27), dict(n_free=2 ** 31)):
        assert call(**bad) == 3, bad
    for bad in (dict(c=P(0x10002)), dict(slots=P(0x10004)), dict(taken=P(0x10001)), dict(counts=P(0x10002))):
        assert call(**bad) == 2, bad


def _info(**kw):
    d = dict(k=0x10000, v=0x10000, k_scale=0x10000, v_scale=0x10000, blocks=4, block_size=16, kv_heads=2, head_dim=64, fmt=0)
    d.update(kw)
    return binding.KVCacheInfo(**d)


CACHE_REFUSALS = [(dict(k=None), 1), (dict(v_scale=None), 1), (dict(blocks=-1), 1), (dict(block_size=0), 1),
                  (dict(kv_heads=0), 1), (dict(head_dim=0), 1), (dict(fmt=2), 1), (dict(block_size=24), 3),
                  (dict(block_size=1040), 3), (dict(head_dim=80), 3), (dict(kv_heads=32768), 3), (dict(blocks=2 ** 31), 3),
                  (dict(k=0x10008), 2), (dict(v=0x10004), 2), (dict(k_scale=0x10002), 2)]


def test_append_refusals(lib):
    f = lib.i8_kv_cache_append

    def call(info=None, k=OK, kt=128, kh=64, v=OK, vt=128, vh=64, slots=OK, T=4):
        return f(k, kt, kh, v, vt, vh, slots, T, ctypes.byref(info or _info()), None)

    assert call(T=0) == 0 and call(info=_info(blocks=0, k=None, v=None, k_scale=None, v_scale=None)) == 0
    assert f(OK, 128, 64, OK, 128, 64, OK, 4, None, None) == 1
    for kw, code in CACHE_REFUSALS:
        assert call(info=_info(**kw)) == code, kw
    for bad in (dict(T=-1), dict(k=None), dict(v=None), dict(slots=None), dict(kt=-128), dict(vh=-64)):
        assert call(**bad) == 1, bad
    assert call(T=2 ** 31) == 3
    for bad in (dict(k=P(0x10008)), dict(v=P(0x10002)), dict(slots=P(0x10004)), dict(kt=130), dict(vh=68)):
        assert call(**bad) == 2, bad


def test_attention_refusals(lib):
    f = lib.i8_paged_attention

    def call(info=None, q=OK, qt=256, qh=64, T=2, Hq=4, table=OK, width=4, ld=4, lens=OK, cu=OK, R=2, max_new=1, scale=0.1,
             out=OK, ot=256, oh=64, lse=None, ws=OK, wsb=1 << 30):
        return f(q, qt, qh, T, Hq, ctypes.byref(info or _info()), table, width, ld, lens, cu, R, max_new, scale, out, ot, oh,
                 lse, ws, wsb, None)

    assert call(T=0) == 0 and call(R=0) == 0 and call(max_new=0) == 0
    for kw, code in CACHE_REFUSALS:
        assert call(info=_info(**kw)) == code, kw
    for bad in (dict(T=-1), dict(R=-1), dict(width=-1), dict(ld=3), dict(max_new=-1), dict(Hq=0), dict(Hq=3), dict(q=None),
                dict(out=None), dict(lens=None), dict(cu=None), dict(table=None), dict(qt=-8), dict(oh=-8),
                dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**bad) == 1, bad
    for bad in (dict(T=2 ** 31), dict(width=2 ** 27, ld=2 ** 27), dict(Hq=65538)):
        assert call(**bad) == 3, bad
    for bad in (dict(q=P(0x10008)), dict(out=P(0x10002)), dict(qt=260), dict(oh=68), dict(table=P(0x10002)),
                dict(lens=P(0x10001)), dict(cu=P(0x10003)), dict(lse=P(0x10002))):
        assert call(**bad) == 2, bad


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        i8.add_rmsnorm_quant_act_pertoken(x)
    with pytest.raises(ValueError):
        i8.add_rmsnorm_quant_act_pertoken(x, fmt="fp4")
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        i8.build_block_tables(i32, i32, torch.zeros(2, 3, dtype=torch.int32), i32, 16, 8)
    with pytest.raises(ValueError):
        i8.QuantKVCache.empty(2, 1, 16, 64, fmt="f16codes", device="cpu")
    cache = i8.QuantKVCache.empty(2, 1, 16, 64, device="cpu")
    assert cache.block_size == 16 and cache.k.dtype == torch.int8
    k = torch.zeros(3, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        i8.kv_cache_append(k, k, torch.zeros(3, dtype=torch.int64), cache)
    with pytest.raises(ValueError):
        i8.paged_attention(k, cache, torch.zeros(2, 3, dtype=torch.int32), i32, torch.zeros(3, dtype=torch.int32))
