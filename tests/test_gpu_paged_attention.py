"""paged_attention against the formula in 64 bits, within bounds that count
its roundings (tests/_serving.py)."""
import random

import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from tests import _serving as ref

pytestmark = pytest.mark.gpu


def _state(lens, news, block, Hq, Hkv, D, fmt, seed, spread=1.0, extra_cols=1):
    """A cache whose blocks outside the requests hold NaN scales and, like the
    ends of the last blocks, any codes at all (NaN codes of E4M3 among them)."""
    g, rng = torch.Generator().manual_seed(seed), random.Random(seed)
    need = [max(0, -(-n // block)) for n in lens]
    P = sum(need) + 3
    ids = list(range(P))
    rng.shuffle(ids)
    width = max(need + [0]) + extra_cols
    table = [[ids.pop() for _ in range(n)] + [10 ** 8] * (width - n) for n in need]
    code, scale = {}, {}
    for name in "kv":
        bits = torch.randint(0, 256, (P, Hkv, block, D), generator=g, dtype=torch.int32).to(torch.uint8)
        clean = bits.clone()
        if fmt == "e4m3":
            clean[(clean & 0x7F) == 0x7F] = 0x30
            # mostly moderate values, so that no block is all about its loudest codes
            clean = torch.where(torch.rand(clean.shape, generator=g) < 0.9, clean & 0xBF, clean)
        for r, n in enumerate(lens):
            for t0 in range(0, n, block):
                m = min(block, n - t0)
                bits[table[r][t0 // block], :, :m] = clean[table[r][t0 // block], :, :m]
        code[name] = bits
        s = torch.full((P, Hkv), float("nan"))
        for r, n in enumerate(need):
            s[table[r][:n]] = (torch.rand(n, Hkv, generator=g) + 0.1) * (0.02 if fmt == "int8" else 0.01) * spread
        scale[name] = s
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    q = (torch.randn(cu[-1], Hq, D, generator=g) * 1.5).bfloat16()
    return dict(q=q, code=code, scale=scale, table=table, lens=lens, cu=cu, fmt=fmt, width=width)


def _cache(st):
    dt = torch.int8 if st["fmt"] == "int8" else torch.float8_e4m3fn
    c = {n: st["code"][n].cuda().view(dt) for n in "kv"}
    return i8.QuantKVCache(c["k"], c["v"], st["scale"]["k"].cuda(), st["scale"]["v"].cuda())


def _table(st):
    return torch.tensor(st["table"], dtype=torch.int32).reshape(len(st["lens"]), st["width"]).cuda()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _expect(st, scale):
    dt = torch.int8 if st["fmt"] == "int8" else torch.float8_e4m3fn
    k, v = (st["code"][n].cuda().view(dt).float().double() for n in "kv")
    return ref.attention_reference(st["q"].cuda(), k, v, st["scale"]["k"].cuda(), st["scale"]["v"].cuda(), st["table"],
                                   st["lens"], st["cu"], scale)


def _check(st, out, lse, scale=None):
    D = st["q"].shape[2]
    o, l, bound, lse_bound = _expect(st, D ** -0.5 if scale is None else scale)
    err = (out.double() - o).abs()
    assert (err <= bound).all(), f"worst {float((err - bound).max()):.3g} over the bound, error {float(err.max()):.3g}"
    empty = torch.isinf(l)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    assert (out[empty] == 0).all()
    assert ((lse.double() - l).abs()[~empty] <= lse_bound[~empty]).all()


def _run(st, max_new=None, **kw):
    out, lse = i8.paged_attention(st["q"].cuda(), _cache(st), _table(st), _i32(st["lens"]), _i32(st["cu"]),
                                  max_new=max_new, want_lse=True, **kw)
    i8.sync_check()
    return out, lse


SHAPES = [(1, 1, 64), (8, 1, 128), (24, 8, 128), (16, 16, 64), (10, 2, 256), (32, 2, 128), (9, 3, 64), (20, 1, 256)]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D", SHAPES)
def test_decode(Hq, Hkv, D, fmt):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500, 1030]
    st = _state(lens, [1] * len(lens), 16, Hq, Hkv, D, fmt, 1)
    _check(st, *_run(st, max_new=1))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("block", [16, 48, 128])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 4, 64), (6, 2, 128), (5, 1, 128), (4, 4, 256)])
def test_several_new_tokens(Hq, Hkv, D, block, fmt):
    lens, news = [9, 40, 200, 7, 130, 65, 3], [2, 5, 8, 7, 1, 33, 3]
    st = _state(lens, news, block, Hq, Hkv, D, fmt, 2)
    _check(st, *_run(st, max_new=33))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (3, 1, 64), (4, 2, 256)])
def test_chunks(Hq, Hkv, D, fmt):
    lens, news = [300, 257, 64, 700], [300, 129, 63, 200]
    st = _state(lens, news, 32, Hq, Hkv, D, fmt, 3)
    _check(st, *_run(st))


@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (16, 4), (32, 2)])
def test_long_context(Hq, Hkv):
    st = _state([20001, 4097, 16], [1, 1, 1], 64, Hq, Hkv, 128, "int8", 4)
    _check(st, *_run(st, max_new=1))


def test_empty_requests_and_rows():
    """No new tokens, no tokens at all, and more new tokens than the sequence
    holds (rows that see nothing)."""
    st = _state([50, 0, 3, 20, 0], [0, 2, 5, 1, 0], 16, 6, 2, 64, "int8", 5)
    out, lse = _run(st, max_new=5)
    _check(st, out, lse)
    assert torch.isinf(lse[:2]).all() and torch.isinf(lse[2:4]).all() and not torch.isinf(lse[4:]).any()


def test_zero_blocks_and_uneven_scales():
    """Blocks of zeros (scale 0), and scales that differ by a factor of 10^6
    between blocks, louder ones first and last."""
    st = _state([160, 160], [1, 3], 16, 4, 2, 128, "int8", 6)
    for r in range(2):
        for i, b in enumerate(st["table"][r][:10]):
            f = [1e3, 1.0, 0.0, 1e-3, 1.0, 1e-3, 0.0, 1.0, 30.0, 1e3][i if r else 9 - i]
            st["scale"]["v"][b] *= f
            if f == 0.0:
                st["code"]["v"][b] = 0
                st["code"]["k"][b] = 0
                st["scale"]["k"][b] = 0.0
    _check(st, *_run(st, max_new=3))


@pytest.mark.parametrize("spread,factor", [(1e-20, 1.0), (1e4, 1.0), (1.0, 1e-30), (1.0, 1e30), (1.0, 0.0)])
def test_far_magnitudes_of_q_and_cache(spread, factor):
    st = _state([100, 33], [1, 2], 16, 4, 2, 64, "e4m3", 7, spread=spread)
    st["q"] = (st["q"].float() * factor).bfloat16()
    scale = 0.125 / spread / (factor or 1.0)
    if not 1e-37 < scale < 1e37:
        pytest.skip("the scale leaves fp32")
    _check(st, *_run(st, max_new=2, scale=scale), scale=scale)


def test_strides_and_padding_rows():
    """q a view of a fused projection, out a view of a wider buffer, the table
    a view of a wider one; rows past the requests are not written."""
    st = _state([40, 90], [3, 2], 16, 6, 2, 64, "int8", 8)
    wide = torch.zeros(7, 10 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    q = wide[:, 8:8 + 6 * 64].unflatten(1, (6, 64))
    q[:5] = st["q"].cuda()
    buf = torch.full((7, 8, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    tab = torch.full((2, st["width"] + 5), -1, dtype=torch.int32, device="cuda")
    tab[:, : st["width"]] = _table(st)
    out, lse = i8.paged_attention(q, _cache(st), tab[:, : st["width"]], _i32(st["lens"]), _i32(st["cu"]), max_new=3,
                                  want_lse=True, out=buf[:, 1:7])
    i8.sync_check()
    _check(st, out[:5], lse[:5])
    assert (buf[:, 0] == 5).all() and (buf[:, 7] == 5).all() and (buf[5:] == 5).all()


def test_one_head_order_and_repeatability():
    st = _state([3000, 77, 1500], [1, 1, 1], 16, 16, 2, 128, "int8", 9)
    a, la = _run(st, max_new=1)
    for _ in range(3):
        b, lb = _run(st, max_new=1)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_other_stream_and_graph():
    st = _state([900, 17], [1, 1], 16, 8, 2, 128, "e4m3", 10)
    cache, tab, lens, cu, q = _cache(st), _table(st), _i32(st["lens"]), _i32(st["cu"]), st["q"].cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, lse = i8.paged_attention(q, cache, tab, lens, cu, max_new=1, want_lse=True)
    side.synchronize()
    _check(st, out, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = i8.paged_attention(q, cache, tab, lens, cu, max_new=1, want_lse=True)
    st["lens"] = [333, 16]
    lens.copy_(_i32(st["lens"]))
    graph.replay()
    i8.sync_check()
    _check(st, out, lse)


def test_missing_blocks_are_left_out_and_reported():
    """Ids below 0 or past the pool inside a request: those tokens count as
    absent, the rest is right, and sync_check says so."""
    st = _state([100, 40], [1, 2], 16, 4, 2, 64, "int8", 11)
    st["table"][0][2], st["table"][0][6], st["table"][1][0] = -1, 10 ** 6, -2 ** 31
    out, lse = i8.paged_attention(st["q"].cuda(), _cache(st), _table(st), _i32(st["lens"]), _i32(st["cu"]), max_new=2,
                                  want_lse=True)
    with pytest.raises(i8.I8Error) as e:
        i8.sync_check()
    assert e.value.status == 7
    _check(st, out, lse)


def test_lengths_out_of_range_are_reported():
    """A sequence longer than its table, offsets past q, and more new tokens
    than max_new."""
    st = _state([40, 40], [1, 1], 16, 4, 2, 64, "int8", 12, extra_cols=0)
    args = (st["q"].cuda(), _cache(st), _table(st))
    for lens, cu in (([1000, 40], [0, 1, 2]), ([40, 40], [0, 1, 7]), ([40, 40], [-1, 0, 2]), ([40, 40], [0, 2, 2])):
        out = i8.paged_attention(*args, _i32(lens), _i32(cu), max_new=1)
        with pytest.raises(i8.I8Error) as e:
            i8.sync_check()
        assert e.value.status == 7, (lens, cu)
        assert torch.isfinite(out[:0].float()).all()
    _check(st, *_run(st, max_new=1))                       # the context is as good as before


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,news,heads", [
    ([5000], [30], (4, 1)),                       # a few rows, a long context: one item over all SMs
    ([129, 1, 4000, 260], [129, 1, 200, 33], (8, 2)),   # some requests by either kernel
    ([0, 50, 700], [100, 97, 96], (1, 1)),        # rows that see nothing, odd counts
    ([256, 128, 385], [256, 128, 385], (3, 3)),   # whole prompts that end on and past a tile
])
def test_many_rows(lens, news, heads, D, fmt):
    st = _state(lens, news, 48 if D == 64 else 64, *heads, D, fmt, 21)
    out, lse = _run(st)
    _check(st, out, lse)
    again, _ = _run(st)
    assert torch.equal(out, again)


def test_many_rows_zero_and_uneven_blocks():
    st = _state([700, 300], [200, 300], 16, 4, 2, 128, "int8", 22)
    for r, n in enumerate(st["lens"]):
        for i, b in enumerate(st["table"][r][: -(-n // 16)]):
            f = [1.0, 1e-3, 0.0, 1e2, 0.0, 1.0, 10.0][(i + r) % 7]
            st["scale"]["v"][b] *= f
            if f == 0.0:
                for c in "kv":
                    st["code"][c][b] = 0
                st["scale"]["k"][b] = 0.0
    _check(st, *_run(st))


@pytest.mark.parametrize("scale", [-0.1, 0.0, 3.0])
def test_many_rows_other_scales(scale):
    st = _state([400, 130], [120, 130], 32, 2, 1, 64, "e4m3", 23)
    _check(st, *_run(st, scale=scale), scale=scale)
    few = _state([400, 130], [1, 2], 32, 2, 1, 64, "e4m3", 23)
    _check(few, *_run(few, scale=scale), scale=scale)


@pytest.mark.parametrize("D", [64, 128])
def test_many_rows_missing_blocks(D):
    st = _state([500, 300], [150, 120], 16, 4, 2, D, "e4m3", 24)
    st["table"][0][3], st["table"][0][20], st["table"][1][0], st["table"][1][18] = -1, 10 ** 6, -7, 2 ** 31 - 1
    out, lse = i8.paged_attention(st["q"].cuda(), _cache(st), _table(st), _i32(st["lens"]), _i32(st["cu"]), want_lse=True)
    with pytest.raises(i8.I8Error) as e:
        i8.sync_check()
    assert e.value.status == 7
    _check(st, out, lse)


def test_many_rows_in_a_graph_and_on_another_stream():
    st = _state([300, 900], [150, 200], 64, 4, 2, 128, "int8", 25)
    cache, tab, lens, cu, q = _cache(st), _table(st), _i32(st["lens"]), _i32(st["cu"]), st["q"].cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, lse = i8.paged_attention(q, cache, tab, lens, cu, max_new=200, want_lse=True)
    side.synchronize()
    _check(st, out, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = i8.paged_attention(q, cache, tab, lens, cu, max_new=200, want_lse=True)
    st["lens"] = [260, 640]
    lens.copy_(_i32(st["lens"]))
    graph.replay()
    i8.sync_check()
    _check(st, out, lse)


def test_workspace_of_the_caller():
    st = _state([300, 40], [100, 1], 16, 4, 2, 128, "int8", 26)
    cache = _cache(st)
    need = i8.paged_attention_workspace_bytes(4, cache, 100)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    _check(st, *_run(st, max_new=100, workspace=ws))
    with pytest.raises(i8.I8Error) as e:
        _run(st, max_new=100, workspace=ws[: need - 16])
    assert e.value.status == 4
