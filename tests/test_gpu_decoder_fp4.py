"""The decoder with 4-bit layers, head norms and rotation: the operators together.

Every stage of a step is compared with its definition in 64 bits on what the step
itself put into it: the projections and the gated MLP on their codes, the rotation
on the projection's output (the product gives the same bits again), the
attention on what the cache holds."""
import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from tests import _fp4
from tests import _serving as ref
from w8a8_int8_quantized_i8_gb300 import decoder

pytestmark = pytest.mark.gpu


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _rows(n, width, seed):
    return torch.randn(n, width, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def _shape(**kw):
    d = dict(blocks=2, width=512, q_heads=8, kv_heads=2, head_dim=64, mlp=1024, block_size=16, rope_theta=10000.0,
             head_norms=True)
    d.update(kw)
    return decoder.Shape(**d)


def _product(codes, lin):
    """(value in 64 bits, bound of the fp32 sum's error) of a layer on these codes."""
    a, w = _fp4.values(codes), _fp4.values(lin.wq)
    want, size = a @ w.T + lin.bias.double(), a.abs() @ w.abs().T + lin.bias.double().abs()
    return want, (a.shape[1] + 4) * 2.0 ** -24 * size


def _close(got, want, err):
    assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + err).all()


@pytest.mark.parametrize("fmt,cache_fmt,activation", [("nvfp4", "int8", "silu"), ("mxfp4", "e4m3", "gelu")])
def test_every_stage_of_a_step(fmt, cache_fmt, activation):
    shape = _shape(fmt=fmt, cache_fmt=cache_fmt, activation=activation)
    model = decoder.Decoder(shape, 60)
    reqs = decoder.Requests(3, 26, 60, shape.block_size)
    for step, lens in enumerate([[70, 1, 33], [1, 1, 1], [5, 40, 0], [100, 1, 1], [200, 100, 90]]):
        seen = {}
        plan = reqs.plan(_ints(lens), sum(lens))
        y = model.step(_rows(sum(lens), shape.width, step), plan, reqs.block_tables, max(lens),
                       record=lambda b, name, t: seen.__setitem__((b, name), t))
        i8.sync_check()
        assert torch.isfinite(y).all()
        for b, layers in enumerate(model.layers):
            q, k, v, o = seen[b, "attention"]
            (codes,) = seen[b, "qkv"]
            want, err = _product(codes, layers["qkv"])
            qkv = i8.gemm_fp4_bias_bf16(codes, layers["qkv"].wq, layers["qkv"].bias)
            _close(qkv, want, err)
            heads = qkv.unflatten(1, (12, 64)).double()
            assert torch.equal(heads[:, 10:], v.double())
            turn = plan.positions.double()[:, None] * model.inv_freq.double()
            for x, got, weight in ((heads[:, :8], q, layers["head_norms"][0]), (heads[:, 8:10], k, layers["head_norms"][1])):
                x = x / (x.square().mean(2, keepdim=True) + 1e-6).sqrt() * weight.double()
                one, two = x[:, :, :32], x[:, :, 32:]
                c, s = turn.cos()[:, None], turn.sin()[:, None]
                # (angles to 2 pi 2^-24, the norm and the products to a few 2^-24: of the pair's size)
                size = 40 * 2.0 ** -24 * (one.abs() + two.abs()).repeat(1, 1, 2)
                _close(got, torch.cat((one * c - two * s, two * c + one * s), 2), size)
            cache = model.caches[b]
            want, _, bound, _ = ref.attention_reference(q, cache.k.float().double(), cache.v.float().double(),
                                                        cache.k_scale, cache.v_scale, reqs.block_tables.tolist(),
                                                        plan.seq_lens.tolist(), plan.cu_new.tolist(), shape.head_dim ** -0.5)
            assert ((o.double() - want).abs() <= bound).all()
            o, x = seen[b, "out"]
            _close(x, *_product(i8.quant_rows_fp4(o.flatten(1), fmt), layers["out"]))
            codes, u, x = seen[b, "mlp"]
            (g, eg), (up, eu) = _product(codes[0], layers["gate"]), _product(codes[0], layers["up"])
            act = torch.nn.functional.silu(g) if activation == "silu" else torch.nn.functional.gelu(g)
            # both activations change by at most 1.13 times their argument's change
            _close(u, act * up, 1.13 * eg * (up.abs() + eu) + act.abs() * eu + 2.0 ** -18 * (act * up).abs() + 1e-12)
            _close(x, *_product(i8.quant_rows_fp4(u, fmt), layers["down"]))


@pytest.mark.parametrize("fmt", ["nvfp4", "int8"])
def test_a_step_in_a_graph(fmt):
    """A decode step captured once and replayed, lengths and tables kept on the
    device, equals the same steps run one by one."""
    shape = _shape(blocks=1, fmt=fmt)
    results = []
    for graphed in (False, True):
        model = decoder.Decoder(shape, 12)
        reqs = decoder.Requests(2, 6, 12, shape.block_size)
        model.step(_rows(20, shape.width, 1), reqs.plan(_ints([13, 7]), 20), reqs.block_tables, 13)
        x, new = torch.zeros(2, shape.width, dtype=torch.bfloat16, device="cuda"), _ints([1, 1])
        if graphed:
            live = [reqs.context_lens, reqs.taken, reqs.block_tables, *(t for c in model.caches for t in c)]
            kept = [t.clone() for t in live]
            model.step(x, reqs.plan(new, 2), reqs.block_tables, 1)   # tables of the GELU are built outside of a capture
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                y = model.step(x, reqs.plan(new, 2), reqs.block_tables, 1)
            for t, saved in zip(live, kept):
                t.copy_(saved)
        out = []
        for i in range(5):
            x.copy_(_rows(2, shape.width, 100 + i))
            if graphed:
                graph.replay()
            else:
                y = model.step(x, reqs.plan(new, 2), reqs.block_tables, 1)
            out.append(y.clone())
        i8.sync_check()
        results.append(torch.stack(out))
    assert torch.equal(results[0], results[1])


@pytest.mark.parametrize("fmt", ["mxfp4", "int8"])
def test_positions_are_the_requests_own(fmt):
    """The same tokens in one request and, behind another request's, in a batch: their keys' rotation goes by
    their own positions, so the projections, rotated, agree bit for bit (a row's product does not depend on the
    other rows of a tile)."""
    shape = _shape(blocks=1, fmt=fmt)
    model, x = decoder.Decoder(shape, 20), _rows(40, shape.width, 3)
    keys = []
    for lens, first in (([40], 0), ([9, 40], 9)):
        reqs = decoder.Requests(len(lens), 4, 20, shape.block_size)
        seen = {}
        rows = x if first == 0 else torch.cat((_rows(9, shape.width, 4), x))
        model.step(rows, reqs.plan(_ints(lens), sum(lens)), reqs.block_tables, max(lens),
                   record=lambda b, name, t: seen.__setitem__(name, t))
        q, k, _, _ = seen["attention"]
        keys.append(torch.cat((q, k), 1)[first:].clone())
    assert torch.equal(keys[0], keys[1])
