"""The decoder stack: the serving operators and the W8A8 layer together.

Prompts, a chunk of a prompt and single tokens run through the same caches.
Every block's attention is checked against the formula over what the cache then
holds, the cache against the keys and values that went in (a coded value is off
by at most half a code of its block's scale, and a re-coding adds at most half
a code each time), and a decode step after a prompt against the prompt's last
token when it comes at once.
"""
import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from tests import _serving as ref
from w8a8_int8_quantized_i8_gb300 import decoder

pytestmark = pytest.mark.gpu


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _shape(**kw):
    d = dict(blocks=2, width=512, q_heads=8, kv_heads=2, head_dim=64, mlp=1024, block_size=16)
    d.update(kw)
    return decoder.Shape(**d)


def _rows(n, width, seed):
    return torch.randn(n, width, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


@pytest.mark.parametrize("fmt,cache_fmt,head_dim", [("int8", "int8", 64), ("e4m3", "e4m3", 64), ("int8", "e4m3", 128)])
def test_steps_of_mixed_requests(fmt, cache_fmt, head_dim):
    shape = _shape(fmt=fmt, cache_fmt=cache_fmt, head_dim=head_dim)
    pool = 40
    model = decoder.Decoder(shape, pool)
    reqs = decoder.Requests(3, 14, pool, shape.block_size)
    held = [[], [], []]                               # block 0's keys of each request, as they went in
    for step, lens in enumerate([[70, 1, 33], [1, 1, 1], [5, 40, 0], [1, 1, 1], [100, 1, 1]]):
        seen = {}
        plan = reqs.plan(_ints(lens), sum(lens))
        x = _rows(sum(lens), shape.width, step)
        y = model.step(x, plan, reqs.block_tables, max(lens), record=lambda b, name, t: seen.setdefault(b, t))
        i8.sync_check()
        assert plan.counts.tolist()[2] == 0 and torch.isfinite(y).all() and y.shape == x.shape
        total, cu = plan.seq_lens.tolist(), plan.cu_new.tolist()
        for b, (q, k, v, o) in seen.items():
            cache = model.caches[b]
            want, _, bound, _ = ref.attention_reference(q, cache.k.float().double(), cache.v.float().double(),
                                                        cache.k_scale, cache.v_scale, reqs.block_tables.tolist(), total,
                                                        cu, shape.head_dim ** -0.5)
            assert ((o.double() - want).abs() <= bound).all(), (step, b)
        k = seen[0][1].float()
        for r in range(3):
            held[r].append(k[cu[r]:cu[r + 1]])
    cache, tables = model.caches[0], reqs.block_tables.long()
    limit = ref.LIMIT[cache_fmt]
    for r in range(3):
        put = torch.cat(held[r])
        ids = tables[r, torch.arange(len(put), device="cuda") // shape.block_size]
        at = torch.arange(len(put), device="cuda") % shape.block_size
        scale = cache.k_scale[ids]
        got = cache.k[ids, :, at].float() * scale[..., None] if cache_fmt == "int8" else \
            cache.k.view(torch.uint8)[ids, :, at].view(torch.float8_e4m3fn).float() * scale[..., None]
        # half a step of the value's code, once when written and once for each of
        # the 15 tokens after it that may have raised the block's scale
        step_size = 0.5 if cache_fmt == "int8" else 2.0 ** -4 * (put.abs() / scale[..., None]).clamp(min=2.0 ** -6)
        assert ((got - put).abs() <= 16 * step_size * scale[..., None] * 1.001).all()
        assert scale.max() <= put.abs().max() / limit * 1.001


def test_a_decode_step_is_the_prompt_s_last_token():
    """The same tokens as one prompt of 48 and as a prompt of 47 and one token:
    the cache's codes differ at most by the last block's re-coding, so the last
    rows agree closely (their cosine is above 0.99)."""
    shape = _shape(blocks=1)
    x = _rows(48, shape.width, 3)
    rows = []
    for parts in ([48], [47, 1], [16, 31, 1]):
        model = decoder.Decoder(shape, 4)
        reqs = decoder.Requests(1, 4, 4, shape.block_size)
        at = 0
        for n in parts:
            y = model.step(x[at:at + n], reqs.plan(_ints([n]), n), reqs.block_tables, n)
            at += n
        i8.sync_check()
        rows.append(y[-1].double())
    for other in rows[1:]:
        assert torch.nn.functional.cosine_similarity(rows[0], other, dim=0) > 0.99


def test_a_step_in_a_graph():
    """A decode step captured once and replayed, lengths and tables kept on the
    device, equals the same steps run one by one."""
    shape = _shape(blocks=1)
    results = []
    for graphed in (False, True):
        model = decoder.Decoder(shape, 12)
        reqs = decoder.Requests(2, 6, 12, shape.block_size)
        model.step(_rows(20, shape.width, 1), reqs.plan(_ints([13, 7]), 20), reqs.block_tables, 13)
        x, new = torch.empty(2, shape.width, dtype=torch.bfloat16, device="cuda"), _ints([1, 1])
        keep = (reqs.context_lens.clone(), reqs.taken.clone(), reqs.block_tables.clone())
        caches = [tuple(t.clone() for t in c) for c in model.caches]

        def step():
            return model.step(x, reqs.plan(new, 2), reqs.block_tables, 1)

        if graphed:
            x.copy_(_rows(2, shape.width, 50))
            step()                                    # tables of the GELU are built outside of a capture
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                y = step()
            for live, saved in zip((reqs.context_lens, reqs.taken, reqs.block_tables), keep):
                live.copy_(saved)
            for live, saved in zip(model.caches, caches):
                for a, b in zip(live, saved):
                    a.view(torch.uint8).copy_(b.view(torch.uint8)) if a.dtype != torch.float32 else a.copy_(b)
        out = []
        for i in range(5):
            x.copy_(_rows(2, shape.width, 100 + i))
            if graphed:
                graph.replay()
            else:
                y = step()
            out.append(y.clone())
        i8.sync_check()
        results.append(torch.stack(out))
    assert torch.equal(results[0], results[1])
