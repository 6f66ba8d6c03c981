"""A synthetic decoder stack on the W8A8 layer and the serving operators.

What runs at every step, for a batch of requests of any lengths (prompts,
chunks of prompts and single tokens mixed):

    block tables, slots, positions             build_block_tables, once a step
    per block:
      x + residual, RMS norm, 8-bit codes      add_rmsnorm_quant_act_pertoken
      QKV projection                           the fused W8A8 GEMM
      new keys and values into the cache       kv_cache_append
      causal attention over the cache          paged_attention
      out projection                           the W8A8 layer
      x + residual, RMS norm, 8-bit codes      add_rmsnorm_quant_act_pertoken
      MLP up, GELU + 8-bit codes, MLP down     the fused GEMMs, gelu_quant_act_pertoken

Weights are random (seeded), as in dit_stack; there is no position encoding, no
vocabulary and no sampling: a step takes the new tokens' hidden rows and gives
theirs back.  Nothing in a step waits for the device, so a step of fixed sizes
can be captured into a CUDA graph.
"""
from __future__ import annotations

import dataclasses

import torch

from . import binding as i8
from . import serving
from .dit_stack import Linear, layer_weight


@dataclasses.dataclass(frozen=True)
class Shape:
    """Sizes of a decoder; the defaults' width is the DiT workloads' (24 heads
    of 128)."""
    blocks: int = 2
    width: int = 3072
    q_heads: int = 24
    kv_heads: int = 8
    head_dim: int = 128
    mlp: int = 12288
    fmt: str = "int8"            # codes of activations and weights: int8 or e4m3
    cache_fmt: str = "int8"      # codes of the cache: int8 or e4m3
    block_size: int = 64


class Decoder:
    """Quantized weights of a decoder and one cache a block."""

    def __init__(self, shape: Shape, cache_blocks: int, seed: int = 7, device="cuda"):
        self.shape = shape
        s = shape
        qkv = (s.q_heads + 2 * s.kv_heads) * s.head_dim
        sizes = (("qkv", s.width, qkv), ("out", s.q_heads * s.head_dim, s.width), ("up", s.width, s.mlp),
                 ("down", s.mlp, s.width))
        quant = i8.quant_weight_perchannel_e4m3 if s.fmt == "e4m3" else i8.quant_weight_perchannel
        self.layers, self.caches = [], []
        for blk in range(s.blocks):
            layers = {}
            for li, (name, K, N) in enumerate(sizes):
                at = seed * 100003 + blk * 8 + li
                w, b = layer_weight(at, N, K, device)
                wq, s_w = quant(w)
                layers[name] = Linear(wq, s_w, b, at, s.fmt)
            g = torch.Generator(device=device).manual_seed(seed * 100003 + blk * 8 + 7)
            layers["norms"] = [(1 + 0.1 * torch.randn(s.width, generator=g, device=device)).bfloat16()
                               for _ in range(2)]
            self.layers.append(layers)
            self.caches.append(serving.QuantKVCache.empty(cache_blocks, s.kv_heads, s.block_size, s.head_dim,
                                                          s.cache_fmt, device))

    def _gemm(self, lin: Linear, codes, scale):
        fn = i8.gemm_e4m3_dequant_bias_bf16 if lin.fmt == "e4m3" else i8.gemm_dequant_bias_bf16
        return fn(codes, scale, lin.wq, lin.s_w, lin.bias)

    def step(self, x: torch.Tensor, plan: serving.BlockPlan, block_tables: torch.Tensor, max_new: int,
             record=None) -> torch.Tensor:
        """One step: x bf16 [T, width], the new tokens' rows in request order
        (T = the plan's slots).  ``max_new`` bounds the new tokens of a request.
        ``record(block, name, tensors)`` sees what goes in and out of the
        attention."""
        s = self.shape
        h = torch.zeros_like(x)          # the residual stream: x joins it in the first norm
        for blk, (layers, cache) in enumerate(zip(self.layers, self.caches)):
            codes, scale, h = serving.add_rmsnorm_quant_act_pertoken(x, h, layers["norms"][0], fmt=s.fmt,
                                                                     residual_out=h)
            qkv = self._gemm(layers["qkv"], codes, scale)
            heads = qkv.unflatten(1, (s.q_heads + 2 * s.kv_heads, s.head_dim))
            q, k, v = heads.split((s.q_heads, s.kv_heads, s.kv_heads), dim=1)
            serving.kv_cache_append(k, v, plan.slots, cache)
            o = serving.paged_attention(q, cache, block_tables, plan.seq_lens, plan.cu_new, max_new)
            if record:
                record(blk, "attention", (q, k, v, o))
            linear = i8.linear_e4m3 if s.fmt == "e4m3" else i8.linear
            x = linear(o.flatten(1), layers["out"].wq, layers["out"].s_w, layers["out"].bias)
            codes, scale, h = serving.add_rmsnorm_quant_act_pertoken(x, h, layers["norms"][1], fmt=s.fmt,
                                                                     residual_out=h)
            up = self._gemm(layers["up"], codes, scale)
            codes, scale = i8.gelu_quant_act_pertoken(up, fmt=s.fmt)
            x = self._gemm(layers["down"], codes, scale)
        return x + h


class Requests:
    """The block tables of a batch of requests over one pool of blocks, kept on
    the device from step to step."""

    def __init__(self, requests: int, max_blocks: int, pool: int, block_size: int, device="cuda"):
        def ints(*shape, fill=0):
            return torch.full(shape, fill, dtype=torch.int32, device=device)
        self.block_size = block_size
        self.context_lens, self.taken = ints(requests), ints(1)
        self.block_tables = ints(requests, max_blocks, fill=-1)
        self.free_blocks = torch.arange(pool, dtype=torch.int32, device=device)

    def plan(self, new_lens: torch.Tensor, tokens: int) -> serving.BlockPlan:
        """Blocks for a step of ``tokens`` tokens, new_lens (int32 [R]) of each
        request; afterwards the requests hold them."""
        plan = serving.build_block_tables(self.context_lens, new_lens, self.block_tables, self.free_blocks,
                                          self.block_size, tokens, taken=self.taken)
        self.context_lens.copy_(plan.seq_lens)
        self.taken.copy_(plan.counts[1:2])
        return plan


def main() -> None:
    """python -m w8a8_int8_quantized_i8_gb300.decoder: a prompt, a few single
    tokens, and how long a step of either takes."""
    shape = Shape()
    prompts, steps = [700, 64, 1, 333], 4
    need = sum(-(-(n + steps) // shape.block_size) for n in prompts)
    model = Decoder(shape, need)
    requests = Requests(len(prompts), -(-(max(prompts) + steps) // shape.block_size), need, shape.block_size)
    g = torch.Generator(device="cuda").manual_seed(1)

    def run(lens):
        x = torch.randn(sum(lens), shape.width, generator=g, device="cuda").bfloat16()
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        plan = requests.plan(torch.tensor(lens, dtype=torch.int32, device="cuda"), sum(lens))
        y = model.step(x, plan, requests.block_tables, max(lens))
        end.record()
        i8.sync_check()
        print(f"{sum(lens)} new tokens: {begin.elapsed_time(end):.3f} ms, finite: {bool(torch.isfinite(y).all())}, "
              f"[tokens, blocks in use, tokens without a block] = {plan.counts.tolist()}")

    run(prompts)
    for _ in range(steps):
        run([1] * len(prompts))


if __name__ == "__main__":
    main()
