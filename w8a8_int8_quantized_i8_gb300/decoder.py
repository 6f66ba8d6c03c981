"""A synthetic decoder stack on the W8A8 layer and the serving operators.

What runs at every step, for a batch of requests of any lengths (prompts,
chunks of prompts and single tokens mixed):

    block tables, slots, positions             build_block_tables, once a step
    per block:
      x + residual, RMS norm, 8-bit codes      add_rmsnorm_quant_act_pertoken
      QKV projection                           the fused W8A8 GEMM
      norm of q and k heads, rotation          heads_rmsnorm_rotate (rope_theta, head_norms)
      new keys and values into the cache       kv_cache_append
      causal attention over the cache          paged_attention
      out projection                           the W8A8 layer
      x + residual, RMS norm, 8-bit codes      add_rmsnorm_quant_act_pertoken
      MLP up, GELU + 8-bit codes, MLP down     the fused GEMMs, gelu_quant_act_pertoken

In the 4-bit formats (nvfp4, mxfp4) the norms are add_rmsnorm_quant_fp4, the
layers gemm_fp4_bias_bf16 and linear_fp4, and the MLP is gated: act(gate) * up
in one kernel (gemm_fp4_gated_bf16), then down.

Weights are random (seeded), as in dit_stack; there is no vocabulary and no
sampling: a step takes the new tokens' hidden rows and gives theirs back.
Nothing in a step waits for the device, so a step of fixed sizes can be captured
into a CUDA graph.
"""
from __future__ import annotations

import dataclasses
import sys

import torch

from . import binding as i8
from . import fp4, serving
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
    fmt: str = "int8"            # codes of activations and weights: int8, e4m3, nvfp4 or mxfp4
    cache_fmt: str = "int8"      # codes of the cache: int8 or e4m3
    block_size: int = 64
    rope_theta: float | None = None   # base of the rotation's frequencies; None: no rotation
    head_norms: bool = False     # RMS norm of each query and key head, with a gain
    activation: str = "silu"     # of the 4-bit formats' gated MLP: silu or gelu


class Decoder:
    """Quantized weights of a decoder and one cache a block."""

    def __init__(self, shape: Shape, cache_blocks: int, seed: int = 7, device="cuda"):
        self.shape = shape
        s = shape
        qkv = (s.q_heads + 2 * s.kv_heads) * s.head_dim
        sizes = (("qkv", s.width, qkv), ("out", s.q_heads * s.head_dim, s.width), ("up", s.width, s.mlp),
                 ("down", s.mlp, s.width))
        self.four_bits = s.fmt in fp4.FORMATS
        if self.four_bits:
            sizes += (("gate", s.width, s.mlp),)
        quant = i8.quant_weight_perchannel_e4m3 if s.fmt == "e4m3" else i8.quant_weight_perchannel
        self.layers, self.caches = [], []
        self.inv_freq = None
        if s.rope_theta is not None or s.head_norms:
            pairs = torch.arange(s.head_dim // 2 if s.rope_theta is not None else 0, dtype=torch.float64, device=device)
            self.inv_freq = ((s.rope_theta or 1.0) ** (-2 * pairs / s.head_dim)).float()
        for blk in range(s.blocks):
            layers = {}
            for li, (name, K, N) in enumerate(sizes):
                at = seed * 100003 + blk * 8 + li
                w, b = layer_weight(at, N, K, device)
                wq, s_w = (fp4.quant_rows_fp4(w, s.fmt), None) if self.four_bits else quant(w)
                layers[name] = Linear(wq, s_w, b, at, s.fmt)
            g = torch.Generator(device=device).manual_seed(seed * 100003 + blk * 8 + 7)
            layers["norms"] = [(1 + 0.1 * torch.randn(s.width, generator=g, device=device)).bfloat16()
                               for _ in range(2)]
            layers["head_norms"] = [(1 + 0.1 * torch.randn(s.head_dim, generator=g, device=device)).bfloat16()
                                    for _ in range(2)] if s.head_norms else (None, None)
            self.layers.append(layers)
            self.caches.append(serving.QuantKVCache.empty(cache_blocks, s.kv_heads, s.block_size, s.head_dim,
                                                          s.cache_fmt, device))

    def _norm(self, x, h, weight):
        """x + h, its norm's codes (what _gemm takes) and the sum in h's place."""
        if self.four_bits:
            rows, h = fp4.add_rmsnorm_quant_fp4(x, h, weight, fmt=self.shape.fmt, residual_out=h)
            return (rows,), h
        codes, scale, h = serving.add_rmsnorm_quant_act_pertoken(x, h, weight, fmt=self.shape.fmt, residual_out=h)
        return (codes, scale), h

    def _gemm(self, lin: Linear, codes):
        if self.four_bits:
            return fp4.gemm_fp4_bias_bf16(codes[0], lin.wq, lin.bias)
        fn = i8.gemm_e4m3_dequant_bias_bf16 if lin.fmt == "e4m3" else i8.gemm_dequant_bias_bf16
        return fn(*codes, lin.wq, lin.s_w, lin.bias)

    def _linear(self, lin: Linear, x):
        if self.four_bits:
            return fp4.linear_fp4(x, lin.wq, lin.bias)
        return (i8.linear_e4m3 if lin.fmt == "e4m3" else i8.linear)(x, lin.wq, lin.s_w, lin.bias)

    def _mlp(self, layers, codes):
        """(what goes into the down projection, what comes out of it)"""
        if self.four_bits:
            gate, up = layers["gate"], layers["up"]
            u = fp4.gemm_fp4_gated_bf16(codes[0], gate.wq, up.wq, gate.bias, up.bias, self.shape.activation)
            return u, self._linear(layers["down"], u)
        u = self._gemm(layers["up"], codes)
        return u, self._gemm(layers["down"], i8.gelu_quant_act_pertoken(u, fmt=self.shape.fmt))

    def step(self, x: torch.Tensor, plan: serving.BlockPlan, block_tables: torch.Tensor, max_new: int,
             record=None) -> torch.Tensor:
        """One step: x bf16 [T, width], the new tokens' rows in request order
        (T = the plan's slots).  ``max_new`` bounds the new tokens of a request.
        ``record(block, name, tensors)`` sees what goes in and out of the
        attention, and then of the block's layers."""
        s = self.shape
        h = torch.zeros_like(x)          # the residual stream: x joins it in the first norm
        for blk, (layers, cache) in enumerate(zip(self.layers, self.caches)):
            codes, h = self._norm(x, h, layers["norms"][0])
            qkv = self._gemm(layers["qkv"], codes)
            heads = qkv.unflatten(1, (s.q_heads + 2 * s.kv_heads, s.head_dim))
            q, k, v = heads.split((s.q_heads, s.kv_heads, s.kv_heads), dim=1)
            if self.inv_freq is not None:
                serving.heads_rmsnorm_rotate(q, k, plan.positions, self.inv_freq, *layers["head_norms"], out=(q, k))
            serving.kv_cache_append(k, v, plan.slots, cache)
            o = serving.paged_attention(q, cache, block_tables, plan.seq_lens, plan.cu_new, max_new)
            if record:
                record(blk, "attention", (q, k, v, o))
                record(blk, "qkv", codes)
            x = self._linear(layers["out"], o.flatten(1))
            if record:
                record(blk, "out", (o, x))
            codes, h = self._norm(x, h, layers["norms"][1])
            u, x = self._mlp(layers, codes)
            if record:
                record(blk, "mlp", (codes, u, x))
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
    """python -m w8a8_int8_quantized_i8_gb300.decoder [fmt]: a prompt, a few single
    tokens, and how long a step of either takes."""
    shape = Shape(fmt=sys.argv[1] if len(sys.argv) > 1 else "int8", rope_theta=10000.0, head_norms=True)
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
