"""GB300 (sm_103a) W8A8 INT8 linear layer.

Per-token activation quantization and a fused int8 x int8 -> int32 GEMM whose
epilogue applies the per-token x per-channel dequantization and the bias and
writes bf16 ("Realizing Native INT8 Compute for Diffusion Transformers on
Consumer GPUs: A Fused INT8 GEMM Kernel for Ideogram 4.0", arXiv 2606.14598,
abstract).  The computation lives in libi8.so (CUDA, include/i8.h); the
functions below are its torch-tensor binding: the linear layer in binding.py,
its 4-bit route in fp4.py, and in serving.py what a decoder runs besides it at
every step (the norm with an 8-bit output, the rotation of queries and keys,
block tables, and attention over an 8-bit paged cache).
"""
from .binding import (I8Error, e4m3_workspace_bytes, f16codes_workspace_bytes,
                      gelu_quant_act_pertoken, gemm_dequant_bias_bf16_f16codes,
                      gemm_int32_f16codes, get_option, linear_f16codes,
                      quant_act_pertoken_f16codes, gemm_dequant_bias_bf16,
                      gemm_e4m3_dequant_bias_bf16, gemm_e4m3_f32, gemm_int32,
                      layernorm_quant_act_pertoken, linear, linear_e4m3, load, plan_query,
                      quant_act_pertoken,
                      quant_act_pertoken_e4m3, quant_weight_perchannel,
                      quant_weight_perchannel_e4m3, set_option, sync_check, widen_weight_codes,
                      workspace_bytes)
from .serving import (BlockPlan, QuantKVCache, add_rmsnorm_quant_act_pertoken, build_block_tables,
                      heads_rmsnorm_rotate, kv_cache_append, paged_attention,
                      paged_attention_workspace_bytes)
from .fp4 import (FP4Rows, add_rmsnorm_quant_fp4, gated_linear_fp4, gemm_fp4_bias_bf16,
                  gemm_fp4_gated_bf16, linear_fp4, linear_fp4_workspace_bytes, quant_rows_fp4)

__all__ = [
    "BlockPlan", "QuantKVCache", "add_rmsnorm_quant_act_pertoken", "build_block_tables",
    "kv_cache_append", "paged_attention", "paged_attention_workspace_bytes", "heads_rmsnorm_rotate",
    "FP4Rows", "add_rmsnorm_quant_fp4", "gated_linear_fp4", "gemm_fp4_bias_bf16", "gemm_fp4_gated_bf16",
    "linear_fp4", "linear_fp4_workspace_bytes", "quant_rows_fp4",
    "I8Error", "e4m3_workspace_bytes", "f16codes_workspace_bytes", "gelu_quant_act_pertoken",
    "gemm_dequant_bias_bf16_f16codes", "gemm_int32_f16codes", "get_option", "linear_f16codes",
    "quant_act_pertoken_f16codes", "gemm_dequant_bias_bf16", "gemm_e4m3_dequant_bias_bf16",
    "gemm_e4m3_f32", "gemm_int32", "layernorm_quant_act_pertoken", "linear", "linear_e4m3", "load", "plan_query", "quant_act_pertoken",
    "quant_act_pertoken_e4m3", "quant_weight_perchannel", "quant_weight_perchannel_e4m3",
    "set_option", "sync_check", "widen_weight_codes", "workspace_bytes",
]
