"""QSPEC hot path on GB300 (sm_103a): one shared INT4 weight set, a W4A4
draft linear, a W4A16 verify linear, an INT4 activation quantiser, greedy and
sampled verification, the KV overwrite, and draft-side sampling with the
draft statistics (confidence, entropy); and, between the linears of a decoder
layer, the residual RMSNorm with an E4M3 output, a 4-bit KV cache with the
attention of draft and verify steps over it, and causal attention over packed
prompts -- CUDA kernels behind the C ABI in include/qspec.h, bound here with
ctypes.

Importing the package does not load the library; the first call does, and
raises if libqspec.so has not been built (``build.build()``).
"""
from .binding import (QspecError, attn_kv4, attn_kv4_workspace, attn_prompt, draft_sample, draft_workspace,
                      kv4_append, kv4_cache, kv4_load, kv_overwrite, linear_w4a4, linear_w4a4_bf16,
                      linear_w4a16, load_library, pack_weights, quant_act_int4, rmsnorm_fp8, verify_greedy,
                      verify_sample, verify_workspace)

__all__ = ["QspecError", "attn_kv4", "attn_kv4_workspace", "attn_prompt", "draft_sample", "draft_workspace",
           "kv4_append", "kv4_cache", "kv4_load", "kv_overwrite", "linear_w4a4", "linear_w4a4_bf16",
           "linear_w4a16", "load_library", "pack_weights", "quant_act_int4", "rmsnorm_fp8", "verify_greedy",
           "verify_sample", "verify_workspace"]
