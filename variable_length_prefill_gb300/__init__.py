"""GB300-native packed variable-length attention forward (prefill).

The computation is atrex-bench "attention_forward" (page #001, reference.py,
Model.forward): per packed sequence and head, softmax(Q K^T / sqrt(D)) V,
non-causal (or, as an option, causal), bf16 in and out.  It runs in a
hand-written sm_103a CUDA library (TMA, tcgen05 MMA into TMEM,
warp-specialised online softmax) behind the C ABI in include/attn_varlen.h;
the same library holds the paged single-query decode of
include/paged_attn_decode.h, the attention of drafted tokens over the same
cache (include/paged_attn_tree.h), the operators that fill and manage it
(include/paged_attn_cache.h) and the chunked gated delta-rule output of
include/chunk_delta_rule.h.  This package is a thin ctypes binding.
"""
from ._binding import (AttnVarlenError, SYMBOLS, attn_varlen_fwd, attn_varlen_fwd_noalloc,
                       check, chunk_delta_rule_output, load, paged_attn_cache_accept,
                       paged_attn_cache_compact, paged_attn_cache_fork, paged_attn_cache_free,
                       paged_attn_cache_write, paged_attn_decode, paged_attn_tree, strerror,
                       workspace_size)
from .build import build, lib_path
from .shard import head_shard

__all__ = ["AttnVarlenError", "SYMBOLS", "attn_varlen_fwd", "attn_varlen_fwd_noalloc", "build",
           "check", "chunk_delta_rule_output", "head_shard", "lib_path", "load",
           "paged_attn_cache_accept", "paged_attn_cache_compact", "paged_attn_cache_fork",
           "paged_attn_cache_free", "paged_attn_cache_write", "paged_attn_decode",
           "paged_attn_tree", "strerror", "workspace_size"]
