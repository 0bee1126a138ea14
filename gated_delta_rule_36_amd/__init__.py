"""Gated Delta Rule-2 token mixer for MI355X (gfx950): HIP kernels behind a C ABI.

    from gated_delta_rule_36_amd import chunk_fwd, decode_step

`chunk_fwd` runs the chunkwise-parallel forward over whole (optionally packed)
sequences, two-phase (with a workspace) or fused; `chunk_bwd` its gradients;
`decode_step` advances a pool of recurrent states by one token, `decode_tokens` by
several (with slot indexing and committed prefixes, for serving); `block_prologue` and
`block_epilogue` are the block's branches around the mixer. The softmax-attention layer that a
hybrid stack puts beside the mixer: `qk_norm_rope` (norms of queries and keys with the
position rotation, differentiable), `attn_prologue` (the same for serving, filling a paged
8-bit `kv_cache`) and `cache_attention` over that cache. What stands around the mixer in a stack:
`linear_recurrence` (a state per channel, differentiable; `linear_recurrence_tokens` for serving),
`residual_norm` (the norm between layers with the residual's addition, differentiable;
`residual_norm_8bit` for e4m3 projections) and `verify_drafts` (how many drafted tokens a pool of
states commits). All call libgdn2.so, built in-tree by `python -m gated_delta_rule_36_amd.build`.
"""
from ._attn import (CACHE_BLOCK, KVCache, attn_prologue, cache_attention,
                    cache_attention_workspace_bytes, kv_cache, qk_norm_rope, qk_norm_rope_bwd,
                    qk_norm_rope_fwd, value_columns)
from ._lib import (Gdn2Error, SavedForBackward, block_epilogue, block_prologue,
                   chunk_bwd, chunk_fwd, chunk_fwd_train, decode_step, decode_tokens,
                   gated_delta_rule2, lib, lib_path, uses_split, workspace_bytes)
from ._stack import (linear_recurrence, linear_recurrence_bwd, linear_recurrence_fwd,
                     linear_recurrence_fwd_train, linear_recurrence_tokens, residual_norm,
                     residual_norm_8bit, residual_norm_bwd, residual_norm_fwd, verify_drafts,
                     verify_drafts_workspace_bytes)

__all__ = ["chunk_fwd", "chunk_fwd_train", "chunk_bwd", "gated_delta_rule2", "SavedForBackward",
           "decode_step", "decode_tokens", "block_prologue", "block_epilogue", "workspace_bytes",
           "qk_norm_rope", "qk_norm_rope_fwd", "qk_norm_rope_bwd", "KVCache", "kv_cache",
           "CACHE_BLOCK", "value_columns", "attn_prologue", "cache_attention",
           "cache_attention_workspace_bytes", "linear_recurrence", "linear_recurrence_fwd",
           "linear_recurrence_fwd_train", "linear_recurrence_bwd", "linear_recurrence_tokens",
           "residual_norm", "residual_norm_fwd", "residual_norm_bwd", "residual_norm_8bit",
           "verify_drafts", "verify_drafts_workspace_bytes", "uses_split", "lib", "lib_path", "Gdn2Error"]
