"""GB300-native tree speculative-decoding verify step.

One verify round is five calls of the C ABI in ``include/tsv.h`` (built from
``csrc/`` into ``libtsv.so``): ``tree_mask`` -> ``tree_verify_attention`` ->
``lm_head_argmax`` -> ``tree_accept_walk`` -> ``kv_gather_positions``.  Ahead of
the head stand, where a target has them, ``add_rms_norm`` and products with 8-bit
weights (``matmul_e4m3``); ``token_logprobs`` tells about the emitted tokens.  This
package is only the Python binding (argument marshalling over ctypes); it has
no fallback and raises if the library is not built.
"""
from ._abi import (ATTN_AUTO, ATTN_SIMT, ATTN_TCGEN05, BF16, E4M3_B128, F32, DEV_TIMEOUT, DEV_BAD_KV_LEN, DEV_BAD_PARENT, DEV_BAD_PATH, DEV_BAD_ROOT, DEV_BAD_SEQ_LEN, DEV_OK, F16, I4_G64, I8_SCALED,
                   MAX_LAYERS, MAX_T, Q4_G64, AttnDesc, GdnDesc, KvDesc, TsvError, load)
from .api import (VerifyRound, append_desc, draft_children, tree_select, attention_workspace_size, attn_desc, gdn_commit, gdn_desc, gdn_scan, gdn_tree_verify, kv_desc, kv_gather_positions, gather_positions, lm_head_argmax,
                  lm_head_logits, lm_head_workspace_size, sample_nucleus, sample_workspace_size, sliding_band_mask, tree_accept_walk, tree_append, tree_mask,
                  tree_verify_attention,
                  add_rms_norm, greedy_tokens, matmul_e4m3, matmul_e4m3_argmax, quantize_e4m3, token_logprobs, token_logprobs_workspace_size)

__all__ = [
    "load", "TsvError", "ATTN_AUTO", "ATTN_SIMT", "ATTN_TCGEN05", "DEV_TIMEOUT", "AttnDesc", "KvDesc", "F16", "BF16", "I8_SCALED", "Q4_G64", "MAX_T", "MAX_LAYERS",
    "DEV_OK", "DEV_BAD_ROOT", "DEV_BAD_PARENT", "DEV_BAD_PATH", "DEV_BAD_KV_LEN",
    "draft_children", "tree_select", "tree_mask", "sliding_band_mask", "append_desc", "tree_append", "attn_desc", "attention_workspace_size", "tree_verify_attention", "lm_head_workspace_size",
    "lm_head_argmax", "lm_head_logits", "sample_workspace_size", "sample_nucleus", "tree_accept_walk", "kv_desc", "kv_gather_positions", "gather_positions", "VerifyRound",
    "I4_G64", "DEV_BAD_SEQ_LEN", "GdnDesc", "gdn_desc", "gdn_tree_verify", "gdn_commit", "gdn_scan",
    "E4M3_B128", "F32", "add_rms_norm", "quantize_e4m3", "matmul_e4m3", "matmul_e4m3_argmax", "token_logprobs", "token_logprobs_workspace_size",
    "greedy_tokens",
]
