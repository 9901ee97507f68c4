"""GB300-native batched draft-token verification for speculative decoding.

The verification step of speculative decoding (the Leviathan/Chen rule as the
pages "Speculative decoding and EAGLE", "Speculative decoding: draft, verify,
repeat" and "Speculative Decoding: from idea to SOTA" define it) as hand-written
sm_103a CUDA behind a C ABI (include/spec_verify.h, libspecverify.so); this
package is the thin binding plus the seeded workload generators.
"""
from .binding import (  # noqa: F401
    SPEC_BF16, SPEC_DRAFT_LOGITS, SPEC_DRAFT_PROBS, SPEC_F32, SPEC_MAX_K, SPEC_MAX_TREE_NODES,
    SpecError, declared_functions, last_error, lib, spec_debug_residual, spec_debug_stall, spec_profile_begin,
    spec_profile_end, spec_tree_workspace_bytes, spec_verify_greedy, spec_verify_sample,
    spec_verify_sample_noalloc, spec_tree_mask, spec_kv_commit, spec_row_stats, spec_tree_draft,
    spec_verify_tree_greedy, spec_workspace_bytes, status_string, workspace,
    q4_cache, spec_adjust_logits, spec_attend_q4, spec_attend_workspace_bytes, spec_kv_commit_q4, spec_kv_store_q4,
    spec_page_map, spec_q4_block_bytes, spec_debug_attend_stall,
    spec_kv_evict_plan, spec_kv_move_q4, spec_kv_weigh_q4, spec_page_trim, spec_token_logprobs,
)
