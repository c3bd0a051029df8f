"""GB300 (sm_103a) attention hot path of sparse self-speculative decoding.

Verify attention with fused criticality, Top-K selection, sparse draft attention, the unified
verify/draft launch and the block-granular variant, the same verify and draft over a 4-bit cache, the
calls that share, reserve, release and compact a cache's pages, and those of a step that drafts trees of
tokens (tree and sliding-window attention, scores, acceptance, commit), as CUDA kernels behind the C ABI in
``include/ssd.h``.  ``binding`` is the thin Python layer over that ABI; ``round`` strings the calls
of one speculative round together; ``workloads`` draws the seeded synthetic inputs.
"""

from .binding import (KV4Cache, KVCache, LibraryNotBuilt, PagePool, SSDError, Workspace, ssd_block_sparse_attn,
                      ssd_block_union, ssd_combine, ssd_draft_attn, ssd_draft_attn_packed, ssd_draft_attn_static,
                      ssd_draft_pack_bytes, ssd_kv4_append, ssd_kv4_draft_attn, ssd_kv4_read, ssd_kv4_verify_attn,
                      ssd_kv_advance, ssd_kv_append, ssd_kv_compact, ssd_kv_fork, ssd_kv_release, ssd_kv_reserve,
                      ssd_phase_assign, ssd_phase_fill, ssd_select_topk, ssd_select_topp, ssd_status,
                      ssd_token_logprobs, ssd_tree_accept, ssd_tree_attn, ssd_tree_commit, ssd_unified_attn,
                      ssd_verify_attn, ssd_verify_select, ssd_version, ssd_window_attn)
from .round import SpecRound, TreeRound

__all__ = ["KV4Cache", "KVCache", "LibraryNotBuilt", "PagePool", "SSDError", "SpecRound", "TreeRound", "Workspace",
           "ssd_block_sparse_attn", "ssd_block_union", "ssd_combine", "ssd_draft_attn", "ssd_draft_attn_packed",
           "ssd_draft_attn_static", "ssd_draft_pack_bytes", "ssd_kv4_append", "ssd_kv4_draft_attn", "ssd_kv4_read",
           "ssd_kv4_verify_attn", "ssd_kv_advance", "ssd_kv_append", "ssd_kv_compact", "ssd_kv_fork",
           "ssd_kv_release", "ssd_kv_reserve", "ssd_phase_assign", "ssd_phase_fill", "ssd_select_topk",
           "ssd_select_topp", "ssd_status", "ssd_token_logprobs", "ssd_tree_accept", "ssd_tree_attn", "ssd_tree_commit",
           "ssd_unified_attn", "ssd_verify_attn", "ssd_verify_select", "ssd_version", "ssd_window_attn"]
