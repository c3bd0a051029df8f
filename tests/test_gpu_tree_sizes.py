"""Sizes that a C int does not hold, in the calls of a step that drafts trees: refused (nothing is launched or allocated)."""

import pytest
import torch

import sparse_self_speculative_verify_gb300 as F

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32, F32 = torch.int32, torch.float32
MANY = (1 << 32) + 3


def test_scores():
    one = torch.zeros((1, 1), device=DEV)
    tok = torch.zeros((1, 1), dtype=I32, device=DEV)
    before = torch.cuda.memory_allocated()
    with pytest.raises(ValueError, match="rows .* out of range"):
        F.ssd_token_logprobs(one.expand(MANY, 1))
    with pytest.raises(ValueError, match="top_k .* out of range|top_k .* outside"):
        F.ssd_token_logprobs(one, top_k=MANY)
    assert torch.cuda.memory_allocated() == before
    wide = torch.empty((1, MANY), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="vocab .* out of range"):
        F.ssd_token_logprobs(wide, tok)
    del wide
    many = torch.empty((1, MANY), dtype=I32, device=DEV)
    before = torch.cuda.memory_allocated()
    with pytest.raises(ValueError, match="tokens .* out of range"):
        F.ssd_token_logprobs(one, many)
    with pytest.raises(ValueError, match="tokens .* out of range"):
        F.ssd_token_logprobs(one, many.view(-1), rows=many.view(-1))
    assert torch.cuda.memory_allocated() == before


def test_trees():
    many = torch.empty((MANY,), dtype=I32, device=DEV)
    before = torch.cuda.memory_allocated()
    for shape, match in (((MANY, 1), "batch"), ((1, MANY), "n")):
        t = many.view(shape)
        with pytest.raises(ValueError, match=f"{match} .* out of range"):
            F.ssd_tree_accept(t, t, t)
    kv = F.KVCache(torch.zeros((2, 2, 1, 8, 64), device=DEV), torch.zeros((1, 1), dtype=I32, device=DEV), torch.ones((1,), dtype=I32, device=DEV), 8)
    with pytest.raises(ValueError, match="max_path .* out of range"):
        F.ssd_tree_commit(kv, many.view(1, MANY), torch.ones((1,), dtype=I32, device=DEV), 1)
    q = torch.zeros((1, 1, 1, 1), device=DEV)
    assert q.expand(1, MANY, 1, 64).shape[1] == MANY
    for call in (lambda x: F.ssd_window_attn(kv, x, 8, 0, 0.1), lambda x: F.ssd_tree_attn(kv, x, many.view(1, MANY), 0.1)):
        with pytest.raises(ValueError):  # (an expanded q is not contiguous, a contiguous one this long does not fit a GPU)
            call(q.expand(1, MANY, 1, 64))
    del kv, q
    assert torch.cuda.memory_allocated() <= before
