"""One speculative round on one attention layer: verify (with criticality) -> Top-K select -> k
sparse drafts, with every buffer allocated once so the round can be replayed or captured in a CUDA
graph.

SparseSpec ("Accelerating Large-Scale Reasoning Model Inference: Self-Speculative Decoding with
Sparse Attention") §4.1: the sparse pattern is refreshed by every verify and stays fixed for the k
drafts that follow it (the refresh stride equals k); §2.3 / §3.2: a round is k drafts plus one
verify of the k+1 positions.

The cache may be a 4-bit one (``KV4Cache``): the same round runs on ``ssd_kv4_verify_attn`` and
``ssd_kv4_draft_attn``.  Its rows are read where they are (no row pack: four 72-byte rows fill what one
packed bf16 row does), and ``verify_select`` is a verify followed by a select.
"""

from __future__ import annotations

import math
from contextlib import nullcontext as _nullcontext
from typing import Optional, Union

import torch

from . import binding as B


class SpecRound:
    def __init__(self, kv: Union[B.KVCache, B.KV4Cache], h_q: int, n_cand: int, k_max: int, scale: Optional[float] = None,
                 workspace: Optional[B.Workspace] = None, pack_rows: bool = True, pack_in_select: bool = False):
        self.kv = kv
        self._nvfp4 = isinstance(kv, B.KV4Cache)
        if self._nvfp4 and pack_in_select:
            raise ValueError("a 4-bit cache has no row pack")
        self.h_q = h_q
        self.n_cand = n_cand
        self.k_max = k_max
        self.scale = scale if scale is not None else 1.0 / math.sqrt(kv.d)
        dev = kv.device
        Bsz, hkv, d = kv.batch, kv.h_kv, kv.d
        self.ws = workspace or B.Workspace()
        self.out_v = torch.empty((Bsz, n_cand, h_q, d), dtype=torch.float32, device=dev)
        self.lse_v = torch.empty((Bsz, n_cand, h_q), dtype=torch.float32, device=dev)
        self.scores = torch.zeros((Bsz, hkv, max(kv.max_seq_len, 1)), dtype=torch.float32, device=dev)
        self.idx = torch.empty((Bsz * hkv, k_max), dtype=torch.int32, device=dev)
        self.cnt = torch.empty((Bsz * hkv,), dtype=torch.int32, device=dev)
        self.out_d = torch.empty((Bsz, h_q, d), dtype=torch.float32, device=dev)
        self.lse_d = torch.empty((Bsz, h_q), dtype=torch.float32, device=dev)
        # Row pack: the selected K / V rows stored contiguously, by the first draft after a selection
        # or (pack_in_select) by the fused verify-select itself; the other drafts of the round read
        # them from there.  On the Qwen3-8B round the first draft's gather is the cheaper of the two
        # (the criticality pass's copy lengthens the verify call by more than it saves the draft).
        self.pack_in_select = pack_in_select
        self.pack = None
        if pack_rows and not self._nvfp4:
            n = B.ssd_draft_pack_bytes(kv, k_max)
            self.pack = torch.empty(n + 256, dtype=torch.uint8, device=dev)
            off = (-self.pack.data_ptr()) % 256
            self.pack = self.pack[off:off + n]
        self._packed = False

    def verify(self, q_verify: torch.Tensor, stream=None):
        call = B.ssd_kv4_verify_attn if self._nvfp4 else B.ssd_verify_attn
        return call(self.kv, q_verify, self.n_cand, self.scale, out=self.out_v, lse=self.lse_v, scores=self.scores,
                    workspace=self.ws, stream=stream)

    def verify_select(self, q_verify: torch.Tensor, k_per_req: torch.Tensor, stream=None):
        """verify + select in one call: the selection runs inside the criticality pass, which also
        stores the selected rows in the row pack (pack_in_select), so every draft reads it."""
        if self._nvfp4:
            r = self.verify(q_verify, stream)
            return dict(r, **dict(zip(("idx", "cnt"), self.select(k_per_req, stream))))
        pack = self.pack if self.pack_in_select else None
        r = B.ssd_verify_select(self.kv, q_verify, self.n_cand, self.scale, k_per_req, self.k_max, out=self.out_v,
                                lse=self.lse_v, scores=self.scores, idx=self.idx, cnt=self.cnt, pack=pack,
                                workspace=self.ws, stream=stream)
        self._packed = pack is not None
        return r

    def select(self, k_per_req: torch.Tensor, stream=None):
        self._packed = False
        return B.ssd_select_topk(self.scores, self.kv.seq_lens, k_per_req, self.k_max, self.kv.h_kv,
                                 max_len=self.kv.max_seq_len, idx=self.idx, cnt=self.cnt, stream=stream)

    def set_selection(self, idx: torch.Tensor, cnt: torch.Tensor, stream=None):
        """Install a selection made elsewhere (idx [B, H_kv, k_max] int32, cnt [B, H_kv]) in place
        of the last select's; the next draft stores the row pack again."""
        self._packed = False
        with torch.cuda.stream(stream) if stream is not None else _nullcontext():
            self.idx.view(self.kv.batch, self.kv.h_kv, self.k_max).copy_(idx)
            self.cnt.view(self.kv.batch, self.kv.h_kv).copy_(cnt)

    def draft(self, q_draft: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None, last: bool = False):
        """One draft over the current selection.  With the row pack, the first draft after a select
        stores the selected rows and the following ones read them (same results within the oracle
        tolerance).  The choice is made when the call is issued, so a captured CUDA graph keeps the
        choice of its capture: capture the drafts together with the selection (as ``run`` does), so
        that the graph's first draft writes the pack on every replay.  ``last`` marks the round's last
        draft: it reads the pack and then drops it from L2 unwritten, so the next draft writes it
        again."""
        idx = self.idx.view(self.kv.batch, self.kv.h_kv, self.k_max)
        cnt = self.cnt.view(self.kv.batch, self.kv.h_kv)
        o = out if out is not None else self.out_d
        if self.pack is None:
            call = B.ssd_kv4_draft_attn if self._nvfp4 else B.ssd_draft_attn
            return call(self.kv, q_draft, idx, cnt, self.scale, out=o, lse=self.lse_d, workspace=self.ws,
                        stream=stream)
        if not self._packed:
            mode = B.PACK_WRITE
        else:
            mode = B.PACK_READ_DISCARD if last else B.PACK_READ
        self._packed = not (self._packed and last)
        return B.ssd_draft_attn_packed(self.kv, q_draft, idx, cnt, self.scale, self.pack, mode, out=o, lse=self.lse_d,
                                       workspace=self.ws, stream=stream)

    def draft_oracle_topk(self, q_draft: torch.Tensor, k_per_req: torch.Tensor, out: Optional[torch.Tensor] = None,
                          stream=None) -> dict:
        """Draft with the "oracle top-k" pattern (SparseSpec §3.3, the reference the pages measure
        drafts against): the draft query selects by its own exact criticality instead of by the last
        verify's.  Three calls: a verify pass with the draft query as the single candidate (it sees
        the whole cache) gives that criticality and the dense output; Top-K selects K_b tokens per
        (request, KV head); the sparse draft attends them.  Buffers are allocated on first use.
        Returns the sparse draft's ``out`` / ``lse`` plus ``dense`` (the full-attention output) and
        the selection ``idx`` / ``cnt``."""
        kv = self.kv
        Bsz, hkv, d = kv.batch, kv.h_kv, kv.d
        if not hasattr(self, "_o_scores"):
            dev = kv.device
            self._o_dense = torch.empty((Bsz, 1, self.h_q, d), dtype=torch.float32, device=dev)
            self._o_lse = torch.empty((Bsz, 1, self.h_q), dtype=torch.float32, device=dev)
            self._o_scores = torch.zeros((Bsz, hkv, max(kv.max_seq_len, 1)), dtype=torch.float32, device=dev)
            self._o_idx = torch.empty((Bsz * hkv, self.k_max), dtype=torch.int32, device=dev)
            self._o_cnt = torch.empty((Bsz * hkv,), dtype=torch.int32, device=dev)
            self._o_out = torch.empty((Bsz, self.h_q, d), dtype=torch.float32, device=dev)
            self._o_lse_d = torch.empty((Bsz, self.h_q), dtype=torch.float32, device=dev)
        verify, draft = (B.ssd_kv4_verify_attn, B.ssd_kv4_draft_attn) if self._nvfp4 else (B.ssd_verify_attn, B.ssd_draft_attn)
        verify(kv, q_draft.view(Bsz, 1, self.h_q, d), 1, self.scale, out=self._o_dense, lse=self._o_lse,
               scores=self._o_scores, workspace=self.ws, stream=stream)
        B.ssd_select_topk(self._o_scores, kv.seq_lens, k_per_req, self.k_max, hkv, max_len=kv.max_seq_len,
                          idx=self._o_idx, cnt=self._o_cnt, stream=stream)
        o = out if out is not None else self._o_out
        draft(kv, q_draft, self._o_idx.view(Bsz, hkv, self.k_max), self._o_cnt.view(Bsz, hkv), self.scale,
              out=o, lse=self._o_lse_d, workspace=self.ws, stream=stream)
        return {"out": o, "lse": self._o_lse_d, "dense": self._o_dense.view(Bsz, self.h_q, d),
                "scores": self._o_scores, "idx": self._o_idx, "cnt": self._o_cnt}

    def run(self, q_verify: torch.Tensor, q_drafts: torch.Tensor, k_per_req: torch.Tensor,
            draft_outs: Optional[torch.Tensor] = None, stream=None, fused_select: bool = False):
        """verify -> select -> len(q_drafts) drafts.  draft_outs [k, B, h_q, d] keeps every draft's
        output (else each overwrites ``out_d``).  fused_select runs the selection inside the verify's
        criticality pass (one launch fewer, same results)."""
        if fused_select:
            self.verify_select(q_verify, k_per_req, stream)
        else:
            self.verify(q_verify, stream)
            self.select(k_per_req, stream)
        k = q_drafts.shape[0]
        for j in range(k):
            self.draft(q_drafts[j], out=None if draft_outs is None else draft_outs[j], stream=stream,
                       last=j == k - 1)


class TreeRound:
    """One step that verifies a drafted tree of tokens, on one attention layer, with every buffer allocated once: a draft token's
    cheap attention (a window of recent tokens and the first ones), the tree's verify attention, the nodes' log probabilities, the
    path that stays and its commit to the cache (SpecSA "branch handling"; SparseSpec §2.3 verifies a chain, the tree in which
    every node hangs on the one before it).  ``draft`` is for a request's last token, a tree's root or a chain's; trees grow from
    the alternatives that ``score`` gives (``draft`` of an inner node would see its siblings, which lie beside it in the cache).

    A step: append the nodes' K and V (``ssd_kv_append``), advance the lengths by the nodes' counts (``ssd_kv_advance``),
    ``verify``; from the logits ``score`` and ``accept``; ``commit`` on every layer's cache; ``advance`` once.  With caches
    that share their lengths, one round accepts and advances and the others only ``verify`` and ``commit``."""

    def __init__(self, kv: B.KVCache, h_q: int, n_nodes: int, window: int, sink: int = 4, max_path: Optional[int] = None,
                 scale: Optional[float] = None, workspace: Optional[B.Workspace] = None):
        self.kv, self.h_q, self.n, self.window, self.sink = kv, h_q, n_nodes, window, sink
        self.max_path = min(max_path or n_nodes, n_nodes)
        self.scale = scale if scale is not None else 1.0 / math.sqrt(kv.d)
        self.ws = workspace
        b, dev, dt = kv.batch, kv.device, kv.pool.dtype
        new = lambda *shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
        self.out_t, self.lse_t = new(b, n_nodes, h_q, kv.d, dtype=dt), new(b, n_nodes, h_q, dtype=torch.float32)
        self.out_d, self.lse_d = new(b, 1, h_q, kv.d, dtype=dt), new(b, 1, h_q, dtype=torch.float32)
        self.logprob, self.lse, self.entropy = (new(b, n_nodes, dtype=torch.float32) for _ in range(3))
        self.path, self.cnt, self.next, self.back = new(b, self.max_path), new(b), new(b), new(b)
        self._first = (torch.arange(b, dtype=torch.int32, device=dev) * n_nodes)[:, None]  # a tree's first row of logits
        self._rows = new(b, n_nodes)

    def draft(self, q: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> dict:
        """Attention of one draft token per request, the last of its cache: q [B, 1, h_q, d]."""
        return B.ssd_window_attn(self.kv, q, self.window, self.sink, self.scale, out=self.out_d if out is None else out,
                                 lse=self.lse_d, workspace=self.ws, stream=stream)

    def verify(self, q: torch.Tensor, parents: torch.Tensor, counts: Optional[torch.Tensor] = None, stream=None) -> dict:
        """Attention of the trees' nodes, the last of their caches: q [B, n, h_q, d]."""
        return B.ssd_tree_attn(self.kv, q, parents, self.scale, counts=counts, out=self.out_t, lse=self.lse_t, workspace=self.ws,
                               stream=stream)

    def score(self, logits: torch.Tensor, tokens: torch.Tensor, parents: torch.Tensor, top_k: int = 0, stream=None) -> dict:
        """Every node's log probability under its parent's row (a root's: 0), every row's entropy and top_k alternatives.
        logits [B * n, vocab]; tokens, parents int32 [B, n], a parent of -1 behind a tree's counts."""
        with torch.cuda.stream(stream) if stream is not None else _nullcontext():
            torch.add(parents, self._first, out=self._rows)
            self._rows.masked_fill_(parents < 0, -1)
        return B.ssd_token_logprobs(logits, tokens.view(-1), rows=self._rows.view(-1), top_k=top_k, logprob=self.logprob.view(-1),
                                    lse=self.lse.view(-1), entropy=self.entropy.view(-1), stream=stream)

    def accept(self, parents: torch.Tensor, tokens: torch.Tensor, target: torch.Tensor, counts: Optional[torch.Tensor] = None,
               epsilon: Optional[float] = None, delta: Optional[float] = None, stream=None) -> dict:
        """The path that stays, by equality with ``target`` or, with epsilon and delta, by the last ``score``."""
        if (epsilon is None) != (delta is None):
            raise ValueError("epsilon and delta go together")
        more = {} if epsilon is None else dict(logprob=self.logprob, entropy=self.entropy, epsilon=epsilon, delta=delta)
        return B.ssd_tree_accept(parents, tokens, target, counts=counts, max_path=self.max_path, path=self.path, cnt=self.cnt,
                                 next=self.next, advance=self.back, stream=stream, **more)

    def commit(self, counts: Optional[torch.Tensor] = None, kv: Optional[B.KVCache] = None, stream=None) -> None:
        """Moves the accepted rows of this round's cache, or of another layer's, together."""
        B.ssd_tree_commit(self.kv if kv is None else kv, self.path, self.cnt, self.n, counts=counts, stream=stream)

    def advance(self, stream=None) -> None:
        """Shortens the lengths to what was accepted."""
        B.ssd_kv_advance(self.kv.seq_lens, self.back, self.kv.max_seq_len, stream=stream)
