"""Acceptance of drafted trees and the commit of their rows, against plain forms."""

import numpy as np
import pytest
import torch

import sparse_self_speculative_verify_gb300 as F
from sparse_self_speculative_verify_gb300 import binding
from tests import _tree

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def dev(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype)).to(DEV)


def expect(r, parents, target, counts, max_path, **kw):
    torch.cuda.synchronize()
    for b in range(len(parents)):
        one = {k: v[b] if isinstance(v, np.ndarray) else v for k, v in kw.items()}
        path, nxt = _tree.accept(parents[b], target[b], int(counts[b]), max_path, **one)
        assert r["path"][b].tolist() == path + [-1] * (max_path - len(path)), b
        assert (int(r["cnt"][b]), int(r["next"][b]), int(r["advance"][b])) == (len(path), nxt, len(path) - int(counts[b])), b


@pytest.mark.parametrize("B,n,max_path", [(1, 1, 1), (7, 5, 5), (40, 16, 8), (9, 64, 64), (33, 129, 3), (5, 512, 20)])
def test_accept_equal(B, n, max_path):
    rng = np.random.default_rng(B * n)
    par = _tree.random_trees(B, n, rng, back=5)
    par[rng.random((B, n)) < 0.05] = -1  # more roots: none but node 0 stays
    par[0] = np.arange(n) - 1            # a chain
    tok = rng.integers(0, 3, (B, n)).astype(np.int32)
    tgt = rng.integers(0, 3, (B, n)).astype(np.int32)
    tok[0] = tgt[0] = 1                  # accepted to its end
    counts = rng.integers(0, n + 1, B).astype(np.int32)
    counts[0] = n
    r = F.ssd_tree_accept(dev(par), dev(tok), dev(tgt), counts=dev(counts), max_path=max_path)
    expect(r, par, tgt, counts, max_path, tokens=tok)
    r = F.ssd_tree_accept(dev(par), dev(tok), dev(tgt))
    expect(r, par, tgt, np.full(B, n), n, tokens=tok)
    assert F.ssd_status() == 0


@pytest.mark.parametrize("B,n,max_path", [(1, 2, 2), (40, 16, 8), (5, 300, 9)])
def test_accept_by_probability(B, n, max_path):
    rng = np.random.default_rng(n)
    par = _tree.random_trees(B, n, rng)
    lp = (-3 * rng.random((B, n))).astype(np.float32)
    ent = (4 * rng.random((B, n))).astype(np.float32)
    lp[rng.random((B, n)) < 0.05] = -np.inf
    lp[rng.random((B, n)) < 0.05] = np.nan
    ent[rng.random((B, n)) < 0.05] = np.nan
    tgt = rng.integers(0, 99, (B, n)).astype(np.int32)
    kw = dict(epsilon=0.3, delta=0.7)
    r = F.ssd_tree_accept(dev(par), None, dev(tgt), logprob=dev(lp, np.float32), entropy=dev(ent, np.float32), max_path=max_path, **kw)
    expect(r, par, tgt, np.full(B, n), max_path, logprob=lp, entropy=ent, **kw)
    # At the border itself: not above it.
    lo = np.float32(np.log(0.3))
    lp2, ent2 = np.full((1, 3), lo, np.float32), np.zeros((1, 3), np.float32)
    lp2[0, 2] = np.nextafter(lo, np.float32(0))
    p2 = np.array([[-1, 0, 0]], np.int32)
    r = F.ssd_tree_accept(dev(p2), None, dev(p2 + 50), logprob=dev(lp2, np.float32), entropy=dev(ent2, np.float32), epsilon=0.3, delta=1.0)
    assert r["path"].tolist() == [[0, 2, -1]] and r["next"].tolist() == [50]


def test_accept_reports_bad_trees():
    par = np.array([[-1, 0, 5, 2], [0, 0, 1, -7], [-1, 0, 1, 2]], np.int32)
    tok = np.ones((3, 4), np.int32)
    r = F.ssd_tree_accept(dev(par), dev(tok), dev(tok), counts=dev([4, 4, 9]))
    assert F.ssd_status() == binding.FAULT_INDEX | binding.FAULT_SEQLEN
    assert r["path"].tolist() == [[0, 1, -1, -1], [0, 1, 2, -1], [0, 1, 2, 3]]


def cache(B, lens, h, page, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    cap = -(-(max(lens) + 1) // page)
    perm = torch.randperm(B * cap + 3, generator=g)[:B * cap].view(B, cap).int()
    pool = torch.randn((B * cap + 3, 2, h, page, d), generator=g).to(dtype)
    return F.KVCache(pool.to(DEV), perm.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), max(lens)), pool.clone(), perm


def moved(pool, perm, lens, counts, path, cnt, page, skip=()):
    for b in range(len(lens)):
        if b in skip:
            continue
        base = lens[b] - counts[b]
        src = [base + int(x) for x in path[b][:cnt[b]]]
        rows = torch.stack([pool[perm[b, t // page], :, :, t % page] for t in src]) if src else None
        for j in range(len(src)):
            pool[perm[b, (base + j) // page], :, :, (base + j) % page] = rows[j]
    return pool


@pytest.mark.parametrize("dtype,d,h,page,n", [(torch.bfloat16, 128, 8, 16, 16), (torch.bfloat16, 64, 3, 1, 40), (torch.float32, 128, 1, 8, 300),
                                              (torch.float32, 64, 2, 512, 5)])
def test_commit(dtype, d, h, page, n):
    rng = np.random.default_rng(n)
    B = 6
    counts = [n, 1, n, max(1, n // 2), 0, n]
    lens = [n + 37, 1, n, 90 + n, 11, n + 5]
    kv, pool, perm = cache(B, lens, h, page, d, dtype, n)
    m = min(n, 40)
    path = np.full((B, m), -1, np.int32)
    cnt = []
    for b in range(B):
        k = min(m, counts[b]) if b != 2 else 0
        k = int(rng.integers(1, k + 1)) if k else 0
        path[b, :k] = np.sort(rng.choice(counts[b], k, replace=False)) if k else []
        cnt.append(k)
    path[5] = np.arange(m) + n - m  # the last m nodes, shifted as a whole
    cnt[5] = m
    F.ssd_tree_commit(kv, dev(path), dev(cnt), n, counts=dev(counts))
    torch.cuda.synchronize()
    assert F.ssd_status() == 0
    want = moved(pool, perm, lens, counts, path, cnt, page)
    assert torch.equal(kv.pool.cpu().view(torch.uint8), want.view(torch.uint8))
    assert kv.seq_lens.tolist() == lens


def test_commit_leaves_bad_requests_alone():
    B, n, page = 9, 6, 8
    lens = [20, 20, 20, 20, 4, 20, 20, 20, 20]
    kv, pool, perm = cache(B, lens, 2, page, 64, torch.bfloat16, 3)
    counts = [6, 6, 6, 6, 6, 7, -1, 6, 6]
    path = np.tile(np.array([[1, 3, 5, -1]], np.int32), (B, 1))
    cnt = [3, 3, 3, 5, 3, 3, 3, -2, 3]
    path[1] = [3, 3, 5, -1]
    path[2] = [1, 3, 6, -1]
    table = kv.page_table
    table[8, 2] = pool.shape[0]  # page of the last tokens outside the pool
    F.ssd_tree_commit(kv, dev(path), dev(cnt), n, counts=dev(counts))
    torch.cuda.synchronize()
    assert F.ssd_status() == binding.FAULT_INDEX | binding.FAULT_KMAX | binding.FAULT_SEQLEN | binding.FAULT_PAGE
    want = moved(pool, perm, lens, counts, path, cnt, page, skip=range(1, 9))
    assert torch.equal(kv.pool.cpu().view(torch.uint8), want.view(torch.uint8))
