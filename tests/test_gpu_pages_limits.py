"""The page calls at the ends of their ranges on the GPU: sums, positions and byte offsets past 32 bits."""

import pytest
import torch

from sparse_self_speculative_verify_gb300 import (KVCache, PagePool, binding, ssd_kv_compact, ssd_kv_fork, ssd_kv_reserve,
                                                 ssd_status)
from tests import _gpu

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_reserve_of_2_to_the_31_pages_in_one_call():
    """1024 rows that each ask for 2^21 pages: far more than the pool has, so nothing changes."""
    _gpu.lib()
    rows, cap, page = 1024, 1 << 21, 8
    pool = torch.ones((64, 2, 1, page, 64), dtype=torch.bfloat16, device=DEV)
    table = torch.full((rows, cap), -1, dtype=torch.int32, device=DEV)
    table[3, 0] = 5
    lens = torch.zeros(rows, dtype=torch.int32, device=DEV)
    lens[3] = 2
    kv = KVCache(pool, table, lens, cap * page)
    pages = PagePool(torch.zeros(64, dtype=torch.int32, device=DEV))
    pages.refs[5] = 1
    counts = torch.full((rows,), cap * page, dtype=torch.int32, device=DEV)
    counts[3] -= 2
    ssd_kv_reserve(kv, pages, counts)
    torch.cuda.synchronize()
    assert ssd_status() == binding.FAULT_NOPAGE
    assert table[3, 0].item() == 5 and (table.sum(1, dtype=torch.int64) == -cap).sum().item() == rows - 1
    assert table[3].sum(dtype=torch.int64).item() == 5 - (cap - 1)
    assert pages.refs.tolist() == [int(p == 5) for p in range(64)]
    assert lens.tolist() == [2 * (b == 3) for b in range(rows)]
    # The same rows, asking for what there is.
    counts.fill_(0)
    counts[3], counts[1023] = page, page
    ssd_kv_reserve(kv, pages, counts)
    torch.cuda.synchronize()
    assert ssd_status() == 0
    assert table[3, :3].tolist() == [5, 0, -1] and table[1023, :2].tolist() == [1, -1]
    del table, kv
    torch.cuda.empty_cache()


def test_pages_whose_rows_lie_past_2_gb():
    """One page per request, as of a cache that is not paged: fp32 rows of 512 bytes, 2^22 and more of them."""
    _gpu.lib()
    page, d, L = 1 << 23, 128, (1 << 22) + 5
    pool = torch.empty((3, 2, 1, page, d), dtype=torch.float32, device=DEV)
    pool[2, :, 0, :L] = torch.arange(L, dtype=torch.float32, device=DEV)[:, None]
    pool[2, 1, 0, :L] += 0.5
    pool[0].zero_()
    table = torch.tensor([[2], [-1], [1]], dtype=torch.int32, device=DEV)
    kv = KVCache(pool, table, torch.tensor([L, 0, 0], dtype=torch.int32, device=DEV), page)
    pages = PagePool.from_table(table, 3)
    row = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    # Compaction out of slots behind 2 GB, and one of its rows to such a slot.
    n = L - 3
    idx = torch.arange(n, dtype=torch.int32, device=DEV).flip(0)[None, None].contiguous()  # the last tokens first
    ssd_kv_compact(kv, kv, row(0), row(2), idx, torch.full((1, 1), n, dtype=torch.int32, device=DEV), pages=pages)
    torch.cuda.synchronize()
    assert ssd_status() == 0 and kv.seq_lens.tolist() == [L, 0, n]
    for w in range(2):
        assert torch.equal(pool[1, w, 0, :n], pool[2, w, 0, :n].flip(0)), w
    # A branch: its page is replaced by a free one, with all of the live tokens.
    ssd_kv_fork(kv, pages, row(0), row(1))
    ssd_kv_reserve(kv, pages, row(2, 2, 0))
    torch.cuda.synchronize()
    assert ssd_status() == 0
    assert table.tolist() == [[2], [0], [1]] and pages.refs.tolist() == [1, 1, 1]
    for w in range(2):
        assert torch.equal(pool[0, w, 0, :L], pool[2, w, 0, :L]), w
    del pool, kv
    torch.cuda.empty_cache()


def test_compact_between_two_caches_with_the_same_lengths():
    """Row 0 of one cache into row 0 of the other would write the length that its own blocks still read."""
    _gpu.lib()
    page, d, n, k = 16, 64, 4096, 3000
    g = torch.Generator(device=DEV).manual_seed(1)
    lens = torch.tensor([n, 0], dtype=torch.int32, device=DEV)
    pools = [torch.randn((n // page + 4, 2, 2, page, d), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    tables = [torch.arange(n // page, dtype=torch.int32, device=DEV).expand(2, -1).contiguous() for _ in range(2)]
    kv, to = (KVCache(p, t, lens, n) for p, t in zip(pools, tables))
    before = pools[1].clone()
    idx = torch.arange(n - k, n, dtype=torch.int32, device=DEV).expand(1, 2, k).contiguous()
    cnt = torch.full((1, 2), k, dtype=torch.int32, device=DEV)
    row = lambda x: torch.tensor([x], dtype=torch.int32, device=DEV)  # noqa: E731
    ssd_kv_compact(kv, to, row(0), row(0), idx, cnt)
    torch.cuda.synchronize()
    assert ssd_status() == binding.FAULT_INDEX
    assert lens.tolist() == [n, 0] and torch.equal(pools[1], before)
    ssd_kv_compact(kv, to, row(0), row(1), idx, cnt)  # another row's length
    torch.cuda.synchronize()
    assert ssd_status() == 0 and lens.tolist() == [n, k]
    flat = lambda p: p[tables[0][0].long()].transpose(0, 2).transpose(0, 1).reshape(2, 2, n, d)  # noqa: E731
    assert torch.equal(flat(pools[1])[:, :, :k], flat(pools[0])[:, :, n - k:])
