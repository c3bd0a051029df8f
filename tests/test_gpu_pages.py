"""Pages shared, taken, given back and compacted on the GPU, against a plain implementation: every value
(table, lengths, counts, pool) is equal, for every cache type; and what is refused or skipped."""

import numpy as np
import pytest
import torch

from sparse_self_speculative_verify_gb300 import (KV4Cache, KVCache, PagePool, Workspace, binding, ssd_kv_advance,
                                                 ssd_kv_compact, ssd_kv_fork, ssd_kv_release, ssd_kv_reserve, ssd_status)
from tests import _gpu
from tests._pages import Pages

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BITS = dict(index=binding.FAULT_INDEX, page=binding.FAULT_PAGE, seqlen=binding.FAULT_SEQLEN, nopage=binding.FAULT_NOPAGE,
            kmax=binding.FAULT_KMAX)


def _make(kind, lens, page, h=2, d=64, spare=8, cap=None, rows=0, seed=0, room=0):
    """(cache on the GPU, PagePool, plain Pages) with `rows` empty rows behind the requests."""
    rng = np.random.default_rng(seed)
    lens = list(lens) + [0] * rows
    need = [-(-n // page) for n in lens]
    cap = cap or max(need) + -(-room // page) + 1
    total = sum(need) + spare
    perm = rng.permutation(total)
    table = np.full((len(lens), cap), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    refs = np.zeros(total, np.int32)
    refs[table[table >= 0]] = 1
    width = {"bf16": d, "f32": d, "nvfp4": d // 2 + d // 16}[kind]
    raw = rng.integers(0, 256 if kind == "nvfp4" else 30000, (total, 2, h, page, width))
    pool = raw.astype({"bf16": np.int16, "f32": np.int32, "nvfp4": np.uint8}[kind])
    t = torch.from_numpy(pool).to(DEV)
    t = t.view({"bf16": torch.bfloat16, "f32": torch.float32, "nvfp4": torch.uint8}[kind])
    cls = KV4Cache if kind == "nvfp4" else KVCache
    kv = cls(t, torch.from_numpy(table).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), cap * page)
    pages = PagePool.from_table(kv.page_table, total)
    assert np.array_equal(pages.refs.cpu().numpy(), refs)
    return kv, pages, Pages(pool, table, lens, refs, cap * page, d if kind == "nvfp4" else None)


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _same(kv, pages, want, what=""):
    torch.cuda.synchronize()
    st = ssd_status()
    bits = 0
    for f in want.faults:
        bits |= BITS[f]
    want.faults.clear()
    assert st == bits, f"{what}: status {st:#x}, expected {bits:#x}"
    np.testing.assert_array_equal(kv.page_table.cpu().numpy(), want.table, err_msg=what)
    assert kv.seq_lens.cpu().tolist() == want.lens, what
    if pages is not None:
        np.testing.assert_array_equal(pages.refs.cpu().numpy(), want.refs, err_msg=what)
    got = kv.pool.view({2: torch.int16, 4: torch.int32, 1: torch.uint8}[kv.pool.element_size()]).cpu().numpy()
    np.testing.assert_array_equal(got, want.pool, err_msg=what)


@pytest.mark.parametrize("kind,page", [("bf16", 16), ("f32", 1), ("bf16", 4), ("nvfp4", 8), ("nvfp4", 64)])
@pytest.mark.parametrize("d", [64, 128])
def test_random_run_of_branching(kind, page, d):
    """Many steps of forking, reserving, advancing, rolling back and releasing."""
    _gpu.lib()
    kv, pages, P = _make(kind, [5 * page + 3, page, 1, 0, 2 * page - 1], page, h=3, d=d, spare=70, rows=7, cap=16)
    rng = np.random.default_rng(page)
    for step in range(25):
        empty = [b for b in range(12) if not (P.table[b] >= 0).any()]
        full = [b for b in range(12) if P.lens[b] > 0]
        if empty and full:
            n = int(rng.integers(1, len(empty) + 1))
            dst = [int(x) for x in rng.choice(empty, n, replace=False)]
            src = [int(x) for x in rng.choice(full, n)]
            P.fork(src, dst)
            ssd_kv_fork(kv, pages, _i32(src), _i32(dst))
            _same(kv, pages, P, f"fork {step}")
        counts = [int(x) if rng.random() < 0.7 else 0 for x in rng.integers(0, 2 * page + 2, 12)]
        counts = [min(c, P.max_len - n) for c, n in zip(counts, P.lens)]
        P.reserve(counts)
        ssd_kv_reserve(kv, pages, _i32(counts))
        failed = "nopage" in P.faults
        _same(kv, pages, P, f"reserve {step}")
        P.check()
        if not failed:
            ssd_kv_advance(kv.seq_lens, _i32(counts), kv.max_seq_len)
            P.lens = [a + b for a, b in zip(P.lens, counts)]
        back = [int(rng.integers(0, min(n, 3) + 1)) for n in P.lens]
        ssd_kv_advance(kv.seq_lens, -_i32(back), kv.max_seq_len)
        P.lens = [a - b for a, b in zip(P.lens, back)]
        keep = [-1 if rng.random() < 0.6 else (0 if rng.random() < 0.5 else int(rng.integers(0, P.max_len + 5))) for _ in range(12)]
        P.release(keep)
        ssd_kv_release(kv, pages, _i32(keep))
        _same(kv, pages, P, f"release {step}")
        P.check()


def test_lowest_holder_keeps_when_all_ask_and_everybody_copies_when_not():
    _gpu.lib()
    for ask in ([3, 3, 3, 3], [0, 3, 3, 3], [3, 0, 0, 0], [0, 0, 0, 3]):
        kv, pages, P = _make("bf16", [21], 16, rows=3, spare=6)
        P.fork([0, 0, 0], [3, 1, 2])
        ssd_kv_fork(kv, pages, _i32([0, 0, 0]), _i32([3, 1, 2]))
        P.reserve(ask)
        ssd_kv_reserve(kv, pages, _i32(ask))
        _same(kv, pages, P, str(ask))
        P.check()


def test_reserve_is_all_or_nothing_and_uses_the_last_free_page():
    _gpu.lib()
    kv, pages, P = _make("nvfp4", [16, 9, 30], 8, spare=3)
    for counts in ([8, 8, 10], [8, 8, 2], [8, 0, 0]):
        P.reserve(counts)
        ssd_kv_reserve(kv, pages, _i32(counts))
        _same(kv, pages, P, str(counts))
        P.check()


def test_many_rows_and_a_large_pool():
    """More rows than the reserve's lanes take at once, free pages far into the pool."""
    _gpu.lib()
    kv, pages, P = _make("bf16", [17 + 3 * (b % 5) for b in range(300)], 4, h=1, spare=20000, rows=300, cap=40)
    src, dst = list(range(300)), list(range(300, 600))
    P.fork(src, dst)
    ssd_kv_fork(kv, pages, _i32(src), _i32(dst))
    P.refs[:9000] += 1  # as if another cache held the low pages
    pages.refs[:9000] += 1
    counts = [(7 * b) % 90 for b in range(600)]
    P.reserve(counts)
    ssd_kv_reserve(kv, pages, _i32(counts))
    _same(kv, pages, P)


def test_fork_refusals():
    _gpu.lib()
    kv, pages, P = _make("bf16", [21, 40, 7], 16, rows=5)
    cases = [([0, 1], [3, 3]), ([0, 3], [4, 5]), ([0, 4], [4, 6]), ([0], [0]), ([-1, 0], [5, 8]), ([9], [6]), ([1], [2])]
    for src, dst in cases:
        P.fork(src, dst)
        ssd_kv_fork(kv, pages, _i32(src), _i32(dst))
        _same(kv, pages, P, f"{src} -> {dst}")
    P.check()
    # A page that nobody holds, and a length out of range.
    P.refs[P.table[2, 0]] = 0
    pages.refs[int(P.table[2, 0])] = 0
    P.lens[1] = P.max_len + 1
    kv.seq_lens[1] = P.max_len + 1
    P.fork([2, 1], [6, 7])
    ssd_kv_fork(kv, pages, _i32([2, 1]), _i32([6, 7]))
    _same(kv, pages, P, "unheld page, bad length")


def test_reserve_and_release_faults():
    _gpu.lib()
    kv, pages, P = _make("bf16", [21, 40, 7, 10, 12], 16, spare=9, room=32)
    total = len(P.refs)
    for b, j, p in ((1, 2, total + 5), (2, 0, -1)):  # a page id outside the pool; a live page missing
        if P.table[b, j] >= 0:
            P.refs[P.table[b, j]] = 0
            pages.refs[int(P.table[b, j])] = 0
        P.table[b, j] = p
        kv.page_table[b, j] = p
    P.refs[P.table[3, 0]] = 0  # held by nobody, says the count
    pages.refs[int(P.table[3, 0])] = 0
    for counts in ([20, 20, 20, 20, 20], [-1, 0, 0, 0, P.max_len]):
        P.reserve(counts)
        ssd_kv_reserve(kv, pages, _i32(counts))
        _same(kv, pages, P, str(counts))
    P.lens[4] = -3
    kv.seq_lens[4] = -3
    P.release([0, 0, 0, 0, 0])
    ssd_kv_release(kv, pages, _i32([0, 0, 0, 0, 0]))
    _same(kv, pages, P, "release")
    assert (pages.refs >= 0).all()


@pytest.mark.parametrize("kind,page,to_page", [("bf16", 16, 16), ("f32", 1, 8), ("nvfp4", 8, 32), ("nvfp4", 64, 16)])
@pytest.mark.parametrize("d", [64, 128])
def test_compact_into_another_cache(kind, page, to_page, d):
    _gpu.lib()
    kv, _, P = _make(kind, [300, 1, 77, 50], page, h=3, d=d)
    kept = [137, 1, 0, 50]
    to, to_pages, Q = _make(kind, [150, 9, 64, 50], to_page, h=3, d=d, seed=5)
    rng = np.random.default_rng(3)
    src, dst = [0, 3, 1, 2], [3, 0, 1, 2]
    kept = [kept[s] for s in src]
    kept[0] = 50  # row 3 of `to` holds pages for 50 tokens
    idx = np.full((4, 3, 140), -1, np.int32)
    for i, s in enumerate(src):
        for g in range(3):
            idx[i, g, :kept[i]] = np.sort(rng.choice(P.lens[s], kept[i], replace=False))
    cnt = np.repeat(np.array(kept, np.int32)[:, None], 3, 1)
    P.compact_to(Q, src, dst, idx, cnt)
    ssd_kv_compact(kv, to, _i32(src), _i32(dst), _i32(idx), _i32(cnt), pages=to_pages)
    _same(to, to_pages, Q, "to")
    _same(kv, None, P, "from")


def test_eviction_in_one_cache_and_the_move_back():
    """Keep some tokens of a request in a spare row, give its pages back, and hand it the kept ones."""
    _gpu.lib()
    kv, pages, P = _make("bf16", [200, 90], 16, rows=1, spare=10)
    idx = np.stack([np.sort(np.random.default_rng(g).choice(200, 60, replace=False)) for g in range(2)]).astype(np.int32)[None]
    cnt = np.full((1, 2), 60, np.int32)
    P.reserve([0, 0, 60])
    ssd_kv_reserve(kv, pages, _i32([0, 0, 60]))
    P.compact_to(P, [0], [2], idx, cnt)
    ssd_kv_compact(kv, kv, _i32([0]), _i32([2]), _i32(idx), _i32(cnt), pages=pages)
    _same(kv, pages, P, "compact")
    P.release([0, -1, -1])
    ssd_kv_release(kv, pages, _i32([0, -1, -1]))
    P.fork([2], [0])
    ssd_kv_fork(kv, pages, _i32([2]), _i32([0]))
    P.release([-1, -1, 0])
    ssd_kv_release(kv, pages, _i32([-1, -1, 0]))
    _same(kv, pages, P, "moved")
    P.check()
    assert P.lens == [60, 90, 0]


def test_compact_refusals():
    _gpu.lib()
    kv, pages, P = _make("bf16", [40, 40, 40, 33], 16, rows=2)
    ones = np.zeros((2, 2, 4), np.int32)
    cnt = np.full((2, 2), 2, np.int32)
    before = kv.pool.clone()

    def call(src, dst, idx=ones, cnt=cnt, bits=0, **k):
        ssd_kv_compact(kv, kv, _i32(src), _i32(dst), _i32(idx[:len(src)]), _i32(cnt[:len(src)]), **k)
        torch.cuda.synchronize()
        assert ssd_status() == bits
        assert torch.equal(kv.pool.view(torch.int16), before.view(torch.int16))
        assert kv.seq_lens.cpu().tolist() == P.lens

    call([0], [0], bits=binding.FAULT_INDEX)
    call([0, 1], [1, 0], bits=binding.FAULT_INDEX)
    call([6, 0], [1, -1], bits=binding.FAULT_INDEX)
    call([0], [1], cnt=np.array([[2, 1]], np.int32), bits=binding.FAULT_KMAX)
    call([0], [1], cnt=np.array([[5, 5]], np.int32), bits=binding.FAULT_KMAX)
    # A list entry past the end stores zeros; a destination that is not there, or shared, is not written.
    idx = np.array([[[3, 40], [3, -1]]], np.int32)
    ssd_kv_compact(kv, kv, _i32([0]), _i32([1]), _i32(idx), _i32(cnt[:1]))
    torch.cuda.synchronize()
    assert ssd_status() == binding.FAULT_INDEX
    p = int(P.table[1, 0])
    assert not kv.pool[p, :, :, 1].view(torch.int16).any()
    assert torch.equal(kv.pool[p, :, :, 0].view(torch.int16), before[int(P.table[0, 0]), :, :, 3].view(torch.int16))
    before = kv.pool.clone()
    P.lens[1] = 2
    ssd_kv_fork(kv, pages, _i32([3]), _i32([4]))
    P.lens[4] = 33
    P.lens[4] = 2
    call([0], [4], bits=binding.FAULT_PAGE, pages=pages)
    P.lens[5] = 2
    call([0], [5], bits=binding.FAULT_PAGE)


def test_page_calls_captured_in_a_graph_and_on_another_stream():
    """release -> fork -> reserve, replayed: each replay ends in the state of the plain run."""
    _gpu.lib()
    kv, pages, P = _make("bf16", [37, 50], 16, rows=4, spare=20)
    keep, src, dst, counts = [37, 50, 0, 0, 0, 0], [0, 0, 1, 1], [2, 3, 4, 5], [5] * 6
    args = [_i32(x) for x in (keep, src, dst, counts)]
    ws = Workspace()

    def step(stream=None, workspace=None):
        ssd_kv_release(kv, pages, args[0], stream=stream)
        ssd_kv_fork(kv, pages, args[1], args[2], stream=stream)
        ssd_kv_reserve(kv, pages, args[3], stream=stream, workspace=workspace)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    for workspace in (None, ws):
        if workspace is ws:
            step(workspace=ws)  # sizes the workspace before the capture
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(workspace=workspace)
        for _ in range(3):
            g.replay()
    P.release(keep), P.fork(src, dst), P.reserve(counts)
    _same(kv, pages, P)
    P.check()
