"""Tree and window attention where they go wrong most easily: bad pages, lengths and trees, batches and groups of every size,
long caches shared by many blocks, pools past 4 GB, workspaces that hold something, streams and threads."""

import threading

import numpy as np
import pytest
import torch

import sparse_self_speculative_verify_gb300 as F
from sparse_self_speculative_verify_gb300 import binding
from tests._tree import Case
from tests.test_gpu_span import BF, DEV, F32, check, run

pytestmark = pytest.mark.gpu


def kv_of(c, **over):
    d = dict(pool=c.pool.to(DEV), table=c.table.to(DEV), lens=torch.tensor(c.lens, dtype=torch.int32, device=DEV))
    d.update(over)
    return F.KVCache(d["pool"], d["table"], d["lens"], c.max_len)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("G", [1, 3, 17, 64, 128])
def test_groups_of_every_size(dtype, G):
    n = 3 if G < 64 else 2
    check(c := Case([200, n], [n, n], n, G, 1, 64, 16, dtype, seed=G), run(c))
    check(c := Case([200, 70], [n, 1], n, 2 * G, 2, 128, 8, dtype, seed=G, window=33, sink=3), run(c))


@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 64, 128, 256, 1024])
def test_pages_of_every_size(page):
    check(c := Case([300, 17, 129], [5, 5, 2], 5, 4, 2, 64, page, BF, seed=page), run(c))
    check(c := Case([300, 17, 129], [5, 5, 2], 5, 4, 2, 64, page, BF, seed=page, window=100, sink=9), run(c))


def test_more_requests_than_a_launch_holds():
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 40, 1100)]
    counts = [min(x, int(y)) for x, y in zip(lens, rng.integers(0, 3, 1100))]
    c = Case(lens, counts, 2, 2, 1, 64, 8, BF, seed=1, window=20, sink=1)
    check(c, run(c))


@pytest.mark.parametrize("n,h_q", [(1, 8), (7, 8), (60, 8)])
def test_few_long_requests_that_many_blocks_share(n, h_q):
    """One request's units are cut into many parts (d = 128, 2 heads)."""
    c = Case([20000], [n], n, h_q, 2, 128, 64, BF, seed=n)
    check(c, run(c))
    c = Case([20000, 300], [n, 1], n, h_q, 2, 128, 64, BF, seed=n, window=9000, sink=700)
    check(c, run(c))


@pytest.mark.parametrize("dtype,d,page", [(F32, 128, 16), (F32, 64, 8), (BF, 128, 4), (BF, 64, 2)])
@pytest.mark.parametrize("n", [3, 5, 9, 18, 33])
def test_row_blocks_of_every_size_on_cuda_cores(dtype, d, page, n):
    """12, 20, 36, 72 and 132 rows a head, more units than fit the SMs at once."""
    lens = [n + (61 * b) % 280 for b in range(40)]
    counts = [n - b % 3 for b in range(40)]
    check(c := Case(lens, counts, n, 8, 2, d, page, dtype, seed=n), run(c))
    check(c := Case(lens, counts, n, 8, 2, d, page, dtype, seed=n, window=70, sink=2), run(c))


@pytest.mark.parametrize("B,n", [(1, 1), (9, 3), (40, 1), (110, 2)])
@pytest.mark.parametrize("window", [900, 1300, 2000])
def test_units_around_the_size_that_is_cut(B, n, window):
    """Units of 8 to 17 tiles, fewer and more of them than blocks."""
    lens = [n + (97 * b) % 2100 if b % 5 else 2150 for b in range(B)]
    check(c := Case(lens, [n] * B, n, 8, 4, 64, 16, BF, seed=B, window=window, sink=6), run(c))


def test_scores_that_grow_along_the_cache():
    """The reference of a row moves many times, by more than the exponent of a half."""
    c = Case([3000], [4], 4, 4, 1, 128, 16, BF, seed=3)
    t = torch.arange(3000)
    rows = c.pool[c.table[0].long()[t // 16], 0, 0, t % 16].float()
    rows += (t / 3000 * 400)[:, None] * c.q[0, 0, 0].float() / c.q[0, 0, 0].float().square().sum()
    c.pool[c.table[0].long()[t // 16], 0, 0, t % 16] = rows.to(BF)
    c.scale = 1.0
    check(c, run(c))


def test_same_bits_twice_whatever_the_workspace_holds():
    c = Case([5000, 900, 40], [20, 20, 7], 20, 8, 2, 128, 16, BF, seed=5)
    ws = F.Workspace()
    a = run(c, workspace=ws)
    a = {k: v.clone() for k, v in a.items()}
    buf = ws._bufs[(DEV, "span")]
    buf[binding.COUNTER_BYTES + 256:].fill_(255)  # (the counters stay zero)
    b = run(c, workspace=ws)
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    check(c, b)


def test_rows_without_a_query_are_zeroed_and_others_written():
    for dtype in (BF, F32):
        c = Case([50, 3, 0, 20], [4, 3, 0, 0], 6, 4, 2, 64, 8, dtype, seed=2)
        out = torch.full((4, 6, 4, 64), float("nan"), dtype=dtype, device=DEV)
        lse = torch.full((4, 6, 4), float("nan"), device=DEV)
        check(c, run(c, out=out, lse=lse))


@pytest.mark.parametrize("dtype,page", [(BF, 16), (BF, 4), (F32, 16)])
def test_lengths_and_counts_out_of_range(dtype, page):
    c = Case([40, 40, 40, 40], [5, 5, 5, 5], 5, 4, 2, 64, page, dtype, seed=4)
    good = run(c)
    lens = torch.tensor([40, 41, 3, -7], dtype=torch.int32, device=DEV)  # fine, above max_seq_len, below the count, negative
    cnt = torch.tensor([9, 5, 5, 5], dtype=torch.int32, device=DEV)
    kv = kv_of(c, lens=lens)
    r = F.ssd_tree_attn(kv, c.q.to(DEV), torch.from_numpy(c.parents).to(DEV), c.scale, counts=cnt)
    torch.cuda.synchronize()
    assert F.ssd_status() == binding.FAULT_SEQLEN
    assert torch.equal(r["out"][:2], good["out"][:2])  # clamped to 40 tokens and 5 queries
    assert (r["out"][2, :2] == 0).all() and torch.isinf(r["lse"][2, :2]).all() and torch.isfinite(r["lse"][2, 2:]).all()
    assert (r["out"][3] == 0).all() and torch.isinf(r["lse"][3]).all()


@pytest.mark.parametrize("dtype,page", [(BF, 16), (BF, 8), (BF, 4), (F32, 16)])
def test_pages_outside_the_pool_read_as_zeros(dtype, page):
    c = Case([100, 60], [3, 3], 3, 4, 2, 64, page, dtype, seed=6)
    table = c.table.clone()
    table[0, 2], table[1, 0] = c.pool.shape[0], -5
    r = F.ssd_tree_attn(kv_of(c, table=table.to(DEV)), c.q.to(DEV), torch.from_numpy(c.parents).to(DEV), c.scale)
    torch.cuda.synchronize()
    assert F.ssd_status() == binding.FAULT_PAGE
    c.pool[c.table[0, 2]] = 0
    c.pool[c.table[1, 0]] = 0
    check(c, r)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_bad_parents_end_a_node_s_ancestors(dtype):
    c = Case([90], [6], 6, 4, 2, 64, 16, dtype, seed=7, parents=np.array([[-1, 0, 1, -1, -1, 4]], np.int32))
    bad = torch.tensor([[-1, 0, 1, 3, 5, 4]], dtype=torch.int32, device=DEV)
    r = F.ssd_tree_attn(kv_of(c), c.q.to(DEV), bad, c.scale)
    torch.cuda.synchronize()
    assert F.ssd_status() == binding.FAULT_INDEX
    check(c, r)


def test_pool_past_4_gb():
    """Pages whose byte offsets need more than 32 bits (and element offsets more than 31)."""
    c = Case([700, 90], [9, 9], 9, 8, 8, 128, 16, BF, seed=8)
    pages = 140_000  # 64 KB each
    pool = torch.empty((pages, 2, 8, 16, 128), dtype=BF, device=DEV)
    pool[pages - c.pool.shape[0]:] = c.pool.to(DEV)
    table = torch.where(c.table >= 0, c.table + (pages - c.pool.shape[0]), -1).to(DEV)
    cnt = torch.tensor(c.counts, dtype=torch.int32, device=DEV)
    kv = kv_of(c, pool=pool, table=table)
    par = torch.from_numpy(c.parents).to(DEV)
    check(c, F.ssd_tree_attn(kv, c.q.to(DEV), par, c.scale, counts=cnt))
    path = torch.tensor([[0, 4, 8], [1, 2, 6]], dtype=torch.int32, device=DEV)
    before = [kv.pool[table[b, (L - 9 + int(j)) // 16], :, :, (L - 9 + int(j)) % 16].clone() for b, L in enumerate(c.lens) for j in path[b]]
    F.ssd_tree_commit(kv, path, torch.tensor([3, 3], dtype=torch.int32, device=DEV), 9)
    after = [kv.pool[table[b, (L - 9 + j) // 16], :, :, (L - 9 + j) % 16] for b, L in enumerate(c.lens) for j in range(3)]
    assert all(torch.equal(x, y) for x, y in zip(before, after)) and F.ssd_status() == 0
    del pool, kv
    c32 = Case([70], [3], 3, 4, 2, 64, 4, BF, seed=8)  # CUDA cores
    pages = 2_200_000  # 2 KB each
    pool = torch.empty((pages, 2, 2, 4, 64), dtype=BF, device=DEV)
    pool[pages - c32.pool.shape[0]:] = c32.pool.to(DEV)
    table = torch.where(c32.table >= 0, c32.table + (pages - c32.pool.shape[0]), -1).to(DEV)
    check(c32, F.ssd_tree_attn(kv_of(c32, pool=pool, table=table), c32.q.to(DEV), torch.from_numpy(c32.parents).to(DEV), c32.scale))


def test_requests_that_share_pages():
    """Two requests over the same pages, and one request's tokens as another's beginning."""
    c = Case([320], [4], 4, 8, 2, 128, 16, BF, seed=9)
    lens = torch.tensor([320, 320], dtype=torch.int32, device=DEV)
    table = c.table.repeat(2, 1).to(DEV)
    kv = F.KVCache(c.pool.to(DEV), table, lens, 320)
    r = F.ssd_tree_attn(kv, c.q.repeat(2, 1, 1, 1).to(DEV), torch.from_numpy(c.parents).repeat(2, 1).to(DEV), c.scale)
    for b in range(2):
        check(c, {k: v[b:b + 1] for k, v in r.items()})


def test_other_streams_and_threads():
    """Calls of different shapes at once on several streams, and from two threads on one."""
    cases = [Case([3000 + 100 * i, 50], [5 + i, 5], 5 + i, 8, 2, 128, 16, BF, seed=10 + i) for i in range(3)]
    want = [run(c) for c in cases]
    torch.cuda.synchronize()
    kvs = [kv_of(c) for c in cases]
    q, par = [c.q.to(DEV) for c in cases], [torch.from_numpy(c.parents).to(DEV) for c in cases]
    cnt = [torch.tensor(c.counts, dtype=torch.int32, device=DEV) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[F.ssd_tree_attn(kvs[i], q[i], par[i], cases[i].scale, counts=cnt[i], stream=streams[i]) for i in range(3)] for _ in range(20)]
    torch.cuda.synchronize()
    for rs in got:
        assert all(torch.equal(r["out"], w["out"]) and torch.equal(r["lse"], w["lse"]) for r, w in zip(rs, want))
    results, errors = [[], []], []

    def body(i):
        try:
            for _ in range(200):
                results[i].append(F.ssd_tree_attn(kvs[i], q[i], par[i], cases[i].scale, counts=cnt[i])["out"])
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=body, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not errors and F.ssd_status() == 0
    assert all(torch.equal(o, want[i]["out"]) for i in range(2) for o in results[i])


def test_two_graphs_replayed_at_once():
    """Each has its own workspace, captured without a call before it on that stream."""
    cases = [Case([5000 + 900 * i, 60], [6, 5 + i], 6, 8, 2, 128, 16, BF, seed=30 + i) for i in range(2)]
    want = [run(c) for c in cases]
    kvs = [kv_of(c) for c in cases]
    q, par = [c.q.to(DEV) for c in cases], [torch.from_numpy(c.parents).to(DEV) for c in cases]
    cnt = [torch.tensor(c.counts, dtype=torch.int32, device=DEV) for c in cases]
    streams, graphs, outs = [torch.cuda.Stream() for _ in cases], [torch.cuda.CUDAGraph() for _ in cases], []
    torch.cuda.synchronize()
    for i in range(2):
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            outs.append(F.ssd_tree_attn(kvs[i], q[i], par[i], cases[i].scale, counts=cnt[i]))
    torch.cuda.synchronize()
    for _ in range(10):
        for o in outs:
            o["out"].zero_()
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                for _ in range(5):
                    graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o["out"], w["out"]) and torch.equal(o["lse"], w["lse"]) for o, w in zip(outs, want))
    assert F.ssd_status() == 0


def test_refusals_name_what_is_wrong():
    c = Case([40], [3], 3, 4, 2, 64, 8, BF, seed=11)
    kv, q, par = kv_of(c), c.q.to(DEV), torch.from_numpy(c.parents).to(DEV)
    for what, match in ((lambda: F.ssd_tree_attn(kv, q.float(), par, 0.1), "q must be"), (lambda: F.ssd_tree_attn(kv, q[:, :2], par, 0.1), "contiguous|must be"),
                        (lambda: F.ssd_tree_attn(kv, q, par.long(), 0.1), "parents must be"), (lambda: F.ssd_tree_attn(kv, q, par[:, :2].contiguous(), 0.1), "parents must be"),
                        (lambda: F.ssd_tree_attn(kv, q, par, -1.0), "scale"), (lambda: F.ssd_window_attn(kv, q, 0, 0, 0.1), "window"),
                        (lambda: F.ssd_window_attn(kv, q, (1 << 32) + 8, 0, 0.1), "window"), (lambda: F.ssd_window_attn(kv, q, 8, 1 << 32, 0.1), "sink"),
                        (lambda: F.TreeRound(kv, 4, 3, 8).accept(par, par, par, epsilon=0.1), "go together"),
                        (lambda: F.ssd_window_attn(kv, q, 5, 0, 0.1, out=torch.empty(q.shape, device=DEV)), "out must be"),
                        (lambda: F.ssd_window_attn(kv, q, 5, 0, 0.1, counts=par), "counts must be"),
                        (lambda: F.ssd_window_attn(kv, q[0], 5, 0, 0.1), "q must be"),
                        (lambda: F.ssd_tree_commit(kv, par.long(), par[:, 0].contiguous(), 3), "path must be")):
        with pytest.raises((ValueError, TypeError, F.SSDError), match=match):
            what()
