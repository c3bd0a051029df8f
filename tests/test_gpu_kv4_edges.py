"""The 4-bit cache where it can go wrong: bad page ids, lengths, list entries and values, logits that grow
along the context, alignment, large pools, empty batches, graphs and streams.  The definitions and the
tolerances (`_check`, `_bounds`) are those of test_gpu_kv4."""

import math

import numpy as np
import pytest
import torch

from sparse_self_speculative_verify_gb300 import (KV4Cache, Workspace, binding, ssd_kv4_append, ssd_kv4_draft_attn,
                                                 ssd_kv4_read, ssd_kv4_verify_attn, ssd_kv_compact, ssd_status)
from tests import _gpu, _kv4
from tests.test_gpu_kv4 import _bounds, _cache, _check, _rows

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# h_kv, G, d, n_cand: the kernels' forms (8 rows at most, tcgen05 with 32, 64 rows in two passes, d = 64).
FORMS = [(2, 4, 128, 1), (2, 4, 128, 5), (1, 8, 128, 8), (2, 4, 64, 5)]
form = pytest.mark.parametrize("form", FORMS, ids=lambda f: f"h{f[0]}G{f[1]}d{f[2]}n{f[3]}")


def _dev(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV, dtype)


def _with_zero_page(pool, table, bad):
    """The pool with a page of zeros behind it, and a table whose bad entries name that page."""
    zero = np.concatenate([pool, np.zeros_like(pool[:1])])
    return zero, np.where(bad, len(pool), table)


@form
@pytest.mark.parametrize("page", [8, 64, 256])
def test_pages_outside_the_pool_read_as_zeros(form, page):
    _gpu.lib()
    h, G, d, nc = form
    lens = [517, 300, 40]
    kv, pool, table = _cache(lens, h, d, page, seed=21)
    last = [(n - 1) // page for n in lens]
    table[0, last[0]] = -1
    table[1, 0] = len(pool)
    if page < 256:
        table[0, 1] = 2 ** 31 - 1
    bad = np.zeros(table.shape, bool)
    for b, n in enumerate(lens):
        bad[b, :last[b] + 1] = (table[b, :last[b] + 1] < 0) | (table[b, :last[b] + 1] >= len(pool))
    kv.page_table.copy_(_dev(table))
    q = _rows((3, nc, G * h, d), torch.bfloat16, 5, 1.5)
    r = ssd_kv4_verify_attn(kv, q.to(DEV), nc, 0.1)
    torch.cuda.synchronize()
    assert ssd_status() == binding.FAULT_PAGE
    zpool, ztable = _with_zero_page(pool, table, bad)
    q64 = q.double().numpy()
    X, A = _bounds(zpool, ztable, lens, q64, d, 0.1, 1, 1)
    _check(r, _kv4.verify(zpool, ztable, lens, q64, d, 0.1), A, X, False, nc * G, "verify")


@form
def test_lengths_out_of_range_are_clamped(form):
    _gpu.lib()
    h, G, d, nc = form
    lens = [200, 200, 90]
    kv, pool, table = _cache(lens, h, d, 16, seed=22)
    kv = KV4Cache(kv.pool, kv.page_table, _dev([-7, 2 ** 31 - 1, 90]), 200)
    q = _rows((3, nc, G * h, d), torch.bfloat16, 5, 1.5)
    r = ssd_kv4_verify_attn(kv, q.to(DEV), nc, 0.1)
    torch.cuda.synchronize()
    assert ssd_status() == binding.FAULT_SEQLEN
    lens = [0, 200, 90]
    q64 = q.double().numpy()
    X, A = _bounds(pool, table, lens, q64, d, 0.1, 1, 1)
    _check(r, _kv4.verify(pool, table, lens, q64, d, 0.1), A, X, False, nc * G, "verify")


@pytest.mark.parametrize("d,G", [(128, 4), (128, 16), (64, 8)])
def test_lists_with_entries_and_counts_out_of_range(d, G):
    _gpu.lib()
    lens, h, page = [300, 90, 300], 2, 16
    kv, pool, table = _cache(lens, h, d, page, seed=23)
    rng = np.random.default_rng(4)
    k = 70
    idx = np.stack([np.stack([np.sort(rng.choice(n, k, replace=False)) for _ in range(h)]) for n in lens]).astype(np.int32)
    cnt = np.full((3, h), k, np.int32)
    idx[0, 0, 3], idx[0, 1, 40], idx[1, 0, 0], idx[1, 1, 69] = -1, 300, 2 ** 31 - 1, 90
    idx[2, 1, 50:] = 10 ** 9  # behind the count: not looked at
    cnt[2, 1], cnt[2, 0], cnt[1, 0] = 50, -3, k + 5
    table[0, 2] = len(pool) + 7
    kv.page_table.copy_(_dev(table))
    q = _rows((3, G * h, d), torch.bfloat16, 6, 1.5)
    r = ssd_kv4_draft_attn(kv, q.to(DEV), _dev(idx), _dev(cnt), 0.1)
    torch.cuda.synchronize()
    assert ssd_status() == binding.FAULT_INDEX | binding.FAULT_KMAX | binding.FAULT_PAGE
    # An entry that is not there counts as a token of zeros.
    bad = np.zeros(table.shape, bool)
    bad[0, 2] = True
    zpool, ztable = _with_zero_page(pool, table, bad)
    ztable = np.concatenate([ztable, np.full((3, 1), len(pool), np.int32)], 1)
    beyond = (ztable.shape[1] - 1) * page
    zidx = np.where((idx < 0) | (idx >= np.array(lens)[:, None, None]), beyond, idx)
    zcnt = np.clip(cnt, 0, k)
    q64 = q.double().numpy()
    X, A = _bounds(zpool, ztable, lens, q64, d, 0.1, 1, 1)
    _check(r, _kv4.draft(zpool, ztable, q64, zidx, zcnt, d, 0.1), A, X, False, G, "draft")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_of_nan_and_infinities(dtype):
    _gpu.lib()
    h, d, page = 2, 64, 16
    kv, pool, table = _cache([5, 30], h, d, page, room=3, seed=24)
    x = torch.randn((2, 2, 3, h, d), generator=torch.Generator().manual_seed(1)).to(dtype)
    x[0, 0, 0, 0, 3] = math.nan
    x[0, 0, 1, 1, 16:32] = math.nan
    x[1, 0, 2, 0, 5] = math.inf
    x[1, 1, 0, 1, 60] = -math.inf
    x[1, 1, 1, 1, 60:62] = torch.tensor([-math.inf, math.nan], dtype=dtype)
    want = pool.copy()
    for w in range(2):
        c, e = _kv4.quantise(x[w].double().numpy())
        for b, n in enumerate([5, 30]):
            for j in range(3):
                for g in range(h):
                    _kv4.write_row(want, table[b, (n + j) // page], w, g, (n + j) % page, d, c[b, j, g], e[b, j, g])
    ssd_kv4_append(kv, x[0].contiguous().to(DEV), x[1].contiguous().to(DEV))
    torch.cuda.synchronize()
    assert ssd_status() == binding.FAULT_VALUE
    np.testing.assert_array_equal(kv.pool.cpu().numpy(), want)
    ssd_kv4_append(kv, *(torch.nan_to_num(t, 0, 1, -1).contiguous().to(DEV) for t in x))
    torch.cuda.synchronize()
    assert ssd_status() == 0


@pytest.mark.parametrize("mul", [1.0, 2.0 ** -20, 2.0 ** 32])
def test_every_bf16_as_the_largest_of_a_group(mul):
    """Scales of all 32640 finite magnitudes, and codes of multiples and neighbours of e2m1's ties under them."""
    _gpu.lib()
    d, page, h = 128, 64, 1
    top = np.arange(0, 0x7f80, dtype=np.uint16).view(np.int16)
    rng = np.random.default_rng(3)
    frac = rng.choice([0.25 / 6, 0.75 / 6, 1.25 / 6, 1.75 / 6, 2.5 / 6, 3.5 / 6, 5.0 / 6], (len(top), 16)) * rng.choice([1.0, -1.0], (len(top), 16))
    m = torch.from_numpy(top.copy()).view(torch.bfloat16)
    x = (m.double()[:, None] * torch.from_numpy(frac)).to(torch.bfloat16)
    near = torch.from_numpy(rng.integers(-1, 2, x.shape).astype(np.int16))
    x = torch.where(x.abs() > 1e-30, (x.view(torch.int16) + near).view(torch.bfloat16), x)
    x = torch.where(x.abs() > m[:, None], m[:, None], x)
    x[:, 5] = m
    n = len(top) // 8
    rows = x.view(1, n, h, d)
    kv, pool, table = _cache([0], h, d, page, room=n, seed=34, k_scale=mul, v_scale=mul)
    ssd_kv4_append(kv, rows.to(DEV), rows.flip(1).contiguous().to(DEV))
    k, v = ssd_kv4_read(kv, kv.seq_lens, n, dtype=torch.float32)
    torch.cuda.synchronize()
    assert ssd_status() == 0
    c, s = _kv4.quantise(rows.double().numpy(), mul)
    want = _kv4.values(c, s, mul)
    np.testing.assert_array_equal(k.double().cpu().numpy(), want)
    np.testing.assert_array_equal(v.double().cpu().numpy(), want[:, ::-1])
    got = kv.pool.cpu().numpy()[table[0, 0], 0, 0].reshape(-1)  # bytes of the first page's K rows
    want = np.zeros((page, d // 2), np.uint8)
    want[:] = c[0, :page, 0, 0::2] | (c[0, :page, 0, 1::2] << 4)
    np.testing.assert_array_equal(got[:page * d // 2], want.reshape(-1))


def test_append_and_read_out_of_range():
    _gpu.lib()
    h, d, page = 2, 128, 16
    lens = [5, 30, 60, 20, -1, 16]
    kv, pool, table = _cache([max(n, 0) for n in lens], h, d, page, room=8, seed=25)
    kv = KV4Cache(kv.pool, kv.page_table, _dev(lens), 64)
    table[3, 1] = len(pool)
    table[5, 0] = -1  # of earlier tokens: not looked at
    kv.page_table.copy_(_dev(table))
    counts = [9, -1, 5, 4, 2, 8]  # more than n_new; negative; past 64; a bad page; a bad length; good
    x = torch.randn((2, 6, 8, h, d), generator=torch.Generator().manual_seed(1))
    want = pool.copy()
    for w in range(2):
        c, e = _kv4.quantise(x[w].double().numpy())
        for j in range(8):
            for g in range(h):
                _kv4.write_row(want, table[5, 1], w, g, j, d, c[5, j, g], e[5, j, g])
    ssd_kv4_append(kv, x[0].contiguous().to(DEV), x[1].contiguous().to(DEV), counts=_dev(counts))
    torch.cuda.synchronize()
    assert ssd_status() == binding.FAULT_SEQLEN | binding.FAULT_PAGE
    np.testing.assert_array_equal(kv.pool.cpu().numpy(), want)
    first = [-1, 0, 60, 10, 0, 16]
    counts = [2, 9, 5, 8, -1, 3]
    k, v = ssd_kv4_read(kv, _dev(first), 8, counts=_dev(counts), dtype=torch.float32)
    torch.cuda.synchronize()
    assert ssd_status() == binding.FAULT_SEQLEN | binding.FAULT_PAGE
    for w, got in ((0, k), (1, v)):
        ref = np.zeros((6, 8, h, d))
        for g in range(h):
            ref[3, :6, g] = _kv4.read_rows(want, table[3], w, g, range(10, 16), d)  # page 1 is bad
            ref[5, :3, g] = _kv4.read_rows(want, table[5], w, g, range(16, 19), d)
        np.testing.assert_array_equal(got.double().cpu().numpy(), ref)


@form
@pytest.mark.parametrize("order", ["up", "down", "spikes"])
@pytest.mark.parametrize("types", ["bf16-bf16", "bf16-f32", "f32-f32"])
def test_logits_that_grow_along_the_context(form, order, types):
    """The softmax's reference moves many times, or the first tiles' weights vanish altogether."""
    _gpu.lib()
    h, G, d, nc = form
    n, page = 900, 16
    qt, ot = (torch.bfloat16 if t == "bf16" else torch.float32 for t in types.split("-"))
    kv, pool, table = _cache([n], h, d, page, seed=26)
    ramp = np.linspace(-1, 1, n) * (1 if order == "up" else -1)
    if order == "spikes":
        ramp = np.where(np.arange(n) % 97 == 3, np.arange(n) / n, -1.0)
    rng = np.random.default_rng(5)
    dirs = np.sign(rng.standard_normal(d))
    for g in range(h):
        c, s = _kv4.quantise(ramp[:, None] * dirs * 4 + 0.1 * rng.standard_normal((n, d)))
        for t in range(n):
            _kv4.write_row(pool, table[0, t // page], 0, g, t % page, d, c[t], s[t])
    kv.pool.copy_(torch.from_numpy(pool))
    q = (torch.from_numpy(dirs).float() * (0.7 + 0.3 * torch.rand((1, nc, G * h, 1), generator=torch.Generator().manual_seed(2)))).to(qt)
    scale = 60.0 / (4 * d)  # logits from about -60 to 60
    r = ssd_kv4_verify_attn(kv, q.to(DEV), nc, scale, out_dtype=ot)
    torch.cuda.synchronize()
    assert ssd_status() == 0
    q64 = q.double().numpy()
    X, A = _bounds(pool, table, [n], q64, d, scale, 1, 1)
    _check(r, _kv4.verify(pool, table, [n], q64, d, scale), A, X, ot == torch.bfloat16, nc * G, order)


@pytest.mark.parametrize("scale", [0.0, -0.125])
@form
def test_zero_and_negative_scale(form, scale):
    _gpu.lib()
    h, G, d, nc = form
    kv, pool, table = _cache([150, 33], h, d, 32, seed=27)
    q = _rows((2, nc, G * h, d), torch.bfloat16, 8)
    r = ssd_kv4_verify_attn(kv, q.to(DEV), nc, scale)
    q64 = q.double().numpy()
    X, A = _bounds(pool, table, [150, 33], q64, d, abs(scale), 1, 1)
    _check(r, _kv4.verify(pool, table, [150, 33], q64, d, scale), A, X, False, nc * G, "verify")
    assert ssd_status() == 0


@form
@pytest.mark.parametrize("lens", [[0, 7, 0, 31, 1, 0, 260, 5] * 20, [6000], [0, 0, 0]], ids=["ragged", "long", "empty"])
def test_units_dealt_out_to_blocks(form, lens):
    """Hundreds of units of a tile or none, and one that many blocks share."""
    _gpu.lib()
    h, G, d, nc = form
    if len(lens) == 1:
        h = 1
    kv, pool, table = _cache(lens, h, d, 16, seed=28)
    q = _rows((len(lens), nc, G * h, d), torch.bfloat16, 9, 1.5)
    r = ssd_kv4_verify_attn(kv, q.to(DEV), nc, 0.1)
    torch.cuda.synchronize()
    assert ssd_status() == (binding.FAULT_SEQLEN if min(lens) < nc else 0)
    q64 = q.double().numpy()
    X, A = _bounds(pool, table, lens, q64, d, 0.1, 1, 1)
    _check(r, _kv4.verify(pool, table, lens, q64, d, 0.1), A, X, False, nc * G, "verify")
    again = ssd_kv4_verify_attn(kv, q.to(DEV), nc, 0.1)
    for name in ("out", "lse"):
        assert torch.equal(r[name], again[name]), name  # the order of the sums does not depend on timing
    ssd_status()


@form
def test_tensors_aligned_to_16_bytes_only(form):
    _gpu.lib()
    h, G, d, nc = form
    lens = [37, 260]
    kv, pool, table = _cache(lens, h, d, 16, room=nc, seed=29)

    def shifted(t):
        n = 16 // t.element_size()
        buf = torch.zeros(t.numel() + n, dtype=t.dtype, device=DEV)
        out = buf[n:].view(t.shape)
        out.copy_(t)
        assert out.data_ptr() % 32 == 16
        return out

    kv2 = KV4Cache(shifted(kv.pool), kv.page_table, kv.seq_lens.clone(), kv.max_seq_len)
    q = _rows((2, nc, G * h, d), torch.bfloat16, 5, 1.5).to(DEV)
    qf = q.float()
    rows = _rows((2, 2, nc, h, d), torch.bfloat16, 6).to(DEV)
    idx = torch.arange(30, dtype=torch.int32, device=DEV).expand(2, h, 30).contiguous()
    cnt = torch.tensor([[30] * h, [11] * h], dtype=torch.int32, device=DEV)
    for cache, f in ((kv, lambda t: t), (kv2, shifted)):
        ssd_kv4_append(cache, f(rows[0]), f(rows[1]))
    assert torch.equal(kv.pool, kv2.pool)
    a, b = (ssd_kv4_read(c, c.seq_lens, nc, k=f(torch.zeros_like(rows[0])), v=f(torch.zeros_like(rows[0])))
            for c, f in ((kv, lambda t: t), (kv2, shifted)))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and not torch.equal(a[0], a[1])
    for x in (q, qf):
        a, b = (ssd_kv4_verify_attn(c, f(x), nc, 0.1, out=f(torch.zeros_like(qf))) for c, f in ((kv, lambda t: t), (kv2, shifted)))
        for name in ("out", "lse", "scores"):
            n = [slice(None)] * a[name].dim()
            if name == "scores":
                n[2] = slice(0, 37)
            assert torch.equal(a[name][tuple(n)], b[name][tuple(n)]), name
        if G <= 16:
            a, b = (ssd_kv4_draft_attn(c, f(x[:, 0].contiguous()), idx, cnt, 0.1, out=f(torch.zeros_like(qf[:, 0].contiguous())))
                    for c, f in ((kv, lambda t: t), (kv2, shifted)))
            assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    assert ssd_status() == 0


@pytest.mark.parametrize("G,nc", [(4, 1), (4, 5)])
def test_pool_past_4_gb(G, nc):
    """Pages whose byte offsets pass 32 bits: the same bits as in a small pool."""
    _gpu.lib()
    h, d, page, n = 8, 128, 16, 150
    n_pages = (5 << 30) // (h * page * 144)
    kv, pool, table = _cache([n], h, d, page, room=8, seed=30)
    used = table[0][table[0] >= 0]
    far = torch.empty((n_pages, 2, h, page, 72), dtype=torch.uint8, device=DEV)
    ftable = np.full_like(table, -1)
    ftable[0, :len(used)] = n_pages - 1 - np.arange(len(used))
    far[torch.from_numpy(ftable[0, :len(used)].astype(np.int64)).to(DEV)] = kv.pool[torch.from_numpy(used.astype(np.int64)).to(DEV)]
    big = KV4Cache(far, _dev(ftable), kv.seq_lens.clone(), kv.max_seq_len)
    q = _rows((1, nc, G * h, d), torch.bfloat16, 5).to(DEV)
    rows = _rows((2, 1, 8, h, d), torch.bfloat16, 6).to(DEV)
    idx = torch.arange(0, 120, 3, dtype=torch.int32, device=DEV).expand(1, h, 40).contiguous()
    cnt = torch.full((1, h), 40, dtype=torch.int32, device=DEV)
    results = []
    for c in (kv, big):
        ssd_kv4_append(c, rows[0], rows[1])
        k, v = ssd_kv4_read(c, torch.zeros_like(c.seq_lens), n + 8)
        scores = torch.zeros((1, h, c.max_seq_len), device=DEV)
        r = ssd_kv4_verify_attn(c, q, nc, 0.1, scores=scores)
        s = ssd_kv4_draft_attn(c, q[:, 0].contiguous(), idx, cnt, 0.1)
        results.append([k, v, r["out"], r["lse"], scores, s["out"], s["lse"]])
    for i, (x, y) in enumerate(zip(*results)):
        assert torch.equal(x, y), i
    # Compaction out of the far pages into near ones.
    near = KV4Cache(torch.zeros_like(kv.pool), kv.page_table, torch.zeros_like(kv.seq_lens), kv.max_seq_len)
    row = torch.zeros(1, dtype=torch.int32, device=DEV)
    ssd_kv_compact(big, near, row, row, idx, cnt)
    k, _ = ssd_kv4_read(near, row, 40)
    assert torch.equal(k, results[0][0][:, 0:120:3])
    assert near.seq_lens.item() == 40
    assert ssd_status() == 0
    del far, big
    torch.cuda.empty_cache()


@form
def test_graphs_and_streams(form):
    """Two captured graphs (each with a workspace of its own, or one that both share in turn) and calls on two
    streams at once give the bits of the plain calls."""
    _gpu.lib()
    h, G, d, nc = form
    lens = [[600, 20, 411], [33, 1200, 700]]
    caches = [_cache(n, h, d, 16, seed=31 + i)[0] for i, n in enumerate(lens)]
    q = _rows((3, nc, G * h, d), torch.bfloat16, 5).to(DEV)
    qd = q[:, 0].contiguous()
    idx = torch.arange(20, dtype=torch.int32, device=DEV).expand(3, h, 20).contiguous()
    cnt = torch.full((3, h), 20, dtype=torch.int32, device=DEV)

    def call(kv, buf, ws=None, stream=None):
        ssd_kv4_verify_attn(kv, q, nc, 0.1, out=buf[0], lse=buf[1], scores=buf[2], workspace=ws, stream=stream)
        ssd_kv4_draft_attn(kv, qd, idx, cnt, 0.1, out=buf[3], lse=buf[4], workspace=ws, stream=stream)

    def buffers(kv):
        return [torch.zeros(s, device=DEV) for s in (q.shape, q.shape[:3], (3, h, kv.max_seq_len), qd.shape, qd.shape[:2])]

    want = [buffers(kv) for kv in caches]
    for kv, buf in zip(caches, want):
        call(kv, buf)
    shared = Workspace()
    for kv in caches:
        call(kv, buffers(kv), shared)  # sizes it
    for ws in (None, shared):
        got = [buffers(kv) for kv in caches]
        graphs = []
        for kv, buf in zip(caches, got):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                call(kv, buf, ws)
            graphs.append(g)
        for _ in range(3):
            for buf in got:
                for t in buf:
                    t.fill_(7.0)
            for t in (got[0][2], got[1][2]):
                t.zero_()
            for g in graphs:
                g.replay()
            for a, b in zip(want, got):
                for i, (x, y) in enumerate(zip(a, b)):
                    assert torch.equal(x, y), i
    streams = [torch.cuda.Stream() for _ in caches]
    got = [buffers(kv) for kv in caches]
    torch.cuda.synchronize()
    for _ in range(20):
        for kv, buf, s in zip(caches, got, streams):
            call(kv, buf, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for i, (x, y) in enumerate(zip(a, b)):
            assert torch.equal(x, y), i
    assert ssd_status() == 0


def test_empty_calls():
    _gpu.lib()
    h, d = 2, 128
    kv, _, _ = _cache([20], h, d, 16, seed=33)
    none = KV4Cache(kv.pool, kv.page_table[:0].contiguous(), kv.seq_lens[:0].contiguous(), 32)
    r = ssd_kv4_verify_attn(none, torch.empty((0, 5, 8, d), dtype=torch.bfloat16, device=DEV), 5, 0.1)
    assert r["out"].shape == (0, 5, 8, d)
    z = torch.empty((0, h, 4), dtype=torch.int32, device=DEV)
    ssd_kv4_draft_attn(none, torch.empty((0, 8, d), dtype=torch.bfloat16, device=DEV), z, z[:, :, 0].contiguous(), 0.1)
    rows = torch.empty((0, 3, h, d), dtype=torch.bfloat16, device=DEV)
    ssd_kv4_append(none, rows, rows)
    rows = torch.empty((1, 0, h, d), dtype=torch.bfloat16, device=DEV)
    ssd_kv4_append(kv, rows, rows)
    k, v = ssd_kv4_read(kv, kv.seq_lens, 0)
    assert k.shape == (1, 0, h, d)
    # A list without entries, and one without room for any.
    q = torch.ones((1, 8, d), dtype=torch.bfloat16, device=DEV)
    for k_max in (0, 5):
        idx = torch.zeros((1, h, k_max), dtype=torch.int32, device=DEV)
        r = ssd_kv4_draft_attn(kv, q, idx, torch.zeros((1, h), dtype=torch.int32, device=DEV), 0.1)
        assert not r["out"].any() and (r["lse"] == -math.inf).all()
    assert ssd_status() == 0
