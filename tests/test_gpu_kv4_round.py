"""The 4-bit cache's calls together, as a server runs them: prompts appended, requests branched, rounds of
append, verify, select and drafts through SpecRound, rejected tokens rolled back, branches given back, a
context evicted down to its critical tokens.  Definitions and tolerances are those of test_gpu_kv4; the plain
side keeps every row's values itself and never reads the library's pool."""

import numpy as np
import pytest
import torch

from sparse_self_speculative_verify_gb300 import (KV4Cache, PagePool, SpecRound, Workspace, binding, ssd_kv4_append,
                                                 ssd_kv4_read, ssd_kv_advance, ssd_kv_compact, ssd_kv_fork, ssd_kv_release,
                                                 ssd_kv_reserve, ssd_status)
from tests import _gpu, _kv4
from tests.test_gpu_kv4 import _check, _rows

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _bounds(rows, q, scale):
    X = max((float((np.abs(K) @ np.abs(q[b]).reshape(-1, K.shape[1]).T).max()) * scale
             for b, heads in enumerate(rows) for K, _ in heads if len(K)), default=0.0)
    return X, max((float(np.abs(V).max()) for heads in rows for _, V in heads if len(V)), default=0.0)


def _verify(rows, q, scale):
    """rows[b][g] = (K, V) values [L, d]."""
    B, nc, hq, d = q.shape
    h = len(rows[0])
    G = hq // h
    out, lse, scores = np.zeros(q.shape), np.zeros(q.shape[:3]), []
    for b, heads in enumerate(rows):
        sc = np.zeros((h, len(heads[0][0])))
        for g, (K, V) in enumerate(heads):
            lim = np.repeat([len(K) - nc + 1 + i for i in range(nc)], G)
            o, z, P = _kv4.attend(q[b, :, g * G:(g + 1) * G].reshape(-1, d), K, V, lim, scale)
            out[b, :, g * G:(g + 1) * G], lse[b, :, g * G:(g + 1) * G] = o.reshape(nc, G, d), z.reshape(nc, G)
            sc[g] = P.sum(0)
        scores.append(sc)
    return {"out": out, "lse": lse, "scores": scores}


def _draft(rows, q, idx, cnt, scale):
    h = len(rows[0])
    G = q.shape[1] // h
    out, lse = np.zeros(q.shape), np.zeros(q.shape[:2])
    for b, heads in enumerate(rows):
        for g, (K, V) in enumerate(heads):
            t = idx[b, g, :cnt[b, g]]
            o, z, _ = _kv4.attend(q[b, g * G:(g + 1) * G], K[t], V[t], [len(t)] * G, scale)
            out[b, g * G:(g + 1) * G], lse[b, g * G:(g + 1) * G] = o, z
    return {"out": out, "lse": lse}


def _stored(x, scale):
    """[n, h, d] -> per head the values the cache keeps."""
    c, s = _kv4.quantise(x.double().numpy(), scale)
    return [_kv4.values(c[:, g], s[:, g], scale) for g in range(x.shape[1])]


class _Plain:
    """Rows of values per request and head."""

    def __init__(self, batch, h, d):
        self.rows = [[(np.zeros((0, d)), np.zeros((0, d))) for _ in range(h)] for _ in range(batch)]

    def append(self, b, k, v, ks, vs):
        self.rows[b] = [(np.concatenate([K, a]), np.concatenate([V, c]))
                        for (K, V), a, c in zip(self.rows[b], _stored(k, ks), _stored(v, vs))]

    def keep(self, b, n):
        self.rows[b] = [(K[:n], V[:n]) for K, V in self.rows[b]]


@pytest.mark.parametrize("d,G,n_cand,page", [(128, 4, 5, 16), (128, 4, 2, 8), (64, 8, 4, 32)])
def test_serving_with_branches_rounds_and_eviction(d, G, n_cand, page):
    _gpu.lib()
    h, batch, k_max, ks, vs = 2, 8, 24, 0.5, 2.0
    prompts = [70, 133, 45]
    cap = 12 if page > 8 else 32
    kv = KV4Cache(torch.randint(0, 256, KV4Cache.pool_shape(90, h, page, d), dtype=torch.uint8, device=DEV),
                  torch.full((batch, cap), -1, dtype=torch.int32, device=DEV), _i32([0] * batch), min(cap * page, 256), ks, vs)
    pages = PagePool.from_table(kv.page_table, 90)
    plain = _Plain(batch, h, d)
    gen = torch.Generator().manual_seed(3)

    def rows(n, dtype=torch.bfloat16):
        return (torch.randn((2, batch, n, h, d), generator=gen) * 1.5).to(dtype)

    def append(counts, n):
        x = rows(n)
        ssd_kv_reserve(kv, pages, _i32(counts))
        ssd_kv4_append(kv, x[0].contiguous().to(DEV), x[1].contiguous().to(DEV), counts=_i32(counts))
        ssd_kv_advance(kv.seq_lens, _i32(counts), kv.max_seq_len)
        for b, c in enumerate(counts):
            plain.append(b, x[0, b, :c], x[1, b, :c], ks, vs)

    append(prompts + [0] * 5, max(prompts))
    # Rows 3 .. 7 branch off rows 0, 0, 1, 1, 1; their pages are shared until they are written.
    src, dst = [0, 0, 1, 1, 1], [3, 4, 5, 6, 7]
    ssd_kv_fork(kv, pages, _i32(src), _i32(dst))
    for s, t in zip(src, dst):
        plain.rows[t] = list(plain.rows[s])
    held = int((pages.refs > 0).sum())
    rnd = SpecRound(kv, G * h, n_cand, k_max)
    lens = [len(r[0][0]) for r in plain.rows]
    assert held == sum(-(-n // page) for n in prompts)
    for step in range(3):
        append([n_cand] * batch, n_cand)
        q = _rows((batch, n_cand, G * h, d), torch.bfloat16, 40 + step, 1.5)
        qd = _rows((3, batch, G * h, d), torch.bfloat16, 50 + step, 1.5)
        k_req = [5, 24, 9, 24, 1, 30, 0, 11]
        outs = torch.empty(qd.shape, dtype=torch.float32, device=DEV)
        rnd.run(q.to(DEV), qd.to(DEV), _i32(np.minimum(k_req, k_max)), draft_outs=outs, fused_select=step == 1)
        torch.cuda.synchronize()
        assert ssd_status() == 0
        ref = _verify(plain.rows, q.double().numpy(), rnd.scale)
        X, A = _bounds(plain.rows, q.double().numpy(), rnd.scale)
        lens = [len(r[0][0]) for r in plain.rows]
        assert kv.seq_lens.tolist() == lens
        sc = rnd.scores.clone()
        for b, n in enumerate(lens):
            sc[b, :, n:] = 0  # entries past the end keep older calls' values
        _check({"out": rnd.out_v, "lse": rnd.lse_v, "scores": sc}, ref, A, X, False, n_cand * G, "verify")
        idx = rnd.idx.view(batch, h, k_max).cpu().numpy()
        cnt = rnd.cnt.view(batch, h).cpu().numpy()
        own = rnd.scores.cpu().numpy()
        for b, n in enumerate(lens):
            K = min(k_req[b], k_max, n)
            for g in range(h):
                assert cnt[b, g] == K
                want = np.sort(np.lexsort((np.arange(n), -own[b, g, :n]))[:K])
                np.testing.assert_array_equal(idx[b, g, :K], want)
        for j in range(3):
            ref = _draft(plain.rows, qd[j].double().numpy(), idx, cnt, rnd.scale)
            X, A = _bounds(plain.rows, qd[j].double().numpy(), rnd.scale)
            _check({"out": outs[j]}, ref, A, X, False, G, f"draft {j}")
        # Row b accepts b % (n_cand + 1) tokens; the rest, and the pages behind, go back.
        keep = [n - n_cand + b % (n_cand + 1) for b, n in enumerate(lens)]
        ssd_kv_release(kv, pages, _i32(keep))
        for b, n in enumerate(keep):
            plain.keep(b, n)
    # Branches 3 .. 6 are given up; row 1 keeps its selected tokens only, in row 3.
    lens = [len(r[0][0]) for r in plain.rows]
    ssd_kv_release(kv, pages, _i32([-1, -1, -1, 0, 0, 0, 0, -1]))
    for b in (3, 4, 5, 6):
        plain.keep(b, 0)
    idx = rnd.idx.view(batch, h, k_max)[1:2].clamp(max=lens[1] - 1).contiguous()
    ssd_kv_reserve(kv, pages, _i32([0, 0, 0, k_max, 0, 0, 0, 0]))
    ssd_kv_compact(kv, kv, _i32([1]), _i32([3]), idx, _i32([[k_max] * h]), pages=pages)
    t = idx[0].cpu().numpy()
    plain.rows[3] = [(K[t[g]], V[t[g]]) for g, (K, V) in enumerate(plain.rows[1])]
    append([n_cand, 0, n_cand, n_cand, 0, 0, 0, n_cand], n_cand)
    q = _rows((batch, 1, G * h, d), torch.float32, 60, 1.5)
    one = SpecRound(kv, G * h, 1, k_max)
    one.verify(q.to(DEV))
    topk = one.draft_oracle_topk(q[:, 0].contiguous().to(DEV), _i32([k_max] * batch))
    torch.cuda.synchronize()
    ref = _verify(plain.rows, q.double().numpy(), one.scale)
    X, A = _bounds(plain.rows, q.double().numpy(), one.scale)
    _check({"out": one.out_v, "lse": one.lse_v, "scores": one.scores}, ref, A, X, False, G, "after eviction")
    assert torch.equal(topk["dense"], one.out_v[:, 0])
    idx, cnt = topk["idx"].view(batch, h, k_max).cpu().numpy(), topk["cnt"].view(batch, h).cpu().numpy()
    _check({"out": topk["out"], "lse": topk["lse"]}, _draft(plain.rows, q[:, 0].double().numpy(), idx, cnt, one.scale), A, X,
           False, G, "oracle top-k")
    assert ssd_status() == binding.FAULT_SEQLEN  # the given-up rows hold fewer tokens than candidates
    # What the cache holds, read back, is what the plain side holds.
    longest = max(len(r[0][0]) for r in plain.rows)
    k, v = ssd_kv4_read(kv, _i32([0] * batch), longest, counts=kv.seq_lens, dtype=torch.float32)
    for b in range(batch):
        for g in range(h):
            for got, want in zip((k, v), plain.rows[b][g]):
                np.testing.assert_array_equal(got[b, :len(want), g].double().cpu().numpy(), want)
    # Every page is given back.
    ssd_kv_release(kv, pages, _i32([0] * batch))
    assert not pages.refs.any() and (kv.page_table == -1).all() and not kv.seq_lens.any()
    assert ssd_status() == 0


def test_a_captured_round_replayed():
    """reserve -> append -> advance -> verify -> select -> drafts -> roll back in one graph: every replay gives
    the bits of the calls made one by one on a copy of the cache."""
    _gpu.lib()
    h, G, d, n_cand, page, k_max, batch = 2, 4, 128, 5, 16, 20, 3
    ws = Workspace()

    def make():
        g = torch.Generator(device=DEV).manual_seed(4)
        kv = KV4Cache(torch.randint(0, 256, KV4Cache.pool_shape(40, h, page, d), dtype=torch.uint8, device=DEV, generator=g),
                      torch.full((batch, 10), -1, dtype=torch.int32, device=DEV), _i32([0] * batch), 160)
        pages = PagePool.from_table(kv.page_table, 40)
        x = torch.randn((2, batch, 100, h, d), device=DEV, generator=g).bfloat16()
        ssd_kv_reserve(kv, pages, _i32([100, 64, 3]))
        ssd_kv4_append(kv, x[0].contiguous(), x[1].contiguous(), counts=_i32([100, 64, 3]))
        ssd_kv_advance(kv.seq_lens, _i32([100, 64, 3]), 160)
        rnd = SpecRound(kv, G * h, n_cand, k_max, workspace=ws)
        rnd.scores.zero_()
        return kv, pages, rnd

    new = torch.randn((2, batch, n_cand, h, d), device=DEV).bfloat16()
    q = torch.randn((batch, n_cand, G * h, d), device=DEV).bfloat16()
    qd = torch.randn((2, batch, G * h, d), device=DEV).bfloat16()
    counts, back, k_req = _i32([n_cand] * batch), _i32([-2, -5, 0]), _i32([20, 7, 3])

    def step(kv, pages, rnd, outs):
        ssd_kv_reserve(kv, pages, counts, workspace=ws)
        ssd_kv4_append(kv, new[0], new[1], counts=counts)
        ssd_kv_advance(kv.seq_lens, counts, kv.max_seq_len)
        rnd.run(q, qd, k_req, draft_outs=outs)
        ssd_kv_advance(kv.seq_lens, back, kv.max_seq_len)

    a, b = make(), make()
    outs = [torch.zeros(qd.shape, device=DEV) for _ in range(2)]
    step(*make(), torch.zeros(qd.shape, device=DEV))  # sizes the workspace
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(*b, outs[1])
    for _ in range(4):
        step(*a, outs[0])
        g.replay()
        pairs = [(a[0].pool, b[0].pool), (a[0].page_table, b[0].page_table), (a[0].seq_lens, b[0].seq_lens),
                 (a[1].refs, b[1].refs), (outs[0], outs[1])]
        pairs += [(getattr(a[2], n), getattr(b[2], n)) for n in ("out_v", "lse_v", "scores", "lse_d", "cnt")]
        for i, (x, y) in enumerate(pairs):
            assert torch.equal(x, y), i
    assert a[0].seq_lens.tolist() == [100 + 4 * 3, 64, 3 + 4 * 5]
    assert ssd_status() == 0
