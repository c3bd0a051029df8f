"""The 4-bit and the page calls from several host threads at once, all on the default stream: the same bits as from
one thread after the other."""

import threading

import pytest
import torch

from sparse_self_speculative_verify_gb300 import (Workspace, binding, ssd_kv4_draft_attn, ssd_kv4_verify_attn, ssd_kv_fork,
                                                 ssd_kv_release, ssd_kv_reserve, ssd_status)
from tests import _gpu
from tests.test_gpu_kv4 import _cache, _rows
from tests.test_gpu_kv4_long import _cache as _shared, _tokens
from tests.test_gpu_pages import _i32, _make, _same

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _long(kind, h, d):
    return _shared(_tokens(kind, h, d)[0], 1)


def _run(work, n):
    """work(i) for every i < n, each in a thread of its own, all started together."""
    errors, start = [], threading.Barrier(n)

    def body(i):
        try:
            torch.cuda.set_device(0)
            start.wait()
            work(i)
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=body, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("shared", [False, True], ids=["stream's workspace", "one Workspace"])
def test_attention_from_two_threads(shared):
    """Requests that many blocks share (their parts go through the workspace, to a join and the scores' pass), so many
    calls that the launch queue fills: a thread then waits inside a call, between its launches, and the other goes on."""
    _gpu.lib()
    h, G, d, nc = 2, 4, 128, 5
    caches = [_long(kind, h, d) for kind in ("spread", "positive")]
    q = [_rows((1, nc, G * h, d), torch.bfloat16, 52 + i, 1.5).to(DEV) for i in range(2)]
    idx = torch.arange(0, 32768, 2, dtype=torch.int32, device=DEV).expand(1, h, 16384).contiguous()
    cnt = torch.full((1, h), 16384, dtype=torch.int32, device=DEV)
    ws = Workspace() if shared else None

    def call(i):
        r = ssd_kv4_verify_attn(caches[i], q[i], nc, 0.1, workspace=ws)
        s = ssd_kv4_draft_attn(caches[i], q[i][:, 0].contiguous(), idx, cnt, 0.1, workspace=ws)
        return [r["out"], r["lse"], r["scores"], s["out"], s["lse"]]

    want = [call(0), call(1)]
    torch.cuda.synchronize()
    got = [[], []]
    torch.cuda._sleep(1_000_000_000)  # half a second, in which the queue fills

    def work(i):
        for _ in range(700):
            got[i].append(call(i))

    _run(work, 2)
    assert ssd_status() == 0
    wrong = [sum(not all(torch.equal(x, y) for x, y in zip(r, want[i])) for r in got[i]) for i in range(2)]
    assert wrong == [0, 0]


def test_workspace_that_grows_under_another_thread(monkeypatch):
    _gpu.lib()
    monkeypatch.setattr(binding, "_STREAM_WS", {})
    h, G, d = 1, 4, 128
    kv, _, _ = _cache([2000], h, d, 16, seed=55)
    qs = [_rows((1, nc, G * h, d), torch.bfloat16, 56, 1.5).to(DEV) for nc in (1, 2, 5, 8)]
    want = [ssd_kv4_verify_attn(kv, q, q.shape[1], 0.1) for q in qs]
    torch.cuda.synchronize()
    wrong = [0, 0]

    def work(i):
        for _ in range(40):
            if i == 0:
                binding._STREAM_WS.clear()
            for q, w in zip(qs, want):
                r = ssd_kv4_verify_attn(kv, q, q.shape[1], 0.1)
                wrong[i] += not all(torch.equal(r[k], w[k]) for k in w)

    _run(work, 2)
    assert ssd_status() == 0 and wrong == [0, 0]


def test_branching_from_two_threads():
    """Two caches of different sizes, each branched by its thread: what a reserve copies is its own."""
    _gpu.lib()
    made = [_make("bf16", [37, 50, 3], 16, rows=9, spare=40, cap=6),
            _make("bf16", [5, 90, 20, 33], 8, rows=8, spare=60, seed=7, cap=14)]

    def args(P):
        n = len(P.lens)
        live = [b for b in range(n) if P.lens[b]]
        empty = [b for b in range(n) if not P.lens[b]]
        src = [live[i % len(live)] for i in range(len(empty))]
        keep = [-1 if b in live else 0 for b in range(n)]
        return keep, src, empty, [5] * n

    lists = [args(m[2]) for m in made]
    dev = [[_i32(x) for x in a] for a in lists]
    torch.cuda.synchronize()

    def work(i):
        kv, pages, _ = made[i]
        for _ in range(200):
            ssd_kv_release(kv, pages, dev[i][0])
            ssd_kv_fork(kv, pages, dev[i][1], dev[i][2])
            ssd_kv_reserve(kv, pages, dev[i][3])

    for (_, _, P), (keep, src, dst, counts) in zip(made, lists):  # what one thread leaves, by the plain definition
        for _ in range(200):
            P.release(keep), P.fork(src, dst), P.reserve(counts)
        assert not P.faults
    _run(work, 2)
    for kv, pages, P in made:
        _same(kv, pages, P)
        P.check()
