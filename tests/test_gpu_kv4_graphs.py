"""Workspaces of the 4-bit calls under stream capture: not sized before, and grown after."""

import pytest
import torch

from sparse_self_speculative_verify_gb300 import SpecRound, Workspace, binding, ssd_kv4_verify_attn, ssd_status
from tests import _gpu
from tests.test_gpu_kv4 import _rows
from tests.test_gpu_kv4_long import _cache, _tokens

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
H, G, D = 2, 4, 128


def _call(kv, q, ws, out):
    r = ssd_kv4_verify_attn(kv, q, q.shape[1], 0.1, out=out[0], lse=out[1], scores=out[2], workspace=ws)
    return [r["out"], r["lse"], r["scores"]]


def _out(q, kv):
    return [torch.zeros(q.shape, device=DEV), torch.zeros(q.shape[:3], device=DEV), torch.zeros((1, H, kv.max_seq_len), device=DEV)]


def _equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_capture_with_a_workspace_that_no_call_has_sized():
    """The graph's calls take memory of the graph; an eager call before its first replay finds counters that are zero."""
    _gpu.lib()
    kv = _cache(_tokens("spread", H, D)[0], 1)
    q = _rows((1, 1, G * H, D), torch.bfloat16, 61, 1.5).to(DEV)  # mma.sync: the last block of a unit joins its parts
    want = [t.clone() for t in _call(kv, q, None, _out(q, kv))]
    torch.cuda.synchronize()
    # A graph pool whose memory holds something.
    dirty = torch.cuda.CUDAGraph()
    with torch.cuda.graph(dirty):
        full = torch.full((256 << 20,), 255, dtype=torch.uint8, device=DEV)
    dirty.replay()
    torch.cuda.synchronize()
    del full
    ws, out, eager = Workspace(), _out(q, kv), _out(q, kv)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, pool=dirty.pool()):
        _call(kv, q, ws, out)
    _call(kv, q, ws, eager)
    torch.cuda.synchronize()
    assert _equal(eager, want)
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        assert _equal(out, want)
    assert ssd_status() == 0


def test_workspace_that_grows_after_a_capture():
    """A larger call replaces the workspace's buffer; the graph that holds the smaller one keeps it."""
    _gpu.lib()
    kv = _cache(_tokens("spread", H, D)[0], 1)
    small, large = (_rows((1, nc, G * H, D), torch.bfloat16, 62, 1.5).to(DEV) for nc in (1, 16))
    ws, out, big = Workspace(), _out(small, kv), _out(large, kv)
    want = [t.clone() for t in _call(kv, small, ws, out)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(kv, small, ws, out)
    held = ws._bufs[(DEV, "kv4")]
    lo, hi, size = held.data_ptr(), held.data_ptr() + held.numel(), held.numel()
    del held
    _call(kv, large, ws, big)
    torch.cuda.synchronize()
    assert ws._bufs[(DEV, "kv4")].data_ptr() != lo
    others = [torch.full((size,), 7, dtype=torch.uint8, device=DEV) for _ in range(4)]  # whoever asks for memory next
    assert not any(lo <= t.data_ptr() < hi for t in others)
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        assert _equal(out, want)
    assert all((t == 7).all() for t in others) and ssd_status() == 0


def test_round_captured_without_a_run_before():
    _gpu.lib()
    kv = _cache(_tokens("spread", H, D)[0], 1)
    q = _rows((1, 5, G * H, D), torch.bfloat16, 63, 1.5).to(DEV)
    qd = _rows((4, 1, G * H, D), torch.bfloat16, 64, 1.5).to(DEV)
    ks = torch.full((1,), 300, dtype=torch.int32, device=DEV)
    binding.load()

    def results(r):
        return [t.clone() for t in (r.out_v, r.lse_v, r.scores, r.idx, r.cnt, r.out_d)]

    plain, captured = SpecRound(kv, G * H, 5, 300), SpecRound(kv, G * H, 5, 300)
    plain.run(q, qd, ks)
    want = results(plain)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.run(q, qd, ks)
    captured.run(q, qd, ks)
    assert _equal(results(captured), want)
    graph.replay()
    assert _equal(results(captured), want)
    assert ssd_status() == 0
