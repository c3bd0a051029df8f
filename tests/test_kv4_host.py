"""Argument checks of the 4-bit cache and the page calls, on the host (no kernel is launched)."""

import ctypes

import pytest
import torch

import sparse_self_speculative_verify_gb300 as F
from sparse_self_speculative_verify_gb300 import binding
from sparse_self_speculative_verify_gb300 import build as libbuild

E, U, W, OK = binding.SSD_ERR_INVALID_ARG, binding.SSD_ERR_UNSUPPORTED, binding.SSD_ERR_WORKSPACE, binding.SSD_OK


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return binding.load()


def _kv(**over):
    d = dict(pool=16, dtype=binding.SSD_DTYPE_NVFP4, num_pages=10, page_size=16, h_kv=8, d=128, page_table=256,
             max_pages=4, seq_lens=512, batch=2, max_seq_len=64)
    d.update(over)
    return binding.PagedKVStruct(**d)


BAD_CACHES = [(dict(pool=None), E), (dict(seq_lens=None), E), (dict(d=96), U), (dict(page_size=4, max_seq_len=16), U), (dict(page_size=24), U),
              (dict(max_seq_len=65), E), (dict(pool=24), E), (dict(num_pages=0), E), (dict(batch=-1), E)]


def _verify(lib, kv, **o):
    return lib.ssd_kv4_verify_attn(kv, o.get("q", 4096), o.get("qt", 1), o.get("h_q", 32), o.get("n", 5), o.get("scale", 0.1),
                                   o.get("ks", 1.0), o.get("vs", 1.0), o.get("out", 8192), o.get("ot", 0), None,
                                   o.get("scores"), o.get("stride", 0), o.get("ws", 1 << 20), o.get("wsb", 1 << 40), None)


def _draft(lib, kv, **o):
    return lib.ssd_kv4_draft_attn(kv, o.get("q", 4096), o.get("qt", 1), o.get("h_q", 32), o.get("idx", 64), o.get("k", 8),
                                  o.get("cnt", 64), o.get("scale", 0.1), o.get("ks", 1.0), o.get("vs", 1.0),
                                  o.get("out", 8192), o.get("ot", 0), None, o.get("ws", 1 << 20), o.get("wsb", 1 << 40), None)


def _append(lib, kv, **o):
    return lib.ssd_kv4_append(kv, o.get("k", 4096), o.get("v", 4096), o.get("t", 1), o.get("n", 3), None, o.get("ks", 1.0),
                              o.get("vs", 1.0), None)


def _read(lib, kv, **o):
    return lib.ssd_kv4_read(kv, o.get("first", 64), None, o.get("n", 3), o.get("ks", 1.0), o.get("vs", 1.0), o.get("t", 1),
                            o.get("k", 4096), o.get("v", 4096), None)


@pytest.mark.parametrize("call", [_verify, _draft, _append, _read])
def test_kv4_calls_check_the_cache(lib, call):
    assert call(lib, None) == E
    for over, code in BAD_CACHES:
        assert call(lib, ctypes.byref(_kv(**over))) == code, over
        assert lib.ssd_last_error()
    for t in (binding.SSD_DTYPE_BF16, binding.SSD_DTYPE_F32, 7):  # a cache of another element type
        assert call(lib, ctypes.byref(_kv(dtype=t))) == U
    for s in (0.0, -1.0, 3.0, float("nan"), float("inf"), 2.0 ** 40):
        assert call(lib, ctypes.byref(_kv()), ks=s) == E
        assert call(lib, ctypes.byref(_kv()), vs=s) == E


def test_other_calls_refuse_a_4_bit_cache(lib):
    kv = ctypes.byref(_kv())
    assert lib.ssd_verify_attn(kv, 4096, 32, 5, 0.1, 8192, None, None, 0, None, 0, 64, 1 << 20, 1 << 40, None) == U
    assert lib.ssd_draft_attn(kv, 16, 32, 16, 8, 16, 0.1, 16, None, 1 << 20, 1 << 40, None) == U
    assert lib.ssd_kv_append(kv, 4096, 4096, 2, None) == U


def test_attention_arguments(lib):
    kv = ctypes.byref(_kv())
    for call in (_verify, _draft):
        for o, code in ((dict(q=None), E), (dict(out=None), E), (dict(q=4104), E), (dict(out=8200), E), (dict(qt=2), U),
                        (dict(ot=5), U), (dict(h_q=30), E), (dict(h_q=0), E), (dict(scale=float("nan")), E),
                        (dict(ws=None), W), (dict(wsb=100), W), (dict(ws=(1 << 20) + 16), E)):
            assert call(lib, kv, **o) == code, o
    assert _verify(lib, kv, n=0) == E
    assert _verify(lib, kv, n=17) == U  # 68 rows
    assert _verify(lib, kv, scores=4096, stride=63) == E
    assert _draft(lib, kv, h_q=8 * 17) == U
    assert _draft(lib, kv, k=-1) == E
    assert _draft(lib, kv, idx=None) == E
    assert _draft(lib, kv, cnt=None) == E
    empty = ctypes.byref(_kv(batch=0))
    assert _verify(lib, empty) == OK and _draft(lib, empty) == OK  # nothing to do, nothing launched


def test_attention_limits(lib):
    """What the kernels' 32-bit positions, rows and grids do not hold is refused before a launch."""
    far = dict(max_pages=1 << 27, max_seq_len=(1 << 24) + 1)
    for call in (_verify, _draft):
        assert call(lib, ctypes.byref(_kv(**far))) == U and b"2^24" in lib.ssd_last_error()
        assert call(lib, ctypes.byref(_kv(batch=8192))) == U
    assert _draft(lib, ctypes.byref(_kv()), k=(1 << 24) + 1) == U
    assert _verify(lib, ctypes.byref(_kv()), n=17) == U  # 68 rows
    assert _draft(lib, ctypes.byref(_kv(h_kv=1)), h_q=17) == U


def test_workspace_queries(lib):
    kv = _kv()
    a = lib.ssd_kv4_verify_workspace_bytes(ctypes.byref(kv), 32, 5)
    assert a > 0 and a % 256 == 0
    assert lib.ssd_kv4_verify_workspace_bytes(ctypes.byref(_kv(max_seq_len=1024, max_pages=64)), 32, 5) > a
    for bad in ((None, 32, 5), (ctypes.byref(kv), 30, 5), (ctypes.byref(kv), 32, 0), (ctypes.byref(kv), 32, 17)):
        assert lib.ssd_kv4_verify_workspace_bytes(*bad) == 0
    assert lib.ssd_kv4_draft_workspace_bytes(ctypes.byref(kv), 32, 410) > 0
    assert lib.ssd_kv4_draft_workspace_bytes(ctypes.byref(kv), 32, -1) == 0
    assert lib.ssd_kv_reserve_workspace_bytes(None) == 0
    assert lib.ssd_kv_reserve_workspace_bytes(ctypes.byref(kv)) > 10 * 16


def test_append_and_read_arguments(lib):
    kv = ctypes.byref(_kv())
    for call in (_append, _read):
        assert call(lib, kv, n=-1) == E
        assert call(lib, kv, k=None) == E
        assert call(lib, kv, v=4104) == E
        assert call(lib, kv, t=2) == U
        assert call(lib, kv, n=0) == OK
    assert _read(lib, kv, first=None) == E


def test_page_arguments(lib):
    kv = _kv()
    r = ctypes.byref(kv)
    assert lib.ssd_kv_fork(r, None, 64, 64, 1, None) == E
    assert lib.ssd_kv_fork(r, 64, None, 64, 1, None) == E
    assert lib.ssd_kv_fork(r, 64, 64, 64, -1, None) == E
    assert lib.ssd_kv_fork(r, 64, None, None, 0, None) == OK
    assert lib.ssd_kv_fork(ctypes.byref(_kv(dtype=9)), 64, 64, 64, 1, None) == U
    assert lib.ssd_kv_reserve(r, 64, None, 1 << 20, 1 << 30, None) == E
    assert lib.ssd_kv_reserve(r, 64, 64, None, 1 << 30, None) == W
    assert lib.ssd_kv_reserve(r, 64, 64, 1 << 20, 64, None) == W
    assert lib.ssd_kv_reserve(r, 64, 64, (1 << 20) + 8, 1 << 30, None) == E
    assert lib.ssd_kv_reserve(ctypes.byref(_kv(batch=0)), 64, None, 1 << 20, 1 << 30, None) == OK
    assert lib.ssd_kv_release(r, 64, None, None) == E
    assert lib.ssd_kv_release(r, None, 64, None) == E
    c = lambda to, n=1, k=4, idx=64, cnt=64: lib.ssd_kv_compact(r, ctypes.byref(to), None, 64, 64, n, idx, k, cnt, None)  # noqa: E731
    assert c(_kv(h_kv=4)) == E
    assert c(_kv(d=64)) == E
    assert c(_kv(dtype=binding.SSD_DTYPE_BF16)) == E
    assert c(kv, n=-1) == E and c(kv, k=-1) == E and c(kv, idx=None) == E and c(kv, cnt=None) == E
    assert c(kv, n=0) == OK
    assert lib.ssd_kv_compact(r, None, None, 64, 64, 1, 64, 4, 64, None) == E


def test_binding_refuses_what_is_not_a_cuda_tensor():
    t = torch.zeros((4, 2, 1, 16, 72), dtype=torch.uint8)
    with pytest.raises(ValueError):
        F.KV4Cache(t, torch.zeros((1, 4), dtype=torch.int32), torch.zeros((1,), dtype=torch.int32), 16)
    with pytest.raises(ValueError):
        F.PagePool(torch.zeros((4,), dtype=torch.int32))
    with pytest.raises(TypeError):
        F.ssd_kv4_read(object(), None, 3)
    assert F.KV4Cache.pool_shape(4, 1, 16, 128) == (4, 2, 1, 16, 72)


def test_round_over_a_4_bit_cache(monkeypatch):
    """SpecRound on a KV4Cache makes the 4-bit calls, with no row pack."""
    class _KV4(F.KV4Cache):
        device = torch.device("cpu")
        batch, h_kv, d = 2, 2, 64

        def __init__(self):
            self.max_seq_len, self.seq_lens = 128, torch.tensor([100, 128], dtype=torch.int32)

    calls = []
    for name in ("ssd_verify_attn", "ssd_verify_select", "ssd_draft_attn", "ssd_draft_attn_packed", "ssd_select_topk",
                 "ssd_kv4_verify_attn", "ssd_kv4_draft_attn"):
        out = (0, 1) if name == "ssd_select_topk" else {"out": 2}
        monkeypatch.setattr(binding, name, lambda *a, _n=name, _o=out, **k: calls.append(_n) or _o)
    r = F.SpecRound(_KV4(), h_q=4, n_cand=3, k_max=8)
    assert r.pack is None
    q, qd, ks = torch.zeros((2, 3, 4, 64)), torch.zeros((2, 2, 4, 64)), torch.full((2,), 8, dtype=torch.int32)
    want = ["ssd_kv4_verify_attn", "ssd_select_topk", "ssd_kv4_draft_attn", "ssd_kv4_draft_attn"]
    r.run(q, qd, ks)
    assert calls == want
    calls.clear()
    r.run(q, qd, ks, fused_select=True)
    assert calls == want
    assert r.verify_select(q, ks) == {"out": 2, "idx": 0, "cnt": 1}
    calls.clear()
    r.draft_oracle_topk(qd[0], ks)
    assert calls == want[:3]
    with pytest.raises(ValueError):
        F.SpecRound(_KV4(), h_q=4, n_cand=3, k_max=8, pack_in_select=True)
