"""Argument checks of the calls of a step that drafts trees, on the host (no kernel is launched)."""

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
    d = dict(pool=16, dtype=binding.SSD_DTYPE_BF16, num_pages=10, page_size=16, h_kv=8, d=128, page_table=256,
             max_pages=4, seq_lens=512, batch=2, max_seq_len=64)
    d.update(over)
    return binding.PagedKVStruct(**d)


def _tree(lib, kv, **o):
    return lib.ssd_tree_attn(kv, o.get("q", 4096), o.get("h_q", 32), o.get("n", 16), o.get("parents", 64), o.get("counts"),
                             o.get("scale", 0.1), o.get("out", 8192), None, o.get("ws", 1 << 20), o.get("wsb", 1 << 40), None)


def _window(lib, kv, **o):
    return lib.ssd_window_attn(kv, o.get("q", 4096), o.get("h_q", 32), o.get("n", 16), o.get("counts"), o.get("window", 32),
                               o.get("sink", 4), o.get("scale", 0.1), o.get("out", 8192), None, o.get("ws", 1 << 20),
                               o.get("wsb", 1 << 40), None)


BAD = [(dict(q=None), E), (dict(out=None), E), (dict(q=4104), E), (dict(out=8200), E), (dict(h_q=30), E), (dict(h_q=0), E), (dict(n=0), E),
       (dict(n=-3), E), (dict(h_q=8 * 129), U), (dict(scale=0.0), E), (dict(scale=-0.5), E), (dict(scale=float("nan")), E),
       (dict(scale=float("inf")), E), (dict(scale=3e38), E), (dict(ws=None), W), (dict(wsb=100), W), (dict(ws=(1 << 20) + 16), E)]


@pytest.mark.parametrize("dtype", [binding.SSD_DTYPE_BF16, binding.SSD_DTYPE_F32])
def test_attention_arguments(lib, dtype):
    kv = ctypes.byref(_kv(dtype=dtype))
    for call in (_tree, _window):
        for o, code in BAD:
            assert call(lib, kv, **o) == code, (o, lib.ssd_last_error())
            assert lib.ssd_last_error()
        assert call(lib, None) == E
        assert call(lib, ctypes.byref(_kv(dtype=dtype, d=96))) == U
        assert call(lib, ctypes.byref(_kv(dtype=dtype, page_size=12))) == U
        assert call(lib, ctypes.byref(_kv(dtype=binding.SSD_DTYPE_NVFP4))) == U
        assert call(lib, ctypes.byref(_kv(dtype=dtype, batch=0)), q=None, ws=None) == OK  # nothing to do
    assert _tree(lib, kv, parents=None) == E
    assert _tree(lib, kv, n=513) == U
    assert _tree(lib, kv, n=300, h_q=8 * 32) == U  # 9600 rows per KV head
    for o in (dict(window=0), dict(window=-1), dict(sink=-1), dict(window=(1 << 30) + 1), dict(sink=(1 << 30) + 1)):
        assert _window(lib, kv, **o) == E, o
    assert _window(lib, kv, n=1 << 27) == U


def test_workspace_queries(lib):
    for dtype, page in ((binding.SSD_DTYPE_BF16, 16), (binding.SSD_DTYPE_BF16, 4), (binding.SSD_DTYPE_F32, 16)):
        kv = ctypes.byref(_kv(dtype=dtype, page_size=page, max_pages=64 // page))
        for b in (lib.ssd_tree_workspace_bytes(kv, 32, 16), lib.ssd_window_workspace_bytes(kv, 32, 1, 100, 4)):
            assert b >= binding.COUNTER_BYTES and b % 256 == 0
        assert lib.ssd_tree_workspace_bytes(kv, 30, 16) == 0 and lib.ssd_window_workspace_bytes(kv, 32, 1, 0, 4) == 0
    assert lib.ssd_tree_workspace_bytes(None, 32, 16) == 0


def _score(lib, **o):
    return lib.ssd_token_logprobs(o.get("logits", 4096), o.get("dtype", 1), o.get("stride", 1000), o.get("N", 4), o.get("V", 1000),
                                  o.get("tokens", 64), o.get("rows"), o.get("M", 4), o.get("logprob", 64), o.get("lse", 64), None,
                                  o.get("ids", 64), o.get("lps", 64), o.get("k", 5), None)


def test_score_arguments(lib):
    for o, code in ((dict(logits=None), E), (dict(logits=4097), E), (dict(logits=4098, dtype=0), E), (dict(dtype=2), U), (dict(stride=-1), E),
                    (dict(N=-1), E), (dict(V=0), E), (dict(M=-1), E), (dict(M=5), E), (dict(tokens=None), E), (dict(logprob=None), E),
                    (dict(lse=None), E), (dict(ids=None), E), (dict(lps=None), E), (dict(k=-1), E), (dict(k=65), E), (dict(k=8, V=7), E),
                    (dict(N=0, M=0), OK), (dict(N=0, M=3, rows=64), E)):
        assert _score(lib, **o) == code, (o, lib.ssd_last_error())


def _accept(lib, **o):
    return lib.ssd_tree_accept(o.get("parents", 64), o.get("tokens", 64), o.get("target", 64), o.get("lp"), o.get("h"), o.get("eps", 0.3),
                               o.get("delta", 0.3), None, o.get("B", 2), o.get("n", 8), o.get("m", 4), o.get("path", 64), o.get("cnt", 64),
                               o.get("next", 64), o.get("advance", 64), None)


def test_accept_and_commit_arguments(lib):
    for name in ("parents", "tokens", "target", "path", "cnt", "next", "advance"):
        assert _accept(lib, **{name: None}) == E, name
    for o, code in ((dict(B=-1), E), (dict(n=0), E), (dict(m=0), E), (dict(n=513), U), (dict(lp=64), E), (dict(h=64), E),
                    (dict(lp=64, h=64, eps=0.0), E), (dict(lp=64, h=64, delta=-1.0), E), (dict(lp=64, h=64, eps=float("nan")), E),
                    (dict(lp=64, h=64, delta=float("inf")), E), (dict(B=0, parents=None), OK)):
        assert _accept(lib, **o) == code, (o, lib.ssd_last_error())
    kv = ctypes.byref(_kv())
    commit = lambda k, n=8, path=64, m=4, cnt=64: lib.ssd_tree_commit(k, n, None, path, m, cnt, None)  # noqa: E731
    assert commit(None) == E and commit(kv, path=None) == E and commit(kv, cnt=None) == E and commit(kv, n=0) == E
    assert commit(kv, m=0) == E and commit(kv, m=513) == U and commit(ctypes.byref(_kv(dtype=binding.SSD_DTYPE_NVFP4))) == U
    assert commit(ctypes.byref(_kv(batch=70000))) == U
    assert commit(ctypes.byref(_kv(batch=0)), path=None) == OK


def test_binding_refuses_what_is_not_on_the_device():
    i32 = torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(ValueError):
        F.ssd_tree_accept(i32, i32, i32)
    with pytest.raises(ValueError):
        F.ssd_token_logprobs(torch.zeros((2, 10)), i32[:, 0].contiguous())
    with pytest.raises(TypeError):
        F.ssd_token_logprobs(torch.zeros((2, 10), dtype=torch.float16))
    with pytest.raises(TypeError):
        F.ssd_tree_attn(None, i32, i32, 0.1)
    with pytest.raises(TypeError):
        F.ssd_tree_commit(None, i32, i32[:, 0], 4)


def test_binding_refuses_what_an_int_does_not_hold():
    assert binding._c_int(-(1 << 31), "x") == -(1 << 31) and binding._c_int((1 << 31) - 1, "x") == (1 << 31) - 1
    for v in (1 << 31, (1 << 32) + 5, -(1 << 31) - 1):
        with pytest.raises(ValueError, match="x .* out of range"):
            binding._c_int(v, "x")
