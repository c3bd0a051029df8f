"""What the 4-bit and the page calls refuse at the ends of their ranges, on the host (no kernel is launched)."""

import ctypes
import os
import subprocess
import sys
import threading
import time

import pytest
import torch

from sparse_self_speculative_verify_gb300 import KV4Cache, PagePool, binding
from sparse_self_speculative_verify_gb300 import build as libbuild
from tests.test_kv4_host import _kv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E, U, W, OK = binding.SSD_ERR_INVALID_ARG, binding.SSD_ERR_UNSUPPORTED, binding.SSD_ERR_WORKSPACE, binding.SSD_OK


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return binding.load()


def test_compact_refuses_lists_whose_positions_pass_32_bits(lib):
    kv = ctypes.byref(_kv())
    for k_max in ((1 << 24) + 1, (1 << 31) - 200, (1 << 31) - 1):
        assert lib.ssd_kv_compact(kv, kv, None, 64, 64, 1, 64, k_max, 64, None) == U
        assert b"2^24" in lib.ssd_last_error()
    assert lib.ssd_kv_compact(kv, kv, None, 64, 64, 0, 64, 1 << 24, 64, None) == OK  # no pairs: nothing is launched


def test_pages_of_2_gb_are_refused_by_every_call_on_a_4_bit_cache(lib):
    """Offsets inside a page are 32 bits in all of them."""
    big = ctypes.byref(_kv(page_size=1 << 24, max_seq_len=1 << 24))
    ok = ctypes.byref(_kv())
    calls = {
        "append": lambda: lib.ssd_kv4_append(big, 4096, 4096, 1, 3, None, 1.0, 1.0, None),
        "read": lambda: lib.ssd_kv4_read(big, 64, None, 3, 1.0, 1.0, 1, 4096, 4096, None),
        "verify": lambda: lib.ssd_kv4_verify_attn(big, 4096, 1, 32, 5, 0.1, 1.0, 1.0, 8192, 0, None, None, 0, 1 << 20, 1 << 40, None),
        "draft": lambda: lib.ssd_kv4_draft_attn(big, 4096, 1, 32, 64, 8, 64, 0.1, 1.0, 1.0, 8192, 0, None, 1 << 20, 1 << 40, None),
        "fork": lambda: lib.ssd_kv_fork(big, 64, 64, 64, 1, None),
        "reserve": lambda: lib.ssd_kv_reserve(big, 64, 64, 1 << 20, 1 << 30, None),
        "release": lambda: lib.ssd_kv_release(big, 64, 64, None),
        "compact from": lambda: lib.ssd_kv_compact(big, ok, None, 64, 64, 1, 64, 4, 64, None),
        "compact to": lambda: lib.ssd_kv_compact(ok, big, None, 64, 64, 1, 64, 4, 64, None),
    }
    for name, call in calls.items():
        assert call() == U, name
        assert b"2 GB" in lib.ssd_last_error(), name


def test_page_counts_of_a_table_with_ids_outside_the_pool():
    """Refused before the counts are scattered: on a GPU an id past their end fails a device assertion."""
    table = torch.tensor([[3, -1], [0, 7]], dtype=torch.int32)
    for num_pages in (7, 1):
        with pytest.raises(ValueError, match="page 7 of a pool"):
            PagePool.from_table(table, num_pages)
    with pytest.raises(ValueError, match="CUDA"):  # the table is fine; counts live on the GPU
        PagePool.from_table(table, 8)


def test_import_without_torchs_private_names():
    """The host parts import on a torch that lacks them (one built without CUDA, or of another version)."""
    code = ("import torch\n"
            "for name in ('_cuda_getCurrentRawStream', '_cuda_getDevice', '_cuda_isCurrentStreamCapturing'):\n"
            "    if hasattr(torch._C, name): delattr(torch._C, name)\n"
            "from sparse_self_speculative_verify_gb300 import binding\n"
            "assert binding._current_device is torch.cuda.current_device\n"
            "assert binding._capturing is torch.cuda.is_current_stream_capturing\n"
            "assert callable(binding._raw_stream)\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0, r.stderr


class _Cache(KV4Cache):
    """Enough of a cache for the calls' host side, on the CPU."""

    def __init__(self):
        self.max_seq_len, self.k_scale, self.v_scale, self._need = 64, 1.0, 1.0, {}
        self._geometry, self._struct = (-1, 2, 1, 64), _kv(batch=2, h_kv=1, d=64)
        self._ref = ctypes.byref(self._struct)


class _Pages(PagePool):
    def __init__(self):
        self.refs = torch.zeros(10, dtype=torch.int32)


def test_threads_on_one_stream_take_turns_with_its_workspace(monkeypatch):
    """A call's launches hand their results on through the workspace, and ctypes lets other threads run meanwhile."""
    inside, most = [], []

    def native(*args):
        inside.append(1)
        most.append(len(inside))
        time.sleep(0.02)
        inside.pop()
        return OK

    class Lib:
        ssd_kv4_verify_attn = ssd_kv4_draft_attn = ssd_kv_reserve = staticmethod(native)
        ssd_kv4_verify_workspace_bytes = ssd_kv4_draft_workspace_bytes = ssd_kv_reserve_workspace_bytes = staticmethod(lambda *a: 1024)

    monkeypatch.setattr(binding, "_lib", Lib)
    monkeypatch.setattr(binding, "_current_device", lambda: -1)
    monkeypatch.setattr(binding, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(binding, "_capturing", lambda: False)
    monkeypatch.setattr(binding, "_STREAM_WS", {(-1, 0, name): (None, 256, 1 << 20) for name in ("kv4", "pages")})
    kv, pages = _Cache(), _Pages()
    q, out = torch.zeros((2, 1, 4, 64)), torch.zeros((2, 1, 4, 64))
    idx, cnt = torch.zeros((2, 1, 3), dtype=torch.int32), torch.zeros((2, 1), dtype=torch.int32)
    calls = [
        lambda: binding.ssd_kv4_verify_attn(kv, q, 1, 0.1, out=out, want_lse=False, want_scores=False),
        lambda: binding.ssd_kv4_draft_attn(kv, q[:, 0].contiguous(), idx, cnt, 0.1, out=out[:, 0].contiguous(), want_lse=False),
        lambda: binding.ssd_kv_reserve(kv, pages, torch.zeros(2, dtype=torch.int32)),
    ]
    threads = [threading.Thread(target=c) for c in calls for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(most) == 9 and max(most) == 1
