"""What the 4-bit and the page calls refuse at the ends of their ranges, on the host (no kernel is launched)."""

import ctypes

import pytest

from sparse_self_speculative_verify_gb300 import binding
from sparse_self_speculative_verify_gb300 import build as libbuild
from tests.test_kv4_host import _kv

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
