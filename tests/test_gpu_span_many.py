"""Tree and window attention where a block walks dozens of short units, most of which leave its second tile of rows without
a query: padded batches of small trees, prompts among decoding requests."""

import numpy as np
import pytest

import sparse_self_speculative_verify_gb300 as F
from tests._tree import Case
from tests.test_gpu_span import BF, check, run

pytestmark = pytest.mark.gpu

# d, n, requests, requests from one with all n queries to the next (0: none has more than a tile of rows holds), window
MANY = [(64, 40, 900, 25, None), (64, 40, 900, 0, None), (64, 40, 900, 300, 30), (128, 33, 600, 0, None), (128, 33, 600, 40, 50),
        (64, 5, 1000, 0, None), (128, 32, 500, 9, 20)]


@pytest.mark.parametrize("d,n,B,full,window", MANY)
def test_dozens_of_short_units_a_block(d, n, B, full, window):
    """4 heads of 4 queries: a tile holds 32 queries, a block of more than 32 two of them."""
    rng = np.random.default_rng(B + n)
    counts = [n if full and b % full == 0 else int(rng.integers(0, 3)) for b in range(B)]
    if not full:
        counts[B // 2] = min(n, 32)
    lens = [c + int(x) for c, x in zip(counts, rng.integers(0, 90, B))]
    c = Case(lens, counts, n, 16, 4, d, 8, BF, seed=B, window=window, sink=2 if window else 0)
    first = run(c)
    check(c, first)
    again = [run(c) for _ in range(5)]
    for r in again:
        assert all((a == b).all() for a, b in ((r["out"], first["out"]), (r["lse"], first["lse"])))
    assert F.ssd_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_prompts_among_decoding_requests(d):
    """A prompt of several groups of queries, then requests of one, over and over."""
    rng = np.random.default_rng(d)
    n, B = 150, 240
    counts = [n - int(rng.integers(0, 9)) if b % 80 == 0 else 1 for b in range(B)]
    lens = [c + int(x) for c, x in zip(counts, rng.integers(0, 200, B))]
    c = Case(lens, counts, n, 8, 4, d, 16, BF, seed=d, window=64, sink=4)
    check(c, run(c))
