"""Tree and window attention against the definition in 64 bits.  Tokens that no query sees hold NaN and their pages are
free, so anything read beyond the masks shows."""

import numpy as np
import pytest
import torch

import sparse_self_speculative_verify_gb300 as F
from tests import _gpu
from tests._tree import Case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def run(c, want_lse=True, counts=True, **kw):
    kv = F.KVCache(c.pool.to(DEV), c.table.to(DEV), torch.tensor(c.lens, dtype=torch.int32, device=DEV), c.max_len)
    cnt = torch.tensor(c.counts, dtype=torch.int32, device=DEV) if counts else None
    if c.window is None:
        return F.ssd_tree_attn(kv, c.q.to(DEV), torch.from_numpy(c.parents).to(DEV), c.scale, counts=cnt, want_lse=want_lse, **kw)
    return F.ssd_window_attn(kv, c.q.to(DEV), c.window, c.sink, c.scale, counts=cnt, want_lse=want_lse, **kw)


def check(c, r, status=0):
    torch.cuda.synchronize()
    assert F.ssd_status() == status
    out, lse, tol, tol_lse = c.reference()
    got = r["out"].double().cpu().numpy()
    assert r["out"].dtype == c.dtype and np.isfinite(got).all()
    bad = np.abs(got - out) > tol
    assert not bad.any(), (bad.sum(), np.abs(got - out).max(), np.argwhere(bad)[:4], tol[bad][:4])
    if r["lse"] is not None:
        got = r["lse"].double().cpu().numpy()
        assert np.array_equal(np.isinf(got), np.isinf(lse))
        fin = np.isfinite(lse)
        assert (np.abs(got - lse)[fin] <= tol_lse[fin]).all(), np.abs(got - lse)[fin].max()


# dtype, d, h_q, h_kv, page, n, lens, counts
TREES = [
    (BF, 128, 32, 8, 16, 16, [700, 129, 16, 1500], None),
    (BF, 128, 8, 2, 8, 1, [1, 2, 127, 128, 129, 4000], None),       # a chain of one: plain decoding
    (BF, 128, 10, 2, 32, 33, [33, 40, 900, 513], [33, 7, 20, 0]),   # counts below n, none at all
    (BF, 64, 4, 4, 64, 7, [300, 0, 65, 7], [7, 0, 1, 7]),           # an empty request; G = 1
    (BF, 64, 6, 2, 256, 100, [1000, 100, 3001], [100, 100, 64]),    # 300 rows: more than one row tile
    (BF, 128, 40, 8, 16, 64, [2100, 64], None),                     # 320 rows
    (BF, 128, 3, 1, 512, 200, [1300], None),                        # 600 rows of one head
    (BF, 128, 16, 1, 16, 512, [700], None),                         # the most rows a tree may have
    (BF, 128, 7, 1, 4, 5, [300, 77], None),                         # pages below 8 tokens
    (BF, 64, 5, 1, 1, 40, [90], None),
    (F32, 64, 8, 2, 512, 5, [512, 300], None),
    (F32, 128, 4, 1, 16, 40, [1000, 41], [40, 17]),
    (F32, 128, 2, 2, 2, 3, [5, 64, 65], None),
]


@pytest.mark.parametrize("dtype,d,h_q,h_kv,page,n,lens,counts", TREES)
def test_tree(dtype, d, h_q, h_kv, page, n, lens, counts):
    c = Case(lens, counts or [n] * len(lens), n, h_q, h_kv, d, page, dtype, seed=n + page)
    check(c, run(c, counts=counts is not None))


# dtype, d, h_q, h_kv, page, n, lens, counts, window, sink
WINDOWS = [
    (BF, 128, 32, 8, 16, 1, [4000, 1, 130, 1025, 1024], None, 1024, 4),
    (BF, 128, 8, 2, 16, 1, [4000, 300, 131], None, 1, 0),           # itself alone
    (BF, 128, 8, 2, 16, 1, [4000, 300, 131], None, 1, 129),
    (BF, 128, 8, 2, 64, 5, [5, 640, 2000], None, 100, 0),
    (BF, 64, 9, 3, 8, 33, [40, 3000, 33, 500], [33, 33, 20, 0], 301, 5),
    (BF, 128, 4, 1, 32, 700, [700, 2300], [700, 511], 256, 1),      # a chunk of a prompt
    (BF, 128, 2, 1, 16, 600, [600], None, 1 << 20, 0),              # a whole prompt, plainly causal
    (BF, 64, 10, 2, 128, 300, [400, 1000], None, 64, 200),          # more sinks than window
    (BF, 128, 8, 2, 4, 3, [300, 77], None, 50, 3),
    (F32, 128, 4, 2, 16, 1, [4000, 3], None, 512, 4),
    (F32, 64, 5, 1, 8, 300, [300, 900], [300, 200], 77, 2),
    (F32, 128, 2, 1, 512, 20, [2000], None, 1 << 30, 1 << 30),
]


@pytest.mark.parametrize("dtype,d,h_q,h_kv,page,n,lens,counts,window,sink", WINDOWS)
def test_window(dtype, d, h_q, h_kv, page, n, lens, counts, window, sink):
    c = Case(lens, counts or [n] * len(lens), n, h_q, h_kv, d, page, dtype, seed=n + window % 1000, window=window, sink=sink)
    check(c, run(c, counts=counts is not None))
