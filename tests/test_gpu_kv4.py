"""The 4-bit cache on the GPU: append and read back bit for bit, attention against 64 bits.

Tolerances.  Stored values and query values enter the products exactly (a stored value has 6 significant
bits and is held in f16, a bf16 query in f16 up to a power of two, an fp32 query in two f16: 22 bits).
 * A logit x (in units of ln): the products are summed in fp32 over d = 128 elements in at most 8 steps of
   16, each step off by at most 2^-21 of the largest partial sum (tensor cores add with truncation after
   aligning 16 products and the sum to the largest), so by 8 * 2^-21 * scale * sum |q k| in all; an fp32
   query adds 2^-22 * scale * sum |q k|.  With X = the largest scale * sum |q k| of the case the logit's
   error is at most E = X * 2^-17.9.
 * A probability is then off by E relative, twice that after the division by the sum, plus exp2's and the
   f32 subtraction's 2^-21 * (1 + |x| / 8): we take 2 E + 2^-18.
 * out = sum p v / sum p: off by (2 E + 2^-18) * sum p |v| plus, for bf16 outputs, P's rounding to f16 (2^-11
   at most) and the output's own half step, 2^-9: under (2 E + 2^-18 + 2^-11) A + 2^-8 |out| with A = sum p |v|.
   fp32 outputs carry P in 22 bits: 2^-22, inside the 2^-18.
 * lse: E + 2^-20 * max(1, |lse|).   scores: (2 E + 2^-18) relative, and 2^-24 absolute per query row for
   what exp2 flushes."""

import math

import numpy as np
import pytest
import torch

from sparse_self_speculative_verify_gb300 import (KV4Cache, binding, ssd_kv4_append, ssd_kv4_draft_attn, ssd_kv4_read,
                                                 ssd_kv4_verify_attn, ssd_status)
from tests import _gpu, _kv4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _cache(lens, h, d, page, room=0, seed=0, k_scale=1.0, v_scale=1.0, fill=True, max_extra=0):
    """A cache whose pages are shuffled and whose every byte is arbitrary, filled for `lens` tokens (through
    numpy, not through the library); returns it with its numpy pool and table."""
    rng = np.random.default_rng(seed)
    need = [-(-(n + room) // page) for n in lens]
    cap = max(max(need), 1) + 1
    total = sum(need) + 4
    perm = rng.permutation(total)
    table = np.full((len(lens), cap), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    pool = rng.integers(0, 256, (total, 2, h, page, d // 2 + d // 16), dtype=np.uint8)
    if fill:
        for b, n in enumerate(lens):
            x = rng.standard_normal((2, h, n, d))
            x[0] += 3.0 * (rng.random((h, n, 1)) < 0.05) * rng.standard_normal((h, 1, d))
            c, s = _kv4.quantise(x)
            for t in range(n):
                for w in range(2):
                    for g in range(h):
                        _kv4.write_row(pool, table[b, t // page], w, g, t % page, d, c[w, g, t], s[w, g, t])
    kv = KV4Cache(torch.from_numpy(pool.copy()).to(DEV), torch.from_numpy(table).to(DEV),
                  torch.tensor(lens, dtype=torch.int32, device=DEV), max(lens) + room + max_extra, k_scale, v_scale)
    return kv, pool, table


def _rows(shape, dtype, seed, sd=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * sd).to(dtype)


def _check(got, ref, A, X, out_bf16, rows, what):
    E = X * 2.0 ** -17.9
    rel = 2 * E + 2.0 ** -18
    o = got["out"].float().cpu().numpy().astype(np.float64)
    lim = (rel + (2.0 ** -11 if out_bf16 else 0)) * A + (2.0 ** -8 if out_bf16 else 0) * np.abs(ref["out"]) + 1e-30
    assert np.isfinite(o).all(), what
    assert (np.abs(o - ref["out"]) <= lim).all(), f"{what}: out off by {(np.abs(o - ref['out']) / lim).max():.2f} limits"
    if got.get("lse") is not None:
        z = got["lse"].cpu().numpy().astype(np.float64)
        fin = np.isfinite(ref["lse"])
        assert np.array_equal(z[~fin], ref["lse"][~fin]), what
        assert (np.abs(z[fin] - ref["lse"][fin]) <= E + 2.0 ** -20 * np.maximum(1, np.abs(ref["lse"][fin]))).all(), f"{what}: lse"
    if got.get("scores") is not None:
        s = got["scores"].cpu().numpy().astype(np.float64)
        for b, want in enumerate(ref["scores"]):
            n = want.shape[1]
            off = np.abs(s[b, :, :n] - want)
            assert (off <= rel * want + rows * 2.0 ** -24).all(), f"{what}: scores"
            assert not s[b, :, n:].any(), f"{what}: scores past the end were written"


def _bounds(pool, table, lens, q, d, scale, ks, vs):
    """X (largest scale * sum |q k|) and A (sum p |v| is at most the largest |v|): per case bounds."""
    X, A = 0.0, 0.0
    h = pool.shape[2]
    for b, n in enumerate(lens):
        for g in range(h):
            if n == 0:
                continue
            K = np.abs(_kv4.read_rows(pool, table[b], 0, g, range(n), d, ks))
            V = np.abs(_kv4.read_rows(pool, table[b], 1, g, range(n), d, vs))
            qa = np.abs(q[b].reshape(-1, d))
            X = max(X, float((K @ qa.T).max()) * scale)
            A = max(A, float(V.max()))
    return X, A


VERIFY = [
    # lens, h_kv, G, d, n_cand, page
    ([1], 1, 1, 64, 1, 8),
    ([5, 33, 64], 2, 4, 128, 1, 16),
    ([7, 31, 32, 65, 200], 2, 4, 128, 5, 16),
    ([300], 1, 1, 128, 8, 8),
    ([130, 257], 1, 8, 64, 4, 32),
    ([130, 61], 2, 5, 128, 5, 64),
    ([515], 1, 7, 128, 8, 16),   # 56 rows: two passes over the cache
    ([90, 40], 1, 16, 64, 4, 128),  # 64 rows
    ([2100, 3], 1, 4, 128, 3, 16),
]


@pytest.mark.parametrize("types", ["bf16-f32", "bf16-bf16", "f32-f32"])
@pytest.mark.parametrize("case", VERIFY, ids=lambda c: f"L{'_'.join(map(str, c[0]))}-h{c[1]}G{c[2]}d{c[3]}n{c[4]}p{c[5]}")
def test_verify_against_64_bits(case, types):
    _gpu.lib()
    lens, h, G, d, nc, page = case
    qt, ot = (torch.bfloat16 if x == "bf16" else torch.float32 for x in types.split("-"))
    kv, pool, table = _cache(lens, h, d, page, seed=3, k_scale=0.5, v_scale=2.0)
    q = _rows((len(lens), nc, G * h, d), qt, 5, 1.5)
    scale = 1 / math.sqrt(d)
    r = ssd_kv4_verify_attn(kv, q.to(DEV), nc, scale, out_dtype=ot)
    q64 = q.double().numpy()
    ref = _kv4.verify(pool, table, lens, q64, d, scale, 0.5, 2.0)
    X, A = _bounds(pool, table, lens, q64, d, scale, 0.5, 2.0)
    torch.cuda.synchronize()
    assert ssd_status() == (binding.FAULT_SEQLEN if min(lens) < nc else 0)
    _check(r, ref, A, X, ot == torch.bfloat16, nc * G, "verify")


DRAFT = [
    # lens, counts per request, h_kv, G, d, page
    ([3], [1], 1, 1, 64, 8),
    ([300, 50, 9], [100, 0, 9], 2, 4, 128, 16),
    ([700, 800], [33, 64], 1, 16, 128, 16),
    ([400], [31], 3, 5, 64, 64),
    ([1500, 40], [1100, 40], 2, 8, 128, 8),
]


@pytest.mark.parametrize("types", ["bf16-f32", "bf16-bf16", "f32-f32"])
@pytest.mark.parametrize("case", DRAFT, ids=lambda c: f"L{'_'.join(map(str, c[0]))}-k{'_'.join(map(str, c[1]))}-h{c[2]}G{c[3]}d{c[4]}p{c[5]}")
def test_draft_against_64_bits(case, types):
    _gpu.lib()
    lens, counts, h, G, d, page = case
    qt, ot = (torch.bfloat16 if x == "bf16" else torch.float32 for x in types.split("-"))
    kv, pool, table = _cache(lens, h, d, page, seed=7)
    rng = np.random.default_rng(1)
    k_max = max(counts) + 2
    idx = np.full((len(lens), h, k_max), -1, np.int32)
    cnt = np.zeros((len(lens), h), np.int32)
    for b, (n, c) in enumerate(zip(lens, counts)):
        for g in range(h):
            cnt[b, g] = max(0, c - g)  # lists of different lengths
            idx[b, g, :cnt[b, g]] = np.sort(rng.choice(n, cnt[b, g], replace=False))
    if cnt[0, 0] > 1:
        idx[0, 0, 1] = idx[0, 0, 0]  # a token listed twice counts twice
    q = _rows((len(lens), G * h, d), qt, 11, 1.5)
    scale = 1 / math.sqrt(d)
    r = ssd_kv4_draft_attn(kv, q.to(DEV), torch.from_numpy(idx).to(DEV), torch.from_numpy(cnt).to(DEV), scale, out_dtype=ot)
    q64 = q.double().numpy()
    ref = _kv4.draft(pool, table, q64, idx, cnt, d, scale)
    X, A = _bounds(pool, table, lens, q64, d, scale, 1.0, 1.0)
    torch.cuda.synchronize()
    assert ssd_status() == 0
    _check(r, ref, A, X, ot == torch.bfloat16, G, "draft")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", [([0], 1, 1, 64, 8), ([13, 250, 0], 7, 2, 128, 16), ([5, 5], 300, 1, 64, 64)],
                         ids=lambda c: f"L{'_'.join(map(str, c[0]))}-n{c[1]}d{c[3]}p{c[4]}")
def test_append_and_read_bit_for_bit(case, dtype):
    _gpu.lib()
    lens, n, h, d, page = case
    B = len(lens)
    kv, pool, table = _cache(lens, h, d, page, room=n, seed=9, k_scale=0.25, v_scale=2.0)
    rng = np.random.default_rng(2)
    x = rng.standard_normal((2, B, n, h, d)) * np.exp(rng.uniform(-12, 9, (2, B, n, h, 1)))  # scales from 0 to saturated
    x[0, 0, 0, 0, :16] = 0.0
    # Ties of the codes (x = tie * scale) and of the scales (max = 6 * midpoint of two e4m3 values).
    x[1, 0, 0, 0, :16] = 2.0 * 0.5 * np.array([6, .25, -.25, .75, -.75, 1.25, 1.75, 2.5, -2.5, 3.5, 5, -5, 3, 0, -6, .5])
    x[1, 0, 0, 0, 16:32] = 2.0 * np.array([6 * 1.0625] + [1.0] * 15)
    x[1, 0, 0, 0, 32:48] = 2.0 * np.array([6 * 1.1875] + [-0.3] * 15)
    t = torch.from_numpy(x).to(dtype)
    counts = np.array([max(0, n - 2 * b) for b in range(B)], np.int32)
    want = pool.copy()
    vals = np.zeros((2, B, n, h, d))
    for w, s in ((0, 0.25), (1, 2.0)):
        c, e = _kv4.quantise(t[w].double().numpy(), s)
        for b in range(B):
            for j in range(counts[b]):
                for g in range(h):
                    pos = lens[b] + j
                    _kv4.write_row(want, table[b, pos // page], w, g, pos % page, d, c[b, j, g], e[b, j, g])
                    vals[w, b, j, g] = _kv4.values(c[b, j, g], e[b, j, g], s)
    cd = torch.from_numpy(counts).to(DEV)
    ssd_kv4_append(kv, t[0].contiguous().to(DEV), t[1].contiguous().to(DEV), counts=cd)
    k, v = ssd_kv4_read(kv, kv.seq_lens, n, counts=cd, dtype=dtype)
    torch.cuda.synchronize()
    assert ssd_status() == 0
    got = kv.pool.cpu().numpy()
    # A zero group's codes may be +0 or -0; everything else, and every byte not appended, is equal.
    np.testing.assert_array_equal(got, want)
    np.testing.assert_array_equal(k.double().cpu().numpy(), vals[0])
    np.testing.assert_array_equal(v.double().cpu().numpy(), vals[1])
    assert kv.seq_lens.cpu().tolist() == lens
