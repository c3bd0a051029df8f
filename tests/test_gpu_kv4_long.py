"""The 4-bit attention on stretches as long as a user's: hundreds of rows share the pages of one request of 32768
tokens, so that every block walks 200 tiles of 128 tokens, or every warp 100 of 32, of a unit.  Against 64 bits on the
GPU, from the values that the pool's bytes stand for, every row of the batch.

Limits, as relative 2-norms over all outputs of a head (`fp32 outputs`; F = 64 products in a row, 4 tiles x 16 on tcgen05
and 16 x 4 on mma.sync, between two times that O is added up to nearest):
 * the tensor cores add with truncation: a step loses less than 2^-23 of the sum so far, which grows from nothing over
   F = 64 steps: 2^-23 * 64 / 2 = 2^-18 at most, where V is positive; the sums of the periods (64 at most, to nearest)
   and of the blocks' parts 2^-25 * 8, with errors of either sign;
 * a logit x: d / 16 <= 8 truncating steps (16 for fp32 queries, whose second half is 2^-11 of the first), which take up to
   2^-23 * 4 relative off |q k| <= 20: as all logits shrink alike, outputs move by 2^-21 times the spread of x under the
   softmax (under 4): 2^-19; exp2 and the subtraction 2^-21, either sign;
 * P in 22 bits, or 2^-35 of the largest: 2^-23, and 32768 * 2^-35 = 2^-20 at most.
In all under 6e-6 (2^-18 + 2^-19 + ...).  lse: 2^-21 * 20 and its own half steps at 16 to 32 (2^-20): 2^-16.  Scores:
the same shrinking logits, weighted by p, 2^-18, as a norm.  bf16 outputs: their half step 2^-9 (rms 2^-9 / sqrt 3) and
P's 2^-12: under 2^-8.

Where logits grow ("grow"), all products of a logit have one sign and add up to 60.  A step then truncates 16 products and
the sum so far, each by less than 2^-25 of that sum: 17 * 2^-25 < 2^-20.9, or 2^-21 with the products' spread.  Over d / 16
= 8 steps the sum grows evenly: 8 / 2 of them.  The second half of an fp32 query adds 8 steps at its full height: 12 in
all.  The softmax is sharp (its neighbours' logits lose alike, but not equally), so outputs, lse and scores may be off by
all of it: 60 * 2^-21 * 4, and * 12 for fp32 queries, on top of the above."""

import functools
import math

import numpy as np
import pytest
import torch

from sparse_self_speculative_verify_gb300 import KV4Cache, ssd_kv4_draft_attn, ssd_kv4_verify_attn, ssd_status
from tests import _gpu, _kv4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
L, PAGE = 32768, 16
F32_OUT, F32_LSE, F32_SCORES, BF16_OUT = 6e-6, 2.0 ** -16, 2.0 ** -18, 2.0 ** -8


def _bytes(codes, scales):
    """Codes [h, n, d] and scales [h, n, d / 16] as pages' blocks [n / PAGE, h, PAGE * 9 d / 16]."""
    h, n, d = codes.shape
    packed = (codes[..., 0::2] | (codes[..., 1::2] << 4)).reshape(h, n // PAGE, PAGE * d // 2)
    return np.concatenate([packed, scales.reshape(h, n // PAGE, PAGE * d // 16)], -1).transpose(1, 0, 2)


@functools.lru_cache(maxsize=4)
def _tokens(kind, h, d, n=L):
    """(pool, K, V in 64 bits [h, n, d]) on the GPU."""
    rng = np.random.default_rng(41)
    k, v = rng.standard_normal((2, h, n, d))
    if kind == "positive":
        v = np.abs(v)
    if kind == "grow":  # logits that rise all along, with falls in between; q holds the signs
        t = np.arange(n)
        ramp = 2.0 * t / n - 1 - 0.15 * (t // 700 % 3 == 1)
        k = 4.0 * ramp[:, None] * _signs(d) + 0.05 * k
    ck, cv = _kv4.quantise(k), _kv4.quantise(v)
    pool = np.stack([_bytes(*ck), _bytes(*cv)], 1)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
    return dev(pool).view(KV4Cache.pool_shape(n // PAGE, h, PAGE, d)), dev(_kv4.values(*ck)), dev(_kv4.values(*cv))


def _signs(d):
    return np.sign(np.random.default_rng(5).standard_normal(d))


def _cache(pool, B, n=L):
    table = torch.arange(n // PAGE, dtype=torch.int32, device=DEV).expand(B, -1).contiguous()
    return KV4Cache(pool, table, torch.full((B,), n, dtype=torch.int32, device=DEV), n)


def _queries(kind, shape, dtype):
    g = torch.Generator(device=DEV).manual_seed(6)
    if kind == "grow":
        s = torch.from_numpy(_signs(shape[-1])).to(DEV, torch.float32)
        return (s * (0.7 + 0.3 * torch.rand(shape[:-1] + (1,), generator=g, device=DEV))).to(dtype)
    return (1.5 * torch.randn(shape, generator=g, device=DEV)).to(dtype)


def _attend(q, K, V, limit, scale):
    """Rows q [r, d] that see the first limit[r] tokens: out, lse, probabilities [n, r]; 64 bits."""
    x = scale * (K @ q.double().T)
    x.masked_fill_(torch.arange(len(K), device=DEV)[:, None] >= limit[None], -math.inf)
    lse = torch.logsumexp(x, 0)
    P = x.sub_(lse).exp_()
    return P.T @ V, lse, P


def _off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


def _types(types):
    return (torch.bfloat16 if t == "bf16" else torch.float32 for t in types.split("-"))


FORMS = [  # h_kv, G, d, n_cand
    (2, 4, 128, 1), (2, 8, 128, 1), (2, 4, 128, 3), (2, 4, 128, 4), (2, 4, 128, 5), (2, 8, 128, 4), (1, 16, 128, 3),
    (1, 16, 128, 4),
    (2, 4, 64, 1), (2, 3, 64, 3), (2, 4, 64, 4), (2, 4, 64, 5), (2, 8, 64, 4), (1, 16, 64, 3),
]


@pytest.mark.parametrize("types", ["bf16-f32", "f32-f32", "bf16-bf16"])
@pytest.mark.parametrize("kind", ["spread", "positive", "grow"])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: f"h{f[0]}G{f[1]}d{f[2]}n{f[3]}")
def test_verify_over_long_stretches(form, kind, types):
    _verify(form, kind, types, 330 // form[0])


@pytest.mark.parametrize("types", ["bf16-f32", "bf16-bf16"])
@pytest.mark.parametrize("B", [1, 3, 20])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: f"h{f[0]}G{f[1]}d{f[2]}n{f[3]}")
def test_verify_of_few_long_requests(form, B, types):
    """Units of a hundred parts down to eight, joined by the last block to arrive or, on tcgen05, by a launch of their own."""
    _verify(form, "spread", types, B)


def _verify(form, kind, types, B):
    _gpu.lib()
    h, G, d, nc = form
    qt, ot = _types(types)
    pool, K, V = _tokens(kind, h, d)
    kv = _cache(pool, B)
    q = _queries(kind, (B, nc, G * h, d), qt)
    scale = 60.0 / (4 * d) if kind == "grow" else 1 / math.sqrt(d)
    r = ssd_kv4_verify_attn(kv, q, nc, scale, out_dtype=ot)
    again = ssd_kv4_verify_attn(kv, q, nc, scale, out_dtype=ot)
    torch.cuda.synchronize()
    assert ssd_status() == 0
    for name in ("out", "lse", "scores"):
        assert torch.equal(r[name], again[name]), name
    more = 60 * 2.0 ** -21 * (12 if qt == torch.float32 else 4) if kind == "grow" else 0.0
    for g in range(h):
        heads = slice(g * G, (g + 1) * G)
        rows = q[:, :, heads].reshape(-1, d)
        limit = (L - nc + 1 + torch.arange(nc, device=DEV)).repeat_interleave(G).repeat(B)
        out, lse, P = _attend(rows, K[g], V[g], limit, scale)
        scores = P.view(L, B, nc * G).sum(2).T
        del P
        off = _off(r["out"][:, :, heads].reshape(-1, d), out)
        assert off <= more + (F32_OUT if ot == torch.float32 else BF16_OUT), f"out off by {off:.2e}"
        off = (r["lse"][:, :, heads].reshape(-1).double() - lse).abs().max().item()
        assert off <= more + F32_LSE, f"lse off by {off:.2e}"
        off = _off(r["scores"][:, g], scores)
        assert off <= more + F32_SCORES, f"scores off by {off:.2e}"


@pytest.mark.parametrize("types", ["bf16-f32", "f32-f32", "bf16-bf16"])
@pytest.mark.parametrize("kind", ["spread", "positive", "grow"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [4, 9, 16])
def test_draft_over_long_lists(G, d, kind, types):
    """Lists in any order: all the tokens but some, shuffled except where the logits grow."""
    _gpu.lib()
    h, B = 2, 165
    qt, ot = _types(types)
    pool, K, V = _tokens(kind, h, d)
    kv = _cache(pool, B)
    q = _queries(kind, (B, G * h, d), qt)
    scale = 60.0 / (4 * d) if kind == "grow" else 1 / math.sqrt(d)
    g = torch.Generator().manual_seed(7)
    perm = (torch.arange(L) if kind == "grow" else torch.randperm(L, generator=g))[:L - 37].to(DEV)
    idx = perm.to(torch.int32).expand(B, h, -1).contiguous()
    cnt = torch.full((B, h), len(perm), dtype=torch.int32, device=DEV)
    r = ssd_kv4_draft_attn(kv, q, idx, cnt, scale, out_dtype=ot)
    torch.cuda.synchronize()
    assert ssd_status() == 0
    more = 60 * 2.0 ** -21 * (12 if qt == torch.float32 else 4) if kind == "grow" else 0.0
    for g in range(h):
        heads = slice(g * G, (g + 1) * G)
        out, lse, _ = _attend(q[:, heads].reshape(-1, d), K[g][perm], V[g][perm], torch.full((B * G,), L, device=DEV), scale)
        off = _off(r["out"][:, heads].reshape(-1, d), out)
        assert off <= more + (F32_OUT if ot == torch.float32 else BF16_OUT), f"out off by {off:.2e}"
        off = (r["lse"][:, heads].reshape(-1).double() - lse).abs().max().item()
        assert off <= more + F32_LSE, f"lse off by {off:.2e}"


def _sink(d, n, below):
    """One token `below` powers of two above n - 1 others of equal weight, and of the opposite value: the cache of 330
    such requests, the query and scale that make it so, and the output."""
    k, v = np.zeros((1, n, d)), np.ones((1, n, d))
    k[0, 0], v[0, 0] = 4.0 * _signs(d), -1.0
    ck, cv = _kv4.quantise(k), _kv4.quantise(v)
    pool = torch.from_numpy(np.ascontiguousarray(np.stack([_bytes(*ck), _bytes(*cv)], 1))).to(DEV)
    K, V = _kv4.values(ck[0][:, :2], ck[1][:, :2]), _kv4.values(cv[0][:, :2], cv[1][:, :2])
    scale = below * math.log(2) / (K[0, 0] @ _signs(d))
    w = (n - 1) * 2.0 ** -below
    return _cache(pool.view(KV4Cache.pool_shape(n // PAGE, 1, PAGE, d)), 330, n), scale, (V[0, 0, 0] + w * V[0, 1, 0]) / (1 + w)


@pytest.mark.parametrize("below", [31, 32.4])
@pytest.mark.parametrize("q_type", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("form", [(4, 128, 1), (4, 128, 5), (16, 128, 2), (4, 64, 1), (4, 64, 4), (4, 64, 5), (8, 64, 4), (4, 128, 0),
                                  (16, 128, 0), (4, 64, 0), (16, 64, 0)], ids=lambda f: f"G{f[0]}d{f[1]}n{f[2]}")
def test_a_flat_tail_far_below_one_token(form, q_type, below):
    """131071 tokens, each 2^-31 and less of the first one's weight: together 6.1e-5 (and 2.3e-5) of it, so without them
    the outputs are off by twice that, 1.2e-4 (4.6e-5).  What fp32 may lose: O is added up at most 256 times to nearest,
    half a step of the first token's part each, 256 * 2^-24 = 2^-16; P holds steps of 2^-34 of the largest, half of one a
    token, 2^17 * 2^-35 = 2^-18, twice (O and its sign against the first token's): 2^-17; the sum of the one thread that has
    the first token loses its tail, 1 / 64 of 6.1e-5, and the logits' rounding is 32 * 2^-24 of the tail: under 2^-19.
    n_cand 0: a draft over all the tokens."""
    _gpu.lib()
    G, d, nc = form
    n = 131072
    kv, scale, want = _sink(d, n, below)
    q = torch.from_numpy(_signs(d)).to(DEV, q_type).expand(330, max(nc, 1), G, d).contiguous()
    if nc:
        r = ssd_kv4_verify_attn(kv, q, nc, scale, want_scores=False)
    else:
        idx = torch.arange(n, dtype=torch.int32, device=DEV).expand(330, 1, n).contiguous()
        r = ssd_kv4_draft_attn(kv, q[:, 0].contiguous(), idx, torch.full((330, 1), n, dtype=torch.int32, device=DEV), scale)
    torch.cuda.synchronize()
    assert ssd_status() == 0
    off = ((r["out"].double() - want).abs().max() / abs(want)).item()
    assert off <= 2.0 ** -16 + 2.0 ** -17 + 2.0 ** -19, f"out off by {off:.2e}"
