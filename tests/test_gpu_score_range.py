"""Scores of rows whose logits are large: banned tokens that hold a large negative number, rows far from 0."""

import numpy as np
import pytest
import torch

import sparse_self_speculative_verify_gb300 as F

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
E = 2.0 ** -24


def check(x, tokens, k, r, row=None):
    """x: the logits' values, float64 [N, V], all finite; tokens [N, m], or [M] with row [M].  Everything relative to the row's maximum m, so that
    no tolerance but that of the log-sum-exp, m + ln s, grows with m."""
    torch.cuda.synchronize()
    N, V = x.shape
    m = x.max(1)
    z = x - m[:, None]
    p = np.exp(z)
    s = p.sum(1)
    p /= s[:, None]
    lns = np.log(s)
    ent = lns - (p * z).sum(1)
    # Sums of positive terms: at most V / 512 + 40 additions in fp32 follow one another.  A term's exponent is rounded to half a
    # step of its size (the factor log2 e too), the exponential lies within 4 half steps; where sums get another reference they take
    # a factor within 4 more, and those of before it count e^-4 at most.  An exponent's error counts with the term, in the entropy
    # times the term's own logarithm.
    rel = E * (V / 512 + 48)
    far = (p * (1 - z)).sum(1)
    far2 = (p * (1 - z) ** 2).sum(1)
    tol = rel + 4 * E * far
    got = {n: r[n].double().cpu().numpy() for n in ("lse", "entropy", "logprob")}
    assert all(np.isfinite(v).all() for v in got.values()), {n: np.argwhere(~np.isfinite(v))[:4].tolist() for n, v in got.items()}
    # One addition more; the last step of m + ln s.
    assert (np.abs(got["lse"] - (m + lns)) <= tol + 2 * E * (np.abs(m + lns) + lns)).all()
    assert (np.abs(got["entropy"] - ent) <= 2 * rel * (1 + far) + 8 * E * far2 + 4 * E * lns).all(), np.abs(got["entropy"] - ent).max()

    def close(lp, want, at, more=0.0):  # x - m, ln s and their difference are rounded
        diff = np.abs(lp - want)
        assert (diff <= tol[at] + 4 * E * (np.abs(want) + 2 * lns[at] + 1) + more).all(), diff.max()

    if row is None:
        at = np.arange(N)[:, None].repeat(tokens.shape[1], 1)
        close(got["logprob"], z[at, tokens] - lns[at], at)
    else:  # (many tokens: relative to the rounded log-sum-exp)
        close(got["logprob"], z[row, tokens] - lns[row], row, 4 * E * np.abs(m + lns)[row])
    if k:
        order = np.argsort(-x, axis=1, kind="stable")[:, :k]
        assert np.array_equal(r["top_ids"].cpu().numpy(), order)
        at = np.arange(N)[:, None].repeat(k, 1)
        lp = r["top_logprobs"].double().cpu().numpy()
        assert np.isfinite(lp).all()
        close(lp, np.take_along_axis(z, order, 1) - lns[:, None], at)


def banned_rows(V, ban):
    """Rows whose banned tokens hold `ban`: a tenth of them, nine tenths, all but a few, long stretches, everything."""
    rng = np.random.default_rng(V)
    rows = [np.where(rng.random(V) < share, ban, 3 * rng.standard_normal(V)) for share in (0.1, 0.9)]
    few = np.full(V, ban)
    few[[0, V // 3, V // 2 + 1]] = [1.5, -2.0, 1.0]
    last = np.full(V, ban)
    last[-1] = 0.25
    half = np.arange(V) < V // 2
    rows += [few, last, np.where(half, ban, 3 * rng.standard_normal(V)), np.where(half, 3 * rng.standard_normal(V), ban), np.full(V, ban)]
    rows.append(np.where(half, ban, ban / 2))
    return np.stack(rows)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [61, 5000, 151936])
@pytest.mark.parametrize("ban", [-1e4, -1e5, -1e7, -1e9, -1e10, -1e12, -1e15, -1e18, -1e20, -1e30, -1e35, -1e36, -3e37, -1e38, -3e38])
def test_banned_by_a_finite_number(dtype, V, ban):
    x = torch.from_numpy(banned_rows(V, ban)).to(dtype)
    tok = torch.stack([torch.zeros(len(x)), torch.full((len(x),), V // 3), torch.full((len(x),), V - 1)], 1).int()
    check(x.double().numpy(), tok.long().numpy(), 20, F.ssd_token_logprobs(x.to(DEV), tok.to(DEV), top_k=20))
    assert F.ssd_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [8, 61, 5000, 151936])
@pytest.mark.parametrize("size", [2000.0, 3e4, 1e5, 1e6, 4e6, 5e6, 1e7, 2e7, 1e8, 1e9, 1e10, 1e20, 1e30, 1e38])
def test_rows_far_from_zero(dtype, V, size):
    """All of one value, spread around it, rising and falling between 0 and it, either sign."""
    rng = np.random.default_rng(V)
    ramp = np.linspace(0, 1, V)
    rows = [np.full(V, size), size + 3 * rng.standard_normal(V), size * (1 + 1e-3 * rng.standard_normal(V)), size * ramp, size * ramp[::-1],
            size + 40 * ramp, size + 40 * ramp[::-1]]
    x = torch.from_numpy(np.stack(rows + [-r for r in rows])).to(dtype)
    tok = torch.stack([torch.zeros(len(x)), torch.full((len(x),), V // 2), torch.full((len(x),), V - 1)], 1).int()
    check(x.double().numpy(), tok.long().numpy(), 5, F.ssd_token_logprobs(x.to(DEV), tok.to(DEV), top_k=5))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_a_batch_beside_one_another(dtype):
    """As many rows as leave one block for each; and more tokens than the rows' blocks look up themselves."""
    rng = np.random.default_rng(4)
    x = np.concatenate([banned_rows(4099, b) for b in (-1e4, -1e10, -1e20, -1e30)] * 30)
    x[3::11] += 1e6
    x = torch.from_numpy(x).to(dtype)
    N, V = x.shape
    tok = torch.from_numpy(rng.integers(0, V, (N, 2))).int()
    check(x.double().numpy(), tok.long().numpy(), 7, F.ssd_token_logprobs(x.to(DEV), tok.to(DEV), top_k=7))
    row, tok = (torch.from_numpy(rng.integers(0, n, 5000)).int() for n in (N, V))
    check(x.double().numpy(), tok.long().numpy(), 0, F.ssd_token_logprobs(x.to(DEV), tok.to(DEV), rows=row.to(DEV)), row.long().numpy())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_infinities_and_nan_among_banned_tokens(dtype):
    V = 5003
    x = torch.full((5, V), -1e10)
    x[:, 4000] = 1.0
    x[0, 9], x[1, 4500], x[2, 11] = float("nan"), float("nan"), float("inf")
    x[3, ::2] = -float("inf")
    x[4, ::2], x[4, 4000] = -float("inf"), -1e10
    x = x.to(dtype)
    tok = torch.full((5,), 4001, dtype=torch.int32)
    r = F.ssd_token_logprobs(x.to(DEV), tok.to(DEV), top_k=1)
    torch.cuda.synchronize()
    for name in ("lse", "entropy", "logprob"):
        assert r[name][:3].isnan().all() and r[name][3:].isfinite().all(), name
    # Rows 3 and 4: the odd tokens are equal (V // 2 of them), and in row 4 token 4000 as well; the other even ones are -inf.
    for row, n in ((3, V // 2), (4, V // 2 + 1)):
        assert r["lse"][row] == x[row, 1].float()  # (ln n is far below a step)
        # A few steps of 2^-24 of 8.
        assert abs(r["entropy"][row].item() - np.log(n)) < 1e-5 and abs(r["logprob"][row].item() + np.log(n)) < 1e-5
    assert r["top_ids"].flatten().tolist() == [4000, 4000, 11, 1, 1]
