"""Token log probabilities, entropies and top alternatives against their definition in 64 bits."""

import numpy as np
import pytest
import torch

import sparse_self_speculative_verify_gb300 as F

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def reference(x):
    """lse, entropy of rows x (float64 numpy)."""
    m = x.max(1)
    with np.errstate(invalid="ignore", divide="ignore"):
        z = np.where(np.isneginf(m)[:, None], 0.0, np.exp(x - m[:, None]))
        s = z.sum(1)
        lse = m + np.log(s)
        p = z / np.where(s > 0, s, 1)[:, None]
        ent = -(np.where(p > 0, p * np.log(np.where(p > 0, p, 1)), 0)).sum(1)
    return lse, ent


def check(x, r, k=0, tokens=None, rows=None):
    """x: the logits' values, float64 numpy [N, V]."""
    torch.cuda.synchronize()
    N, V = x.shape
    lse, ent = reference(x)
    # Sums of positive terms in fp32, each within 4 half steps of 2^-24 (the exponential) and its argument's own rounding
    # (2 of |x - m|, weighted by the term); at most V / 512 + 40 additions follow one another.
    with np.errstate(invalid="ignore"):
        p = np.where(np.isneginf(lse)[:, None], 0.0, np.exp(x - np.where(np.isneginf(lse), 0, lse)[:, None]))
        far = np.where(p > 0, p * (np.where(p > 0, np.abs(x - lse[:, None]), 0) + 1), 0).sum(1)
        far2 = np.where(p > 0, p * (np.where(p > 0, np.abs(x - lse[:, None]), 0) + 1) ** 2, 0).sum(1)
    e = 2.0 ** -24
    rel = e * (V / 512 + 48)
    tol = rel + 4 * e * far + 2 * e * np.abs(np.where(np.isneginf(lse), 0, lse))
    got = r["lse"].double().cpu().numpy()
    assert np.array_equal(np.isinf(got), np.isinf(lse))
    fin = np.isfinite(lse)
    assert (np.abs(got - lse)[fin] <= tol[fin]).all(), np.abs(got - lse)[fin].max()
    got = r["entropy"].double().cpu().numpy()
    assert (np.abs(got - ent) <= 2 * rel * (1 + far) + 8 * e * far2).all(), np.abs(got - ent).max()

    def close(lp, want, row):
        lp = lp.double().cpu().numpy()
        assert np.array_equal(np.isinf(lp), np.isinf(want))
        f = np.isfinite(want)
        assert (np.abs(lp - want)[f] <= (tol[row] + 4 * e * (np.abs(want) + np.abs(np.where(np.isneginf(lse), 0, lse))[row]))[f]).all()

    if tokens is not None:
        row = np.arange(N).repeat(tokens.size // N).reshape(tokens.shape) if rows is None else rows
        with np.errstate(invalid="ignore"):
            want = np.where(np.isneginf(x[row, tokens]), -np.inf, x[row, tokens] - lse[row])
        close(r["logprob"], want, row)
    if k:
        order = np.argsort(-x, axis=1, kind="stable")[:, :k]
        assert np.array_equal(r["top_ids"].cpu().numpy(), order)
        with np.errstate(invalid="ignore"):
            v = np.take_along_axis(x, order, 1)
            want = np.where(np.isneginf(v), -np.inf, v - lse[:, None])
        close(r["top_logprobs"], want, np.arange(N)[:, None].repeat(k, 1))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,V,k", [(1, 1, 1), (3, 7, 7), (2, 513, 5), (1, 32000, 8), (5, 50257, 20), (160, 4099, 64), (3, 151936, 32), (40, 1000, 0)])
def test_rows(dtype, N, V, k):
    g = torch.Generator().manual_seed(N * V)
    x = (torch.randn((N, V), generator=g) * 3).to(dtype)
    tok = torch.randint(0, V, (N, 3), generator=g, dtype=torch.int32)
    r = F.ssd_token_logprobs(x.to(DEV), tok.to(DEV), top_k=k)
    check(x.double().numpy(), r, k, tok.numpy())
    assert F.ssd_status() == 0


def test_strided_rows_of_every_alignment():
    g = torch.Generator().manual_seed(5)
    for dtype in (BF, F32):
        base = torch.randn((9, 1003), generator=g).to(dtype)
        for off in range(8):
            x = base.to(DEV)[:, off:off + 700 + off]
            tok = torch.randint(0, 700, (9,), generator=g, dtype=torch.int32)
            check(base[:, off:off + 700 + off].double().numpy(), F.ssd_token_logprobs(x, tok.to(DEV), top_k=9), 9, tok.numpy())


def special_rows(V):
    """Rows where a reduction goes wrong most easily."""
    rng = np.random.default_rng(3)
    rows = [np.full(V, 0.5), np.full(V, -np.inf), np.where(rng.random(V) < 0.9, -np.inf, rng.standard_normal(V)),
            np.linspace(-20, 20, V), np.linspace(20, -20, V), np.where(np.arange(V) == V - 1, 60.0, -60.0),
            np.where(np.arange(V) % 3 == 0, 2.0, 1.0), rng.integers(0, 3, V).astype(float)]
    few = np.full(V, -np.inf)
    few[[V // 7, V // 3, V - 2]] = [1.0, 3.0, 1.0]
    rows.append(few)
    low = np.full(V, float(torch.finfo(BF).min))
    rows += [low, np.where(np.arange(V) == 5, 0.0, low)]
    return np.stack(rows)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [64, 5000, 40001])
def test_special_rows(dtype, V):
    x = torch.from_numpy(special_rows(V)).to(dtype)
    tok = torch.stack([torch.full((len(x),), V - 2), torch.zeros(len(x))], 1).int()
    k = 20
    check(x.double().numpy(), F.ssd_token_logprobs(x.to(DEV), tok.to(DEV), top_k=k), k, tok.numpy())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_nan_and_infinity(dtype):
    V = 3001
    x = torch.randn((4, V), generator=torch.Generator().manual_seed(1)).to(dtype)
    x[0, 17] = float("nan")
    x[1, 2999] = float("inf")
    x[2, :] = float("nan")
    x[2, 5] = 1.0
    tok = torch.zeros((4,), dtype=torch.int32)
    r = F.ssd_token_logprobs(x.to(DEV), tok.to(DEV), top_k=4)
    for name in ("lse", "entropy", "logprob"):
        assert r[name][:3].isnan().all() and r[name][3:].isfinite().all(), name
    ids = r["top_ids"].cpu()
    assert 17 not in ids[0].tolist() and ids[1, 0] == 2999 and ids[2].tolist() == [5, -1, -1, -1]
    order = np.argsort(-x[0].double().nan_to_num(nan=-1e9).numpy(), kind="stable")[:4]
    assert ids[0].tolist() == order.tolist()


def test_tokens_of_chosen_rows():
    g = torch.Generator().manual_seed(2)
    x = torch.randn((6, 5003), generator=g).to(BF)
    rows = torch.randint(0, 6, (400,), generator=g, dtype=torch.int32)
    tok = torch.randint(0, 5003, (400,), generator=g, dtype=torch.int32)
    check(x.double().numpy(), F.ssd_token_logprobs(x.to(DEV), tok.to(DEV), rows=rows.to(DEV)), 0, tok.numpy(), rows.numpy())
    assert F.ssd_status() == 0
    rows[3], rows[7], tok[9], tok[11] = -1, 6, 5003, -1
    lp = F.ssd_token_logprobs(x.to(DEV), tok.to(DEV), rows=rows.to(DEV))["logprob"]
    assert F.ssd_status() == F.binding.FAULT_INDEX
    assert lp[3] == 0 and lp[[7, 9, 11]].isnan().all() and lp[0].isfinite()
    lp = F.ssd_token_logprobs(x.to(DEV), torch.tensor([0, 1, 2, 3, -1, 5003], dtype=torch.int32, device=DEV))["logprob"]
    assert F.ssd_status() == F.binding.FAULT_INDEX
    assert lp[4:].isnan().all() and lp[:4].isfinite().all()
