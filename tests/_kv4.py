"""Plain 64-bit definitions of the 4-bit (NVFP4) cache and of attention over it, for the tests.

numpy, token by token from the bytes of the pool; nothing here is shared with the library."""

import math

import numpy as np

MAGNITUDE = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1 = np.concatenate([MAGNITUDE, -MAGNITUDE])
E4M3 = np.array([math.ldexp(b & 7, -9) if b < 8 else math.ldexp(8 + (b & 7), (b >> 3) - 10) for b in range(127)])


def nearest_even(x, grid):
    """Index into an ascending grid of the value nearest to x >= 0; ties to the even index, saturating."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    with np.errstate(invalid="ignore"):
        up, down = grid[hi] - x, x - grid[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def quantise(x, scale=1.0):
    """(codes uint8 [..., d], scale bytes uint8 [..., d / 16]) of float values x [..., d]."""
    y = np.asarray(x, np.float64) / scale
    y = np.where(np.isnan(y), 0.0, y).reshape(*y.shape[:-1], y.shape[-1] // 16, 16)
    s = nearest_even(np.minimum(np.abs(y).max(-1) / 6, 448.0), E4M3)
    sv = E4M3[s][..., None]
    with np.errstate(invalid="ignore", divide="ignore"):
        a = np.where(sv > 0, np.minimum(np.abs(y), 1e300) / np.where(sv > 0, sv, 1.0), 0.0)
    c = nearest_even(a, MAGNITUDE).astype(np.uint8)
    c |= (np.signbit(y) & (sv > 0)).astype(np.uint8) << 3
    return c.reshape(*c.shape[:-2], c.shape[-2] * 16), s.astype(np.uint8)


def values(codes, scales, scale=1.0):
    return E2M1[codes] * np.repeat(E4M3[scales], 16, axis=-1) * scale


def write_row(pool, page, which, head, slot, d, codes, scales):
    """Stores one row into pool uint8 [pages, 2, h_kv, page_size, 9 d / 16] (numpy, in place)."""
    ps = pool.shape[3]
    block = pool[page, which, head].reshape(-1)
    block[slot * d // 2:(slot + 1) * d // 2] = codes[0::2] | (codes[1::2] << 4)
    at = ps * d // 2 + slot * (d // 16)
    block[at:at + d // 16] = scales


def read_rows(pool, table, which, head, tokens, d, scale=1.0):
    """Values [len(tokens), d] of a request's tokens (table: its row of the page table)."""
    ps = pool.shape[3]
    out = np.zeros((len(tokens), d))
    for i, t in enumerate(tokens):
        block = pool[table[t // ps], which, head].reshape(-1)
        slot = t % ps
        b = block[slot * d // 2:(slot + 1) * d // 2]
        codes = np.empty(d, np.uint8)
        codes[0::2], codes[1::2] = b & 15, b >> 4
        at = ps * d // 2 + slot * (d // 16)
        out[i] = values(codes, block[at:at + d // 16], scale)
    return out


def attend(q, K, V, limit, scale):
    """Rows q [r, d] over K, V [n, d], row i seeing the first limit[i] tokens: out, lse, probabilities."""
    out, lse, P = np.zeros((len(q), V.shape[1])), np.full(len(q), -np.inf), np.zeros((len(q), len(K)))
    for i, n in enumerate(limit):
        n = min(max(int(n), 0), len(K))
        if n == 0:
            continue
        x = scale * (K[:n] @ q[i])
        m = x.max()
        z = np.exp(x - m).sum()
        lse[i] = m + np.log(z)
        P[i, :n] = np.exp(x - lse[i])
        out[i] = P[i, :n] @ V[:n]
    return out, lse, P


def verify(pool, table, lens, q, d, scale, k_scale=1.0, v_scale=1.0):
    """q [B, n_cand, h_q, d] (float64): dict of out, lse, scores (list of [h_kv, L_b])."""
    B, nc, hq, _ = q.shape
    h = pool.shape[2]
    G = hq // h
    out, lse, scores = np.zeros(q.shape), np.zeros(q.shape[:3]), []
    for b in range(B):
        L = int(lens[b])
        sc = np.zeros((h, L))
        for g in range(h):
            K, V = (read_rows(pool, table[b], w, g, range(L), d, s) for w, s in ((0, k_scale), (1, v_scale)))
            qs = q[b, :, g * G:(g + 1) * G].reshape(-1, d)
            lim = np.repeat([L - nc + 1 + i for i in range(nc)], G)
            o, z, P = attend(qs, K, V, lim, scale)
            out[b, :, g * G:(g + 1) * G] = o.reshape(nc, G, d)
            lse[b, :, g * G:(g + 1) * G] = z.reshape(nc, G)
            sc[g] = P.sum(0)
        scores.append(sc)
    return {"out": out, "lse": lse, "scores": scores}


def draft(pool, table, q, idx, cnt, d, scale, k_scale=1.0, v_scale=1.0):
    """q [B, h_q, d]; idx [B, h_kv, k], cnt [B, h_kv]."""
    B, hq, _ = q.shape
    h = pool.shape[2]
    G = hq // h
    out, lse = np.zeros(q.shape), np.zeros(q.shape[:2])
    for b in range(B):
        for g in range(h):
            toks = [int(t) for t in idx[b, g, :cnt[b, g]]]
            K, V = (read_rows(pool, table[b], w, g, toks, d, s) for w, s in ((0, k_scale), (1, v_scale)))
            o, z, _ = attend(q[b, g * G:(g + 1) * G], K, V, [len(toks)] * G, scale)
            out[b, g * G:(g + 1) * G], lse[b, g * G:(g + 1) * G] = o, z
    return {"out": out, "lse": lse}
