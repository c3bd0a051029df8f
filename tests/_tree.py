"""Plain 64-bit definitions for the tests of a step that drafts trees: attention by tree and by window over a paged cache,
token log probabilities, acceptance.  numpy, from the definitions; nothing here is shared with the library."""

import math

import numpy as np
import torch

EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step, relative


def sees(p, base, i, t, parents=None, window=None, sink=0):
    """Whether the query at position p = base + i sees token t."""
    if p < 0 or t > p:
        return False
    if window is not None:
        return t < sink or t > p - window
    if t < base:
        return True
    j = i
    while j >= 0:
        if base + j == t:
            return True
        j = int(parents[j])
    return False


def visible(L, c, n, parents=None, window=None, sink=0):
    """bool [n, L]."""
    m = np.zeros((n, max(L, 1)), bool)[:, :L]
    base = L - c
    for i in range(c):
        p = base + i
        if p < 0:
            continue
        if window is not None:
            m[i, max(0, p - window + 1):p + 1] = True
            m[i, :min(sink, p + 1)] = True
        else:
            m[i, :max(base, 0)] = True
            j = i
            while j >= 0 and base + j >= 0:
                m[i, base + j] = True
                j = int(parents[j])
    return m


def random_trees(B, n, rng, back=6):
    par = np.full((B, n), -1, np.int32)
    for i in range(1, n):
        par[:, i] = np.maximum(i - rng.integers(1, back + 1, B), 0)
    return par


class Case:
    """A cache on the CPU with NaN wherever no query of the call sees a token (slots behind the end among them), and free
    (-1) page-table entries where a page holds no seen token; queries, and the reference in 64 bits."""

    def __init__(self, lens, counts, n, h_q, h_kv, d, page, dtype, seed=0, parents=None, window=None, sink=0, lean=2.0, kscale=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        self.__dict__.update(lens=lens, counts=counts, n=n, h_q=h_q, h_kv=h_kv, d=d, page=page, dtype=dtype, B=B, window=window, sink=sink)
        self.parents = parents if parents is not None else random_trees(B, n, rng)
        self.max_len = max(max(lens), 1)
        cap = -(-self.max_len // page) + 1
        total = B * cap + 2
        perm = torch.randperm(total, generator=g)[:B * cap].view(B, cap)
        self.table = torch.full((B, cap), -1, dtype=torch.int32)
        self.pool = torch.full((total, 2, h_kv, page, d), float("nan"), dtype=dtype)
        u = torch.randn(d, generator=g) / math.sqrt(d)
        self.q = (torch.randn((B, n, h_q, d), generator=g) + lean * u).to(dtype)
        self.masks = []
        for b, (L, c) in enumerate(zip(lens, counts)):
            m = visible(L, c, n, self.parents[b], window, sink)
            self.masks.append(m)
            any_ = torch.from_numpy(m.any(0))
            for j in range(-(-L // page)):
                if any_[j * page:(j + 1) * page].any():
                    self.table[b, j] = perm[b, j]
            t = torch.nonzero(any_)[:, 0]
            if t.numel():
                k = torch.randn((t.numel(), h_kv, d), generator=g) * kscale
                k[torch.rand(t.numel(), generator=g) < 0.02] += 4.0 * u * math.sqrt(d) / 8
                self.pool[perm[b][t // page], 0, :, t % page] = k.to(dtype)
                self.pool[perm[b][t // page], 1, :, t % page] = torch.randn((t.numel(), h_kv, d), generator=g).to(dtype)
        self.scale = 1.0 / math.sqrt(d)

    def reference(self):
        """out, lse and their tolerances, float64 numpy."""
        B, n, G = self.B, self.n, self.h_q // self.h_kv
        out = np.zeros((B, n, self.h_q, self.d))
        lse = np.full((B, n, self.h_q), -np.inf)
        tol, tol_lse = np.zeros_like(out), np.zeros_like(lse)
        pool = self.pool.double().numpy()
        q = self.q.double().numpy()
        bf = self.dtype == torch.bfloat16
        e32 = 2.0 ** -24
        for b, (L, c) in enumerate(zip(self.lens, self.counts)):
            m = self.masks[b]
            t = np.nonzero(m.any(0))[0]
            if not t.size:
                continue
            pg = self.table[b].numpy()[t // self.page]
            for g in range(self.h_kv):
                K, V = (pool[pg, w, g, t % self.page] for w in (0, 1))
                for h in range(g * G, (g + 1) * G):
                    for i in range(c):
                        s = m[i, t]
                        if not s.any():
                            continue
                        k, v, qi = K[s], V[s], q[b, i, h]
                        x = k @ qi * self.scale
                        mx = x.max()
                        p = np.exp(x - mx)
                        z = p.sum()
                        lse[b, i, h] = mx + math.log(z)
                        p /= z
                        out[b, i, h] = p @ v
                        # Products are exact or rounded once, sums of d and of the tokens in fp32 (a tensor core may truncate: 2
                        # half steps), the exponential within 4 half steps, its argument within 2 of its size; each
                        # probability's error counts in the numerator and in the sum.
                        a = np.abs(k) @ np.abs(qi) * self.scale
                        logit = 2 * e32 * (self.d + 4) * a + 4 * e32 * np.abs(x - mx) + 4 * e32 * abs(mx) + 4 * e32
                        sums = 2 * e32 * (s.sum() + 16)
                        pv = p @ np.abs(v)
                        tol[b, i, h] = (p * logit) @ np.abs(v) + (p @ logit) * pv + 2 * sums * pv
                        if bf:  # probabilities and the result are rounded to bf16
                            tol[b, i, h] += EPS[torch.bfloat16] * (pv + np.abs(out[b, i, h]) + tol[b, i, h])
                        else:
                            tol[b, i, h] += 4 * e32 * np.abs(out[b, i, h])
                        tol_lse[b, i, h] = p @ logit + sums + 8 * e32 * (1 + abs(lse[b, i, h]))
        return out, lse, tol, tol_lse


def accept(parents, target, count, max_path, tokens=None, logprob=None, entropy=None, epsilon=0.0, delta=0.0):
    """(path, next) of one tree."""
    f = np.float32
    keep, depth = [], []
    for c in range(count):
        if c == 0:
            keep.append(True), depth.append(0)
            continue
        p = int(parents[c])
        ok = 0 <= p < c and keep[p]
        if ok and logprob is not None:
            low = f(math.log(delta)) - f(entropy[p])
            low = low if np.isnan(low) else min(low, f(math.log(epsilon)))
            ok = bool(f(logprob[c]) > low)
        elif ok:
            ok = tokens[c] == target[p]
        keep.append(ok), depth.append(depth[p] + 1 if ok else 0)
    good = [c for c in range(count) if keep[c] and depth[c] < max_path]
    if not good:
        return [], -1
    best = max(good, key=lambda c: (depth[c], -c))
    path, c = [], best
    while c > 0:
        path.append(c)
        c = int(parents[c])
    return [0] + path[::-1], int(target[best])
