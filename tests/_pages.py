"""The page calls' definitions in plain Python, for the tests: lists of pages, one row after the other."""

import numpy as np


class Pages:
    """A cache's pages: pool (numpy, [pages, 2, h_kv, page_size, ...]; 4-bit pools uint8 with d given), table,
    lens, refs; the methods do what the calls of the same name do."""

    def __init__(self, pool, table, lens, refs, max_len, d4=None):
        self.pool, self.table, self.lens, self.refs = pool.copy(), table.copy(), list(lens), refs.copy()
        self.max_len, self.d4, self.ps = max_len, d4, pool.shape[3]
        self.faults = set()

    def fork(self, src, dst):
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < len(self.lens) and 0 <= d < len(self.lens)) or s in dst or d in dst[:i]:
                self.faults.add("index")
                continue
            if not 0 <= self.lens[s] <= self.max_len:
                self.faults.add("seqlen")
                continue
            n = -(-self.lens[s] // self.ps)
            held = self.table[s, :n]
            if (self.table[d] >= 0).any() or any(not (0 <= p < len(self.refs)) or self.refs[p] <= 0 for p in held):
                self.faults.add("page")
                continue
            self.table[d, :n] = held
            for p in held:
                self.refs[p] += 1
            self.lens[d] = self.lens[s]

    def release(self, keep):
        for b, k in enumerate(keep):
            if k < 0:
                continue
            for j in range(-(-k // self.ps), self.table.shape[1]):
                p = self.table[b, j]
                if p < 0:
                    continue
                self.table[b, j] = -1
                if p >= len(self.refs) or self.refs[p] <= 0:
                    self.faults.add("page")
                else:
                    self.refs[p] -= 1
            if not 0 <= self.lens[b] <= self.max_len:
                self.faults.add("seqlen")
            else:
                self.lens[b] = min(self.lens[b], k)

    def reserve(self, counts):
        before = (self.table.copy(), self.refs.copy(), self.pool.copy())
        asks = {}
        for b, n in enumerate(counts):
            L = self.lens[b]
            if n < 0 or not 0 <= L <= L + n <= self.max_len:
                self.faults.add("seqlen")
                continue
            js = range(L // self.ps, -(-(L + n) // self.ps)) if n else []
            bad = False
            for j in js:
                p = self.table[b, j]
                bad |= (p >= len(self.refs) or self.refs[p] <= 0) if p >= 0 else (j == L // self.ps and L % self.ps > 0)
            if bad:
                self.faults.add("page")
            else:
                asks[b] = js
        holders = {}
        for b, js in asks.items():
            for j in js:
                holders.setdefault(int(self.table[b, j]), []).append(b)
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        for b, js in asks.items():
            for j in js:
                p = int(self.table[b, j])
                if p >= 0:
                    rows = holders[p]
                    if before[1][p] == 1 or (len(rows) == before[1][p] and rows[0] == b):
                        continue
                if not free:
                    self.table, self.refs, self.pool = before
                    self.faults.add("nopage")
                    return
                f = free.pop(0)
                self.table[b, j] = f
                self.refs[f] = 1
                if p >= 0:
                    self.refs[p] -= 1
                    live = self.lens[b] % self.ps
                    if j == self.lens[b] // self.ps and live:
                        for t in range(live):
                            self._copy(self.pool, p, t, self.pool, f, t)

    def _copy(self, a, p, t, b, q, u, heads=None):
        for g in range(a.shape[2]) if heads is None else heads:
            for w in range(2):
                if self.d4 is None:
                    b[q, w, g, u] = a[p, w, g, t]
                else:
                    d, x, y = self.d4, a[p, w, g].reshape(-1), b[q, w, g].reshape(-1)
                    psa, psb = a.shape[3], b.shape[3]
                    y[u * d // 2:(u + 1) * d // 2] = x[t * d // 2:(t + 1) * d // 2]
                    y[psb * d // 2 + u * d // 16:psb * d // 2 + (u + 1) * d // 16] = \
                        x[psa * d // 2 + t * d // 16:psa * d // 2 + (t + 1) * d // 16]

    def compact_to(self, to, src, dst, idx, cnt):
        """Only lists that are in order; faults are tested one by one."""
        old = self.pool.copy()
        for i, (s, d) in enumerate(zip(src, dst)):
            n = int(cnt[i, 0])
            for g in range(idx.shape[1]):
                for j in range(n):
                    t = int(idx[i, g, j])
                    self._copy(old, self.table[s, t // self.ps], t % self.ps, to.pool, to.table[d, j // to.ps], j % to.ps, [g])
            to.lens[d] = n

    def check(self):
        """Counts agree with the table."""
        want = np.bincount(self.table[self.table >= 0], minlength=len(self.refs))
        assert np.array_equal(want, self.refs)
