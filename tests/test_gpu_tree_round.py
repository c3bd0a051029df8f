"""Steps that draft trees, strung together as a server would: the tokens that a toy model emits are those that it emits one
after the other."""

import numpy as np
import pytest
import torch

import sparse_self_speculative_verify_gb300 as F

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
V, H_Q, H, D = 97, 4, 2, 64


class Toy:
    """One attention layer between an embedding and a readout: everything after a token follows from the tokens before."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
        self.q, self.k, self.v, self.w = r(V, H_Q, D), r(V, H, D), r(V, H, D), r(V, H_Q * D)
        for name in "qkvw":  # what the cache holds is what the definition uses
            setattr(self, name, getattr(self, name).float().double())

    def logits(self, tokens):
        """float64, after each token of a sequence."""
        t = torch.tensor(tokens)
        q, k, v = self.q[t], self.k[t].repeat_interleave(H_Q // H, 1), self.v[t].repeat_interleave(H_Q // H, 1)
        x = torch.einsum("ihd,jhd->hij", q, k) / D ** 0.5
        x = x.masked_fill(torch.ones(len(t), len(t)).triu(1).bool(), -float("inf"))
        return torch.einsum("hij,jhd->ihd", x.softmax(-1), v).reshape(len(t), -1) @ self.w.T

    def greedy(self, tokens, n):
        tokens = list(tokens)
        for _ in range(n):
            tokens.append(int(self.logits(tokens)[-1].argmax()))
        return tokens


def trees(rng, truth, at, n):
    """Parents and tokens of a tree that starts with truth[at]: the true continuation as far as chance has it, other tokens beside."""
    par, tok, right = [-1], [truth[at]], [0]  # (a true node's depth, or None)
    while len(par) < n:
        p = int(rng.integers(max(0, len(par) - 5), len(par)))
        true = right[p] is not None and rng.random() < 0.7
        par.append(p)
        tok.append(truth[at + right[p] + 1] if true else int(rng.integers(V)))
        right.append(right[p] + 1 if right[p] is not None and tok[-1] == truth[at + right[p] + 1] else None)
    return par, tok


@pytest.mark.parametrize("typical", [False, True])
def test_steps_emit_the_model_s_own_tokens(typical):
    rng = np.random.default_rng(5)
    toy, n, page, steps = Toy(1), 9, 16, 7
    prompts = [list(rng.integers(0, V, m)) for m in (3, 17, 40)]
    B = len(prompts)
    truth = [toy.greedy(p, steps * n + n + 2) for p in prompts]
    top = max(map(len, truth)) + 2 * n
    cap = -(-top // page)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)  # noqa: E731
    pool = torch.full((B * cap, 2, H, page, D), float("nan"), device=DEV)
    # The caches hold everything before the last token, which the first tree begins with.
    kv = F.KVCache(pool, torch.randperm(B * cap).int().view(B, cap).to(DEV), i32([0] * B), top)
    k, v, q = (getattr(toy, x).float().to(DEV) for x in "kvq")
    w = toy.w.float().to(DEV)
    longest = max(map(len, prompts)) - 1
    padded = i32([p[:-1] + [0] * (longest - len(p) + 1) for p in prompts]).long()
    F.ssd_kv_append(kv, k[padded].contiguous(), v[padded].contiguous())
    F.ssd_kv_advance(kv.seq_lens, i32([len(p) - 1 for p in prompts]), top)
    rnd = F.TreeRound(kv, H_Q, n, window=8, sink=2, max_path=6)
    said, accepted = [list(p) for p in prompts], 0
    for _ in range(steps):
        drawn = [trees(rng, truth[b], len(said[b]) - 1, n) for b in range(B)]
        parents, tokens = i32([d[0] for d in drawn]), i32([d[1] for d in drawn])
        counts = i32(rng.integers(1, n + 1, B))
        F.ssd_kv_append(kv, k[tokens.long()].contiguous(), v[tokens.long()].contiguous())
        # The draft's attention over the cache as it is: the newest token is the tree's root.
        F.ssd_kv_advance(kv.seq_lens, i32([1] * B), top)
        root = q[tokens[:, :1].long()].contiguous()
        d = rnd.draft(root)["out"]
        for b in range(B):
            L = len(said[b])
            seen = [t for t in range(L) if t < 2 or t > L - 1 - 8]
            rep = lambda x: x[torch.tensor(said[b])[seen]].repeat_interleave(H_Q // H, 1)  # noqa: E731
            x = torch.einsum("hd,jhd->hj", toy.q[said[b][-1]], rep(toy.k)) / D ** 0.5
            want = torch.einsum("hj,jhd->hd", x.softmax(-1), rep(toy.v))
            assert (d[b, 0].double().cpu() - want).abs().max() < 1e-4  # (sums of 64 and of 10 terms of size 1 to 10 in 32 bits: 1e-5)
        F.ssd_kv_advance(kv.seq_lens, counts - 1, top)
        out = rnd.verify(q[tokens.long()].contiguous(), parents, counts)["out"]
        logits = (out.flatten(2) @ w.T).view(B * n, V)
        s = rnd.score(logits, tokens, parents, top_k=2)
        target = s["top_ids"][:, 0].contiguous().view(B, n)
        if typical:  # so high a threshold that only the model's own token passes it
            lp = s["top_logprobs"][:, 1].max().item()
            r = rnd.accept(parents, tokens, target, counts, epsilon=float(np.exp(lp + 1e-4)), delta=1e9)
        else:
            r = rnd.accept(parents, tokens, target, counts)
        rnd.commit(counts)
        rnd.advance()
        for b in range(B):
            m = int(r["cnt"][b])
            said[b] += [int(tokens[b, j]) for j in r["path"][b, 1:m].tolist()] + [int(r["next"][b])]
            accepted += m - 1
        assert kv.seq_lens.tolist() == [len(t) - 1 for t in said]
        assert F.ssd_status() == 0
    assert accepted >= 5  # (0.7 per node that hangs on a true one)
    for b in range(B):
        assert said[b] == truth[b][:len(said[b])]
        at = torch.arange(len(said[b]) - 1)
        rows = kv.pool[kv.page_table[b].long().cpu()[at // page].to(DEV), :, :, (at % page).to(DEV)]
        t = torch.tensor(said[b][:-1], device=DEV)
        assert torch.equal(rows[:, 0], k[t]) and torch.equal(rows[:, 1], v[t])


def test_a_captured_step_replays():
    """verify, score, accept and commit as one graph, replayed on other inputs: the eager calls' results."""
    g = torch.Generator().manual_seed(2)
    B, n, h_q, h, d, page, top = 3, 12, 8, 2, 128, 16, 600
    cap = -(-top // page)
    table = torch.randperm(B * cap, generator=g).int().view(B, cap).to(DEV)
    pool = torch.randn((B * cap, 2, h, page, d), generator=g).bfloat16().to(DEV)
    caches = [F.KVCache(pool.clone(), table, torch.zeros((B,), dtype=torch.int32, device=DEV), top) for _ in range(2)]
    w = torch.randn((V, h_q * d), generator=g).bfloat16().to(DEV)
    q = torch.empty((B, n, h_q, d), dtype=torch.bfloat16, device=DEV)
    par, tok, cnt = (torch.zeros((B, n), dtype=torch.int32, device=DEV) for _ in range(2)), None, torch.full((B,), n, dtype=torch.int32, device=DEV)
    par, tok = par
    par[:, 0] = -1
    rounds = [F.TreeRound(c, h_q, n, window=64, max_path=5) for c in caches]

    def step(r):
        out = r.verify(q, par, cnt)["out"]
        s = r.score((out.flatten(2) @ w.T).view(B * n, V), tok, par, top_k=4)
        r.accept(par, tok, s["top_ids"][:, 0].contiguous().view(B, n), cnt)
        r.commit(cnt)
        return [r.out_t, r.lse_t, r.logprob, r.entropy, r.path, r.cnt, r.next, r.back, r.kv.pool, s["top_logprobs"]]

    q.normal_()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for c in caches:
            c.seq_lens.fill_(100)
        step(rounds[0])
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            kept = step(rounds[0])
    torch.cuda.synchronize()
    for k in range(4):
        lens = torch.randint(n, top + 1, (B,), generator=g, dtype=torch.int32)
        for c in caches:
            c.seq_lens.copy_(lens)
        caches[0].pool.copy_(pool)
        caches[1].pool.copy_(pool)
        q.copy_(torch.randn(q.shape, generator=g))
        parents = torch.stack([torch.tensor([-1] + [int(torch.randint(0, i, (1,), generator=g)) for i in range(1, n)]) for _ in range(B)])
        par.copy_(parents)
        tok.copy_(torch.randint(0, V, (B, n), generator=g))
        cnt.copy_(torch.randint(1, n + 1, (B,), generator=g))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in kept]
        want = step(rounds[1])
        torch.cuda.synchronize()
        assert F.ssd_status() == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want))
