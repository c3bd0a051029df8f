"""Operators of a decoding step that drafts a tree of tokens, as cases to be measured.

Five operators over a paged KV cache and the logits that belong to its tokens:
  tree     attention of a request's drafted tree over its whole cache: the nodes are the last tokens of
           the cache, a node sees all tokens before the tree, its ancestors and itself
  window   attention of a request's last tokens with a sliding window and a few first tokens that stay
           visible: the draft's cheap attention (one token), and prompts of a model that has such layers
  score    log probabilities of given tokens under rows of logits, with each row's entropy and its
           top alternatives
  accept   the longest accepted path of a drafted tree, by equality with the model's own tokens or by a
           threshold on the drafted tokens' probabilities
  commit   the accepted path's K and V rows moved together behind the tokens before the tree
"""

import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------


def listed():
    return [
        # One short request in 32 bits: the smallest attention call, where latency counts.
        dict(name="tree one short", op="tree", batch=1, n=5, ragged=False, lo=300, hi=300, h_q=8, h_kv=2, d=64, page=16, dtype="f32"),
        # A batch of conversations, 16 drafted nodes each.
        dict(name="tree batch", op="tree", batch=32, n=16, ragged=False, lo=2048, hi=8192, h_q=32, h_kv=8, d=128, page=16, dtype="bf16"),
        # Long contexts with wide trees of different sizes: 320 query rows a KV head.
        dict(name="tree wide long", op="tree", batch=8, n=64, ragged=True, lo=16384, hi=65536, h_q=40, h_kv=8, d=128, page=32, dtype="bf16"),
        # The draft's token of a batch: 1024 recent tokens and 4 first ones of a long cache.
        dict(name="window draft", op="window", batch=32, n=1, ragged=False, lo=2048, hi=8192, window=1024, sink=4, h_q=32, h_kv=8, d=128, page=16, dtype="bf16"),
        # Chunks of prompts behind earlier ones: the compute bound end.
        dict(name="window prompts", op="window", batch=4, n=4096, ragged=True, lo=4096, hi=8192, window=2048, sink=64, h_q=32, h_kv=8, d=128, page=16, dtype="bf16"),
        # Odd sizes: three heads a group, d = 64, a window that ends inside pages.
        dict(name="window odd chunk", op="window", batch=17, n=33, ragged=True, lo=40, hi=3000, window=301, sink=5, h_q=9, h_kv=3, d=64, page=8, dtype="bf16"),
        # One sampled token of one request.
        dict(name="score one row", op="score", rows=1, vocab=32000, tokens=1, k=8, dtype="f32", banned=0.0),
        # Every node of 32 trees of 16 under its parent's row, with the top alternatives that the next tree grows from.
        dict(name="score trees", op="score", rows=512, vocab=151936, tokens=512, k=20, dtype="bf16", banned=0.01),
        # Greedy or sampled: a node is kept where the model gave the same token.
        dict(name="accept equal", op="accept", batch=32, n=16, ragged=False, most=8, typical=False),
        # By probability, many requests with wide trees.
        dict(name="accept typical", op="accept", batch=512, n=255, ragged=True, most=16, typical=True),
        # One layer's cache after a step of a batch: the accepted nodes' rows close up.
        dict(name="commit batch", op="commit", batch=32, n=16, ragged=False, lo=20, hi=500, most=8, h_kv=8, d=128, page=16, dtype="bf16"),
        dict(name="commit many", op="commit", batch=160, n=63, ragged=True, lo=1, hi=400, most=12, h_kv=8, d=128, page=32, dtype="bf16"),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "window", "window", "window", "score", "score", "accept", "commit"])
    ragged = rng.random() < 0.6
    if op == "score":
        vocab = _logint(rng, 90, 160000)
        rows = _logint(rng, 1, min(2000, 70_000_000 // vocab))
        return dict(op=op, rows=rows, vocab=vocab, tokens=_logint(rng, 1, 700), k=rng.choice([0, 1, 5, 20, 32]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    banned=rng.choice([0.0, 0.02, 0.5]))
    if op == "accept":
        return dict(op=op, batch=_logint(rng, 1, 512), n=_logint(rng, 1, 256), ragged=ragged, most=rng.randint(1, 16), typical=rng.random() < 0.5)
    h_kv = rng.choice([1, 2, 3, 8])
    d = rng.choice([64, 128, 128])
    page = rng.choice([8, 16, 16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    batch = _logint(rng, 1, 40)
    if op == "commit":
        n = _logint(rng, 1, 128)
        hi = _logint(rng, 2, 600)
        return dict(op=op, batch=batch, n=n, ragged=ragged, lo=max(1, hi // 4), hi=hi, most=rng.randint(1, 12), h_kv=h_kv, d=d, page=page, dtype=dtype)
    G = rng.choice([1, 2, 3, 4, 4, 5, 8])
    if op == "tree":
        n = _logint(rng, 1, 96)
        top = _logint(rng, n + 1, max(n + 2, min(200000 // batch, (40_000_000 if dtype == "bf16" else 4_000_000) // (batch * n * G))))
        return dict(op=op, batch=batch, n=n, ragged=ragged, lo=max(n, top // rng.choice([1, 2, 4])), hi=top, h_q=G * h_kv, h_kv=h_kv, d=d, page=page, dtype=dtype)
    n = rng.choice([1, 1, _logint(rng, 2, 40), _logint(rng, 40, 3000)])
    top = _logint(rng, n + 1, max(n + 2, min(200000 // batch, (60_000_000 if dtype == "bf16" else 4_000_000) // (batch * n * G), 16384)))
    return dict(op=op, batch=batch, n=n, ragged=ragged, lo=max(n, top // rng.choice([1, 2, 4])), hi=top, window=_logint(rng, 1, 4096), sink=rng.choice([0, 1, 4, 130]),
                h_q=G * h_kv, h_kv=h_kv, d=d, page=page, dtype=dtype)


# ------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _sizes(case, seed):
    """Lengths (with the tree or chunk) and counts of a case's requests."""
    g = torch.Generator().manual_seed(int(seed) * 7919 + 17)
    B, n = case["batch"], case["n"]
    counts = torch.randint((n + 1) // 2, n + 1, (B,), generator=g) if case["ragged"] else torch.full((B,), n)
    lens = torch.randint(case["lo"], case["hi"] + 1, (B,), generator=g) if "lo" in case else counts
    return [int(x) for x in lens], [int(x) for x in counts]


def _trees(B, n, gen):
    """parents [B, n]: node 0 is the root (parent -1), every other node hangs on one of the eight before it."""
    i = torch.arange(n, device=DEV)
    back = torch.randint(1, 9, (B, n), generator=gen, device=DEV)
    par = (i[None] - back).clamp(min=0)
    par[:, 0] = -1
    return par.to(torch.int32)


def _table(gen, lens, page, most):
    """A shuffled page table for rows of `lens` tokens, and the pool's size, which holds rows of `most`."""
    cap = -(-most // page)
    total = len(lens) * cap + 3
    perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)[:len(lens) * cap].view(len(lens), cap)
    need = torch.tensor([-(-x // page) for x in lens], device=DEV)
    table = torch.where(torch.arange(cap, device=DEV)[None] < need[:, None], perm, -1)
    return table.contiguous(), total


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    i32 = dict(dtype=torch.int32, device=DEV)
    rnd = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    s = dict(case=dict(case))
    op = case["op"]
    if op == "score":
        R, V, M = case["rows"], case["vocab"], case["tokens"]
        x = rnd(R, V) * 2.5
        x[torch.rand((R, V), generator=gen, device=DEV) < case["banned"]] = -math.inf  # tokens that a grammar forbids
        x[:, 0] = 0.0  # one at least is allowed
        s["logits"] = x.to(_type(case))
        s["at"] = torch.randint(0, R, (M,), generator=gen, **i32)
        s["tokens"] = torch.randint(0, V, (M,), generator=gen, **i32)
        return s
    B, n = case["batch"], case["n"]
    lens, counts = _sizes(case, seed)
    s["counts"] = torch.tensor(counts, **i32)
    if op in ("tree", "accept", "commit"):
        s["parents"] = _trees(B, n, gen)
    if op == "accept":
        # Few tokens, so that children often match; probabilities around the thresholds.
        s["tokens"] = torch.randint(0, 50000, (B, n), generator=gen, **i32)
        s["target"] = torch.randint(0, 50000, (B, n), generator=gen, **i32)
        child = torch.rand((B, n), generator=gen, device=DEV) < 0.6
        at = torch.where(child, s["parents"].clamp(min=0), n).long()  # the model's token after a node: often its last child's
        last = torch.full((B, n + 1), -1, device=DEV).scatter_reduce_(1, at, torch.arange(n, device=DEV).expand(B, n).contiguous(), "amax")[:, :n]
        s["target"] = torch.where(last >= 0, s["tokens"].gather(1, last.clamp(min=0)), s["target"])
        if case["typical"]:
            s["logprob"] = -3.0 * torch.rand((B, n), generator=gen, device=DEV)
            s["entropy"] = 4.0 * torch.rand((B, n), generator=gen, device=DEV)
        return s
    h, d, page = case["h_kv"], case["d"], case["page"]
    if op == "commit":
        lens = [a + c for a, c in zip(lens, counts)]  # the tokens before the tree, and its nodes
        most = case["hi"] + n
        # An accepted path: ascending nodes from the root on.
        pick = torch.rand((B, n), generator=gen, device=DEV)
        pick[:, 0] = -1.0
        live = torch.arange(n, device=DEV)[None] < s["counts"][:, None]
        m = min(case["most"], n)
        s["cnt"] = (torch.randint(1, m + 1, (B,), generator=gen, device=DEV)).minimum(s["counts"]).to(torch.int32)
        order = torch.where(live, pick, 2.0).argsort(dim=1)[:, :m]
        kept = torch.arange(m, device=DEV)[None] < s["cnt"][:, None]
        path = torch.where(kept, order, n).sort(dim=1).values
        s["path"] = torch.where(kept, path, -1).to(torch.int32).contiguous()
    else:
        most = case["hi"]
    s["lens"] = torch.tensor(lens, **i32)
    s["max_len"] = most
    s["table"], total = _table(gen, lens, page, most)
    s["pool"] = torch.empty((total, 2, h, page, d), dtype=_type(case), device=DEV)
    s["pool"].normal_(generator=gen)
    if op != "commit":
        # Some keys lean on a direction that the queries share, as attention that concentrates does.
        u = rnd(d) / math.sqrt(d)
        some = torch.rand((total, h, page, 1), generator=gen, device=DEV) < 0.02
        s["pool"][:, 0] += (4.0 * some * u).to(_type(case))
        s["q"] = (rnd(B, n, case["h_q"], d) + 2.0 * u).to(_type(case))
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:-1], dtype=torch.float32, device=DEV)
    return s


# ------------------------------------------------------------------------------------------------
# The plain forms
# ------------------------------------------------------------------------------------------------


def _rows_of(s, which):
    """K or V of every request in 32 bits: [B, h, max_len, d], zeros behind its end."""
    t = torch.arange(s["max_len"], device=DEV)
    page = s["case"]["page"]
    p = s["table"][:, t // page].clamp(min=0).long()
    x = s["pool"][p, which, :, t % page].transpose(1, 2).float()  # indexing puts the heads last but one
    return torch.where((t[None] < s["lens"][:, None])[:, None, :, None], x, 0.0)


def _ancestors(parents):
    """[B, n, n]: whether node j is node i or an ancestor of it, by doubling the reach."""
    B, n = parents.shape
    a = torch.zeros((B, n, n + 1), device=DEV)
    a.scatter_(2, torch.where(parents >= 0, parents, n).long()[..., None], 1.0)
    a = a[..., :n] + torch.eye(n, device=DEV)
    for _ in range(max(1, (n - 1).bit_length())):
        a = (a @ a > 0).float()
    return a > 0


def _visible(s):
    """[B, n, max_len]: what the queries see."""
    case = s["case"]
    n = case["n"]
    t = torch.arange(s["max_len"], device=DEV)[None, None]
    i = torch.arange(n, device=DEV)[None, :, None]
    base = (s["lens"] - s["counts"])[:, None, None]
    live = i < s["counts"][:, None, None]
    if case["op"] == "window":
        p = base + i
        return live & (t <= p) & ((t < case["sink"]) | (t > p - case["window"]))
    j = (t - base).clamp(0, n - 1).expand(-1, n, -1)
    seen = _ancestors(s["parents"]).gather(2, j)
    return live & ((t < base) | ((t < s["lens"][:, None, None]) & seen))


def _plain_attention(s):
    case = s["case"]
    B, n, h, d = case["batch"], case["n"], case["h_kv"], case["d"]
    G = case["h_q"] // h
    q = s["q"].float().view(B, n, h, G, d).transpose(1, 2).reshape(B, h, n * G, d)
    seen = _visible(s).repeat_interleave(G, dim=1)[:, None]
    x = q @ _rows_of(s, 0).transpose(-1, -2)
    x *= 1.0 / math.sqrt(d)
    x.masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    x -= torch.where(m == -math.inf, 0.0, m)
    x.exp_()
    z = x.sum(-1, keepdim=True)
    o = (x @ _rows_of(s, 1)) / torch.where(z > 0, z, 1.0)
    lse = torch.where(z > 0, m + torch.log(z), -math.inf)
    back = lambda y: y.view(B, h, n, G, -1).transpose(1, 2).reshape(B, n, h * G, -1)  # noqa: E731
    return {"out": back(o).to(s["q"].dtype), "lse": back(lse).squeeze(-1)}


def _plain_score(s):
    k = s["case"]["k"]
    x = s["logits"].float()
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1)
    lse = m[:, 0] + torch.log(z)
    entropy = torch.log(z) - torch.where(e > 0, e * (x - m), 0.0).sum(-1) / z
    at = s["at"].long()
    res = {"logprob": x[at, s["tokens"].long()] - lse[at], "entropy": entropy, "lse": lse}
    if k:
        v, i = torch.sort(x, dim=-1, descending=True, stable=True)  # equal ones: the lowest index first
        res["top_ids"] = i[:, :k].to(torch.int32)
        res["top_logprobs"] = v[:, :k] - lse[:, None]
    return res


EPSILON, DELTA = 0.3, 0.6


def _plain_accept(s):
    case = s["case"]
    B, n, most = case["batch"], case["n"], case["most"]
    par = s["parents"].clamp(min=0).long()
    i = torch.arange(n, device=DEV)
    if case["typical"]:
        low = torch.full((), math.log(EPSILON), device=DEV)
        ok = s["logprob"] > torch.minimum(low, math.log(DELTA) - s["entropy"].gather(1, par))
    else:
        ok = s["tokens"] == s["target"].gather(1, par)
    ok = (ok & (s["parents"] >= 0)) | (i == 0)
    ok &= i[None] < s["counts"][:, None]
    depth = (s["parents"] >= 0).long()
    up = par
    for _ in range(max(1, (n - 1).bit_length())):
        ok = ok & ok.gather(1, up)
        depth = depth + depth.gather(1, up)
        up = up.gather(1, up)
    best = torch.where(ok & (depth < most), depth * n + (n - 1 - i), -1).amax(1)
    node = torch.where(best >= 0, n - 1 - best % n, 0)
    cnt = torch.where(best >= 0, torch.div(best, n, rounding_mode="floor") + 1, 0)
    path = torch.full((B, most), -1, dtype=torch.int64, device=DEV)
    cur = node
    for k in range(min(most, n)):  # from the deepest node up
        at = (cnt - 1 - k).clamp(min=0)[:, None]
        path.scatter_(1, at, torch.where((k < cnt)[:, None], cur[:, None], path.gather(1, at)))
        cur = par.gather(1, cur[:, None])[:, 0]
    nxt = torch.where(cnt > 0, s["target"].gather(1, node[:, None])[:, 0], -1)
    i32 = torch.int32
    return {"path": path.to(i32), "cnt": cnt.to(i32), "next": nxt.to(i32), "advance": (cnt - s["counts"]).to(i32)}


def _plain_commit(s):
    m, page, table = s["path"].shape[1], s["case"]["page"], s["table"].long()
    j = torch.arange(m, device=DEV)[None]
    live = j < s["cnt"][:, None]
    base = (s["lens"] - s["counts"])[:, None]
    frm, to = (base + s["path"])[live].long(), (base + j)[live].long()
    b = torch.arange(live.shape[0], device=DEV)[:, None].expand_as(live)[live]
    s["pool"][table[b, to // page], :, :, to % page] = s["pool"][table[b, frm // page], :, :, frm % page]
    return s["pool"]


# ------------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------------


def run(state):
    s = state
    case = s["case"]
    op = case["op"]
    if not own:
        return {"tree": _plain_attention, "window": _plain_attention, "score": _plain_score, "accept": _plain_accept, "commit": _plain_commit}[op](s)
    import sparse_self_speculative_verify_gb300 as F
    if op == "score":
        r = F.ssd_token_logprobs(s["logits"], s["tokens"], rows=s["at"], top_k=case["k"])
        return {k: v for k, v in r.items() if v is not None}
    if op == "accept":
        more = dict(logprob=s["logprob"], entropy=s["entropy"], epsilon=EPSILON, delta=DELTA) if case["typical"] else {}
        return F.ssd_tree_accept(s["parents"], s["tokens"], s["target"], counts=s["counts"], max_path=case["most"], **more)
    if "cache" not in s:  # the framework's handle of a cache, made once and kept beside its tensors
        s["cache"] = F.KVCache(s["pool"], s["table"], s["lens"], s["max_len"])
    if op == "commit":
        F.ssd_tree_commit(s["cache"], s["path"], s["cnt"], case["n"], counts=s["counts"])
        return s["pool"]
    scale = 1.0 / math.sqrt(case["d"])
    if op == "tree":
        return F.ssd_tree_attn(s["cache"], s["q"], s["parents"], scale, counts=s["counts"], out=s["out"], lse=s["lse"])
    return F.ssd_window_attn(s["cache"], s["q"], case["window"], case["sink"], scale, counts=s["counts"], out=s["out"], lse=s["lse"])


def work(case):
    """Bytes and operations that a pass cannot do without, with every length and count at the middle of its range."""
    op = case["op"]
    if op == "score":
        e = 2 if case["dtype"] == "bf16" else 4
        R, V = case["rows"], case["vocab"]
        return {"bytes": R * V * e + R * (8 + 8 * case["k"]) + case["tokens"] * 12, "flops": 6.0 * R * V}
    B, n = case["batch"], case["n"]
    c = n * 0.75 if case["ragged"] else float(n)
    if op == "accept":
        return {"bytes": B * (c * (20 if case["typical"] else 12) + 4 * case["most"] + 16), "flops": 8.0 * B * c}
    h, d = case["h_kv"], case["d"]
    e = 2 if case["dtype"] == "bf16" else 4
    row = 2 * h * d * e
    if op == "commit":
        m = (1 + min(case["most"], n)) / 2
        return {"bytes": B * m * (2 * row + 4), "flops": 0}
    mid = (case["lo"] + case["hi"]) / 2
    rows = B * c * case["h_q"]
    if op == "tree":
        tokens, pairs = mid, c * (mid - c / 2)
    else:
        W, S = case["window"], case["sink"]
        tokens = min(mid, W + c - 1 + S)
        first = mid - c  # tokens before the chunk
        seen = lambda p: min(p + 1, W + S)  # noqa: E731
        pairs = c * (seen(first) + 4 * seen(first + c / 2) + seen(mid - 1)) / 6
    return {"bytes": B * tokens * row + rows * (2 * d * e + 4), "flops": 4.0 * B * pairs * case["h_q"] * d}


# ------------------------------------------------------------------------------------------------
# The definition in 64 bits
# ------------------------------------------------------------------------------------------------


def _seen_by(case, s, b, i, L, c):
    """The tokens that query i of request b sees, from the definition."""
    p = L - c + i
    if case["op"] == "window":
        first = list(range(min(case["sink"], p + 1)))
        return first + list(range(max(case["sink"], p - case["window"] + 1), p + 1))
    up, chain = i, []
    par = s["par_host"][b]
    while up >= 0:
        chain.append(L - c + up)
        up = par[up]
    return (L - c, chain)


def _exact_attention(case, s):
    h, G, page = case["h_kv"], case["h_q"] // case["h_kv"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    if case["op"] == "tree":
        s["par_host"] = s["parents"].tolist()
    for b, (L, c) in enumerate(zip(s["lens"].tolist(), s["counts"].tolist())):
        pages = s["table"][b, :-(-L // page)].long()
        for i0 in range(0, c, 512):  # so many queries at once
            i1 = min(c, i0 + 512)
            hidden = torch.ones((i1 - i0, L), dtype=torch.bool)
            for i in range(i0, i1):
                seen = _seen_by(case, s, b, i, L, c)
                if case["op"] == "tree":
                    hidden[i - i0, :seen[0]] = False
                    seen = seen[1]
                hidden[i - i0, seen] = False
            hidden = hidden.to(DEV)[:, None]
            for g in range(h):
                K, V = (s["pool"][pages, w, g].flatten(0, 1)[:L].double() for w in (0, 1))
                y = s["q"][b, i0:i1, g * G:(g + 1) * G].double() @ K.T / math.sqrt(case["d"])
                y = y.masked_fill(hidden, -math.inf)
                z = torch.logsumexp(y, dim=-1)
                lse[b, i0:i1, g * G:(g + 1) * G] = z
                out[b, i0:i1, g * G:(g + 1) * G] = torch.exp(y - z[..., None]) @ V
    return {"out": out, "lse": lse}


def _exact_score(case, s):
    k = case["k"]
    R = case["rows"]
    lse = torch.empty((R,), dtype=torch.float64, device=DEV)
    entropy = torch.empty_like(lse)
    top = torch.empty((R, k), dtype=torch.float64, device=DEV)
    for r in range(R):
        x = s["logits"][r].double()
        lse[r] = torch.logsumexp(x, 0)
        lp = (x - lse[r])[torch.isfinite(x)]
        entropy[r] = -(lp.exp() * lp).sum()
        if k:
            top[r] = (x - lse[r]).sort(descending=True).values[:k]
    at = s["at"].long()
    res = {"logprob": s["logits"][at, s["tokens"].long()].double() - lse[at], "entropy": entropy, "lse": lse}
    return res | ({"top_ids": None, "top_logprobs": top} if k else {})


def _exact_commit(case, s):
    pool, page = s["pool"].double(), case["page"]
    for b, (L, c, m) in enumerate(zip(s["lens"].tolist(), s["counts"].tolist(), s["cnt"].tolist())):
        pages = s["table"][b].long()
        t = torch.arange(L - c, L, device=DEV)
        rows = pool[pages[t // page], :, :, t % page]
        rows[:m] = rows[s["path"][b, :m].long()]  # behind the kept ones lies what lay there
        pool[pages[t // page], :, :, t % page] = rows
    return pool


def exact(case, seed):
    if case["op"] == "accept":
        return None  # whole numbers
    s = prepare(case, seed)
    return {"score": _exact_score, "commit": _exact_commit}.get(case["op"], _exact_attention)(case, s)
