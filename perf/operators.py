"""Operators of a 4-bit paged KV cache and of page management, as cases to be measured.

The 4-bit cache holds K and V rows in NVFP4: per 16 consecutive elements of a row one scale in e4m3,
per element one e2m1 code.  A (page, K|V, head) block is page_size * d / 2 bytes of codes (token after
token, the even element of a pair in the low nibble), then page_size * d / 16 scale bytes.  A stored
value stands for code * scale * (the cache's k_scale or v_scale).

Five operators:
  append   quantise new tokens' K and V rows into their pages, and read them back
  verify   attention of a request's last n_cand tokens over its whole 4-bit cache (n_cand = 1: plain
           decoding), with or without the tokens' criticality
  draft    single-query attention over a list of selected tokens of the 4-bit cache
  branch   drop the last step's branches of every request, fork each request into new ones, and make
           room for everybody's next tokens (copying the last page where it is shared)
  compact  gather the listed tokens of each request into the pages of a smaller cache
"""

import math

import torch

own = False

DEV = "cuda"
GROUP = 16  # elements that share a scale


# ------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------


def listed():
    return [
        # One decoding step's candidates (k = 4 drafts and a bonus token) of a batch of 32: latency counts.
        dict(name="append candidates", op="append", batch=32, n=5, lo=5, hi=5, h_kv=8, d=128, page=16, dtype="bf16", ksc=1.0, vsc=1.0),
        # Prompts of different lengths entering the cache together.
        dict(name="append prompts", op="append", batch=8, n=8192, lo=2048, hi=8192, h_kv=8, d=128, page=16, dtype="bf16", ksc=1.0, vsc=0.5),
        # One short request: the smallest attention call.
        dict(name="verify one short", op="verify", batch=1, lo=700, hi=900, h_q=8, h_kv=2, d=64, n_cand=5, page=16, q="bf16", out="f32", scores=True, ksc=1.0, vsc=1.0),
        # Plain decoding of a batch from the 4-bit cache.
        dict(name="verify decode", op="verify", batch=32, lo=2048, hi=8192, h_q=32, h_kv=8, d=128, n_cand=1, page=16, q="bf16", out="bf16", scores=False, ksc=1.0, vsc=1.0),
        # The verify of a speculative round on the same batch, with the criticality that selects the drafts' tokens.
        dict(name="verify round", op="verify", batch=32, lo=2048, hi=8192, h_q=32, h_kv=8, d=128, n_cand=5, page=16, q="bf16", out="f32", scores=True, ksc=1.0, vsc=1.0),
        # Long contexts, few requests: work split along the tokens.
        dict(name="verify long", op="verify", batch=8, lo=131072, hi=131072, h_q=32, h_kv=8, d=128, n_cand=5, page=16, q="bf16", out="bf16", scores=False, ksc=1.0, vsc=1.0),
        # A draft of one short request.
        dict(name="draft one short", op="draft", batch=1, lo=700, hi=900, h_q=8, h_kv=2, d=64, k=41, page=16, q="bf16", out="f32", ksc=1.0, vsc=1.0),
        # A draft of the round: 5 % of 8192 tokens at most.
        dict(name="draft round", op="draft", batch=32, lo=2048, hi=8192, h_q=32, h_kv=8, d=128, k=410, page=16, q="bf16", out="bf16", ksc=1.0, vsc=1.0),
        # Eight requests, three new branches each, next to a 16-bit cache.
        dict(name="branch 8 to 32", op="branch", parents=8, children=3, lo=2048, hi=8192, n=5, h_kv=8, d=128, page=16, dtype="bf16"),
        # Sampling of many answers for each prompt from a large 4-bit pool.
        dict(name="branch 64 to 512", op="branch", parents=64, children=7, lo=4096, hi=16384, n=5, h_kv=8, d=128, page=16, dtype="nvfp4"),
        # Keeping the critical 5 % of a batch's 16-bit cache.
        dict(name="compact round", op="compact", batch=32, lo=2048, hi=8192, k=410, h_kv=8, d=128, page=16, dtype="bf16"),
        # Keeping a tenth of long 4-bit contexts.
        dict(name="compact long", op="compact", batch=8, lo=131072, hi=131072, k=13107, h_kv=8, d=128, page=16, dtype="nvfp4"),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "verify", "verify", "verify", "draft", "draft", "branch", "compact"])
    h_kv = rng.choice([1, 2, 3, 8])
    d = rng.choice([64, 128, 128])
    page = rng.choice([8, 16, 16, 32, 64])
    sc = dict(ksc=rng.choice([0.5, 1.0, 2.0]), vsc=rng.choice([0.25, 1.0]))
    batch = _logint(rng, 1, 40)
    if op == "append":
        n = _logint(rng, 1, 4096)
        return dict(op=op, batch=batch, n=n, lo=max(1, n // 4), hi=n, h_kv=h_kv, d=d, page=page, dtype=rng.choice(["bf16", "bf16", "f32"]), **sc)
    top = _logint(rng, 40, 200000 // batch)
    lo = max(1, int(top * rng.choice([0.25, 0.5, 1.0])))
    if op in ("verify", "draft"):
        G = rng.choice([1, 2, 4, 4, 5, 7, 8, 16])
        q = rng.choice(["bf16", "bf16", "bf16", "f32"])
        out = "f32" if q == "f32" else rng.choice(["bf16", "f32"])
        if op == "draft":
            return dict(op=op, batch=batch, lo=lo, hi=top, h_q=G * h_kv, h_kv=h_kv, d=d, k=_logint(rng, 1, max(2, min(top, 4096) // 3)), page=page, q=q, out=out, **sc)
        nc = min(rng.choice([1, 1, 2, 4, 5, 7, 8]), 64 // G)
        return dict(op=op, batch=batch, lo=max(lo, nc), hi=max(top, nc), h_q=G * h_kv, h_kv=h_kv, d=d, n_cand=nc, page=page, q=q, out=out, scores=rng.random() < 0.5, **sc)
    dtype = rng.choice(["bf16", "f32", "nvfp4", "nvfp4"])
    if op == "branch":
        parents = _logint(rng, 1, 24)
        top = min(top, 8192)
        return dict(op=op, parents=parents, children=rng.randint(1, 6), lo=min(lo, top), hi=top, n=_logint(rng, 1, 300), h_kv=h_kv, d=d, page=page, dtype=dtype)
    return dict(op=op, batch=batch, lo=lo, hi=top, k=_logint(rng, 1, max(2, top // 2)), h_kv=h_kv, d=d, page=page, dtype=dtype)


# ------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------


def _lens(case, seed):
    g = torch.Generator().manual_seed(int(seed) * 7919 + 13)
    rows = case.get("parents", case.get("batch"))
    lens = torch.randint(case["lo"], case["hi"] + 1, (rows,), generator=g)
    return [int(x) for x in lens]


def _row_bytes(dtype, d):
    return {"bf16": 2 * d, "f32": 4 * d, "nvfp4": d // 2 + d // GROUP}[dtype]


def _codes(x):
    """(codes in 0..15, e4m3 scale bytes) of x [..., d]: s = e4m3(amax / 6) per 16 elements, code =
    e2m1(x / s), both to nearest with ties to the even code; a group whose scale is 0 holds zeros."""
    y = x.float().unflatten(-1, (-1, GROUP))
    s = (y.abs().amax(-1) / torch.full((1,), 6.0, device=x.device)).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.float().unsqueeze(-1)
    a = torch.where(sf > 0, y.abs() / torch.where(sf > 0, sf, 1.0), 0.0)
    c = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    c = c.to(torch.uint8) | ((y < 0).to(torch.uint8) << 3)
    return c.flatten(-2), s.view(torch.uint8)


def _pack(c):
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _halves(pool, page, d):
    """The code and scale parts of a pool, as views [pages, 2, heads, page_size, d / 2 | d / 16]."""
    flat = pool.flatten(3)
    return (flat[..., :page * d // 2].unflatten(-1, (page, d // 2)), flat[..., page * d // 2:].unflatten(-1, (page, d // GROUP)))


def _table(gen, lens, page, most, cap, spare):
    """A shuffled page table for rows of `lens` tokens (at most `most`), `cap` entries a row, and the
    pool's size, which holds rows of `most` tokens."""
    need = [-(-x // page) for x in lens]
    total = len(lens) * -(-most // page) + spare
    perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(lens), cap), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, total


def _cache4(case, lens, gen):
    """A filled 4-bit cache; the slots behind each request hold arbitrary bytes.  Keys lean on a
    direction of their head at some positions, as attention that concentrates does."""
    page, d, h = case["page"], case["d"], case["h_kv"]
    table, total = _table(gen, lens, page, case["hi"], -(-case["hi"] // page) + 1, 3)
    pool = torch.randint(0, 256, (total, 2, h, page, d // 2 + d // GROUP), dtype=torch.uint8, generator=gen, device=DEV)
    code, scale = _halves(pool, page, d)
    u = torch.randn((len(lens), h, d), generator=gen, device=DEV)
    u = u / u.norm(dim=-1, keepdim=True)
    step = 16384
    for b, n in enumerate(lens):
        for t0 in range(0, n, step):
            m = min(step, n - t0)
            x = torch.randn((2, h, m, d), generator=gen, device=DEV)
            x[0] += 4.0 * (torch.rand((h, m, 1), generator=gen, device=DEV) < 0.02) * u[b][:, None]
            c, s = _codes(x.bfloat16())
            p = table[b, t0 // page:-(-(t0 + m) // page)].long()
            full = m // page * page
            if full:
                code[p[:full // page]] = _pack(c)[:, :, :full].unflatten(2, (-1, page)).permute(2, 0, 1, 3, 4)
                scale[p[:full // page]] = s[:, :, :full].unflatten(2, (-1, page)).permute(2, 0, 1, 3, 4)
            if full < m:
                code[p[-1], :, :, :m - full] = _pack(c)[:, :, full:]
                scale[p[-1], :, :, :m - full] = s[:, :, full:]
    return pool, table, u


def _lists(case, lens, gen, rows):
    """Ascending lists of distinct tokens for every (request, head): [rows, h_kv, k] and counts."""
    h, k = case["h_kv"], case["k"]
    idx = torch.full((rows, h, k), -1, dtype=torch.int32, device=DEV)
    cnt = torch.empty((rows, h), dtype=torch.int32, device=DEV)
    frac = k / case["hi"]
    for b, n in enumerate(lens):
        m = max(1, min(k, int(math.ceil(frac * n))))
        pick = torch.rand((h, n), generator=gen, device=DEV).topk(m, dim=-1).indices
        idx[b, :, :m] = pick.sort(dim=-1).values.to(torch.int32)
        cnt[b] = m
    return idx, cnt


def _any_pool(gen, pages, case):
    """A pool of arbitrary bytes: what the page operators move they do not read."""
    d, page, h, dtype = case["d"], case["page"], case["h_kv"], case["dtype"]
    raw = torch.randint(-2**31, 2**31 - 1, (pages, 2, h, page, _row_bytes(dtype, d) // 4), dtype=torch.int32, generator=gen, device=DEV)
    return raw.view({"bf16": torch.bfloat16, "f32": torch.float32, "nvfp4": torch.uint8}[dtype])


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    lens = _lens(case, seed)
    i32 = dict(dtype=torch.int32, device=DEV)
    s = dict(case=dict(case), lens=torch.tensor(lens, **i32), max_len=case["hi"])
    op, page, h, d = case["op"], case["page"], case["h_kv"], case["d"]
    if op == "append":
        # The requests already hold some tokens; `lens` are the counts of new ones.
        before = torch.randint(0, 200, (case["batch"],), generator=gen, device=DEV).tolist()
        end = [a + n for a, n in zip(before, lens)]
        table, total = _table(gen, end, page, 200 + case["n"], -(-(200 + case["n"]) // page), 3)
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        shape = (case["batch"], case["n"], h, d)
        mk = lambda sd: (torch.randn(shape, generator=gen, device=DEV) * sd).to(dt)  # noqa: E731
        s.update(k=mk(1.5), v=mk(0.7), table=table, counts=s["lens"], max_len=200 + case["n"])
        s["lens"] = torch.tensor(before, **i32)
        s["pool"] = torch.zeros((total, 2, h, page, d // 2 + d // GROUP), dtype=torch.uint8, device=DEV)
        s.update(k_out=torch.empty(shape, dtype=torch.bfloat16, device=DEV), v_out=torch.empty(shape, dtype=torch.bfloat16, device=DEV))
    elif op in ("verify", "draft"):
        s["pool"], s["table"], u = _cache4(case, lens, gen)
        B, nc, G = case["batch"], case.get("n_cand", 1), case["h_q"] // h
        q = torch.randn((B, nc, h, G, d), generator=gen, device=DEV) + 2.0 * u[:, None, :, None]
        q = q.flatten(2, 3).to(torch.bfloat16 if case["q"] == "bf16" else torch.float32)
        dt = torch.bfloat16 if case["out"] == "bf16" else torch.float32
        s["out"] = torch.empty_like(q, dtype=dt)
        s["lse"] = torch.empty(q.shape[:-1], dtype=torch.float32, device=DEV)
        if op == "draft":
            s["idx"], s["cnt"] = _lists(case, lens, gen, B)
            q, s["out"], s["lse"] = q[:, 0].contiguous(), s["out"][:, 0].contiguous(), s["lse"][:, 0].contiguous()
        elif case["scores"]:
            s["scores"] = torch.zeros((B, h, case["hi"]), dtype=torch.float32, device=DEV)
        s["q"] = q
    elif op == "branch":
        P, C, n = case["parents"], case["children"], case["n"]
        cap = -(-(case["hi"] + n) // page)
        rows = P * (1 + C)
        spare = rows * (-(-n // page) + 1) + 8
        table, total = _table(gen, lens, page, case["hi"], cap, spare)
        s["table"] = torch.full((rows, cap), -1, **i32)
        s["table"][:P] = table
        s["refs"] = torch.zeros((total,), **i32)
        s["refs"][table[table >= 0].long()] = 1
        s["pool"] = _any_pool(gen, total, case)
        s["lens"] = torch.cat([s["lens"], torch.zeros((P * C,), **i32)])
        s["max_len"] = cap * page
        s["keep"] = torch.cat([s["lens"][:P], torch.zeros((P * C,), **i32)])
        s["src"] = torch.arange(P, **i32).repeat_interleave(C)
        s["dst"] = torch.arange(P, rows, **i32)
        s["counts"] = torch.full((rows,), n, **i32)
    else:
        table, total = _table(gen, lens, page, case["hi"], -(-case["hi"] // page), 3)
        s.update(table=table, pool=_any_pool(gen, total, case))
        s["idx"], s["cnt"] = _lists(case, lens, gen, case["batch"])
        kept = s["cnt"][:, 0].tolist()
        s["dst_table"], total = _table(gen, kept, page, case["k"], -(-case["k"] // page), 3)
        s["dst_pool"] = _any_pool(gen, total, case)
        s["dst_lens"] = torch.zeros((case["batch"],), **i32)
        s["rows"] = torch.arange(case["batch"], **i32)
        s["max_kept"] = case["k"]
    return s


# ------------------------------------------------------------------------------------------------
# The plain forms
# ------------------------------------------------------------------------------------------------


def _values(code, scale, mult):
    """What codes [..., d / 2] and scales [..., d / 16] stand for, in 32 bits (exact)."""
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=code.device)
    c = torch.stack([code & 15, code >> 4], dim=-1).flatten(-2)
    v = lut[c.int()].unflatten(-1, (-1, GROUP))
    return (v * (scale.contiguous().view(torch.float8_e4m3fn).float() * mult).unsqueeze(-1)).flatten(-2)


def _plain_append(s):
    case = s["case"]
    page, d, n = case["page"], case["d"], case["n"]
    j = torch.arange(n, device=DEV)
    live = j[None] < s["counts"][:, None]
    t = s["lens"][:, None] + j[None]
    p = s["table"].long().gather(1, torch.div(t, page, rounding_mode="floor").long())
    code, scale = _halves(s["pool"], page, d)
    outs = []
    for which, x, mult in ((0, s["k"], case["ksc"]), (1, s["v"], case["vsc"])):
        c, e = _codes(x.float() / mult)
        c = _pack(c)
        at = (p[live], (t % page)[live].long())
        code[at[0], which, :, at[1]] = c[live]
        scale[at[0], which, :, at[1]] = e[live]
        outs.append(torch.where(live[:, :, None, None], _values(c, e, mult), 0.0).bfloat16())
    return outs


def _attend(s, q, K, V, mask):
    """Softmax attention of q [B, h, r, d] over K, V [B, h, t, d]; mask [B, h | 1, r | 1, t]."""
    x = q.float() @ K.transpose(-1, -2) * (1.0 / math.sqrt(q.shape[-1]))
    x = torch.where(mask, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.where(mask, torch.exp(x - torch.where(m == -math.inf, 0.0, m)), 0.0)
    z = p.sum(-1, keepdim=True)
    p = p / torch.where(z > 0, z, 1.0)
    lse = torch.where(z > 0, m + torch.log(z), -math.inf)
    return p @ V, lse.squeeze(-1), p


def _plain_verify(s):
    case = s["case"]
    page, d, h, nc = case["page"], case["d"], case["h_kv"], case["n_cand"]
    n = s["max_len"]
    code, scale = _halves(s["pool"], page, d)
    pages = s["table"][:, :-(-n // page)].clamp(min=0).long()
    t = torch.arange(n, device=DEV)
    inside = t[None] < s["lens"][:, None]

    def rows(which, mult):
        c = code[pages, which].transpose(1, 2).flatten(2, 3)[:, :, :n]
        e = scale[pages, which].transpose(1, 2).flatten(2, 3)[:, :, :n]
        return torch.where(inside[:, None, :, None], _values(c, e, mult), 0.0)

    B, G = case["batch"], case["h_q"] // h
    q = s["q"].view(B, nc, h, G, d).transpose(1, 2).flatten(2, 3)
    seen = t[None, None] <= (s["lens"][:, None] - nc + torch.arange(nc, device=DEV)[None])[:, :, None]
    mask = (seen & inside[:, None]).repeat_interleave(G, dim=1)[:, None]
    o, lse, p = _attend(s, q, rows(0, case["ksc"]), rows(1, case["vsc"]), mask)
    res = {"out": o.view(B, h, nc, G, d).transpose(1, 2).flatten(2, 3).to(s["out"].dtype),
           "lse": lse.view(B, h, nc, G).transpose(1, 2).flatten(2, 3)}
    if case["scores"]:
        res["scores"] = p.sum(2)
    return res


def _plain_draft(s):
    case = s["case"]
    page, d, h = case["page"], case["d"], case["h_kv"]
    B, G, k = case["batch"], case["h_q"] // h, case["k"]
    live = torch.arange(k, device=DEV)[None, None] < s["cnt"][:, :, None]
    t = s["idx"].clamp(min=0).long()
    p = s["table"].long()[:, None].expand(B, h, -1).gather(2, t // page)
    head = torch.arange(h, device=DEV)[None, :, None]
    code, scale = _halves(s["pool"], page, d)
    K = _values(code[p, 0, head, t % page], scale[p, 0, head, t % page], case["ksc"])
    V = _values(code[p, 1, head, t % page], scale[p, 1, head, t % page], case["vsc"])
    o, lse, _ = _attend(s, s["q"].view(B, h, G, d), K, torch.where(live[..., None], V, 0.0), live[:, :, None])
    return {"out": o.reshape(B, h * G, d).to(s["out"].dtype), "lse": lse.reshape(B, h * G)}


def _ceil_pages(n, page):
    return torch.div(n + page - 1, page, rounding_mode="floor")


def _plain_branch(s):
    case = s["case"]
    page = case["page"]
    table, lens, refs, pool = s["table"], s["lens"], s["refs"], s["pool"]
    rows, cap = table.shape
    j = torch.arange(cap, device=DEV)[None]
    # Drop what lies behind `keep`.
    drop = (j >= _ceil_pages(s["keep"], page)[:, None]) & (table >= 0)
    refs.scatter_add_(0, torch.where(drop, table, 0).flatten().long(), -drop.flatten().int())
    table.masked_fill_(drop, -1)
    lens.copy_(torch.minimum(lens, s["keep"]))
    # Fork: the new rows share the pages of theirs.
    src, dst = s["src"].long(), s["dst"].long()
    new = torch.where(j < _ceil_pages(lens[src], page)[:, None], table[src], -1)
    table[dst] = new
    lens[dst] = lens[src]
    refs.scatter_add_(0, new.clamp(min=0).flatten().long(), (new >= 0).flatten().int())
    # Room for the next tokens: missing pages, and a page of its own where one is shared.  The lowest
    # of a page's holders keeps it when all of them ask.
    need = (j >= torch.div(lens, page, rounding_mode="floor")[:, None]) & (j < _ceil_pages(lens + s["counts"], page)[:, None])
    held = need & (table >= 0)
    at = table.clamp(min=0).flatten().long()
    asked = torch.zeros_like(refs).scatter_add_(0, at, held.flatten().int())
    row = torch.arange(rows, dtype=torch.int32, device=DEV)[:, None].expand(rows, cap)
    low = torch.full_like(refs, rows).scatter_reduce_(0, at, torch.where(held, row, rows).flatten(), "amin")
    keeps = held & ((refs[at] == 1) | ((asked[at] == refs[at]) & (low[at] == row.flatten()))).view(rows, cap)
    takes = need & ~keeps
    rank = takes.flatten().long().cumsum(0) - 1
    free = refs == 0
    place = torch.where(free, free.long().cumsum(0) - 1, refs.numel())
    order = torch.zeros(refs.numel() + 1, dtype=torch.int64, device=DEV).scatter_(0, place, torch.arange(refs.numel(), device=DEV))
    fresh = order[rank.clamp(min=0)].view(rows, cap)
    leaves = takes & (table >= 0)
    refs.scatter_add_(0, at, -leaves.flatten().int())
    old = table.clone()
    table.copy_(torch.where(takes, fresh.int(), table))
    refs.scatter_add_(0, table.clamp(min=0).flatten().long(), takes.flatten().int())
    # The live slots of a page that was shared move along.
    b = torch.arange(rows, device=DEV)
    jl = torch.div(lens, page, rounding_mode="floor").long()
    jl_in = jl.clamp(max=cap - 1)
    moves = leaves[b, jl_in] & (lens % page > 0) & (jl < cap)
    frm, to, slots = old[b, jl_in].long()[moves], table[b, jl_in].long()[moves], (lens % page)[moves]
    live = (torch.arange(page, device=DEV)[None] < slots[:, None])[:, None, None, :, None]
    if case["dtype"] == "nvfp4":
        for part in _halves(pool, page, case["d"]):
            part[to] = torch.where(live, part[frm], part[to])
    else:
        raw = pool.view(torch.int32)
        raw[to] = torch.where(live, raw[frm], raw[to])
    return _branch_out(s)


def _branch_out(s):
    return {"table": s["table"], "lens": s["lens"], "refs": s["refs"], "pool": s["pool"].view(torch.int16)}


def _plain_compact(s):
    case = s["case"]
    page, h, k = case["page"], case["h_kv"], case["k"]
    B = case["batch"]
    j = torch.arange(k, device=DEV)
    live = j[None, None] < s["cnt"][:, :, None]
    t = s["idx"].clamp(min=0).long()
    p = s["table"].long()[:, None].expand(B, h, -1).gather(2, t // page)[live]
    to = s["dst_table"].long()[:, (j // page).clamp(max=s["dst_table"].shape[1] - 1)][:, None].expand(B, h, k)[live]
    head = torch.arange(h, device=DEV)[None, :, None].expand(B, h, k)[live]
    slot, slot_to = (t % page)[live], (j % page)[None, None].expand(B, h, k)[live]
    if case["dtype"] == "nvfp4":
        pairs = zip(_halves(s["dst_pool"], page, case["d"]), _halves(s["pool"], page, case["d"]))
    else:
        pairs = [(s["dst_pool"].view(torch.int32), s["pool"].view(torch.int32))]
    for a, b in pairs:
        a[to, :, head, slot_to] = b[p, :, head, slot]
    s["dst_lens"].copy_(s["cnt"][:, 0])
    return {"pool": s["dst_pool"].view(torch.int16), "lens": s["dst_lens"]}


# ------------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------------


def _cache(s, pool="pool", table="table", lens="lens", max_len="max_len"):
    """The framework's handle of a cache, made once and kept beside its tensors."""
    from sparse_self_speculative_verify_gb300 import KV4Cache, KVCache
    c = s["case"]
    if s[pool].dtype == torch.uint8:
        return KV4Cache(s[pool], s[table], s[lens], s[max_len], k_scale=c.get("ksc", 1.0), v_scale=c.get("vsc", 1.0))
    return KVCache(s[pool], s[table], s[lens], s[max_len])


def run(state):
    s = state
    case = s["case"]
    op = case["op"]
    if not own:
        return {"append": _plain_append, "verify": _plain_verify, "draft": _plain_draft, "branch": _plain_branch,
                "compact": _plain_compact}[op](s)
    import sparse_self_speculative_verify_gb300 as F
    if "cache" not in s:
        s["cache"] = _cache(s)
        if op == "branch":
            s["pages"] = F.PagePool(s["refs"])
        if op == "compact":
            s["dst_cache"] = _cache(s, "dst_pool", "dst_table", "dst_lens", "max_kept")
    kv = s["cache"]
    if op == "append":
        F.ssd_kv4_append(kv, s["k"], s["v"], counts=s["counts"])
        return list(F.ssd_kv4_read(kv, s["lens"], case["n"], counts=s["counts"], k=s["k_out"], v=s["v_out"]))
    scale = 1.0 / math.sqrt(case["d"])
    if op == "verify":
        r = F.ssd_kv4_verify_attn(kv, s["q"], case["n_cand"], scale, out=s["out"], lse=s["lse"], scores=s.get("scores"),
                                  want_scores=case["scores"])
        return {k: v for k, v in r.items() if v is not None}
    if op == "draft":
        return F.ssd_kv4_draft_attn(kv, s["q"], s["idx"], s["cnt"], scale, out=s["out"], lse=s["lse"])
    if op == "branch":
        F.ssd_kv_release(kv, s["pages"], s["keep"])
        F.ssd_kv_fork(kv, s["pages"], s["src"], s["dst"])
        F.ssd_kv_reserve(kv, s["pages"], s["counts"])
        return _branch_out(s)
    F.ssd_kv_compact(kv, s["dst_cache"], s["rows"], s["rows"], s["idx"], s["cnt"])
    return {"pool": s["dst_pool"].view(torch.int16), "lens": s["dst_lens"]}


def work(case):
    """Bytes and operations that a pass cannot do without, with every length at the middle of its range."""
    op, h, d = case["op"], case["h_kv"], case["d"]
    mid = (case["lo"] + case["hi"]) / 2
    q4 = 2 * h * (d // 2 + d // GROUP)  # K and V bytes of a token in 4 bits
    if op == "append":
        n = case["batch"] * mid * 2 * h * d
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * (e + 0.5625) + case["batch"] * case["n"] * 2 * h * d * 2, "flops": 4 * n}
    size = {"bf16": 2, "f32": 4}
    if op in ("verify", "draft"):
        rows = case["batch"] * case.get("n_cand", 1) * case["h_q"]
        tok = case["batch"] * (mid if op == "verify" else max(1.0, case["k"] * mid / case["hi"]))
        b = tok * q4 + rows * (d * (size[case["q"]] + size[case["out"]]) + 4)
        b += 4 * h * tok if op == "draft" or case["scores"] else 0
        return {"bytes": b, "flops": 4.0 * tok * case["h_q"] * case.get("n_cand", 1) * d}
    row = 2 * h * _row_bytes(case["dtype"], d)
    if op == "branch":
        P, C = case["parents"], case["children"]
        pages = mid / case["page"]
        # every fork copies its row of the table; every new branch moves half a page at the mean
        return {"bytes": P * C * (pages * 4 * 3 + case["page"] * row) + P * pages * 8, "flops": 0}
    kept = case["batch"] * max(1.0, case["k"] * mid / case["hi"])
    return {"bytes": kept * (2 * row + 4 * h), "flops": 0}


# ------------------------------------------------------------------------------------------------
# The definition in 64 bits
# ------------------------------------------------------------------------------------------------

_MAGNITUDE = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _e4m3(byte):
    """The values of e4m3 bytes, from the definition: sign, 4 bits of exponent (bias 7), 3 of fraction."""
    size = [math.ldexp(b & 7, -9) if b < 8 else math.ldexp(8 + (b & 7), (b >> 3) - 10) for b in range(127)] + [math.nan]
    return torch.tensor(size + [-x for x in size], dtype=torch.float64, device=byte.device)[byte.to(torch.int64)]


def _all_e4m3():
    return _e4m3(torch.arange(127, device=DEV))  # 0 .. 448, ascending with the byte


def _nearest_even(x, grid):
    """Index of the value of an ascending grid nearest to x >= 0, ties to the even index."""
    hi = torch.searchsorted(grid, x).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - x, x - grid[lo]
    pick_hi = (up < down) | ((up == down) & (hi % 2 == 0)) | (x >= grid[-1])
    return torch.where(pick_hi, hi, lo)


def _exact_append(case, s):
    out = []
    for x, mult in ((s["k"], case["ksc"]), (s["v"], case["vsc"])):
        mag, scales = torch.tensor(_MAGNITUDE, dtype=torch.float64, device=DEV), _all_e4m3()
        res = torch.zeros(x.shape, dtype=torch.float64, device=DEV)
        for b, n in enumerate(s["counts"].tolist()):
            y = x[b, :n].double().div(mult).reshape(-1, GROUP)
            sc = scales[_nearest_even(y.abs().max(dim=1).values / 6, scales)][:, None]
            c = _nearest_even(torch.where(sc > 0, y.abs() / sc.clamp(min=1e-300), torch.zeros_like(y)), mag)
            res[b, :n] = (mag[c] * sc * y.sign() * mult).reshape(res[b, :n].shape)
        out.append(res)
    return out


def _token_rows(case, s, b, head, which, tokens):
    """Rows of listed tokens of one head in 64 bits, byte by byte from the pool."""
    page, d = case["page"], case["d"]
    block = s["pool"][s["table"][b].long()[tokens // page], which, head].flatten(1)
    slot = (tokens % page)[:, None]
    codes = block.gather(1, slot * (d // 2) + torch.arange(d // 2, device=DEV)).to(torch.int64)
    sc = _e4m3(block.gather(1, page * d // 2 + slot * (d // GROUP) + torch.arange(d // GROUP, device=DEV)))
    lut = torch.tensor(_MAGNITUDE + [-m for m in _MAGNITUDE], dtype=torch.float64, device=DEV)
    row = torch.empty((tokens.numel(), d), dtype=torch.float64, device=DEV)
    row[:, 0::2], row[:, 1::2] = lut[codes % 16], lut[codes // 16]
    return row * sc.repeat_interleave(GROUP, dim=1) * (case["vsc"] if which else case["ksc"])


def _exact_attention(case, s):
    verify = case["op"] == "verify"
    h, G = case["h_kv"], case["h_q"] // case["h_kv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    crit = torch.zeros(s["scores"].shape, dtype=torch.float64, device=DEV) if "scores" in s else None
    for b, n in enumerate(s["lens"].tolist()):
        for g in range(h):
            tok = torch.arange(n, device=DEV) if verify else s["idx"][b, g, :int(s["cnt"][b, g])].long()
            K, V = _token_rows(case, s, b, g, 0, tok), _token_rows(case, s, b, g, 1, tok)
            for i in range(case["n_cand"] if verify else 1):
                m = n - case["n_cand"] + i + 1 if verify else tok.numel()
                at = (b, i) if verify else (b,)
                hs = slice(g * G, (g + 1) * G)
                x = s["q"][at][hs].double() @ K[:m].T / math.sqrt(case["d"])
                lse[at][hs] = torch.logsumexp(x, dim=1)
                w = torch.exp(x - lse[at][hs, None])
                out[at][hs] = w @ V[:m]
                if crit is not None:
                    crit[b, g, :m] += w.sum(0)
    return {"out": out, "lse": lse} | ({"scores": crit} if crit is not None else {})


def exact(case, seed):
    if case["op"] in ("branch", "compact"):
        return None  # copies and counts: nothing is computed in floating point
    s = prepare(case, seed)
    return _exact_append(case, s) if case["op"] == "append" else _exact_attention(case, s)
