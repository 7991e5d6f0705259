"""Cases of the verify forward's attention operators: the norms and position
rotation of query and key heads, the append of a round's keys and values to a
paged cache, and the attention of a verify block over that cache with prefixes
that requests share.

``own`` selects what ``run`` does: the plain form in elementary torch
operations, or the calls a user makes of ``logprob_epilogue_gb300.AttnPlan``.

A verify round of a batch: group g owns the rows group_indptr[g] ..
group_indptr[g + 1] - 1 (the last committed token and its drafts), ``lens[g]``
tokens of its own are committed in the paged cache, row j of the group is token
lens[g] + j, and a run of groups may share a prefix held in pages of its own.
"""
import math

import numpy as np
import torch

own = False

MAX_GROUP_ROWS = 32  # rows of one group in the attention cases
TABLE_POSITIONS = 1 << 17  # positions the rotation table covers
THETA = 1.0e6
EPS = 1.0e-6


def listed():
    """Twelve cases; the head counts are a grouped-query layout of 32 query and 8 key-value heads
    unless a case says otherwise."""
    rope = {"op": "norm_rope", "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "head_dim": 128, "rot": 128,
            "interleaved": False, "norm": True, "fused": True}
    app = {"op": "append", "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "head_dim": 128, "page": 64, "rot": 128,
           "interleaved": False, "norm": True, "fused": True, "idle": 0}
    att = {"op": "attend", "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "head_dim": 128, "page": 64, "idle": 0,
           "prefixes": 0, "prefix": 0, "tree": False}
    return [
        # a verify step of one request outside a cache: latency alone
        dict(rope, name="norm_rope_round", rows=4),
        # a training-sized or prompt-sized block with small heads, half of each rotated, pairs interleaved
        dict(rope, name="norm_rope_block", rows=8191, dtype="f16", q_heads=24, kv_heads=4, head_dim=64, rot=32,
             interleaved=True, fused=False),
        # one request decoding one token: the smallest call
        dict(app, name="append_token", groups=1, rows_lo=1, rows_hi=1, len_lo=1000, len_hi=1000, page=16),
        # the verify round of 128 requests with 3 drafts each, three slots of the batch idle
        dict(app, name="append_verify", groups=128, rows_lo=4, rows_hi=4, len_lo=0, len_hi=8192, idle=3),
        # five prompts entering the cache at once, of ragged lengths
        dict(app, name="append_prompts", groups=5, rows_lo=1501, rows_hi=5003, len_lo=0, len_hi=777, norm=False),
        # one request decoding one token at a moderate context: latency, and one row's work over the whole GPU
        dict(att, name="attend_token", groups=1, rows_lo=1, rows_hi=1, len_lo=4095, len_hi=4095, page=16),
        # the verify round of 128 requests with 3 drafts each, ragged contexts, three slots idle: bandwidth
        dict(att, name="attend_verify", groups=128, rows_lo=4, rows_hi=4, len_lo=0, len_hi=8192, idle=3),
        # four requests at very long contexts with small heads
        dict(att, name="attend_long", groups=4, rows_lo=1, rows_hi=4, len_lo=100_001, len_hi=131_071, head_dim=64,
             q_heads=16, kv_heads=2, dtype="f16", page=128),
        # trees of drafts, up to 16 rows a group, small pages
        dict(att, name="attend_tree", groups=16, rows_lo=7, rows_hi=16, len_lo=1, len_hi=4001, page=32, tree=True),
        # 64 requests decoding one token each behind one shared prefix (a long instruction text)
        dict(att, name="attend_prefix", groups=64, rows_lo=1, rows_hi=1, len_lo=0, len_hi=512, prefixes=1,
             prefix=8191),
        # three prefixes of ragged length, drafts, multi-query heads
        dict(att, name="attend_prefixes", groups=47, rows_lo=2, rows_hi=6, len_lo=5, len_hi=1500, prefixes=3,
             prefix=12_345, q_heads=40, kv_heads=4),
        # 256 requests with 7 drafts each behind one long shared prefix: arithmetic
        dict(att, name="attend_prefix_large", groups=256, rows_lo=8, rows_hi=8, len_lo=0, len_hi=1024, prefixes=1,
             prefix=32_768),
    ]


def draw(rng):
    """One more case of the same ranges."""
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["norm_rope", "append", "attend", "attend", "attend"])
    dim = rng.choice([64, 128])
    kv = rng.choice([1, 2, 4, 8])
    share = rng.choice([1, 2, 3, 4, 5, 8, 12])  # query heads of one key-value head
    while kv * share > 48:
        share = rng.choice([1, 2, 3, 4])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16"]), "q_heads": kv * share, "kv_heads": kv, "head_dim": dim}
    if op != "attend":
        c.update(rot=rng.choice([0, 16, dim // 2, dim, dim]), interleaved=rng.random() < 0.3, norm=rng.random() < 0.7,
                 fused=rng.random() < 0.5)
        if op == "norm_rope":
            c.update(rows=log_int(1, 16_384))
            return c
        c.update(page=rng.choice([8, 16, 32, 64, 128, 256]), groups=log_int(1, 256), len_lo=0, len_hi=log_int(1, 8192))
        hi = log_int(1, max(1, 20_000 // c["groups"]))
        c.update(rows_lo=max(1, hi // 2), rows_hi=hi, idle=min(c["groups"] - 1, rng.choice([0, 0, 1, 4])))
        return c
    groups = log_int(1, 256)
    rows_hi = rng.choice([1, 1, 2, 4, 5, 8, 16])
    len_hi = log_int(1, min(131_000, 1_000_000 // groups))
    prefixes = rng.choice([0, 0, 1, 1, 2, 4])
    prefix = log_int(1, 32_768) if prefixes else 0
    while groups * rows_hi * c["q_heads"] * prefix > 1_000_000_000:  # at most half the arithmetic of the largest listed case
        prefix = max(1, prefix // 2)
    c.update(page=rng.choice([8, 16, 32, 64, 128, 256]), groups=groups, rows_lo=rng.randint(1, rows_hi), rows_hi=rows_hi,
             len_lo=rng.randint(0, len_hi), len_hi=len_hi, idle=min(groups - 1, rng.choice([0, 0, 1, 5])),
             prefixes=min(prefixes, groups), prefix=prefix, tree=rows_hi > 1 and rng.random() < 0.4)
    return c


# ---- the shape of a case's batch, from the case alone


def _shape(case):
    """(rows of each group, committed tokens of each group, -1 for an idle slot; tokens and first group of each prefix)."""
    r = np.random.RandomState((case["groups"] * 7919 + case["len_hi"] * 31 + case["rows_hi"]) % (1 << 31))
    n = r.randint(case["rows_lo"], case["rows_hi"] + 1, case["groups"])
    lens = r.randint(case["len_lo"], case["len_hi"] + 1, case["groups"])
    if case["groups"] > 1:
        lens[r.randint(case["groups"])] = case["len_hi"]
    if case["idle"]:
        lens[r.choice(case["groups"], case["idle"], replace=False)] = -1
    count = case.get("prefixes", 0)
    shared = np.array([max(1, case["prefix"] * (count - i) // count) for i in range(count)], np.int64)
    first = np.array([case["groups"] * i // count for i in range(count + 1)], np.int64) if count else np.zeros(1, np.int64)
    return n.astype(np.int64), lens.astype(np.int64), shared, first


def _pages_of(tokens, page):
    return -(-np.maximum(tokens, 0) // page)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def work(case):
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "norm_rope":
        rows, heads = case["rows"], hq + hk
        return {"bytes": rows * (heads * d * 4 + case["rot"] * 4 + 4), "flops": rows * heads * (4 * d * case["norm"] + 3 * case["rot"])}
    n, lens, shared, first = _shape(case)
    rows = int(n.sum())
    if case["op"] == "append":
        live = int(n[lens >= 0].sum())
        return {"bytes": rows * (hq * d * 4 + case["rot"] * 4 + 4) + live * hk * d * 8,
                "flops": rows * (hq + hk) * (4 * d * case["norm"] + 3 * case["rot"])}
    live = lens >= 0
    tokens = int((lens + n)[live].sum()) + int(shared.sum())
    seen = int((n * lens + n * (n + 1) // 2)[live].sum())
    for i in range(len(shared)):
        part = slice(int(first[i]), int(first[i + 1]))
        seen += int(n[part][live[part]].sum()) * int(shared[i])
    return {"bytes": tokens * hk * d * 4 + rows * hq * (d * 4 + 4), "flops": 4 * d * hq * seen}


# ---- inputs


def prepare(case, seed):
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = _dtype(case)
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    randn = lambda *s: torch.randn(*s, generator=gen, device=dev, dtype=torch.float32)  # noqa: E731
    ints = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(dev)  # noqa: E731
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device=dev)}
    if case["op"] == "norm_rope":
        rows = case["rows"]
        n = lens = None
    else:
        n, lens, shared, first = _shape(case)
        rows = int(n.sum())
    if case["op"] != "attend":
        # activations of a projection, one row after another; fused: the columns q, k, v of one matrix
        if case["fused"]:
            both = (randn(rows, (hq + 2 * hk) * d) * 1.5).to(dt)
            s["q"] = both[:, :hq * d].unflatten(1, (hq, d))
            s["k"] = both[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
            s["v"] = both[:, (hq + hk) * d:].unflatten(1, (hk, d))
        else:
            s["q"], s["k"], s["v"] = ((randn(rows, h, d) * 1.5).to(dt) for h in (hq, hk, hk))
        s["q_out"], s["k_out"] = torch.empty(rows, hq, d, dtype=dt, device=dev), torch.empty(rows, hk, d, dtype=dt, device=dev)
        s["q_weight"] = (1 + 0.2 * randn(d)).to(dt) if case["norm"] else None
        s["k_weight"] = (1 + 0.2 * randn(d)).to(dt) if case["norm"] else None
        half = case["rot"] // 2
        angle = torch.arange(TABLE_POSITIONS, device=dev, dtype=torch.float64)[:, None] * (
            THETA ** (-torch.arange(half, device=dev, dtype=torch.float64) / max(half, 1)))
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
    if case["op"] == "norm_rope":
        s["positions"] = torch.randint(0, TABLE_POSITIONS, (rows,), generator=gen, device=dev, dtype=torch.int32)
    if case["op"] != "norm_rope":
        page = case["page"]
        need = _pages_of(np.where(lens >= 0, lens + n, 0), page)
        width = max(1, int(need.max()))
        pneed = _pages_of(shared, page)
        total = int(need.sum() + pneed.sum()) + 3  # a few pages that nobody holds
        order = torch.randperm(total, generator=gen, device=dev).to(torch.int32).cpu().numpy()
        tables = np.full((case["groups"], width), -1, np.int32)
        used = 0
        for g in range(case["groups"]):
            tables[g, :need[g]] = order[used:used + need[g]]
            used += int(need[g])
        s["block_tables"], s["group_indptr"], s["lens"] = ints(tables), ints(np.concatenate([[0], np.cumsum(n)])), ints(lens)
        if case["op"] == "append":
            s["positions"] = ints(np.concatenate([np.where(lens[g] >= 0, lens[g] + np.arange(n[g]), 0) for g in range(case["groups"])]))
        s["k_cache"] = randn(total, hk, page, d).to(dt)
        s["v_cache"] = randn(total, hk, page, d).to(dt)
        s["pages"], s["longest"], s["most_rows"] = total, int((lens + n).max()), int(n.max())
    if case["op"] == "attend":
        # a few query heads look at few tokens, the others at many
        s["q"] = (randn(rows, hq, d) * (0.5 + 3.0 * torch.rand(1, hq, 1, generator=gen, device=dev))).to(dt)
        s["out"], s["lse_out"] = torch.empty(rows, hq, d, dtype=dt, device=dev), torch.empty(rows, hq, device=dev)
        if len(shared):
            ptab = np.full((len(shared), int(pneed.max())), -1, np.int32)
            for i in range(len(shared)):
                ptab[i, :pneed[i]] = order[used:used + pneed[i]]
                used += int(pneed[i])
            s["prefix_tables"], s["prefix_lens"], s["prefix_indptr"] = ints(ptab), ints(shared), ints(first)
            ends = np.concatenate([[0], np.cumsum(n)])[first]
            s["prefix_longest"], s["prefix_most_rows"] = int(shared.max()), int(np.diff(ends).max())
        if case["tree"]:
            # row j hangs on an earlier row of its group (the first row is the root) and sees its ancestors and itself
            r = np.random.RandomState(seed % (1 << 31))
            masks = []
            for g in range(case["groups"]):
                m = [1]
                for j in range(1, int(n[g])):
                    m.append(m[r.randint(0, j)] | (1 << j))
                masks += m
            s["row_masks"] = ints(np.array(masks, np.int64))
    if own:
        import logprob_epilogue_gb300 as lpe
        prefixes = len(shared) if case["op"] == "attend" else 0
        s["plan"] = lpe.AttnPlan(
            max_rows=rows, max_groups=case.get("groups", 1), q_heads=hq, kv_heads=hk, head_dim=d, page_size=case.get("page", 64),
            num_pages=s.get("pages", 1), max_pages=s["block_tables"].shape[1] if "block_tables" in s else 1,
            max_prefixes=prefixes, max_prefix_pages=s["prefix_tables"].shape[1] if prefixes else 0,
            max_group_rows=MAX_GROUP_ROWS if case["op"] == "attend" else 1, dtype=case["dtype"], device=0)
    return s


# ---- the framework's calls and the plain forms


def run(s):
    op = s["case"]["op"]
    if own:
        if op == "norm_rope":
            s["plan"].norm_rope(q=s["q"], k=s["k"], q_out=s["q_out"], k_out=s["k_out"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                eps=EPS, cos_sin=s["cos_sin"], interleaved=s["case"]["interleaved"], positions=s["positions"], status=s["status"])
            return {"q": s["q_out"], "k": s["k_out"]}
        if op == "append":
            s["plan"].append(q=s["q"], k=s["k"], v=s["v"], q_out=s["q_out"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                             cos_sin=s["cos_sin"], interleaved=s["case"]["interleaved"], positions=s["positions"],
                             group_indptr=s["group_indptr"], lens=s["lens"], block_tables=s["block_tables"],
                             k_cache=s["k_cache"], v_cache=s["v_cache"], status=s["status"])
            return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        s["plan"].attend(q=s["q"], k_cache=s["k_cache"], v_cache=s["v_cache"], group_indptr=s["group_indptr"], lens=s["lens"],
                         block_tables=s["block_tables"], out=s["out"], lse_out=s["lse_out"], status=s["status"],
                         row_masks=s.get("row_masks"), prefix_indptr=s.get("prefix_indptr"), prefix_lens=s.get("prefix_lens"),
                         prefix_tables=s.get("prefix_tables"))
        return {"out": s["out"], "lse": s["lse_out"]}
    if op == "norm_rope":
        return {"q": _plain_heads(s, s["q"], s["q_weight"]).to(s["q"].dtype), "k": _plain_heads(s, s["k"], s["k_weight"]).to(s["k"].dtype)}
    if op == "append":
        return _plain_append(s)
    return _plain_attend(s)


def _plain_heads(s, x, weight):
    """Each head's norm and rotation in 32 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    rot = s["cos_sin"].shape[1]
    if rot:
        cs = s["cos_sin"][s["positions"].long()][:, None, :]
        cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
        if s["case"]["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        x = torch.cat([turned, x[..., rot:]], -1)
    return x


def _row_groups(s, rows):
    """Each row's group and its place in it."""
    row = torch.arange(rows, device=s["lens"].device, dtype=torch.int32)
    g = torch.searchsorted(s["group_indptr"], row, right=True) - 1
    return g, row.long() - s["group_indptr"].long()[g]


def _plain_append(s):
    g, j = _row_groups(s, s["q"].shape[0])
    live = s["lens"][g] >= 0
    page = s["case"]["page"]
    token = (s["lens"].long()[g] + j)[live]
    at, off = s["block_tables"].long()[g[live], token // page], token % page
    k = _plain_heads(s, s["k"], s["k_weight"]).to(s["k"].dtype)
    s["k_cache"][at, :, off] = k[live]
    s["v_cache"][at, :, off] = s["v"][live]
    return {"q": _plain_heads(s, s["q"], s["q_weight"]).to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_part(s, q, tables, tokens, visible):
    """Softmax parts of q [B, n, Hq, D] over the first `tokens` tokens of tables [B, pages]; visible
    [B, n, tokens]: each row's maximum, sum of exponentials and unnormalised result."""
    case = s["case"]
    hk, d, page = case["kv_heads"], case["head_dim"], case["page"]
    b, n, hq, _ = q.shape
    at = tables[:, :-(-tokens // page)].long().clamp(min=0)
    k, v = (c[at].transpose(1, 2).flatten(2, 3)[:, :, :tokens].float() for c in (s["k_cache"], s["v_cache"]))
    q = q.float().view(b, n, hk, hq // hk, d).transpose(1, 2).flatten(2, 3)  # [B, Hk, n * share, D]
    x = (q @ k.transpose(2, 3)) * d ** -0.5
    x = x.view(b, hk, n, hq // hk, tokens).masked_fill(~visible[:, None, :, None, :], -math.inf)
    m = x.amax(-1)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m)[..., None])
    o = (p.flatten(2, 3) @ v).view(b, hk, n, hq // hk, d)
    back = lambda t: t.transpose(1, 2).flatten(2, 3)  # noqa: E731  [B, n, Hq, ...]
    return back(m), back(p.sum(-1)), back(o)


def _plain_attend(s):
    rows = s["q"].shape[0]
    dev = s["q"].device
    g, j = _row_groups(s, rows)
    lens, begin = s["lens"].long(), s["group_indptr"].long()
    # each group's own tokens: rows gathered to [groups, most rows], tokens padded to the longest
    most, longest = s["most_rows"], s["longest"]
    i = torch.arange(most, device=dev)
    at = (begin[:-1, None] + i).clamp(max=rows - 1)
    t = torch.arange(longest, device=dev)
    past = t[None, None, :] - lens[:, None, None]  # place among the round's own rows
    if "row_masks" in s:
        bits = s["row_masks"].long()[at][:, :, None]
        seen = (past < 0) | ((past < 32) & ((bits >> past.clamp(0, 31)) & 1 == 1))
    else:
        seen = past <= i[None, :, None]
    seen = seen & (lens >= 0)[:, None, None]
    m, l, o = (x[g, j] for x in _plain_part(s, s["q"][at], s["block_tables"], longest, seen))
    if "prefix_lens" in s:
        first = begin[s["prefix_indptr"].long()]  # first row of each prefix
        row = torch.arange(rows, device=dev)
        of = torch.searchsorted(first, row, right=True) - 1
        at = (first[:-1, None] + torch.arange(s["prefix_most_rows"], device=dev)).clamp(max=rows - 1)
        t = torch.arange(s["prefix_longest"], device=dev)
        seen = (t < s["prefix_lens"].long()[:, None])[:, None, :] & (lens >= 0)[g[at]][:, :, None]
        m2, l2, o2 = (x[of, row - first[of]] for x in _plain_part(s, s["q"][at], s["prefix_tables"], s["prefix_longest"], seen))
        top = torch.maximum(m, m2)
        safe = torch.where(top == -math.inf, 0.0, top)
        a, b = torch.exp(m - safe), torch.exp(m2 - safe)
        m, l, o = top, a * l + b * l2, a[..., None] * o + b[..., None] * o2
    out = torch.where(l[..., None] > 0, o / l[..., None], 0.0)
    return {"out": out.to(s["q"].dtype), "lse": m + torch.log(l)}


# ---- the definitions in 64 bits


def _exact_heads(s, x, weight):
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / y.shape[-1] + EPS) * weight.double()
    rot = s["case"]["rot"]
    z = y.clone()
    table = s["cos_sin"].double()[s["positions"].long()]
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if s["case"]["interleaved"] else (i, i + rot // 2)
        c, n = table[:, i, None], table[:, rot // 2 + i, None]
        z[..., a] = y[..., a] * c - y[..., b] * n
        z[..., b] = y[..., a] * n + y[..., b] * c
    return z


def exact(case, seed):
    global own
    keep, own = own, False  # the inputs alone
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    if case["op"] == "norm_rope":
        return {"q": _exact_heads(s, s["q"], s["q_weight"]), "k": _exact_heads(s, s["k"], s["k_weight"])}
    n, lens, shared, first = _shape(case)
    start = np.concatenate([[0], np.cumsum(n)])
    page, hk = case["page"], case["kv_heads"]
    tables = s["block_tables"].cpu().numpy()
    if case["op"] == "append":
        k = _exact_heads(s, s["k"], s["k_weight"])
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        dst, src = [], []
        for g in range(case["groups"]):
            for j in range(int(n[g]) if lens[g] >= 0 else 0):
                t = int(lens[g]) + j
                dst.append(int(tables[g, t // page]) * page + t % page)
                src.append(int(start[g]) + j)
        dst, src = torch.tensor(dst, device=kc.device), torch.tensor(src, device=kc.device)
        for c, new in ((kc, k), (vc, s["v"].double())):
            for h in range(hk):
                flat = c[:, h].reshape(-1, case["head_dim"])
                flat[dst] = new[src, h]
                c[:, h] = flat.view(c[:, h].shape)
        return {"q": _exact_heads(s, s["q"], s["q_weight"]), "k_cache": kc, "v_cache": vc}
    if work(case)["flops"] > 5e12:
        return None
    share = case["q_heads"] // hk
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device=out.device)
    ptables = s["prefix_tables"].cpu().numpy() if len(shared) else None
    masks = s["row_masks"].cpu().numpy() if "row_masks" in s else None

    def tokens_of(cache, h, table, count):
        at = torch.from_numpy(np.ascontiguousarray(table[:-(-count // page)])).long().to(out.device)
        return cache[at, h].reshape(-1, case["head_dim"])[:count].double()

    for h in range(hk):
        heads = slice(h * share, (h + 1) * share)
        for i in range(max(1, len(shared))):
            if len(shared):
                pk, pv = (tokens_of(s[c], h, ptables[i], int(shared[i])) for c in ("k_cache", "v_cache"))
                lo, hi = int(first[i]), int(first[i + 1])
                r0, r1 = int(start[lo]), int(start[hi])
                px = torch.einsum("rsd,td->rst", s["q"][r0:r1, heads].double(), pk) / math.sqrt(case["head_dim"])
                ptop = px.amax(-1)
                pe = torch.exp(px - ptop[..., None])
                pl, po = pe.sum(-1), torch.einsum("rst,td->rsd", pe, pv)
                del px, pe
            else:
                lo, hi, r0 = 0, case["groups"], 0
            for g in range(lo, hi):
                if lens[g] < 0:
                    continue
                a, b, count = int(start[g]), int(start[g + 1]), int(lens[g] + n[g])
                k, v = (tokens_of(s[c], h, tables[g], count) for c in ("k_cache", "v_cache"))
                x = torch.einsum("rsd,td->rst", s["q"][a:b, heads].double(), k) / math.sqrt(case["head_dim"])
                for j in range(int(n[g])):
                    bits = int(masks[a + j]) if masks is not None else (2 << j) - 1
                    for m in range(int(n[g])):
                        if not bits >> m & 1:
                            x[j, :, int(lens[g]) + m] = -math.inf
                top = x.amax(-1)
                if len(shared):
                    top = torch.maximum(top, ptop[a - r0:b - r0])
                e = torch.exp(x - top[..., None])
                l, o = e.sum(-1), torch.einsum("rst,td->rsd", e, v)
                if len(shared):
                    f = torch.exp(ptop[a - r0:b - r0] - top)
                    l, o = l + f * pl[a - r0:b - r0], o + f[..., None] * po[a - r0:b - r0]
                out[a:b, heads], lse[a:b, heads] = o / l[..., None], top + torch.log(l)
    return {"out": out, "lse": lse}
