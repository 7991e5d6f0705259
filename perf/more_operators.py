"""Cases of the operators around a paged cache held in 4 bits: the reservation of
a round's pages with its positions and slots, the append of keys and values in
4 bits, and the attention of verify rows over that cache.

``own`` selects what ``run`` does: the plain form in elementary torch
operations, or the calls a user makes of ``logprob_epilogue_gb300.AttnPlan``.

A round of a batch: group g owns ``counts[g]`` rows (the last committed token
and its drafts, or a prompt), ``lens[g]`` tokens of its own are committed in the
cache (negative: an idle slot of the batch), row j of the group is token
lens[g] + j.  A cached head of a token is head_dim codes of type e2m1, two to a
byte, and one e4m3 scale for each 16 of them.
"""
import math

import numpy as np
import torch

own = False

MAX_GROUP_ROWS = 32  # rows of one group in the attention cases
BLOCK = 16  # lanes that share a scale
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of e2m1


def listed():
    """Twelve cases; the head counts are a grouped-query layout of 32 query and 8 key-value heads
    unless a case says otherwise."""
    res = {"op": "reserve", "page": 64, "idle": 0, "short": 0, "spare": 7}
    app = {"op": "append", "dtype": "bf16", "kv_heads": 8, "head_dim": 128, "page": 64, "fused": True, "idle": 0}
    att = {"op": "attend", "dtype": "bf16", "q_heads": 32, "kv_heads": 8, "head_dim": 128, "page": 64, "idle": 0,
           "prefixes": 0, "prefix": 0, "tree": False}
    return [
        # the verify round of 128 requests with 3 drafts each, three of them finished: latency
        dict(res, name="reserve_verify", groups=128, rows_lo=4, rows_hi=4, len_lo=0, len_hi=8192, idle=3),
        # a large batch of single tokens, small pages, more requests than the free pages serve
        dict(res, name="reserve_batch", groups=4099, rows_lo=1, rows_hi=1, len_lo=0, len_hi=2000, page=16, idle=101, short=9),
        # ragged prompts entering the cache at once
        dict(res, name="reserve_prompts", groups=37, rows_lo=1001, rows_hi=32_003, len_lo=0, len_hi=777),
        # one request decoding one token: the smallest call
        dict(app, name="append4_token", groups=1, rows_lo=1, rows_hi=1, len_lo=1000, len_hi=1000, page=16),
        # the verify round of 128 requests with 3 drafts each, three slots of the batch idle
        dict(app, name="append4_verify", groups=128, rows_lo=4, rows_hi=4, len_lo=0, len_hi=2048, idle=3),
        # five prompts entering the cache at once, of ragged lengths
        dict(app, name="append4_prompts", groups=5, rows_lo=1501, rows_hi=5003, len_lo=0, len_hi=777, fused=False),
        # one request decoding one token at a moderate context: latency, and one row's work over the whole GPU
        dict(att, name="attend4_token", groups=1, rows_lo=1, rows_hi=1, len_lo=4095, len_hi=4095, page=16),
        # the verify round of 128 requests with 3 drafts each, ragged contexts, three slots idle: bandwidth
        dict(att, name="attend4_verify", groups=128, rows_lo=4, rows_hi=4, len_lo=0, len_hi=8192, idle=3),
        # four requests at very long contexts with small heads
        dict(att, name="attend4_long", groups=4, rows_lo=1, rows_hi=4, len_lo=100_001, len_hi=131_071, head_dim=64,
             q_heads=16, kv_heads=2, dtype="f16", page=128),
        # trees of drafts, up to 16 rows a group, small pages
        dict(att, name="attend4_tree", groups=16, rows_lo=7, rows_hi=16, len_lo=1, len_hi=4001, page=32, tree=True),
        # three prefixes of ragged length, drafts, multi-query heads
        dict(att, name="attend4_prefixes", groups=47, rows_lo=2, rows_hi=6, len_lo=5, len_hi=1500, prefixes=3,
             prefix=12_345, q_heads=40, kv_heads=4),
        # 256 requests with 7 drafts each behind one long shared prefix: arithmetic
        dict(att, name="attend4_prefix_large", groups=256, rows_lo=8, rows_hi=8, len_lo=0, len_hi=1024, prefixes=1,
             prefix=32_768),
    ]


def draw(rng):
    """One more case of the same ranges."""
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["reserve", "append", "attend", "attend", "attend"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    if op == "reserve":
        groups = log_int(1, 4099)
        len_hi = log_int(1, min(131_000, 8_000_000 // groups))
        hi = log_int(1, max(1, min(40_000, 700_000 // groups)))
        return {"op": op, "page": page, "groups": groups, "rows_lo": rng.randint(1, hi), "rows_hi": hi, "len_lo": 0, "len_hi": len_hi,
                "idle": min(groups - 1, rng.choice([0, 0, 3, 50])), "short": rng.choice([0, 0, 2, 30]), "spare": rng.randint(0, 100)}
    dim = rng.choice([64, 128])
    kv = rng.choice([1, 2, 4, 8])
    if op == "append":
        c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16"]), "kv_heads": kv, "head_dim": dim, "page": page,
             "groups": log_int(1, 256), "len_lo": 0, "len_hi": log_int(1, 2048), "fused": rng.random() < 0.5}
        hi = log_int(1, max(1, 20_000 // c["groups"]))
        c.update(rows_lo=max(1, hi // 2), rows_hi=hi, idle=min(c["groups"] - 1, rng.choice([0, 0, 1, 4])))
        return c
    share = rng.choice([1, 2, 3, 4, 5, 8, 12])  # query heads of one key-value head
    while kv * share > 48:
        share = rng.choice([1, 2, 3, 4])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16"]), "q_heads": kv * share, "kv_heads": kv, "head_dim": dim}
    groups = log_int(1, 256)
    rows_hi = rng.choice([1, 1, 2, 4, 5, 8, 16])
    len_hi = log_int(1, min(131_000, 1_000_000 // groups))
    prefixes = rng.choice([0, 0, 1, 1, 2, 4])
    prefix = log_int(1, 32_768) if prefixes else 0
    while groups * rows_hi * c["q_heads"] * prefix > 1_000_000_000:  # at most half the arithmetic of the largest listed case
        prefix = max(1, prefix // 2)
    c.update(page=page, groups=groups, rows_lo=rng.randint(1, rows_hi), rows_hi=rows_hi, len_lo=rng.randint(0, len_hi), len_hi=len_hi,
             idle=min(groups - 1, rng.choice([0, 0, 1, 5])), prefixes=min(prefixes, groups), prefix=prefix,
             tree=rows_hi > 1 and rng.random() < 0.4)
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


def _holdings(case):
    """Of a reservation: pages that each group holds and needs, and how many pages are free."""
    n, lens, _, _ = _shape(case)
    live = lens >= 0
    held = np.where(live, _pages_of(lens, case["page"]), 1 + np.arange(len(lens)) % 5)  # a finished request still holds some
    need = np.where(live, np.maximum(0, _pages_of(lens + n, case["page"]) - held), 0)
    free = int(need.sum()) + case["spare"] if not case["short"] else max(0, int(need.sum()) - case["short"])
    return held, need, free


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def work(case):
    n, lens, shared, first = _shape(case)
    rows = int(n.sum())
    live = lens >= 0
    if case["op"] == "reserve":
        held, need, free = _holdings(case)
        new = min(free, int(need.sum()))
        return {"bytes": 24 * len(n) + 12 * rows + 8 * new + 8 * int(held[~live].sum()), "flops": 2 * rows + 4 * len(n)}
    hk, d = case["kv_heads"], case["head_dim"]
    token = 2 * hk * (d // 2 + d // BLOCK)  # bytes of a cached token
    if case["op"] == "append":
        return {"bytes": rows * hk * d * 8 + rows * 4 + int(n[live].sum()) * token, "flops": rows * hk * d * 2 * 4}
    hq = case["q_heads"]
    tokens = int((lens + n)[live].sum()) + int(shared.sum())
    seen = int((n * lens + n * (n + 1) // 2)[live].sum())
    for i in range(len(shared)):
        part = slice(int(first[i]), int(first[i + 1]))
        seen += int(n[part][live[part]].sum()) * int(shared[i])
    return {"bytes": tokens * token + rows * hq * (d * 4 + 4), "flops": 4 * d * hq * seen}


# ---- inputs


def _fill(gen, pages, hk, page, d, outlier):
    """(codes, scales) of a cache whose values are normal, some lanes of the keys larger; a few pages at a time."""
    dev = gen.device
    codes = torch.empty(pages, hk, page, d // 2, dtype=torch.uint8, device=dev)
    scales = torch.empty(pages, hk, page, d // BLOCK, dtype=torch.float8_e4m3fn, device=dev)
    step = max(1, (1 << 26) // (hk * page * d))
    for at in range(0, pages, step):
        x = torch.randn(min(step, pages - at), hk, page, d, generator=gen, device=dev) * outlier
        codes[at:at + step], scales[at:at + step] = _plain_quantise(x)[:2]
    return codes, scales


def prepare(case, seed):
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device=dev, dtype=torch.float32)  # noqa: E731
    ints = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(dev)  # noqa: E731
    n, lens, shared, first = _shape(case)
    groups, rows, page = case["groups"], int(n.sum()), case["page"]
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device=dev), "lens": ints(lens)}
    hq, hk, d = case.get("q_heads", case.get("kv_heads", 1)), case.get("kv_heads", 1), case.get("head_dim", 64)
    if case["op"] == "reserve":
        held, need, free = _holdings(case)
        width = max(1, int((held + need).max()))
        total = int(held.sum()) + free
        ring = total + 5  # room for every page, and the queue of free ones goes round its end
        order = torch.randperm(total, generator=gen, device=dev).to(torch.int32).cpu().numpy()
        tables = np.full((groups, width), -1, np.int32)
        tables[np.arange(width)[None, :] < held[:, None]] = order[:int(held.sum())]
        head = 3 * ring - max(1, free // 2)
        queue = np.zeros(ring, np.int32)
        queue[(head + np.arange(free)) % ring] = order[int(held.sum()):]
        empty = lambda *z: torch.empty(*z, dtype=torch.int32, device=dev)  # noqa: E731
        s.update(counts=ints(n), held=ints(held), free_pages=ints(queue), block_tables=ints(tables),
                 queue=torch.tensor([head, head + free], dtype=torch.int64, device=dev), queue_out=torch.empty(2, dtype=torch.int64, device=dev),
                 group_indptr=empty(groups + 1), round_lens=empty(groups), held_out=empty(groups), positions=empty(rows + 3),
                 slots=torch.empty(rows + 3, dtype=torch.int64, device=dev))  # three rows of padding
        pages = total
    else:
        dt = _dtype(case)
        need = _pages_of(np.where(lens >= 0, lens + n, 0), page)
        width = max(1, int(need.max()))
        pneed = _pages_of(shared, page)
        pages = int(need.sum() + pneed.sum()) + 3  # a few pages that nobody holds
        order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32).cpu().numpy()
        tables = np.full((groups, width), -1, np.int32)
        tables[np.arange(width)[None, :] < need[:, None]] = order[:int(need.sum())]
        s["block_tables"], s["group_indptr"] = ints(tables), ints(np.concatenate([[0], np.cumsum(n)]))
        outlier = torch.where(torch.rand(d, generator=gen, device=dev) < 0.05, 4.0, 1.0)
        s["k_cache"], s["k_scales"] = _fill(gen, pages, hk, page, d, outlier)
        s["v_cache"], s["v_scales"] = _fill(gen, pages, hk, page, d, 1.0)
    if case["op"] == "append":
        s["positions"] = ints(np.concatenate([np.where(lens[g] >= 0, lens[g] + np.arange(n[g]), 0) for g in range(groups)]))
        # keys already rotated, and values; fused: the columns of one matrix
        if case["fused"]:
            both = randn(rows, 2 * hk * d).to(dt)
            s["k"], s["v"] = both[:, :hk * d].unflatten(1, (hk, d)), both[:, hk * d:].unflatten(1, (hk, d))
        else:
            s["k"], s["v"] = (randn(rows, hk, d) * outlier).to(dt), randn(rows, hk, d).to(dt)
        s["k_held"], s["v_held"] = (torch.empty(rows, hk, d, dtype=dt, device=dev) for _ in range(2))
    if case["op"] == "attend":
        s["longest"], s["most_rows"] = int((lens + n).max()), int(n.max())
        # a few query heads look at few tokens, the others at many
        s["q"] = (randn(rows, hq, d) * (0.5 + 2.0 * torch.rand(1, hq, 1, generator=gen, device=dev))).to(dt)
        s["out"], s["lse_out"] = torch.empty(rows, hq, d, dtype=dt, device=dev), torch.empty(rows, hq, device=dev)
        if len(shared):
            ptab = np.full((len(shared), int(pneed.max())), -1, np.int32)
            ptab[np.arange(ptab.shape[1])[None, :] < pneed[:, None]] = order[int(need.sum()):int(need.sum() + pneed.sum())]
            s["prefix_tables"], s["prefix_lens"], s["prefix_indptr"] = ints(ptab), ints(shared), ints(first)
            ends = np.concatenate([[0], np.cumsum(n)])[first]
            s["prefix_longest"], s["prefix_most_rows"] = int(shared.max()), int(np.diff(ends).max())
        if case["tree"]:
            # row j hangs on an earlier row of its group (the first row is the root) and sees its ancestors and itself
            r = np.random.RandomState(seed % (1 << 31))
            masks = []
            for g in range(groups):
                m = [1]
                for j in range(1, int(n[g])):
                    m.append(m[r.randint(0, j)] | (1 << j))
                masks += m
            s["row_masks"] = ints(np.array(masks, np.int64))
    if own:
        import logprob_epilogue_gb300 as lpe
        attend = case["op"] == "attend"
        s["plan"] = lpe.AttnPlan(
            max_rows=rows + 3, max_groups=groups, q_heads=hq, kv_heads=hk, head_dim=d, page_size=page, num_pages=pages,
            max_pages=s["block_tables"].shape[1], max_prefixes=len(shared), max_prefix_pages=s["prefix_tables"].shape[1] if len(shared) else 0,
            max_group_rows=MAX_GROUP_ROWS if attend else 1, dtype=case.get("dtype", "bf16"), device=0, kv_bits=4)
    return s


# ---- the framework's calls and the plain forms


def run(s):
    op = s["case"]["op"]
    if op == "reserve":
        if not own:
            return _plain_reserve(s)
        s["plan"].reserve(lens=s["lens"], counts=s["counts"], held=s["held"], queue=s["queue"], free_pages=s["free_pages"],
                          block_tables=s["block_tables"], group_indptr=s["group_indptr"], round_lens=s["round_lens"],
                          held_out=s["held_out"], queue_out=s["queue_out"], positions=s["positions"], slots=s["slots"], status=s["status"])
        return {x: s[x] for x in ("group_indptr", "round_lens", "held_out", "queue_out", "positions", "slots", "block_tables", "free_pages")}
    if op == "append":
        if own:
            s["plan"].append4(k=s["k"], v=s["v"], k_cache=s["k_cache"], v_cache=s["v_cache"], k_scales=s["k_scales"], v_scales=s["v_scales"],
                              group_indptr=s["group_indptr"], lens=s["lens"], block_tables=s["block_tables"], positions=s["positions"],
                              k_held=s["k_held"], v_held=s["v_held"], status=s["status"])
        else:
            _plain_append(s)
        # the rows as the values that the cache now holds, and the cache itself
        return {x: s[x] for x in ("k_held", "v_held", "k_cache", "v_cache", "k_scales", "v_scales")}
    if not own:
        return _plain_attend(s)
    s["plan"].attend4(q=s["q"], k_cache=s["k_cache"], v_cache=s["v_cache"], k_scales=s["k_scales"], v_scales=s["v_scales"],
                      group_indptr=s["group_indptr"], lens=s["lens"], block_tables=s["block_tables"], out=s["out"], lse_out=s["lse_out"],
                      status=s["status"], row_masks=s.get("row_masks"), prefix_indptr=s.get("prefix_indptr"),
                      prefix_lens=s.get("prefix_lens"), prefix_tables=s.get("prefix_tables"))
    return {"out": s["out"], "lse": s["lse_out"]}


def _plain_reserve(s):
    """Groups in order take the pages they lack from the queue's head until it runs out; finished groups' pages join its tail."""
    page, cap, width = s["case"]["page"], s["free_pages"].numel(), s["block_tables"].shape[1]
    lens, n, held = s["lens"].long(), s["counts"].long(), s["held"].long()
    head, tail = s["queue"][0], s["queue"][1]
    live = lens >= 0
    need = torch.where(live, ((lens + n + page - 1) // page - held).clamp(min=0), 0)
    upto = need.cumsum(0)
    served = live & ((need == 0) | (upto <= tail - head))
    taken = torch.where(served, need, 0)
    before = upto - need
    column = torch.arange(width, device=lens.device)
    new = served[:, None] & (column >= held[:, None]) & (column < (held + need)[:, None])
    at = (head + before[:, None] + column - held[:, None]) % cap
    tables = torch.where(new, s["free_pages"][at], s["block_tables"])
    # pages of finished groups, in the order of the groups
    gone = ~live[:, None] & (column < held[:, None])
    back = s["block_tables"][gone]
    queue = s["free_pages"].clone()
    queue[(tail + torch.arange(back.numel(), device=lens.device)) % cap] = back
    indptr = torch.nn.functional.pad(n.cumsum(0), (1, 0))
    row = torch.arange(s["positions"].numel(), device=lens.device)
    g = (torch.searchsorted(indptr, row, right=True) - 1).clamp(max=len(n) - 1)
    ok = (row < indptr[-1]) & served[g]
    token = torch.where(ok, lens[g] + row - indptr[g], 0)
    slot = tables[g, token // page].long() * page + token % page
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return {"group_indptr": i32(indptr), "round_lens": i32(torch.where(served | ~live, lens, -1)), "held_out": i32(torch.where(live, held + taken, 0)),
            "queue_out": torch.stack([head + taken.sum(), tail + back.numel()]), "positions": i32(torch.where(ok, token, -1)),
            "slots": torch.where(ok, slot, -1), "block_tables": tables, "free_pages": queue}


def _plain_quantise(x):
    """(codes, scales, the values they stand for) of x [..., lanes]: the scale of 16 lanes is the e4m3 value nearest to a
    sixth of the largest magnitude, a code the e2m1 value nearest to the lane over its scale (ties to the even code)."""
    x = x.float().unflatten(-1, (-1, BLOCK))
    scale = (x.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = scale.float()[..., None]
    y = torch.where(step > 0, x.abs() / step, 0.0)
    level = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    code = (level + 8 * torch.signbit(x).to(torch.uint8)).flatten(-2)
    value = torch.tensor(LEVELS, device=x.device)[level.int()] * step
    value = torch.where(torch.signbit(x), -value, value).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale, value


def _row_groups(s, rows):
    """Each row's group and its place in it."""
    row = torch.arange(rows, device=s["lens"].device, dtype=torch.int32)
    g = torch.searchsorted(s["group_indptr"], row, right=True) - 1
    return g, row.long() - s["group_indptr"].long()[g]


def _plain_append(s):
    g, j = _row_groups(s, s["k"].shape[0])
    live = s["lens"][g] >= 0
    page = s["case"]["page"]
    token = (s["lens"].long()[g] + j)[live]
    at, off = s["block_tables"].long()[g[live], token // page], token % page

    def put(x, codes, scales, held):
        code, scale, value = _plain_quantise(x)
        codes[at, :, off] = code[live]
        scales.view(torch.uint8)[at, :, off] = scale.view(torch.uint8)[live]
        held.copy_(value)

    put(s["k"], s["k_cache"], s["k_scales"], s["k_held"])
    put(s["v"], s["v_cache"], s["v_scales"], s["v_held"])


def _values(codes, scales):
    """What cached codes [..., lanes / 2] and scales [..., lanes / 16] stand for, in 32 bits."""
    levels = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=codes.device)
    pairs = torch.stack([levels.repeat(16), levels.repeat_interleave(16)], -1)  # of a byte: low half first
    x = pairs[codes.int()].flatten(-2)
    return (x.unflatten(-1, (-1, BLOCK)) * scales.float()[..., None]).flatten(-2)


def _plain_part(s, q, tables, tokens, visible):
    """Softmax parts of q [B, n, Hq, D] over the first `tokens` tokens of tables [B, pages]; visible
    [B, n, tokens]: each row's maximum, sum of exponentials and unnormalised result."""
    case = s["case"]
    hk, d, page = case["kv_heads"], case["head_dim"], case["page"]
    b, n, hq, _ = q.shape
    at = tables[:, :-(-tokens // page)].long().clamp(min=0)
    k, v = (_values(s[x + "_cache"][at], s[x + "_scales"].view(torch.uint8)[at].view(torch.float8_e4m3fn))
            .transpose(1, 2).flatten(2, 3)[:, :, :tokens] for x in "kv")
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


def _nearest(x, values):
    """The entries of an ascending list of representable values nearest to x >= 0, ties to the even entry."""
    values = torch.tensor(values, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(values, x.contiguous()).clamp(1, len(values) - 1)
    lo = hi - 1
    below, above = x - values[lo], values[hi] - x
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return torch.where(x >= values[-1], values[-1], torch.where(up, values[hi], values[lo]))


def _exact_quantise(x):
    """(scales, values) of x [rows, heads, lanes] in 64 bits."""
    e4m3 = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]
    x = x.double()
    blocks = x.reshape(*x.shape[:-1], -1, BLOCK)
    scale = _nearest(blocks.abs().max(-1).values / 6, e4m3)
    over = torch.where(scale > 0, scale, 1.0)[..., None]
    value = _nearest(blocks.abs() / over, list(LEVELS)) * scale[..., None] * blocks.sign()
    return scale, value.reshape(x.shape)


def _exact_tokens(s, x, h, table, count):
    """The first `count` tokens of a page table, head h, in 64 bits."""
    at = torch.from_numpy(np.ascontiguousarray(table[:-(-count // s["case"]["page"])])).long().to(s["q"].device)
    raw = s[x + "_cache"][at, h].reshape(-1, s["case"]["head_dim"] // 2)[:count].int()
    level = torch.tensor(LEVELS, dtype=torch.float64, device=raw.device)
    half = [level[c & 7] * (1.0 - 2.0 * (c >> 3 & 1)) for c in (raw & 15, raw >> 4)]
    scale = s[x + "_scales"].view(torch.uint8)[at, h].reshape(-1, s["case"]["head_dim"] // BLOCK)[:count].view(torch.float8_e4m3fn).double()
    return torch.stack(half, -1).flatten(-2) * scale.repeat_interleave(BLOCK, -1)


def exact(case, seed):
    global own
    if case["op"] == "reserve":
        return None  # whole numbers
    keep, own = own, False  # the inputs alone
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    n, lens, shared, first = _shape(case)
    start = np.concatenate([[0], np.cumsum(n)])
    page, hk = case["page"], case["kv_heads"]
    tables = s["block_tables"].cpu().numpy()
    if case["op"] == "append":
        dst, src = [], []
        for g in range(case["groups"]):
            for j in range(int(n[g]) if lens[g] >= 0 else 0):
                t = int(lens[g]) + j
                dst.append(int(tables[g, t // page]) * page + t % page)
                src.append(int(start[g]) + j)
        dev = s["k"].device
        dst, src = torch.tensor(dst, device=dev), torch.tensor(src, device=dev)
        found = {"k_cache": None, "v_cache": None}  # codes
        for x in "kv":
            scale, found[x + "_held"] = _exact_quantise(s[x])
            cache = s[x + "_scales"].double()
            for h in range(hk):
                flat = cache[:, h].reshape(-1, cache.shape[-1])
                flat[dst] = scale[src, h]
                cache[:, h] = flat.view(cache[:, h].shape)
            found[x + "_scales"] = cache
        return found
    if work(case)["flops"] > 5e12:
        return None
    share = case["q_heads"] // hk
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device=out.device)
    ptables = s["prefix_tables"].cpu().numpy() if len(shared) else None
    masks = s["row_masks"].cpu().numpy() if "row_masks" in s else None
    for h in range(hk):
        heads = slice(h * share, (h + 1) * share)
        for i in range(max(1, len(shared))):
            if len(shared):
                pk, pv = (_exact_tokens(s, x, h, ptables[i], int(shared[i])) for x in "kv")
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
                k, v = (_exact_tokens(s, x, h, tables[g], count) for x in "kv")
                x = torch.einsum("rsd,td->rst", s["q"][a:b, heads].double(), k) / math.sqrt(case["head_dim"])
                own_rows = torch.arange(int(n[g]), device=x.device)
                if masks is None:
                    hidden = own_rows[None, :] > own_rows[:, None]
                else:
                    hidden = (torch.from_numpy(masks[a:b].astype(np.int64)).to(x.device)[:, None] >> own_rows) & 1 == 0
                x[:, :, int(lens[g]):].masked_fill_(hidden[:, None, :], -math.inf)
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
