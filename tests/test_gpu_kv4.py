"""The operators around a cache in 4 bits on the GPU: reservation of a round's
pages, append, attention."""
import numpy as np
import pytest

import attn_ref as R
import kv4_ref as K
from test_gpu_attn import batch, dev, generator, i32, plan_of, rand, status_word, table

pytestmark = pytest.mark.gpu


# ---- reservation


def reserve_inputs(counts, lens, page, seed, *, free=None, spare=3, extra=0, ring_extra=5, idle_holds=2):
    """Host lists of a reservation: what groups hold covers their committed tokens; random pages."""
    r = np.random.RandomState(seed)
    held = [(-(-l // page) if l >= 0 else int(r.randint(0, idle_holds + 1))) for l in lens]
    need = [max(0, -(-(l + max(n, 0)) // page) - h) if l >= 0 else 0 for l, n, h in zip(lens, counts, held)]
    free = sum(need) + spare if free is None else free
    width = max([1] + [h + m for h, m in zip(held, need)]) + extra
    total = sum(held) + free
    order = r.permutation(total).tolist()
    tables = np.full((len(lens), width), -1, np.int64)
    at = 0
    for g, h in enumerate(held):
        tables[g, :h] = order[at:at + h]
        at += h
    ring = total + ring_extra
    head = int(r.randint(0, 3 * ring))
    queue = np.full(ring, -7, np.int64)
    for i in range(free):
        queue[(head + i) % ring] = order[at + i]
    return dict(lens=list(lens), counts=list(counts), held=held, queue=[head, head + free], free_pages=queue, tables=tables, pages=total)


def run_reserve(x, page, rows, *, starts=None, inplace=False, slots=True, plan=None, stream=None, max_pages=None):
    import torch
    G = len(x["lens"])
    t = dict(lens=i32(x["lens"]), counts=i32(x["counts"]), held=i32(x["held"]), free_pages=i32(x["free_pages"]),
             block_tables=i32(x["tables"]), queue=torch.tensor(x["queue"], dtype=torch.int64, device=dev()),
             starts=None if starts is None else i32(starts))
    full = lambda n, dtype=torch.int32: torch.full((n,), -99, dtype=dtype, device=dev())  # noqa: E731
    t.update(group_indptr=full(G + 1), round_lens=full(G), held_out=t["held"] if inplace else full(G),
             queue_out=t["queue"] if inplace else full(2, torch.int64), positions=full(rows), slots=full(rows, torch.int64) if slots else None)
    st = status_word()
    p = plan or plan_of(max_rows=max(rows, 1), max_groups=max(G, 1), page_size=page, num_pages=x["pages"], max_pages=x["tables"].shape[1], kv_bits=4)
    p.reserve(**t, status=st)
    torch.cuda.synchronize()
    return t, int(st[0])


def check_reserve(t, st, want):
    import logprob_epilogue_gb300 as lpe
    for name in ("group_indptr", "round_lens", "held_out", "queue_out", "positions", "slots", "block_tables", "free_pages"):
        if t[name] is not None:
            got = t[name].cpu().numpy()
            assert np.array_equal(got, np.asarray(want[name]).reshape(got.shape)), name
    assert st == (lpe.STATUS_BAD_GROUP if want["bad"] else 0) | (lpe.STATUS_NO_PAGES if want["none"] else 0) | (
        lpe.STATUS_BAD_PAGE if want["bad_page"] else 0)


def both_reserve(x, page, rows, starts=None, **kw):
    want = K.reserve(x["lens"], x["counts"], x["held"], x["queue"], x["free_pages"], x["tables"], rows=rows, page=page,
                     max_pages=x["tables"].shape[1], num_pages=x["pages"], starts=starts)
    t, st = run_reserve(x, page, rows, starts=starts, **kw)
    check_reserve(t, st, want)
    return t, want


@pytest.mark.parametrize("page", [8, 64, 256])
@pytest.mark.parametrize("groups,hi,len_hi", [(1, 1, 0), (1, 4, 1000), (3, 700, 20), (33, 8, 300), (1024, 4, 50), (1025, 3, 200), (2049, 1, 40), (5, 3001, 9)])
@pytest.mark.parametrize("inplace", [False, True])
def test_reserve(page, groups, hi, len_hi, inplace):
    r = np.random.RandomState(groups + hi)
    lens = r.randint(-1 if groups > 2 else 0, len_hi + 1, groups).tolist()
    counts = r.randint(0, hi + 1, groups).tolist()
    x = reserve_inputs(counts, lens, page, seed=groups)
    both_reserve(x, page, sum(counts) + 5, inplace=inplace, starts=r.randint(0, 1000, groups).tolist() if inplace else None)


@pytest.mark.parametrize("groups", [40, 1500])
def test_reserve_runs_out_of_pages(groups):
    r = np.random.RandomState(1)
    counts, lens = r.randint(0, 20, groups).tolist(), r.randint(-1, 60, groups).tolist()
    full = reserve_inputs(counts, lens, 8, seed=2, spare=0)
    need = full["queue"][1] - full["queue"][0]
    for free in (0, 1, need // 2, need - 1, need):
        x = reserve_inputs(counts, lens, 8, seed=2, free=free)
        x["tables"] = np.pad(x["tables"], ((0, 0), (0, 3)), constant_values=-1)
        _, want = both_reserve(x, 8, sum(counts))
        assert want["none"] == (free < need)


@pytest.mark.parametrize("groups", [12, 1100])
def test_reserve_malformed_groups(groups):
    r = np.random.RandomState(3)
    counts, lens = r.randint(1, 9, groups).tolist(), r.randint(0, 40, groups).tolist()
    lens[5], lens[7] = -3, -1
    x = reserve_inputs(counts, lens, 8, seed=4, extra=1, spare=40)
    width = x["tables"].shape[1]
    x["counts"][2] = -4                # a negative count
    x["held"][4] = -1                  # holds less than nothing
    x["held"][5] = width + 1           # an idle group past its table
    x["lens"][6] = 8 * width           # more tokens than its table takes
    x["counts"][9] = 8 * width
    rows = sum(max(n, 0) for n in x["counts"])
    both_reserve(x, 8, rows)
    both_reserve(x, 8, rows - counts[-1] - 1)  # the last two groups are past the rows
    both_reserve(x, 8, 0)
    for lens6, held6 in ((2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (0, -2 ** 31)):
        x["lens"][6], x["held"][6] = lens6, held6
        both_reserve(x, 8, rows)


def test_reserve_counts_past_32_bits():
    x = dict(
        lens=[3, 0, 0, 0, 5], counts=[1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 4], held=[1, 0, 0, 0, 1], queue=[0, 5],
        free_pages=np.arange(2, 9), tables=np.array([[0, -1]] + [[-1, -1]] * 3 + [[1, -1]]), pages=9)
    both_reserve(x, 8, 20)


def test_reserve_unsound_queues_and_full_rings():
    counts, lens = [4, 4, 1, 4], [30, -1, 8, -1]
    for queue in ([5, 4], [-1, 3], [0, 10 ** 12], [2 ** 62, 2 ** 62 + 3]):
        x = reserve_inputs(counts, lens, 8, seed=1)
        x["queue"] = queue
        both_reserve(x, 8, 13)
    # room in the ring for one idle group's pages and not for the other's
    x = dict(lens=[-1, -1, 4], counts=[1, 1, 1], held=[2, 2, 1], queue=[7, 8], free_pages=np.array([9, 9, 9, 8]), tables=np.array([[0, 1, -1], [2, 3, -1], [4, -1, -1]]), pages=9)
    both_reserve(x, 8, 3)


def test_reserve_pages_and_positions_out_of_range():
    import logprob_epilogue_gb300 as lpe
    x = reserve_inputs([2, 3, 4], [9, 0, 20], 8, seed=1)
    x["tables"][0, 1] = x["pages"]     # a page that does not exist
    both_reserve(x, 8, 9)
    x = reserve_inputs([2, 3], [9, 0], 8, seed=1)
    t, st = run_reserve(x, 8, 5, starts=[2 ** 31 - 1 - 9, 7])
    assert st == lpe.STATUS_BAD_POSITION
    assert t["positions"].tolist() == [2 ** 31 - 1, -1, 7, 8, 9]


def test_reserve_again_gives_the_same():
    import torch
    r = np.random.RandomState(0)
    for groups in (50, 3000):
        counts, lens = r.randint(0, 5, groups).tolist(), r.randint(-1, 90, groups).tolist()
        x = reserve_inputs(counts, lens, 16, seed=6)
        t, want = both_reserve(x, 16, sum(counts))
        p = plan_of(max_rows=sum(counts), max_groups=groups, page_size=16, num_pages=x["pages"], max_pages=x["tables"].shape[1])  # a plan of 16 bits
        st = status_word()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            p.reserve(**t, status=st)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            p.reserve(**t, status=st)
        for name in ("positions", "group_indptr", "round_lens", "held_out", "slots"):
            t[name].fill_(5)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        check_reserve(t, int(st[0]), want)


def test_reserve_nothing():
    import torch
    p = plan_of(max_rows=4, max_groups=2, page_size=16, num_pages=4, max_pages=2)
    e = i32([])
    indptr, pos, q = i32([7]), i32([3, 3, 3]), torch.tensor([2, 5], dtype=torch.int64, device=dev())
    qo, st = torch.zeros_like(q), status_word()
    p.reserve(lens=e, counts=e, held=e, queue=q, free_pages=i32([0, 1, 2, 3]), block_tables=i32(np.zeros((0, 2))), group_indptr=indptr, round_lens=e,
              held_out=e, queue_out=qo, positions=pos, status=st)
    assert indptr.tolist() == [0] and pos.tolist() == [-1] * 3 and qo.tolist() == [2, 5] and int(st[0]) == 0


def test_reserve_through_rounds_of_requests_that_come_and_go():
    """Every page belongs to one request or to the queue, after every round."""
    import torch
    r = np.random.RandomState(11)
    groups, page, pages, width = 9, 8, 60, 12
    p = plan_of(max_rows=groups * 5, max_groups=groups, page_size=page, num_pages=pages, max_pages=width)
    lens, held = i32([-1] * groups), i32([0] * groups)
    tables = i32(np.full((groups, width), -1))
    queue, free = torch.tensor([0, pages], dtype=torch.int64, device=dev()), i32(np.arange(pages))
    indptr, round_lens = i32([0] * (groups + 1)), i32([0] * groups)
    pos, slots, st = i32([0] * (groups * 5)), torch.zeros(groups * 5, dtype=torch.int64, device=dev()), status_word()
    for _ in range(60):
        for g in range(groups):
            if r.rand() < 0.3:
                lens[g] = -1 if int(lens[g]) >= 0 else 0
        counts = r.randint(1, 6, groups)
        p.reserve(lens=lens, counts=i32(counts), held=held, queue=queue, free_pages=free, block_tables=tables, group_indptr=indptr,
                  round_lens=round_lens, held_out=held, queue_out=queue, positions=pos, slots=slots, status=st)
        h, (a, b) = held.tolist(), queue.tolist()
        owned = [int(tables[g, i]) for g in range(groups) for i in range(h[g])] + [int(free[i % pages]) for i in range(a, b)]
        assert sorted(owned) == list(range(pages))
        live = slots[slots >= 0].tolist()
        assert len(set(live)) == len(live) == sum(int(n) for g, n in enumerate(counts) if int(round_lens[g]) >= 0)
        grow = torch.minimum(round_lens + i32(r.randint(1, counts + 1)), i32([page * width - 6] * groups))
        lens = torch.where(round_lens >= 0, torch.maximum(grow, lens), lens)
    assert int(st[0]) & ~0x200 == 0


# ---- append


def four_caches(pages, hk, page, d, seed=0):
    """Codes and scales of random bytes: what a call must leave alone."""
    import torch
    g = generator(seed)
    b = lambda w: torch.randint(0, 256, (pages, hk, page, w), generator=g, device=dev(), dtype=torch.int32).to(torch.uint8)  # noqa: E731
    return b(d // 2), b(d // 2), b(d // 16), b(d // 16)


def test_quantise_reference_agrees_with_exact_arithmetic():
    import torch
    g = torch.Generator().manual_seed(0)
    for dtype in (torch.bfloat16, torch.float16):
        x = (torch.randn(60, 16, generator=g) * torch.exp(3 * torch.randn(60, 1, generator=g))).to(dtype)
        x[0] = 0.0
        x[1] = torch.tensor([6, 5, 3.5, 2.5, 1.75, 1.25, .75, .25, -5, -3.5, -2.5, -1.75, -1.25, -.75, -.25, -0.0])
        x[2] = x[1] * 3.5
        x[3] = 1e-6
        for f in (1.0, 0.25):
            codes, scales = K.quantise_rows(x, f)
            for i in range(60):
                c, s = K.quantise(x[i].tolist(), f)
                assert codes[i].tolist() == c and scales[i].tolist() == s, i


def append4(dtype, d, hq, hk, page, n, lens, *, factors=(1.0, 1.0), held=True, rope=True, k=None, v=None, seed=0):
    """lp_norm_rope and the reference's quantisation against lp_kv_append4: keys and values."""
    import torch
    gen = generator(len(n) + page + seed)
    indptr, tables, pages, _ = batch(n, lens, page, seed=page)
    rows = indptr[-1] + 2  # the last two rows belong to no group
    dt = R.DTYPE[dtype]
    both = rand(gen, rows, (hq + 2 * hk) * d, dtype=dtype)
    q = both[:, :hq * d].unflatten(1, (hq, d))
    k = both[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)) if k is None else k
    v = both[:, (hq + hk) * d:].unflatten(1, (hk, d)) if v is None else v
    pos = torch.randint(0, 500, (rows,), generator=gen, device=dev(), dtype=torch.int32)
    pos[-1] = -1
    more = dict(cos_sin=table(d, positions=500), k_weight=(1 + 0.3 * rand(gen, d, dtype=dtype)).to(dt)) if rope else {}
    caches = four_caches(pages, hk, page, d)
    kc, vc, ks, vs = (x.clone() for x in caches)
    full = lambda h: torch.full((rows, h, d), 7.0, dtype=dt, device=dev())  # noqa: E731
    ko, want_k, kh, vh, qo = full(hk), full(hk), full(hk), full(hk), full(hq)
    st = status_word()
    p = plan_of(max_rows=rows, max_groups=len(n), q_heads=hq, kv_heads=hk, head_dim=d, page_size=page, num_pages=pages,
                max_pages=tables.shape[1], dtype=dtype, kv_bits=4)
    p.norm_rope(k=k, k_out=want_k, positions=pos, status=st, **more)
    p.append4(q=q if rope else None, q_out=qo if rope else None, k=k, v=v, k_out=ko, positions=pos, group_indptr=i32(indptr), lens=i32(lens),
              block_tables=i32(tables), k_cache=kc, v_cache=vc, k_scales=ks.view(torch.float8_e4m3fn), v_scales=vs.view(torch.float8_e4m3fn),
              k_factor=factors[0], v_factor=factors[1], k_held=kh if held else None, v_held=vh if held else None, status=st, **more)
    torch.cuda.synchronize()
    assert int(st[0]) == 0
    assert torch.equal(ko, want_k) or bool(want_k.isnan().any())
    hit = torch.zeros(pages, page, dtype=torch.bool, device=dev())
    at, off, rowsof = [], [], []
    for g in range(len(n)):
        for j in range(n[g] if lens[g] >= 0 else 0):
            t = lens[g] + j
            rowsof.append(indptr[g] + j), at.append(int(tables[g, t // page])), off.append(t % page)
    hit[at, off] = True
    for x, codes, scales, h, f, was in ((want_k, kc, ks, kh, factors[0], (caches[0], caches[2])), (v, vc, vs, vh, factors[1], (caches[1], caches[3]))):
        want_codes, want_scales = K.quantise_rows(x, f)
        sound = want_scales != 0x7F
        assert torch.equal(scales[at, :, off], want_scales[rowsof])
        lanes = sound.repeat_interleave(K.BLOCK, -1)
        got = torch.where(lanes[rowsof], K.unpack(codes[at, :, off]), 255)
        assert torch.equal(got, want_codes[rowsof])
        for c, w in zip((codes, scales), was):  # every other slot is untouched
            assert torch.equal(c.transpose(1, 2)[~hit], w.transpose(1, 2)[~hit])
        if held:
            stands = K.values(K.pack(want_codes & 15), want_scales, f)
            assert torch.equal(torch.where(lanes, h.double(), 0.0)[:-1], torch.where(lanes, stands, 0.0)[:-1])
            assert bool(h[:-1][~lanes[:-1]].isnan().all()) and bool((h[-1] == 7.0).all())
    return kc, vc, ks, vs


@pytest.mark.parametrize("dtype,d,hq,hk,page,n,lens,held,rope", [
    ("bf16", 128, 32, 8, 16, [1], [1000], True, True),
    ("bf16", 128, 8, 8, 64, [4] * 9, [0, 5, 63, 64, 65, -1, 127, 200, 60], False, True),
    ("f16", 64, 6, 2, 8, [3, 0, 17, 1, 250], [5, 9, 7, -1, 3], True, False),
    ("f16", 128, 5, 1, 256, [300, 1, 1], [10, 255, 256], True, True),
    ("bf16", 64, 12, 4, 32, [2] * 300, [i % 71 - 1 for i in range(300)], True, False),
    ("bf16", 128, 24, 8, 64, [8200], [3], True, True),  # eight heads per task
])
def test_append4(dtype, d, hq, hk, page, n, lens, held, rope):
    append4(dtype, d, hq, hk, page, n, lens, held=held, rope=rope)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("factors", [(1.0, 1.0), (0.25, 2.0 ** -9), (64.0, 1024.0)])
def test_append4_ties_ranges_and_what_is_not_finite(dtype, factors):
    import torch
    rows, hk, d = 64, 2, 64
    gen = generator(5)
    x = rand(gen, rows + 2, 2 * hk, d, dtype=dtype).float()
    ties = torch.tensor([6, 5, 3.5, 2.5, 1.75, 1.25, .75, .25, -5, -3.5, -2.5, -1.75, -1.25, -.75, -.25, -0.0], device=dev())
    for i in range(16):  # every significand of a scale, at the ties of the codes and just beside them
        x[i] = (ties * (1 + i % 8 / 8) * 2.0 ** (i // 8 - 3)).repeat(d // 16)
    x[16:24] = x[0:8] * (1 + 2.0 ** -7)
    for m in range(8):   # ties of the scale itself: six times a number of five bits
        x[24 + m] = x[24 + m].clamp(-1, 1)
        x[24 + m, :, ::16] = 6 * (17 + 2 * m) / 16
    x[32] = 0.0
    x[33] = -0.0
    x[34], x[35] = 2.0 ** -14, 2.0 ** -24
    x[36] *= 2.0 ** 9
    x[37] *= 2.0 ** 15
    x[38, 0, 5], x[39, 1, 20], x[40, 3, 63] = float("nan"), float("inf"), float("-inf")
    if dtype == "bf16":
        x[41] *= 2.0 ** 120
        x[42] *= 2.0 ** -120
    x = x.to(R.DTYPE[dtype])
    held = dtype == "bf16" or factors[1] <= 1.0  # F16 holds no value of 2688 * 1024
    append4(dtype, d, hk, hk, 8, [rows], [0], factors=factors, rope=False, k=x[:, :hk], v=x[:, hk:], held=held and factors[0] <= 1.0)


def test_append4_malformed_groups_and_pages_write_nothing():
    import logprob_epilogue_gb300 as lpe
    import torch
    d, hk, page = 64, 2, 8
    caches = four_caches(4, hk, page, d)
    for indptr, lens, tables, bit in (
            ([0, 3], [14], [[0, 1]], lpe.STATUS_BAD_GROUP), ([0, 9], [0], [[0, 1]], lpe.STATUS_BAD_GROUP),
            ([0, 3], [0], [[4, 1]], lpe.STATUS_BAD_PAGE), ([0, 3], [0], [[-1, 1]], lpe.STATUS_BAD_PAGE), ([0, 3], [-1], [[0, 1]], 0)):
        kc, vc, ks, vs = (x.clone() for x in caches)
        x = rand(generator(0), 3, hk, d, dtype="bf16")
        st = status_word()
        plan_of(max_rows=3, head_dim=d, page_size=page, num_pages=4, max_pages=2, kv_bits=4).append4(
            k=x, v=x, positions=i32([0, 1, 2]), group_indptr=i32(indptr), lens=i32(lens), block_tables=i32(tables), k_cache=kc, v_cache=vc,
            k_scales=ks.view(torch.float8_e4m3fn), v_scales=vs.view(torch.float8_e4m3fn), status=st)
        assert int(st[0]) == bit
        for a, b in zip((kc, vc, ks, vs), caches):
            assert torch.equal(a, b)


def test_append4_twice_and_captured_is_the_same():
    import torch
    n, lens = [4] * 20, [i * 3 for i in range(20)]
    indptr, tables, pages, _ = batch(n, lens, 16, seed=1)
    kc, vc, ks, vs = four_caches(pages, 2, 16, 128)
    k, v = (rand(generator(i), 80, 2, 128, dtype="bf16") for i in (1, 2))
    st = status_word()
    p = plan_of(max_rows=80, max_groups=20, num_pages=pages, max_pages=tables.shape[1], kv_bits=4)
    call = lambda: p.append4(k=k, v=v, positions=pos, group_indptr=ptr, lens=ln, block_tables=tb, k_cache=kc, v_cache=vc,  # noqa: E731
                             k_scales=ks.view(torch.float8_e4m3fn), v_scales=vs.view(torch.float8_e4m3fn), status=st)
    pos, ptr, ln, tb = i32(range(80)), i32(indptr), i32(lens), i32(tables)
    call()
    torch.cuda.synchronize()
    first = [x.clone() for x in (kc, vc, ks, vs)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for x in (kc, vc, ks, vs):
        x.random_(0, 256)
    keep = [x.clone() for x in (kc, vc, ks, vs)]
    graph.replay()
    torch.cuda.synchronize()
    at = [int(tables[g, (lens[g] + j) // 16]) for g in range(20) for j in range(4)]
    off = [(lens[g] + j) % 16 for g in range(20) for j in range(4)]
    for x, f, w in zip((kc, vc, ks, vs), first, keep):
        assert torch.equal(x[at, :, off], f[at, :, off])
        w[at, :, off] = f[at, :, off]
        assert torch.equal(x, w)
