"""The operators around a cache in 4 bits on the GPU: reservation of a round's
pages, append, attention."""
import numpy as np
import pytest

import attn_ref as R
import kv4_ref as K
from test_gpu_attn import EDGES, Case, batch, dev, generator, i32, plan_of, rand, status_word, table

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


# ---- attention
#
# The bounds are those of attend (see attn_ref), whose terms cover this kernel's: a query is exact in F16 after its power of two
# (a lane under 2^-28 of the row's largest is off by 2^-39 of that), a code times its scale is exact, and a probability is
# rounded to F16, 2^-11 of it or 2^-31 of the largest.


class Case4(Case):
    """A Case over a cache in 4 bits: its keys and values quantised, with NaN scales in slots that nothing owns."""

    def __init__(self, factors=(1.0, 1.0), **kw):
        super().__init__(**kw)
        self.factors = factors
        self.raw = [self.kc, self.vc]
        self.quantise()

    def quantise(self, seed=3):
        """Codes and scales of the raw caches; kc and vc become what these stand for, in 64 bits."""
        import torch
        self.codes, self.scales, stand = [], [], []
        for raw, f in zip(self.raw, self.factors):
            codes, scales = K.quantise_rows(raw, f)
            junk = torch.randint(0, 16, codes.shape, generator=generator(seed), device=dev(), dtype=torch.int32).to(torch.uint8)
            codes = K.pack(torch.where(codes == 255, junk, codes))
            self.codes.append(codes), self.scales.append(scales), stand.append(K.values(codes, scales, f))
        self.kc, self.vc = stand

    def plan(self, **kw):
        return super().plan(kv_bits=4, **kw)

    def tensors(self):
        import torch
        t = super().tensors()
        t.update(k_cache=self.codes[0], v_cache=self.codes[1], k_scales=self.scales[0].view(torch.float8_e4m3fn),
                 v_scales=self.scales[1].view(torch.float8_e4m3fn), k_factor=self.factors[0], v_factor=self.factors[1])
        return t

    def run(self, plan=None, stream=None, **more):
        import torch
        out = torch.full((self.rows, self.hq, self.d), 7.0, dtype=R.DTYPE[self.dtype], device=dev())
        lse = torch.full((self.rows, self.hq), 7.0, device=dev())
        st = status_word()
        plan = plan or self.plan()
        plan.attend4(**{**self.tensors(), **more}, out=out, lse_out=lse, status=st, stream=stream)
        torch.cuda.synchronize()
        return out, lse, int(st[0])


@pytest.mark.parametrize("dtype,d,hq,hk,page", [
    ("bf16", 128, 4, 1, 16), ("f16", 64, 6, 2, 8), ("bf16", 64, 2, 2, 256), ("f16", 128, 12, 1, 64), ("bf16", 128, 10, 2, 128),
    ("f16", 128, 5, 1, 32), ("bf16", 64, 128, 1, 64), ("bf16", 128, 8, 1, 8),
])
def test_attend4_lengths(dtype, d, hq, hk, page):
    """Every length about a page's and a tile's end, groups of one to five rows, unused slots NaN."""
    n = [1 + i % 5 for i in range(len(EDGES))]
    Case4(dtype=dtype, d=d, hq=hq, hk=hk, page=page, n=n, lens=EDGES, pad_rows=2).check()


@pytest.mark.parametrize("prefix", [1, 7, 64, 127, 128, 129, 300, 1025])
@pytest.mark.parametrize("dtype,d,hq,hk,page,n,lens", [
    ("bf16", 128, 4, 1, 16, [1], [0]),
    ("bf16", 128, 8, 2, 64, [4] * 11, [0, 1, 2, 130, 5, 64, 9, 31, 256, 77, 3]),
    ("f16", 64, 3, 3, 32, [32, 1, 9, 31, 32], [5, 0, 700, 1, 128]),
    ("f16", 128, 24, 2, 8, [16, 16, 16], [1, 0, 140]),
])
def test_attend4_shared_prefix(prefix, dtype, d, hq, hk, page, n, lens):
    Case4(dtype=dtype, d=d, hq=hq, hk=hk, page=page, n=n, lens=lens, prefixes=[prefix]).check()


@pytest.mark.parametrize("hq,n", [(1, 1), (1, 15), (4, 4), (1, 17), (8, 4), (3, 11), (4, 12), (3, 21), (4, 16), (5, 13), (12, 8), (5, 25), (8, 16), (12, 32)])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64)])
def test_attend4_query_rows(dtype, d, hq, n):
    """From one (row, head) pair of a group to three units of them, about every number of fragments; one token tile, two and several."""
    Case4(dtype=dtype, d=d, hq=hq, hk=1, n=[n] * 4, lens=[1, 129, 700, 300], page=32).check()


@pytest.mark.parametrize("factors", [(2.0 ** -8, 2.0 ** 5), (3.0, 0.7), (2.0 ** 20, 2.0 ** -20)])
def test_attend4_factors(factors):
    c = Case4(n=[2, 3], lens=[300, 40], prefixes=[150])
    c.factors = factors  # what the same codes stand for under others
    c.kc, c.vc = (K.values(x, s, f) for x, s, f in zip(c.codes, c.scales, factors))
    c.scale /= factors[0]
    c.check()


def test_attend4_several_prefixes_and_groups_without_one():
    n = [2, 3, 1, 4, 1, 1, 5, 2, 2]
    lens = [10, 0, 300, 5, -1, 129, 0, 64, 1]
    Case4(n=n, lens=lens, prefixes=[200, 5, 400], prefix_indptr=[1, 3, 3, 8], hq=6, hk=3).check()
    Case4(n=n, lens=lens, prefixes=[200, 0], prefix_indptr=[0, 4, 9], hq=6, hk=3, dtype="f16", d=64).check()


def test_attend4_many_rows_behind_a_prefix():
    n = [1 + i % 8 for i in range(66)]
    lens = [(37 * i) % 150 - 1 for i in range(66)]
    Case4(n=n, lens=lens, prefixes=[517], hq=10, hk=2).check()
    Case4(n=n, lens=lens, prefixes=[517], hq=10, hk=2, d=64, dtype="f16", page=64).check()


def test_attend4_more_units_than_blocks():
    n = [20, 31, 7, 32, 32, 28, 12]
    Case4(n=n, lens=[0, 140, -1, 3, 0, 128, 9], prefixes=[260, 129], prefix_indptr=[0, 5, 7], hq=32 * 12, hk=32, d=64).check()
    Case4(n=n, lens=[0, 140, -1, 3, 0, 128, 9], prefixes=[140], hq=16 * 40, hk=16, dtype="f16").check()


def test_attend4_trees_and_empty_rows():
    r = np.random.RandomState(0)
    n, lens = [7, 32, 1, 16, 3], [0, 50, 0, 131, 0]
    masks = []
    for m in n:
        rows = [1]
        for j in range(1, m):
            rows.append(rows[r.randint(j)] | 1 << j)
        masks += rows
    masks[3] = 0                 # no context, no row: nothing to see
    masks[39] = 0                # a single row that does not see itself
    masks[8] = 0xFFFFFFFF        # rows after its own, too
    masks[-1] = 0xFFFFFFF8       # bits past the group's rows name nothing
    c = Case4(n=n, lens=lens, masks=masks)
    out, lse = c.check()
    for row in (3, 39, c.rows - 1):
        assert bool((out[row] == 0).all()) and bool((lse[row] == -np.inf).all())
    Case4(n=n, lens=lens, masks=masks, prefixes=[33], d=64).check()


def test_attend4_idle_and_malformed_groups():
    import logprob_epilogue_gb300 as lpe
    c = Case4(n=[2, 3, 2, 1], lens=[20, -1, 40, -7], prefixes=[30])
    out, lse = c.check()
    assert bool((out[2:5] == 0).all()) and bool((lse[2:5] == -np.inf).all())
    ref = c.ref()
    good = list(range(0, 2)) + [7]
    out, lse, st = c.run(lens=i32([20, -1, c.tables.shape[1] * c.page - 1, -7]))  # more tokens than the table holds
    assert st == lpe.STATUS_BAD_GROUP
    assert bool((out[5:7] == 0).all()) and bool((lse[5:7] == -np.inf).all())
    R.check_attend(out, lse, ref, c.dtype, good)
    small = Case4(n=[2, 3, 2, 1], lens=[20, -1, 40, -7], prefixes=[30], max_group_rows=2)
    out, lse, st = small.run(lens=i32([20, 3, 40, -7]))
    assert st == lpe.STATUS_BAD_GROUP and bool((out[2:5] == 0).all())
    R.check_attend(out, lse, ref, c.dtype, good)
    for indptr in ([0, 2, 5, 7, 9], [-2, 2, 5, 7, 8], [0, 5, 2, 7, 8], [0, 2, 5, 2147483647, 8]):
        _, _, st = c.run(group_indptr=i32(indptr))
        assert st & lpe.STATUS_BAD_GROUP, indptr
    alone = R.attend(c.q, c.kc, c.vc, c.indptr, c.lens, c.tables, scale=c.scale)
    for bad in (dict(prefix_indptr=i32([0, 5])), dict(prefix_indptr=i32([3, 2])), dict(prefix_indptr=i32([-1, 4])),
                dict(prefix_lens=i32([-1])), dict(prefix_lens=i32([c.prefix_tables.shape[1] * c.page + 1]))):
        out, lse, st = c.run(**bad)
        assert st == lpe.STATUS_BAD_PREFIX, bad
        R.check_attend(out, lse, alone, c.dtype, slice(0, c.rows))


@pytest.mark.parametrize("page", [16, 256])
def test_attend4_pages_out_of_range_read_as_zeros(page):
    import logprob_epilogue_gb300 as lpe
    c = Case4(n=[1, 2], lens=[40, 300], page=page, fill=0.0)
    at = 300 // page
    for i in {0, at}:
        for bad in (-1, -2147483648, c.pages, 2147483647):
            tab = c.tables.copy()
            tab[1, i] = bad
            out, lse, st = c.run(block_tables=i32(tab))
            assert st == lpe.STATUS_BAD_PAGE
            kc, vc = c.kc.clone(), c.vc.clone()
            kc[int(c.tables[1, i])] = 0
            vc[int(c.tables[1, i])] = 0
            R.check_attend(out, lse, R.attend(c.q, kc, vc, c.indptr, c.lens, c.tables, scale=c.scale), c.dtype)


def test_attend4_what_is_not_finite_stays_with_the_rows_that_see_it():
    import torch
    c = Case4(n=[4, 4], lens=[200, 129], hq=4, hk=2)
    clean, clean_lse = c.check()
    t = 203  # the last draft of group 0: only row 3 sees it
    page, off = int(c.tables[0, t // c.page]), t % c.page
    for scales in c.scales:
        keep = scales[page, :, off].clone()
        scales[page, :, off] = 0x7F
        out, lse, st = c.run()
        scales[page, :, off] = keep
        rows = [0, 1, 2, 4, 5, 6, 7]
        assert st == 0 and torch.equal(out[rows], clean[rows]) and torch.equal(lse[rows], clean_lse[rows])
        assert not bool(out[3].isfinite().all())
    # a committed token of group 0: its rows, and no others
    page, off = int(c.tables[0, 60 // c.page]), 60 % c.page
    for scales in c.scales:
        keep = scales[page, :, off].clone()
        scales[page, :, off] = 0xFF
        out, lse, st = c.run()
        scales[page, :, off] = keep
        assert st == 0 and torch.equal(out[4:], clean[4:]) and not bool(out[:4].isfinite().all(-1).any())
    # a query that is not finite: its head of its row
    for bad in (float("nan"), float("inf")):
        keep = c.q[1, 2, 7].clone()
        c.q[1, 2, 7] = bad
        out, lse, st = c.run()
        c.q[1, 2, 7] = keep
        rest = torch.ones(c.rows, c.hq, dtype=torch.bool, device=dev())
        rest[1, 2] = False
        assert st == 0 and torch.equal(out[rest], clean[rest]) and torch.equal(lse[rest], clean_lse[rest])
        assert not bool(out[1, 2].isfinite().all())


@pytest.mark.parametrize("size", [2.0 ** -120, 2.0 ** -30, 2.0 ** 20, 2.0 ** 100])
def test_attend4_queries_of_any_size(size):
    """BF16 queries far outside F16's range, with a scale that brings their scores back."""
    c = Case4(n=[3, 2], lens=[200, 40], prefixes=[20])
    c.q = (c.q.float() * size).bfloat16()
    c.q[0, 0, 3] = 2.0 ** -100 * size if size > 1 else 0.0
    c.q[2] = 0.0
    c.scale /= size
    c.check()


def test_attend4_extreme_scores():
    """Scores of magnitude 1e3, rising and falling along the context: the running maximum moves often."""
    import torch
    c = Case4(n=[3, 1], lens=[900, 513], hq=4, hk=1, width=0.0)
    c.q = torch.full_like(c.q, 8.0)
    t = torch.arange(903, device=dev())
    for g, count in ((0, 903), (1, 514)):
        at, off = torch.from_numpy(c.tables[g]).to(dev())[t[:count] // c.page], t[:count] % c.page
        ramp = (t[:count].float() - 300.0) * (1 if g == 0 else -1) / 64.0
        c.raw[0][at, :, off] = ramp[:, None, None].expand(count, 1, 128).to(c.raw[0].dtype)
    c.quantise()
    c.check()


def test_attend4_offsets_past_32_bits():
    """Codes past 2^32 bytes, the batch in the cache's last pages."""
    import torch
    if torch.cuda.get_device_properties(0).total_memory < 60e9:
        pytest.skip("needs a large card")
    pages, hk, page, d = 70_000, 4, 256, 128
    small = Case4(n=[1, 3], lens=[300, 77], hq=4, hk=hk, page=page, prefixes=[200])
    big = [torch.zeros(pages, hk, page, x.shape[-1], dtype=torch.uint8, device=dev()) for x in (*small.codes, *small.scales)]
    for x, y in zip(big, (*small.codes, *small.scales)):
        x[pages - small.pages:] = y
    up = lambda tab: i32(np.where(tab >= 0, tab + pages - small.pages, -1))  # noqa: E731
    e4m3 = torch.float8_e4m3fn
    assert big[0].numel() > 2 ** 32
    plan = plan_of(max_rows=4, max_groups=2, q_heads=4, kv_heads=hk, page_size=page, num_pages=pages, max_pages=small.tables.shape[1], max_prefixes=1,
                   max_prefix_pages=small.prefix_tables.shape[1], kv_bits=4)
    moved = dict(k_cache=big[0], v_cache=big[1], k_scales=big[2].view(e4m3), v_scales=big[3].view(e4m3), block_tables=up(small.tables))
    out, lse, st = small.run(plan, **moved, prefix_tables=up(small.prefix_tables))
    assert st == 0
    R.check_attend(out, lse, small.ref(), small.dtype)
    # and the append that reaches them
    k, v = (rand(generator(5), 4, hk, d, dtype="bf16") for _ in range(2))
    st = status_word()
    plan.append4(k=k, v=v, positions=i32([0] * 4), group_indptr=i32(small.indptr), lens=i32(small.lens), status=st, **moved)
    t = small.lens[1] + 2
    at = int(small.tables[1, t // page]) + pages - small.pages
    for x, codes, scales in ((k, big[0], big[2]), (v, big[1], big[3])):
        want = K.quantise_rows(x[-1])
        assert torch.equal(codes[at, :, t % page], K.pack(want[0])) and torch.equal(scales[at, :, t % page], want[1])


def test_attend4_strided_tensors_other_streams_and_graphs():
    import torch
    c = Case4(n=[4, 2, 1], lens=[100, 333, 0], prefixes=[150])
    ref = c.ref()
    wide = torch.zeros(c.rows, (c.hq + 3) * c.d, dtype=c.q.dtype, device=dev())
    wide[:, c.d:(c.hq + 1) * c.d] = c.q.flatten(1)
    q = wide[:, c.d:(c.hq + 1) * c.d].unflatten(1, (c.hq, c.d))
    outs = torch.full((c.rows, (c.hq + 1) * c.d), 7.0, dtype=c.q.dtype, device=dev())
    out = outs[:, :c.hq * c.d].unflatten(1, (c.hq, c.d))
    plan, st, t = c.plan(), status_word(), c.tensors()
    t["q"] = q
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan.attend4(**t, out=out, status=st, stream=side)
    side.synchronize()
    R.check_attend(out, None, ref, c.dtype)
    assert bool((outs[:, c.hq * c.d:] == 7.0).all())
    # captured once, replayed on new lengths
    lse = torch.zeros(c.rows, c.hq, device=dev())
    t["q"] = c.q
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.attend4(**t, out=out, lse_out=lse, status=st)
    for lens in ([100, 333, 0], [3, -1, 0], [0, 0, 0], [100, 12, 0]):
        t["lens"].copy_(i32(lens))
        c.lens = lens
        for g, l in enumerate(lens):
            for j in range(c.n[g] if l >= 0 else 0):
                at, off = int(c.tables[g, (l + j) // c.page]), (l + j) % c.page
                c.raw[0][at, :, off], c.raw[1][at, :, off] = 0.25 * (j + 1), 0.5 * j
        was = [*c.codes, *c.scales]
        c.quantise()
        for x, y in zip(was, (*c.codes, *c.scales)):  # the tensors that the graph reads
            x.copy_(y)
        c.codes, c.scales = was[:2], was[2:]
        graph.replay()
        torch.cuda.synchronize()
        R.check_attend(out, lse, c.ref(), c.dtype)
    assert int(st[0]) == 0


def test_attend4_repeats_bit_for_bit_after_other_calls():
    import torch
    a = Case4(n=[4] * 30, lens=[(97 * i) % 500 for i in range(30)], prefixes=[700])
    plan = a.plan()
    first = a.run(plan)
    for lens in ([0] * 30, [-1] * 29 + [3], [min(l, 31 * i % 300) for i, l in enumerate(a.lens)]):  # within the groups' pages
        out, lse, st = a.run(plan, lens=i32(lens), prefix_lens=i32([lens[-1]]))
        assert st == 0
    again = a.run(plan)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_attend4_zero_rows_and_zero_groups():
    import torch
    c = Case4(n=[1], lens=[5])
    plan = c.plan()
    empty = torch.empty(0, c.hq, c.d, dtype=c.q.dtype, device=dev())
    t = c.tensors()
    t["q"] = empty
    t["group_indptr"], t["lens"], t["block_tables"] = i32([0]), i32([]), i32(np.zeros((0, c.tables.shape[1])))
    plan.attend4(**t, out=empty, status=status_word())
    t["q"] = c.q
    out = torch.full_like(c.q, 7.0)
    plan.attend4(**t, out=out, status=status_word())
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())


def test_a_call_of_attend4_that_gave_up_gives_zeros():
    """Waits that run out: the status, 0 and -inf for every row of a group, and the next plan gets the right result."""
    import time
    import torch
    import logprob_epilogue_gb300 as lpe
    for c in (Case4(n=[2, 3], lens=[300, 40], prefixes=[150], pad_rows=2), Case4(n=[1], lens=[5000], hq=8, hk=1, d=64, dtype="f16")):
        good, good_lse, st = c.run()
        assert st == 0
        rows = c.indptr[-1]
        plan = c.plan(debug_force_timeout=True, timeout_ns=2_000_000)
        for _ in range(2):
            began = time.perf_counter()
            out, lse, st = c.run(plan)
            assert time.perf_counter() - began < 5.0
            assert st == lpe.STATUS_TIMEOUT
            assert bool((out[:rows] == 0).all()) and bool((lse[:rows] == -np.inf).all())
            assert bool((out[rows:] == 7.0).all()) and bool((lse[rows:] == 7.0).all())
        plan.close()
        out, lse, st = c.run()
        assert st == 0 and torch.equal(out[:rows], good[:rows]) and torch.equal(lse[:rows], good_lse[:rows])


# ---- a round


def test_rounds_of_reserve_append4_attend4_commit():
    """Rounds of requests that come, grow and leave: pages reserved, keys and values appended, attention, commit."""
    import torch
    gen = generator(11)
    hq, hk, d, page, groups, rows_g, width = 8, 2, 128, 16, 6, 4, 9
    rows, pages = groups * rows_g, 45
    plan = plan_of(max_rows=rows, max_groups=groups, q_heads=hq, kv_heads=hk, head_dim=d, page_size=page, num_pages=pages,
                   max_pages=width, max_group_rows=rows_g, max_prefixes=1, max_prefix_pages=5, kv_bits=4)
    order = np.random.RandomState(1).permutation(pages)
    ptab, free = order[:5].reshape(1, 5), i32(order[5:])
    kc, vc, ks, vs = four_caches(pages, hk, page, d)
    e4m3 = torch.float8_e4m3fn
    ks, vs = (x.bitwise_and(0x37).view(e4m3) for x in (ks, vs))  # finite, as the prefix's are
    lens, held, tables = i32([0, 0, 0, 0, 0, -1]), i32([0] * groups), i32(np.full((groups, width), -1))
    queue, st, cs = torch.tensor([0, pages - 5], dtype=torch.int64, device=dev()), status_word(), table(d)
    indptr, round_lens, pos = i32([0] * (groups + 1)), i32([0] * groups), i32([0] * rows)
    caches = dict(k_cache=kc, v_cache=vc, k_scales=ks, v_scales=vs)
    for step in range(7):
        counts = i32([(g + step) % rows_g + 1 for g in range(groups)])
        qkv = rand(gen, rows, (hq + 2 * hk) * d, dtype="bf16")
        q, k, v = (qkv[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, hq), (hq, hq + hk), (hq + hk, hq + 2 * hk)))
        qo, out = (torch.full((rows, hq, d), 7.0, dtype=torch.bfloat16, device=dev()) for _ in range(2))
        lse, kh = torch.empty(rows, hq, device=dev()), torch.full((rows, hk, d), 7.0, dtype=torch.bfloat16, device=dev())
        plan.reserve(lens=lens, counts=counts, held=held, queue=queue, free_pages=free, block_tables=tables, group_indptr=indptr,
                     round_lens=round_lens, held_out=held, queue_out=queue, positions=pos, starts=i32([70] * groups), status=st)
        batch_of = dict(group_indptr=indptr, lens=round_lens, block_tables=tables, status=st, **caches)
        plan.append4(q=q, k=k, v=v, q_out=qo, cos_sin=cs, positions=pos, k_held=kh, **batch_of)
        plan.attend4(q=qo, out=out, lse_out=lse, prefix_indptr=i32([0, groups]), prefix_lens=i32([70]), prefix_tables=i32(ptab), **batch_of)
        ref = R.attend(qo, K.values(kc, ks), K.values(vc, vs), indptr.tolist(), round_lens.tolist(), tables.cpu().numpy(), scale=d ** -0.5,
                       prefix_indptr=[0, groups], prefix_lens=[70], prefix_tables=ptab)
        n = int(indptr[-1])
        R.check_attend(out, lse, ref, "bf16", slice(0, n))
        assert bool((out[n:] == 7.0).all()) and bool((kh[n:] == 7.0).all()) and bool((pos[n:] == -1).all())
        # the appended keys are the rotated ones, in 4 bits
        g = 3
        row, t = int(indptr[g]), int(lens[g])
        if int(round_lens[g]) >= 0:
            at = K.values(kc, ks)[int(tables[g, t // page]), :, t % page]
            assert torch.equal(kh[row].double(), at) and int(pos[row]) == 70 + t
        accepted = torch.minimum(counts, i32([1, 4, 2, 3, 1, 2]))
        lens = torch.where(round_lens >= 0, lens + accepted, lens).int()
        if step == 3:
            lens[1], lens[5] = -1, 0  # one leaves, one comes
    assert int(st[0]) == 0


def test_the_example_decodes_over_a_cache_in_4_bits():
    """It runs, every request grows by what was accepted, and free slots stay free."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "verify_rounds.py")
    spec = importlib.util.spec_from_file_location("verify_rounds", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    target, prompt, firsts = example.Target(), list(range(3, 40)), [5, 6, 7]
    for idle in (0, 1, 5):
        emitted, accepted, lens = example.decode(target, prompt, firsts, rounds=8, idle=idle, kv_bits=4)
        assert lens == [sum(a[g] + 1 for a in accepted) for g in range(3)] + [-1] * idle
        assert all(len(e) == 1 + n for e, n in zip(emitted, lens))


@pytest.mark.parametrize("groups", [900, 5000])
def test_reserve_rows_among_groups_without_any(groups):
    """Long runs of groups without rows before, between and after those that have some: neighbouring rows lie thousands of groups apart."""
    r = np.random.RandomState(groups)
    counts = np.zeros(groups, np.int64)
    some = np.sort(r.choice(groups, 40, replace=False))
    counts[some] = r.randint(1, 3, 40)
    counts[some[7]] = 90
    counts[some[8]] = 33
    lens = r.randint(0, 30, groups)
    lens[r.choice(groups, groups // 3, replace=False)] = -1
    counts, lens = counts.tolist(), lens.tolist()
    both_reserve(reserve_inputs(counts, lens, 8, seed=5), 8, sum(counts) + 37)


def test_reserve_largest_counts_and_holdings_side_by_side():
    """Warps full of groups with the largest counts: their sums pass 32 bits, what follows sits out and what is before them does not."""
    groups, first = 2100, 1030
    counts, lens = [1] * first + [2 ** 31 - 1] * 70 + [2] * (groups - first - 70), [3 + g % 9 for g in range(groups)]
    x = reserve_inputs([1] * groups, lens, 8, seed=1, extra=1)
    x["counts"] = counts
    both_reserve(x, 8, first + 100)
    x["held"][5] = x["held"][1200] = x["tables"].shape[1]
    x["lens"][5] = x["lens"][1200] = -1  # idle groups with full tables
    x["tables"][5] = x["tables"][1200] = np.arange(x["tables"].shape[1])
    both_reserve(x, 8, first + 100)


@pytest.mark.parametrize("dtype,d,hq", [("bf16", 64, 2), ("f16", 128, 2), ("bf16", 128, 3), ("f16", 64, 4)])
def test_attend4_units_of_one_and_two_fragments_side_by_side(dtype, d, hq):
    """Blocks that go through several units, of 16 rows and fewer and of more, whole ones and cut ones."""
    r = np.random.RandomState(d + hq)
    groups = 330
    n, lens = r.randint(1, 32 // hq, groups).tolist(), r.randint(-1, 300, groups)
    n[0] = 32 // hq
    lens[r.choice(groups, 6, replace=False)] = r.randint(1000, 2500, 6)
    Case4(dtype=dtype, d=d, hq=hq, hk=1, page=32, n=n, lens=lens.tolist()).check()


@pytest.mark.parametrize("page", [16, 256])
def test_attend4_pages_out_of_range_of_groups_of_many_rows(page):
    """The same zeros where a group's rows take query tiles."""
    import logprob_epilogue_gb300 as lpe
    c = Case4(n=[12, 20], lens=[40, 300], page=page, fill=0.0, hq=8, hk=1)
    at = 300 // page
    for i in {0, at}:
        for bad in (-1, c.pages, 2147483647):
            tab = c.tables.copy()
            tab[1, i] = bad
            out, lse, st = c.run(block_tables=i32(tab))
            assert st == lpe.STATUS_BAD_PAGE
            kc, vc = c.kc.clone(), c.vc.clone()
            kc[int(c.tables[1, i])] = 0
            vc[int(c.tables[1, i])] = 0
            R.check_attend(out, lse, R.attend(c.q, kc, vc, c.indptr, c.lens, c.tables, scale=c.scale), c.dtype)
