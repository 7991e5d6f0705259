"""Attention over a cache in 4 bits by each of its two kernels: groups of at most 32 (row, head) pairs take fragments,
larger ones query tiles; prefixes likewise by the rows behind them."""
import math

import numpy as np
import pytest

import attn_ref as R
import kv4_ref as K
from test_gpu_attn import EDGES, batch, dev, generator, i32, plan_of, rand, status_word, table
from test_gpu_kv4 import Case4, append4, both_reserve, four_caches, reserve_inputs

pytestmark = pytest.mark.gpu


def restate(c, k_factor, v_factor):
    """What the same codes stand for under other factors."""
    c.factors = (k_factor, v_factor)
    c.kc, c.vc = (K.values(x, s, f) for x, s, f in zip(c.codes, c.scales, c.factors))


def close(out, lse, ref, dtype, rows=slice(None)):
    """Results against 64 bits, with the probabilities' own rounding beside the output's.

    Both kernels round a probability to F16 after a power of two that brings a row's largest to 2^6 or more: by 2^-11 of it, or,
    below F16's normal numbers, by 2^-25, which is 2^-31 of the largest.  Where the results are divided by the sum of the rounded
    ones, sum p (1 + d) v / sum p (1 + d) differs from o = sum p v by sum p d (v - o) / (1 + d'): 2^-11 (sum p |v| + |o|) and a
    2^-10th of that.  Scores are off as they are for attend (see attn_ref)."""
    o, want_lse, mag, bound, count, vmax = (x[rows] for x in ref)
    tol = R.U[dtype] * o.abs() + (2.0 ** -11 + 2.0 ** -20 + 2 * bound + 2.0 ** -18)[..., None] * (mag + o.abs())
    tol = tol + (2.0 ** -30 * count * vmax)[..., None] + R.STEP[dtype]
    err = (out[rows].double() - o).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), int((~(err <= tol)).sum()))
    none = want_lse == -math.inf
    assert bool((out[rows][none] == 0).all())
    if lse is not None:
        got = lse[rows].double()
        assert bool((got[none] == -math.inf).all())
        off = (got - want_lse).abs()[~none]
        assert bool((off <= (bound + 2.0 ** -18)[~none]).all()), float(off.max())


def check(c, ref=None, **more):
    out, lse, st = c.run(**more)
    assert st == 0, hex(st)
    close(out, lse, ref or c.ref(), c.dtype, slice(0, c.indptr[-1]))
    return out, lse


@pytest.mark.parametrize("dtype,d", [("f16", 128), ("f16", 64), ("bf16", 128)])
@pytest.mark.parametrize("n,hq", [([2, 3], 4), ([12, 20], 8)])  # fragments; query tiles (more than 32 pairs a group)
@pytest.mark.parametrize("scale,factor", [(2.0 ** -100, 2.0 ** -100), (2.0 ** -149, 1.0), (2.0 ** -3, 2.0 ** -149)])
def test_attend4_scores_whose_factor_vanishes(dtype, d, n, hq, scale, factor):
    """scale * k_factor below FP32's range: every score is 0 to within the bound, and tokens past a length stay out."""
    c = Case4(dtype=dtype, d=d, hq=hq, hk=1, n=n, lens=[40, 300], prefixes=[70])
    c.scale = scale
    restate(c, factor, 1.0)
    check(c)


@pytest.mark.parametrize("dtype,d", [("f16", 128), ("f16", 64), ("bf16", 128)])
@pytest.mark.parametrize("n,hq", [([2, 3], 4), ([12, 20], 8)])
def test_attend4_scores_of_zero_under_a_factor_past_the_range(dtype, d, n, hq):
    """scale * k_factor past FP32's range: a score of 0 is 0."""
    import torch
    c = Case4(dtype=dtype, d=d, hq=hq, hk=1, n=n, lens=[40, 300], prefixes=[70])
    c.q = torch.zeros_like(c.q)
    c.scale = 2.0 ** 80
    restate(c, 2.0 ** 80, 1.0)
    check(c)


@pytest.mark.parametrize("n,hq", [([2, 3], 4), ([12, 20], 8)])
@pytest.mark.parametrize("size,scale,factor", [
    (2.0 ** -105, 2.0 ** 40, 2.0 ** 62), (2.0 ** -128, 2.0 ** 70, 2.0 ** 58), (2.0 ** -110, 1.75 * 2.0 ** 127, 2.0 ** -20),
    (2.0 ** 100, 2.0 ** -60, 2.0 ** -43), (2.0 ** 100, 2.0 ** 20, 2.0 ** -123),
])
def test_attend4_factors_that_bring_one_another_back(size, scale, factor, n, hq):
    """BF16 queries far from 1 under a scale and a factor that bring their scores back, whatever the products on the way."""
    c = Case4(hq=hq, hk=1, n=n, lens=[40, 300], prefixes=[70])
    c.q = (c.q.float() * size).bfloat16()
    c.scale = scale
    restate(c, factor, 1.0)
    check(c)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64)])
@pytest.mark.parametrize("n,hq", [([2], 4), ([12], 8)])
@pytest.mark.parametrize("factor", [2.0 ** -126, 2.0 ** -128, 2.0 ** -131, 2.0 ** 116])
def test_attend4_values_under_a_factor_at_the_ends_of_the_range(dtype, d, n, hq, factor):
    """Values of 2,688 factor, which BF16 holds: the factor alone, divided by the sum of 5,000 probabilities, would leave FP32's normal numbers."""
    import torch
    c = Case4(dtype=dtype, d=d, hq=hq, hk=1, n=n, lens=[5001])
    c.raw[1][~c.raw[1].isnan()] = 2688.0
    c.quantise()
    restate(c, 1.0, factor)
    out, _ = check(c)
    assert torch.equal(out.double(), torch.full_like(out, 2688.0 * factor).double())


@pytest.mark.parametrize("dtype,d,bits", [("bf16", 128, 4), ("f16", 128, 4), ("f16", 64, 4), ("f16", 128, 16), ("bf16", 128, 16)])
@pytest.mark.parametrize("n,hq", [([2, 3, 1], 4), ([12, 20, 9], 8)])
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 15, 2.0 ** 18])
def test_scores_far_from_zero(dtype, d, bits, n, hq, size):
    """Scores to 2^22, where neighbouring FP32 numbers lie whole units apart: a row whose largest score is far above its others
    takes that token's value."""
    import torch
    from test_gpu_attn import Case
    c = (Case4 if bits == 4 else Case)(dtype=dtype, d=d, hq=hq, hk=1, n=n, lens=[40, 700, 0], prefixes=[70], prefix_indptr=[0, 2])
    c.scale *= size
    p = 2.0 ** -11 if bits == 4 else R.U[dtype]  # the probability's rounding; its FP32 sum is off by 2^-18 and the join's
    out, lse, st = c.run()
    assert st == 0 and bool(out.isfinite().all()) and bool(lse.isfinite().all())
    clear = 0
    for g in range(len(n)):
        pre = 70 if g < 2 else 0
        k, v = ([R.gather(x, c.prefix_tables[0], pre, 0, c.page)] if pre else [] for x in (c.kc, c.vc))
        k, v = (torch.cat(x + [R.gather(y, c.tables[g], c.lens[g] + n[g], 0, c.page)]) for x, y in ((k, c.kc), (v, c.vc)))
        for j in range(n[g]):
            row, see = c.indptr[g] + j, pre + c.lens[g] + j + 1
            s = c.scale * c.q[row].double() @ k[:see].T
            off = 2 * d * 2.0 ** -24 * c.scale * (c.q[row].double().abs() @ k[:see].abs().T).amax(-1) + 2.0 ** -21 * s.abs().amax(-1)
            top, at = s.max(-1)
            assert bool(((lse[row].double() - top).abs() <= off + math.log(see)).all())
            rest = s.scatter(1, at[:, None], -math.inf).amax(-1)
            alone = top - rest > 2 * off + 40
            clear += int(alone.sum())
            err = (out[row].double() - v[at]).abs()
            assert bool((err[alone] <= (R.U[dtype] + p + 2.0 ** -17) * v[at][alone].abs() + R.STEP[dtype] + 2.0 ** -40).all())
    assert clear > 0.9 * sum(n) * hq


# The tests below take their calls through query tiles: groups of more than 32 pairs on average.
TILES = dict(n=[12, 20], hq=8, hk=1)


@pytest.mark.parametrize("dtype,d,hq,hk,page,rows", [
    ("bf16", 128, 4, 1, 16, 1), ("bf16", 64, 16, 2, 256, 1), ("bf16", 128, 16, 2, 8, 7), ("bf16", 64, 12, 1, 64, 5), ("f16", 128, 10, 2, 128, 9),
    ("f16", 64, 128, 1, 32, 3),
])
def test_attend4_within_the_probabilities_own_rounding(dtype, d, hq, hk, page, rows):
    """Every length about a page's and a tile's end."""
    check(Case4(dtype=dtype, d=d, hq=hq, hk=hk, page=page, n=[rows + i % 5 for i in range(len(EDGES))], lens=EDGES, prefixes=[333],
                prefix_indptr=[0, 9]))


@pytest.mark.parametrize("factors", [(2.0 ** -8, 2.0 ** 5), (3.0, 0.7), (2.0 ** 20, 2.0 ** -20)])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64)])
def test_attend4_factors_of_query_tiles(dtype, d, factors):
    c = Case4(dtype=dtype, d=d, lens=[300, 40], prefixes=[150], **TILES)
    restate(c, *factors)
    if dtype == "f16" and factors[1] > 1:  # within F16
        c.factors, c.vc = (factors[0], 1.0), K.values(c.codes[1], c.scales[1], 1.0)
    c.scale /= factors[0]
    check(c)


def test_attend4_idle_and_malformed_groups_of_many_rows():
    import logprob_epilogue_gb300 as lpe
    kw = dict(n=[12, 13, 20, 9], lens=[20, -1, 140, -7], prefixes=[30], hq=8, hk=1)
    c = Case4(**kw)
    ref = c.ref()
    out, lse = check(c, ref=ref)
    starts = c.indptr
    group = lambda g: slice(starts[g], starts[g + 1])  # noqa: E731
    nothing = lambda o, x, g: bool((o[group(g)] == 0).all()) and bool((x[group(g)] == -math.inf).all())  # noqa: E731
    assert nothing(out, lse, 1) and nothing(out, lse, 3)
    good, good_lse, _ = c.run()
    out, lse, st = c.run(lens=i32([20, -1, c.tables.shape[1] * c.page - 1, -7]))  # more tokens than the table holds
    assert st == lpe.STATUS_BAD_GROUP and nothing(out, lse, 2)
    close(out, lse, ref, c.dtype, group(0))
    small = Case4(max_group_rows=12, **kw)
    out, lse, st = small.run()
    assert st == lpe.STATUS_BAD_GROUP and nothing(out, lse, 2)
    close(out, lse, ref, c.dtype, group(0))
    for indptr in ([0, 12, 25, 45, 55], [-2, 12, 25, 45, 54], [0, 25, 12, 45, 54], [0, 12, 25, 2147483647, 54]):
        _, _, st = c.run(group_indptr=i32(indptr))
        assert st & lpe.STATUS_BAD_GROUP, indptr
    alone = R.attend(c.q, c.kc, c.vc, c.indptr, c.lens, c.tables, scale=c.scale)
    for bad in (dict(prefix_indptr=i32([0, 5])), dict(prefix_indptr=i32([3, 2])), dict(prefix_indptr=i32([-1, 4])),
                dict(prefix_lens=i32([-1])), dict(prefix_lens=i32([c.prefix_tables.shape[1] * c.page + 1]))):
        out, lse, st = c.run(**bad)
        assert st == lpe.STATUS_BAD_PREFIX, bad
        close(out, lse, alone, c.dtype, slice(0, c.rows))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attend4_what_is_not_finite_stays_with_the_rows_of_a_query_tile_that_see_it(dtype):
    import torch
    c = Case4(dtype=dtype, lens=[200, 129], **TILES)
    clean, clean_lse = check(c)
    t = 200 + 11  # the last draft of group 0: only row 11 sees it
    page, off = int(c.tables[0, t // c.page]), t % c.page
    for scales in c.scales:
        keep = scales[page, :, off].clone()
        scales[page, :, off] = 0x7F
        out, lse, st = c.run()
        scales[page, :, off] = keep
        rows = [r for r in range(32) if r != 11]
        assert st == 0 and torch.equal(out[rows], clean[rows]) and torch.equal(lse[rows], clean_lse[rows])
        assert not bool(out[11].isfinite().all())
    for token in (60, 199):  # committed tokens of group 0: its rows, and no others
        page, off = int(c.tables[0, token // c.page]), token % c.page
        for scales in c.scales:
            keep = scales[page, :, off].clone()
            scales[page, :, off] = 0xFF
            out, lse, st = c.run()
            scales[page, :, off] = keep
            assert st == 0 and torch.equal(out[12:], clean[12:]) and not bool(out[:12].isfinite().all(-1).any())
    for bad in (math.nan, math.inf):  # a query that is not finite: its head of its row
        keep = c.q[1, 2, 7].clone()
        c.q[1, 2, 7] = bad
        out, lse, st = c.run()
        c.q[1, 2, 7] = keep
        rest = torch.ones(c.rows, c.hq, dtype=torch.bool, device=dev())
        rest[1, 2] = False
        assert st == 0 and torch.equal(out[rest], clean[rest]) and torch.equal(lse[rest], clean_lse[rest])
        assert not bool(out[1, 2].isfinite().all())


@pytest.mark.parametrize("size", [2.0 ** -120, 2.0 ** -30, 2.0 ** 20, 2.0 ** 100])
@pytest.mark.parametrize("n", [[5, 9], [20, 32]])  # units of one tile, and of two
def test_attend4_queries_of_any_size_in_query_tiles(size, n):
    c = Case4(n=n, hq=16, hk=1, lens=[200, 40], prefixes=[20])
    c.q = (c.q.float() * size).bfloat16()
    c.q[0, 0, 3] = 2.0 ** -100 * size if size > 1 else 0.0
    c.q[2] = 0.0
    c.q[3] *= 2.0 ** -9  # rows of a tile with factors of their own
    c.scale /= size
    check(c)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("n", [[12, 9], [32, 20]])
def test_attend4_extreme_scores_in_query_tiles(dtype, d, n):
    """Scores of magnitude 1e3, rising and falling along the context: the running maximum moves often."""
    import torch
    c = Case4(dtype=dtype, d=d, n=n, lens=[900, 513], hq=8, hk=1, width=0.0)
    c.q = torch.full_like(c.q, 8.0)
    t = torch.arange(932, device=dev())
    for g, count in ((0, 900 + n[0]), (1, 513 + n[1])):
        at, off = torch.from_numpy(c.tables[g]).to(dev())[t[:count] // c.page], t[:count] % c.page
        ramp = (t[:count].float() - 300.0) * (1 if g == 0 else -1) / 64.0
        c.raw[0][at, :, off] = ramp[:, None, None].expand(count, 1, d).to(c.raw[0].dtype)
    c.quantise()
    check(c)


def test_attend4_offsets_past_32_bits_in_query_tiles():
    """Codes past 2^32 bytes, the batch in the cache's last pages."""
    import torch
    if torch.cuda.get_device_properties(0).total_memory < 60e9:
        pytest.skip("needs a large card")
    pages, hk, page = 70_000, 4, 256
    c = Case4(n=[10, 30], lens=[300, 77], hq=32, hk=hk, page=page, prefixes=[200])
    big = [torch.zeros(pages, hk, page, x.shape[-1], dtype=torch.uint8, device=dev()) for x in (*c.codes, *c.scales)]
    for x, y in zip(big, (*c.codes, *c.scales)):
        x[pages - c.pages:] = y
    up = lambda tab: i32(np.where(tab >= 0, tab + pages - c.pages, -1))  # noqa: E731
    e4m3 = torch.float8_e4m3fn
    assert big[0].numel() > 2 ** 32
    plan = plan_of(max_rows=40, max_groups=2, max_group_rows=32, q_heads=32, kv_heads=hk, page_size=page, num_pages=pages, max_pages=c.tables.shape[1],
                   max_prefixes=1, max_prefix_pages=c.prefix_tables.shape[1], kv_bits=4)
    check(c, plan=plan, k_cache=big[0], v_cache=big[1], k_scales=big[2].view(e4m3), v_scales=big[3].view(e4m3), block_tables=up(c.tables),
          prefix_tables=up(c.prefix_tables))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attend4_strides_streams_and_graphs_of_query_tiles(dtype):
    import torch
    c = Case4(dtype=dtype, n=[14, 20, 9], lens=[100, 333, 0], prefixes=[150], hq=8, hk=1)
    ref = c.ref()
    wide = torch.zeros(c.rows, (c.hq + 3) * c.d, dtype=c.q.dtype, device=dev())
    wide[:, c.d:(c.hq + 1) * c.d] = c.q.flatten(1)
    outs = torch.full((c.rows, (c.hq + 1) * c.d), 7.0, dtype=c.q.dtype, device=dev())
    out = outs[:, :c.hq * c.d].unflatten(1, (c.hq, c.d))
    plan, st, t = c.plan(), status_word(), c.tensors()
    t["q"] = wide[:, c.d:(c.hq + 1) * c.d].unflatten(1, (c.hq, c.d))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan.attend4(**t, out=out, status=st, stream=side)
    side.synchronize()
    close(out, None, ref, c.dtype)
    assert bool((outs[:, c.hq * c.d:] == 7.0).all())
    lse = torch.zeros(c.rows, c.hq, device=dev())
    t["q"] = c.q
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.attend4(**t, out=out, lse_out=lse, status=st)
    for lens, pre in (([100, 333, 0], 150), ([3, -1, 0], 7), ([0, 0, 0], 0), ([100, 12, 0], 129)):  # captured once, replayed on new lengths
        t["lens"].copy_(i32(lens)), t["prefix_lens"].copy_(i32([pre]))
        c.lens, c.prefix_lens = lens, [pre]
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
        close(out, lse, c.ref(), c.dtype)
    assert int(st[0]) == 0


# Which kernel takes a call's prefixes and which its groups: 32 pairs for each of them, on average.
MIXED = {
    "prefixes in tiles, groups in fragments": dict(n=[2] * 9, hq=8, hk=1, lens=[40, 0, 300, -1, 129, 7, 64, 1, 500], prefixes=[333]),
    "groups in tiles, prefixes in fragments": dict(n=[16], hq=4, hk=1, lens=[300], prefixes=[200, 5, 7], prefix_indptr=[0, 1, 1, 1]),
    "both in tiles": dict(n=[12, 20], hq=8, hk=1, lens=[40, 300], prefixes=[150]),
    "both in fragments": dict(n=[1, 3], hq=4, hk=1, lens=[40, 300], prefixes=[150]),
}


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("kernels", MIXED)
def test_attend4_kernels_side_by_side(dtype, d, kernels):
    """Each pair of kernels in one call: results, pages out of range in either kind of table, and waits that run out."""
    import torch
    import logprob_epilogue_gb300 as lpe
    c = Case4(dtype=dtype, d=d, fill=0.0, pad_rows=3, **MIXED[kernels])
    good, good_lse = check(c)
    rows = c.indptr[-1]
    for tables, name, last in ((c.tables, "block_tables", 300 // c.page if len(c.n) < 9 else 299 // c.page), (c.prefix_tables, "prefix_tables", 0)):
        g = {"block_tables": c.lens.index(300), "prefix_tables": 0}[name]
        for i in {0, last}:
            for bad in (-1, c.pages, 2147483647):
                tab = tables.copy()
                tab[g, i] = bad
                out, lse, st = c.run(**{name: i32(tab)})
                assert st == lpe.STATUS_BAD_PAGE
                kc, vc = c.kc.clone(), c.vc.clone()
                kc[int(tables[g, i])] = 0
                vc[int(tables[g, i])] = 0
                ref = R.attend(c.q, kc, vc, c.indptr, c.lens, c.tables, scale=c.scale, prefix_indptr=c.prefix_indptr, prefix_lens=c.prefix_lens,
                               prefix_tables=c.prefix_tables)
                close(out, lse, ref, c.dtype, slice(0, rows))
    plan = c.plan(debug_force_timeout=True, timeout_ns=2_000_000)
    for _ in range(2):
        out, lse, st = c.run(plan)
        assert st == lpe.STATUS_TIMEOUT
        assert bool((out[:rows] == 0).all()) and bool((lse[:rows] == -math.inf).all())
        assert bool((out[rows:] == 7.0).all()) and bool((lse[rows:] == 7.0).all())
    plan.close()
    out, lse, st = c.run()
    assert st == 0 and torch.equal(out[:rows], good[:rows]) and torch.equal(lse[:rows], good_lse[:rows])


def test_attend4_one_plan_through_every_pair_of_kernels():
    """The parts and tables that a call leaves mean nothing to the next one, whichever kernels it takes."""
    import torch
    cases = [Case4(hq=8, hk=2, n=n, lens=lens, prefixes=prefixes, prefix_indptr=ptr, seed=i, max_group_rows=32) for i, (n, lens, prefixes, ptr) in enumerate([
        ([2] * 9, [40, 0, 300, -1, 129, 7, 64, 1, 500], [333], [0, 9]), ([32], [900], [200, 5, 7], [0, 1, 1, 1]), ([12, 20], [40, 300], [150], [0, 2]),
        ([1, 3], [40, 300], [150], [0, 2]), ([1] * 31 + [32], [5] * 31 + [700], [], None)])]
    pages = max(c.pages for c in cases)
    plans = [c.plan() for c in cases]
    first = [c.run(p) for c, p in zip(cases, plans)]
    for c, (out, lse, st) in zip(cases, first):
        assert st == 0
        close(out, lse, c.ref(), c.dtype, slice(0, c.indptr[-1]))
    width, pwidth = max(c.tables.shape[1] for c in cases), max(c.prefix_tables.shape[1] for c in cases)
    one = plan_of(max_rows=max(c.rows for c in cases), max_groups=max(len(c.n) for c in cases), max_group_rows=32, q_heads=8, kv_heads=2, page_size=16,
                  num_pages=pages, max_pages=width, max_prefixes=3, max_prefix_pages=pwidth, kv_bits=4)
    pad = lambda tab, w: i32(np.pad(tab, ((0, 0), (0, w - tab.shape[1])), constant_values=-1))  # noqa: E731

    def again(c):
        t = {}
        for name, x in (("k_cache", c.codes[0]), ("v_cache", c.codes[1]), ("k_scales", c.scales[0]), ("v_scales", c.scales[1])):
            y = torch.zeros(pages, *x.shape[1:], dtype=torch.uint8, device=dev())
            y[:c.pages] = x
            t[name] = y.view(torch.float8_e4m3fn) if "scales" in name else y
        if c.prefix_lens:
            t["prefix_tables"] = pad(c.prefix_tables, pwidth)
        return c.run(one, block_tables=pad(c.tables, width), **t)

    for i in (0, 1, 2, 3, 4, 1, 0, 3, 2, 4, 0):
        out, lse, st = again(cases[i])
        assert st == 0 and torch.equal(out, first[i][0]) and torch.equal(lse, first[i][1]), i


def test_attend4_a_large_group_among_single_rows():
    """One group of 256 pairs at a long context beside 60 of eight: one kernel for all, whichever, and padding rows that count for neither."""
    n, lens = [32] + [1] * 60, [2500] + [17 * i % 200 for i in range(60)]
    for pad in (0, 400):  # as many rows as make the average 32 pairs
        check(Case4(n=n, lens=lens, hq=8, hk=1, pad_rows=pad))


# ---- append and reserve


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rope", [False, True])
def test_append4_keys_out_beside_what_is_not_finite(dtype, rope):
    """k_out is norm_rope's, lane for lane, in heads with a NaN or an infinity too."""
    import torch
    d, hk, page, rows = 64, 2, 8, 24
    gen = generator(9)
    k, v, q = (rand(gen, rows, h, d, dtype=dtype) for h in (hk, hk, 4))
    for row, lane, x in ((3, 0, math.nan), (5, 63, math.inf), (7, 17, -math.inf)):
        k[row, row % hk, lane] = v[row, row % hk, lane] = x
    indptr, tables, pages, _ = batch([rows], [5], page, seed=2)
    more = dict(cos_sin=table(d), k_weight=(1 + 0.1 * rand(gen, d, dtype=dtype)).to(R.DTYPE[dtype])) if rope else {}
    pos, st = i32(range(rows)), status_word()
    p = plan_of(max_rows=rows, head_dim=d, page_size=page, num_pages=pages, max_pages=tables.shape[1], dtype=dtype, kv_bits=4)
    want, got, qo = torch.empty_like(k), torch.empty_like(k), torch.empty_like(q)
    p.norm_rope(k=k, k_out=want, positions=pos, status=st, **more)
    kc, vc, ks, vs = four_caches(pages, hk, page, d)
    e4m3 = torch.float8_e4m3fn
    p.append4(q=q, q_out=qo, k=k, v=v, k_out=got, positions=pos, group_indptr=i32(indptr), lens=i32([5]), block_tables=i32(tables), k_cache=kc, v_cache=vc,
              k_scales=ks.view(e4m3), v_scales=vs.view(e4m3), status=st, **more)
    torch.cuda.synchronize()
    assert int(st[0]) == 0 and bool(want.isnan().any())
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got[~want.isnan()], want[~want.isnan()])


@pytest.mark.parametrize("dtype,hk,n,held", [("bf16", 8, [9001], True), ("f16", 3, [20_000, 1, 4100], False), ("bf16", 9, [8000], True), ("f16", 12, [5999], False)])
def test_append4_many_keys_without_queries(dtype, hk, n, held):
    """Eight heads per task and four, at counts of heads that are multiples of neither."""
    append4(dtype, 128, hk, hk, 64, n, [3] * len(n), held=held, rope=False)


@pytest.mark.parametrize("groups", [3, 1200])
def test_reserve_long_requests_that_leave_and_come(groups):
    """Thousands of pages given back by one group and taken by another, in one block and across all."""
    page, long = 8, 40_003
    lens, counts = [5] * groups, [1] * groups
    lens[0], lens[-1], counts[1] = -1, -1, long
    x = reserve_inputs(counts, lens, page, seed=groups, ring_extra=12_000)
    width = max(x["tables"].shape[1], 6000)
    tables = np.full((groups, width), -1, np.int64)
    tables[:, :x["tables"].shape[1]] = x["tables"]
    for g, held in ((0, 5001), (groups - 1, 1023)):  # more pages than the random ones
        tables[g, :held] = x["pages"] + np.arange(held)
        x["held"][g], x["pages"] = held, x["pages"] + held
    x["tables"] = tables
    both_reserve(x, page, sum(counts) + 3)
    both_reserve(x, page, sum(counts), inplace=True)


@pytest.mark.parametrize("groups,rows", [(256, 2048), (257, 2048), (256, 2049), (1, 2048), (1, 2049), (257, 257)])
def test_reserve_about_where_a_second_kernel_begins(groups, rows):
    r = np.random.RandomState(groups + rows)
    counts = np.bincount(r.randint(0, groups, rows), minlength=groups).tolist()
    lens = r.randint(-1 if groups > 1 else 0, 99, groups).tolist()
    both_reserve(reserve_inputs(counts, lens, 16, seed=rows), 16, rows)
    both_reserve(reserve_inputs(counts, lens, 16, seed=rows, free=rows // 40), 16, rows, inplace=True)


def example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "verify_rounds.py")
    spec = importlib.util.spec_from_file_location("verify_rounds", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("free", [0, 1, 3, 4, 5])
def test_rounds_whose_pages_run_out(free):
    """A request without pages keeps its length and emits nothing; the others' lengths stay within the pages that they hold."""
    e = example()
    page, drafts, rounds = 16, 3, 24
    emitted, accepted, lens = e.decode(e.Target(), list(range(3, 40)), [5, 6, 7], rounds=rounds, drafts=drafts, page=page, idle=1, kv_bits=4, free=free)
    held, want, left = [0, 0, 0], [0, 0, 0], free
    for a in accepted:
        short = False  # groups in order; from the first that the rest does not cover, those that lack pages get none
        for g in range(3):
            lack = -(-(want[g] + drafts + 1) // page) - held[g]
            short |= lack > left
            served = lack == 0 or not short
            assert (a[g] >= 0) == served, (a, g)
            if served:
                held[g], left, want[g] = held[g] + lack, left - lack, want[g] + a[g] + 1
    assert lens == want + [-1] and any(-1 in a for a in accepted)
    assert [len(x) for x in emitted] == [1 + n for n in want]
