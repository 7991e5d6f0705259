"""CPU checks of the entries around a cache in 4 bits, and what the host refuses."""
import ctypes
import os
import subprocess

import pytest

import logprob_epilogue_gb300 as lpe
from logprob_epilogue_gb300 import attn as A
from logprob_epilogue_gb300 import build as B
from test_attn_abi import BASE, EALIGN, EINVAL, ESHAPE

ESTATE = -7
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    B.build()
    return lpe.lib()


def test_null_arguments_and_descriptors(L):
    for f in (L.lp_kv_reserve, L.lp_kv_append4, L.lp_attend4):
        assert f(None, None, None) == EINVAL
    assert A.attn_scratch_bytes(**BASE, kv_bits=4) > A.attn_scratch_bytes(**BASE) > 0  # parts of either kernel
    with pytest.raises(ValueError, match="kv_bits"):
        A.make_attn_desc(**BASE, kv_bits=8)
    d = A.make_attn_desc(**BASE)
    d.flags = 0x800
    assert L.lp_attn_scratch_bytes(ctypes.byref(d)) == 0


def test_struct_sizes_match_the_header(L, tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "lp_epilogue.h"\nint main(void) { printf("%zu %zu %zu %zu %zu %d %d\\n", '
                   "sizeof(lp_reserve_io), sizeof(lp_append4_io), sizeof(lp_attend4_io), offsetof(lp_append4_io, k_factor), "
                   "offsetof(lp_attend4_io, k_scales), (int)LP_ATTN_KV4, (int)LP_STATUS_NO_PAGES); return 0; }\n")
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    structs = (A.ReserveIO, A.Append4IO, A.Attend4IO)
    assert got[:3] == [ctypes.sizeof(t) for t in structs] == [s.size for s in (A._PACK_RESERVE, A._PACK_APPEND4, A._PACK_ATTEND4)]
    assert got[3:] == [A.Append4IO.k_factor.offset, A.Attend4IO.k_scales.offset, lpe.ATTN_KV4, lpe.STATUS_NO_PAGES]


def test_packed_fields_land_where_the_structs_have_them():
    """Every field of the io structures, set by one native pack."""
    n = len(A._PACK_RESERVE.unpack(bytes(A._PACK_RESERVE.size)))
    io = A.ReserveIO.from_buffer_copy(A._PACK_RESERVE.pack(*range(1, n + 1)))
    assert [getattr(io, f) for f, _ in io._fields_] == list(range(1, n + 1))
    for pack, struct, inner in ((A._PACK_APPEND4, A.Append4IO, A._PACK_APPEND), (A._PACK_ATTEND4, A.Attend4IO, A._PACK_ATTEND)):
        n, m = (len(p.unpack(bytes(p.size))) for p in (pack, inner))
        io = struct.from_buffer_copy(pack.pack(*range(1, n + 1)))
        assert [getattr(io, f) for f, _ in io._fields_[1:]] == list(range(m + 1, n + 1))
        assert bytes(getattr(io, io._fields_[0][0])) == inner.pack(*range(1, m + 1))


@pytest.mark.gpu
class TestRefusals:
    """Argument errors of the three calls (a plan needs a device)."""

    def plan(self, **kw):
        return lpe.AttnPlan(**{**BASE, **dict(max_prefixes=1, max_prefix_pages=2, kv_bits=4), **kw})

    def append(self, **kw):
        io = A.Append4IO()
        a, r, at = io.append, io.append.rope, 1 << 20  # never followed: refused first
        r.k = r.positions = r.status = a.v = a.group_indptr = a.lens = a.block_tables = a.k_cache = a.v_cache = io.k_scales = io.v_scales = at
        r.k_stride = a.v_stride = 2 * 128
        r.eps, r.max_positions, r.rows, a.groups, io.k_factor, io.v_factor = 1e-6, 10, 4, 2, 1.0, 1.0
        for k, v in kw.items():
            setattr(next(x for x in (io, a, r) if hasattr(x, k)), k, v)
        return io

    def attend(self, **kw):
        io = A.Attend4IO()
        a = io.attend
        for n in ("q", "k_cache", "v_cache", "group_indptr", "lens", "block_tables", "prefix_indptr", "prefix_lens", "prefix_tables", "out", "status"):
            setattr(a, n, 1 << 20)
        io.k_scales = io.v_scales = 1 << 20
        a.q_stride = a.out_stride = 8 * 128
        a.scale, a.rows, a.groups, a.prefixes, io.k_factor, io.v_factor = 0.1, 4, 2, 1, 1.0, 1.0
        for k, v in kw.items():
            setattr(io if hasattr(io, k) else a, k, v)
        return io

    @pytest.mark.parametrize("kw,code", [
        (dict(k_factor=0.0), EINVAL), (dict(k_factor=3.0), EINVAL), (dict(v_factor=-2.0), EINVAL), (dict(v_factor=float("nan")), EINVAL),
        (dict(v_factor=2.0 ** 61), EINVAL), (dict(k_factor=2.0 ** -61), EINVAL), (dict(k_scales=None), EINVAL), (dict(v_scales=(1 << 20) + 8), EALIGN),
        (dict(k_cache=(1 << 20) + 8), EALIGN), (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(rows=65), ESHAPE), (dict(groups=9), ESHAPE),
        (dict(k_held=1 << 20, k_held_stride=128), ESHAPE), (dict(v_held=(1 << 20) + 2, v_held_stride=256), EALIGN),
        (dict(v_held=1 << 20, v_held_stride=260), EALIGN), (dict(status=None), EINVAL), (dict(positions=None), EINVAL),
    ])
    def test_append4(self, kw, code):
        p = self.plan()
        assert lpe.lib().lp_kv_append4(p._h, ctypes.byref(self.append(**kw)), None) == code

    @pytest.mark.parametrize("kw,code", [
        (dict(k_factor=0.0), EINVAL), (dict(v_factor=float("inf")), EINVAL), (dict(v_factor=-1.0), EINVAL), (dict(k_scales=None), EINVAL),
        (dict(v_scales=(1 << 20) + 4), EALIGN), (dict(rows=65), ESHAPE), (dict(prefixes=2), ESHAPE), (dict(scale=0.0), EINVAL), (dict(q=None), EINVAL),
        (dict(prefix_lens=None), EINVAL), (dict(q_stride=512), ESHAPE), (dict(out_stride=1028), EALIGN), (dict(status=None), EINVAL),
    ])
    def test_attend4(self, kw, code):
        p = self.plan()
        assert lpe.lib().lp_attend4(p._h, ctypes.byref(self.attend(**kw)), None) == code

    def test_a_plan_has_one_kind_of_cache(self):
        four, half = self.plan(), self.plan(kv_bits=16)
        L = lpe.lib()
        assert L.lp_kv_append(four._h, ctypes.byref(self.append().append), None) == ESTATE
        assert L.lp_attend(four._h, ctypes.byref(self.attend().attend), None) == ESTATE
        assert L.lp_kv_append4(half._h, ctypes.byref(self.append()), None) == ESTATE
        assert L.lp_attend4(half._h, ctypes.byref(self.attend()), None) == ESTATE

    @pytest.mark.parametrize("kw,code", [
        (dict(rows=65), ESHAPE), (dict(rows=-1), ESHAPE), (dict(groups=9), ESHAPE), (dict(ring=0), ESHAPE), (dict(queue=None), EINVAL),
        (dict(queue_out=None), EINVAL), (dict(group_indptr=None), EINVAL), (dict(lens=None), EINVAL), (dict(counts=None), EINVAL), (dict(held=None), EINVAL),
        (dict(held_out=None), EINVAL), (dict(round_lens=None), EINVAL), (dict(round_lens=1 << 20), EINVAL), (dict(positions=None), EINVAL),
        (dict(free_pages=None), EINVAL), (dict(block_tables=None), EINVAL), (dict(status=None), EINVAL), (dict(queue=(1 << 20) + 4), EALIGN),
        (dict(slots=(1 << 20) + 4), EALIGN), (dict(counts=(1 << 20) + 2), EALIGN), (dict(starts=(1 << 20) + 1), EALIGN),
    ])
    def test_reserve(self, kw, code):
        io = A.ReserveIO()
        for n, _ in io._fields_[:14]:
            setattr(io, n, 1 << 20)
        io.round_lens, io.rows, io.groups, io.ring = 2 << 20, 4, 2, 10
        for k, v in kw.items():
            setattr(io, k, v)
        assert lpe.lib().lp_kv_reserve(self.plan()._h, ctypes.byref(io), None) == code

    def test_python_checks(self):
        import torch
        p = self.plan()
        dev = torch.device("cuda", 0)
        z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device=dev)  # noqa: E731
        i = lambda *s: z(*s, dtype=torch.int32)  # noqa: E731
        e4m3 = torch.float8_e4m3fn
        caches = dict(k_cache=z(100, 2, 16, 64, dtype=torch.uint8), v_cache=z(100, 2, 16, 64, dtype=torch.uint8),
                      k_scales=z(100, 2, 16, 8, dtype=e4m3), v_scales=z(100, 2, 16, 8, dtype=e4m3))
        batch = dict(caches, group_indptr=torch.tensor([0, 4], dtype=torch.int32, device=dev), lens=i(1), block_tables=i(1, 10), status=i(1))
        k = z(4, 2, 128)
        append = dict(batch, k=k, v=k, positions=i(4), k_held=torch.empty_like(k))
        attend = dict(batch, q=z(4, 8, 128), out=z(4, 8, 128))
        p.append4(**append)
        p.attend4(**attend)
        wrong = [dict(k_cache=caches["k_cache"][..., :32]), dict(v_cache=caches["v_cache"].float()), dict(k_scales=caches["k_scales"].view(torch.uint8)),
                 dict(v_scales=caches["v_scales"][:50]), dict(group_indptr=None), dict(status=None), dict(block_tables=i(1, 9)), dict(lens=i(1).long())]
        for kw in wrong + [dict(v=None), dict(k=k[:3]), dict(k_held=k[:3]), dict(v_held=k.float()), dict(positions=i(3))]:
            with pytest.raises((ValueError, AttributeError)):
                p.append4(**{**append, **kw})
        for kw in wrong + [dict(q=None), dict(out=None), dict(q=k), dict(lse_out=z(4, 8)), dict(prefix_lens=i(1))]:
            with pytest.raises((ValueError, lpe.LPError)):
                p.attend4(**{**attend, **kw})
        long = lambda *s: z(*s, dtype=torch.int64)  # noqa: E731
        reserve = dict(lens=i(1), counts=i(1), held=i(1), queue=long(2), free_pages=i(5), block_tables=i(1, 10), group_indptr=i(2), round_lens=i(1),
                       held_out=i(1), queue_out=long(2), positions=i(4), slots=long(4), status=i(1))
        p.reserve(**reserve)
        for kw in (dict(queue=i(2)), dict(slots=i(4)), dict(slots=long(3)), dict(positions=None), dict(free_pages=None), dict(lens=None), dict(group_indptr=None),
                   dict(block_tables=i(1, 9)), dict(counts=i(0)), dict(held=i(1).cpu()), dict(status=None)):
            with pytest.raises(ValueError):
                p.reserve(**{**reserve, **kw})
        torch.cuda.synchronize()
