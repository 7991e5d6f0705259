"""CPU checks of the attention entries: what the host refuses before any CUDA call."""
import ctypes

import pytest

import logprob_epilogue_gb300 as lpe
from logprob_epilogue_gb300 import attn as A
from logprob_epilogue_gb300 import build as B

EINVAL, ESHAPE, EALIGN, ECAPACITY, EDTYPE, ECUDA = -1, -2, -3, -4, -5, -6


@pytest.fixture(scope="module")
def L():
    B.build()
    return lpe.lib()


BASE = dict(max_rows=64, max_groups=8, q_heads=8, kv_heads=2, head_dim=128, page_size=16, num_pages=100, max_pages=10)


@pytest.mark.parametrize("kw,code", [
    (dict(max_rows=0), ESHAPE), (dict(max_groups=0), ESHAPE), (dict(max_pages=0), ESHAPE), (dict(num_pages=0), ESHAPE),
    (dict(q_heads=7), ESHAPE), (dict(kv_heads=0), ESHAPE), (dict(q_heads=1), ESHAPE), (dict(head_dim=96), ESHAPE),
    (dict(page_size=24), ESHAPE), (dict(page_size=4), ESHAPE), (dict(page_size=512), ESHAPE),
    (dict(max_prefixes=1), ESHAPE), (dict(max_prefixes=-1), ESHAPE),
    (dict(max_group_rows=0), ECAPACITY), (dict(max_group_rows=33), ECAPACITY), (dict(q_heads=516, kv_heads=4), ECAPACITY),
    (dict(num_pages=1 << 31), ECAPACITY), (dict(max_pages=1 << 27), ECAPACITY),
    (dict(dtype="f32"), EDTYPE), (dict(timeout_ns=-1), EINVAL),
])
def test_create_refuses(L, kw, code):
    d = A.make_attn_desc(**{**BASE, **kw})
    h = ctypes.c_void_p()
    assert L.lp_attn_create(ctypes.byref(h), ctypes.byref(d)) == code
    assert not h.value
    assert L.lp_attn_scratch_bytes(ctypes.byref(d)) == 0


def test_scratch_bytes_and_null_arguments(L):
    assert A.attn_scratch_bytes(**BASE) > 0
    assert L.lp_attn_create(None, None) == EINVAL
    assert L.lp_attn_destroy(None) == EINVAL
    assert L.lp_norm_rope(None, None, None) == EINVAL
    assert L.lp_kv_append(None, None, None) == EINVAL
    assert L.lp_attend(None, None, None) == EINVAL


def test_struct_sizes_match_the_header(L, tmp_path):
    import os
    import subprocess
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "lp_epilogue.h"\nint main(void) { printf("%zu %zu %zu %zu\\n", '
                   "sizeof(lp_attn_desc), sizeof(lp_rope_io), sizeof(lp_append_io), sizeof(lp_attend_io)); return 0; }\n")
    exe = tmp_path / "s"
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    sizes = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert sizes == [ctypes.sizeof(t) for t in (A.AttnDesc, A.RopeIO, A.AppendIO, A.AttendIO)]
    assert sizes[1:] == [s.size for s in (A._PACK_ROPE, A._PACK_APPEND, A._PACK_ATTEND)]


def test_a_table_entry_names_only_parts_that_exist(tmp_path):
    """What the join takes from an entry (a unit's first slot and its pieces), whatever the entry holds: no pieces, or at most
    one per block, in slots of the region."""
    import os
    import subprocess
    src = tmp_path / "e.cpp"
    src.write_text('#include <cstdio>\n#include "lp_attn.h"\nint main() { int s, n, g; long long slots;\n'
                   '    while (std::scanf("%d %d %lld %d", &s, &n, &slots, &g) == 4) std::printf("%d\\n", lp::entry_pieces(s, n, slots, g)); }\n')
    exe = tmp_path / "e"
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    cuda = os.path.dirname(os.path.dirname(B._nvcc()))
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(root, "logprob_epilogue_gb300", "csrc"), "-I", os.path.join(cuda, "include"),
                    str(src), "-o", str(exe)], check=True)
    slots, grid = 1000, 152
    words = [0, 1, 2, 151, 152, 153, 847, 848, 849, 998, 999, 1000, 1001, 0x3F800000, 0x7FFFFFFF, -1, -2, -0x80000000]
    cases = [(s, n) for s in words for n in words]
    text = "".join(f"{s} {n} {slots} {grid}\n" for s, n in cases)
    got = [int(x) for x in subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split()]
    assert got == [n if 1 <= n <= grid and 0 <= s and s + n <= slots else 0 for s, n in cases]


@pytest.mark.gpu
class TestRefusals:
    """Argument errors of the three calls (a plan needs a device)."""

    def plan(self):
        return lpe.AttnPlan(**BASE, max_prefixes=1, max_prefix_pages=2)

    def rope(self, **kw):
        io = A.RopeIO()
        io.q = io.k = io.q_out = io.k_out = io.cos_sin = io.positions = io.status = 1 << 20  # never followed: refused first
        io.q_stride = io.q_out_stride = 8 * 128
        io.k_stride = io.k_out_stride = 2 * 128
        io.eps, io.max_positions, io.rot_dim, io.rows = 1e-6, 10, 128, 4
        for k, v in kw.items():
            setattr(io, k, v)
        return io

    @pytest.mark.parametrize("kw,code", [
        (dict(rows=65), ESHAPE), (dict(rows=-1), ESHAPE), (dict(rot_dim=8), ESHAPE), (dict(rot_dim=144), ESHAPE),
        (dict(rot_dim=-16), ESHAPE), (dict(max_positions=-1), ESHAPE), (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL),
        (dict(status=None), EINVAL), (dict(positions=None), EINVAL), (dict(cos_sin=None), EINVAL), (dict(q=None, k=None), EINVAL),
        (dict(q_out=None), EINVAL), (dict(k_out=None), EINVAL), (dict(q=(1 << 20) + 2), EALIGN), (dict(q_stride=8 * 128 + 4), EALIGN),
        (dict(k_stride=128), ESHAPE), (dict(q_weight=(1 << 20) + 4), EALIGN), (dict(positions=(1 << 20) + 1), EALIGN),
        (dict(weight_offset=float("inf")), EINVAL),
    ])
    def test_norm_rope(self, kw, code):
        p = self.plan()
        assert lpe.lib().lp_norm_rope(p._h, ctypes.byref(self.rope(**kw)), None) == code

    @pytest.mark.parametrize("kw,code", [
        (dict(groups=9), ESHAPE), (dict(groups=-1), ESHAPE), (dict(v=None), EINVAL), (dict(v_stride=8), ESHAPE), (dict(k_cache=None), EINVAL),
        (dict(v_cache=(1 << 20) + 8), EALIGN), (dict(group_indptr=None), EINVAL), (dict(lens=None), EINVAL),
        (dict(block_tables=(1 << 20) + 2), EALIGN), (dict(rope=dict(k=None)), EINVAL),
    ])
    def test_append(self, kw, code):
        p = self.plan()
        io = A.AppendIO()
        io.rope = self.rope(**kw.pop("rope", {}))
        io.v = io.group_indptr = io.lens = io.block_tables = io.k_cache = io.v_cache = 1 << 20
        io.v_stride, io.groups = 2 * 128, 2
        for k, v in kw.items():
            setattr(io, k, v)
        assert lpe.lib().lp_kv_append(p._h, ctypes.byref(io), None) == code

    @pytest.mark.parametrize("kw,code", [
        (dict(rows=65), ESHAPE), (dict(groups=9), ESHAPE), (dict(prefixes=2), ESHAPE), (dict(prefixes=-1), ESHAPE), (dict(scale=0.0), EINVAL),
        (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(scale=-1.0), EINVAL), (dict(status=None), EINVAL),
        (dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(k_cache=None), EINVAL), (dict(lens=None), EINVAL),
        (dict(prefix_tables=None), EINVAL), (dict(q=(1 << 20) + 8), EALIGN), (dict(out_stride=1028), EALIGN),
        (dict(q_stride=512), ESHAPE), (dict(lse_out=(1 << 20) + 2), EALIGN), (dict(row_masks=(1 << 20) + 1), EALIGN),
    ])
    def test_attend(self, kw, code):
        p = self.plan()
        io = A.AttendIO()
        for n in ("q", "k_cache", "v_cache", "group_indptr", "lens", "block_tables", "prefix_indptr", "prefix_lens", "prefix_tables", "out", "status"):
            setattr(io, n, 1 << 20)
        io.q_stride = io.out_stride = 8 * 128
        io.scale, io.rows, io.groups, io.prefixes = 0.1, 4, 2, 1
        for k, v in kw.items():
            setattr(io, k, v)
        assert lpe.lib().lp_attend(p._h, ctypes.byref(io), None) == code

    def test_python_checks(self):
        import torch
        p = self.plan()
        dev = torch.device("cuda", 0)
        q = torch.zeros(4, 8, 128, dtype=torch.bfloat16, device=dev)
        ok = dict(q=q, q_out=torch.zeros_like(q), cos_sin=torch.zeros(4, 128, device=dev),
                  positions=torch.zeros(4, dtype=torch.int32, device=dev), status=torch.zeros(1, dtype=torch.int32, device=dev))
        p.norm_rope(**ok)
        for kw in (dict(q=q.half()), dict(q=q.cpu()), dict(q=q[:, :7]), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)),
                   dict(q_out=q[:3]), dict(cos_sin=torch.zeros(4, 128, dtype=torch.float64, device=dev)),
                   dict(positions=torch.zeros(3, dtype=torch.int32, device=dev)), dict(positions=torch.zeros(4, device=dev)),
                   dict(cos_sin=torch.zeros(128, 4, device=dev).t()), dict(q=None, q_out=None)):
            with pytest.raises(ValueError):
                p.norm_rope(**{**ok, **kw})
        torch.cuda.synchronize()

    def test_python_takes_no_table_and_names_what_is_missing(self):
        import torch
        p = self.plan()
        dev = torch.device("cuda", 0)
        z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device=dev)  # noqa: E731
        i = lambda *s: z(*s, dtype=torch.int32)  # noqa: E731
        q, k = torch.randn(4, 8, 128, device=dev).bfloat16(), torch.randn(4, 2, 128, device=dev).bfloat16()
        out, st, pos = z(4, 8, 128), i(1), torch.tensor([0, 5, 1 << 30, -1], dtype=torch.int32, device=dev)
        out[3] = 7.0
        p.norm_rope(q=q, q_out=out, positions=pos, status=st)  # no table: nothing is rotated
        assert torch.equal(out[:3], q[:3]) and bool((out[3] == 7.0).all())
        kc, vc = z(100, 2, 16, 128), z(100, 2, 16, 128)
        batch = dict(k_cache=kc, v_cache=vc, group_indptr=torch.tensor([0, 4], dtype=torch.int32, device=dev), lens=i(1), block_tables=i(1, 10), status=st)
        append = dict(batch, k=k, v=k, positions=pos)
        p.append(**append)
        torch.cuda.synchronize()
        assert torch.equal(kc[0, :, :3].transpose(0, 1), k[:3]) and torch.equal(vc[0, :, :3].transpose(0, 1), k[:3]) and int(st[0]) == 0
        assert not bool(kc[0, :, 3:].any()) and not bool(vc[0, :, 3:].any())  # the row that is skipped, too
        attend = dict(batch, q=q, out=out)
        p.attend(**attend)
        for call, args, names in ((p.append, append, ("status", "group_indptr", "v")), (p.attend, attend, ("status", "group_indptr", "q", "out")),
                                  (p.norm_rope, dict(q=q, q_out=out, positions=pos, status=st), ("status", "q_out"))):
            for name in names:
                with pytest.raises(ValueError, match=name):
                    call(**{**args, name: None})
        with pytest.raises(ValueError, match="neither q nor k"):
            p.append(**{**append, "k": None})
        torch.cuda.synchronize()
