"""Attention of the verify forward: ``AttnPlan``, the Python side of the
``lp_norm_rope``, ``lp_kv_append`` and ``lp_attend`` entries (argument
marshalling only; see ``include/lp_epilogue.h`` for the contract)."""
from __future__ import annotations

import ctypes

from . import LP_BF16, LP_F16, PLAN_DEBUG_FORCE_TIMEOUT, _check, lib

ATTN_MAX_GROUP_ROWS = 32


class AttnDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "max_rows", "max_groups", "max_group_rows", "q_heads", "kv_heads", "head_dim", "page_size", "max_pages",
        "max_prefixes", "max_prefix_pages", "dtype", "device")] + [
        ("num_pages", ctypes.c_int64), ("flags", ctypes.c_uint32), ("timeout_ns", ctypes.c_int64)]


class RopeIO(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "q_out", "k_out")] + [
        (n, ctypes.c_int64) for n in ("q_stride", "k_stride", "q_out_stride", "k_out_stride")] + [
        (n, ctypes.c_void_p) for n in ("q_weight", "k_weight", "cos_sin", "positions", "status")] + [
        ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float)] + [
        (n, ctypes.c_int32) for n in ("max_positions", "rot_dim", "interleaved", "rows")]


class AppendIO(ctypes.Structure):
    _fields_ = [("rope", RopeIO), ("v", ctypes.c_void_p), ("v_stride", ctypes.c_int64)] + [
        (n, ctypes.c_void_p) for n in ("group_indptr", "lens", "block_tables", "k_cache", "v_cache")] + [
        ("groups", ctypes.c_int32)]


class AttendIO(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_stride", ctypes.c_int64)] + [
        (n, ctypes.c_void_p) for n in ("k_cache", "v_cache", "group_indptr", "lens", "block_tables", "row_masks",
                                       "prefix_indptr", "prefix_lens", "prefix_tables", "out")] + [
        ("out_stride", ctypes.c_int64), ("lse_out", ctypes.c_void_p), ("status", ctypes.c_void_p),
        ("scale", ctypes.c_float), ("rows", ctypes.c_int32), ("groups", ctypes.c_int32), ("prefixes", ctypes.c_int32)]


def make_attn_desc(*, max_rows, max_groups, q_heads, kv_heads, head_dim, page_size, num_pages, max_pages,
                   max_group_rows=16, max_prefixes=0, max_prefix_pages=0, dtype="bf16", device=0, timeout_ns=0,
                   debug_force_timeout=False) -> AttnDesc:
    code = {"bf16": LP_BF16, "f16": LP_F16}.get(dtype, 99)
    return AttnDesc(int(max_rows), int(max_groups), int(max_group_rows), int(q_heads), int(kv_heads), int(head_dim),
                    int(page_size), int(max_pages), int(max_prefixes), int(max_prefix_pages), code, int(device),
                    int(num_pages), PLAN_DEBUG_FORCE_TIMEOUT if debug_force_timeout else 0, int(timeout_ns))


def attn_scratch_bytes(**desc_kw) -> int:
    return int(lib().lp_attn_scratch_bytes(ctypes.byref(make_attn_desc(**desc_kw))))


class AttnPlan:
    """Attention operators of a verify forward on one device: the head norms and
    position rotation (``norm_rope``), the append of a round's keys and values
    to the paged cache (``append``), and the attention of the verify rows over
    it (``attend``).

    Caches are [num_pages, kv_heads, page_size, head_dim].  ``lens`` counts each
    group's committed tokens and is changed by none of the calls: after the
    epilogue, ``lens += accepted + 1`` commits the round.  Every call only
    enqueues on ``stream`` (default: torch's current stream) and ORs its status
    bits into ``status`` without resetting it."""

    def __init__(self, **desc_kw):
        import torch
        self.desc = make_attn_desc(**desc_kw)
        self.device = int(self.desc.device)
        self._dtype = torch.bfloat16 if self.desc.dtype == LP_BF16 else torch.float16
        self._h = None
        h = ctypes.c_void_p()
        _check(lib().lp_attn_create(ctypes.byref(h), ctypes.byref(self.desc)), "lp_attn_create")
        self._h = h
        self._i32, self._f32 = torch.int32, torch.float32
        self._current = torch.cuda.current_stream

    def close(self) -> None:
        if getattr(self, "_h", None) is not None:
            _check(lib().lp_attn_destroy(self._h), "lp_attn_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _stream(self, stream):
        if stream is None:
            return self._current(self.device).cuda_stream
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)

    def _heads(self, name, x, rows, heads):
        """A [rows, heads, head_dim] tensor with dense heads: (pointer, row stride)."""
        d = self.desc.head_dim
        if x.dtype != self._dtype or x.device.index != self.device or not x.is_cuda:
            raise ValueError(f"{name}: expected {self._dtype} on CUDA device {self.device}")
        if x.shape != (rows, heads, d):
            raise ValueError(f"{name}: expected shape [{rows}, {heads}, {d}], got {list(x.shape)}")
        s = x.stride()
        if (heads > 1 and s[1] != d) or s[2] != 1:
            raise ValueError(f"{name}: the heads of a row must be dense")
        return x.data_ptr(), s[0] if rows > 1 else heads * d

    def _flat(self, name, x, dtype, shape=None, numel=0):
        """A contiguous tensor of a type and a shape (or a least number of elements); None passes."""
        if x is None:
            return None
        if x.dtype != dtype or x.device.index != self.device or not x.is_cuda or not x.is_contiguous():
            raise ValueError(f"{name}: expected contiguous {dtype} on CUDA device {self.device}")
        if shape is not None and x.shape != shape or x.numel() < numel:
            raise ValueError(f"{name}: expected {list(shape) if shape is not None else f'at least {numel} elements'}, got {list(x.shape)}")
        return x.data_ptr()

    def _status(self, x):
        if x.element_size() != 4 or x.numel() < 1 or not x.is_cuda or x.device.index != self.device:
            raise ValueError(f"status: expected one 32-bit word on CUDA device {self.device}")
        return x.data_ptr()

    def _caches(self, k_cache, v_cache):
        d = self.desc
        shape = (d.num_pages, d.kv_heads, d.page_size, d.head_dim)
        return (self._flat("k_cache", k_cache, self._dtype, shape), self._flat("v_cache", v_cache, self._dtype, shape))

    def _rope(self, q, k, q_out, k_out, q_weight, k_weight, eps, weight_offset, cos_sin, interleaved, positions, status):
        d = self.desc
        if q is None and k is None:
            raise ValueError("norm_rope: neither q nor k")
        rows = int((k if q is None else q).shape[0])
        io = RopeIO()
        if q is not None:
            io.q, io.q_stride = self._heads("q", q, rows, d.q_heads)
            io.q_out, io.q_out_stride = self._heads("q_out", q_out, rows, d.q_heads)
        if k is not None:
            io.k, io.k_stride = self._heads("k", k, rows, d.kv_heads)
            if k_out is not None:
                io.k_out, io.k_out_stride = self._heads("k_out", k_out, rows, d.kv_heads)
        io.q_weight = self._flat("q_weight", q_weight, self._dtype, (d.head_dim,))
        io.k_weight = self._flat("k_weight", k_weight, self._dtype, (d.head_dim,))
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin: expected [positions, rot_dim]")
        io.cos_sin = self._flat("cos_sin", cos_sin, self._f32)
        io.max_positions, io.rot_dim = cos_sin.shape
        io.positions = self._flat("positions", positions, self._i32, None, rows)
        io.status = self._status(status)
        io.eps, io.weight_offset, io.interleaved, io.rows = eps, weight_offset, int(bool(interleaved)), rows
        return io

    def norm_rope(self, *, cos_sin, positions, status, q=None, k=None, q_out=None, k_out=None, q_weight=None,
                  k_weight=None, eps=1e-6, weight_offset=0.0, interleaved=False, stream=None) -> None:
        """RMS norm (where a weight is given) and position rotation of each head of
        ``q`` [rows, q_heads, head_dim] and ``k`` [rows, kv_heads, head_dim].
        ``cos_sin`` is float32 [positions, rot_dim]: the cosines of the rot_dim / 2
        angles, then their sines.  Rows with a negative position are skipped."""
        io = self._rope(q, k, q_out, k_out, q_weight, k_weight, eps, weight_offset, cos_sin, interleaved, positions, status)
        _check(lib().lp_norm_rope(self._h, ctypes.byref(io), self._stream(stream)), "lp_norm_rope")

    def append(self, *, k, v, k_cache, v_cache, group_indptr, lens, block_tables, cos_sin, positions, status, q=None,
               q_out=None, k_out=None, q_weight=None, k_weight=None, eps=1e-6, weight_offset=0.0, interleaved=False,
               stream=None) -> None:
        """``norm_rope``, with the keys and values of row j of group g written to
        token ``lens[g] + j`` of the paged caches (``block_tables`` int32 [groups,
        max_pages]); ``k_out`` is optional."""
        d = self.desc
        io = AppendIO()
        io.rope = self._rope(q, k, q_out, k_out, q_weight, k_weight, eps, weight_offset, cos_sin, interleaved, positions, status)
        io.v, io.v_stride = self._heads("v", v, io.rope.rows, d.kv_heads)
        groups = group_indptr.numel() - 1
        io.group_indptr = self._flat("group_indptr", group_indptr, self._i32, None, 1)
        io.lens = self._flat("lens", lens, self._i32, None, groups)
        io.block_tables = self._flat("block_tables", block_tables, self._i32, (groups, d.max_pages))
        io.k_cache, io.v_cache = self._caches(k_cache, v_cache)
        io.groups = groups
        _check(lib().lp_kv_append(self._h, ctypes.byref(io), self._stream(stream)), "lp_kv_append")

    def attend(self, *, q, k_cache, v_cache, group_indptr, lens, block_tables, out, status, lse_out=None, row_masks=None,
               prefix_indptr=None, prefix_lens=None, prefix_tables=None, scale=None, stream=None) -> None:
        """Attention of the verify rows ``q`` over their group's committed tokens, the
        round's own rows (causal, or those set in the int32 ``row_masks`` [rows]) and
        the prefix that serves their group (``prefix_indptr`` int32 [prefixes + 1]
        over groups, ``prefix_lens`` [prefixes], ``prefix_tables`` [prefixes,
        max_prefix_pages]).  ``lse_out`` is float32 [rows, q_heads]."""
        d = self.desc
        io = AttendIO()
        rows = int(q.shape[0])
        io.q, io.q_stride = self._heads("q", q, rows, d.q_heads)
        io.out, io.out_stride = self._heads("out", out, rows, d.q_heads)
        io.k_cache, io.v_cache = self._caches(k_cache, v_cache)
        groups = group_indptr.numel() - 1
        io.group_indptr = self._flat("group_indptr", group_indptr, self._i32, None, 1)
        io.lens = self._flat("lens", lens, self._i32, None, groups)
        io.block_tables = self._flat("block_tables", block_tables, self._i32, (groups, d.max_pages))
        io.row_masks = self._flat("row_masks", row_masks, self._i32, None, rows)
        if prefix_lens is not None:
            n = prefix_lens.numel()
            io.prefix_indptr = self._flat("prefix_indptr", prefix_indptr, self._i32, (n + 1,))
            io.prefix_lens = self._flat("prefix_lens", prefix_lens, self._i32)
            io.prefix_tables = self._flat("prefix_tables", prefix_tables, self._i32, (n, d.max_prefix_pages))
            io.prefixes = n
        io.lse_out = self._flat("lse_out", lse_out, self._f32, (rows, d.q_heads))
        io.status = self._status(status)
        io.scale = d.head_dim ** -0.5 if scale is None else scale
        io.rows, io.groups = rows, groups
        _check(lib().lp_attend(self._h, ctypes.byref(io), self._stream(stream)), "lp_attend")
