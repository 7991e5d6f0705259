"""Attention of the verify forward: ``AttnPlan``, the Python side of the
``lp_norm_rope``, ``lp_kv_append`` and ``lp_attend`` entries, of
``lp_kv_reserve``, and of ``lp_kv_append4`` and ``lp_attend4`` over a cache in 4
bits (argument marshalling only; see ``include/lp_epilogue.h`` for the
contract)."""
from __future__ import annotations

import ctypes
import struct

from . import ATTN_KV4, LP_BF16, LP_F16, PLAN_DEBUG_FORCE_TIMEOUT, _check, lib

ATTN_MAX_GROUP_ROWS = 32
BLOCK4 = 16  # lanes that share a scale in a cache of 4 bits


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


class ReserveIO(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "lens", "counts", "starts", "held", "queue", "free_pages", "block_tables", "group_indptr", "round_lens", "held_out",
        "queue_out", "positions", "slots", "status")] + [(n, ctypes.c_int32) for n in ("rows", "groups", "ring")]


class Append4IO(ctypes.Structure):
    _fields_ = [("append", AppendIO)] + [(n, ctypes.c_void_p) for n in ("k_scales", "v_scales", "k_held", "v_held")] + [
        (n, ctypes.c_int64) for n in ("k_held_stride", "v_held_stride")] + [(n, ctypes.c_float) for n in ("k_factor", "v_factor")]


class Attend4IO(ctypes.Structure):
    _fields_ = [("attend", AttendIO)] + [(n, ctypes.c_void_p) for n in ("k_scales", "v_scales")] + [
        (n, ctypes.c_float) for n in ("k_factor", "v_factor")]


def make_attn_desc(*, max_rows, max_groups, q_heads, kv_heads, head_dim, page_size, num_pages, max_pages,
                   max_group_rows=16, max_prefixes=0, max_prefix_pages=0, dtype="bf16", device=0, timeout_ns=0,
                   debug_force_timeout=False, kv_bits=16) -> AttnDesc:
    if kv_bits not in (4, 16):
        raise ValueError(f"kv_bits: expected 4 or 16, got {kv_bits}")
    flags = (PLAN_DEBUG_FORCE_TIMEOUT if debug_force_timeout else 0) | (ATTN_KV4 if kv_bits == 4 else 0)
    code = {"bf16": LP_BF16, "f16": LP_F16}.get(dtype, 99)
    return AttnDesc(int(max_rows), int(max_groups), int(max_group_rows), int(q_heads), int(kv_heads), int(head_dim),
                    int(page_size), int(max_pages), int(max_prefixes), int(max_prefix_pages), code, int(device),
                    int(num_pages), flags, int(timeout_ns))


def attn_scratch_bytes(**desc_kw) -> int:
    return int(lib().lp_attn_scratch_bytes(ctypes.byref(make_attn_desc(**desc_kw))))


# The io structures as one native pack each: a call sets every field at once (field by field through ctypes takes longer
# than the kernel of a small call).
_ROPE = "PPPPqqqqPPPPPffiiii"
_PACK_ROPE = struct.Struct("@" + _ROPE + "0P")
_APPEND, _ATTEND = _ROPE + "PqPPPPPi", "PqPPPPPPPPPPqPPfiii"
_PACK_APPEND = struct.Struct("@" + _APPEND + "0P")
_PACK_ATTEND = struct.Struct("@" + _ATTEND + "0P")
_PACK_APPEND4 = struct.Struct("@" + _APPEND + "0PPPPPqqff0P")
_PACK_ATTEND4 = struct.Struct("@" + _ATTEND + "0PPPff0P")
_PACK_RESERVE = struct.Struct("@PPPPPPPPPPPPPPiii0P")
_ANY_POSITION = 2 ** 31 - 1  # max_positions of a call without a table


class AttnPlan:
    """Attention operators of a verify forward on one device: the head norms and
    position rotation (``norm_rope``), the append of a round's keys and values
    to the paged cache (``append``), the attention of the verify rows over it
    (``attend``), and the pages, positions and slots of a round (``reserve``).

    Caches are [num_pages, kv_heads, page_size, head_dim].  With ``kv_bits=4``
    they are held in 4 bits, and ``append4`` and ``attend4`` take the place of
    ``append`` and ``attend``: uint8 codes [num_pages, kv_heads, page_size,
    head_dim / 2] and float8_e4m3fn scales [num_pages, kv_heads, page_size,
    head_dim / 16].

    ``lens`` counts each group's committed tokens, negative for an idle group,
    and is changed by none of the calls: after the epilogue, ``lens +=
    torch.where(lens < 0, 0, accepted + 1)`` commits the round (``round_lens < 0``
    after ``reserve``, whose groups without pages sit out).  Every call only
    enqueues on ``stream`` (default: torch's current stream) and ORs its status
    bits into ``status`` without resetting it.  Like a ``Plan``, one plan serves
    one stream, and one thread, at a time."""

    def __init__(self, **desc_kw):
        import torch
        self.desc = d = make_attn_desc(**desc_kw)
        self._i64, self._u8, self._e4m3 = torch.int64, torch.uint8, torch.float8_e4m3fn
        self.device = int(d.device)
        self._dtype = torch.bfloat16 if d.dtype == LP_BF16 else torch.float16
        self._i32, self._f32 = torch.int32, torch.float32
        self._h = None
        h = ctypes.c_void_p()
        _check(lib().lp_attn_create(ctypes.byref(h), ctypes.byref(d)), "lp_attn_create")
        self._h = h
        self._current = torch._C._cuda_getCurrentRawStream
        self._io = ctypes.create_string_buffer(max(_PACK_ROPE.size, _PACK_APPEND4.size, _PACK_ATTEND4.size, _PACK_RESERVE.size))
        self._at = ctypes.addressof(self._io)
        self._q_heads, self._kv_heads, self._dim = int(d.q_heads), int(d.kv_heads), int(d.head_dim)
        self._one_head = (self._dim,)
        self._cache_shape = (int(d.num_pages), int(d.kv_heads), int(d.page_size), int(d.head_dim))
        self._codes_shape = self._cache_shape[:3] + (self._dim // 2,)
        self._scales_shape = self._cache_shape[:3] + (self._dim // BLOCK4,)
        self._norm_rope, self._append, self._attend = lib().lp_norm_rope, lib().lp_kv_append, lib().lp_attend
        self._reserve, self._append4, self._attend4 = lib().lp_kv_reserve, lib().lp_kv_append4, lib().lp_attend4

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
            return self._current(self.device)
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)

    def _rows(self, name, x, want):
        """A tensor of shape ``want``, [rows, heads, head_dim], with dense heads: (pointer, row stride)."""
        if x is not None and x.dtype is self._dtype and x.shape == want and x.get_device() == self.device:
            s, t, u = x.stride()
            rows, heads, d = want
            if u == 1 and (t == d or heads == 1):
                return x.data_ptr(), s if rows > 1 else heads * d
            raise ValueError(f"{name}: the heads of a row must be dense")
        if x is None:
            raise ValueError(f"{name}: missing")
        if x.dtype is not self._dtype or x.get_device() != self.device:
            raise ValueError(f"{name}: expected {self._dtype} on CUDA device {self.device}")
        raise ValueError(f"{name}: expected shape {list(want)}, got {list(x.shape)}")

    def _flat(self, name, x, dtype, numel):
        """Pointer of a contiguous tensor of a type and at least so many elements; 0 for None."""
        if x is None:
            return 0
        if x.dtype is dtype and x.get_device() == self.device and x.is_contiguous():
            if x.numel() >= numel:
                return x.data_ptr()
            raise ValueError(f"{name}: expected at least {numel} elements, got {list(x.shape)}")
        raise ValueError(f"{name}: expected contiguous {dtype} on CUDA device {self.device}")

    def _shaped(self, name, x, dtype, shape):
        """Pointer of a contiguous tensor of a type and a shape; 0 for None."""
        if x is None:
            return 0
        if x.shape != shape:
            raise ValueError(f"{name}: expected shape {list(shape)}, got {list(x.shape)}")
        if x.dtype is dtype and x.get_device() == self.device and x.is_contiguous():
            return x.data_ptr()
        raise ValueError(f"{name}: expected contiguous {dtype} on CUDA device {self.device}")

    def _status(self, x):
        if x is None or x.element_size() != 4 or x.numel() < 1 or x.get_device() != self.device:
            raise ValueError(f"status: expected one 32-bit word on CUDA device {self.device}")
        return x.data_ptr()

    def _groups(self, group_indptr):
        if group_indptr is None:
            raise ValueError("group_indptr: missing")
        return group_indptr.numel() - 1

    def _rope(self, q, k, q_out, k_out, q_weight, k_weight, eps, weight_offset, cos_sin, interleaved, positions, status):
        """The fields of lp_rope_io, in order, and the rows."""
        qp = qs = qo = qos = kp = ks = ko = kos = 0
        if q is not None:
            rows = q.shape[0]
            want = (rows, self._q_heads, self._dim)
            qp, qs = self._rows("q", q, want)
            qo, qos = self._rows("q_out", q_out, want)
        elif k is None:
            raise ValueError("neither q nor k")
        else:
            rows = k.shape[0]
        if k is not None:
            want = (rows, self._kv_heads, self._dim)
            kp, ks = self._rows("k", k, want)
            if k_out is not None:
                ko, kos = self._rows("k_out", k_out, want)
        if cos_sin is None:
            table, rot = _ANY_POSITION, 0
        elif cos_sin.dim() != 2:
            raise ValueError("cos_sin: expected [positions, rot_dim]")
        else:
            table, rot = cos_sin.shape
        return rows, (qp, kp, qo, ko, qs, ks, qos, kos,
                      self._shaped("q_weight", q_weight, self._dtype, self._one_head),
                      self._shaped("k_weight", k_weight, self._dtype, self._one_head),
                      self._flat("cos_sin", cos_sin, self._f32, 0), self._flat("positions", positions, self._i32, rows),
                      self._status(status), eps, weight_offset, table, rot, 1 if interleaved else 0, rows)

    def _appended(self, q, k, q_out, k_out, q_weight, k_weight, eps, weight_offset, cos_sin, interleaved, positions, status, v,
                  group_indptr, lens, block_tables, k_cache, v_cache):
        """The fields of lp_append_io, in order; the caches as pointers."""
        rows, rope = self._rope(q, k, q_out, k_out, q_weight, k_weight, eps, weight_offset, cos_sin, interleaved, positions, status)
        vp, vs = self._rows("v", v, (rows, self._kv_heads, self._dim))
        groups = self._groups(group_indptr)
        return (*rope, vp, vs, self._flat("group_indptr", group_indptr, self._i32, 1), self._flat("lens", lens, self._i32, groups),
                self._shaped("block_tables", block_tables, self._i32, (groups, self.desc.max_pages)), k_cache, v_cache, groups)

    def _attended(self, q, out, k_cache, v_cache, group_indptr, lens, block_tables, status, lse_out, row_masks, prefix_indptr,
                  prefix_lens, prefix_tables, scale):
        """The fields of lp_attend_io, in order; the caches as pointers."""
        i32 = self._i32
        if q is None:
            raise ValueError("q: missing")
        rows = q.shape[0]
        want = (rows, self._q_heads, self._dim)
        qp, qs = self._rows("q", q, want)
        op, os_ = self._rows("out", out, want)
        groups = self._groups(group_indptr)
        prefixes = pi = pl = pt = 0
        if prefix_lens is not None:
            prefixes = prefix_lens.numel()
            pi = self._flat("prefix_indptr", prefix_indptr, i32, prefixes + 1)
            pl = self._flat("prefix_lens", prefix_lens, i32, 0)
            pt = self._shaped("prefix_tables", prefix_tables, i32, (prefixes, self.desc.max_prefix_pages))
        return (qp, qs, k_cache, v_cache, self._flat("group_indptr", group_indptr, i32, 1), self._flat("lens", lens, i32, groups),
                self._shaped("block_tables", block_tables, i32, (groups, self.desc.max_pages)),
                self._flat("row_masks", row_masks, i32, rows), pi, pl, pt, op, os_,
                self._shaped("lse_out", lse_out, self._f32, (rows, self._q_heads)), self._status(status),
                self._dim ** -0.5 if scale is None else scale, rows, groups, prefixes)

    def _held(self, name, x, rows):
        """Pointer and row stride of an optional output [rows, kv_heads, head_dim]."""
        return (0, 0) if x is None else self._rows(name, x, (rows, self._kv_heads, self._dim))

    def norm_rope(self, *, positions, status, cos_sin=None, q=None, k=None, q_out=None, k_out=None, q_weight=None,
                  k_weight=None, eps=1e-6, weight_offset=0.0, interleaved=False, stream=None) -> None:
        """RMS norm (where a weight is given) and position rotation of each head of
        ``q`` [rows, q_heads, head_dim] and ``k`` [rows, kv_heads, head_dim].
        ``cos_sin`` is float32 [positions, rot_dim]: the cosines of the rot_dim / 2
        angles, then their sines; without one nothing is rotated and any position
        below 2^31 - 1 will do.  Rows with a negative position are skipped."""
        _, rope = self._rope(q, k, q_out, k_out, q_weight, k_weight, eps, weight_offset, cos_sin, interleaved, positions, status)
        _PACK_ROPE.pack_into(self._io, 0, *rope)
        rc = self._norm_rope(self._h, self._at, self._stream(stream))
        if rc:
            _check(rc, "lp_norm_rope")

    def append(self, *, k, v, k_cache, v_cache, group_indptr, lens, block_tables, positions, status, cos_sin=None, q=None,
               q_out=None, k_out=None, q_weight=None, k_weight=None, eps=1e-6, weight_offset=0.0, interleaved=False,
               stream=None) -> None:
        """``norm_rope``, with the keys and values of row j of group g written to
        token ``lens[g] + j`` of the paged caches (``block_tables`` int32 [groups,
        max_pages]); ``k_out`` is optional."""
        _PACK_APPEND.pack_into(self._io, 0, *self._appended(
            q, k, q_out, k_out, q_weight, k_weight, eps, weight_offset, cos_sin, interleaved, positions, status, v, group_indptr, lens,
            block_tables, self._shaped("k_cache", k_cache, self._dtype, self._cache_shape),
            self._shaped("v_cache", v_cache, self._dtype, self._cache_shape)))
        rc = self._append(self._h, self._at, self._stream(stream))
        if rc:
            _check(rc, "lp_kv_append")

    def attend(self, *, q, k_cache, v_cache, group_indptr, lens, block_tables, out, status, lse_out=None, row_masks=None,
               prefix_indptr=None, prefix_lens=None, prefix_tables=None, scale=None, stream=None) -> None:
        """Attention of the verify rows ``q`` over their group's committed tokens, the
        round's own rows (causal, or those set in the int32 ``row_masks`` [rows]) and
        the prefix that serves their group (``prefix_indptr`` int32 [prefixes + 1]
        over groups, ``prefix_lens`` [prefixes], ``prefix_tables`` [prefixes,
        max_prefix_pages]).  ``lse_out`` is float32 [rows, q_heads]."""
        _PACK_ATTEND.pack_into(self._io, 0, *self._attended(
            q, out, self._shaped("k_cache", k_cache, self._dtype, self._cache_shape),
            self._shaped("v_cache", v_cache, self._dtype, self._cache_shape), group_indptr, lens, block_tables, status, lse_out,
            row_masks, prefix_indptr, prefix_lens, prefix_tables, scale))
        rc = self._attend(self._h, self._at, self._stream(stream))
        if rc:
            _check(rc, "lp_attend")

    def append4(self, *, k, v, k_cache, v_cache, k_scales, v_scales, group_indptr, lens, block_tables, positions, status, k_factor=1.0,
                v_factor=1.0, k_held=None, v_held=None, cos_sin=None, q=None, q_out=None, k_out=None, q_weight=None, k_weight=None,
                eps=1e-6, weight_offset=0.0, interleaved=False, stream=None) -> None:
        """``append`` to a cache in 4 bits (a plan with ``kv_bits=4``): codes in
        ``k_cache`` and ``v_cache``, the scales of 16 lanes each in ``k_scales`` and
        ``v_scales``; a value is code * scale * factor, the factor a power of two.
        ``k_held`` and ``v_held`` [rows, kv_heads, head_dim], where given, receive
        the values as the cache holds them."""
        fields = self._appended(
            q, k, q_out, k_out, q_weight, k_weight, eps, weight_offset, cos_sin, interleaved, positions, status, v, group_indptr, lens,
            block_tables, self._shaped("k_cache", k_cache, self._u8, self._codes_shape),
            self._shaped("v_cache", v_cache, self._u8, self._codes_shape))
        rows = v.shape[0]
        kh, khs = self._held("k_held", k_held, rows)
        vh, vhs = self._held("v_held", v_held, rows)
        _PACK_APPEND4.pack_into(self._io, 0, *fields, self._shaped("k_scales", k_scales, self._e4m3, self._scales_shape),
                                self._shaped("v_scales", v_scales, self._e4m3, self._scales_shape), kh, vh, khs, vhs, k_factor, v_factor)
        rc = self._append4(self._h, self._at, self._stream(stream))
        if rc:
            _check(rc, "lp_kv_append4")

    def attend4(self, *, q, k_cache, v_cache, k_scales, v_scales, group_indptr, lens, block_tables, out, status, k_factor=1.0,
                v_factor=1.0, lse_out=None, row_masks=None, prefix_indptr=None, prefix_lens=None, prefix_tables=None, scale=None,
                stream=None) -> None:
        """``attend`` over a cache in 4 bits (a plan with ``kv_bits=4``), as
        ``append4`` writes it."""
        fields = self._attended(
            q, out, self._shaped("k_cache", k_cache, self._u8, self._codes_shape),
            self._shaped("v_cache", v_cache, self._u8, self._codes_shape), group_indptr, lens, block_tables, status, lse_out, row_masks,
            prefix_indptr, prefix_lens, prefix_tables, scale)
        _PACK_ATTEND4.pack_into(self._io, 0, *fields, self._shaped("k_scales", k_scales, self._e4m3, self._scales_shape),
                                self._shaped("v_scales", v_scales, self._e4m3, self._scales_shape), k_factor, v_factor)
        rc = self._attend4(self._h, self._at, self._stream(stream))
        if rc:
            _check(rc, "lp_attend4")

    def reserve(self, *, lens, counts, held, queue, free_pages, block_tables, group_indptr, round_lens, held_out, queue_out, positions,
                status, starts=None, slots=None, stream=None) -> None:
        """Lays a round out: group g owns the next ``counts[g]`` rows
        (``group_indptr``), takes the pages that its tokens need beyond the
        ``held[g]`` of ``block_tables[g]`` from the queue of free pages (int64
        ``queue`` = [head, tail] into the ring ``free_pages``), and idle groups
        (``lens`` < 0) give theirs back.  ``round_lens`` are the lens for the
        round's other calls and for its commit (-1 where the pages ran out: that
        group sits the round out, and its ``lens`` stays), ``positions`` and the
        int64 ``slots`` those of every row (-1: padding); their length is the
        batch's rows.  ``held_out`` and ``queue_out`` may be ``held`` and
        ``queue``."""
        i32, i64, flat, groups = self._i32, self._i64, self._flat, self._groups(group_indptr)
        for name, x in (("positions", positions), ("free_pages", free_pages), ("lens", lens)):
            if x is None:
                raise ValueError(f"{name}: missing")
        rows = positions.numel()
        _PACK_RESERVE.pack_into(
            self._io, 0, flat("lens", lens, i32, groups), flat("counts", counts, i32, groups), flat("starts", starts, i32, groups),
            flat("held", held, i32, groups), flat("queue", queue, i64, 2), flat("free_pages", free_pages, i32, 1),
            self._shaped("block_tables", block_tables, i32, (groups, self.desc.max_pages)),
            flat("group_indptr", group_indptr, i32, 1), flat("round_lens", round_lens, i32, groups), flat("held_out", held_out, i32, groups),
            flat("queue_out", queue_out, i64, 2), flat("positions", positions, i32, 0), flat("slots", slots, i64, rows),
            self._status(status), rows, groups, free_pages.numel())
        rc = self._reserve(self._h, self._at, self._stream(stream))
        if rc:
            _check(rc, "lp_kv_reserve")
