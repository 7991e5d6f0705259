"""64-bit reference of the attention operators, written from the formulas, and
the bounds its comparisons use.

Bounds.  u is the plan type's unit roundoff (2^-8 BF16, 2^-11 F16).

norm_rope: FP32 arithmetic (a handful of roundings on a and b of a pair, a
relative 2^-20 at most) and one rounding:
    |y - ref| <= u |ref| + 2^-20 (|a| + |b|) + the type's smallest step.

attend: scores carry the FP32 error of a D-term dot product, at most
e_s = 2 D 2^-24 max_t scale sum_i |q_i k_ti| (twice the rounding bound, as a
tensor product may truncate), plus 2^-21 max |s| for the scaling into base 2.
Each probability then carries a relative u (rounded to the type before it
multiplies v) + 2 e_s + 2^-18 (exponential, FP32 sums), so
    |out - ref| <= u |ref| + (u + 2 e_s + 2^-18) sum_t p_t |v_t| + steps,
    |lse - ref| <= e_s + 2^-18.
F16 probabilities below the normal range carry an absolute 2^-24 of the largest
instead: N 2^-24 max |v| more, N the tokens seen.
"""
import math

import torch

U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
STEP = {"bf16": 0.0, "f16": 2.0 ** -24}
DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16}


def heads(x, weight, cos_sin, positions, *, eps, offset, interleaved):
    """(y, sum of the magnitudes a rotated lane is made of) of x [rows, heads, D]."""
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * (offset + weight.double())
    rot = cos_sin.shape[1]
    z, mag = y.clone(), y.abs()
    t = cos_sin.double()[positions.long().clamp(0, max(cos_sin.shape[0] - 1, 0))][:, None, :]
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = t[..., i], t[..., rot // 2 + i]
        z[..., a] = y[..., a] * c - y[..., b] * s
        z[..., b] = y[..., b] * c + y[..., a] * s
        mag[..., a] = mag[..., b] = y[..., a].abs() + y[..., b].abs()
    return z, mag


def check_heads(got, ref, mag, dtype):
    err = (got.double() - ref).abs()
    tol = U[dtype] * ref.abs() + 2.0 ** -20 * mag + STEP[dtype]
    assert bool((err <= tol).all()), float((err - tol).max())


def gather(cache, table, count, h, page):
    at = torch.as_tensor(table[: -(-count // page)], device=cache.device).long()
    return cache[at, h].reshape(-1, cache.shape[-1])[:count].double()


def attend(q, k_cache, v_cache, indptr, lens, tables, *, scale, masks=None, prefix_indptr=None, prefix_lens=None,
           prefix_tables=None):
    """(out, lse, sum p |v|, score bound, tokens seen, largest |v|), in 64 bits; rows that see nothing: 0, -inf."""
    rows, hq, d = q.shape
    hk, page = k_cache.shape[1], k_cache.shape[2]
    share = hq // hk
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device=q.device)  # noqa: E731
    out, lse, mag = z(rows, hq, d), torch.full((rows, hq), -math.inf, dtype=torch.float64, device=q.device), z(rows, hq, d)
    bound, count, vmax = z(rows, hq), z(rows, hq), z(rows, hq)
    for g in range(len(lens)):
        if lens[g] < 0:
            continue
        r0, n = indptr[g], indptr[g + 1] - indptr[g]
        for h in range(hk):
            k, v = (gather(c, tables[g], lens[g] + n, h, page) for c in (k_cache, v_cache))
            pre = 0
            for p in range(len(prefix_lens) if prefix_lens is not None else 0):
                if prefix_indptr[p] <= g < prefix_indptr[p + 1]:
                    pre = prefix_lens[p]
                    k = torch.cat([gather(k_cache, prefix_tables[p], pre, h, page), k])
                    v = torch.cat([gather(v_cache, prefix_tables[p], pre, h, page), v])
            for j in range(n):
                bits = (2 << j) - 1 if masks is None else int(masks[r0 + j]) & 0xFFFFFFFF
                see = list(range(pre + lens[g])) + [pre + lens[g] + i for i in range(n) if bits >> i & 1]
                if not see:
                    continue
                kk, vv = k[see], v[see]
                hs = slice(h * share, (h + 1) * share)
                qq = q[r0 + j, hs].double()
                s = scale * qq @ kk.T
                top = s.amax(-1, keepdim=True)
                e = torch.exp(s - top)
                l = e.sum(-1, keepdim=True)
                out[r0 + j, hs] = e @ vv / l
                mag[r0 + j, hs] = e @ vv.abs() / l
                lse[r0 + j, hs] = (top + torch.log(l))[:, 0]
                bound[r0 + j, hs] = (2 * d * 2.0 ** -24 * scale * (qq.abs() @ kk.abs().T) + 2.0 ** -21 * s.abs()).amax(-1)
                count[r0 + j, hs] = len(see)
                vmax[r0 + j, hs] = vv.abs().max()
    return out, lse, mag, bound, count, vmax


def check_attend(out, lse, ref, dtype, rows=slice(None)):
    o, want_lse, mag, bound, count, vmax = (x[rows] for x in ref)
    u = U[dtype]
    err = (out[rows].double() - o).abs()
    tol = u * o.abs() + (u + 2 * bound + 2.0 ** -18)[..., None] * mag + STEP[dtype]
    if dtype == "f16":
        tol = tol + (2.0 ** -24 * count * vmax)[..., None]
    assert bool((err <= tol).all()), ("out", float((err - tol).max()), int((~(err <= tol)).sum()))
    if lse is not None:
        none = want_lse == -math.inf
        got = lse[rows].double()
        assert bool((got[none] == -math.inf).all())
        assert bool((out[rows][none] == 0).all())
        el = (got - want_lse).abs()[~none]
        assert bool((el <= (bound + 2.0 ** -18)[~none]).all()), ("lse", float(el.max()))
