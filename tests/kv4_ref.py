"""References of the operators around a cache in 4 bits, written from their
definitions: quantisation and reservation in exact arithmetic on the host, the
cache's values in 64 bits."""
import math
from fractions import Fraction

import numpy as np
import torch

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = 16
E4M3 = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]


def nearest(x, table):
    """Index of the entry of an ascending table nearest to the fraction x >= 0, ties to the even index."""
    if x >= table[-1]:
        return len(table) - 1
    hi = next(i for i, t in enumerate(table) if t > x)
    below, above = x - Fraction(table[hi - 1]), Fraction(table[hi]) - x
    return hi if above < below or (above == below and hi % 2 == 0) else hi - 1


def quantise(x, factor=1.0):
    """(codes, scale bytes) of x [lanes], floats: exact quotients, on the host."""
    codes, scales = [], []
    f = Fraction(factor)
    for b in range(0, len(x), BLOCK):
        block = [float(v) for v in x[b:b + BLOCK]]
        if not all(math.isfinite(v) for v in block):
            scales.append(0x7F)
            codes += [None] * BLOCK
            continue
        s = nearest(max(abs(Fraction(v)) for v in block) / (6 * f), E4M3)
        scales.append(s)
        for v in block:
            c = nearest(abs(Fraction(v)) / (Fraction(E4M3[s]) * f), LEVELS) if s else 0
            codes.append(c + (8 if math.copysign(1.0, v) < 0 else 0))
    return codes, scales


def quantise_rows(x, factor=1.0):
    """The same for a tensor [..., lanes] of 16-bit floats, in 64 bits: codes (uint8, one each) and scales (e4m3 bytes);
    blocks with a NaN or infinity have scale byte 0x7F and codes 255.

    64 bits decide as the exact quotients do: a tie is a product of at most 7 bits, a lane has at most 11, and so lies on
    a tie (where the quotient is exact) or 2^-11 from it."""
    x = x.double().unflatten(-1, (-1, BLOCK))
    bad = ~torch.isfinite(x).all(-1)
    table = torch.tensor(E4M3, dtype=torch.float64, device=x.device)
    scale = _nearest(torch.where(bad, 0.0, x.abs().amax(-1)) / (6 * factor), table)
    step = table[scale][..., None] * factor
    code = _nearest(torch.where(step > 0, x.abs() / step, 0.0).nan_to_num(0.0), torch.tensor(LEVELS, dtype=torch.float64, device=x.device))
    code = code + 8 * torch.signbit(x)
    return (torch.where(bad[..., None], 255, code).flatten(-2).to(torch.uint8), torch.where(bad, 0x7F, scale).to(torch.uint8))


def _nearest(x, table):
    hi = torch.searchsorted(table, x.contiguous(), right=True).clamp(1, len(table) - 1)
    below, above = x - table[hi - 1], table[hi] - x
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return torch.where(x >= table[-1], len(table) - 1, torch.where(up, hi, hi - 1))


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(packed):
    return torch.stack([packed & 15, packed >> 4], -1).flatten(-2)


def values(packed, scales, factor=1.0):
    """What a cache stands for, in 64 bits."""
    table = torch.tensor(LEVELS + tuple(-x for x in LEVELS), dtype=torch.float64, device=packed.device)
    x = table[unpack(packed).long()].unflatten(-1, (-1, BLOCK))
    return (x * scales.view(torch.float8_e4m3fn).double()[..., None]).flatten(-2) * factor


def reserve(lens, counts, held, queue, free_pages, tables, *, rows, page, max_pages, num_pages, starts=None):
    """lp_kv_reserve group by group: a dict of its outputs (lists and arrays) and whether pages ran out or groups were bad."""
    G, ring = len(lens), len(free_pages)
    head, tail = queue
    sound = 0 <= head <= tail <= head + ring
    free, room = (tail - head, ring - (tail - head)) if sound else (0, 0)
    tables, free_pages = np.array(tables), np.array(free_pages)
    before = free_pages.copy()
    out = dict(group_indptr=[0], round_lens=[], held_out=[], positions=[-1] * rows, slots=[-1] * rows, none=False, bad=False, bad_page=not sound)
    total, taken, back, lack = 0, 0, 0, 0
    for g in range(G):
        n = max(counts[g], 0)
        holds = 0 <= held[g] <= max_pages
        idle = lens[g] < 0
        bad = counts[g] < 0 or not holds or (not idle and -(-(lens[g] + n) // page) > max_pages)
        past = total + n > rows
        need = 0 if idle or bad else max(0, -(-(lens[g] + n) // page) - held[g])
        serves = not idle and not bad and not past and (need == 0 or lack + need <= free)
        out["bad"] |= bad or past
        out["none"] |= not idle and not bad and not past and not serves
        new_held = held[g]
        if idle and holds and held[g]:
            if back + held[g] <= room:
                for i in range(held[g]):
                    free_pages[(tail + back + i) % ring] = tables[g][i]
                new_held = 0
            else:
                out["bad_page"] = True
            back += held[g]
        if serves:
            for i in range(need):
                tables[g][held[g] + i] = before[(head + lack + i) % ring]
            taken = max(taken, lack + need) if need else taken
            new_held = held[g] + need
            for j in range(n):
                t = lens[g] + j
                out["positions"][total + j] = (0 if starts is None else starts[g]) + t
                p = int(tables[g][t // page])
                if 0 <= p < num_pages:
                    out["slots"][total + j] = p * page + t % page
                else:
                    out["bad_page"] = True
        lack += need
        out["round_lens"].append(lens[g] if idle or serves else -1)
        out["held_out"].append(new_held)
        total += n
        out["group_indptr"].append(min(total, rows))
    given = 0  # what came back, up to the first group that had no room
    for g in range(G):
        if lens[g] < 0 and 0 < held[g] <= max_pages:
            if given + held[g] > room:
                break
            given += held[g]
    out.update(queue_out=[head + taken, tail + given], block_tables=tables, free_pages=free_pages)
    return out
