"""The key-value cache and the attention over it in 64 bits, position by
position (definitions: include/gdnspec.h), and the inputs that their tests share."""
from __future__ import annotations

import math
import random

import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
LEAST = 2.0 ** -100
# every e4m3 value that is a number and not negative, ascending
_E4M3 = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8) if (e, m) != (8, 7)]


def is_small(kind):
    return kind in ("e4m3", "int8")


def quantise(row, kind):
    """(values the codes stand for without the scale, scale) of one row, float64."""
    if not bool(torch.isfinite(row).all()):
        return torch.zeros_like(row), math.nan
    a = float(row.abs().max())
    if kind == "e4m3":
        e = -100
        while a > 448 * 2.0 ** e:
            e += 1
        scale = 2.0 ** e
        table = torch.tensor(_E4M3, dtype=torch.float64)
        x = row.abs() / scale
        hi = torch.searchsorted(table, x).clamp(max=len(_E4M3) - 1)
        lo = (hi - 1).clamp(min=0)
        up = (table[hi] - x < x - table[lo]) | ((table[hi] - x == x - table[lo]) & (hi % 2 == 0))    # codes ascend: even ones end in 0
        return torch.where(up, table[hi], table[lo]) * torch.sign(row), scale
    m, e = math.frexp(a / 127)
    scale = max(LEAST, math.ldexp(math.ceil(m * 256) / 256, e))
    return torch.round(row / scale), scale


def place(table, i, x, page, pages):
    """Page and row of position x of sequence i, or None where it has no page."""
    p = int(table[i, x // page])
    return (p, x % page) if 0 <= p < pages else None


def make_cache(pages, page, G, D, kind, layout="nhd", device="cpu"):
    """k_cache, v_cache, k_scale, v_scale with NaN (or its codes) everywhere.  layout: nhd (pages, positions, heads),
    hnd (pages, heads, positions), pair (K and V halves of one tensor)."""
    dt = TYPES[kind]

    def new(shape, dtype):
        t = torch.full(shape, 0x7F if dtype.itemsize == 1 else 0x7FFF if dtype.itemsize == 2 else 0x7FC00000,
                       dtype={1: torch.int8, 2: torch.int16, 4: torch.int32}[dtype.itemsize], device=device)
        return t.view(dtype)

    if layout == "hnd":
        k, v = (new((pages, G, page, D), dt).transpose(1, 2) for _ in range(2))
        ks, vs = (new((pages, G, page), torch.float32).transpose(1, 2) for _ in range(2))
    elif layout == "pair":
        both = new((pages, 2, page, G, D), dt)
        k, v = both[:, 0], both[:, 1]
        s = new((pages, 2, page, G), torch.float32)
        ks, vs = s[:, 0], s[:, 1]
    else:
        k, v = (new((pages, page, G, D), dt) for _ in range(2))
        ks, vs = (new((pages, page, G), torch.float32) for _ in range(2))
    return (k, v, ks, vs) if is_small(kind) else (k, v, None, None)


def tables(past, n, page, seed, spare=2, extra_cols=1):
    """A page table for past[i] + n[i] positions a sequence, pages in random order; -1 behind."""
    need = [-(-(p + m) // page) for p, m in zip(past, n)]
    pages = sum(need) + spare
    order = list(range(pages))
    random.Random(seed).shuffle(order)
    t = torch.full((len(past), max(max(need), 1) + extra_cols), -1, dtype=torch.int32)
    for i, m in enumerate(need):
        t[i, :m] = torch.tensor(order[:m], dtype=torch.int32)
        order = order[m:]
    return t, pages


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32)


def pick(cache, pages, rows):
    """float64 rows [n, G, D] at (pages, rows); torch does not index 8-bit floats on the CPU."""
    return (cache.view(torch.int8)[pages, rows].view(cache.dtype) if cache.dtype.itemsize == 1 else cache[pages, rows]).double()


def held(cache, scale, where):
    """float64 rows [G, D] at (page, row)."""
    x = cache[where[0], where[1]].double()
    return x if scale is None else x * scale[where[0], where[1]].double()[:, None]


def attend(q, k, v, seen, scale, z=None):
    """One row q [H, D] over k, v [L, G, D] float64 where seen [L]: (out [H, D], sum p |v|, the largest sum |q k| scale, the largest |score|)."""
    H, D = q.shape
    G = k.shape[1]
    if not bool(seen.any()):
        return torch.zeros(H, D, dtype=torch.float64), torch.zeros(H, D, dtype=torch.float64), 0.0, 0.0
    k, v = k[seen], v[seen]
    qg = q.double().view(G, H // G, D)
    s = torch.einsum("grd,lgd->grl", qg, k) * scale
    size = torch.einsum("grd,lgd->grl", qg.abs(), k.abs()) * scale
    p = torch.softmax(s, -1)
    o = torch.einsum("grl,lgd->grd", p, v).reshape(H, D)
    a = torch.einsum("grl,lgd->grd", p, v.abs()).reshape(H, D)
    if z is not None:
        o, a = o * torch.sigmoid(z.double()), a * torch.sigmoid(z.double())
    return o, a, float(size.max()), float(s.abs().max())
