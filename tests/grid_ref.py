"""64-bit reference of rotary positions on several axes for the tests, pair by pair from
the definition, with error bounds next to the values (those of dense_ref.rotary)."""
import math

import torch

import dense_ref


def pairs(columns, span, layout):
    """(axis, place on its ladder, length of the ladder, first column, second column) of every pair."""
    half = [c // 2 for c in columns]
    total = sum(half)
    got, used, turn = [], [0] * len(columns), 0
    for i in range(total):
        if span == "dealt":
            while used[turn % len(half)] == half[turn % len(half)]:
                turn += 1
            axis, turn = turn % len(half), turn + 1
        else:
            axis = next(a for a, h in enumerate(half) if used[a] < h)
        if layout == "interleaved":
            ia, ib = 2 * i, 2 * i + 1
        elif span == "axis":
            ia = 2 * sum(half[:axis]) + used[axis]
            ib = ia + half[axis]
        else:
            ia, ib = i, i + total
        got.append((axis, used[axis], columns[axis], ia, ib) if span == "axis" else (axis, i, 2 * total, ia, ib))
        used[axis] += 1
    return got


def frequency(place, length, base=10000.0, scaling="none", factor=1.0, orig_len=0, low=1.0, high=32.0):
    if scaling == "base":
        base = base * factor ** (length / (length - 2))
    w = base ** (-2.0 * place / length)
    if scaling == "linear":
        w /= factor
    if scaling == "wavelength":
        g = min(1.0, max(0.0, (orig_len * w / (2 * math.pi) - low) / (high - low)))
        w *= g + (1 - g) / factor
    return w


def turned(x, pos, columns, span="axis", layout="half", step=None, inverse=False, amplitude=0.0, dtype=None, **kw):
    """(value, bound) of x [batch, heads, n, d] turned by pos [1 or batch, n, axes]."""
    A = amplitude or (0.1 * math.log(kw["factor"]) + 1 if kw.get("scaling") == "wavelength" and kw["factor"] > 1 else 1.0)
    x = x.double()
    out, bound = x.clone(), torch.zeros_like(x)
    for axis, place, length, ia, ib in pairs(columns, span, layout):
        p = pos[..., axis].double()
        s1 = step[axis] if step else 1.0
        ang = (-p if inverse else p) * frequency(place, length, **kw) * s1
        c, s = (A * ang.cos())[:, None], (A * ang.sin())[:, None]
        X, Y = x[..., ia], x[..., ib]
        out[..., ia], out[..., ib] = X * c - Y * s, X * s + Y * c
        # cos and sin are good to 2^-22; w step carries roundings of 2^-52 that the position multiplies
        bound[..., ia] = bound[..., ib] = abs(A) * (X.abs() + Y.abs()) * (2.0 ** -21 + 2.0 ** -50 * max(1.0, s1) * p.abs()[:, None])
    u = dense_ref.half_step(dtype) if dtype is not None else 0.0
    bound[..., :sum(columns)] += u * out[..., :sum(columns)].abs()
    return out, bound


def tile_digits(t, side):
    """(row, column) of tile positions t: base-16 digits, each a row and a column digit in base 4."""
    r, c, place = torch.zeros_like(t), torch.zeros_like(t), 1
    while place < side:
        r, c = r + place * ((t & 15) >> 2), c + place * (t & 3)
        t, place = t >> 4, place * 4
    return r, c


def places(extent, offset=None, order="raster"):
    """Positions of the grid's tokens, [n, axes]."""
    t, cols = torch.arange(math.prod(extent)), []
    rest = list(extent)
    if order == "tile":
        side = extent[-1]
        r, c = tile_digits(t % (side * side), side)
        cols, t, rest = [c, r], t // (side * side), rest[:-2]
    for e in reversed(rest):
        cols.append(t % e)
        t = t // e
    got = torch.stack(cols[::-1], -1)
    return got + torch.tensor(offset) if offset else got
