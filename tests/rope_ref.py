"""Plain implementations of rotary positions and of the 8-bit cache's rows,
from include/ss.h's definitions, in 64 bits (turns in whole numbers)."""
import math

import numpy as np

from tests import cache_ref as R

BLOCK = 16


def e4m3(x):
    """The nearest e4m3 value, ties to even, |x| <= 448; what is not finite becomes NaN."""
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        _, e = np.frexp(x)  # |x| in [2^(e-1), 2^e)
        step = np.exp2(np.maximum(e - 4, -9).astype(np.float64))
        return np.where(np.isfinite(x), np.rint(x / step) * step, np.nan)


def e4m3_of(b):
    """What bytes stand for."""
    b = np.asarray(b).astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    x = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e - 10.0))
    x = np.where((b & 127) == 127, np.nan, x)
    return np.where(b >= 128, -x, x)


def scale_of(rows):
    """The scale of a block's rows (any shape), a float."""
    x = np.abs(rows[np.isfinite(rows)])
    top = x.max() if x.size else 0.0
    e = -100
    while 448 * 2.0 ** e < top:
        e += 1
    return 2.0 ** e


def turns(rot_dim, base, scaling=None, factor=1.0, length=0.0, low=1.0, high=4.0):
    """Turns per position as fractions of 2^64 (Python integers), from long floats."""
    out = []
    for i in range(rot_dim // 2):
        f = np.longdouble(base) ** (np.longdouble(-2 * i) / rot_dim)
        if scaling == "linear":
            f /= factor
        if scaling == "by_parts":
            g = min(1.0, max(0.0, (length * float(f) / (2 * math.pi) - low) / (high - low)))
            f = f * g + f / factor * (1 - g)
        out.append(f / (2 * np.arccos(np.longdouble(-1))))
    return out


def turn(x, positions, table, rot_dim, layout, magnitude):
    """Rows x [tokens, heads, dim] turned, float64; table: turns as 64-bit integers."""
    y = np.array(x, np.float64)
    half = rot_dim // 2
    a = slice(0, half) if layout == "halves" else slice(0, rot_dim, 2)
    b = slice(half, rot_dim) if layout == "halves" else slice(1, rot_dim, 2)
    frac = np.array([[(int(p) * int(t)) % 2 ** 64 / 2.0 ** 64 for t in table] for p in positions]).reshape(len(positions), half)
    cos, sin = (magnitude * f(2 * np.pi * frac)[:, None] for f in (np.cos, np.sin))
    u, v = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = u * cos - v * sin, v * cos + u * sin
    return y


class Cache8:
    """One of the two arrays of an 8-bit cache's layer: values [pages, heads, slots, dim] and scales."""

    def __init__(self, data, scale):
        self.n, self.s = e4m3_of(data), np.array(scale, np.float64)
        self.page = self.n.shape[2]
        self.block = min(BLOCK, self.page)

    def values(self, page, head, slot):
        with np.errstate(all="ignore"):
            return self.n[page, head, slot] * self.s[page, head, np.arange(self.page)[slot] // self.block][..., None]

    def rewrite(self, page, head, block, rows):
        """rows: {slot in block: values} become the block's rows."""
        s = scale_of(np.stack(list(rows.values())))
        for slot, x in rows.items():
            self.n[page, head, block * self.block + slot] = e4m3(x / s)
        self.s[page, head, block] = s

    def append(self, table_row, base, new):
        """new [tokens, heads, dim] at the slots from base."""
        for b in range(base // self.block, -(-(base + len(new)) // self.block)):
            at = b * self.block
            e = at // self.page
            page = table_row[e] if e < len(table_row) else -1
            if not 0 <= page < len(self.n):
                continue
            inside = at % self.page // self.block
            for h in range(self.n.shape[1]):
                rows = {}
                for slot in range(self.block):
                    i = at + slot - base
                    if i < 0:
                        rows[slot] = self.values(page, h, at % self.page + slot)
                    elif i < len(new):
                        rows[slot] = new[i, h]
                self.rewrite(page, h, inside, rows)

    def compact(self, table_row, base, path):
        """The rows at base + path[j] to base + 1 + j."""
        end = base + 1 + len(path)
        for b in range((base + 1) // self.block, -(-end // self.block)):
            at = b * self.block
            src = {slot: at + slot if at + slot <= base else base + path[at + slot - base - 1]
                   for slot in range(self.block) if at + slot < end}
            if all(x == at + slot for slot, x in src.items()):
                continue
            page, inside = table_row[at // self.page], at % self.page // self.block
            for h in range(self.n.shape[1]):
                self.rewrite(page, h, inside, {slot: self.values(table_row[x // self.page], h, x % self.page)
                                               for slot, x in src.items()})


def positions(lens, news, parents=None):
    """Each new token's position; parents: per request, or None."""
    out = []
    for r, (a, n) in enumerate(zip(lens, news)):
        depth = R.paths(parents[r])[0] if parents is not None and n else range(n)
        out += [a + d for d in depth]
    return out
