"""Plain implementations of the paged-cache operators, from include/ss.h's
definitions: attention and row values in 64 bits, the pages with Python lists."""
import numpy as np


def bf16(x):
    """Values as bf16 (round to nearest even), held in float32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7fff + ((u >> 16) & 1)) & 0xffff0000
    return u.astype(np.uint32).view(np.float32)


def quantise(x):
    """Rows x [..., dim] of bf16 values: (n uint8 [..., dim], step, low), fp32 arithmetic as defined."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        low, high = x.min(-1), x.max(-1)
        span = high - low
        bad = ~np.isfinite(x).all(-1) | ~np.isfinite(span)
        step = ((np.where(bad, 0, span / np.float32(15)).astype(np.float32).view(np.uint32) + np.uint32(0xffff))
                & np.uint32(0xffff0000)).view(np.float32)
        n = np.rint((x - low[..., None]) / np.where(step == 0, 1, step)[..., None])
        n = np.where((step == 0)[..., None] | bad[..., None], 0, np.minimum(n, 15)).astype(np.uint8)
    return n, np.where(bad, np.float32("nan"), step), np.where(bad, np.float32("nan"), low)


def pack(n):
    """Channels [..., dim] of 0..15 to the packed bytes [..., dim / 2]."""
    w = np.zeros(n.shape[:-1] + (n.shape[-1] // 8,), np.uint32)
    for i in range(8):
        w |= n[..., i::8].astype(np.uint32) << np.uint32(4 * (i // 2) + 16 * (i % 2))
    return np.ascontiguousarray(w).view(np.uint8).reshape(n.shape[:-1] + (n.shape[-1] // 2,))


def unpack(b):
    w = np.ascontiguousarray(b).view(np.uint32)
    n = np.zeros(b.shape[:-1] + (w.shape[-1] * 8,), np.uint8)
    for i in range(8):
        n[..., i::8] = (w >> np.uint32(4 * (i // 2) + 16 * (i % 2))) & 15
    return n


def paths(parents):
    """Per node of one tree its depth and the set of nodes it sees (itself and its ancestors)."""
    depth, line = [0], [{0}]
    for i in range(1, len(parents)):
        p = parents[i] if 0 <= parents[i] < i else 0
        depth.append(depth[p] + 1)
        line.append(line[p] | {i})
    return depth, line


def attend(q, rows, table_row, page, base, scale, window, sinks, parents, num_pages):
    """One request: q [n, heads, dim]; rows(slots' pages, slots' rows) -> (k, v, weight of v's error)
    [keys, kv heads, dim] float64.  Returns out, lse, and for tolerances sum p |v|-like / sum p and max sum |q k| scale."""
    n, heads, dim = q.shape
    out, lse = np.zeros((n, heads, dim)), np.full((n, heads), -np.inf)
    mag, reach = np.zeros((n, heads, dim)), np.zeros((n, heads))
    depth, line = paths(parents) if parents is not None else (list(range(n)), None)
    for i in range(n):
        p = base + depth[i]
        slots = np.arange(base + n)
        place = slots.copy()
        if line is None:
            see = slots <= p
        else:
            place[base:] = base + np.array(depth)
            see = slots < base
            see[[base + u for u in line[i]]] = True
        if window:
            see &= (place > p - window) | (place < sinks)
        entry = slots // page
        see &= entry < len(table_row)
        pages = np.array([table_row[e] if e < len(table_row) else -1 for e in entry], np.int64).reshape(-1)
        see &= (pages >= 0) & (pages < num_pages)
        if not see.any():
            continue
        k, v, m = rows(pages[see], slots[see] % page)
        group = heads // k.shape[1]
        for h in range(heads):
            with np.errstate(all="ignore"):
                s = (k[:, h // group] @ q[i, h]) * scale
                top = s.max()
                e = np.exp(s - top)
                out[i, h] = e @ v[:, h // group] / e.sum()
                mag[i, h] = e @ m[:, h // group] / e.sum()
                lse[i, h] = top + np.log(e.sum())
                reach[i, h] = (np.abs(k[:, h // group]) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, mag, reach


class Pages:
    """The pages' bookkeeping with lists."""

    def __init__(self, table, refs, free, page):
        self.table, self.refs, self.free, self.page = [list(r) for r in table], list(refs), list(free), page

    def hole(self, e):
        return not 0 <= e < len(self.refs)

    def _most(self):
        return len(self.table[0]) * self.page

    def reserve(self, rows, start, stop):
        status, short = [], False
        for r, a, b in zip(rows, start, stop):
            if not (0 <= r < len(self.table) and 0 <= a <= b <= self._most()):
                status.append(4)
                continue
            need = [e for e in range(a // self.page, -(-b // self.page)) if self.hole(self.table[r][e])] if a < b else []
            short = short or len(need) > len(self.free)
            if need and short:
                status.append(6)
                continue
            for e in need:
                p = self.free.pop()
                self.table[r][e], self.refs[p] = p, 1
            status.append(0)
        return status

    def fork(self, parent, child, length):
        """Statuses, and the page copies (source, destination, slots)."""
        status, copies, short = [], [], False
        for a, b, n in zip(parent, child, length):
            inside = 0 <= a < len(self.table) and 0 <= b < len(self.table) and 0 <= n <= self._most()
            if not inside or any(e >= 0 for e in self.table[b]):
                status.append(4)
                continue
            full, rest = divmod(n, self.page)
            need = rest > 0 and not self.hole(self.table[a][full])
            short = short or (need and not self.free)
            if need and short:
                status.append(6)
                continue
            row = [e if not self.hole(e) else -1 for e in self.table[a][:full]]
            for e in row:
                if e >= 0:
                    self.refs[e] += 1
            if need:
                p = self.free.pop()
                self.refs[p] = 1
                copies.append((self.table[a][full], p, rest))
                row.append(p)
            self.table[b] = row + [-1] * (len(self.table[b]) - len(row))
            status.append(0)
        return status, copies

    def trim(self, rows, length, window, sinks):
        status, dropped = [], []
        for r, n in zip(rows, length):
            if not (0 <= r < len(self.table) and n >= 0):
                status.append(4)
                continue
            bad = False
            for e, p in enumerate(self.table[r]):
                keep = any(s < sinks or window == 0 or s >= n - window
                           for s in range(e * self.page, min((e + 1) * self.page, n)))
                if p < 0 or keep:
                    continue
                self.table[r][e] = -1
                if self.hole(p) or self.refs[p] <= 0:
                    bad = True
                else:
                    self.refs[p] -= 1
                    dropped.append(p)
            status.append(5 - 2 if bad else 0)
        seen = set()
        for p in reversed(dropped):
            if self.refs[p] == 0 and p not in seen:
                seen.add(p)
                self.free.append(p)
        return status
