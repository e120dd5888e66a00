"""Rotary positions, alone and with the cache's append, and the rows of the
8-bit cache on the GPU, against tests/rope_ref.py.

Tolerances.  A turned channel is one bf16 rounding (2^-8 of it at most) of fp32
sums: the angle is off by 2^-25 of half a turn (2^-23.3 radians), sine and
cosine by two units of 2^-24, magnitude, product and sum by one each, so by less
than 2^-21 of |x| + |y| times the magnitude.  What is cached in 8 bits is
defined bit by bit.  Keys on their way into 8 or 4 bits are bf16 roundings of
sums that are off by 2^-33 of |x| + |y|: compared bit by bit with the 64-bit
sums' after an assertion that none of these lies that near to where a rounding
turns.
"""
import random

import numpy as np
import pytest

from tests import cache_ref as R
from tests import rope_ref as P
from tests.test_cache_gpu import ints, np32, random_parents, ss  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def half(rng, *shape, spread=1.0):
    return torch.from_numpy(R.bf16(rng.standard_normal(shape) * spread)).to(torch.bfloat16).cuda()


def offsets_of(news):
    return [sum(news[:i]) for i in range(len(news) + 1)]


def check_turned(got, x, at, rope, layout, magnitude, what=""):
    table = [int(v) for v in rope.turns.cpu().numpy().view(np.uint64)]
    x64 = np32(x).astype(np.float64)
    want = P.turn(x64, at, table, rope.rot_dim, layout, magnitude)
    pair = P.turn(np.abs(x64), [0] * len(at), table, rope.rot_dim, layout, 1.0)
    h = rope.rot_dim // 2
    a, b = (slice(0, h), slice(h, 2 * h)) if layout == "halves" else (slice(0, 2 * h, 2), slice(1, 2 * h, 2))
    both = np.zeros_like(pair)
    both[..., a] = both[..., b] = pair[..., a] + pair[..., b]
    err = np.abs(np32(got) - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * both * abs(magnitude)).all(), (what, err.max())
    assert np.array_equal(np32(got)[..., 2 * h:], np32(x)[..., 2 * h:])


def keys_to_cache(x, at, rope, layout, magnitude):
    """The keys that ss_rope_append puts into 8 or 4 bits, from 64-bit sums."""
    table = [int(v) for v in rope.turns.cpu().numpy().view(np.uint64)]
    x64 = np32(x).astype(np.float64)
    want = P.turn(x64, at, table, rope.rot_dim, layout, magnitude)
    h = rope.rot_dim // 2
    a, b = (slice(0, h), slice(h, 2 * h)) if layout == "halves" else (slice(0, 2 * h, 2), slice(1, 2 * h, 2))
    off = np.zeros_like(want)
    off[..., a] = off[..., b] = 2.0 ** -33 * abs(magnitude) * (np.abs(x64[..., a]) + np.abs(x64[..., b]))
    off[np.array(at) == 0] = 0.0  # cosine 1 and sine 0 are exact, and so are two products that one of them takes part in
    y, low, high = (R.bf16((want + d).astype(np.float32)) for d in (0, -off, off))
    assert np.array_equal(low, high)
    return torch.from_numpy(y).to(torch.bfloat16).cuda()


SHAPES = [  # dim, rot_dim, heads, kv heads
    (128, 128, 4, 2), (128, 64, 3, 1), (64, 64, 8, 8), (80, 80, 5, 5), (96, 24, 4, 2), (80, 20, 2, 1), (8, 8, 1, 1),
    (16, 2, 3, 3), (128, 126, 2, 2), (40, 36, 7, 1), (72, 16, 1, 3)]


@pytest.mark.parametrize("layout", ["halves", "interleaved"])
@pytest.mark.parametrize("dim,rot,heads,kv", SHAPES)
def test_queries_and_keys(ss, dim, rot, heads, kv, layout):
    rng = np.random.default_rng(dim * 1000 + rot)
    rope = ss.Rope(dim, rot_dim=rot, layout=layout, base=500.0, magnitude=1.25)
    lens, news = [0, 7, 1000000, 33], [1, 0, 37, 16]
    total = sum(news)
    qkv = half(rng, total + 3, heads + 2 * kv, dim)  # three rows behind the last request
    q, k = qkv[:, :heads], qkv[:, heads:heads + kv]
    q_out, k_out = torch.full((total + 3, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full(
        (kv, total + 3, dim), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    st = ints([-1] * 4)
    args = dict(token_offsets=ints(offsets_of(news)), max_tokens=37)
    ss.ss_rope(rope, q, q_out, k, k_out, ints(lens), st, **args)
    assert st.tolist() == [0] * 4
    at = P.positions(lens, news)
    check_turned(q_out[:total], q[:total], at, rope, layout, 1.25)
    check_turned(k_out[:total], k[:total], at, rope, layout, 1.25)
    assert (q_out[total:] == 7).all() and (k_out[total:] == 7).all()
    # in place; and one of the two alone
    mine = qkv.clone()
    ss.ss_rope(rope, mine[:, :heads], mine[:, :heads], mine[:, heads:heads + kv], mine[:, heads:heads + kv], ints(lens), st, **args)
    assert torch.equal(mine[:total, :heads], q_out[:total]) and torch.equal(mine[:total, heads:heads + kv], k_out[:total])
    assert torch.equal(mine[:, heads + kv:], qkv[:, heads + kv:]) and torch.equal(mine[total:], qkv[total:])
    alone = torch.zeros_like(q_out)
    ss.ss_rope(rope, q, alone, None, None, ints(lens), st, **args)
    assert torch.equal(alone[:total], q_out[:total])
    alone = torch.zeros_like(k_out)
    ss.ss_rope(rope, None, None, k, alone, ints(lens), st, **args)
    assert torch.equal(alone[:total], k_out[:total])


@pytest.mark.parametrize("scaling", [dict(), dict(scaling="linear", factor=4.0), dict(
    scaling="by_parts", factor=8.0, length=8192, low=1.0, high=4.0)])
def test_positions_of_ones_own_far_and_negative(ss, scaling):
    rng = np.random.default_rng(5)
    rope = ss.Rope(128, base=500000.0, **scaling)
    at = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 123456789, 5, 5, 1 << 30, 77, 3]
    q = half(rng, 12, 2, 128)
    out, st = torch.empty_like(q), ints([-1, -1])
    ss.ss_rope(rope, q, out, None, None, None, st, token_offsets=ints([0, 5, 12]), max_tokens=7, positions=ints(at))
    assert st.tolist() == [0, 0]
    check_turned(out, q, at, rope, "halves", 1.0)
    # against angles in 64-bit floats, at positions where these still have the bits
    f = [500000.0 ** (-i / 64) for i in range(64)]
    if scaling.get("scaling") == "linear":
        f = [x / 4 for x in f]
    if not scaling or "linear" in scaling.values():
        angle = np.outer(at, f)
        x = np32(q).astype(np.float64)
        u, v = x[..., :64], x[..., 64:]
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        want = np.concatenate([u * c - v * s, v * c + u * s], -1)
        # the frequency's 2^-48 (test_frequencies) times 2^31 positions of a radian
        assert (np.abs(np32(out) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -16 * 8).all()


@pytest.mark.parametrize("seed", range(3))
def test_trees_stand_at_their_depths(ss, seed):
    rng, pr = np.random.default_rng(seed), random.Random(seed)
    lens, news = [100, 0, 5000, 31], [64, 1, 17, 40]
    parents = [random_parents(pr, n) for n in news]
    if seed == 1:
        parents[0] = [0] + list(range(63))  # a chain
    if seed == 2:
        parents[3] = [0] * 40  # all children of the root
    rope = ss.Rope(64, layout="interleaved")
    q = half(rng, sum(news), 3, 64)
    out, st = torch.empty_like(q), ints([-1] * 4)
    flat = [p for row in parents for p in row]
    ss.ss_rope(rope, q, out, None, None, ints(lens), st, token_offsets=ints(offsets_of(news)), max_tokens=64,
               parents=ints(flat))
    assert st.tolist() == [0] * 4
    at = P.positions(lens, news, parents)
    check_turned(out, q, at, rope, "interleaved", 1.0)
    # a parent that is none: the node is the root's child
    bad = list(flat)
    bad[10], bad[64 + 1 + 3] = 10, -1
    for r, i, first in ((0, 10, 0), (2, 3, 65)):
        parents[r] = list(parents[r])
        parents[r][i] = 0
    ss.ss_rope(rope, q, out, None, None, ints(lens), st, token_offsets=ints(offsets_of(news)), max_tokens=64,
               parents=ints(bad))
    assert st.tolist() == [4, 0, 4, 0]
    check_turned(out, q, P.positions(lens, news, parents), rope, "interleaved", 1.0)


def test_requests_that_cannot_be(ss):
    rng = np.random.default_rng(1)
    rope = ss.Rope(32)
    q = half(rng, 70, 1, 32)

    def call(offsets, lens, most, **kw):
        out, st = torch.full_like(q, 7.0), ints([-1] * len(lens))
        ss.ss_rope(rope, q, out, None, None, ints(lens), st, token_offsets=ints(offsets), max_tokens=most, **kw)
        return out, st.tolist()

    out, st = call([0, 3, 10, 11, 11], [5, 5, -1, 5], 6)
    assert st == [0, 4, 4, 0]  # too many tokens; a negative length; no tokens
    assert (out[3:] == 7).all() and not (out[:3] == 7).all()
    out, st = call([-1, 3, 2, 71], [5, 5, 5], 80)
    assert st == [4, 4, 4] and (out == 7).all()
    out, st = call([0, 65, 70], [5, 5], 65, parents=ints([0] + [0] * 64 + [0] * 5))
    assert st == [4, 0] and (out[:65] == 7).all()
    # nothing at all
    st = ints([-1])
    ss.ss_rope(rope, q[:0], q[:0], None, None, ints([3]), st, token_offsets=ints([0, 0]), max_tokens=0)
    assert st.tolist() == [0]
    # one token each, by default
    out, st = torch.empty_like(q[:3]), ints([-1] * 3)
    ss.ss_rope(rope, q[:3], out, None, None, ints([9, 2, 0]), st)
    assert st.tolist() == [0] * 3
    check_turned(out, q[:3], [9, 2, 0], rope, "halves", 1.0)


# ------------------------------------------------------- rows of 8 bits --

def cache8(ss, rng, pages, heads, page, dim, layers=1, order="phsd"):
    blocks = max(1, page // 16)
    names = [0] + [1 + order[:3].index(x) for x in "phs"] + [4]
    front = [0] + ["phs".index(x) + 1 for x in order[:3]] + [4]
    parts = []
    for _ in range(2):
        b = rng.integers(0, 256, (layers, pages, heads, page, dim), dtype=np.uint8)
        b[(b & 127) == 127] = 0x38
        parts.append(torch.from_numpy(b).cuda().permute(*front).contiguous().permute(*names).view(torch.float8_e4m3fn))
    scales = [torch.from_numpy(np.exp2(rng.integers(-10, -6, (layers, pages, heads, blocks))).astype(np.float32)).cuda()
              for _ in range(2)]
    return ss.KVCache(*parts, *scales)


def plain8(cache, layer=0):
    return [P.Cache8(x[layer].view(torch.uint8).cpu().numpy(), s[layer].cpu().numpy())
            for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]


def same8(cache, want, layer=0):
    for x, s, w in ((cache.k, cache.k_scale, want[0]), (cache.v, cache.v_scale, want[1])):
        assert np.array_equal(s[layer].cpu().numpy().astype(np.float64), w.s, equal_nan=True)
        got = P.e4m3_of(x[layer].view(torch.uint8).cpu().numpy())
        assert np.array_equal(got, w.n, equal_nan=True), np.argwhere(~((got == w.n) | (np.isnan(got) & np.isnan(w.n))))[:5]


class Rows:
    """Requests over a shuffled page table, and their new keys and values."""

    def __init__(self, ss, seed, lens, news, heads, page, dim, order="phsd", layers=1, holes=()):
        rng = np.random.default_rng(seed)
        need = [-(-(a + b) // page) for a, b in zip(lens, news)]
        used = sum(need)
        perm = rng.permutation(used + 2).tolist()
        self.table, at = [], 0
        for n in need:
            self.table.append(perm[at:at + n] + [-1] * (max(need + [1]) - n))
            at += n
        for r, e in holes:
            self.table[r][e] = -1
        self.lens, self.news, self.offsets, self.rng = lens, news, offsets_of(news), rng
        self.cache = cache8(ss, rng, used + 2, heads, page, dim, layers, order)
        kv = half(rng, sum(news), 2 * heads, dim)
        kv *= torch.exp2(torch.from_numpy(rng.integers(-4, 5, sum(news))).cuda())[:, None, None].to(torch.bfloat16)
        self.k, self.v = kv[:, :heads], kv[:, heads:]
        self.st = ints([-1] * len(lens))
        self.kw = dict(token_offsets=ints(self.offsets), max_tokens=max(news + [0]))

    def plain(self, want, k=None, v=None):
        for x, w in ((self.k if k is None else k, want[0]), (self.v if v is None else v, want[1])):
            x = np32(x).astype(np.float64)
            for r, a in enumerate(self.lens):
                w.append(self.table[r], a, x[self.offsets[r]:self.offsets[r + 1]])


@pytest.mark.parametrize("heads,page,dim,order", [(1, 8, 16, "phsd"), (2, 16, 128, "phsd"), (8, 64, 128, "shpd"),
                                                  (3, 32, 80, "hpsd"), (5, 128, 64, "pshd"), (2, 8, 96, "sphd")])
def test_append_and_read(ss, heads, page, dim, order):
    lens = [0, 1, 15, 16, 17, 100, 3, 250, 31]
    news = [1, 1, 1, 5, 40, 0, 70, 8, 2]
    p = Rows(ss, heads * page, lens, news, heads, page, dim, order=order)
    want = plain8(p.cache)
    p.plain(want)
    ss.ss_cache_append(p.cache, 0, p.k, p.v, ints(p.table), ints(lens), p.st, **p.kw)
    assert p.st.tolist() == [0] * len(lens)
    same8(p.cache, want)
    again = [x.clone() for x in (p.cache.k.view(torch.uint8), p.cache.v.view(torch.uint8), p.cache.k_scale, p.cache.v_scale)]
    ss.ss_cache_append(p.cache, 0, p.k, p.v, ints(p.table), ints(lens), p.st, **p.kw)
    for x, y in zip(again, (p.cache.k.view(torch.uint8), p.cache.v.view(torch.uint8), p.cache.k_scale, p.cache.v_scale)):
        assert torch.equal(x, y)
    # back, from the first token on
    upto = [a + b for a, b in zip(lens, news)]
    k, v = (torch.full((sum(upto) + 1, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ss.ss_cache_read(p.cache, 0, k, v, ints(p.table), ints([0] * len(lens)), p.st, token_offsets=ints(offsets_of(upto)),
                     max_tokens=max(upto))
    assert p.st.tolist() == [0] * len(lens) and (k[-1] == 7).all()
    at = 0
    for r, n in enumerate(upto):
        for i in range(n):
            where = (p.table[r][i // page], slice(None), i % page)
            # e4m3 times a power of two: no rounding
            assert np.array_equal(np32(k[at + i]), want[0].values(*where)) and np.array_equal(np32(v[at + i]), want[1].values(*where))
        at += n


def test_append_one_token_after_another(ss):
    """A step at a time, as decoding writes: the plain form takes the same steps."""
    p = Rows(ss, 3, [0, 13, 60], [70, 70, 70], 2, 16, 64)
    want = plain8(p.cache)
    at = list(p.lens)
    for step in (1, 1, 2, 5, 1, 16, 7, 31, 1):
        rows = [o + a - b for o, a, b in zip(p.offsets, at, p.lens)]
        pick = torch.cat([torch.arange(x, x + step) for x in rows]).cuda()
        k, v = p.k[pick].contiguous(), p.v[pick].contiguous()
        for x, w in ((k, want[0]), (v, want[1])):
            for r in range(3):
                w.append(p.table[r], at[r], np32(x[r * step:(r + 1) * step]).astype(np.float64))
        ss.ss_cache_append(p.cache, 0, k, v, ints(p.table), ints(at), p.st, token_offsets=ints([0, step, 2 * step, 3 * step]),
                           max_tokens=step)
        assert p.st.tolist() == [0] * 3
        same8(p.cache, want)
        at = [a + step for a in at]
        if step == 5:
            at = [a - 3 for a in at]  # three drafts were rejected


def test_values_that_are_not_finite_and_scales_of_others(ss):
    p = Rows(ss, 9, [0, 5, 20], [9, 6, 4], 2, 16, 32)
    k = p.k.clone()
    k[0, 0, 3], k[1, 0, 0], k[2, 1], k[5, 0, 31] = float("nan"), float("inf"), float("-inf"), 3e38
    k[9:15] = 0
    v = p.v.clone()
    v[:9] *= 2.0 ** -60
    v[:9] *= 2.0 ** -55  # scales end at 2^-100
    for s, where, x in ((p.cache.k_scale, (0, p.table[1][0], 0, 0), 0.3), (p.cache.k_scale, (0, p.table[1][0], 1, 0), float("nan")),
                        (p.cache.v_scale, (0, p.table[2][1], 0, 0), float("inf")), (p.cache.v_scale, (0, p.table[2][1], 1, 0), -2.0)):
        s[where] = x
    want = plain8(p.cache)
    for x, w in ((k, want[0]), (v, want[1])):
        x = np32(x).astype(np.float64)
        for r, a in enumerate(p.lens):
            # (the old values as fp32 makes them: scale times e4m3 rounded once)
            w.s = w.s.astype(np.float32).astype(np.float64)
            w.append(p.table[r], a, x[p.offsets[r]:p.offsets[r + 1]])
    ss.ss_cache_append(p.cache, 0, k, v, ints(p.table), ints(p.lens), p.st, **p.kw)
    assert p.st.tolist() == [0] * 3
    same8(p.cache, want)


def test_append_into_holes_and_beyond(ss):
    p = Rows(ss, 4, [10, 40, 0, 5], [30, 30, 3, 2], 2, 16, 64, holes=[(0, 1), (1, 4)])
    p.table[2][0] = 10 ** 6
    short = [row[:5] for row in p.table]
    want = plain8(p.cache)
    for x, w in ((p.k, want[0]), (p.v, want[1])):
        x = np32(x).astype(np.float64)
        for r, a in enumerate(p.lens):
            w.append(short[r], a, x[p.offsets[r]:p.offsets[r + 1]])
    lens = list(p.lens)
    ss.ss_cache_append(p.cache, 0, p.k, p.v, ints(short), ints(lens), p.st, **p.kw)
    assert p.st.tolist() == [3, 3, 3, 0]
    same8(p.cache, want)
    ss.ss_cache_append(p.cache, 0, p.k, p.v, ints(short), ints([-1, 0, 0, 0]), p.st, token_offsets=ints([0, 5, 40, 39, 70]),
                       max_tokens=9, table_rows=ints([0, 1, 2, 4]))
    assert p.st.tolist() == [4, 4, 4, 4]
    same8(p.cache, want)


def test_layers_are_apart(ss):
    p = Rows(ss, 6, [3, 30], [20, 9], 2, 16, 64, layers=3, order="hspd")
    want = [plain8(p.cache, i) for i in range(3)]
    p.plain(want[1])
    ss.ss_cache_append(p.cache, 1, p.k, p.v, ints(p.table), ints(p.lens), p.st, **p.kw)
    for i in range(3):
        same8(p.cache, want[i], i)


# ------------------------------------------------------- both in one call --

def any_cache(ss, rng, fmt, pages, heads, page, dim):
    if fmt == "fp8":
        return cache8(ss, rng, pages, heads, page, dim)
    from tests.test_cache_gpu import make_cache
    return make_cache(ss, rng, fmt, pages, heads, page, dim)


def parts(c):
    return [x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x for x in (c.k, c.v, c.k_scale, c.v_scale) if x is not None]


@pytest.mark.parametrize("fmt", ["bf16", "int4", "fp8"])
@pytest.mark.parametrize("page,dim,rot,heads,kv,layout,mode", [
    (16, 128, 128, 8, 2, "halves", "row"), (64, 64, 32, 5, 5, "interleaved", "tree"), (8, 96, 24, 3, 1, "halves", "positions"),
    (32, 32, 20, 2, 1, "halves", "row"), (128, 64, 64, 0, 4, "halves", "tree"), (16, 128, 64, 32, 8, "interleaved", "one")])
def test_rope_append_is_the_two_calls(ss, fmt, page, dim, rot, heads, kv, layout, mode):
    rng, pr = np.random.default_rng(rot), random.Random(rot)
    lens, news = [0, 30, 16, 100, 7], [33, 1, 0, 64, 9]
    if mode == "one":
        news = [1] * 5
    total, offsets = sum(news), offsets_of(news)
    need = [-(-(a + b) // page) for a, b in zip(lens, news)]
    perm = rng.permutation(sum(need)).tolist()
    table = [[perm.pop() for _ in range(n)] + [-1] * (max(need) - n) for n in need]
    cache = any_cache(ss, rng, fmt, sum(need), kv, page, dim)
    rope = ss.Rope(dim, rot_dim=rot, layout=layout, base=1000.0, magnitude=0.75)
    qkv = half(rng, total + 2, heads + 2 * kv, dim)
    q, k, v = (x[:total] for x in (qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]))
    at = {}
    if mode == "tree":
        trees = [random_parents(pr, n) if n else [] for n in news]
        at["parents"], places = ints(sum(trees, [])), P.positions(lens, news, trees)
    elif mode == "positions":
        places = rng.integers(-2 ** 31, 2 ** 31, total).tolist()
        at["positions"] = ints(places)
    else:
        places = P.positions(lens, news)
    rows = {} if mode == "one" else dict(token_offsets=ints(offsets), max_tokens=max(news))
    t, n, st, st2 = ints(table), ints(lens), ints([-1] * 5), ints([-1] * 5)
    # the two calls (8 and 4 bits: with the keys from closer sums)
    q_want, turned = torch.empty(total, heads, dim, dtype=torch.bfloat16, device="cuda"), torch.empty_like(k)
    before = [x.clone() for x in parts(cache)]
    ss.ss_rope(rope, *((q, q_want) if heads else (None, None)), k, turned, n, st, **rows, **at)
    if fmt != "bf16":
        close = keys_to_cache(k, places, rope, layout, 0.75)
        assert (np.abs(np32(close) - np32(turned)) <= 2.0 ** -7 * np.abs(np32(close)) + 2.0 ** -19).all()
        turned = close
    ss.ss_cache_append(cache, 0, *(x.contiguous() for x in (turned, v)), t, n, st2, **rows)
    assert st.tolist() == [0] * 5 and st2.tolist() == [0] * 5
    want = [x.clone() for x in parts(cache)]
    # and the one
    for x, y in zip(parts(cache), before):
        x.copy_(y)
    q_out = torch.full((total + 2, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    kv_before, st = qkv.clone(), ints([-1] * 5)
    ss.ss_rope_append(rope, cache, 0, *((q, q_out[:total]) if heads else (None, None)), k, v, t, n, st, **rows, **at)
    assert st.tolist() == [0] * 5
    assert torch.equal(q_out[:total], q_want) and (q_out[total:] == 7).all()
    for x, y in zip(parts(cache), want):
        assert torch.equal(x.view(torch.int16) if x.dtype == torch.bfloat16 else x,
                           y.view(torch.int16) if y.dtype == torch.bfloat16 else y)
    assert torch.equal(qkv, kv_before)
    if heads:  # in place
        ss.ss_rope_append(rope, cache, 0, q, q, k, v, t, n, st, **rows, **at)
        assert torch.equal(q, q_want) and torch.equal(qkv[:, heads:], kv_before[:, heads:])


@pytest.mark.parametrize("fmt", ["bf16", "int4", "fp8"])
def test_rope_append_statuses(ss, fmt):
    rng = np.random.default_rng(8)
    cache = any_cache(ss, rng, fmt, 12, 2, 16, 64)
    rope = ss.Rope(64)
    q, k, v = (half(rng, 80, h, 64) for h in (4, 2, 2))
    table = ints([[0, 1, 2], [3, -1, 4], [5, 6, 7], [8, 9, 10]])
    before = [x.clone() for x in parts(cache)]
    out, st = torch.full_like(q, 7.0), ints([-1] * 4)
    # a hole; a parent that is none, whose request has a hole as well (the larger code wins); a table row outside
    parents = [0] * 80
    parents[20 + 3] = 3
    ss.ss_rope_append(rope, cache, 0, q, out, k, v, table, ints([0, 0, 40, 0]), st, token_offsets=ints([0, 20, 40, 50, 52]),
                      max_tokens=20, parents=ints(parents), table_rows=ints([1, 1, 2, 4]))
    assert st.tolist() == [3, 4, 3, 4]
    assert not (out[:50] == 7).all(-1).any() and (out[50:] == 7).all()
    changed = [(x != y).flatten(2).any(-1)[0] for x, y in zip(parts(cache)[:2], before)]
    for c in changed:
        assert sorted(c.nonzero().flatten().tolist()) == [3, 7]
    # more than 64 nodes, more tokens than said
    for x, y in zip(parts(cache), before):
        x.copy_(y)
    out.fill_(7.0)
    ss.ss_rope_append(rope, cache, 0, q, out, k, v, table, ints([0, 0]), st[:2], token_offsets=ints([0, 65, 68]), max_tokens=65,
                      parents=ints([0] * 80), table_rows=ints([3, 2]))
    assert st.tolist()[:2] == [4, 0] and (out[:65] == 7).all() and (out[68:] == 7).all()
    assert not (parts(cache)[0] != before[0]).flatten(2).any(-1)[0][[8, 9, 10]].any()


def test_rope_append_in_a_graph_and_on_a_stream(ss):
    p = Rows(ss, 12, [0, 20, 47], [16, 1, 9], 2, 16, 64)
    rope = ss.Rope(64)
    q, out = half(p.rng, sum(p.news), 4, 64), torch.empty(sum(p.news), 4, 64, dtype=torch.bfloat16, device="cuda")
    state = [x.clone() for x in parts(p.cache)]
    table, lens = ints(p.table), ints(p.lens)
    ss.ss_rope_append(rope, p.cache, 0, q, out, p.k, p.v, table, lens, p.st, **p.kw)
    want = [x.clone() for x in parts(p.cache)] + [out.clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ss.ss_rope_append(rope, p.cache, 0, q, out, p.k, p.v, table, lens, p.st, **p.kw)
    for _ in range(2):
        for x, y in zip(parts(p.cache), state):
            x.copy_(y)
        out.zero_()
        p.st.fill_(-1)
        graph.replay()
        assert p.st.tolist() == [0] * 3
        for x, y in zip(parts(p.cache) + [out], want):
            assert torch.equal(x, y)
    for x, y in zip(parts(p.cache), state):
        x.copy_(y)
    torch.cuda.synchronize()
    ss.ss_rope_append(rope, p.cache, 0, q, out, p.k, p.v, table, lens, p.st, stream=side, **p.kw)
    side.synchronize()
    for x, y in zip(parts(p.cache) + [out], want):
        assert torch.equal(x, y)


# ------------------------------------------------------------- the pages --

@pytest.mark.parametrize("page,heads,dim,layers", [(16, 2, 64, 2), (8, 3, 96, 1), (64, 8, 128, 3), (32, 1, 16, 1)])
def test_compact_of_8_bits(ss, page, heads, dim, layers):
    rng, pr = np.random.default_rng(page), random.Random(page)
    lens = [0, 5, 15, 16, 30, 100, 31, 7, 14]
    paths = [[], [1, 2, 3], [1, 3, 20], [2], sorted(pr.sample(range(1, 64), 40)), [5, 9, 33], list(range(1, 40)), [63], [1, 2, 9]]
    width, n = 64, len(lens)
    need = [-(-(a + 64) // page) for a in lens]
    perm = rng.permutation(sum(need) + 1).tolist()
    table = [[perm.pop() for _ in range(x)] + [-1] * (max(need) - x) for x in need]
    cache = cache8(ss, rng, sum(need) + 1, heads, page, dim, layers)
    # blocks of very different scales
    for s in (cache.k_scale, cache.v_scale):
        s *= torch.exp2(torch.from_numpy(rng.integers(-6, 7, tuple(s.shape))).cuda())
    pool = ss.alloc_pool(n, max(need), sum(need) + 1, page)
    pool.page_table.copy_(ints(table))
    want = [plain8(cache, i) for i in range(layers)]
    for layer in want:
        for w in layer:
            for r in range(n):
                if r != 7:
                    w.compact(table[r], lens[r], paths[r])
    verified = [0] * n
    verified[7] = 2
    new_len, st = ints([-1] * n), ints([-1] * n)
    ss.ss_pages_compact(pool, cache, ints(lens), ints([p + [-1] * (width - len(p)) for p in paths]),
                        ints([len(p) for p in paths]), ints(verified), new_len, st)
    assert st.tolist() == [0] * 7 + [2, 0]
    assert new_len.tolist() == [a + (1 + len(p) if r != 7 else 0) for r, (a, p) in enumerate(zip(lens, paths))]
    for i in range(layers):
        same8(cache, want[i], i)
    # a path that goes back, a slot in a hole, a count past the path: nothing moves
    bad = [[3, 2], [1, 2], [1, 2]]
    pool.page_table[1, (lens[1] + 1) // page] = -1
    ss.ss_pages_compact(pool, cache, ints(lens[:3]), ints([p + [-1] * (width - 2) for p in bad]), ints([2, 2, 65]), None,
                        new_len[:3], st[:3])
    assert st.tolist()[:3] == [3, 3, 4] and new_len.tolist()[:3] == lens[:3]
    for i in range(layers):
        same8(cache, want[i], i)


@pytest.mark.parametrize("page", [8, 16, 64])
def test_fork_of_8_bits(ss, page):
    rng = np.random.default_rng(page)
    lens = [page * 2, page + 3, 17, 1]
    cache = cache8(ss, rng, 20, 3, page, 48, layers=2)
    pool = ss.alloc_pool(8, 4, 20, page)
    st = ints([-1] * 4)
    ss.ss_pages_reserve(pool, ints([0] * 4), ints(lens), st)
    ss.ss_pages_fork(pool, cache, ints([0, 1, 2, 3]), ints([4, 5, 6, 7]), ints(lens), st)
    assert st.tolist() == [0] * 4
    table = pool.page_table.tolist()
    for layer in range(2):
        for w in plain8(cache, layer):
            for r, n in enumerate(lens):
                for s in range(n):
                    a, b = (w.values(table[x][s // page], slice(None), s % page) for x in (r, r + 4))
                    assert np.array_equal(a, b)
    for r, n in enumerate(lens):
        assert (table[r][n // page] != table[r + 4][n // page]) == (n % page > 0)


def test_all_calls_on_the_longest_rows(ss):
    """Slots whose addresses pass 32 bits, in a cache of which few pages are there."""
    heads, page, dim = 2, 1024, 128
    row = 2 ** 21  # bytes between pages: 1.5k of them are more than 2^31 apart
    pages = 1600
    free = torch.cuda.mem_get_info()[0]
    if free < 4 * pages * row:
        pytest.skip("needs %d GB" % (4 * pages * row >> 30))
    big = [torch.empty(pages * row, dtype=torch.uint8, device="cuda") for _ in range(2)]
    shape, strides = (1, pages, heads, page, dim), (pages * row, row, page * dim, dim, 1)
    views = [x.as_strided(shape, strides).view(torch.float8_e4m3fn) for x in big]
    scales = [torch.zeros(1, pages, heads, page // 16, device="cuda") for _ in range(2)]
    cache = ss.KVCache(*views, *scales)
    rng = np.random.default_rng(0)
    k, v = half(rng, 40, heads, dim), half(rng, 40, heads, dim)
    lens = [1599 * 1024 + 1000 - 1024, 1590 * 1024 + 5]
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(2, -1).contiguous()
    st = ints([-1, -1])
    kw = dict(token_offsets=ints([0, 30, 40]), max_tokens=30)
    for x in views:  # the rows before the new ones in their blocks
        x.view(torch.uint8)[0, 1590:].zero_()
    ss.ss_rope_append(ss.Rope(dim), cache, 0, None, None, k, v, table, ints(lens), st, **kw)
    assert st.tolist() == [0, 0]
    back, back_v = torch.empty_like(k), torch.empty_like(v)
    ss.ss_cache_read(cache, 0, back, back_v, table, ints(lens), st, **kw)
    at = P.positions(lens, [30, 10])
    rope = ss.Rope(dim)
    want = P.turn(np32(k).astype(np.float64), at, [int(t) for t in rope.turns.cpu().numpy().view(np.uint64)], dim, "halves", 1.0)
    # e4m3's half step and the bf16 before it; 2^-10 of the block's scale, which is at most 2^-6 here
    assert (np.abs(np32(back) - want) <= (2.0 ** -4 + 2.0 ** -7) * np.abs(want) + 2.0 ** -15).all()
    err = np.abs(np32(back_v) - np32(v))
    assert (err <= 2.0 ** -4 * np.abs(np32(v)) + 2.0 ** -15).all()


@pytest.mark.parametrize("fmt", ["bf16", "int4", "fp8"])
def test_long_chunks_and_generous_limits(ss, fmt):
    """Many chunks of tokens of a request; limits far above the numbers of tokens."""
    rng = np.random.default_rng(11)
    lens, news, heads, page, dim = [5, 70], [21000, 3], 1, 64, 64
    need = [-(-(a + b) // page) for a, b in zip(lens, news)]
    perm = rng.permutation(sum(need)).tolist()
    table = ints([[perm.pop() for _ in range(n)] + [-1] * (max(need) - n) for n in need])
    cache = any_cache(ss, rng, fmt, sum(need), heads, page, dim)
    before = [x.clone() for x in parts(cache)]
    rope = ss.Rope(dim, base=1e6)
    q, k, v = (half(rng, sum(news), h, dim) for h in (2, 1, 1))
    out, turned, st = torch.empty_like(q), torch.empty_like(k), ints([-1] * 2)
    kw = dict(token_offsets=ints(offsets_of(news)), max_tokens=200000)
    ss.ss_rope(rope, q, out, k, turned, ints(lens), st, **kw)
    assert st.tolist() == [0, 0]
    at = P.positions(lens, news)
    check_turned(out, q, at, rope, "halves", 1.0)
    ss.ss_cache_append(cache, 0, turned, v, table, ints(lens), st, **kw)
    assert st.tolist() == [0, 0]
    want = [x.clone() for x in parts(cache)]
    if fmt == "fp8":
        plain = [P.Cache8(x[0].cpu().numpy(), s[0].cpu().numpy()) for x, s in ((before[0], before[2]), (before[1], before[3]))]
        for x, w in ((turned, plain[0]), (v, plain[1])):
            x = np32(x).astype(np.float64)
            for r, a in enumerate(lens):
                w.append(table[r].tolist(), a, x[offsets_of(news)[r]:offsets_of(news)[r + 1]])
        same8(cache, plain)
    def again():
        for x, y in zip(parts(cache), before):
            x.copy_(y)

    if fmt != "bf16":  # (in 1.3 million keys some lie next to where a rounding turns: as with limits that fit)
        again()
        ss.ss_rope_append(rope, cache, 0, q, torch.empty_like(q), k, v, table, ints(lens), st, **dict(kw, max_tokens=21000))
        want = [x.clone() for x in parts(cache)]
    again()
    out2 = torch.empty_like(q)
    ss.ss_rope_append(rope, cache, 0, q, out2, k, v, table, ints(lens), st, **kw)
    assert st.tolist() == [0, 0] and torch.equal(out, out2)
    for x, y in zip(parts(cache), want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_two_calls_at_once(ss):
    """Two streams, each with requests of its own in one cache: the blocks are apart."""
    p = Rows(ss, 21, [3, 40, 0, 17], [500, 300, 77, 130], 4, 16, 128)
    want = plain8(p.cache)
    p.plain(want)
    half_of = [slice(0, 2), slice(2, 4)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    lens, table, st = ints(p.lens), ints(p.table), [ints([-1, -1]) for _ in range(2)]
    off = [ints(p.offsets[h.start:h.stop + 1]) for h in half_of]
    torch.cuda.synchronize()
    for s, h, o, t in zip(streams, half_of, off, st):
        ss.ss_cache_append(p.cache, 0, p.k, p.v, table, lens[h], t, token_offsets=o, max_tokens=500,
                           table_rows=ints([h.start, h.start + 1]), stream=s)
    torch.cuda.synchronize()
    assert [t.tolist() for t in st] == [[0, 0], [0, 0]]
    same8(p.cache, want)
