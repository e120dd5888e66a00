"""ss_rope_append: what its statuses leave behind, in every format; many chunks of
a request's tokens, and the rotation at places of every kind, against 64-bit sums.

Tolerance of a turned channel.  With u = 2^-24 (half a step of fp32): cosine and
sine are fp32 roundings of sums known to 2^-34, off by u + 2^-34 of the
magnitude m at most; y s is rounded by u of it, the sum by u of it: 2 u m |x| +
3 u m |y| and 2^-34 m (|x| + |y|), so less than 3.01 u m (|x| + |y|); and the
result is rounded to bf16, 2^-8 of it.

Keys on their way into 8 or 4 bits carry what fp32 leaves: of cosine and sine a
bf16 more (2^-34.3 of m as far as they are known, and 2^-33 of it half a step of a
bf16 of up to 2^-24), of products and sum all: less than 2^-32 m (|x| + |y|),
before fp32 and then bf16 round them."""
import random

import numpy as np
import pytest

from tests import cache_ref as R
from tests import rope_ref as P
from tests.test_cache_gpu import ints, np32, random_parents, ss  # noqa: F401
from tests.test_rope_gpu import any_cache, half, offsets_of, parts, plain8

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("fmt", ["bf16", "int4", "fp8"])
def test_a_refused_request_is_untouched_and_a_bad_parent_is_the_root(ss, fmt):
    rng = np.random.default_rng(2)
    cache = any_cache(ss, rng, fmt, 9, 2, 16, 64)
    rope = ss.Rope(64)
    offsets, total = [0, 20, 40, 49, 49], 49
    q, k, v = (half(rng, total, h, 64) for h in (4, 2, 2))
    # rows of the table: one with a hole behind the first page; a full one; two more; none
    table, rows, lens = ints([[0, -1], [1, 2], [3, 4], [5, 6]]), ints([0, 1, 2, 7]), ints([5, 9, 5, 0])
    bad, good = [0] * total, [0] * total
    bad[0 + 3], bad[20 + 19] = 3, -5
    before = [x.clone() for x in parts(cache)]

    def call(parents, most=20):
        for x, y in zip(parts(cache), before):
            x.copy_(y)
        out, st = torch.full_like(q, 7.0), ints([-1] * 4)
        ss.ss_rope_append(rope, cache, 0, q, out, k, v, table, lens, st, token_offsets=ints(offsets), max_tokens=most,
                          parents=ints(parents), table_rows=rows)
        return [x.clone() for x in parts(cache)] + [out], st.tolist()

    want, st = call(good)
    assert st == [3, 0, 0, 4]
    got, st = call(bad)
    assert st == [4, 4, 0, 4]
    for x, y in zip(got, want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert not (got[-1] == 7).all(-1).any()
    # more tokens than said: the same code, and nothing of it touched
    got, st = call(bad, most=19)
    assert st == [4, 4, 0, 4] and (got[-1][:40] == 7).all() and not (got[-1][40:] == 7).all(-1).any()
    for x, y in zip(got[:-1], before):
        assert torch.equal(x[0, [0, 1, 2, 5, 6, 7, 8]].view(torch.uint8), y[0, [0, 1, 2, 5, 6, 7, 8]].view(torch.uint8))
        assert not torch.equal(x[0, [3, 4]].view(torch.uint8), y[0, [3, 4]].view(torch.uint8))


def table_of(rope):
    return [int(t) for t in rope.turns.cpu().numpy().view(np.uint64)]


def pairs_of(rope, layout):
    h = rope.rot_dim // 2
    return (slice(0, h), slice(h, 2 * h)) if layout == "halves" else (slice(0, 2 * h, 2), slice(1, 2 * h, 2))


@pytest.mark.parametrize("fmt", ["int4", "fp8"])
@pytest.mark.parametrize("layout,tree", [("halves", False), ("interleaved", False), ("halves", True)])
def test_every_chunk_against_sums_of_ones_own(ss, fmt, layout, tree):
    """Each cached row of a long chunk (or of many trees), from 64-bit sums: positions, rows, scales.  Where a sum lies
    so near to a tie of bf16 that the call may round it either way, its row or block is left out."""
    rng = np.random.default_rng(12)
    if tree:
        lens, news = rng.integers(0, 3000, 60).tolist(), rng.integers(1, 65, 60).tolist()
    else:
        lens, news = [5, 70, 0], [9001, 3, 130]
    heads, page, dim, total, offsets = 2, 64, 64, sum(news), offsets_of(news)
    need = [-(-(a + b) // page) for a, b in zip(lens, news)]
    perm = rng.permutation(sum(need)).tolist()
    table = [[perm.pop() for _ in range(n)] + [-1] * (max(need) - n) for n in need]
    cache = any_cache(ss, rng, fmt, sum(need), heads, page, dim)
    rope = ss.Rope(dim, rot_dim=48, layout=layout, base=1e6, magnitude=1.25)
    q, k, v = (half(rng, total, h, dim) for h in (3, heads, heads))
    pr = random.Random(12)
    trees = [random_parents(pr, n) for n in news] if tree else None
    at = P.positions(lens, news, trees)
    want = plain8(cache) if fmt == "fp8" else None
    out, st = torch.empty_like(q), ints([-1] * len(lens))
    ss.ss_rope_append(rope, cache, 0, q, out, k, v, ints(table), ints(lens), st, token_offsets=ints(offsets),
                      max_tokens=64 if tree else 200000, parents=ints(sum(trees, [])) if tree else None)
    assert st.tolist() == [0] * len(lens)
    # the keys: sums to 2^-32 of the magnitude times |x| + |y|, rounded to fp32 and to bf16
    x = np32(k).astype(np.float64)
    sums = P.turn(x, at, table_of(rope), 48, layout, 1.25)
    a, b = pairs_of(rope, layout)
    off = np.zeros_like(sums)
    off[..., a] = off[..., b] = 2.0 ** -32 * 1.25 * (np.abs(x[..., a]) + np.abs(x[..., b]))
    keys, low, high = (R.bf16((sums + d).astype(np.float32)) for d in (0, -off, off))
    doubt = (low != high).any(-1)  # [token, head]
    assert doubt.sum() <= 20
    new = [keys.astype(np.float64), np32(v).astype(np.float64)]
    if fmt == "fp8":
        for w, y in zip(want, new):
            for r, m in enumerate(lens):
                w.append(table[r], m, y[offsets[r]:offsets[r + 1]])
        skip = np.zeros(want[0].s.shape, bool)
        for r, m in enumerate(lens):
            for i, h in np.argwhere(doubt[offsets[r]:offsets[r + 1]]):
                skip[table[r][(m + i) // page], h, (m + i) % page // 16] = True
        for i, (d, s, w) in enumerate(((cache.k, cache.k_scale, want[0]), (cache.v, cache.v_scale, want[1]))):
            look = ~skip if i == 0 else np.ones_like(skip)
            assert np.array_equal(s[0].cpu().numpy().astype(np.float64)[look], w.s[look])
            got = P.e4m3_of(d[0].view(torch.uint8).cpu().numpy())
            look = np.repeat(look, 16, -1)
            assert np.array_equal(got[look], w.n[look])
        return
    for i, (d, s, y) in enumerate(((cache.k, cache.k_scale, new[0]), (cache.v, cache.v_scale, new[1]))):
        n, step, lowest = R.quantise(y)
        r = np.repeat(np.arange(len(lens)), news)
        slot = np.concatenate([np.arange(m, m + c) for m, c in zip(lens, news)])
        pages = np.array([table[j][e] for j, e in zip(r, slot // page)])
        look = ~doubt if i == 0 else np.ones_like(doubt)
        got, pair = d[0].cpu().numpy()[pages, :, slot % page], np32(s[0])[pages, :, slot % page]
        assert np.array_equal(got[look], R.pack(n)[look])
        assert np.array_equal(pair[look], np.stack([step, lowest], -1)[look])


@pytest.mark.parametrize("layout", ["halves", "interleaved"])
@pytest.mark.parametrize("dim,rot", [(128, 128), (96, 20)])
def test_turned_rows_to_the_last_bits_of_fp32(ss, dim, rot, layout):
    rng = np.random.default_rng(rot)
    rope = ss.Rope(dim, rot_dim=rot, layout=layout, base=10000.0, magnitude=1.5)
    n = 4000
    at = np.concatenate([np.arange(2000), rng.integers(-2 ** 31, 2 ** 31, n - 2000)]).tolist()
    q = half(rng, n, 2, dim)
    x = np32(q).astype(np.float64)
    a, b = pairs_of(rope, layout)
    # half of the rows: pairs whose first result nearly cancels, y = x cos / sin as bf16 has it
    ones = np.zeros((n, 1, dim))
    ones[..., a] = 1.0
    turned = P.turn(ones, at, table_of(rope), rot, layout, 1.0)
    cos, sin = turned[..., a], turned[..., b]
    with np.errstate(all="ignore"):
        y = np.where(np.abs(sin) > 0.05, x[..., a] * cos / sin, x[..., b])
    x[n // 2:, :, b] = R.bf16(y[n // 2:].astype(np.float32))
    x[:1000, :, b] = R.bf16(y[:1000].astype(np.float32))
    q = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()
    out, st = torch.empty_like(q), ints([-1])
    ss.ss_rope(rope, q, out, None, None, None, st, token_offsets=ints([0, n]), max_tokens=n, positions=ints(at))
    assert st.tolist() == [0]
    want = P.turn(x, at, table_of(rope), rot, layout, 1.5)
    both = np.zeros_like(x)
    both[..., a] = both[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    near = 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * 3.01 * 2.0 ** -24 * 1.5 * both
    assert (np.abs(np32(out) - want) <= near).all()
