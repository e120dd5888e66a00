"""What rejected drafts leave in a cache of 8 bits: the rows that were there
before share a block's scale with them.

The bound.  A row's value x is first held to 2^-4 |x| (half of e4m3's step) or,
small, to 2^-10 s.  Encoded again under a larger power of two s', it keeps its
bits where it is at least 2^-6 s', and is off by 2^-10 s' more elsewhere; under
a smaller one it keeps them all.  Errors under growing scales add up to
2^-10 (s + s / 2 + ..) at most: 2^-4 |x| + 2^-9 s, s the largest scale that the
block has had."""
import numpy as np
import pytest

from tests import rope_ref as P
from tests.test_cache_gpu import ints, np32, ss  # noqa: F401
from tests.test_rope_gpu import half, offsets_of, plain8, same8

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HEADS, DIM, PAGE = 2, 64, 32
OUTLIER = 1e6


class Step:
    """Four requests of a few tokens, and calls on them beside the plain forms."""

    def __init__(self, ss):
        self.ss, self.lens = ss, [5, 12, 39, 16]
        self.n, self.rng = len(self.lens), np.random.default_rng(4)
        self.cache, self.pool = ss.alloc_cache(1, 24, HEADS, PAGE, DIM, "fp8"), ss.alloc_pool(2 * self.n, 4, 24, PAGE)
        self.st = ints([-1] * self.n)
        self.want = plain8(self.cache)
        self.rows = list(range(self.n))
        self.first = [[self.draw(m) for m in self.lens] for _ in range(2)]
        self.reserve(self.rows, [0] * self.n, self.lens)
        self.append(self.rows, [0] * self.n, self.first)

    def draw(self, m):
        return half(self.rng, m, HEADS, DIM)

    def reserve(self, rows, start, stop):
        self.ss.ss_pages_reserve(self.pool, ints(start), ints(stop), self.st, table_rows=ints(rows))
        assert self.st.tolist() == [0] * self.n
        self.table = self.pool.page_table.tolist()

    def append(self, rows, lens, kv):
        news = [len(x) for x in kv[0]]
        self.ss.ss_cache_append(self.cache, 0, torch.cat(kv[0]), torch.cat(kv[1]), self.pool, ints(lens), self.st,
                                token_offsets=ints(offsets_of(news)), max_tokens=max(news), table_rows=ints(rows))
        assert self.st.tolist() == [0] * self.n
        for w, new in zip(self.want, kv):
            for r, a, x in zip(rows, lens, new):
                w.append(self.table[r], a, np32(x).astype(np.float64))
        same8(self.cache, self.want)

    def drafts(self, m=6):
        """The last token and drafts, one of which has a value far beyond all others, in K and in V."""
        kv = [[self.draw(m) for _ in self.lens] for _ in range(2)]
        for new in kv:
            for r, x in enumerate(new):
                x[m // 2, r % HEADS, 7 * r] = -OUTLIER
        return kv

    def read(self, rows, lens):
        k, v = (torch.empty(sum(lens), HEADS, DIM, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.ss.ss_cache_read(self.cache, 0, k, v, self.pool, ints([0] * self.n), self.st, token_offsets=ints(offsets_of(lens)),
                              max_tokens=max(lens), table_rows=ints(rows))
        assert self.st.tolist() == [0] * self.n
        return [list(x.split(lens)) for x in (k, v)]


def near(got, want, s):
    x = np.abs(np32(want))
    return (np.abs(np32(got) - np32(want)) <= 2.0 ** -4 * x + 2.0 ** -9 * s).all()


SMALL, LARGE = P.scale_of(np.array([8.0])), P.scale_of(np.array([OUTLIER]))  # (normal values stay below 8)


@pytest.mark.parametrize("tree", [False, True])
def test_what_a_rejected_draft_leaves(ss, tree):
    t = Step(ss)
    new = t.drafts()
    after = [a + 6 for a in t.lens]
    before = t.read(t.rows, t.lens)
    assert all(near(g, w, SMALL) for got, want in zip(before, t.first) for g, w in zip(got, want))
    t.reserve(t.rows, t.lens, after)
    t.append(t.rows, t.lens, new)
    kept = [0, 1, 5] if tree else [0, 1]  # the root, its child, and of a tree a node behind the far one
    if tree:
        new_len = ints([-1] * t.n)
        t.ss.ss_pages_compact(t.pool, t.cache, ints(t.lens), ints([[1, 5]] * t.n), ints([2] * t.n), None, new_len, t.st)
        assert t.st.tolist() == [0] * t.n
        for w in t.want:
            for r, a in enumerate(t.lens):
                w.compact(t.table[r], a, [1, 5])
        same8(t.cache, t.want)
    lens = [a + len(kept) for a in t.lens]
    more = [[t.draw(3) for _ in t.lens] for _ in range(2)]
    t.append(t.rows, lens, more)
    got = t.read(t.rows, [a + 3 for a in lens])
    for old, first, drafted, added, back in zip(before, t.first, new, more, got):
        for r, a in enumerate(t.lens):
            full = a // 16 * 16
            assert torch.equal(back[r][:full], old[r][:full])  # of full blocks: not a bit
            assert near(back[r][full:a], first[r][full:], LARGE)
            assert near(back[r][a:a + len(kept)], drafted[r][kept], LARGE)
            assert near(back[r][a + len(kept):], added[r], SMALL)  # the next step's own values
    # the scales are those of what is there
    for scale, w in ((t.cache.k_scale, t.want[0]), (t.cache.v_scale, t.want[1])):
        for r, m in enumerate(lens):
            at = m + 2
            assert float(scale[0, t.table[r][at // PAGE], :, at % PAGE // 16].max()) <= SMALL


def test_drafts_tried_in_a_fork_leave_nothing(ss):
    t, never = Step(ss), Step(ss)
    assert never.lens == t.lens
    children = [t.n + r for r in t.rows]
    t.ss.ss_pages_fork(t.pool, t.cache, ints(t.rows), ints(children), ints(t.lens), t.st)
    assert t.st.tolist() == [0] * t.n
    new = t.drafts()
    t.reserve(children, t.lens, [a + 6 for a in t.lens])
    t.want = plain8(t.cache)
    t.append(children, t.lens, new)
    tried = t.read(children, [a + 6 for a in t.lens])
    assert all(near(g[a:], w, LARGE) for got, want in zip(tried, new) for g, w, a in zip(got, want, t.lens))
    t.ss.ss_pages_trim(t.pool, ints([0] * t.n), t.st, table_rows=ints(children))
    assert t.st.tolist() == [0] * t.n
    # two of them accepted: appended to the rows that were forked
    accepted = [[x[:2] for x in part] for part in new]
    for s in (t, never):
        s.reserve(s.rows, s.lens, [a + 2 for a in s.lens])
        s.append(s.rows, s.lens, accepted)
    got, want = (s.read(s.rows, [a + 2 for a in s.lens]) for s in (t, never))
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))
