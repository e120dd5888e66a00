"""The paged cache on the GPU: rows in bf16 and in 4 bits, attention over
them, and the pages' bookkeeping, against tests/cache_ref.py.

Tolerances.  An output row is sum_j p_j v_j / sum_j p_j with fp32 sums, the
weights rounded to bf16 (8 significant bits: relative error at most 2^-8 each)
and the result rounded to bf16 (2^-8 of it): |error| <= 2^-8 (|out| +
sum p |v| / sum p), with 1/16 more for the fp32 scores, exponentials and sums.  Over 4 bits the rounded
factor is p s times n - 8, so |v| becomes s |n - 8| + |m + 8 s|.  The log-sum
carries the scores' fp32 error: 128 products and sums of 24 bits, so at most
2^-24 * 128 of sum |q k|, plus a few units of the result's own last place.
"""
import random

import numpy as np
import pytest

from tests import cache_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ss():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_verification_gb300 import build as ss_build
    ss_build.build()
    from speculative_verification_gb300 import ss as _ss
    _ss.load()
    return _ss


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def np32(t):
    return t.float().cpu().numpy()


def make_cache(ss, rng, fmt, pages, heads, page, dim, layers=1, order="phsd", fill=None):
    """A cache with random rows (or all NaN), its rows' dimensions laid out in `order`."""
    names = {"p": pages, "h": heads, "s": page}
    rows = (layers, pages, heads, page)

    def lay(t):
        back = [0] + [1 + order[:3].index(x) for x in "phs"] + [4]
        front = [0] + ["phs".index(x) + 1 for x in order[:3]] + [4]
        return t.permute(*front).contiguous().permute(*back)

    assert names
    if fmt == "bf16":
        parts = []
        for _ in range(2):
            x = torch.from_numpy(R.bf16(rng.standard_normal(rows + (dim,)))).to(torch.bfloat16)
            parts.append(lay(x.cuda() if fill is None else torch.full_like(x, fill).cuda()))
        return ss.KVCache(*parts)
    parts, scales = [], []
    for _ in range(2):
        parts.append(lay(torch.from_numpy(rng.integers(0, 256, rows + (dim // 2,), dtype=np.uint8)).cuda()))
        step = rng.uniform(0.1, 0.4, rows)
        pair = np.stack([step, rng.standard_normal(rows) * 0.3 - 7.5 * step], -1)
        pair = torch.from_numpy(pair.astype(np.float32)).to(torch.bfloat16)
        scales.append((pair if fill is None else torch.full_like(pair, fill)).cuda())
    return ss.KVCache(*parts, *scales)


def dense(cache, layer=0):
    """The cache's values: k, v and the factor of the tolerance, float64 [pages, heads, slots, dim]."""
    out = []
    for x, sc in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        if sc is None:
            f = np32(x[layer]).astype(np.float64)
            out.append((f, np.abs(f)))
        else:
            n = R.unpack(x[layer].contiguous().cpu().numpy()).astype(np.float64)
            p = np32(sc[layer]).astype(np.float64)
            s, m = p[..., :1], p[..., 1:]
            out.append((s * n + m, np.abs(s * (n - 8)) + np.abs(m + 8 * s)))
    (k, _), (v, mv) = out
    return k, v, mv


def random_parents(rng, n):
    return [0] + [rng.randint(max(0, i - 4), i - 1) for i in range(1, n)]


class Problem:
    """A batch over a shuffled page table."""

    def __init__(self, ss, seed, fmt, lens, news, heads, kv_heads, dim, page, window=0, sinks=0, tree=False, order="phsd",
                 evict=False, rows=None):
        rng, pr = np.random.default_rng(seed), random.Random(seed)
        self.lens, self.news, self.window, self.sinks, self.page = lens, news, window, sinks, page
        need = [-(-(a + b) // page) for a, b in zip(lens, news)]
        width = max(need + [1])
        used, table = 0, []
        for a, n in zip(lens, need):
            row = [-1] * width
            for e in range(n):
                if evict and window and e * page >= sinks and (e + 1) * page <= a - window:
                    continue
                row[e] = used
                used += 1
            table.append(row)
        self.num_pages = used + 2
        perm = rng.permutation(self.num_pages)
        self.table = [[int(perm[e]) if e >= 0 else -1 for e in row] for row in table]
        self.cache = make_cache(ss, rng, fmt, self.num_pages, kv_heads, page, dim, order=order)
        self.offsets = [0]
        for n in news:
            self.offsets.append(self.offsets[-1] + n)
        total = self.offsets[-1]
        self.q = torch.from_numpy(R.bf16(rng.standard_normal((total, heads, dim)))).to(torch.bfloat16).cuda()
        self.parents = [random_parents(pr, n) for n in news] if tree else None
        self.scale = dim ** -0.5
        self.heads = heads

    def spoil(self):
        """Every slot that no query sees becomes NaN (K, V and scales)."""
        keep = np.zeros((self.num_pages, self.page), bool)
        for row, a, b in zip(self.table, self.lens, self.news):
            for s in range(a + b):
                if 0 <= row[s // self.page] < self.num_pages:
                    seen = not self.window or s > a - self.window or s < self.sinks
                    keep[row[s // self.page], s % self.page] |= seen
        gone = torch.from_numpy(~keep).cuda()
        for t in ((self.cache.k, self.cache.v) if self.cache.format == "bf16" else
                  (self.cache.k_scale, self.cache.v_scale)):
            t[0].masked_fill_(gone[:, None, :, None], float("nan"))

    def call(self, ss, workspace, lse=True, **kw):
        out = torch.full_like(self.q, 7.0)
        ls = torch.full(self.q.shape[:2], 7.0, dtype=torch.float32, device="cuda") if lse else None
        st = ints([-1] * len(self.lens))
        par = ints([p for row in self.parents for p in row]) if self.parents is not None else None
        ss.ss_cache_attention(self.cache, 0, self.q, out, ints(self.table), ints(self.lens), workspace, st,
                              query_offsets=ints(self.offsets), max_queries=max(self.news), parents=par,
                              scale=self.scale, window=self.window, sinks=self.sinks, lse=ls, **kw)
        return out, ls, st

    def check(self, ss, workspace):
        out, lse, st = self.call(ss, workspace)
        torch.cuda.synchronize()
        assert st.cpu().tolist() == [0] * len(self.lens)
        assert not bool(workspace[:256].any())  # the counters are left at zero
        got, gl = np32(out).astype(np.float64), lse.cpu().numpy().astype(np.float64)
        k, v, mv = dense(self.cache)
        pick = lambda pages, slots: tuple(x[pages, :, slots] for x in (k, v, mv))  # noqa: E731
        q = np32(self.q).astype(np.float64)
        for r, (a, n) in enumerate(zip(self.lens, self.news)):
            lo, hi = self.offsets[r], self.offsets[r + 1]
            par = self.parents[r] if self.parents is not None else None
            o, l, m, reach = R.attend(q[lo:hi], pick, self.table[r], self.page, a, self.scale, self.window, self.sinks, par,
                                      self.num_pages)
            tol = 2.0 ** -8 * (np.abs(o) + m) * (1 + 1 / 16) + 1e-30
            bad = ~(np.abs(got[lo:hi] - o) <= tol)
            assert not bad.any(), (r, a, n, np.argwhere(bad)[:5], got[lo:hi][bad][:5], o[bad][:5], bad.mean())
            empty = np.isneginf(l)
            assert np.array_equal(np.isneginf(gl[lo:hi]), empty)
            tl = 2.0 ** -17 * reach + 2.0 ** -21 * (1 + np.abs(np.where(empty, 0, l)))
            badl = ~empty & ~(np.abs(gl[lo:hi] - np.where(empty, 0, l)) <= tl)
            assert not badl.any(), (r, gl[lo:hi][badl][:5], l[badl][:5])


@pytest.fixture(scope="module")
def workspace(ss):
    return ss.alloc_attention_workspace()


FORMATS = ["bf16", "int4"]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,heads,kv_heads,page", [
    (128, 8, 2, 16), (64, 4, 4, 32), (128, 7, 1, 64), (96, 6, 2, 8), (32, 3, 3, 128), (128, 128, 1, 16),
    (64, 10, 2, 256), (128, 16, 1, 1024)])
def test_lengths_and_layouts(ss, workspace, fmt, dim, heads, kv_heads, page):
    # lengths around the tile of 128 keys and the pages, empty caches, and ragged numbers of queries
    lens = [0, 1, 15, 16, 17, 126, 127, 128, 129, 255, 256, 300, 513, 1000]
    news = [1, 2, 1, 3, 1, 2, 1, 1, 8, 1, 5, 4, 1, 7]
    Problem(ss, 1, fmt, lens, news, heads, kv_heads, dim, page).check(ss, workspace)


@pytest.mark.parametrize("dim", [8, 16, 24, 40, 72, 80, 112, 120])
def test_odd_head_dims_bf16(ss, workspace, dim):
    Problem(ss, 2, "bf16", [5, 130, 400], [1, 3, 2], 4, 2, dim, 16).check(ss, workspace)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (5, 130), (64, 1), (127, 3), (128, 0), (129, 128), (200, 17),
                                          (1000, 4), (100000, 4)])
def test_window_and_sinks(ss, workspace, fmt, window, sinks):
    lens, news = [0, 3, 60, 127, 128, 200, 400, 777, 1200], [1, 5, 3, 2, 4, 1, 8, 1, 6]
    p = Problem(ss, 3, fmt, lens, news, 8, 2, 64, 16, window=window, sinks=sinks)
    p.check(ss, workspace)
    # pages that the window has passed given back, and NaN wherever nothing looks
    p = Problem(ss, 4, fmt, lens, news, 8, 2, 128, 16, window=window, sinks=sinks, evict=True)
    p.spoil()
    p.check(ss, workspace)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 1), (40, 4), (300, 150)])
@pytest.mark.parametrize("heads,kv_heads", [(4, 4), (8, 1), (12, 4)])
def test_trees(ss, workspace, fmt, window, sinks, heads, kv_heads):
    lens, news = [0, 1, 100, 127, 250, 511, 64], [64, 1, 33, 2, 64, 17, 63]
    p = Problem(ss, 5, fmt, lens, news, heads, kv_heads, 64, 16, window=window, sinks=sinks, tree=True)
    p.spoil()
    p.check(ss, workspace)


@pytest.mark.parametrize("fmt", FORMATS)
def test_prompt_chunks(ss, workspace, fmt):
    for seed, (lens, news, window) in enumerate([([0, 300], [300, 201], 0), ([130, 5], [257, 1], 100),
                                                 ([0], [700], 33)]):
        p = Problem(ss, 10 + seed, fmt, lens, news, 4, 2, 128, 32, window=window, sinks=4 if window else 0)
        p.spoil()
        p.check(ss, workspace)


@pytest.mark.parametrize("fmt", FORMATS)
def test_long_context_is_split_and_joined(ss, workspace, fmt):
    for lens, news, heads, kv in [([20011], [1], 2, 1), ([9000, 1, 5000], [3, 1, 4], 16, 2)]:
        Problem(ss, 20, fmt, lens, news, heads, kv, 128, 64).check(ss, workspace)


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_requests(ss, workspace, fmt):
    rng = random.Random(7)
    lens = [rng.choice([0, 1, rng.randint(0, 200), rng.randint(0, 600)]) for _ in range(333)]
    news = [rng.randint(1, 3) for _ in lens]
    Problem(ss, 21, fmt, lens, news, 2, 1, 64, 16).check(ss, workspace)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("group,dim", [(8, 128), (24, 128), (24, 64), (60, 128), (100, 64), (128, 128)])
def test_many_items_for_every_block_of_rows(ss, workspace, fmt, group, dim):
    # several items per SM, whole and in pieces, of 16 to 128 rows
    rng = random.Random(group)
    lens = [rng.randint(0, 500) for _ in range(160)]
    Problem(ss, 40, fmt, lens, [1] * len(lens), 2 * group, 2, dim, 16).check(ss, workspace)


@pytest.mark.parametrize("order", ["pshd", "hpsd", "shpd"])
def test_cache_layouts(ss, workspace, order):
    Problem(ss, 22, "bf16", [100, 300], [2, 5], 4, 2, 64, 16, order=order).check(ss, workspace)
    Problem(ss, 23, "int4", [100, 300], [2, 5], 4, 2, 64, 16, order=order).check(ss, workspace)


@pytest.mark.parametrize("fmt", FORMATS)
def test_scores_far_apart(ss, workspace, fmt):
    # rising and falling scores of hundreds: the running maximum moves at every tile, early keys vanish
    for sign in (1.0, -1.0):
        p = Problem(ss, 24, fmt, [900], [4], 4, 2, 64, 16)
        ramp = torch.linspace(0, 40, 1000).to(torch.bfloat16).cuda() * sign
        for s in range(904):
            page = p.table[0][s // 16]
            if fmt == "bf16":
                p.cache.k[0, page, :, s % 16] = ramp[s]
            else:
                p.cache.k_scale[0, page, :, s % 16, 0] = 0.0625
                p.cache.k_scale[0, page, :, s % 16, 1] = ramp[s]
        p.q.abs_()
        p.check(ss, workspace)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("low,high,zeros", [(-60, -60, False), (60, 60, False), (100, 100, False), (-40, 40, False),
                                            (-20, 0, True)])
def test_values_of_every_size(ss, workspace, fmt, low, high, zeros):
    # values far from 1, keys whose values differ by many powers of two, rows of zeros
    rng = np.random.default_rng(abs(high) + 7)
    for news, heads in (([3, 1], 4), ([8, 5], 16)):
        p = Problem(ss, 31, fmt, [700, 40], news, heads, 2, 64, 16)
        f = torch.from_numpy(2.0 ** rng.integers(low, high + 1, p.cache.v.shape[:4])).to(torch.bfloat16).cuda()
        if zeros:
            f[torch.from_numpy(rng.random(f.shape) < 0.3).cuda()] = 0
        t = p.cache.v if fmt == "bf16" else p.cache.v_scale
        t.mul_(f[..., None])
        p.check(ss, workspace)


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_that_see_nothing(ss, workspace, fmt):
    # the pages of some requests are holes: out = 0, lse = -inf
    p = Problem(ss, 25, fmt, [40, 200, 10], [2, 3, 1], 4, 2, 64, 16)
    p.table[0] = [-1] * len(p.table[0])
    p.table[2] = [p.num_pages + 5] * len(p.table[2])
    p.spoil()
    p.check(ss, workspace)
    # the window of a query has holes but the sinks are there
    p = Problem(ss, 26, fmt, [300], [2], 4, 2, 64, 16, window=20, sinks=2)
    p.table[0][1:] = [-1] * (len(p.table[0]) - 1)
    p.check(ss, workspace)


@pytest.mark.parametrize("fmt", FORMATS)
def test_lengths_far_beyond_the_table(ss, workspace, fmt):
    # 200 requests whose lengths say 2^31 slots, of a table of four pages
    n, page, heads, dim, far = 200, 16, 4, 64, 2 ** 31 - 300
    rng = np.random.default_rng(8)
    cache = make_cache(ss, rng, fmt, 8, 2, page, dim)
    q = torch.randn(n, heads, dim, device="cuda").to(torch.bfloat16)
    table = ints(rng.integers(0, 8, (n, 4)).tolist())
    out, lse, st = torch.full_like(q, 7), torch.full((n, heads), 7.0, device="cuda"), ints([-1] * n)
    ss.ss_cache_attention(cache, 0, q, out, table, ints([far] * n), workspace, st, lse=lse)
    torch.cuda.synchronize()
    assert st.tolist() == [3] * n
    want, want_lse, st2 = torch.empty_like(q), torch.empty_like(lse), ints([-1] * n)
    # all four pages are seen: the same as at the table's last slot
    ss.ss_cache_attention(cache, 0, q, want, table, ints([4 * page - 1] * n), workspace, st2, lse=want_lse)
    torch.cuda.synchronize()
    assert st2.tolist() == [0] * n and torch.equal(out, want) and torch.equal(lse, want_lse)
    # a window that lies beyond the table shows nothing, but for the sinks
    ss.ss_cache_attention(cache, 0, q, out, table, ints([far] * n), workspace, st, lse=lse, window=500)
    torch.cuda.synchronize()
    assert not out.any() and bool((lse == -float("inf")).all()) and st.tolist() == [3] * n


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_draft_that_is_not_finite_stays_on_its_branch(ss, workspace, fmt):
    p = Problem(ss, 27, fmt, [150], [40], 8, 2, 64, 16, tree=True)
    clean, clean_lse, _ = p.call(ss, workspace)
    _, line = R.paths(p.parents[0])
    node = next(i for i in range(1, 40) if 1 < sum(i in x for x in line) < 39)
    s = 150 + node
    page, row = p.table[0][s // 16], s % 16
    for value in (float("nan"), float("inf")):
        for t in ((p.cache.k, p.cache.v) if fmt == "bf16" else (p.cache.k_scale, p.cache.v_scale)):
            t[0, page, :, row] = value
        out, lse, _ = p.call(ss, workspace)
        torch.cuda.synchronize()
        for i in range(40):
            if node in line[i]:
                assert not torch.isfinite(out[i]).all(dim=-1).any()
            else:
                assert torch.equal(out[i], clean[i]) and torch.equal(lse[i], clean_lse[i]), i


@pytest.mark.parametrize("fmt", FORMATS)
def test_extreme_values_in_sight(ss, workspace, fmt):
    # the type's lowest and highest finite values as keys of some tokens: weights of 0 or 1, no NaN
    p = Problem(ss, 28, fmt, [200], [1], 2, 1, 64, 16)
    p.q.abs_()
    big = 3.3895313892515355e38
    for s, value in ((3, -big), (130, -big)):
        page = p.table[0][s // 16]
        if fmt == "bf16":
            p.cache.k[0, page, :, s % 16] = value
        else:
            p.cache.k_scale[0, page, :, s % 16, 0] = 0.0
            p.cache.k_scale[0, page, :, s % 16, 1] = value
    out, lse, _ = p.call(ss, workspace)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


def test_same_bits_every_time_and_on_other_streams(ss, workspace):
    for fmt in FORMATS:
        p = Problem(ss, 29, fmt, [3000, 10, 777, 64], [4, 1, 8, 2], 16, 2, 128, 16, window=0)
        out, lse, _ = p.call(ss, workspace)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for i in range(4):
            o2, l2, _ = p.call(ss, workspace)
            assert torch.equal(out, o2) and torch.equal(lse, l2)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            o3, l3, _ = p.call(ss, workspace)
        side.synchronize()
        assert torch.equal(out, o3) and torch.equal(lse, l3)
        o4, l4, _ = p.call(ss, workspace, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, o4) and torch.equal(lse, l4)


def test_strided_queries_outputs_and_no_lse(ss, workspace):
    p = Problem(ss, 30, "bf16", [100, 33], [3, 1], 8, 2, 64, 16)
    ref, _, _ = p.call(ss, workspace)
    wide = torch.zeros(4, 3, 8, 64 + 8, dtype=torch.bfloat16, device="cuda")
    wide[:, 1, :, :64] = p.q
    out = torch.full((4, 8, 65), 5.0, dtype=torch.bfloat16, device="cuda")
    st = ints([9, 9])
    ss.ss_cache_attention(p.cache, 0, wide[:, 1, :, :64], out[..., 1:], ints(p.table), ints(p.lens), workspace, st,
                          query_offsets=ints(p.offsets), max_queries=5)
    torch.cuda.synchronize()
    assert torch.equal(out[..., 1:], ref) and bool((out[..., 0] == 5).all()) and st.tolist() == [0, 0]


def test_one_query_each_table_rows_and_layers(ss, workspace):
    rng = np.random.default_rng(3)
    cache = make_cache(ss, rng, "bf16", 12, 2, 16, 64, layers=3)
    table = ints([[0, 1, 2], [3, 4, 5], [6, 7, 8]])
    q = torch.randn(2, 4, 64, device="cuda").to(torch.bfloat16)
    out, st = torch.empty_like(q), ints([-1, -1])
    ss.ss_cache_attention(cache, 2, q, out, table, ints([20, 40]), workspace, st, table_rows=ints([2, 0]))
    torch.cuda.synchronize()
    k, v, mv = dense(cache, 2)
    for i, (row, a) in enumerate((([6, 7, 8], 20), ([0, 1, 2], 40))):
        o, _, m, _ = R.attend(np32(q[i:i + 1]).astype(np.float64), lambda p, s: (k[p, :, s], v[p, :, s], mv[p, :, s]), row, 16,
                              a, 0.125, 0, 0, None, 12)
        assert (np.abs(np32(out[i:i + 1]) - o) <= 2.0 ** -8 * (np.abs(o) + m) * (1 + 1 / 16)).all()
    assert st.tolist() == [0, 0]


def test_bad_requests_are_reported_and_the_others_done(ss, workspace):
    p = Problem(ss, 31, "bf16", [50, 60, 70, 80], [2, 3, 1, 2], 4, 2, 64, 16)
    ref, rl, _ = p.call(ss, workspace)

    def run(lens, offsets=None, most=3, rows=None, parents=None):
        out = torch.full_like(p.q, 7.0)
        st = ints([-1] * 4)
        ss.ss_cache_attention(p.cache, 0, p.q, out, ints(p.table), ints(lens), workspace, st,
                              query_offsets=ints(offsets or p.offsets), max_queries=most,
                              table_rows=None if rows is None else ints(rows), parents=parents)
        torch.cuda.synchronize()
        return out, st.tolist()

    out, st = run([50, -1, 70, 80])
    assert st == [0, 4, 0, 0] and torch.equal(out[:2], ref[:2]) and torch.equal(out[5:], ref[5:])
    assert bool((out[2:5] == 7).all())
    out, st = run(p.lens, most=2)  # request 1 has three queries
    assert st == [0, 4, 0, 0] and torch.equal(out[5:], ref[5:]) and bool((out[2:5] == 7).all())
    out, st = run(p.lens, offsets=[0, 2, 5, 6, 9])  # past the rows of q
    assert st == [0, 0, 0, 4] and torch.equal(out[:6], ref[:6])
    out, st = run(p.lens, offsets=[0, 2, 1, 2, 4])  # falling offsets
    assert st[1] == 4
    out, st = run(p.lens, rows=[0, 4, -1, 3])
    assert st == [0, 4, 4, 0] and torch.equal(out[:2], ref[:2]) and torch.equal(out[6:], ref[6:])
    out, st = run([50, 60, 70, len(p.table[0]) * 16 - 1])  # the second query's slot is beyond the table
    assert st == [0, 0, 0, 3] and torch.equal(out[:6], ref[:6])
    out, st = run(p.lens, parents=ints([0, 0, 0, 2, 0, 0, 0, 0]))  # a node that is not before its child
    assert st == [0, 4, 0, 0]


def test_zero_queries(ss, workspace):
    p = Problem(ss, 32, "bf16", [50, 60, 70], [2, 0, 1], 4, 2, 64, 16)
    p.check(ss, workspace)


def test_graph_capture(ss, workspace):
    p = Problem(ss, 33, "int4", [500, 60], [4, 2], 8, 2, 128, 16)
    ref, rl, _ = p.call(ss, workspace)
    out, lse, st = torch.empty_like(ref), torch.empty_like(rl), ints([0, 0])
    table, lens, off = ints(p.table), ints(p.lens), ints(p.offsets)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            ss.ss_cache_attention(p.cache, 0, p.q, out, table, lens, workspace, st, query_offsets=off, max_queries=4,
                                  lse=lse)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, rl)


# ------------------------------------------------------------------ rows --

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,heads,page,order", [(128, 8, 16, "phsd"), (64, 3, 32, "pshd"), (96, 1, 8, "hpsd"),
                                                  (32, 5, 128, "phsd")])
def test_append_and_read(ss, fmt, dim, heads, page, order):
    rng = np.random.default_rng(dim)
    lens, news = [0, 5, 15, 100, 7, 31], [1, 40, 0, 3, 300, 1]
    offsets = np.concatenate([[0], np.cumsum(news)])
    width = max(-(-(a + b) // page) for a, b in zip(lens, news))
    pages = len(lens) * width + 1
    table = rng.permutation(pages)[:len(lens) * width].reshape(len(lens), width).astype(np.int32)
    cache = make_cache(ss, rng, fmt, pages, heads, page, dim, layers=2, order=order)
    x = rng.standard_normal((offsets[-1], 2, heads, dim)) * np.exp(rng.uniform(-3, 3, (offsets[-1], 2, heads, 1)))
    x[3] = 1.5          # no spread: step 0
    x[4, :, :, 0] = 64  # exact ties of the rounding
    x[4, :, :, 1:] = rng.integers(0, 31, (2, heads, dim - 1)) * 0.5
    kv = torch.from_numpy(R.bf16(x)).to(torch.bfloat16).cuda()
    before = [None if t is None else t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    st = ints([-1] * len(lens))
    args = dict(token_offsets=ints(offsets.tolist()), max_tokens=300)
    ss.ss_cache_append(cache, 1, kv[:, 0], kv[:, 1], torch.from_numpy(table).cuda(), ints(lens), st, **args)
    torch.cuda.synchronize()
    assert st.tolist() == [0] * len(lens)
    at = [(int(table[r, (a + i) // page]), (a + i) % page) for r, (a, b) in enumerate(zip(lens, news)) for i in range(b)]
    pg, sl = np.array(at).T
    src = np32(kv)
    for which, (cells, scale, old, olds) in enumerate(((cache.k, cache.k_scale, before[0], before[2]),
                                                      (cache.v, cache.v_scale, before[1], before[3]))):
        want = old.cpu()
        if fmt == "bf16":
            want[1, pg, :, sl] = kv[:, which].cpu()
            assert torch.equal(cells.cpu(), want)
        else:
            n, s, m = R.quantise(src[:, which])
            want[1, pg, :, sl] = torch.from_numpy(R.pack(n))
            assert torch.equal(cells.cpu(), want)
            ws = olds.cpu()
            ws[1, pg, :, sl] = torch.from_numpy(np.stack([s, m], -1)).to(torch.bfloat16)
            assert torch.equal(scale.cpu(), ws)
            assert float(np.abs(s[..., None] * n + m[..., None] - src[:, which]).max() / (s.max())) <= 0.51
    back = torch.empty_like(kv)
    ss.ss_cache_read(cache, 1, back[:, 0], back[:, 1], torch.from_numpy(table).cuda(), ints(lens), st, **args)
    torch.cuda.synchronize()
    if fmt == "bf16":
        assert torch.equal(back, kv)
    else:
        n, s, m = R.quantise(src)
        v = n.astype(np.float64) * s[..., None] + m[..., None]
        assert (np.abs(np32(back) - v) <= 2.0 ** -8 * np.abs(v) + 1e-40).all()


def test_append_rows_that_are_not_finite(ss):
    cache = ss.alloc_cache(1, 4, 1, 16, 64, "int4")
    x = torch.randn(5, 1, 64, device="cuda").to(torch.bfloat16)
    x[0, 0, 3], x[1, 0, 63], x[2, 0, 0] = float("nan"), float("inf"), float("-inf")
    x[3, 0, 0], x[3, 0, 1] = 3e38, -3e38
    st, y, z = ints([0]), torch.zeros_like(x), torch.zeros_like(x)
    kw = dict(token_offsets=ints([0, 5]), max_tokens=5)
    ss.ss_cache_append(cache, 0, x, x, ints([[2]]), ints([0]), st, **kw)
    ss.ss_cache_read(cache, 0, y, z, ints([[2]]), ints([0]), st, **kw)
    torch.cuda.synchronize()
    assert torch.isnan(y[:4]).all() and torch.isfinite(y[4]).all() and torch.isnan(z[:4]).all()


def test_append_rounds_as_defined_at_every_scale(ss):
    # rows over the whole range of bf16, many of them with channels next to or on a half
    rng = np.random.default_rng(3)
    rows, dim = 6000, 64
    x = rng.standard_normal((rows, 1, dim)) * 2.0 ** rng.integers(-133, 120, (rows, 1, 1))
    on = rng.integers(0, 31, (rows // 2, 1, dim)) * 0.5 * 2.0 ** rng.integers(-125, 110, (rows // 2, 1, 1))
    x[::2] = on + rng.integers(-3, 4, (rows // 2, 1, 1)) * on.max(-1, keepdims=True)
    x[1, 0, :2] = 3.3895313892515355e38, -1.2e36  # their difference is finite, just
    x = torch.from_numpy(x).to(torch.bfloat16).cuda()
    cache = ss.alloc_cache(1, 6, 1, 1024, dim, "int4")
    st = ints([-1])
    ss.ss_cache_append(cache, 0, x, x, ints([list(range(6))]), ints([0]), st, token_offsets=ints([0, rows]),
                       max_tokens=rows)
    torch.cuda.synchronize()
    n, step, low = R.quantise(np32(x)[:, 0])
    assert st.tolist() == [0] and np.isfinite(step).all()
    cells = cache.k[0].cpu().numpy().reshape(-1, dim // 2)[:rows]
    assert (cells == R.pack(n)).all()
    pairs = cache.k_scale[0].float().cpu().numpy().reshape(-1, 2)[:rows]
    assert (pairs[:, 0] == step).all() and (pairs[:, 1] == low).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_reports_holes_and_bad_requests(ss, fmt):
    cache = ss.alloc_cache(1, 6, 2, 16, 64, fmt)
    x = torch.randn(40, 2, 64, device="cuda").to(torch.bfloat16)
    table = ints([[0, -1], [1, 2], [3, 9], [4, 5]])
    st = ints([-1] * 4)
    # request 0 runs into a hole, 1 beyond the table, 2 into an entry that is no page, 3 has too many tokens
    ss.ss_cache_append(cache, 0, x, x, table, ints([10, 30, 15, 0]), st, token_offsets=ints([0, 10, 20, 25, 40]),
                       max_tokens=10)
    torch.cuda.synchronize()
    assert st.tolist() == [3, 3, 3, 4]
    y, z = torch.full_like(x, 5), torch.full_like(x, 5)
    ss.ss_cache_read(cache, 0, y, z, table, ints([10, 30, 15, 0]), st, token_offsets=ints([0, 10, 20, 25, 40]),
                     max_tokens=10)
    torch.cuda.synchronize()
    done = [0, 1, 2, 3, 4, 5, 10, 11, 20]
    left = [i for i in range(25) if i not in done]
    assert bool((y[left] == 0).all()) and bool((y[25:] == 5).all()) and bool((y[done] != 0).any(-1).all())
    assert not bool(cache.k[0, 4:].any())
    st = ints([-1] * 3)
    ss.ss_cache_append(cache, 0, x[:3], x[:3], table, ints([0, -2, 3]), st, table_rows=ints([3, 0, 7]))
    torch.cuda.synchronize()
    assert st.tolist() == [0, 4, 4]


# ----------------------------------------------------------------- pages --

def pool_of(ss, table, refs, free, page, pages):
    stack = free + [-7] * (pages - len(free))
    return ss.PagePool(ints(table), ints(refs), ints(stack), ints([len(free)]), page)


def same(pool, ref):
    torch.cuda.synchronize()
    n = int(pool.free_count.item())
    assert pool.page_table.tolist() == ref.table
    assert pool.ref_count.tolist() == ref.refs
    assert pool.free_pages[:n].tolist() == ref.free


@pytest.mark.parametrize("seed", range(6))
def test_pages_against_lists(ss, seed):
    rng = random.Random(seed)
    page, rows, width = 8, 40, [3, 9, 33, 70, 5, 128][seed]
    pages = rng.choice([rows * width // 2, 60, 1000])
    pages = max(pages, 8)
    order = list(range(pages))
    rng.shuffle(order)
    pool = pool_of(ss, [[-1] * width for _ in range(rows)], [0] * pages, order, page, pages)
    ref = R.Pages([[-1] * width for _ in range(rows)], [0] * pages, order, page)
    cache = ss.alloc_cache(1, pages, 1, page, 8, "bf16")
    lens = [0] * rows
    for _ in range(30):
        what = rng.choice(["reserve", "reserve", "fork", "trim", "free"])
        pick = rng.sample(range(rows), rng.randint(1, rows // 2))
        st = ints([-1] * len(pick))
        if what == "reserve":
            start = [lens[r] for r in pick]
            stop = [min(width * page, a + rng.randint(0, 3 * page)) for a in start]
            ss.ss_pages_reserve(pool, ints(start), ints(stop), st, table_rows=ints(pick))
            want = ref.reserve(pick, start, stop)
            for r, s, b in zip(pick, want, stop):
                lens[r] = b if s == 0 else lens[r]
        elif what == "fork":
            empty = [r for r in range(rows) if all(e < 0 for e in ref.table[r])]
            full = [r for r in range(rows) if lens[r] and r not in empty]
            if not empty or not full:
                continue
            child = rng.sample(empty, min(len(empty), rng.randint(1, 8)))
            parent = [rng.choice(full) for _ in child]
            n = [rng.randint(0, lens[p]) for p in parent]
            st = ints([-1] * len(child))
            ss.ss_pages_fork(pool, cache, ints(parent), ints(child), ints(n), st)
            want, _ = ref.fork(parent, child, n)
            for c, s, b in zip(child, want, n):
                lens[c] = b if s == 0 else 0
        else:
            keep = [0 if what == "free" else rng.randint(0, lens[r]) for r in pick]
            window, sinks = (0, 0) if what == "free" else (rng.choice([0, 5, 20, 100]), rng.choice([0, 3, 20]))
            ss.ss_pages_trim(pool, ints(keep), st, window=window, sinks=sinks, table_rows=ints(pick))
            want = ref.trim(pick, keep, window, sinks)
            for r, n in zip(pick, keep):
                lens[r] = n
        torch.cuda.synchronize()
        assert st.tolist() == want, what
        same(pool, ref)


def test_pages_many_requests(ss):
    # more requests than one pass of the bookkeeping takes
    n, page, width = 2500, 16, 3
    pages = n * 2
    pool = ss.alloc_pool(n, width, pages, page)
    ref = R.Pages([[-1] * width for _ in range(n)], [0] * pages, list(range(pages - 1, -1, -1)), page)
    start, stop = [0] * n, [(i * 7) % 40 for i in range(n)]
    st = ints([-1] * n)
    ss.ss_pages_reserve(pool, ints(start), ints(stop), st)
    assert ref.reserve(range(n), start, stop) == st.tolist()
    same(pool, ref)
    keep = [(i * 5) % 33 for i in range(n)]
    ss.ss_pages_trim(pool, ints(keep), st)
    assert ref.trim(range(n), keep, 0, 0) == st.tolist()
    same(pool, ref)


@pytest.mark.parametrize("n,width", [(8, 1024), (9, 1024), (3, 5000), (700, 30)])
def test_pages_wide_tables(ss, n, width):
    # on both sides of the sizes that the bookkeeping holds in registers
    rng = random.Random(n * width)
    page, rows = 8, 2 * n
    pages = n * width + n // 2
    order = list(range(pages))
    rng.shuffle(order)
    pool = pool_of(ss, [[-1] * width for _ in range(rows)], [0] * pages, order, page, pages)
    ref = R.Pages([[-1] * width for _ in range(rows)], [0] * pages, order, page)
    cache = ss.alloc_cache(1, pages, 1, page, 8, "bf16")
    st = ints([-1] * n)
    full = [rng.randint(0, width * page) for _ in range(n)]
    full[0] = width * page
    for part in (0.3, 1.0):  # the second time the first entries are held
        stop = [int(part * x) for x in full]
        ss.ss_pages_reserve(pool, ints([0] * n), ints(stop), st)
        assert ref.reserve(range(n), [0] * n, stop) == st.tolist()
        same(pool, ref)
    child = [n + i for i in range(n)]
    ss.ss_pages_fork(pool, cache, ints(list(range(n))), ints(child), ints(full), st)
    want, _ = ref.fork(list(range(n)), child, full)
    assert st.tolist() == want
    same(pool, ref)
    for rows_, window, sinks in ((list(range(n)), 100, 9), (child, 0, 0), (list(range(n)), 0, 0)):
        keep = full if window else [rng.randint(0, 50) for _ in rows_]
        ss.ss_pages_trim(pool, ints(keep), st, window=window, sinks=sinks, table_rows=ints(rows_))
        assert ref.trim(rows_, keep, window, sinks) == st.tolist()
        same(pool, ref)


def test_pages_bad_arguments_per_row(ss):
    pool = pool_of(ss, [[0, 1], [-1, -1], [2, 9]], [1, 0, 1, 0], [3], 8, 4)
    ref = R.Pages([[0, 1], [-1, -1], [2, 9]], [1, 0, 1, 0], [3], 8)
    st = ints([-1] * 5)
    a, b = [0, 5, 3, -1, 0], [17, 3, 4, 4, 1]
    ss.ss_pages_reserve(pool, ints(a), ints(b), st, table_rows=ints([0, 1, 3, 1, -1]))
    assert ref.reserve([0, 1, 3, 1, -1], a, b) == st.tolist() == [4] * 5
    same(pool, ref)
    # page 1's count is already 0, entry 9 is no page
    st = ints([-1] * 3)
    ss.ss_pages_trim(pool, ints([0, -1, 0]), st)
    assert ref.trim([0, 1, 2], [0, -1, 0], 0, 0) == st.tolist() == [3, 4, 3]
    same(pool, ref)


@pytest.mark.parametrize("fmt", FORMATS)
def test_fork_copies_the_last_page_in_every_layer(ss, fmt):
    rng = np.random.default_rng(5)
    layers, pages, heads, page, dim = 3, 12, 2, 16, 64
    cache = make_cache(ss, rng, fmt, pages, heads, page, dim, layers=layers)
    table = [[3, 7, -1], [5, -1, -1], [-1, -1, -1], [-1, -1, -1], [-1, -1, -1], [-1, -1, -1]]
    refs = [0] * pages
    for p in (3, 7, 5):
        refs[p] = 1
    free = [9, 1, 8]
    pool, ref = pool_of(ss, table, refs, free, page, pages), R.Pages(table, refs, free, page)
    old = [None if t is None else t.cpu().clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    parent, child, length = [0, 0, 1, 0], [2, 3, 4, 5], [21, 16, 9, 32]
    st = ints([-1] * 4)
    ss.ss_pages_fork(pool, cache, ints(parent), ints(child), ints(length), st)
    want, copies = ref.fork(parent, child, length)
    assert st.tolist() == want == [0] * 4 and len(copies) == 2
    same(pool, ref)
    for t, o in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), old):
        if t is None:
            continue
        for src, dst, n in copies:
            o[:, dst, :, :n] = o[:, src, :, :n]
        assert torch.equal(t.cpu().view(torch.uint8), o.view(torch.uint8))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,heads", [(64, 3), (128, 8)])
def test_compact(ss, fmt, dim, heads):
    rng, pr = np.random.default_rng(6), random.Random(6)
    layers, page, n, nodes = 3, 16, 9, 64
    lens = [0, 1, 13, 16, 40, 15, 7, 20, 3]
    width = 8
    pages = n * width + 1
    table = rng.permutation(pages)[:n * width].reshape(n, width).tolist()
    cache = make_cache(ss, rng, fmt, pages, heads, page, dim, layers=layers)
    tensors = (cache.k, cache.v, cache.k_scale, cache.v_scale)
    old = [None if t is None else t.cpu().clone() for t in tensors]
    counts = [0, 1, 5, 63, 12, 3, 4, 2, 2]
    path = []
    for i, c in enumerate(counts):
        p = sorted(pr.sample(range(1, nodes), c))
        path.append(p + [-1] * (nodes - c))
    path[7][:2] = [5, 5]       # not increasing
    table[8][0] = -1           # in a hole
    verified = [0] * n
    verified[6] = 2
    new, st = ints([-1] * n), ints([-1] * n)
    pool = ss.alloc_pool(n, width, pages, page)
    pool.page_table.copy_(ints(table))
    ss.ss_pages_compact(pool, cache, ints(lens), ints(path), ints(counts), ints(verified), new, st)
    torch.cuda.synchronize()
    assert st.tolist() == [0, 0, 0, 0, 0, 0, 2, 3, 3]
    assert new.tolist() == [a + 1 + c for a, c in zip(lens[:6], counts[:6])] + lens[6:]
    for t, o in zip(tensors, old):
        if t is None:
            continue
        w = o.clone()
        for i in range(6):
            for j in range(counts[i]):
                s, d = lens[i] + path[i][j], lens[i] + 1 + j
                w[:, table[i][d // page], :, d % page] = o[:, table[i][s // page], :, s % page]
        assert torch.equal(t.cpu().view(torch.uint8), w.view(torch.uint8))
    st2 = ints([-1] * 3)
    ss.ss_pages_compact(pool, cache, ints([-1, 0, 0]), ints(path[:3]), ints([1, 65, -1]), None, new[:3].clone(), st2)
    torch.cuda.synchronize()
    assert st2.tolist() == [4, 4, 4]
