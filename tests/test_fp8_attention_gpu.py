"""Attention over the 8-bit cache on the GPU, against tests/cache_ref.py.

Tolerances.  An output row is sum_j p_j v_j / sum_j p_j with fp32 sums, p_j
times the block's scale rounded to f16 (2^-11 of it at most) and the result
rounded to bf16 (2^-8 of it): |error| <= 2^-8 |out| + 2^-11 sum p |v| / sum p.
Scores are fp32 sums of exact products (queries are two e4m3 numbers, exact but
for channels below 2^-15 of a row's largest): off by at most 2^-24 * 128 of sum
|q k|, so the weights by 2^-17 of it, in numerator and denominator, and a power
by a few units of 2^-22.  The log-sum carries the scores' error and a few units
of its own last place.
"""
import random

import numpy as np
import pytest

from tests import cache_ref as R
from tests import rope_ref as P
from tests.test_cache_gpu import Problem, ints, np32, random_parents, ss, workspace  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def make8(ss, rng, pages, heads, page, dim, layers=1, order="phsd", spread=3, pow2=True):
    """A cache of ordinary rows, its blocks' scales 2^-spread .. 2^spread apart (a few channels in 100,000, those past
    448, are NaN)."""
    blocks, block = max(1, page // 16), min(16, page)
    front = [0] + ["phs".index(x) + 1 for x in order[:3]] + [4]
    back = [0] + [1 + order[:3].index(x) for x in "phs"] + [4]
    parts, scales = [], []
    for _ in range(2):
        x = rng.standard_normal((layers, pages, heads, blocks, block, dim))
        s = np.exp2(rng.integers(-spread, spread + 1, x.shape[:4])) / 256 * (1 if pow2 else rng.uniform(0.6, 1.4, x.shape[:4]))
        n = torch.from_numpy(x * 100).cuda().to(torch.float8_e4m3fn).view(torch.uint8).flatten(3, 4)
        parts.append(n.permute(*front).contiguous().permute(*back).view(torch.float8_e4m3fn))
        scales.append(torch.from_numpy(s.astype(np.float32)).cuda())
    return ss.KVCache(*parts, *scales)


def dense8(cache, layer=0):
    out = []
    for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        n = P.e4m3_of(x[layer].view(torch.uint8).cpu().numpy())
        out.append(n * np.repeat(s[layer].cpu().numpy().astype(np.float64), min(16, cache.page_size), -1)[..., None])
    return out[0], out[1], np.abs(out[1])


class Problem8(Problem):
    def __init__(self, ss, seed, lens, news, heads, kv_heads, dim, page, spread=3, pow2=True, **kw):
        super().__init__(ss, seed, "bf16", lens, news, heads, kv_heads, dim, page, **kw)
        self.cache = make8(ss, np.random.default_rng(seed + 1000), self.num_pages, kv_heads, page, dim,
                           order=kw.get("order", "phsd"), spread=spread, pow2=pow2)

    def spoil(self):
        """Rows that no query sees become NaN, and the scales of blocks of which none is seen."""
        keep = np.zeros((self.num_pages, self.page), bool)
        for row, a, b in zip(self.table, self.lens, self.news):
            for s in range(a + b):
                if 0 <= row[s // self.page] < self.num_pages:
                    keep[row[s // self.page], s % self.page] |= not self.window or s > a - self.window or s < self.sinks
        gone = torch.from_numpy(~keep).cuda()
        for t in (self.cache.k, self.cache.v):
            t.view(torch.uint8)[0].masked_fill_(gone[:, None, :, None], 0x7f)
        for t in (self.cache.k_scale, self.cache.v_scale):
            t[0].masked_fill_(gone.unflatten(1, (t.shape[3], -1)).all(-1)[:, None], float("nan"))

    def finite(self):
        for t in (self.cache.k, self.cache.v):
            b = t.view(torch.uint8)
            b.masked_fill_((b & 0x7f) == 0x7f, 0x7e)
        return self

    def check(self, ss, workspace):
        out, lse, st = self.call(ss, workspace)
        assert st.cpu().tolist() == [0] * len(self.lens)
        assert not bool(workspace[:256].any())
        got, gl = np32(out).astype(np.float64), lse.cpu().numpy().astype(np.float64)
        k, v, mv = dense8(self.cache)
        q = np32(self.q).astype(np.float64)
        for r, (a, n) in enumerate(zip(self.lens, self.news)):
            lo, hi = self.offsets[r], self.offsets[r + 1]
            par = self.parents[r] if self.parents is not None else None
            o, l, m, reach = R.attend(q[lo:hi], lambda p, s: (k[p, :, s], v[p, :, s], mv[p, :, s]), self.table[r], self.page,
                                      a, self.scale, self.window, self.sinks, par, self.num_pages)
            tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + (2.0 ** -16 * reach[..., None] + 2.0 ** -19)) * m * (1 + 2.0 ** -8) + 1e-30
            # a query that sees a NaN gets a row that is not finite, whatever its channels
            seen = np.isnan(o).any(-1, keepdims=True)
            assert np.array_equal(seen, ~np.isfinite(got[lo:hi]).all(-1, keepdims=True))
            bad = ~(np.abs(got[lo:hi] - o) <= tol) & ~seen
            assert not bad.any(), (r, a, n, np.argwhere(bad)[:5], got[lo:hi][bad][:5], o[bad][:5], bad.mean())
            empty = np.isneginf(l)
            assert np.array_equal(np.isneginf(gl[lo:hi]), empty)
            tl = 2.0 ** -17 * reach + 2.0 ** -21 * (1 + np.abs(np.where(empty, 0, l)))
            badl = ~empty & ~((np.abs(gl[lo:hi] - np.where(empty, 0, l)) <= tl) | (np.isnan(gl[lo:hi]) & np.isnan(l)))
            assert not badl.any(), (r, gl[lo:hi][badl][:5], l[badl][:5])


@pytest.mark.parametrize("dim,heads,kv_heads,page", [
    (128, 8, 2, 16), (64, 4, 4, 32), (128, 7, 1, 64), (96, 6, 2, 8), (32, 3, 3, 128), (128, 128, 1, 16),
    (64, 10, 2, 256), (128, 16, 1, 1024), (128, 32, 1, 64), (48, 64, 1, 8), (80, 20, 4, 8)])
def test_lengths_and_layouts(ss, workspace, dim, heads, kv_heads, page):
    lens = [0, 1, 15, 16, 17, 126, 127, 128, 129, 255, 256, 300, 513, 1000]
    news = [1, 2, 1, 3, 1, 2, 1, 1, 8, 1, 5, 4, 1, 7]
    Problem8(ss, 1, lens, news, heads, kv_heads, dim, page).check(ss, workspace)


@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 96, 112])
def test_head_dims(ss, workspace, dim):
    for heads in (4, 40):
        Problem8(ss, 2, [5, 130, 400], [1, 3, 2], heads, 2, dim, 16, pow2=False).check(ss, workspace)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (5, 130), (64, 1), (127, 3), (128, 0), (129, 128), (200, 17),
                                          (1000, 4), (100000, 4)])
def test_window_and_sinks(ss, workspace, window, sinks):
    lens, news = [0, 3, 60, 127, 128, 200, 400, 777, 1200], [1, 5, 3, 2, 4, 1, 8, 1, 6]
    for heads, dim in ((8, 64), (16, 128)):
        p = Problem8(ss, 4, lens, news, heads, 2, dim, 16, window=window, sinks=sinks, evict=True)
        p.spoil()
        p.check(ss, workspace)


@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 1), (40, 4), (300, 150)])
@pytest.mark.parametrize("heads,kv_heads", [(4, 4), (8, 1), (12, 4)])
def test_trees(ss, workspace, window, sinks, heads, kv_heads):
    lens, news = [0, 1, 100, 127, 250, 511, 64], [64, 1, 33, 2, 64, 17, 63]
    p = Problem8(ss, 5, lens, news, heads, kv_heads, 64, 16, window=window, sinks=sinks, tree=True)
    p.spoil()
    p.check(ss, workspace)


def test_prompt_chunks(ss, workspace):
    for seed, (lens, news, window) in enumerate([([0, 300], [300, 201], 0), ([130, 5], [257, 1], 100), ([0], [700], 33)]):
        p = Problem8(ss, 10 + seed, lens, news, 4, 2, 128, 32, window=window, sinks=4 if window else 0)
        p.spoil()
        p.check(ss, workspace)


def test_long_context_is_split_and_joined(ss, workspace):
    for lens, news, heads, kv in [([20011], [1], 2, 1), ([9000, 1, 5000], [3, 1, 4], 16, 2)]:
        Problem8(ss, 20, lens, news, heads, kv, 128, 64).check(ss, workspace)


def test_many_requests(ss, workspace):
    rng = random.Random(7)
    lens = [rng.choice([0, 1, rng.randint(0, 200), rng.randint(0, 600)]) for _ in range(333)]
    Problem8(ss, 21, lens, [rng.randint(1, 3) for _ in lens], 2, 1, 64, 16).check(ss, workspace)


@pytest.mark.parametrize("group,dim", [(8, 128), (24, 128), (24, 64), (60, 128), (100, 64), (128, 128)])
def test_many_items_for_every_block_of_rows(ss, workspace, group, dim):
    rng = random.Random(group)
    lens = [rng.randint(0, 500) for _ in range(160)]
    Problem8(ss, 40, lens, [1] * len(lens), 2 * group, 2, dim, 16).check(ss, workspace)


@pytest.mark.parametrize("heads,news", [(4, 1), (8, 3), (40, 1), (16, 5)])
@pytest.mark.parametrize("longest", [100, 300])
def test_items_of_few_tiles(ss, workspace, heads, news, longest):
    """Many items a CTA, of a tile each: not every warpgroup that unpacks values has one."""
    rng = random.Random(longest)
    lens = [rng.randint(longest - 100, longest) for _ in range(400)]
    Problem8(ss, 41, lens, [news] * len(lens), heads, 2, 64, 32).check(ss, workspace)


@pytest.mark.parametrize("order", ["pshd", "hpsd", "shpd"])
def test_cache_layouts(ss, workspace, order):
    Problem8(ss, 22, [100, 300], [2, 5], 4, 2, 64, 16, order=order).check(ss, workspace)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("heads", [4, 32])
def test_scores_far_apart(ss, workspace, sign, heads):
    # rising and falling scores of hundreds: the running maximum moves at every tile, early keys vanish
    p = Problem8(ss, 24, [900], [4], heads, 2, 64, 16)
    for b in range(57):
        p.cache.k_scale[0, p.table[0][b]] = sign * b * 0.002
    p.cache.k.view(torch.uint8).fill_(0x78)  # 256
    p.q.abs_()
    p.check(ss, workspace)


@pytest.mark.parametrize("low,high,zeros", [(-60, -60, False), (60, 60, False), (90, 90, False), (-40, 40, False),
                                            (-20, 0, True)])
def test_values_of_every_size(ss, workspace, low, high, zeros):
    rng = np.random.default_rng(abs(high) + 7)
    for news, heads in (([3, 1], 4), ([8, 5], 16)):
        p = Problem8(ss, 31, [700, 40], news, heads, 2, 64, 16, spread=0)
        f = torch.from_numpy(2.0 ** rng.integers(low, high + 1, p.cache.v_scale.shape)).float().cuda()
        if zeros:
            f[torch.from_numpy(rng.random(f.shape) < 0.3).cuda()] = 0
        p.cache.v_scale.mul_(f)
        p.check(ss, workspace)


def test_rows_that_see_nothing(ss, workspace):
    p = Problem8(ss, 25, [40, 200, 10], [2, 3, 1], 4, 2, 64, 16)
    p.table[0] = [-1] * len(p.table[0])
    p.table[2] = [p.num_pages + 5] * len(p.table[2])
    p.spoil()
    p.check(ss, workspace)
    p = Problem8(ss, 26, [300], [2], 4, 2, 64, 16, window=20, sinks=2)
    p.table[0][1:] = [-1] * (len(p.table[0]) - 1)
    p.check(ss, workspace)


@pytest.mark.parametrize("heads", [8, 16, 64])
def test_a_draft_that_is_not_finite_stays_on_its_branch(ss, workspace, heads):
    # one channel of one draft's key or value, or all of them, beside other drafts of its block
    p = Problem8(ss, 27, [150], [40], heads, 2, 64, 16, tree=True).finite()
    clean, clean_lse, _ = p.call(ss, workspace)
    _, line = R.paths(p.parents[0])
    node = next(i for i in range(1, 40) if 1 < sum(i in x for x in line) < 39)
    s = 150 + node
    page, row = p.table[0][s // 16], s % 16
    for which, channels in (("k", slice(None)), ("v", slice(None)), ("v", slice(63, 64)), ("v", slice(0, 1)), ("k", slice(17, 18))):
        t = getattr(p.cache, which).view(torch.uint8)
        before = t[0, page, :, row].clone()
        t[0, page, :, row, channels] = 0xff
        out, lse, _ = p.call(ss, workspace)
        t[0, page, :, row] = before
        for i in range(40):
            if node in line[i]:
                assert not torch.isfinite(out[i, :, channels if which == "v" else slice(None)]).all(dim=-1).any()
            else:
                assert torch.equal(out[i], clean[i]) and torch.equal(lse[i], clean_lse[i]), i


@pytest.mark.parametrize("heads", [4, 32, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_scale_that_is_not_finite(ss, workspace, heads, value):
    # of a block that the window has left for the last query, and that the first still sees
    p = Problem8(ss, 28, [300, 300], [20, 1], heads, 1, 128, 16, window=60).finite()
    for which in ("k_scale", "v_scale"):
        clean, clean_lse, _ = p.call(ss, workspace)
        t = getattr(p.cache, which)
        page = p.table[0][15]  # slots 240 .. 255: query i sees those from 241 + i on
        before = t[0, page].clone()
        t[0, page] = value
        out, lse, st = p.call(ss, workspace)
        t[0, page] = before
        # (keys of an infinite scale may have scores of minus infinity: weights of 0, as defined)
        for i in range(15) if (which, value) != ("k_scale", float("inf")) else ():
            assert not torch.isfinite(out[i]).all(dim=-1).any(), (which, i)
        assert torch.equal(out[15:], clean[15:]) and torch.equal(lse[15:], clean_lse[15:])
        assert st.tolist() == [0, 0]


def test_a_value_that_all_see(ss, workspace):
    # a NaN in a tile that no mask touches
    for heads in (4, 64):
        p = Problem8(ss, 29, [700], [3], heads, 1, 128, 16).finite()
        p.cache.v.view(torch.uint8)[0, p.table[0][3], 0, 5, 77] = 0x7f
        out, lse, _ = p.call(ss, workspace)
        assert torch.isnan(out[..., 77]).all() and torch.isfinite(out[..., :77]).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("spread", [1.0, 0.02])
@pytest.mark.parametrize("heads", [4, 16, 32, 64])
def test_a_sink_over_a_long_context(ss, workspace, heads, spread):
    """One key takes about half of the mass of 64k keys, and all scores have a constant added, -24 to 12: each of the
    others weighs 2^-16 of the first, and together they count as much."""
    dim, page, keys = 128, 1024, 1 << 16
    gen = torch.Generator(device="cuda").manual_seed(heads)
    k = torch.zeros(1, keys // page, 1, page, dim, device="cuda")
    k[..., 2:] = torch.randn(k[..., 2:].shape, generator=gen, device="cuda") * 4 * spread
    k[..., 0] = 1.0
    k[0, 0, 0, 0, 1] = 1.0  # the sink
    v = torch.randn(k.shape, generator=gen, device="cuda") * 64
    k, v = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
    scales = [torch.full((1, keys // page, 1, page // 16), x, device="cuda") for x in (0.25, 2.0 ** -6)]
    cache = ss.KVCache(k, v, *scales)
    q = torch.randn(1, heads, dim, generator=gen, device="cuda").to(torch.bfloat16)
    q[0, :, 0] = torch.linspace(-24 * 4, 12 * 4, heads).to(torch.bfloat16).cuda()
    kk, vv = k[0, :, 0].flatten(0, 1).double() * 0.25, v[0, :, 0].flatten(0, 1).double() * 2.0 ** -6
    rest = (kk[1:, 2:] @ q[0, :, 2:].double().T).logsumexp(0)  # of the others, without the constant
    q[0, :, 1] = ((rest - (kk[0, 2:] @ q[0, :, 2:].double().T)) * 4).to(torch.bfloat16)
    out, lse, st = torch.empty_like(q), torch.empty(1, heads, device="cuda"), ints([-1])
    ss.ss_cache_attention(cache, 0, q, out, ints([list(range(keys // page))]), ints([keys - 1]), workspace, st, scale=1.0, lse=lse)
    assert st.tolist() == [0]
    x = q[0].double() @ kk.T
    p = (x - x.logsumexp(-1, keepdim=True)).exp()
    want, mag = p @ vv, p @ vv.abs()
    reach = (q[0].double().abs() @ kk.abs().T).amax(-1, keepdim=True)
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -16 * reach + 2.0 ** -19) * mag
    assert bool(((out[0].double() - want).abs() <= tol).all())
    assert bool(((lse[0].double() - x.logsumexp(-1)).abs() <= 2.0 ** -17 * reach[:, 0] + 2.0 ** -18).all())


def test_same_bits_every_time_on_streams_and_in_graphs(ss, workspace):
    p = Problem8(ss, 29, [3000, 10, 777, 64], [4, 1, 8, 2], 16, 2, 128, 16).finite()
    out, lse, _ = p.call(ss, workspace)
    for _ in range(4):
        o2, l2, _ = p.call(ss, workspace)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o3, l3, _ = p.call(ss, workspace, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, o3) and torch.equal(lse, l3)
    o4, l4, st = torch.empty_like(out), torch.empty_like(lse), ints([0] * 4)
    table, lens, off = ints(p.table), ints(p.lens), ints(p.offsets)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            ss.ss_cache_attention(p.cache, 0, p.q, o4, table, lens, workspace, st, query_offsets=off, max_queries=8, lse=l4)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o4) and torch.equal(lse, l4)


def test_scales_of_neighbours_with_gaps(ss, workspace):
    # scales that lie next to other data, at addresses that are multiples of 4 alone
    p = Problem8(ss, 33, [100, 300], [2, 5], 4, 2, 64, 32).finite()
    c = p.cache
    wide = [torch.full((1, p.num_pages, 2, 5), float("nan"), device="cuda") for _ in range(2)]
    views = [w[..., 3:5] for w in wide]
    for a, b in zip(views, (c.k_scale, c.v_scale)):
        a.copy_(b)
    ref = p.call(ss, workspace)
    p.cache = ss.KVCache(c.k, c.v, *views)
    out = p.call(ss, workspace)
    assert torch.equal(ref[0], out[0]) and torch.equal(ref[1], out[1])


def test_bad_requests_are_reported_and_the_others_done(ss, workspace):
    p = Problem8(ss, 31, [50, 60, 70, 80], [2, 3, 1, 2], 4, 2, 64, 16).finite()
    ref, _, _ = p.call(ss, workspace)
    out, st = torch.full_like(p.q, 7.0), ints([-1] * 4)
    ss.ss_cache_attention(p.cache, 0, p.q, out, ints(p.table), ints([50, -1, 70, len(p.table[0]) * 16 - 1]), workspace, st,
                          query_offsets=ints(p.offsets), max_queries=3)
    assert st.tolist() == [0, 4, 0, 3] and torch.equal(out[:2], ref[:2]) and torch.equal(out[5:6], ref[5:6])
    assert bool((out[2:5] == 7).all())
    Problem8(ss, 32, [50, 60, 70], [2, 0, 1], 4, 2, 64, 16).check(ss, workspace)


@pytest.mark.parametrize("heads,tree", [(4, False), (16, True), (32, False), (64, True)])
@pytest.mark.parametrize("stall", ["items", "queries", "keys", "values", "scores", "weights", "packed"])
def test_a_wait_that_nothing_ends_gives_up(ss, workspace, heads, tree, stall):
    p = Problem8(ss, 50, [300, 700, 40, 0], [2, 5, 1, 3], heads, 1, 128, 16, window=200, sinks=4, tree=tree)
    out, lse, st = torch.full_like(p.q, 7.0), torch.full(p.q.shape[:2], 7.0, device="cuda"), ints([-1] * 4)
    ss.ss_selftest_attention_timeout(p.cache, 0, p.q, out, ints(p.table), ints(p.lens), workspace, st, stall=stall,
                                     query_offsets=ints(p.offsets), max_queries=max(p.news),
                                     parents=ints([x for r in p.parents for x in r]) if tree else None, scale=p.scale,
                                     window=p.window, sinks=p.sinks, lse=lse)
    torch.cuda.synchronize()
    assert st.tolist() == [ss.SS_ROW_TIMEOUT] * 4
    workspace.zero_()
    p.check(ss, workspace)


def test_a_layer_s_calls_together(ss, workspace):
    """Prompt, then steps of draft trees: turned, written, attended to, the accepted nodes packed; against the same
    from the plain forms."""
    pr, rng = random.Random(3), np.random.default_rng(3)
    heads, kv, dim, page, n = 8, 2, 64, 16, 3
    rope = ss.Rope(dim, rot_dim=48, layout="interleaved", scaling="linear", factor=2.0)
    table_of_turns = [int(t) for t in rope.turns.cpu().numpy().view(np.uint64)]
    cache, pool = ss.alloc_cache(1, 60, kv, page, dim, "fp8"), ss.alloc_pool(n, 20, 60, page)
    want = [P.Cache8(np.zeros((60, kv, page, dim), np.uint8), np.zeros((60, kv, 1))) for _ in range(2)]
    lens, st = [0] * n, ints([-1] * n)
    for step in range(5):
        news = [70, 3, 130] if step == 0 else [pr.randint(1, 30) for _ in range(n)]
        parents = None if step == 0 else [random_parents(pr, m) for m in news]
        offsets = [sum(news[:i]) for i in range(n + 1)]
        qkv = torch.from_numpy(R.bf16(rng.standard_normal((sum(news), heads + 2 * kv, dim)))).to(torch.bfloat16).cuda()
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
        kw = dict(parents=ints([p for r in parents for p in r])) if parents else {}
        ss.ss_pages_reserve(pool, ints(lens), ints([a + b for a, b in zip(lens, news)]), st)
        q_out, out = torch.empty(sum(news), heads, dim, dtype=torch.bfloat16, device="cuda"), None
        ss.ss_rope_append(rope, cache, 0, q, q_out, k, v, pool, ints(lens), st, token_offsets=ints(offsets),
                          max_tokens=max(news), **kw)
        assert st.tolist() == [0] * n
        table = pool.page_table.tolist()
        # the keys as the call turned them (test_rope_gpu.py holds these against the plain form)
        turned = torch.empty_like(k)
        ss.ss_rope(rope, None, None, k, turned, ints(lens), st, token_offsets=ints(offsets), max_tokens=max(news), **kw)
        at = P.positions(lens, news, parents)
        plain = P.turn(np32(k).astype(np.float64), at, table_of_turns, 48, "interleaved", 1.0)
        assert np.abs(np32(turned) - plain).max() <= 2.0 ** -8 * np.abs(plain).max()
        for x, w in ((turned, want[0]), (v, want[1])):
            for r in range(n):
                w.append(table[r], lens[r], np32(x[offsets[r]:offsets[r + 1]]).astype(np.float64))
        out, lse = torch.empty_like(q_out), torch.empty(sum(news), heads, device="cuda")
        ss.ss_cache_attention(cache, 0, q_out, out, pool, ints(lens), workspace, st, query_offsets=ints(offsets),
                              max_queries=max(news), lse=lse, **kw)
        assert st.tolist() == [0] * n
        values = [w.n * np.repeat(w.s, 16, -1)[..., None] for w in want]
        for r in range(n):
            o, l, m, reach = R.attend(np32(q_out[offsets[r]:offsets[r + 1]]).astype(np.float64),
                                      lambda p, s: (values[0][p, :, s], values[1][p, :, s], np.abs(values[1][p, :, s])),
                                      table[r], page, lens[r], dim ** -0.5, 0, 0, parents[r] if parents else None, 60)
            got = np32(out[offsets[r]:offsets[r + 1]])
            assert (np.abs(got - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -16 * reach[..., None] + 2.0 ** -18) * m).all()
        if parents is None:
            lens = list(news)
            continue
        # a node of the first level, then one of its children, and so on
        paths = []
        for row in parents:
            node, path = 0, []
            while True:
                below = [c for c in range(node + 1, len(row)) if row[c] == node]
                if not below or pr.random() < 0.1:
                    break
                node = pr.choice(below)
                path.append(node)
            paths.append(path)
        new_len = ints([-1] * n)
        ss.ss_pages_compact(pool, cache, ints(lens), ints([p + [-1] * (30 - len(p)) for p in paths]),
                            ints([len(p) for p in paths]), None, new_len, st)
        assert st.tolist() == [0] * n
        for r in range(n):
            for w in want:
                w.compact(table[r], lens[r], paths[r])
        lens = new_len.tolist()
        for x, s, w in ((cache.k, cache.k_scale, want[0]), (cache.v, cache.v_scale, want[1])):
            assert np.array_equal(s[0].cpu().numpy().astype(np.float64), w.s)
            assert np.array_equal(P.e4m3_of(x[0].view(torch.uint8).cpu().numpy()), w.n)
        ss.ss_pages_trim(pool, ints(lens), st)
