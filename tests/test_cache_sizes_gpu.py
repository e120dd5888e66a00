"""Sizes at which 32 bits do not count or address everything: sinks and
lengths far beyond the table, more tiles than a call can walk, rows of lse past
2^31, page counts past 2^31.  Small memory where the sizes are only said."""
import numpy as np
import pytest

from tests import cache_ref as R
from tests.test_cache_gpu import FORMATS, dense, ints, make_cache, np32, ss, workspace  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FAR = 2 ** 31 - 300


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sinks", [2 ** 31 - 1, 2 ** 30, 70, 40])
def test_sinks_and_lengths_far_beyond_the_table(ss, workspace, fmt, sinks):
    # 200 requests in a window that has passed the table of four pages: the sinks that are in the table, no tiles
    # for the others
    n, page, heads, dim = 200, 16, 4, 64
    rng = np.random.default_rng(9)
    cache = make_cache(ss, rng, fmt, 8, 2, page, dim)
    q = torch.from_numpy(R.bf16(rng.standard_normal((n, heads, dim)))).to(torch.bfloat16).cuda()
    rows = rng.integers(0, 8, (n, 4)).tolist()
    out, lse, st = torch.full_like(q, 7), torch.full((n, heads), 7.0, device="cuda"), ints([-1] * n)
    ss.ss_cache_attention(cache, 0, q, out, ints(rows), ints([FAR] * n), workspace, st, lse=lse, window=500, sinks=sinks)
    torch.cuda.synchronize()
    assert st.tolist() == [3] * n
    # the keys of a query at the table's last slot, or at the last sink.  Held to the 64-bit results by the attention
    # tests' bound, not to such a call's bits: other lengths are cut over the SMs in other places.
    k, v, mv = dense(cache)
    for r in range(n):
        o, l, m, reach = R.attend(np32(q[r:r + 1]).astype(np.float64), lambda p, s: (k[p, :, s], v[p, :, s], mv[p, :, s]),
                                  rows[r], page, min(sinks, 4 * page) - 1, dim ** -0.5, 0, 0, None, 8)
        assert (np.abs(np32(out[r:r + 1]) - o) <= 2.0 ** -8 * (np.abs(o) + m) * (1 + 1 / 16)).all(), r
        assert (np.abs(lse[r].cpu().numpy() - l[0]) <= 2.0 ** -17 * reach[0] + 2.0 ** -21 * (1 + np.abs(l[0]))).all(), r


@pytest.mark.parametrize("fmt", FORMATS)
def test_more_tiles_than_can_be_walked(ss, workspace, fmt):
    # 2^14 requests of 2^24 tiles each: reported, nothing written, at once
    n, page, dim = 1 << 14, 1024, 64
    cache = make_cache(ss, np.random.default_rng(1), fmt, 2, 1, page, dim)
    q = torch.randn(n, 2, dim, device="cuda").to(torch.bfloat16)
    table = torch.zeros(1, 1 << 21, dtype=torch.int32, device="cuda")
    rows = torch.zeros(n, dtype=torch.int32, device="cuda")
    lens = torch.full((n,), FAR, dtype=torch.int32, device="cuda")
    lens[5] = -1
    out, lse, st = torch.full_like(q, 7), torch.full((n, 2), 7.0, device="cuda"), torch.full_like(lens, -1)
    ss.ss_cache_attention(cache, 0, q, out, table, lens, workspace, st, lse=lse, table_rows=rows)
    torch.cuda.synchronize()
    want = torch.full_like(st, 6)
    want[5] = 4
    assert torch.equal(st, want) and bool((out == 7).all()) and bool((lse == 7).all())
    # a window makes the same requests short
    ss.ss_cache_attention(cache, 0, q, out, table, lens, workspace, st, lse=lse, table_rows=rows, window=100, sinks=3)
    torch.cuda.synchronize()
    want.zero_()
    want[5] = 4
    assert torch.equal(st, want) and bool((lse[6:] != 7).all()) and bool((out[5] == 7).all())


def test_a_request_of_more_tiles_than_31_bits_count(ss, workspace):
    # 2^22 queries of 64 heads over 2^30 keys: refused for itself, the request beside it is done
    heads, dim, page, many = 64, 32, 1024, 1 << 22
    cache = make_cache(ss, np.random.default_rng(2), "int4", 2, 1, page, dim)
    q = torch.randn(1, heads, dim, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 7)
    table = torch.zeros(1, 1 << 21, dtype=torch.int32, device="cuda")
    st = ints([-1, -1])
    ss.ss_cache_attention(cache, 0, q.expand(many + 1, -1, -1), out.expand(many + 1, -1, -1), table, ints([200, 1 << 30]),
                          workspace, st, query_offsets=ints([0, 1, many + 1]), max_queries=many, table_rows=ints([0, 0]))
    torch.cuda.synchronize()
    assert st.tolist() == [0, 4]
    k, v, mv = dense(cache)
    o, _, m, _ = R.attend(np32(q).astype(np.float64), lambda p, s: (k[p, :, s], v[p, :, s], mv[p, :, s]), [0], page, 200,
                          dim ** -0.5, 0, 0, None, 2)
    assert (np.abs(np32(out) - o) <= 2.0 ** -8 * (np.abs(o) + m) * (1 + 1 / 16)).all()


def test_rows_of_lse_past_31_bits(ss, workspace):
    # one query whose row of lse is number 2^24 of 128 heads
    heads, dim, page, first = 128, 32, 16, 1 << 24
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 9 GB of device memory")
    cache = make_cache(ss, np.random.default_rng(3), "int4", 4, 1, page, dim)
    q = torch.from_numpy(R.bf16(np.random.default_rng(4).standard_normal((1, heads, dim)))).to(torch.bfloat16).cuda()
    out, st = torch.full_like(q, 7), ints([-1])
    lse = torch.full((first + 3, heads), 7.0, device="cuda")
    ss.ss_cache_attention(cache, 0, q.expand(first + 3, -1, -1), out.expand(first + 3, -1, -1), ints([[0, 1, 2, 3]]), ints([50]),
                          workspace, st, query_offsets=ints([first + 1, first + 2]), max_queries=1, lse=lse)
    torch.cuda.synchronize()
    assert st.tolist() == [0]
    k, v, mv = dense(cache)
    o, l, m, reach = R.attend(np32(q).astype(np.float64), lambda p, s: (k[p, :, s], v[p, :, s], mv[p, :, s]), [0, 1, 2, 3], page,
                              50, dim ** -0.5, 0, 0, None, 4)
    assert (np.abs(np32(out) - o) <= 2.0 ** -8 * (np.abs(o) + m) * (1 + 1 / 16)).all()
    got = lse[first + 1].cpu().numpy()
    assert (np.abs(got - l[0]) <= 2.0 ** -17 * reach[0] + 2.0 ** -21 * (1 + np.abs(l[0]))).all()
    assert bool((lse[first] == 7).all()) and bool((lse[first + 2] == 7).all()) and bool((lse[:100] == 7).all())


def test_reserving_more_pages_than_31_bits_count(ss):
    # nine rows of 2^28 holes want 2^31 + 2^28 pages of a pool of 16: none fits, none is taken
    rows, entries, page = 9, 1 << 28, 8
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 10 GB of device memory")
    pool = ss.alloc_pool(rows, entries, 16, page)
    st = ints([-1] * rows)
    ss.ss_pages_reserve(pool, ints([0] * rows), ints([2 ** 31 - 1] * rows), st)
    torch.cuda.synchronize()
    assert st.tolist() == [6] * rows
    assert int(pool.free_count) == 16 and not bool(pool.ref_count.any())
    assert pool.free_pages.tolist() == list(range(15, -1, -1))
    assert all(bool((pool.page_table[r] == -1).all()) for r in range(rows))
    # rows that want little get it
    ss.ss_pages_reserve(pool, ints([0] * rows), ints([8] * 4 + [0] * 4 + [2 ** 31 - 1]), st)
    torch.cuda.synchronize()
    assert st.tolist() == [0] * 8 + [6] and pool.page_table[:, 0].tolist() == [0, 1, 2, 3] + [-1] * 5


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_step_in_which_no_request_has_tokens(ss, workspace, fmt):
    cache = make_cache(ss, np.random.default_rng(5), fmt, 4, 2, 16, 64)
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]
    table, offsets = ints([[0], [1], [2]]), ints([0] * 4)
    k = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(0, 4, device="cuda")
    for lens, want in (([3, 0, 15], [0, 0, 0]), ([3, -1, 40], [0, 4, 0])):
        for most in (0, 1, 8):
            st = ints([-1] * 3)
            ss.ss_cache_append(cache, 0, k, k, table, ints(lens), st, token_offsets=offsets, max_tokens=most)
            assert st.tolist() == want
            st = ints([-1] * 3)
            ss.ss_cache_read(cache, 0, k, k, table, ints(lens), st, token_offsets=offsets, max_tokens=most)
            assert st.tolist() == want
            for parents in (None, torch.empty(0, dtype=torch.int32, device="cuda")):
                st = ints([-1] * 3)
                ss.ss_cache_attention(cache, 0, q, q, table, ints(lens), workspace, st, query_offsets=offsets,
                                      max_queries=most, lse=lse, parents=parents)
                assert st.tolist() == want
    after = [t for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]
    assert all(torch.equal(a, b) for a, b in zip(after, before))
    # and none at all
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    ss.ss_cache_append(cache, 0, k, k, table, none, none, max_tokens=1)
    ss.ss_cache_attention(cache, 0, q, q, table, none, workspace, none)
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", FORMATS)
def test_compact_at_the_last_length(ss, fmt):
    # new_len = kv_len + 1 + accepted would pass 2^31 - 1
    cache, pool = ss.alloc_cache(1, 4, 1, 16, 64, fmt), ss.alloc_pool(3, 4, 4, 16)
    lens, new, st = [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 2], ints([-1] * 3), ints([-1] * 3)
    path = ints([[1, 2]] * 3)
    ss.ss_pages_compact(pool, cache, ints(lens), path, ints([0, 0, 1]), None, new, st)
    torch.cuda.synchronize()
    assert st.tolist() == [4, 0, 4] and new.tolist() == [2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 2]


@pytest.mark.parametrize("fmt,heads", [("bf16", 4), ("bf16", 128), ("int4", 4), ("int4", 64)])
def test_items_that_take_a_tenth_of_a_second(ss, workspace, fmt, heads):
    # Several items per SM of 2^24 keys each (one page, 2^14 times): a warp that waits for the end of an item does not
    # give up as one that waits for a tile does.  Each thread adds up 2^17 weights in fp32, so a sum is off by at most
    # 2^17 units of 2^-24 of it, 2^-7, and the quotient of two by twice that, beside the attention tests' bound.
    times, page, dim = 1 << 14, 1024, 64
    n = 3 * torch.cuda.get_device_properties(0).multi_processor_count + 5
    rng = np.random.default_rng(heads)
    cache = make_cache(ss, rng, fmt, 1, 1, page, dim)
    q = torch.from_numpy(R.bf16(rng.standard_normal((3, heads, dim)))).to(torch.bfloat16).cuda()
    batch = q[torch.arange(n, device="cuda") % 3].contiguous()
    out, lse, st = torch.full_like(batch, 7), torch.full((n, heads), 7.0, device="cuda"), ints([-1] * n)
    table, rows = torch.zeros(1, times, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    lens = torch.full((n,), times * page - 1, dtype=torch.int32, device="cuda")
    ss.ss_cache_attention(cache, 0, batch, out, table, lens, workspace, st, table_rows=rows, lse=lse)
    torch.cuda.synchronize()
    late = bool((st == ss.SS_ROW_TIMEOUT).any())
    if late:
        workspace.zero_()
    assert not late and not st.any()
    k, v, mv = dense(cache)
    for i in range(3):
        o, l, m, _ = R.attend(np32(q[i:i + 1]).astype(np.float64), lambda p, s: (k[p, :, s], v[p, :, s], mv[p, :, s]), [0], page,
                              page - 1, dim ** -0.5, 0, 0, None, 1)
        err = np.abs(np32(out[i::3]).astype(np.float64) - o)
        assert (err <= 2.0 ** -8 * (np.abs(o) + m) * (1 + 1 / 16) + 2.0 ** -6 * m).all()
        assert (np.abs(lse[i::3].cpu().numpy() - (l + np.log(times))) <= 2.0 ** -7 + 2.0 ** -12).all()
