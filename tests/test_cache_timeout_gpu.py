"""The bounded waits of the attention kernel: a wait that nothing ends gives
up, the requests' statuses say so, and the next call is right.  Each kind of
barrier by itself, in the kernel's different shapes."""
import time

import pytest

from tests.test_cache_gpu import Problem, ints, ss, workspace  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

STALLS = ["items", "queries", "keys", "values", "scores", "weights", "packed"]


def stalled(ss, p, workspace, stall, lens=None, offsets=None):
    out, lse = torch.full_like(p.q, 7.0), torch.full(p.q.shape[:2], 7.0, device="cuda")
    st = ints([-1] * len(p.lens))
    par = ints([x for row in p.parents for x in row]) if p.parents is not None else None
    ss.ss_selftest_attention_timeout(p.cache, 0, p.q, out, ints(p.table), ints(lens or p.lens), workspace, st, stall=stall,
                                     query_offsets=ints(offsets or p.offsets), max_queries=max(p.news), parents=par,
                                     scale=p.scale, window=p.window, sinks=p.sinks, lse=lse)
    torch.cuda.synchronize()
    return st.tolist()


# rows of an item: 8, 16, 32, 64 (two warpgroups or four), 128
@pytest.mark.parametrize("fmt,heads,tree", [("bf16", 2, False), ("bf16", 16, False), ("bf16", 64, True), ("bf16", 128, False),
                                            ("int4", 4, False), ("int4", 16, True), ("int4", 32, False), ("int4", 64, True)])
@pytest.mark.parametrize("stall", STALLS)
def test_a_wait_that_nothing_ends_gives_up(ss, workspace, fmt, heads, tree, stall):
    p = Problem(ss, 50, fmt, [300, 700, 40, 0], [2, 5, 1, 3], heads, 1, 128, 16, window=200, sinks=4, tree=tree)
    if stall == "packed" and fmt == "bf16":
        with pytest.raises(ss.SSError):
            stalled(ss, p, workspace, stall)
        return
    t0 = time.monotonic()
    assert stalled(ss, p, workspace, stall) == [ss.SS_ROW_TIMEOUT] * 4
    assert time.monotonic() - t0 < 20
    workspace.zero_()
    p.check(ss, workspace)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_only_requests_with_queries_time_out(ss, workspace, fmt):
    # bad requests and those without queries, at the ends and between others, keep their statuses
    lens, news = [50, 60, -1, 70, 80, 90, 10], [0, 2, 1, 0, 3, 1, 0]
    p = Problem(ss, 52, fmt, [max(x, 0) for x in lens], news, 4, 1, 64, 16)
    assert stalled(ss, p, workspace, "scores", lens=lens) == [0, 5, 4, 0, 5, 5, 0]
    # more requests than threads, most of them without queries
    n = 3000
    p = Problem(ss, 53, fmt, [20] * n, [int(i % 100 == 7) for i in range(n)], 4, 1, 64, 16)
    workspace.zero_()
    assert stalled(ss, p, workspace, "keys") == [5 * x for x in p.news]
    workspace.zero_()
    p.check(ss, workspace)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_a_workspace_that_was_not_zeroed_again_says_so(ss, workspace, fmt):
    # the counts of the pieces' joining may be off from then on: no call may pass that over
    p = Problem(ss, 54, fmt, [5000, 30], [2, 0], 4, 1, 64, 16)
    assert stalled(ss, p, workspace, "values") == [5, 0]
    for _ in range(2):
        assert p.call(ss, workspace)[2].tolist() == [5, 0]
    workspace.zero_()
    p.check(ss, workspace)


def test_the_self_test_checks_its_arguments(ss, workspace):
    p = Problem(ss, 51, "bf16", [30], [1], 2, 1, 64, 16)
    lib = ss.load()
    assert lib.ss_selftest_attention_timeout(None, 0, None, 0, None) == 1
    assert lib.ss_selftest_attention_timeout(None, 8, None, 0, None) == 1
    assert lib.ss_selftest_attention_timeout(None, 1, None, 0, None) == 1
    with pytest.raises(ss.SSError):
        stalled(ss, p, workspace.cpu(), "keys")
    p.check(ss, workspace)
