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
    q = torch.randn(n, heads, dim, device="cuda").to(torch.bfloat16)
    rows = rng.integers(0, 8, (n, 4)).tolist()
    out, lse, st = torch.full_like(q, 7), torch.full((n, heads), 7.0, device="cuda"), ints([-1] * n)
    ss.ss_cache_attention(cache, 0, q, out, ints(rows), ints([FAR] * n), workspace, st, lse=lse, window=500, sinks=sinks)
    torch.cuda.synchronize()
    assert st.tolist() == [3] * n
    # the same keys as those of a query at the table's last slot, or at the last sink
    want, want_lse, st2 = torch.empty_like(q), torch.empty_like(lse), ints([-1] * n)
    ss.ss_cache_attention(cache, 0, q, want, ints(rows), ints([min(sinks, 4 * page) - 1] * n), workspace, st2, lse=want_lse)
    torch.cuda.synchronize()
    assert st2.tolist() == [0] * n and torch.equal(out, want) and torch.equal(lse, want_lse)
