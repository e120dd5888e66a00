"""ss_rope_append: what its statuses leave behind, in every format."""
import numpy as np
import pytest

from tests.test_cache_gpu import ints, ss  # noqa: F401
from tests.test_rope_gpu import any_cache, half, parts

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
