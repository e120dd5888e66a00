"""The log-sum over 8 bits where the values are far from 1.

The tolerance.  A row's reference is the largest score plus log2 of its key's
scale, less 8: up to |x| + |log2 s| + 8.  A score less the reference, the
reference's own sums and log2 of the sum (which takes the reference away again)
are rounded to 2^-24 of that each, and a reference moves a few times at most:
2^-21 (|log2 s| + 8) together, beside what the attention's tests allow."""
import numpy as np
import pytest

from tests import cache_ref as R
from tests.test_cache_gpu import np32, ss, workspace  # noqa: F401
from tests.test_fp8_attention_gpu import Problem8, dense8

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("spread,power", [(12, 0), (12, -40), (3, 30), (0, -60)])
@pytest.mark.parametrize("heads", [2, 32])
def test_the_log_sum_beside_small_and_large_values(ss, workspace, heads, spread, power):
    p = Problem8(ss, 70 + spread, [300, 5, 0, 700], [3, 4, 2, 1], heads, 2, 64, 16, spread=spread).finite()
    p.cache.v_scale *= 2.0 ** power
    p.cache.k_scale /= p.cache.k_scale.max() * 128  # (scores of ordinary size)
    _, lse, st = p.call(ss, workspace)
    assert st.tolist() == [0] * 4
    k, v, mv = dense8(p.cache)
    q = np32(p.q).astype(np.float64)
    for r, (a, n) in enumerate(zip(p.lens, p.news)):
        lo, hi = p.offsets[r], p.offsets[r + 1]
        _, want, _, reach = R.attend(q[lo:hi], lambda x, s: (k[x, :, s], v[x, :, s], mv[x, :, s]), p.table[r], p.page, a,
                                     p.scale, 0, 0, None, p.num_pages)
        near = 2.0 ** -17 * reach + 2.0 ** -21 * (1 + np.abs(want)) + 2.0 ** -21 * (spread + 8 + abs(power) + 8)
        assert (np.abs(lse[lo:hi].cpu().numpy() - want) <= near).all()
