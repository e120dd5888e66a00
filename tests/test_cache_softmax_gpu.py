"""The softmax of ss_cache_attention where its references matter: items whose
scores lie far apart one after the other, weights far below a row's largest.
Many requests share a few pages, so that the batch is large and its 64-bit
results are computed once per distinct request."""
import numpy as np
import pytest

from tests import cache_ref as R
from tests.test_cache_gpu import FORMATS, dense, ints, make_cache, np32, ss, workspace  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def exact(cache, q, table_row, base, scale):
    """One request of one query [heads, dim]: out, lse and the tolerance's sum p |v| / sum p."""
    k, v, mv = dense(cache)
    o, l, m, _ = R.attend(np32(q)[None].astype(np.float64), lambda p, s: (k[p, :, s], v[p, :, s], mv[p, :, s]), table_row,
                          cache.page_size, base, scale, 0, 0, None, cache.num_pages)
    return o[0], l[0], m[0]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heads", [4, 16, 32, 64, 128])
def test_an_item_starts_from_references_of_its_own(ss, workspace, fmt, heads):
    # Short requests, several per SM one after the other, whose scores lie around +70, 0 and -90 in turn: a reference
    # left over from the item before would be off by 2^100 and more.  Every request of a kind has the same queries and
    # keys; the batch is cut over the SMs anyhow, and a piece's reference changes the fp32 sums' last places only.
    rng = np.random.default_rng(heads)
    dim, page, n = 64, 16, 1500
    cache = make_cache(ss, rng, fmt, 9, 1, page, dim)
    for t in ((cache.k,) if fmt == "bf16" else ()):
        t[..., 0] = 1.0
    if fmt == "int4":  # channel 0 stands for 15 s + m = 1: the rows' largest nibble
        cache.k[..., 0] |= 15
        step = cache.k_scale[..., 0]
        step.copy_(0.125 * torch.ones_like(step))
        cache.k_scale[..., 1] = 1 - 15 * 0.125
    far = (70.0, 0.0, -90.0)
    q = torch.from_numpy(R.bf16(rng.standard_normal((3, heads, dim)))).to(torch.bfloat16).cuda()
    for i, x in enumerate(far):
        q[i, :, 0] = x
    lens = [100, 131, 17]
    kind = torch.arange(n) % 3
    table = ints([[0, 1, 2, 3, 4, 5, 6, 7, 8]] * n)
    base = ints([lens[i] for i in kind.tolist()])
    batch = q[kind.cuda()].contiguous()
    want = [exact(cache, q[i], list(range(9)), lens[i], 1.0) for i in range(3)]
    first = None
    for _ in range(10):
        out, lse, st = torch.full_like(batch, 7), torch.full((n, heads), 7.0, device="cuda"), ints([-1] * n)
        ss.ss_cache_attention(cache, 0, batch, out, table, base, workspace, st, scale=1.0, lse=lse)
        torch.cuda.synchronize()
        assert not st.any()
        if first is None:
            first = (out, lse)
            for i, (o, l, m) in enumerate(want):
                tol = 2.0 ** -8 * (np.abs(o) + m) * (1 + 1 / 16)
                got = np32(out[i::3]).astype(np.float64)
                assert (np.abs(got - o) <= tol).all(), far[i]
                # scores of up to 90 + 64 products, each to 2^-24 of it
                assert (np.abs(lse[i::3].cpu().numpy() - l) <= 2.0 ** -17 * (90 + 64)).all(), far[i]
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
