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


@pytest.mark.parametrize("spread", [1.0, 0.02])
@pytest.mark.parametrize("heads", [4, 16, 32, 64])
def test_a_sink_over_a_long_4_bit_context(ss, workspace, heads, spread):
    """One key takes about half of the mass of 64k keys, and all scores have a
    constant added to them, -24 to 12: each of the others weighs 2^-16 of the
    first, and together they count as much.

    Tolerance: the result's rounding to bf16 (2^-8 of it); each weight's to f16, 11 significant bits, so 2^-11 of
    sum p (s |n - 8| + |m + 8 s|) / sum p; and half as much for the fp32 scores, exponentials and sums.  A weight that
    loses bits because f16's range ends is not in it."""
    dim, page, keys = 128, 1024, 1 << 16
    gen = torch.Generator(device="cuda").manual_seed(heads)
    n = torch.full((1, keys // page, 1, page, dim), 8, dtype=torch.uint8, device="cuda")
    n[..., 2:] = torch.randint(6, 11, n[..., 2:].shape, generator=gen, device="cuda", dtype=torch.uint8)
    n[..., 1] = 15
    n[0, 0, 0, 0, 0] = 15  # the sink is the first key: 7/8 in channel 0, the others 0
    v = torch.randint(0, 16, n.shape, generator=gen, device="cuda", dtype=torch.uint8)

    def packed(x):
        x = x.unflatten(-1, (-1, 8))[..., [0, 2, 4, 6, 1, 3, 5, 7]].flatten(-2)
        return x[..., 0::2] | (x[..., 1::2] << 4)

    pairs = []
    for step, low in ((0.125, -1.0), (0.25 * spread, -7.5 * 0.25 * spread)):
        pair = torch.empty(1, keys // page, 1, page, 2, device="cuda")
        pair[..., 0], pair[..., 1] = step, low
        pairs.append(pair.to(torch.bfloat16))
    cache = ss.KVCache(packed(n), packed(v), *pairs)
    # enough requests for an item per SM; they take turns at the constants and share the pages
    count = torch.cuda.get_device_properties(0).multi_processor_count
    consts = [x * 0.5 for x in range(-48, 25)]
    q = torch.randn(len(consts), heads, dim, generator=gen, device="cuda") * 0.05
    q[..., 0] = 12.0 / 0.875
    q[..., 1] = torch.tensor(consts, device="cuda")[:, None] / 0.875
    q = q.to(torch.bfloat16)
    kind = torch.arange(count, device="cuda") % len(consts)
    batch = q[kind].contiguous()
    out, lse, st = torch.full_like(batch, 7), torch.full((count, heads), 7.0, device="cuda"), ints([-1] * count)
    ss.ss_cache_attention(cache, 0, batch, out, ints([list(range(keys // page))] * count), ints([keys - 1] * count), workspace,
                          st, scale=1.0, lse=lse)
    torch.cuda.synchronize()
    assert not st.any()
    k64 = (n[0, :, 0].flatten(0, 1).double() * 0.125 - 1.0)
    s, m = (pairs[1][0, 0, 0, 0, i].double() for i in (0, 1))
    v64 = v[0, :, 0].flatten(0, 1).double()
    x = q.double().flatten(0, 1) @ k64.T
    p = torch.softmax(x, -1)
    want = (p @ (s * v64 + m)).view(len(consts), heads, dim)
    mag = (p @ (s * (v64 - 8).abs() + (m + 8 * s).abs())).view(len(consts), heads, dim)
    share = p[:, 0]
    assert 0.3 < float(share.min()) and float(share.max()) < 0.95
    err = (out.double() - want[kind]).abs()
    tol = (2.0 ** -8 + 2.0 ** -12) * want.abs() + (2.0 ** -11 + 2.0 ** -12) * mag
    worst = (err / tol[kind]).amax((1, 2))
    assert float(worst.max()) <= 1, [(consts[i], round(float(worst[i]), 1)) for i in range(len(consts)) if worst[i] > 1]
    reach = (q.double().abs().flatten(0, 1) @ k64.abs().T).amax(-1).view(len(consts), heads)
    want_lse = torch.logsumexp(x, -1).view(len(consts), heads)
    assert ((lse.double() - want_lse[kind]).abs() <= 2.0 ** -17 * (reach + 1)[kind]).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heads", [2, 32, 128])
@pytest.mark.parametrize("power", [92, -80])
def test_large_and_small_values_with_large_and_small_scores(ss, workspace, fmt, heads, power):
    # Scores around -44 to 42 (64 powers of two both ways) with values around 2^92 and 2^-80, 700 keys: the products of
    # weights and values stay in fp32's range.  The file's own tolerance: nothing is lost at either end.
    rng = np.random.default_rng(power + 100)
    dim, page, keys = 64, 16, 700
    entries = -(-keys // page)
    cache = make_cache(ss, rng, fmt, entries, 1, page, dim)
    if fmt == "bf16":
        cache.k[..., 0] = 1.0
        cache.v.mul_(2.0 ** power)
    else:
        cache.k[..., 0] |= 15
        cache.k_scale[..., 0], cache.k_scale[..., 1] = 0.125, 1 - 15 * 0.125
        cache.v_scale.mul_(2.0 ** power)
    consts = list(range(-44, 43, 2))
    q = rng.standard_normal((len(consts), heads, dim)) * 0.1
    q[:, :, 0] = np.array(consts)[:, None]
    q = torch.from_numpy(R.bf16(q)).to(torch.bfloat16).cuda()
    out, st = torch.full_like(q, 7), ints([-1] * len(consts))
    ss.ss_cache_attention(cache, 0, q, out, ints([list(range(entries))] * len(consts)), ints([keys - 1] * len(consts)),
                          workspace, st, scale=1.0)
    torch.cuda.synchronize()
    assert not st.any()
    k, v, mv = (x[:, 0].reshape(-1, dim)[:keys] for x in dense(cache))
    x = np32(q).astype(np.float64) @ k.T
    p = np.exp(x - x.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    o, m = p @ v, p @ mv
    bad = ~(np.abs(np32(out) - o) <= 2.0 ** -8 * (np.abs(o) + m) * (1 + 1 / 16))
    assert not bad.any(), [consts[i] for i in range(len(consts)) if bad[i].any()]
