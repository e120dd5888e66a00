"""ss_cache_read of 8 bits with scales that are no powers of two: s * n, up to 28
bits long, is rounded to bf16 once, held bit for bit against 64-bit products
(exact) rounded once.  A product that fp32 would round onto a tie of bf16 is
where a second rounding shows; such scales are constructed."""
import numpy as np
import pytest

from tests import rope_ref as P
from tests.test_cache_gpu import ints, np32, ss  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def bf16_once(x):
    """float64 to the nearest bf16, ties to even, as float32."""
    with np.errstate(all="ignore"):
        _, e = np.frexp(x)
        step = np.exp2(np.maximum(e - 8, -133).astype(np.float64))
        y = np.rint(x / step) * step
        return np.where(np.isfinite(x), np.where(np.abs(y) >= 2.0 ** 128, np.copysign(np.inf, x), y), x).astype(np.float32)


def beside_ties(rng, count):
    """Scales s of which some e4m3 n has a product beside a tie of bf16 that fp32 rounds onto it."""
    out = []
    while len(out) < count:
        n = rng.integers(8, 16) / 8
        tie = (2 * int(rng.integers(128, 256)) + 1) / 256
        s = np.float32(tie / n) * np.float32(rng.choice([-1, 1]))
        if float(s) * n != np.copysign(tie, s) and np.abs(np.float32(s * np.float32(n))) == tie:
            out.append(float(s) * 2.0 ** int(rng.integers(-20, 20)))
    return out


@pytest.mark.parametrize("heads", [4, 3])
def test_products_are_rounded_once(ss, heads):
    rng = np.random.default_rng(heads)
    pages, page, dim = 160, 16, 16
    count = 2 * pages * heads
    scales = beside_ties(rng, count - 200)
    scales += (rng.uniform(1, 2, 160) * np.exp2(rng.integers(-30, 30, 160))).tolist()  # any
    scales += [0.0, -0.0, 1.0, -2.0, 2.0 ** -126, 2.0 ** 127, float("nan"), float("inf"), float("-inf"), 3e38, -3e38]
    scales += (rng.uniform(1, 2, 29) * np.exp2(rng.integers(-148, -117, 29))).tolist()  # products that are subnormal
    s = np.array(scales, np.float32)[rng.permutation(count)].reshape(2, 1, pages, heads, 1)
    # every byte in every block
    b = np.stack([rng.permutation(256) for _ in range(count)]).astype(np.uint8).reshape(2, 1, pages, heads, page, dim)
    cache = ss.KVCache(*(torch.from_numpy(x).cuda().view(torch.float8_e4m3fn) for x in b),
                       *(torch.from_numpy(x).cuda() for x in s))
    k, v = (torch.empty(pages * page, heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st = ints([-1])
    ss.ss_cache_read(cache, 0, k, v, ints([list(range(pages))]), ints([0]), st, token_offsets=ints([0, pages * page]),
                     max_tokens=pages * page)
    assert st.tolist() == [0]
    twice = 0
    for got, n, x in zip((k, v), b, s):
        with np.errstate(all="ignore"):
            exact = P.e4m3_of(n[0]) * x[0].astype(np.float64)[..., None]
            other = bf16_once(exact.astype(np.float32).astype(np.float64))
        want = bf16_once(exact)
        twice += int((other != want)[~np.isnan(want)].sum())
        assert np.array_equal(np32(got).reshape(pages, page, heads, dim).transpose(0, 2, 1, 3), want, equal_nan=True)
    assert twice > 400  # as many would a second rounding have turned
