"""How many tiles a request may have: the same for bf16 and 4 bits, whose items
count their own tiles; three fewer a block of rows for 8 bits, whose items count
three more.

A request of 2^24 - 64 rows a kv head (the most that 128 kv heads may have) in
blocks of 128 (4 and 8 bits: 64) over a table of 4095 (2047) pages of 512 slots:
2^17 (2^18) blocks of 16380 (8188) tiles, and three for the window's and the
sinks' ends, stay below 2^31; three more for each block pass it.  A call that
may be walked is then beyond what 128 kv heads allow in all (2^30), so that
it is reported, and nothing is computed."""
import numpy as np
import pytest

from tests.test_cache_gpu import ints, make_cache, ss, workspace  # noqa: F401
from tests.test_rope_gpu import cache8

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BAD_PARAM, LIMIT = 4, 6


@pytest.mark.parametrize("fmt,rows,status", [("bf16", 128, LIMIT), ("int4", 64, LIMIT), ("fp8", 64, BAD_PARAM)])
def test_tiles_of_a_request_by_format(ss, workspace, fmt, rows, status):
    heads, dim, page, n = 128, 32, 512, (1 << 24) - 64
    blocks, entries = -(-n // rows), (1 << 31) // (-(-n // rows)) // 4 - 1
    tiles = entries * page // 128
    assert blocks * (tiles + 3) < 1 << 31 <= blocks * (tiles + 6)
    rng = np.random.default_rng(0)
    cache = cache8(ss, rng, 1, heads, page, dim) if fmt == "fp8" else make_cache(ss, rng, fmt, 1, heads, page, dim)
    table, st = torch.zeros(1, entries, dtype=torch.int32, device="cuda"), ints([-1])
    flat = torch.full((n * 8 + heads * dim,), 7.0, dtype=torch.bfloat16, device="cuda")
    q = flat.as_strided((n, heads, dim), (8, dim, 1))  # (tokens overlap: only their addresses count)
    ss.ss_cache_attention(cache, 0, q, q, table, ints([0]), workspace, st, query_offsets=ints([0, n]), max_queries=n)
    torch.cuda.synchronize()
    assert st.tolist() == [status]
    assert bool((flat == 7).all())
