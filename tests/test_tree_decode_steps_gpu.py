"""Every attention call of the example's loop, held to 64-bit sums over what
the cache holds at that moment: prompts, draft trees, windows with sinks, pages
that were forked, compacted and trimmed."""
import numpy as np
import pytest

from tests import cache_ref as R
from tests.test_cache_gpu import FORMATS, dense, np32
from tests.test_tree_decode_gpu import example  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_attention_of_the_loop(example, monkeypatch, fmt):  # noqa: F811
    ss = example.ss
    call, kinds = ss.ss_cache_attention, []

    def checked(cache, layer, q, out, table, kv_len, workspace, status, **kw):
        call(cache, layer, q, out, table, kv_len, workspace, status, **kw)
        torch.cuda.synchronize()
        assert not status.any()
        k, v, mv = dense(cache, layer)
        offsets, parents = kw["query_offsets"].tolist(), kw.get("parents")
        rows = kw["table_rows"].tolist() if kw.get("table_rows") is not None else list(range(kv_len.numel()))
        got, qs = np32(out).astype(np.float64), np32(q).astype(np.float64)
        for r, base in enumerate(kv_len.tolist()):
            lo, hi = offsets[r], offsets[r + 1]
            o, _, m, _ = R.attend(qs[lo:hi], lambda p, s: (k[p, :, s], v[p, :, s], mv[p, :, s]), table[rows[r]].tolist(),
                                  cache.page_size, base, q.shape[2] ** -0.5, kw["window"], kw["sinks"],
                                  parents[lo:hi].tolist() if parents is not None else None, cache.num_pages)
            # the bound of the attention tests: each weight's and the result's rounding to bf16
            assert (np.abs(got[lo:hi] - o) <= 2.0 ** -8 * (np.abs(o) + m) * (1 + 1 / 16)).all(), (len(kinds), layer, r)
        kinds.append("tree" if parents is not None else "prompt")

    monkeypatch.setattr(ss, "ss_cache_attention", checked)
    model = example.Decoder(window=48)
    g = torch.Generator().manual_seed(11)
    prompts = [torch.randint(model.vocab, (m,), generator=g).tolist() for m in (5, 90, 64)]
    *_, bad = example.decode(model, prompts, samples=2, steps=4, page=16, format=fmt)
    assert bad == 0 and kinds.count("prompt") == model.layers and kinds.count("tree") == 4 * model.layers
