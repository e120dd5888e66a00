"""The example with rotary positions: what its loop of draft trees leaves in the
cache, in every format."""
import pytest
import torch

from speculative_verification_gb300 import ss
from tests.test_tree_decode_gpu import example  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "int4", "fp8"])
def test_the_cache_holds_the_turned_keys(example, fmt):  # noqa: F811
    model = example.Decoder(rotary=True)
    g = torch.Generator().manual_seed(6)
    prompts = [torch.randint(model.vocab, (m,), generator=g).tolist() for m in (7, 150, 64)]
    texts, kv_len, cache, pool, bad = example.decode(model, prompts, samples=2, steps=6, page=16, format=fmt)
    assert bad == 0
    n = len(prompts)
    for i, (text, m) in enumerate(zip(texts, kv_len.tolist())):
        assert m == len(text) - 1
        # layer 0's keys depend on the token and its position alone
        _, keys, _ = model.project(0, model.embedded(torch.tensor(text[:m]).cuda(), torch.arange(m).cuda()))
        want, st = torch.empty(m, *keys.shape[1:], dtype=torch.bfloat16, device="cuda"), example.ints([0])
        ss.ss_rope(model.rope, None, None, keys, want, None, st, token_offsets=example.ints([0, m]), max_tokens=m,
                   positions=torch.arange(m, dtype=torch.int32, device="cuda"))
        k, v = torch.zeros_like(want), torch.zeros_like(want)
        ss.ss_cache_read(cache, 0, k, v, pool.page_table, example.ints([0]), st, token_offsets=example.ints([0, m]),
                         max_tokens=m, table_rows=example.ints([n + i]))
        first = max(0, m - model.window)
        kept = [j for j in range(m) if j < model.sinks or j >= first]
        got, want = k[kept].float(), want[kept].float()
        # bf16: the projection's rounding in another batch (one unit), turned (its pair's unit) and rounded again;
        # 4 bits: half a step of the row as well; 8 bits: half of e4m3's step (2^-4), twice where a draft's larger
        # block scale came and went, and the smallest ones 2^-10 of a scale of at most the largest over 224
        size = (want[..., :48:2] ** 2 + want[..., 1:48:2] ** 2).sqrt().repeat_interleave(2, -1)
        near = 2.0 ** -7 * torch.cat([size, want[..., 48:].abs()], -1) + 2.0 ** -7 * want.abs() + 2.0 ** -9
        if fmt == "int4":
            near = near + (want.amax(-1, keepdim=True) - want.amin(-1, keepdim=True)) / 15 * 0.52
        if fmt == "fp8":
            near = near + 2.0 ** -4 * (want.abs() + near) + 2.0 ** -9 * 64 / 224
        assert want.abs().max() < 64
        assert ((got - want).abs() <= near).all()
