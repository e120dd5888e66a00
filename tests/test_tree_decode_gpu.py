"""The example that runs the cache's calls together with tree verification."""
import importlib.util
import os

import pytest
import torch

from speculative_verification_gb300 import ss

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("tree_decode", os.path.join(ROOT, "examples", "tree_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_the_cache_holds_the_text(example, fmt):
    model = example.Decoder()
    g = torch.Generator().manual_seed(5)
    prompts = [torch.randint(model.vocab, (m,), generator=g).tolist() for m in (7, 150, 64)]
    samples, steps, page = 2, 6, 16
    texts, kv_len, cache, pool, bad = example.decode(model, prompts, samples=samples, steps=steps, page=page, format=fmt)
    assert bad == 0
    rows, n = len(texts), len(prompts)
    held = pool.page_table >= 0
    assert int(held.sum()) == int(pool.ref_count.sum())
    assert int(pool.free_count) + int(pool.ref_count.count_nonzero()) == pool.ref_count.numel()
    assert not held[:n].any()
    emitted = 0
    for i, (text, m) in enumerate(zip(texts, kv_len.tolist())):
        prompt = prompts[i // samples]
        assert text[:len(prompt)] == prompt and m == len(text) - 1  # the last token is the next step's root
        emitted += len(text) - len(prompt) - 1
        # layer 0's keys depend on the token and its position alone
        _, want, _ = model.project(0, model.embedded(torch.tensor(text[:m]).cuda(), torch.arange(m).cuda()))
        k, v, st = torch.zeros_like(want).contiguous(), torch.zeros_like(want).contiguous(), example.ints([0])
        ss.ss_cache_read(cache, 0, k, v, pool.page_table, example.ints([0]), st, token_offsets=example.ints([0, m]),
                         max_tokens=m, table_rows=example.ints([n + i]))
        torch.cuda.synchronize()
        first = max(0, m - model.window)
        kept = [j for j in range(m) if j < model.sinks or j >= first]
        got, want = k[kept].float(), want[kept].float()
        # bf16: the projection's rounding in another batch, one unit each; 4 bits: half a step of the row as well
        near = 2.0 ** -7 * want.abs() + 2.0 ** -9
        if fmt == "int4":
            near = near + (want.amax(-1, keepdim=True) - want.amin(-1, keepdim=True)) / 15 * 0.52
        assert ((got - want).abs() <= near).all()
        gone = [j for j in range(m) if j // page * page + page <= first and j // page * page >= model.sinks]
        assert not k[gone].any()
    assert emitted >= steps * rows  # each step emits one token or more
    st = example.ints([0] * rows)
    ss.ss_pages_trim(pool, example.ints([0] * rows), st, table_rows=example.ints([n + i for i in range(rows)]))
    torch.cuda.synchronize()
    assert int(pool.free_count) == pool.ref_count.numel() and not pool.ref_count.any()


def test_a_steps_result_is_that_of_the_accepted_text(example):
    """The logits of a chain of tokens, one call per token or all in one call
    as a draft tree of one branch, are those of the text as a prompt."""
    model = example.Decoder(window=0)
    g = torch.Generator().manual_seed(3)
    text = torch.randint(model.vocab, (40,), generator=g).int().cuda()
    ints = example.ints

    def run(parts, tree):
        cache = ss.alloc_cache(model.layers, 8, model.kv_heads, 16, model.dim)
        pool, ws, st = ss.alloc_pool(1, 8, 8, 16), ss.alloc_attention_workspace(), ints([0])
        out, at = [], 0
        for m in parts:
            ss.ss_pages_reserve(pool, ints([at]), ints([at + m]), st)
            out.append(model.forward(cache, pool, text[at:at + m], torch.arange(at, at + m).cuda(), ints([at]), ints([0, m]),
                                     m, ws, st, **(dict(parents=ints([max(i - 1, 0) for i in range(m)])) if tree else {})))
            at += m
        torch.cuda.synchronize()
        assert int(st) == 0
        return torch.cat(out).float()

    whole = run([40], False)
    # the same sums in another order, three layers of bf16 roundings: up to 5 parts in a hundred of the logits' spread
    # each, and four times that for the largest of 40 x 512
    near = 0.2 * whole.std()
    assert (run([1] * 40, False) - whole).abs().max() <= near
    assert (run([17, 13, 10], True) - whole).abs().max() <= near
