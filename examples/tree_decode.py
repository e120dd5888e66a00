"""Tree-speculative decoding over a paged cache: the calls of one server step
in the order a serving loop makes them.

A small random decoder answers `requests` prompts, `samples` continuations
each.  The prompt is cached once and its pages are shared by the
continuations (ss_pages_fork); every step then

  ss_pages_reserve      pages for the draft tree's tokens
  per layer             ss_cache_append, ss_cache_attention (tree mask, window)
  ss_tree_verify        the accepted path and one token of the target's
  ss_commit_accepted    the emitted tokens into the token buffer
  ss_pages_compact      the accepted nodes' rows next to each other
  ss_pages_trim         pages that left the window back to the pool

without a device-to-host copy in the loop.  The drafts are uniform random
tokens (their q says so), so the verified text follows the target model.

    python examples/tree_decode.py [--format bf16|int4] [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_verification_gb300 import ss  # noqa: E402


class Decoder:
    """Attention layers without an MLP: as much of a model as the calls need."""

    def __init__(self, vocab=512, layers=3, heads=8, kv_heads=2, dim=64, positions=2048, window=96, sinks=4, seed=0):
        g = torch.Generator().manual_seed(seed)

        def weight(*shape, scale):
            return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16).cuda()

        self.vocab, self.layers, self.heads, self.kv_heads, self.dim = vocab, layers, heads, kv_heads, dim
        self.window, self.sinks = window, sinks
        width = self.width = heads * dim
        self.embed = weight(vocab, width, scale=1.0)
        self.place = weight(positions, width, scale=0.5)
        self.qkv = [weight(width, (heads + 2 * kv_heads) * dim, scale=width ** -0.5) for _ in range(layers)]
        self.out = [weight(width, width, scale=width ** -0.5) for _ in range(layers)]
        self.head = weight(width, vocab, scale=2.0 * width ** -0.5)

    def embedded(self, tokens, positions):
        return self.embed[tokens.long()] + self.place[positions.long()]

    def project(self, layer, x):
        """The queries, keys and values of a layer."""
        y = (torch.nn.functional.rms_norm(x, (self.width,)) @ self.qkv[layer]).view(x.shape[0], -1, self.dim)
        return y.split([self.heads, self.kv_heads, self.kv_heads], 1)

    def forward(self, cache, pool, tokens, positions, kv_len, offsets, most, workspace, status, **attention):
        """The logits of the new tokens, whose keys and values go into the cache."""
        x = self.embedded(tokens, positions)
        for layer in range(self.layers):
            q, k, v = self.project(layer, x)
            ss.ss_cache_append(cache, layer, k, v, pool.page_table, kv_len, status, token_offsets=offsets,
                               max_tokens=most, table_rows=attention.get("table_rows"))
            o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            ss.ss_cache_attention(cache, layer, q, o, pool.page_table, kv_len, workspace, status, query_offsets=offsets,
                                  max_queries=most, window=self.window, sinks=self.sinks, **attention)
            x = x + o.view(-1, self.width) @ self.out[layer]
        return torch.nn.functional.rms_norm(x, (self.width,)) @ self.head


def ints(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def decode(model, prompts, samples=2, steps=6, nodes=12, page=16, format="bf16", seed=1):
    """Lists of token ids, one per continuation, and the state they leave:
    (texts, lengths in the cache, cache, pool, statuses that were not 0)."""
    g = torch.Generator().manual_seed(seed)
    n = len(prompts)
    rows, most = n * samples, max(len(p) for p in prompts)
    capacity = most + steps * nodes + 1
    entries = -(-(capacity + nodes) // page)
    pages = (n + rows) * entries
    cache = ss.alloc_cache(model.layers, pages, model.kv_heads, page, model.dim, format)
    pool = ss.alloc_pool(n + rows, entries, pages, page)
    workspace = ss.alloc_attention_workspace()
    verify_ws = torch.zeros(ss.ss_workspace_size(max(n, rows), nodes - 1), dtype=torch.uint8, device="cuda")
    bad = torch.zeros((), dtype=torch.int64, device="cuda")

    # the prompts
    lens = [len(p) for p in prompts]
    start, prompt_len, st = ints([0] * n), ints(lens), ints([0] * n)
    offsets = ints([sum(lens[:i]) for i in range(n + 1)])
    flat = ints([t for p in prompts for t in p])
    position = torch.cat([torch.arange(x) for x in lens]).cuda()
    ss.ss_pages_reserve(pool, start, prompt_len, st)
    bad += st.count_nonzero()
    logits = model.forward(cache, pool, flat, position, start, offsets, most, workspace, st)
    bad += st.count_nonzero()

    # their pages shared by the continuations, the prompts' own rows freed
    of = torch.arange(rows, device="cuda") // samples
    table_rows = ints([n + i for i in range(rows)])
    kv_len, status = prompt_len[of].contiguous(), ints([0] * rows)
    ss.ss_pages_fork(pool, cache, of.int(), table_rows, kv_len, status)
    bad += status.count_nonzero()
    ss.ss_pages_trim(pool, start, st)
    bad += st.count_nonzero()

    # the first token of each continuation
    params = dict(temperature=torch.ones(rows, device="cuda"), seed=torch.arange(rows, device="cuda") + 100 * seed,
                  position=kv_len.long())
    root = torch.empty_like(kv_len)
    ss.ss_process_sample(logits[(offsets[1:] - 1).long()][of].contiguous(), params, root, status, vocab=model.vocab,
                         dtype="bf16")
    bad += status.count_nonzero()
    tokens = torch.full((rows, capacity), -1, dtype=torch.int32, device="cuda")
    for i in range(rows):
        p = prompts[i // samples]
        tokens[i, :len(p)] = ints(p)
        tokens[i, len(p)] = root[i]
    seq_len, next_token = kv_len + 1, root
    params["position"] = seq_len.long()

    offsets = ints([i * nodes for i in range(rows + 1)])
    uniform = torch.full((rows * nodes, model.vocab), 1.0 / model.vocab, device="cuda")
    out_tokens, out_path = (torch.empty(rows, nodes, dtype=torch.int32, device="cuda") for _ in range(2))
    accepted, verified, committed, new_len = (torch.empty(rows, dtype=torch.int32, device="cuda") for _ in range(4))
    for _ in range(steps):
        parents = torch.stack([torch.tensor([0] + [int(torch.randint(u, (1,), generator=g)) for u in range(1, nodes)])
                               for _ in range(rows)])
        depth = torch.zeros(rows, nodes, dtype=torch.int64)
        for u in range(1, nodes):
            depth[:, u] = depth.gather(1, parents[:, u:u + 1])[:, 0] + 1
        drafts = torch.randint(model.vocab, (rows, nodes), generator=g).int().cuda()
        drafts[:, 0] = next_token
        parents, depth = parents.int().cuda().view(-1), depth.cuda()

        ss.ss_pages_reserve(pool, kv_len, kv_len + nodes, status, table_rows=table_rows)
        bad += status.count_nonzero()
        logits = model.forward(cache, pool, drafts.view(-1), (kv_len[:, None] + depth).view(-1), kv_len, offsets, nodes,
                               workspace, status, parents=parents, table_rows=table_rows)
        bad += status.count_nonzero()
        ss.ss_tree_verify(logits, offsets, parents, drafts.view(-1), uniform, params, out_tokens, accepted, verified,
                          verify_ws, vocab=model.vocab, max_nodes=nodes, dtype="bf16", out_path=out_path)
        bad += verified.count_nonzero()
        ss.ss_commit_accepted(out_tokens, accepted, verified, tokens, seq_len, params["position"], next_token, committed)
        bad += committed.count_nonzero()
        ss.ss_pages_compact(pool, cache, kv_len, out_path, accepted, verified, new_len, status, table_rows=table_rows)
        bad += status.count_nonzero()
        kv_len, new_len = new_len, kv_len
        ss.ss_pages_trim(pool, kv_len, status, window=model.window, sinks=model.sinks, table_rows=table_rows)
        bad += status.count_nonzero()
    torch.cuda.synchronize()
    texts = [t[:int(m)] for t, m in zip(tokens.tolist(), seq_len)]
    return texts, kv_len, cache, pool, int(bad)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--format", default="bf16", choices=("bf16", "int4"))
    ap.add_argument("--steps", type=int, default=6)
    args = ap.parse_args()
    g = torch.Generator().manual_seed(5)
    prompts = [torch.randint(512, (m,), generator=g).tolist() for m in (7, 150, 64)]
    texts, lengths, _, pool, bad = decode(Decoder(), prompts, steps=args.steps, format=args.format)
    for i, t in enumerate(texts):
        m = len(prompts[i // 2])
        print("prompt %d, continuation %d: %d tokens in %d steps: %s" % (i // 2, i % 2, len(t) - m, args.steps, t[m:]))
    print("%d of %d pages in use; %s" % (pool.ref_count.count_nonzero(), pool.ref_count.numel(),
                                         "every status 0" if bad == 0 else "%d statuses were not 0" % bad))


if __name__ == "__main__":
    main()
