"""The cache operators around a verification step, as cases that can be timed and compared.

Four operators, over one paged key/value cache:

  append   new keys and values into a request's pages, as bf16 or in 4 bits (and read back)
  attend   attention over the pages: sliding window and sinks, drafts in a row or in a tree, prompt chunks;
           the cache in bf16 or in 4 bits
  pages    the pages themselves: reserve, fork, compact after a verified tree, trim

With `own` false every operator is computed by elementary torch operations in 32 bits; with `own` true by the
library's entry points.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # One decode step's new tokens of a batch with drafts, one layer of a bf16 cache with small pages: the
        # smallest write, all latency.
        dict(name="append bf16, 32 x 1-8 tokens", op="append", format="bf16", requests=32, kv_heads=8, head_dim=128,
             page=16, len_min=100, len_max=3000, tokens_min=1, tokens_max=8),
        # Prompt chunks of four requests into a 4-bit cache, then read back as a program does that moves a request.
        dict(name="append 4-bit, 4 x 2-6k tokens", op="append", format="int4", requests=4, kv_heads=8, head_dim=128,
             page=64, len_min=0, len_max=5000, tokens_min=2011, tokens_max=6143),
        # A single chat request, one token a step, a short window: the smallest attention call.
        dict(name="window 1 x 1 token, 700", op="attend", format="bf16", requests=1, heads=32, kv_heads=8,
             head_dim=128, page=16, len_min=700, len_max=700, queries_min=1, queries_max=1, tree=False, window=512,
             sinks=4),
        # Linear verification: a batch with 1 to 8 queries (the last token and up to 7 drafts) over long contexts with a
        # wide window.
        dict(name="window 32 x 1-8 drafts, 1-32k", op="attend", format="bf16", requests=32, heads=32, kv_heads=8,
             head_dim=128, page=64, len_min=1000, len_max=32000, queries_min=1, queries_max=8, tree=False,
             window=16384, sinks=4),
        # Tree verification: up to 64 nodes a request, small heads, full attention.
        dict(name="window off, 16 trees, 2-12k", op="attend", format="bf16", requests=16, heads=16, kv_heads=4,
             head_dim=64, page=32, len_min=2000, len_max=12000, queries_min=17, queries_max=64, tree=True, window=0,
             sinks=0),
        # Prompt chunks: the second chunk of two prompts, thousands of queries with a window of 1024.
        dict(name="window 1024, 2 x 4096 prompt", op="attend", format="bf16", requests=2, heads=32, kv_heads=8,
             head_dim=128, page=64, len_min=0, len_max=4096, queries_min=4095, queries_max=4096, tree=False,
             window=1024, sinks=4),
        # The smallest call on a 4-bit cache: a few requests, one token each, small heads and pages.
        dict(name="4-bit 4 x 1 token, 1-2k", op="attend", format="int4", requests=4, heads=16, kv_heads=2,
             head_dim=64, page=16, len_min=1000, len_max=2000, queries_min=1, queries_max=1, tree=False, window=0,
             sinks=0),
        # Decode over long contexts, which is what a 4-bit cache is for: bound by reading it.
        dict(name="4-bit 32 x 1 token, 8-64k", op="attend", format="int4", requests=32, heads=32, kv_heads=8,
             head_dim=128, page=64, len_min=8000, len_max=64000, queries_min=1, queries_max=1, tree=False, window=0,
             sinks=0),
        # Verification of 1 to 8 positions over a 4-bit cache, wide head groups.
        dict(name="4-bit 48 x 1-8 drafts, 1-16k", op="attend", format="int4", requests=48, heads=64, kv_heads=8,
             head_dim=128, page=64, len_min=1000, len_max=16000, queries_min=1, queries_max=8, tree=False, window=0,
             sinks=0),
        # Four prompts forked into eight continuations each, and the continuations freed again: a small model's cache.
        dict(name="fork 4 x 8, 4 layers", op="pages", kind="fork", parents=4, children=8, layers=4, kv_heads=4,
             head_dim=64, page=16, len_min=100, len_max=900),
        # After a tree verification: pages for the drafts reserved, the accepted rows of 64 requests moved together
        # in every layer, the pages past them freed.
        dict(name="compact 64 trees, 32 layers", op="pages", kind="compact", requests=64, layers=32, kv_heads=8,
             head_dim=128, page=16, len_min=50, len_max=700, nodes_max=48, depth_max=7),
        # A batch of prompts forked for parallel sampling, pages of 64 slots in 32 layers.
        dict(name="fork 16 x 4, 32 layers", op="pages", kind="fork", parents=16, children=4, layers=32, kv_heads=8,
             head_dim=128, page=64, len_min=200, len_max=900),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["append", "bf16", "int4", "prompt", "tree", "fork", "compact"])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    head_dim = rng.choice([64, 64, 96, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    if kind == "append":
        requests = _log(rng, 1, 48)
        tokens = _log(rng, 1, max(1, 16000 // requests))
        first = _log(rng, 1, 5000)
        return dict(op="append", format=rng.choice(["bf16", "int4"]), requests=requests, kv_heads=kv_heads,
                    head_dim=head_dim, page=page, len_min=first - 1, len_max=first + _log(rng, 1, 3000),
                    tokens_min=max(1, tokens // 3), tokens_max=tokens)
    if kind in ("bf16", "int4"):
        requests = _log(rng, 1, 32)
        group = rng.choice([1, 2, 4, 5, 7, 8])
        longest = _log(rng, 64, 32000 if requests > 8 else 64000)
        return dict(op="attend", format=kind, requests=requests, heads=kv_heads * group, kv_heads=kv_heads,
                    head_dim=head_dim, page=page, len_min=max(0, longest // rng.choice([1, 2, 8]) - 1),
                    len_max=longest, queries_min=1, queries_max=_log(rng, 1, 8), tree=False,
                    window=rng.choice([0, 0, _log(rng, 100, 20000)]), sinks=rng.choice([0, 4, 64, 131]))
    if kind == "prompt":
        queries = _log(rng, 100, 4000)
        return dict(op="attend", format=rng.choice(["bf16", "bf16", "int4"]), requests=rng.choice([1, 2]),
                    heads=kv_heads * 4, kv_heads=kv_heads, head_dim=head_dim, page=page, len_min=0,
                    len_max=_log(rng, 1, 4000), queries_min=queries // 2, queries_max=queries, tree=False,
                    window=rng.choice([0, _log(rng, 100, 2000)]), sinks=rng.choice([0, 4, 64]))
    if kind == "tree":
        longest = _log(rng, 100, 16000)
        return dict(op="attend", format=rng.choice(["bf16", "int4"]), requests=_log(rng, 1, 16),
                    heads=kv_heads * rng.choice([1, 4, 8]), kv_heads=kv_heads, head_dim=head_dim, page=page,
                    len_min=longest // 3, len_max=longest, queries_min=1, queries_max=_log(rng, 2, 64), tree=True,
                    window=rng.choice([0, _log(rng, 100, 8000)]), sinks=rng.choice([0, 4, 64]))
    layers = _log(rng, 1, 32)
    if kind == "fork":
        return dict(op="pages", kind="fork", parents=_log(rng, 1, 16), children=_log(rng, 1, 4), layers=layers,
                    kv_heads=kv_heads, head_dim=head_dim, page=page, len_min=_log(rng, 1, 200),
                    len_max=_log(rng, 200, 900))
    return dict(op="pages", kind="compact", requests=_log(rng, 1, 64), layers=layers, kv_heads=kv_heads,
                head_dim=head_dim, page=page, len_min=_log(rng, 1, 50), len_max=_log(rng, 50, 500),
                nodes_max=_log(rng, 4, 64), depth_max=_log(rng, 1, 7))


# ----------------------------------------------------------------- inputs --

def _lengths(case):
    """Each request's cached length and number of new tokens: a request's two numbers go together, so that the work
    of a case does not depend on the seed (the seed orders the requests)."""
    n = case["requests"]
    lo, hi = case["len_min"], case["len_max"]
    qlo, qhi = (case[k] for k in (("tokens_min", "tokens_max") if case["op"] == "append" else
                                  ("queries_min", "queries_max")))
    lens = [lo + ((hi - lo) * i) // max(1, n - 1) for i in range(n)]
    news = [qlo + (i * 7919 + n // 2) % (qhi - qlo + 1) for i in range(n)]
    return lens, news


def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def _kv(gen, *shape):
    """Keys or values as models make them: unit spread with a few channels that are much larger and off centre."""
    x = _rand(gen, *shape)
    x[..., 3] *= 4
    x[..., 3] += 2
    x[..., -2] *= 3
    return x


def _offsets(news):
    out = [0]
    for n in news:
        out.append(out[-1] + n)
    return out


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _parents(rng, news):
    """Draft trees: a node hangs under one of the few nodes before it."""
    out = []
    for n in news:
        out += [0] + [rng.randint(max(0, v - 5), v - 1) for v in range(1, n)]
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    if case["op"] == "pages":
        return _prepare_pages(case, gen, rng)
    n, page, heads, dim = case["requests"], case["page"], case["kv_heads"], case["head_dim"]
    pairs = list(zip(*_lengths(case)))
    rng.shuffle(pairs)
    lens, news = [a for a, _ in pairs], [b for _, b in pairs]
    # the pages that hold something: all of a request's, or with a window those of the sinks and of the window
    width = max(-(-(a + b) // page) for a, b in pairs)
    rows, used = [], 0
    for a, b in pairs:
        row = [-1] * width
        keep = case.get("window", 0)
        for p in range(-(-(a + b) // page)):
            if not keep or p * page < case["sinks"] or (p + 1) * page > a - keep:
                row[p] = used
                used += 1
        rows.append(row)
    order = torch.randperm(used + 3, generator=gen, device="cuda").to(torch.int32)
    table = _ints(rows)
    table = torch.where(table >= 0, order[table.clamp(min=0).long()], table)
    s = dict(case=case, page_table=table, kv_len=_ints(lens), offsets=_ints(_offsets(news)),
             total=sum(news), most=max(news), longest=max(a + b for a, b in pairs))
    packed = case["format"] == "int4"
    shape = (1, used + 3, heads, page)
    if case["op"] == "append":
        if packed:
            s["cache"] = dict(k=torch.zeros(*shape, dim // 2, dtype=torch.uint8, device="cuda"),
                              v=torch.zeros(*shape, dim // 2, dtype=torch.uint8, device="cuda"),
                              k_scale=torch.zeros(*shape, 2, dtype=torch.bfloat16, device="cuda"),
                              v_scale=torch.zeros(*shape, 2, dtype=torch.bfloat16, device="cuda"))
        else:
            s["cache"] = dict(k=_kv(gen, *shape, dim), v=_kv(gen, *shape, dim))
        # keys and values of one layer's projection, side by side
        kv = _kv(gen, sum(news), 2, heads, dim)
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
        s["k_read"], s["v_read"] = (torch.empty(sum(news), heads, dim, dtype=torch.bfloat16, device="cuda")
                                    for _ in range(2))
    else:
        if packed:
            s["cache"] = {}
            for x in ("k", "v"):
                s["cache"][x] = torch.randint(0, 256, (*shape, dim // 2), generator=gen, dtype=torch.uint8,
                                              device="cuda")
                step = torch.rand(*shape, 1, generator=gen, device="cuda") * 0.3 + 0.2
                low = torch.randn(*shape, 1, generator=gen, device="cuda") * 0.3 - 7.5 * step
                s["cache"][x + "_scale"] = torch.cat([step, low], -1).to(torch.bfloat16)
        else:
            s["cache"] = dict(k=_kv(gen, *shape, dim), v=_kv(gen, *shape, dim))
            # pages that no request holds: whatever was there before
            s["cache"]["v"][:, order[used:].long()] = float("nan")
        s["q"] = _rand(gen, sum(news), case["heads"], dim)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(sum(news), case["heads"], dtype=torch.float32, device="cuda")
        s["parents"] = _ints(_parents(rng, news)) if case["tree"] else None
        s["scale"] = dim ** -0.5
    s["status"] = torch.empty(n, dtype=torch.int32, device="cuda")
    if own:
        from speculative_verification_gb300 import ss
        s["handle"] = ss.KVCache(**s["cache"])
        if case["op"] == "attend":
            s["workspace"] = ss.alloc_attention_workspace()
    return s


def _prepare_pages(case, gen, rng):
    page, layers, heads, dim = case["page"], case["layers"], case["kv_heads"], case["head_dim"]
    lo, hi = case["len_min"], case["len_max"]
    fork = case["kind"] == "fork"
    n = case["parents"] if fork else case["requests"]
    lens = [lo + ((hi - lo) * i) // max(1, n - 1) for i in range(n)]
    rng.shuffle(lens)
    width = -(-(hi + case.get("nodes_max", 0)) // page) + 1
    rows = n * (1 + case["children"]) if fork else n
    table, used = [[-1] * width for _ in range(rows)], 0
    for r, length in enumerate(lens):
        for p in range(-(-length // page)):
            table[r][p] = used
            used += 1
    more = n * case["children"] if fork else n * (case["nodes_max"] // page + 2)
    pages = used + more + 2
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    t = _ints(table)
    t = torch.where(t >= 0, order[t.clamp(min=0).long()], t)
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free[:pages - used] = order[used:]
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[order[:used].long()] = 1
    s = dict(case=case, pool=dict(page_table=t, ref_count=refs, free_pages=free, free_count=_ints([pages - used]),
                                  page_size=page),
             cache=dict(k=_kv(gen, layers, pages, heads, page, dim), v=_kv(gen, layers, pages, heads, page, dim)))
    if fork:
        m = n * case["children"]
        s["parent"] = _ints([i // case["children"] for i in range(m)])
        s["child"] = _ints([n + i for i in range(m)])
        s["length"] = _ints(lens)[s["parent"].long()]
        s["zero"] = torch.zeros(m, dtype=torch.int32, device="cuda")
        s["status"], s["status2"] = (torch.empty(m, dtype=torch.int32, device="cuda") for _ in range(2))
    else:
        # the accepted path of each request's tree: a node of the first level, then one of its children, and so on
        # (a level's nodes come before the next level's, so a path's nodes lie past the slots that they move to)
        most, nodes, paths, counts = case["nodes_max"], [], [], []
        for i in range(n):
            depth = min((i * 5 + n) % (case["depth_max"] + 1), (most - 1) // 2)
            path = sorted(rng.sample(range(depth + 1, most), depth)) if depth else []
            nodes.append(most)
            counts.append(depth)
            paths.append(path + [-1] * (most - depth))
        s["kv_len"], s["nodes"], s["path"], s["accepted"] = _ints(lens), _ints(nodes), _ints(paths), _ints(counts)
        s["to_len"] = s["kv_len"] + s["nodes"]
        s["verified"] = torch.zeros(n, dtype=torch.int32, device="cuda")
        s["new_len"] = torch.empty(n, dtype=torch.int32, device="cuda")
        s["status"], s["status2"], s["status3"] = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(3))
    if own:
        from speculative_verification_gb300 import ss
        s["handle"], s["pages"] = ss.KVCache(**s["cache"]), ss.PagePool(**s["pool"])
    return s


# --------------------------------------------------------------- one pass --

def run(state):
    op = state["case"]["op"]
    if op == "append":
        return _own_append(state) if own else _plain_append(state)
    if op == "attend":
        return _own_attend(state) if own else _plain_attend(state)
    return _own_pages(state) if own else _plain_pages(state)


def _own_append(s):
    from speculative_verification_gb300 import ss
    ss.ss_cache_append(s["handle"], 0, s["k"], s["v"], s["page_table"], s["kv_len"], s["status"],
                       token_offsets=s["offsets"], max_tokens=s["most"])
    if s["case"]["format"] == "bf16":
        return dict(k=s["cache"]["k"], v=s["cache"]["v"], status=s["status"])
    ss.ss_cache_read(s["handle"], 0, s["k_read"], s["v_read"], s["page_table"], s["kv_len"], s["status"],
                     token_offsets=s["offsets"], max_tokens=s["most"])
    return dict(k=s["k_read"], v=s["v_read"], status=s["status"])


def _own_attend(s):
    from speculative_verification_gb300 import ss
    c = s["case"]
    ss.ss_cache_attention(s["handle"], 0, s["q"], s["out"], s["page_table"], s["kv_len"], s["workspace"], s["status"],
                          query_offsets=s["offsets"], max_queries=s["most"], parents=s["parents"], scale=s["scale"],
                          window=c["window"], sinks=c["sinks"], lse=s["lse"])
    return dict(out=s["out"], lse=s["lse"], status=s["status"])


def _own_pages(s):
    from speculative_verification_gb300 import ss
    pool, cache = s["pages"], s["handle"]
    out = dict(page_table=s["pool"]["page_table"], ref_count=s["pool"]["ref_count"],
               free_count=s["pool"]["free_count"], k=s["cache"]["k"], v=s["cache"]["v"], status=s["status"])
    if s["case"]["kind"] == "fork":
        ss.ss_pages_fork(pool, cache, s["parent"], s["child"], s["length"], s["status"])
        # the forked tables, as they are between the two calls
        out["forked"] = s["pool"]["page_table"].clone()
        ss.ss_pages_trim(pool, s["zero"], s["status2"], table_rows=s["child"])
        return out | dict(status2=s["status2"])
    ss.ss_pages_reserve(pool, s["kv_len"], s["to_len"], s["status"])
    ss.ss_pages_compact(pool, cache, s["kv_len"], s["path"], s["accepted"], s["verified"], s["new_len"], s["status2"])
    ss.ss_pages_trim(pool, s["new_len"], s["status3"])
    return out | dict(status2=s["status2"], status3=s["status3"], new_len=s["new_len"])


# ------------------------------------------------------------ plain forms --

def _token_slots(s):
    """For each new token its request, page and row in the page."""
    page = s["case"]["page"]
    at = torch.arange(s["total"], device="cuda", dtype=torch.int32)
    r = torch.searchsorted(s["offsets"][1:].contiguous(), at, right=True)
    slot = s["kv_len"][r] + at - s["offsets"][r]
    return s["page_table"][r, (slot // page).long()].long(), (slot % page).long()


#: Channel order of a packed word's nibbles, least significant byte first: channel 2i in bits 4i.., 2i + 1 in 16 + 4i..
_NIBBLES = [0, 2, 4, 6, 1, 3, 5, 7]


def _pack(x):
    """4-bit rows of x [..., dim] (float32): the packed bytes and (step, lowest)."""
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    step = (high - low) / torch.full_like(low, 15)  # a tensor: by a number, torch multiplies by its reciprocal
    step = ((step.view(torch.int32) + 0xffff) & ~0xffff).view(torch.float32)  # up to a bf16
    n = torch.where(step > 0, ((x - low) / step).round().clamp(max=15), torch.zeros_like(x)).to(torch.uint8)
    n = n.unflatten(-1, (-1, 8))[..., _NIBBLES]
    packed = (n[..., 0::2] | (n[..., 1::2] << 4)).flatten(-2)
    return packed, torch.cat([step, low], -1).to(torch.bfloat16)


def _unpack(packed, scale):
    """The values (float32) that packed rows stand for."""
    b = packed.unflatten(-1, (-1, 4))
    n = torch.stack([b & 15, b >> 4], -1).flatten(-2)[..., [0, 4, 1, 5, 2, 6, 3, 7]].flatten(-2)
    return n.float() * scale[..., :1].float() + scale[..., 1:].float()


def _plain_append(s):
    cache, (page, row) = s["cache"], _token_slots(s)
    s["status"].zero_()
    if s["case"]["format"] == "bf16":
        cache["k"][0, page, :, row] = s["k"]
        cache["v"][0, page, :, row] = s["v"]
        return dict(k=cache["k"], v=cache["v"], status=s["status"])
    (kp, ks), (vp, vs) = _pack(s["k"].float()), _pack(s["v"].float())
    cache["k"][0, page, :, row], cache["k_scale"][0, page, :, row] = kp, ks
    cache["v"][0, page, :, row], cache["v_scale"][0, page, :, row] = vp, vs
    k = _unpack(cache["k"][0, page, :, row], cache["k_scale"][0, page, :, row])
    v = _unpack(cache["v"][0, page, :, row], cache["v_scale"][0, page, :, row])
    return dict(k=k.to(torch.bfloat16), v=v.to(torch.bfloat16), status=s["status"])


def _plain_attend(s):
    c, kv_len, offsets = s["case"], s["kv_len"].long(), s["offsets"].long()
    page, window, sinks, heads = c["page"], c["window"], c["sinks"], c["kv_heads"]
    n, most, group = c["requests"], s["most"], c["heads"] // c["kv_heads"]
    dev = kv_len.device
    news = offsets[1:] - offsets[:-1]
    # the slots that some query of the request may see: the sinks, then from the window's start on
    if window:
        first = (kv_len - window + 1).clamp(min=0)
        slots = first[:, None] + torch.arange(min(window + most, s["longest"]), device=dev)
        slots = torch.cat([torch.arange(sinks, device=dev).expand(n, -1), slots], 1)
        once = torch.arange(slots.shape[1], device=dev) < sinks
        there = once | (slots >= sinks)
    else:
        slots = torch.arange(s["longest"], device=dev).expand(n, -1)
        there = torch.ones_like(slots, dtype=torch.bool)
    there = there & (slots < (kv_len + news)[:, None])
    pages = torch.gather(s["page_table"].long(), 1, (slots // page).clamp(max=s["page_table"].shape[1] - 1))
    there, pages = there & (pages >= 0), pages.clamp(min=0)
    if c["format"] == "int4":
        k = _unpack(s["cache"]["k"][0, pages, :, slots % page], s["cache"]["k_scale"][0, pages, :, slots % page])
        v = _unpack(s["cache"]["v"][0, pages, :, slots % page], s["cache"]["v_scale"][0, pages, :, slots % page])
    else:
        k, v = (s["cache"][x][0, pages, :, slots % page].float() for x in ("k", "v"))
    v = torch.where(there[..., None, None], v, torch.zeros((), device=dev))
    # queries, padded to the most that a request has
    at = (offsets[:-1, None] + torch.arange(most, device=dev)).clamp(max=s["total"] - 1)
    live = torch.arange(most, device=dev) < news[:, None]
    q = s["q"][at].float().view(n, most, heads, group, -1).permute(0, 2, 1, 3, 4).reshape(n, heads, most * group, -1)
    # what each query sees
    node = torch.arange(most, device=dev).expand(n, -1)
    draft = slots - kv_len[:, None]  # the key's own number among the new tokens, or negative
    if c["tree"]:
        up = s["parents"].long()[at]
        up = torch.where(live & (node > 0), up, node)
        hop = torch.zeros(n, most, most, device=dev).scatter_(2, up[..., None], 1.0)
        reach = ((hop + torch.eye(most, device=dev)) > 0).float()
        for _ in range(6):  # 2^6 steps reach every ancestor of 64 nodes
            reach = (reach @ reach > 0).float()
        depth = reach.sum(-1).long() - 1
        sees = torch.gather(reach, 2, draft.clamp(0, most - 1)[:, None].expand(-1, most, -1)) > 0
        sees = torch.where((draft < 0)[:, None], True, sees)
        place = torch.where(draft < 0, slots, kv_len[:, None] + torch.gather(depth, 1, draft.clamp(0, most - 1)))
    else:
        depth, place = node, slots
        sees = draft[:, None] <= node[..., None]
    if window:
        p = kv_len[:, None] + depth
        sees = sees & ((place[:, None] > p[..., None] - window) | (place[:, None] < sinks))
    sees = (sees & there[:, None])[:, None, :, None].expand(-1, -1, -1, group, -1)
    x = (q @ k.permute(0, 2, 3, 1)) * s["scale"]
    del k
    x = x.view(n, heads, most, group, -1).masked_fill_(~sees, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    mass = x.sum(-1, keepdim=True)
    out = (x.view(n, heads, most * group, -1) @ v.permute(0, 2, 1, 3)).view(n, heads, most, group, -1)
    out = torch.where(mass > 0, out / mass, torch.zeros_like(out))
    lse = (top + mass.log()).squeeze(-1)
    s["out"][at[live]] = out.permute(0, 2, 1, 3, 4).flatten(2, 3)[live].to(torch.bfloat16)
    s["lse"][at[live]] = lse.permute(0, 2, 1, 3).flatten(2, 3)[live]
    s["status"].zero_()
    return dict(out=s["out"], lse=s["lse"], status=s["status"])


def _take(pool, need):
    """Pages for a table of `need` (truth values, in order): each its page from the top of the stack, -1 elsewhere."""
    flat = need.flatten().long()
    nth = flat.cumsum(0) - 1
    at = (pool["free_count"].long() - 1 - nth).clamp(min=0)
    got = torch.where(flat > 0, pool["free_pages"][at], torch.full_like(pool["free_pages"][at], -1))
    pool["ref_count"].index_add_(0, got.clamp(min=0).long(), flat.to(torch.int32))
    pool["free_count"] -= flat.sum().to(torch.int32)
    return got.view(need.shape)


def _plain_trim(pool, rows, length, status):
    """Drops the rows' pages past `length`; pages that nothing holds any more go back, the last table entry first."""
    page, table = pool["page_size"], pool["page_table"]
    entries = table[rows]
    width = entries.shape[1]
    drop = (entries >= 0) & (torch.arange(width, device=table.device) * page >= length[:, None])
    table[rows] = torch.where(drop, torch.full_like(entries, -1), entries)
    ids, lin = entries[drop].long(), drop.flatten().nonzero().flatten()
    refs = pool["ref_count"]
    refs.index_add_(0, ids, torch.full_like(ids, -1, dtype=torch.int32))
    owner = torch.full((refs.numel(),), -1, dtype=torch.long, device=table.device)
    owner.scatter_reduce_(0, ids, lin, "amax")
    mine = (owner[ids] == lin) & (refs[ids] == 0)
    back = ids[mine].flip(0).to(torch.int32)
    pool["free_pages"][(pool["free_count"].long() + torch.arange(back.numel(), device=table.device))] = back
    pool["free_count"] += back.numel()
    status.zero_()


def _plain_pages(s):
    pool, cache, page = s["pool"], s["cache"], s["case"]["page"]
    out = dict(page_table=pool["page_table"], ref_count=pool["ref_count"], free_count=pool["free_count"],
               k=cache["k"], v=cache["v"], status=s["status"])
    table = pool["page_table"]
    col = torch.arange(table.shape[1], device=table.device)
    s["status"].zero_()
    if s["case"]["kind"] == "fork":
        parent, child, length = s["parent"].long(), s["child"].long(), s["length"]
        full = (length // page)[:, None]
        old = table[parent]
        shared = (col < full) & (old >= 0)
        pool["ref_count"].index_add_(0, old[shared].long(), torch.ones_like(old[shared]))
        last = (length % page > 0) & (torch.gather(old, 1, full.long())[:, 0] >= 0)
        new = _take(pool, last)
        table[child] = torch.where(shared, old, torch.where((col == full) & last[:, None], new[:, None],
                                                            torch.full_like(old, -1)))
        src, dst = torch.gather(old, 1, full.long())[:, 0][last].long(), new[last].long()
        held = torch.arange(page, device=table.device) < (length % page)[last][:, None]  # [copies, page]
        held = held[None, :, None, :, None]
        for x in ("k", "v"):
            cache[x][:, dst] = torch.where(held, cache[x][:, src], cache[x][:, dst])
        out["forked"] = table.clone()
        _plain_trim(pool, child, s["zero"], s["status2"])
        return out | dict(status2=s["status2"])
    n = s["kv_len"].numel()
    need = (col >= (s["kv_len"] // page)[:, None]) & (col * page < s["to_len"][:, None]) & (table < 0)
    table.copy_(torch.where(need, _take(pool, need), table))
    # accepted rows to consecutive slots
    deep = torch.arange(s["path"].shape[1], device=table.device)
    r, j = (deep < s["accepted"][:, None]).nonzero(as_tuple=True)
    src, dst = s["kv_len"][r] + s["path"][r, j], s["kv_len"][r] + 1 + j
    sp, dp = table[r, (src // page).long()].long(), table[r, (dst // page).long()].long()
    for x in ("k", "v"):
        cache[x][:, dp, :, dst % page] = cache[x][:, sp, :, src % page]
    s["new_len"].copy_(s["kv_len"] + 1 + s["accepted"])
    s["status2"].zero_()
    _plain_trim(pool, torch.arange(n, device=table.device), s["new_len"], s["status3"])
    return out | dict(status2=s["status2"], status3=s["status3"], new_len=s["new_len"])


# ------------------------------------------------------------------- work --

def _visible(base, news, window, sinks, upto):
    """Visible (query, key) pairs of one request, and its keys that some query sees (drafts in a row; a tree's
    queries see about as many)."""
    pairs = 0
    for i in range(news):
        p = base + i
        low = max(0, p - window + 1) if window else 0
        pairs += p - low + 1 + min(low, sinks)
    low = max(0, base - window + 1) if window else 0
    return pairs, upto - low + min(low, sinks)


def work(case):
    if case["op"] == "append":
        tokens = sum(_lengths(case)[1])
        row = case["kv_heads"] * case["head_dim"] * 2
        if case["format"] == "bf16":
            return dict(bytes=4 * tokens * row, flops=0)
        packed = case["kv_heads"] * (case["head_dim"] // 2 + 4)
        # read, quantise and write; then read the 4 bits and write bf16
        return dict(bytes=4 * tokens * row + 4 * tokens * packed, flops=0)
    if case["op"] == "attend":
        lens, news = _lengths(case)
        pairs = keys = 0
        for a, b in zip(lens, news):
            p, k = _visible(a, b, case["window"], case["sinks"], a + b)
            pairs, keys = pairs + p, keys + k
        dim = case["head_dim"]
        row = 2 * (dim * 2 if case["format"] == "bf16" else dim // 2 + 4)
        return dict(bytes=keys * case["kv_heads"] * row + sum(news) * case["heads"] * (4 * dim + 4),
                    flops=4 * pairs * case["heads"] * dim)
    row = case["layers"] * case["kv_heads"] * case["head_dim"] * 4  # one token's keys and values in every layer
    lo, hi = case["len_min"], case["len_max"]
    if case["kind"] == "fork":
        n = case["parents"]
        lens = [lo + ((hi - lo) * i) // max(1, n - 1) for i in range(n)]
        moved = sum(x % case["page"] for x in lens) * case["children"]
        table = 2 * 4 * n * case["children"] * (-(-hi // case["page"]) + 1)
    else:
        n = case["requests"]
        moved = sum(min((i * 5 + n) % (case["depth_max"] + 1), (case["nodes_max"] - 1) // 2) for i in range(n))
        table = 2 * 4 * n * (-(-(hi + case["nodes_max"]) // case["page"]) + 1)
    return dict(bytes=2 * moved * row + table, flops=0)


# ------------------------------------------------------------ in 64 bits --

def exact(case, seed):
    """The outputs from the definitions, in 64 bits, one request at a time."""
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "attend":
        lens, news = _lengths(case)
        pairs = sum(b * (min(a + b, case["window"] + b) if case["window"] else a + b) for a, b in zip(lens, news))
        if pairs * case["heads"] * case["head_dim"] * 4 > 4e12:
            return None
        return _exact_attend(s)
    return None  # whole numbers and copies: nothing is computed


def _exact_row_values(x):
    """What a 4-bit row of x (float64 [dim]) stands for, by the definition."""
    low = x.min(-1, keepdim=True).values
    r = (x.max(-1, keepdim=True).values - low) / 15
    e = torch.floor(torch.log2(torch.where(r > 0, r, torch.ones_like(r))))
    ulp = torch.exp2(e - 7)
    step = torch.ceil(r / ulp) * ulp
    n = torch.where(r > 0, torch.round((x - low) / torch.where(r > 0, step, torch.ones_like(r))).clamp(max=15), 0 * x)
    return n * step + low


def _exact_append(s):
    if s["case"]["format"] == "int4":
        return dict(k=_exact_row_values(s["k"].double()), v=_exact_row_values(s["v"].double()), status=None)
    k, v = s["cache"]["k"].double(), s["cache"]["v"].double()
    page, offsets, lens = s["case"]["page"], s["offsets"].tolist(), s["kv_len"].tolist()
    table = s["page_table"].tolist()
    for r, base in enumerate(lens):
        for i in range(offsets[r + 1] - offsets[r]):
            p, row = table[r][(base + i) // page], (base + i) % page
            k[0, p, :, row] = s["k"][offsets[r] + i].double()
            v[0, p, :, row] = s["v"][offsets[r] + i].double()
    return dict(k=k, v=v, status=None)


def _exact_attend(s):
    c = s["case"]
    page, window, sinks, group = c["page"], c["window"], c["sinks"], c["heads"] // c["kv_heads"]
    offsets, lens, table = s["offsets"].tolist(), s["kv_len"].tolist(), s["page_table"].tolist()
    parents = s["parents"].tolist() if c["tree"] else None
    out = torch.zeros(s["total"], c["heads"], c["head_dim"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["total"], c["heads"], dtype=torch.float64, device="cuda")
    for r, base in enumerate(lens):
        first, n = offsets[r], offsets[r + 1] - offsets[r]
        low = max(0, base - window + 1) if window else 0
        slots = list(range(min(sinks, low))) + list(range(low, base + n))
        slots = torch.tensor([x for x in slots if table[r][x // page] >= 0], device="cuda")
        pages = torch.tensor(table[r], device="cuda")[slots // page]
        values = []
        for x in ("k", "v"):
            rows = s["cache"][x][0, pages, :, slots % page]
            if c["format"] == "int4":
                scale = s["cache"][x + "_scale"][0, pages, :, slots % page].double()
                word = rows.unflatten(-1, (-1, 4)).long()
                word = (word * torch.tensor([1, 1 << 8, 1 << 16, 1 << 24], device="cuda")).sum(-1)
                bits = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device="cuda")
                rows = ((word[..., None] >> bits) & 15).flatten(-2).double() * scale[..., :1] + scale[..., 1:]
            values.append(rows.double())
        k, v = values
        if parents is None:
            depth = list(range(n))
        else:
            depth, line = [0] * n, [{0}]
            for i in range(1, n):
                depth[i] = depth[parents[first + i]] + 1
                line.append(line[parents[first + i]] | {i})
        place = slots.clone()
        if parents is not None:
            new = slots >= base
            place[new] = base + torch.tensor(depth, device="cuda")[slots[new] - base]
        for at in range(0, n, 512):  # in pieces, for the memory
            upto = min(n, at + 512)
            p = base + torch.tensor(depth[at:upto], device="cuda")[:, None]
            if parents is None:
                see = slots <= p
            else:
                see = torch.zeros(upto - at, len(slots), dtype=torch.bool, device="cuda")
                see[:, slots < base] = True
                for i in range(at, upto):
                    mine = torch.tensor(sorted(line[i]), device="cuda") + base
                    see[i - at] |= torch.isin(slots, mine)
            if window:
                see = see & ((place > p - window) | (place < sinks))
            for h in range(c["heads"]):
                x = (s["q"][first + at:first + upto, h].double() @ k[:, h // group].T) * s["scale"]
                x = x.masked_fill(~see, -math.inf)
                top = x.amax(-1, keepdim=True)
                e = torch.exp(x - top)
                mass = e.sum(-1, keepdim=True)
                out[first + at:first + upto, h] = (e @ v[:, h // group]) / mass
                lse[first + at:first + upto, h] = (top + mass.log())[:, 0]
    return dict(out=out, lse=lse, status=None)
