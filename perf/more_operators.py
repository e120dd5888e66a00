"""Rotary positions and the 8-bit cache, as cases that can be timed and compared.

Four operators around one layer of the paged key/value cache:

  rotate  a step's queries and keys turned by their positions: channels paired by halves or interleaved, the whole
          head or its first part, frequencies scaled for contexts longer than the trained one
  write   new keys and values into a cache of 8 bits, whose blocks of 16 slots share a scale for each head; read back
  step    both at once: queries and keys turned, the keys and values written, into a cache of any format; read back
  attend  attention over the 8-bit cache: single tokens, drafts in a row or in a tree, prompt chunks, windows and sinks

With `own` false every operator is computed by elementary torch operations, in 32 bits (angles in 64); with `own`
true by the library's entry points.
"""
import math
import random

import torch

own = False

#: Slots that share a scale (all of a page that is smaller).
_BLOCK = 16


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # One token of one chat request: the smallest call, all latency.
        dict(name="rotate 1 x 1 token", op="rotate", requests=1, heads=32, kv_heads=8, head_dim=128, rot_dim=128,
             layout="halves", scaling="none", len_min=700, len_max=700, tokens_min=1, tokens_max=1, tree=False),
        # Prompt chunks far into a long context, half of the head turned, interleaved, frequencies scaled by parts.
        dict(name="rotate 4 x 4096 prompt, interleaved", op="rotate", requests=4, heads=32, kv_heads=8, head_dim=128,
             rot_dim=64, layout="interleaved", scaling="by_parts", len_min=4096, len_max=60000, tokens_min=4093,
             tokens_max=4096, tree=False),
        # One verification step's new tokens of a batch, small pages: most blocks hold rows already.
        dict(name="write 32 x 1-8 tokens", op="write", format="fp8", requests=32, kv_heads=8, head_dim=128, page=16,
             len_min=100, len_max=3000, tokens_min=1, tokens_max=8),
        # Prompt chunks of four requests, then read back as a program does that moves a request.
        dict(name="write 4 x 2-6k tokens", op="write", format="fp8", requests=4, kv_heads=8, head_dim=128, page=64,
             len_min=0, len_max=5000, tokens_min=2011, tokens_max=6143),
        # Draft trees of a batch before their attention: nodes of one depth share a position.
        dict(name="step 32 trees", op="step", format="fp8", requests=32, heads=32, kv_heads=8, head_dim=128,
             rot_dim=128, layout="halves", scaling="linear", page=64, len_min=500, len_max=12000, tokens_min=9,
             tokens_max=48, tree=True),
        # Prompt chunks into a bf16 cache.
        dict(name="step bf16 2 x 4096 prompt", op="step", format="bf16", requests=2, heads=32, kv_heads=8,
             head_dim=128, rot_dim=128, layout="halves", scaling="none", page=64, len_min=0, len_max=4096,
             tokens_min=4095, tokens_max=4096, tree=False),
        # A single chat request, one token a step, a short window: the smallest attention call.
        dict(name="8-bit window 1 x 1 token, 700", op="attend", format="fp8", requests=1, heads=32, kv_heads=8,
             head_dim=128, page=16, len_min=700, len_max=700, queries_min=1, queries_max=1, tree=False, window=512,
             sinks=4),
        # A few requests with small heads of an odd size, and the smallest pages, each a block of its own.
        dict(name="8-bit 4 x 1-3 tokens, 1-2k, dim 80", op="attend", format="fp8", requests=4, heads=20, kv_heads=4,
             head_dim=80, page=8, len_min=1000, len_max=2000, queries_min=1, queries_max=3, tree=False, window=0,
             sinks=0),
        # Decode over long contexts: bound by reading the cache.
        dict(name="8-bit 32 x 1 token, 8-64k", op="attend", format="fp8", requests=32, heads=32, kv_heads=8,
             head_dim=128, page=64, len_min=8000, len_max=64000, queries_min=1, queries_max=1, tree=False, window=0,
             sinks=0),
        # Verification of 1 to 8 positions, wide head groups.
        dict(name="8-bit 48 x 1-8 drafts, 1-16k", op="attend", format="fp8", requests=48, heads=64, kv_heads=8,
             head_dim=128, page=64, len_min=1000, len_max=16000, queries_min=1, queries_max=8, tree=False, window=0,
             sinks=0),
        # Tree verification: up to 64 nodes a request, small heads, full attention.
        dict(name="8-bit 16 trees, 2-12k", op="attend", format="fp8", requests=16, heads=16, kv_heads=4, head_dim=64,
             page=32, len_min=2000, len_max=12000, queries_min=17, queries_max=64, tree=True, window=0, sinks=0),
        # Prompt chunks: the second chunk of two prompts, thousands of queries with a window of 1024.
        dict(name="8-bit window 1024, 2 x 4096 prompt", op="attend", format="fp8", requests=2, heads=32, kv_heads=8,
             head_dim=128, page=64, len_min=0, len_max=4096, queries_min=4095, queries_max=4096, tree=False,
             window=1024, sinks=4),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rotate", "write", "step", "step tree", "decode", "drafts", "prompt", "tree"])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    head_dim = rng.choice([32, 64, 64, 80, 96, 128, 128, 128])
    page = rng.choice([8, 16, 32, 64, 128])
    rotary = dict(rot_dim=rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4]),
                  layout=rng.choice(["halves", "interleaved"]), scaling=rng.choice(["none", "linear", "by_parts"]))
    if kind in ("rotate", "write", "step", "step tree"):
        tree = kind == "step tree"
        requests = _log(rng, 1, 48)
        tokens = _log(rng, 1, 64 if tree else max(1, 16000 // requests))
        first = _log(rng, 1, 50000 if kind == "rotate" else 5000)
        case = dict(requests=requests, kv_heads=kv_heads, head_dim=head_dim, len_min=first - 1,
                    len_max=first + _log(rng, 1, 3000), tokens_min=max(1, tokens // 3), tokens_max=tokens)
        if kind == "rotate":
            return dict(op="rotate", heads=kv_heads * rng.choice([1, 2, 4, 5, 8]), tree=tokens <= 64 and
                        rng.random() < 0.5, **rotary, **case)
        if kind == "write":
            return dict(op="write", format="fp8", page=page, **case)
        fmt = rng.choice(["fp8", "fp8", "bf16", "int4"])
        if fmt == "int4":
            case["head_dim"] = head_dim = rng.choice([64, 96, 128])
            rotary["rot_dim"] = rng.choice([head_dim, head_dim // 2])
        return dict(op="step", format=fmt, heads=kv_heads * rng.choice([1, 2, 4, 5, 8]), page=page, tree=tree, **rotary,
                    **case)
    if kind in ("decode", "drafts"):
        requests = _log(rng, 1, 32)
        longest = _log(rng, 64, 32000 if requests > 8 else 64000)
        return dict(op="attend", format="fp8", requests=requests, heads=kv_heads * rng.choice([1, 2, 4, 5, 7, 8]),
                    kv_heads=kv_heads, head_dim=head_dim, page=page,
                    len_min=max(0, longest // rng.choice([1, 2, 8]) - 1), len_max=longest, queries_min=1,
                    queries_max=1 if kind == "decode" else _log(rng, 2, 8), tree=False,
                    window=rng.choice([0, 0, _log(rng, 100, 20000)]), sinks=rng.choice([0, 4, 64, 131]))
    if kind == "prompt":
        queries = _log(rng, 100, 4000)
        return dict(op="attend", format="fp8", requests=rng.choice([1, 2]), heads=kv_heads * 4, kv_heads=kv_heads,
                    head_dim=head_dim, page=page, len_min=0, len_max=_log(rng, 1, 4000), queries_min=queries // 2,
                    queries_max=queries, tree=False, window=rng.choice([0, _log(rng, 100, 2000)]),
                    sinks=rng.choice([0, 4, 64]))
    longest = _log(rng, 100, 16000)
    return dict(op="attend", format="fp8", requests=_log(rng, 1, 16), heads=kv_heads * rng.choice([1, 4, 8]),
                kv_heads=kv_heads, head_dim=head_dim, page=page, len_min=longest // 3, len_max=longest, queries_min=1,
                queries_max=_log(rng, 2, 64), tree=True, window=rng.choice([0, _log(rng, 100, 8000)]),
                sinks=rng.choice([0, 4, 64]))


# ----------------------------------------------------------------- inputs --

#: How the frequencies are scaled, as a model's configuration says it: the base, the trained length and by how much
#: positions are stretched; by parts, channels that turn less than `low` times within that length are stretched
#: wholly, those that turn more than `high` times not at all, and all are multiplied by the magnitude.
_SCALING = {"none": dict(base=10000.0), "linear": dict(base=10000.0, scaling="linear", factor=4.0),
            "by_parts": dict(base=500000.0, scaling="by_parts", factor=8.0, length=8192, low=1.0, high=4.0,
                             magnitude=0.1 * math.log(8.0) + 1.0)}


def _lengths(case):
    """Each request's cached length and number of new tokens: a request's two numbers go together, so that the work
    of a case does not depend on the seed (the seed orders the requests)."""
    n = case["requests"]
    lo, hi = case["len_min"], case["len_max"]
    qlo, qhi = (case[k] for k in (("queries_min", "queries_max") if case["op"] == "attend" else
                                  ("tokens_min", "tokens_max")))
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


def _filled(gen, pages, heads, page, dim):
    """An 8-bit cache's bytes and scales as writing ordinary rows leaves them."""
    block = min(_BLOCK, page)
    data = torch.empty(1, pages, heads, page, dim, dtype=torch.uint8, device="cuda")
    scale = torch.empty(1, pages, heads, page // block, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (heads * page * dim))
    for p in range(0, pages, step):
        x = _kv(gen, min(step, pages - p), heads, page // block, block, dim)
        s = _scale_of(x.abs().amax((-1, -2)).float())
        scale[0, p:p + step] = s
        x = (x / s[..., None, None].to(torch.bfloat16)).to(torch.float8_e4m3fn)
        data[0, p:p + step] = x.view(torch.uint8).flatten(2, 3)
    return data, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    n, op, heads, dim = case["requests"], case["op"], case["kv_heads"], case["head_dim"]
    pairs = list(zip(*_lengths(case)))
    rng.shuffle(pairs)
    lens, news = [a for a, _ in pairs], [b for _, b in pairs]
    s = dict(case=case, kv_len=_ints(lens), offsets=_ints(_offsets(news)), total=sum(news), most=max(news),
             longest=max(a + b for a, b in pairs))
    s["parents"] = _ints(_parents(rng, news)) if case.get("tree") else None
    s["status"] = torch.empty(n, dtype=torch.int32, device="cuda")
    if "page" in case:
        page = case["page"]
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
        s["page_table"] = torch.where(table >= 0, order[table.clamp(min=0).long()], table)
        shape = (1, used + 3, heads, page)
        if case["format"] == "fp8":
            k, ks = _filled(gen, used + 3, heads, page, dim)
            v, vs = _filled(gen, used + 3, heads, page, dim)
            # pages that no request holds: whatever was there before
            v[:, order[used:].long()] = 0x7f
            s["cache"] = dict(k=k, v=v, k_scale=ks, v_scale=vs)
        elif case["format"] == "int4":
            s["cache"] = dict(k=torch.zeros(*shape, dim // 2, dtype=torch.uint8, device="cuda"),
                              v=torch.zeros(*shape, dim // 2, dtype=torch.uint8, device="cuda"),
                              k_scale=torch.zeros(*shape, 2, dtype=torch.bfloat16, device="cuda"),
                              v_scale=torch.zeros(*shape, 2, dtype=torch.bfloat16, device="cuda"))
        else:
            s["cache"] = dict(k=_kv(gen, *shape, dim), v=_kv(gen, *shape, dim))
    if op == "attend":
        s["q"] = _rand(gen, sum(news), case["heads"], dim)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(sum(news), case["heads"], dtype=torch.float32, device="cuda")
        s["scale"] = dim ** -0.5
    else:
        # one layer's projection: queries, keys and values side by side
        h = case.get("heads", 0)
        qkv = _kv(gen, sum(news), h + 2 * heads, dim)
        s["q"], s["k"], s["v"] = qkv[:, :h], qkv[:, h:h + heads], qkv[:, h + heads:]
        s["q_out"] = torch.empty(sum(news), h, dim, dtype=torch.bfloat16, device="cuda")
    if op == "rotate":
        s["k_out"] = torch.empty(sum(news), heads, dim, dtype=torch.bfloat16, device="cuda")
    if op in ("write", "step"):
        # read back: the new rows, and the rows before them that share a block with the first
        back = [a % min(_BLOCK, case["page"]) for a in lens]
        s["read_len"] = _ints([a - c for a, c in zip(lens, back)])
        s["read_offsets"] = _ints(_offsets([b + c for b, c in zip(news, back)]))
        s["read_most"] = max(b + c for b, c in zip(news, back))
        s["k_read"], s["v_read"] = (torch.empty(sum(news) + sum(back), heads, dim, dtype=torch.bfloat16, device="cuda")
                                    for _ in range(2))
        s["read_status"] = torch.empty(n, dtype=torch.int32, device="cuda")
    if own:
        from speculative_verification_gb300 import ss
        if "scaling" in case:
            s["rope"] = ss.Rope(dim, rot_dim=case["rot_dim"], layout=case["layout"], **_SCALING[case["scaling"]])
        if "page" in case:
            c = dict(s["cache"])
            if case["format"] == "fp8":
                c["k"], c["v"] = (c[x].view(torch.float8_e4m3fn) for x in ("k", "v"))
            s["handle"] = ss.KVCache(**c)
        if op == "attend":
            s["workspace"] = ss.alloc_attention_workspace()
    return s


# --------------------------------------------------------------- one pass --

def run(state):
    op = state["case"]["op"]
    if own:
        return dict(rotate=_own_rotate, write=_own_write, step=_own_step, attend=_own_attend)[op](state)
    return dict(rotate=_plain_rotate, write=_plain_write, step=_plain_step, attend=_plain_attend)[op](state)


def _own_rotate(s):
    from speculative_verification_gb300 import ss
    ss.ss_rope(s["rope"], s["q"], s["q_out"], s["k"], s["k_out"], s["kv_len"], s["status"], token_offsets=s["offsets"],
               max_tokens=s["most"], parents=s["parents"])
    return dict(q=s["q_out"], k=s["k_out"], status=s["status"])


def _own_read(s):
    from speculative_verification_gb300 import ss
    ss.ss_cache_read(s["handle"], 0, s["k_read"], s["v_read"], s["page_table"], s["read_len"], s["read_status"],
                     token_offsets=s["read_offsets"], max_tokens=s["read_most"])
    return dict(k=s["k_read"], v=s["v_read"], status=s["status"], read_status=s["read_status"])


def _own_write(s):
    from speculative_verification_gb300 import ss
    ss.ss_cache_append(s["handle"], 0, s["k"], s["v"], s["page_table"], s["kv_len"], s["status"],
                       token_offsets=s["offsets"], max_tokens=s["most"])
    return _own_read(s)


def _own_step(s):
    from speculative_verification_gb300 import ss
    ss.ss_rope_append(s["rope"], s["handle"], 0, s["q"], s["q_out"], s["k"], s["v"], s["page_table"], s["kv_len"],
                      s["status"], token_offsets=s["offsets"], max_tokens=s["most"], parents=s["parents"])
    return dict(q=s["q_out"], **_own_read(s))


def _own_attend(s):
    from speculative_verification_gb300 import ss
    c = s["case"]
    ss.ss_cache_attention(s["handle"], 0, s["q"], s["out"], s["page_table"], s["kv_len"], s["workspace"], s["status"],
                          query_offsets=s["offsets"], max_queries=s["most"], parents=s["parents"], scale=s["scale"],
                          window=c["window"], sinks=c["sinks"], lse=s["lse"])
    return dict(out=s["out"], lse=s["lse"], status=s["status"])


# ------------------------------------------------------------ plain forms --

def _frequencies(case):
    """Radians per position of each pair of channels, and the factor on sine and cosine."""
    c, pairs = _SCALING[case["scaling"]], case["rot_dim"] // 2
    f = [c["base"] ** (-i / pairs) for i in range(pairs)]
    if c.get("scaling") == "linear":
        f = [x / c["factor"] for x in f]
    elif c.get("scaling") == "by_parts":
        for i, x in enumerate(f):
            turns = c["length"] * x / (2 * math.pi)
            part = min(1.0, max(0.0, (turns - c["low"]) / (c["high"] - c["low"])))
            f[i] = x / c["factor"] * (1 - part) + x * part
    return f, c.get("magnitude", 1.0)


def _hops(s):
    """Trees: [requests, most, most] truth values, whether node i's path holds node j."""
    offsets, most = s["offsets"].long(), s["most"]
    dev = offsets.device
    news = offsets[1:] - offsets[:-1]
    node = torch.arange(most, device=dev).expand(len(news), -1)
    at = (offsets[:-1, None] + torch.arange(most, device=dev)).clamp(max=s["total"] - 1)
    up = torch.where((node < news[:, None]) & (node > 0), s["parents"].long()[at], node)
    hop = torch.zeros(len(news), most, most, device=dev).scatter_(2, up[..., None], 1.0)
    reach = ((hop + torch.eye(most, device=dev)) > 0).float()
    for _ in range(6):  # 2^6 steps reach every ancestor of 64 nodes
        reach = (reach @ reach > 0).float()
    return reach


def _token_rows(s, offsets, total):
    """For each token its request and number within it."""
    at = torch.arange(total, device="cuda", dtype=torch.int32)
    r = torch.searchsorted(offsets[1:].contiguous(), at, right=True)
    return r, at - offsets[r]


def _positions(s):
    r, i = _token_rows(s, s["offsets"], s["total"])
    if s["parents"] is not None:
        i = (_hops(s).sum(-1).to(torch.int32) - 1)[r, i.long()]
    return s["kv_len"][r] + i


def _turn(case, x, position):
    """Rows x [tokens, heads, dim] (float32) turned, in float32 with the angles in float64."""
    f, magnitude = _frequencies(case)
    angle = position.double()[:, None] * torch.tensor(f, dtype=torch.float64, device=x.device)
    cos, sin = (magnitude * angle.cos()).float()[:, None], (magnitude * angle.sin()).float()[:, None]
    rot = case["rot_dim"]
    if case["layout"] == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)
    a, b = x[..., :rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., rot:]], -1)


def _plain_rotate(s):
    position = _positions(s)
    s["q_out"].copy_(_turn(s["case"], s["q"].float(), position))
    s["k_out"].copy_(_turn(s["case"], s["k"].float(), position))
    s["status"].zero_()
    return dict(q=s["q_out"], k=s["k_out"], status=s["status"])


def _scale_of(top):
    """The power of two for a block's largest magnitude (float32): the smallest 2^e, e >= -100, with 448 2^e >= top."""
    bits = top.contiguous().view(torch.int32) + 0x1fffff  # a mantissa above 1.75 carries
    return (((bits >> 23) - 8).clamp(min=27) << 23).view(torch.float32)


def _slots(s, r, slot):
    page = s["case"]["page"]
    return s["page_table"][r, (slot // page).long()].long(), (slot % page).long()


def _write8(s, data, scale, new):
    """New rows (float32 [tokens, heads, dim]) into one of the cache's two 8-bit arrays, block by block."""
    block = min(_BLOCK, s["case"]["page"])
    kv_len, offsets = s["kv_len"].long(), s["offsets"].long()
    news = offsets[1:] - offsets[:-1]
    first, last = kv_len // block, (kv_len + news - 1) // block
    r, b = (torch.arange((s["most"] + 2 * block - 2) // block, device="cuda") <= (last - first)[:, None]).nonzero(as_tuple=True)
    slot = (first[r] + b)[:, None] * block + torch.arange(block, device="cuda")
    token = slot - kv_len[r][:, None]
    fresh, kept = (token >= 0) & (token < news[r][:, None]), token < 0
    page, row = _slots(s, r[:, None], slot)
    cell = (0, page[:, 0], slice(None), row[:, 0] // block)
    old = data[0, page, :, row].view(torch.float8_e4m3fn).float() * scale[cell][:, None, :, None]
    x = new[(offsets[r][:, None] + token).clamp(0, s["total"] - 1)]
    zero = torch.zeros((), device="cuda")
    x = torch.where(fresh[..., None, None], x, torch.where(kept[..., None, None], old, zero))
    del old
    top = torch.where(x.isfinite(), x.abs(), zero).amax((1, 3))
    step = _scale_of(top)
    x = x / step[:, None, :, None]
    x = torch.where(x.isfinite(), x, torch.full_like(zero, math.nan)).to(torch.float8_e4m3fn).view(torch.uint8)
    scale[cell] = step
    live = fresh | kept
    data[0, page[live], :, row[live]] = x[live]


#: Channel order of a packed word's nibbles, least significant byte first: channel 2i in bits 4i.., 2i + 1 in 16 + 4i..
_NIBBLES = [0, 2, 4, 6, 1, 3, 5, 7]


def _pack4(x):
    """4-bit rows of x [..., dim] (float32): the packed bytes and (step, lowest)."""
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    step = (high - low) / torch.full_like(low, 15)  # a tensor: by a number, torch multiplies by its reciprocal
    step = ((step.view(torch.int32) + 0xffff) & ~0xffff).view(torch.float32)  # up to a bf16
    n = torch.where(step > 0, ((x - low) / step).round().clamp(max=15), torch.zeros_like(x)).to(torch.uint8)
    n = n.unflatten(-1, (-1, 8))[..., _NIBBLES]
    packed = (n[..., 0::2] | (n[..., 1::2] << 4)).flatten(-2)
    return packed, torch.cat([step, low], -1).to(torch.bfloat16)


def _unpack4(packed, scale):
    """The values (float32) that packed rows stand for."""
    b = packed.unflatten(-1, (-1, 4))
    n = torch.stack([b & 15, b >> 4], -1).flatten(-2)[..., [0, 4, 1, 5, 2, 6, 3, 7]].flatten(-2)
    return n.float() * scale[..., :1].float() + scale[..., 1:].float()


def _plain_store(s, k, v):
    """Keys and values (bf16) into the cache, and the rows read back."""
    cache, fmt = s["cache"], s["case"]["format"]
    r, i = _token_rows(s, s["offsets"], s["total"])
    page, row = _slots(s, r, s["kv_len"][r] + i)
    for x, new in (("k", k), ("v", v)):
        if fmt == "fp8":
            _write8(s, cache[x], cache[x + "_scale"], new.float())
        elif fmt == "int4":
            cache[x][0, page, :, row], cache[x + "_scale"][0, page, :, row] = _pack4(new.float())
        else:
            cache[x][0, page, :, row] = new
    r, i = _token_rows(s, s["read_offsets"], s["k_read"].shape[0])
    page, row = _slots(s, r, s["read_len"][r] + i)
    for x in ("k", "v"):
        got = cache[x][0, page, :, row]
        if fmt == "fp8":
            got = got.view(torch.float8_e4m3fn).float() * cache[x + "_scale"][
                0, page, :, row // min(_BLOCK, s["case"]["page"])][..., None]
        elif fmt == "int4":
            got = _unpack4(got, cache[x + "_scale"][0, page, :, row])
        s[x + "_read"].copy_(got)
    s["status"].zero_()
    s["read_status"].zero_()
    return dict(k=s["k_read"], v=s["v_read"], status=s["status"], read_status=s["read_status"])


def _plain_write(s):
    return _plain_store(s, s["k"], s["v"])


def _plain_step(s):
    position = _positions(s)
    s["q_out"].copy_(_turn(s["case"], s["q"].float(), position))
    k = _turn(s["case"], s["k"].float(), position).to(torch.bfloat16)
    return dict(q=s["q_out"], **_plain_store(s, k, s["v"]))


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
    k, v = (s["cache"][x][0, pages, :, slots % page].view(torch.float8_e4m3fn).float() *
            s["cache"][x + "_scale"][0, pages, :, slots % page // min(_BLOCK, page)][..., None] for x in ("k", "v"))
    v = torch.where(there[..., None, None], v, torch.zeros((), device=dev))
    # queries, padded to the most that a request has
    at = (offsets[:-1, None] + torch.arange(most, device=dev)).clamp(max=s["total"] - 1)
    live = torch.arange(most, device=dev) < news[:, None]
    q = s["q"][at].float().view(n, most, heads, group, -1).permute(0, 2, 1, 3, 4).reshape(n, heads, most * group, -1)
    # what each query sees
    node = torch.arange(most, device=dev).expand(n, -1)
    draft = slots - kv_len[:, None]  # the key's own number among the new tokens, or negative
    if c["tree"]:
        reach = _hops(s)
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


# ------------------------------------------------------------------- work --

def _row_bytes(case):
    """Bytes of one row of one head in the cache, its share of the scales included."""
    dim = case["head_dim"]
    if case["format"] == "bf16":
        return 2 * dim
    return dim // 2 + 4 if case["format"] == "int4" else dim + 4 / min(_BLOCK, case["page"])


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
    lens, news = _lengths(case)
    tokens, dim, kv = sum(news), case["head_dim"], case["kv_heads"]
    if case["op"] == "attend":
        pairs = keys = 0
        for a, b in zip(lens, news):
            p, k = _visible(a, b, case["window"], case["sinks"], a + b)
            pairs, keys = pairs + p, keys + k
        return dict(bytes=int(keys * kv * 2 * _row_bytes(case)) + tokens * case["heads"] * (4 * dim + 4),
                    flops=4 * pairs * case["heads"] * dim)
    turned = (case.get("heads", 0) + kv) * tokens if "scaling" in case else 0
    flops = 3 * case.get("rot_dim", 0) * turned
    if case["op"] == "rotate":
        return dict(bytes=4 * dim * turned, flops=flops)
    back = tokens + sum(a % min(_BLOCK, case["page"]) for a in lens)
    # queries read and written, keys and values read as bf16 and written; then the rows read back and written as bf16
    return dict(bytes=int(4 * dim * tokens * case.get("heads", 0) + 2 * kv * tokens * (2 * dim + _row_bytes(case)) +
                          2 * kv * back * (2 * dim + _row_bytes(case))), flops=flops)


# ------------------------------------------------------------ in 64 bits --

def exact(case, seed):
    """The outputs from the definitions, in 64 bits, one request at a time."""
    s = prepare(case, seed)
    if case["op"] == "attend":
        lens, news = _lengths(case)
        pairs = sum(b * (min(a + b, case["window"] + b) if case["window"] else a + b) for a, b in zip(lens, news))
        if pairs * case["heads"] * case["head_dim"] * 4 > 4e12:
            return None
        return _exact_attend(s)
    if case["op"] == "rotate":
        return dict(q=_exact_turn(s, s["q"]), k=_exact_turn(s, s["k"]), status=None)
    out = {}
    k = s["k"].double()
    if case["op"] == "step":
        out["q"] = _exact_turn(s, s["q"])
        k = _exact_turn(s, s["k"]).to(torch.bfloat16).double()  # the keys are cached as bf16 has them
    return dict(out, k=_exact_cached(s, "k", k), v=_exact_cached(s, "v", s["v"].double()), status=None, read_status=None)


def _exact_depths(s):
    """Each token's number of steps from its request's first, and the tokens on its path."""
    offsets = s["offsets"].tolist()
    parents = s["parents"].tolist() if s["parents"] is not None else None
    depth, line = [], []
    for a, b in zip(offsets, offsets[1:]):
        d, p = [0], [{0}]
        for i in range(1, b - a):
            up = i - 1 if parents is None else parents[a + i]
            d.append(d[up] + 1)
            p.append(p[up] | {i} if parents is not None else None)
        depth.append(d)
        line.append(p)
    return depth, line


def _exact_turn(s, x):
    case = s["case"]
    depth, _ = _exact_depths(s)
    at = [a + d for a, row in zip(s["kv_len"].tolist(), depth) for d in row]
    f, magnitude = _frequencies(case)
    angle = torch.outer(torch.tensor(at, dtype=torch.float64, device="cuda"),
                        torch.tensor(f, dtype=torch.float64, device="cuda"))
    turn = torch.polar(torch.full_like(angle, magnitude), angle)[:, None]
    rot, y = case["rot_dim"], x.double().clone()
    if case["layout"] == "halves":
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * turn
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    else:
        z = torch.complex(y[..., 0:rot:2].contiguous(), y[..., 1:rot:2].contiguous()) * turn
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    return y


def _exact_e4m3(x):
    """The nearest numbers with 4 significant bits, exponents from -6 on: steps of 2^-9 at least, ties to even."""
    _, e = torch.frexp(x)  # |x| in [2^(e-1), 2^e)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.round(x / step) * step


def _exact_e4m3_of(byte):
    """What bytes stand for: sign, four bits of exponent, three of mantissa."""
    b = byte.long()
    e, m = (b >> 3) & 15, (b & 7).double()
    x = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10))
    return torch.where(b >= 128, -x, x)


def _exact_row4(x):
    """What a 4-bit row of x (float64 [dim]) stands for, by the definition."""
    low = x.min(-1, keepdim=True).values
    r = (x.max(-1, keepdim=True).values - low) / 15
    e = torch.floor(torch.log2(torch.where(r > 0, r, torch.ones_like(r))))
    ulp = torch.exp2(e - 7)
    step = torch.ceil(r / ulp) * ulp
    n = torch.where(r > 0, torch.round((x - low) / torch.where(r > 0, step, torch.ones_like(r))).clamp(max=15), 0 * x)
    return n * step + low


def _exact_cached(s, name, new):
    """The rows read back after new rows (float64) were written."""
    case, out = s["case"], []
    data, page = s["cache"][name][0], case["page"]
    block = min(_BLOCK, page)
    offsets, table = s["offsets"].tolist(), s["page_table"].tolist()
    for r, base in enumerate(s["kv_len"].tolist()):
        x = new[offsets[r]:offsets[r + 1]]
        before = base % block
        p, row = table[r][base // page], base % page - before
        old = data[p, :, row:row + before].transpose(0, 1)
        if case["format"] == "bf16":
            out.append(torch.cat([old.double(), x]))
            continue
        if case["format"] == "int4":  # rows that nothing was written to yet: zeros
            out.append(torch.cat([old.new_zeros(before, *x.shape[1:], dtype=torch.float64), _exact_row4(x)]))
            continue
        old = _exact_e4m3_of(old) * s["cache"][name + "_scale"][0, p, :, row // block].double()[:, None]
        x = torch.cat([old, x])
        pad = -len(x) % block
        x = torch.cat([x, x.new_zeros(pad, *x.shape[1:])]).unflatten(0, (-1, block))
        top, e = torch.frexp(x.abs().amax((1, 3)))
        step = torch.exp2(torch.where(top <= 0.875, e - 9, e - 8).clamp(min=-100).double())[:, None, :, None]
        x = (_exact_e4m3(x / step) * step).flatten(0, 1)
        out.append(x[:len(x) - pad])
    return torch.cat(out)


def _exact_attend(s):
    c = s["case"]
    page, window, sinks, group = c["page"], c["window"], c["sinks"], c["heads"] // c["kv_heads"]
    offsets, lens, table = s["offsets"].tolist(), s["kv_len"].tolist(), s["page_table"].tolist()
    depths, lines = _exact_depths(s)
    out = torch.zeros(s["total"], c["heads"], c["head_dim"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["total"], c["heads"], dtype=torch.float64, device="cuda")
    for r, base in enumerate(lens):
        first, n = offsets[r], offsets[r + 1] - offsets[r]
        low = max(0, base - window + 1) if window else 0
        slots = list(range(min(sinks, low))) + list(range(low, base + n))
        slots = torch.tensor([x for x in slots if table[r][x // page] >= 0], device="cuda")
        pages = torch.tensor(table[r], device="cuda")[slots // page]
        k, v = (_exact_e4m3_of(s["cache"][x][0, pages, :, slots % page]) *
                s["cache"][x + "_scale"][0, pages, :, slots % page // min(_BLOCK, page)].double()[..., None]
                for x in ("k", "v"))
        depth = torch.tensor(depths[r], device="cuda")
        place = slots.clone()
        if c["tree"]:
            new = slots >= base
            place[new] = base + depth[slots[new] - base]
        for at in range(0, n, 512):  # in pieces, for the memory
            upto = min(n, at + 512)
            p = base + depth[at:upto, None]
            if not c["tree"]:
                see = slots <= p
            else:
                see = torch.zeros(upto - at, len(slots), dtype=torch.bool, device="cuda")
                see[:, slots < base] = True
                for i in range(at, upto):
                    see[i - at] |= torch.isin(slots, torch.tensor(sorted(lines[r][i]), device="cuda") + base)
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
