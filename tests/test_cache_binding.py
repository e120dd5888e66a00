"""The binding of the paged-cache calls refuses memory of the host or of
another GPU, each argument by itself, before the library is called.  Runs
without a GPU: the tensors only say that they are on one, and the library is
a stand-in that counts its calls."""
import pytest

from speculative_verification_gb300 import ss

torch = pytest.importorskip("torch")


class Placed(torch.Tensor):
    """A host tensor that claims to be on GPU `place`."""

    place = 0

    def get_device(self):
        return self.place

    @property
    def is_cuda(self):
        return self.place >= 0


class Elsewhere(Placed):
    place = 1


class Host(Placed):
    place = -1


def on(t, cls=Placed):
    return t.as_subclass(cls)


def ints(*shape):
    return on(torch.zeros(*shape, dtype=torch.int32))


def half(*shape):
    return on(torch.zeros(*shape, dtype=torch.bfloat16))


@pytest.fixture()
def calls(monkeypatch):
    made = []

    def fn(name):
        def call(*args):
            made.append(name)
            return 0
        return call

    class Library:
        def __getattr__(self, name):
            return fn(name)

    monkeypatch.setattr(ss, "load", lambda path=None: Library())
    monkeypatch.setattr(ss, "_quick_call", lambda name, argtypes: fn(name))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    return made


def caches(fmt):
    shape = (1, 4, 2, 16)
    if fmt == "bf16":
        return dict(k=half(*shape, 64), v=half(*shape, 64))
    return dict(k=on(torch.zeros(*shape, 32, dtype=torch.uint8)), v=on(torch.zeros(*shape, 32, dtype=torch.uint8)),
                k_scale=half(*shape, 2), v_scale=half(*shape, 2))


def pools():
    return dict(page_table=ints(3, 2), ref_count=ints(4), free_pages=ints(4), free_count=ints(1))


def rows_call(fn, c, t):
    a = dict(k=half(3, 2, 64), v=half(3, 2, 64), page_table=ints(3, 2), kv_len=ints(3), status=ints(3), token_offsets=ints(4),
             table_rows=ints(3))
    a.update(t)
    fn(c, 0, a.pop("k"), a.pop("v"), a.pop("page_table"), a.pop("kv_len"), a.pop("status"), max_tokens=1, **a)


def attention(c, t):
    a = dict(q=half(3, 4, 64), out=half(3, 4, 64), page_table=ints(3, 2), kv_len=ints(3), workspace=ints(64), status=ints(3),
             query_offsets=ints(4), parents=ints(3), lse=on(torch.zeros(3, 4)), table_rows=ints(3))
    a.update(t)
    ss.ss_cache_attention(c, 0, *(a.pop(x) for x in ("q", "out", "page_table", "kv_len", "workspace", "status")), **a)


CALLS = {
    "ss_cache_append": (lambda c, p, t: rows_call(ss.ss_cache_append, c, t),
                        "k v page_table kv_len status token_offsets table_rows"),
    "ss_cache_read": (lambda c, p, t: rows_call(ss.ss_cache_read, c, t),
                      "k v page_table kv_len status token_offsets table_rows"),
    "ss_cache_attention": (lambda c, p, t: attention(c, t),
                           "q out page_table kv_len workspace status query_offsets parents lse table_rows"),
    "ss_pages_reserve": (lambda c, p, t: ss.ss_pages_reserve(p, **{**{x: ints(3) for x in
                                                                     ("from_len", "to_len", "status", "table_rows")}, **t}),
                         "from_len to_len status table_rows"),
    "ss_pages_fork": (lambda c, p, t: ss.ss_pages_fork(p, c, **{**{x: ints(3) for x in
                                                                  ("parent", "child", "length", "status")}, **t}),
                      "parent child length status"),
    "ss_pages_compact": (lambda c, p, t: ss.ss_pages_compact(p, c, **{**{x: ints(3) for x in (
        "kv_len", "num_accepted", "verify_status", "new_len", "status", "table_rows")}, "path": ints(3, 4), **t}),
        "kv_len path num_accepted verify_status new_len status table_rows"),
    "ss_pages_trim": (lambda c, p, t: ss.ss_pages_trim(p, **{**{x: ints(3) for x in ("length", "status", "table_rows")}, **t}),
                      "length status table_rows"),
}


def moved(t, cls):
    return t.as_subclass(torch.Tensor).as_subclass(cls)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("name", CALLS)
def test_every_argument_is_asked_for_its_gpu(calls, name, fmt):
    call, arguments = CALLS[name]
    cache, pool = ss.KVCache(**caches(fmt)), ss.PagePool(page_size=16, **pools())
    call(cache, pool, {})
    assert calls == [name]
    for x in arguments.split():
        # the argument's own tensor, placed elsewhere
        for cls in (Host, Elsewhere):
            t = {"path": ints(3, 4), "page_table": ints(3, 2), "token_offsets": ints(4), "query_offsets": ints(4),
                 "workspace": ints(64), "lse": on(torch.zeros(3, 4)), "q": half(3, 4, 64), "out": half(3, 4, 64),
                 "k": half(3, 2, 64), "v": half(3, 2, 64)}.get(x, ints(3))
            with pytest.raises(ss.SSError):
                call(cache, pool, {x: moved(t, cls)})
    for cls in (Host, Elsewhere):
        there = ss.KVCache(**{k: moved(t, cls) for k, t in caches(fmt).items()})
        if "pages" not in name or name in ("ss_pages_fork", "ss_pages_compact"):
            with pytest.raises(ss.SSError):
                call(there, pool, {})
    assert calls == [name]


def test_handles_hold_memory_of_one_gpu():
    for fmt in ("bf16", "int4"):
        for x in caches(fmt):
            for cls in (Host, Elsewhere):
                t = caches(fmt)
                t[x] = moved(t[x], cls)
                with pytest.raises(ss.SSError):
                    ss.KVCache(**t)
    for x in pools():
        for cls in (Host, Elsewhere):
            t = pools()
            t[x] = moved(t[x], cls)
            with pytest.raises(ss.SSError):
                ss.PagePool(page_size=16, **t)


def test_a_pool_of_another_gpu_and_a_workspace_with_gaps(calls):
    cache = ss.KVCache(**caches("bf16"))
    pool = ss.PagePool(page_size=16, **{k: moved(t, Elsewhere) for k, t in pools().items()})
    for x in ("ss_cache_append", "ss_cache_read", "ss_cache_attention"):
        with pytest.raises(ss.SSError):
            CALLS[x][0](cache, pool, {"page_table": pool})
    for x in ("ss_pages_reserve", "ss_pages_fork", "ss_pages_compact", "ss_pages_trim"):
        with pytest.raises(ss.SSError):
            CALLS[x][0](cache, pool, {})
    with pytest.raises(ss.SSError):
        CALLS["ss_cache_attention"][0](cache, None, {"workspace": ints(64, 2)[:, 0]})
    assert not calls


def test_the_current_device_and_the_stream_are_the_memorys(calls, monkeypatch):
    cache = ss.KVCache(**caches("bf16"))

    class Stream:
        cuda_stream, device_index = 5, 1

    call = CALLS["ss_cache_attention"][0]
    with pytest.raises(ss.SSError):
        call(cache, None, {"stream": Stream()})
    assert not calls
    Stream.device_index = 0
    call(cache, None, {"stream": Stream()})
    assert calls == ["ss_cache_attention"]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ss.SSError):
        call(cache, None, {})
    assert calls == ["ss_cache_attention"]


def test_a_pool_of_another_page_size(calls):
    # slots would be looked up in the wrong pages
    cache, pool = ss.KVCache(**caches("bf16")), ss.PagePool(page_size=32, **pools())
    for x in ("ss_cache_append", "ss_cache_read", "ss_cache_attention"):
        with pytest.raises(ss.SSError):
            CALLS[x][0](cache, pool, {"page_table": pool})
    assert not calls
    pool = ss.PagePool(page_size=16, **pools())
    CALLS["ss_cache_append"][0](cache, pool, {"page_table": pool})
    assert calls == ["ss_cache_append"]


def test_rows_of_a_request_end_before_31_bits_do():
    # the library itself, which refuses before anything is launched
    from speculative_verification_gb300 import build as ss_build
    from tests.test_cache_abi import attention, attention_args
    ss_build.build()
    lib = ss.load()
    for heads, most, want in ((4, 2 ** 29 - 2048, 4), (4, 2 ** 29 - 2047, 1), (4, 2 ** 29 - 1, 1), (128, 2 ** 24 - 64, 4),
                              (128, 2 ** 24 - 63, 1), (512, 2 ** 31 - 1, 1)):
        a = attention_args(num_heads=heads, max_queries=most)
        # accepted counts go on to the next check, a workspace that is too small
        assert attention(lib, a, size=0) == want, (heads, most)
