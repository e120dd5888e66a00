"""The paged-cache entry points refuse what they cannot do, before anything is
launched (no GPU needed), and the plain implementations agree with themselves."""
import ctypes as C

import numpy as np
import pytest

from speculative_verification_gb300 import build as ss_build
from speculative_verification_gb300 import ss
from tests import cache_ref as R

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    ss_build.build()
    return ss.load()


def cache(**kw):
    c = ss.ss_kv_cache(0, 2, 10, 4, 16, 64, 4096, 8192, 1 << 20, 1 << 14, 1 << 11, 128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def packed(**kw):
    c = cache(format=1, slot_stride=32, k_scale=4096, v_scale=8192, scale_layer_stride=1 << 16,
              scale_page_stride=1 << 10, scale_head_stride=64)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def pool(**kw):
    p = ss.ss_page_pool(3, 5, 5, 4096, 10, 16, 4096, 4096, 4096)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


BAD_CACHES = [dict(format=2), dict(num_layers=0), dict(num_pages=0), dict(num_kv_heads=0), dict(page_size=12),
              dict(page_size=4), dict(page_size=2048), dict(head_dim=0), dict(head_dim=63), dict(head_dim=136), dict(k=None),
              dict(v=None), dict(k=4104), dict(v=8200), dict(slot_stride=112), dict(slot_stride=136), dict(page_stride=-16),
              dict(head_stride=1 << 41), dict(layer_stride=(1 << 20) + 8)]
BAD_PACKED = [dict(k_scale=None), dict(v_scale=None), dict(k_scale=4100), dict(head_dim=48), dict(scale_head_stride=48),
              dict(scale_page_stride=(1 << 10) + 4), dict(slot_stride=16)]
BAD_TABLES = [dict(num_rows=0), dict(max_pages=0), dict(row_stride=4), dict(page_table=None)]


def append_args(c=None, p=None, **kw):
    a = ss.ss_append_args(C.pointer(c or cache()), C.pointer(p or pool()), 0, 2, 4, 8, 4096, None, 4096, 4096, 4096,
                          256, 64, 4096)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def attention_args(c=None, p=None, **kw):
    a = ss.ss_attention_args(C.pointer(c or cache()), C.pointer(p or pool()), 0, 2, 8, 4, 8, 4096, None, 4096, None, 4096,
                             512, 64, 4096, 512, 64, None, 0.125, 0, 0, 4096)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def attention(lib, a, ws=4096, size=None):
    return lib.ss_cache_attention(C.byref(a) if a else None, C.c_void_p(ws),
                                  lib.ss_attention_workspace_size() if size is None else size, None)


def test_caches_and_tables_that_cannot_be(lib):
    for rows in (lib.ss_cache_append, lib.ss_cache_read):
        assert rows(None, None) == INVALID
        for kw in BAD_CACHES:
            assert rows(C.byref(append_args(cache(**kw))), None) == INVALID, kw
        for kw in BAD_PACKED:
            assert rows(C.byref(append_args(packed(**kw))), None) == INVALID, kw
        for kw in BAD_TABLES:
            assert rows(C.byref(append_args(p=pool(**kw))), None) == INVALID, kw
        for kw in (dict(layer=2), dict(layer=-1), dict(num_requests=-1), dict(max_tokens=-1), dict(total_tokens=-1),
                   dict(kv_len=None), dict(out_status=None), dict(k=None), dict(v=4100), dict(token_stride=257),
                   dict(head_stride=60), dict(token_offsets=None, total_tokens=1), dict(num_requests=70000)):
            assert rows(C.byref(append_args(**kw)), None) == INVALID, kw
        assert rows(C.byref(append_args(num_requests=0)), None) == 0  # nothing to do
    for kw in BAD_CACHES:
        assert attention(lib, attention_args(cache(**kw))) == INVALID, kw
    for kw in BAD_PACKED:
        assert attention(lib, attention_args(packed(**kw))) == INVALID, kw
    for kw in BAD_TABLES:
        assert attention(lib, attention_args(p=pool(**kw))) == INVALID, kw


def test_attention_refusals(lib):
    assert attention(lib, None) == INVALID
    for kw in (dict(layer=2), dict(num_requests=-1), dict(max_queries=-1), dict(total_queries=-1), dict(num_heads=0),
               dict(num_heads=6), dict(num_heads=4 * 129), dict(window=-1), dict(sinks=-1), dict(scale=float("inf")),
               dict(scale=float("nan")), dict(kv_len=None), dict(out_status=None), dict(q=None), dict(q=4100), dict(out=None),
               dict(out=4097), dict(q_token_stride=510), dict(q_head_stride=4), dict(query_offsets=None, total_queries=1)):
        assert attention(lib, attention_args(**kw)) == INVALID, kw
    assert attention(lib, attention_args(), ws=None) == WORKSPACE
    assert attention(lib, attention_args(), ws=4096 + 16) == WORKSPACE
    assert attention(lib, attention_args(), size=lib.ss_attention_workspace_size() - 1) == WORKSPACE
    assert attention(lib, attention_args(num_requests=0), ws=None) == 0


def test_pages_refusals(lib):
    ok = C.c_void_p(4096)
    bad_pools = BAD_TABLES + [dict(num_pages=0), dict(page_size=24), dict(page_size=0), dict(ref_count=None),
                              dict(free_pages=None), dict(free_count=None)]
    for kw in bad_pools:
        p = C.byref(pool(**kw))
        assert lib.ss_pages_reserve(p, 1, None, ok, ok, ok, None) == INVALID, kw
        assert lib.ss_pages_fork(p, C.byref(cache()), 1, ok, ok, ok, ok, None) == INVALID, kw
        assert lib.ss_pages_trim(p, 1, None, ok, 0, 0, ok, None) == INVALID, kw
    p, c = C.byref(pool()), C.byref(cache())
    assert lib.ss_pages_reserve(None, 1, None, ok, ok, ok, None) == INVALID
    assert lib.ss_pages_reserve(p, -1, None, ok, ok, ok, None) == INVALID
    assert lib.ss_pages_reserve(p, 1, None, None, ok, ok, None) == INVALID
    assert lib.ss_pages_reserve(p, 1, None, ok, ok, None, None) == INVALID
    assert lib.ss_pages_reserve(p, 0, None, None, None, None, None) == 0
    assert lib.ss_pages_fork(p, c, 1, None, ok, ok, ok, None) == INVALID
    assert lib.ss_pages_fork(p, C.byref(cache(page_size=32, head_stride=1 << 12)), 1, ok, ok, ok, ok, None) == INVALID
    assert lib.ss_pages_fork(p, C.byref(cache(num_pages=11)), 1, ok, ok, ok, ok, None) == INVALID
    assert lib.ss_pages_fork(p, c, 0, None, None, None, None, None) == 0
    assert lib.ss_pages_trim(p, 1, None, ok, -1, 0, ok, None) == INVALID
    assert lib.ss_pages_trim(p, 1, None, ok, 0, -1, ok, None) == INVALID
    assert lib.ss_pages_trim(p, 1, None, None, 0, 0, ok, None) == INVALID
    assert lib.ss_pages_trim(C.byref(pool(max_pages=1 << 20, row_stride=1 << 20)), 1 << 12, None, ok, 0, 0, ok,
                             None) == UNSUPPORTED
    f = lib.ss_pages_compact
    assert f(p, c, 1, None, ok, ok, 4, ok, None, C.c_void_p(8192), None, None) == INVALID
    assert f(p, c, 1, None, ok, ok, 4, ok, None, ok, ok, None) == INVALID  # new_len is kv_len
    assert f(p, c, 1, None, ok, None, 4, ok, None, C.c_void_p(8192), ok, None) == INVALID
    assert f(p, c, 1, None, ok, ok, -1, ok, None, C.c_void_p(8192), ok, None) == INVALID
    assert f(p, c, 0, None, None, None, 4, None, None, None, None, None) == 0


def test_binding_refuses_tensors_that_do_not_fit():
    torch = pytest.importorskip("torch")
    k = torch.zeros(1, 2, 2, 16, 64, dtype=torch.bfloat16)
    ss.KVCache(k, k.clone())
    with pytest.raises(ss.SSError):
        ss.KVCache(k.float(), k.float())
    with pytest.raises(ss.SSError):
        ss.KVCache(k, k[:, :1])
    with pytest.raises(ss.SSError):
        ss.KVCache(k, k.transpose(1, 2).contiguous().transpose(1, 2))  # other strides
    with pytest.raises(ss.SSError):
        ss.KVCache(k, k.clone(), torch.zeros(1, 2, 2, 16, 2), torch.zeros(1, 2, 2, 16, 2))
    with pytest.raises(ss.SSError):
        ss.alloc_cache(1, 1, 1, 16, 64, "int3", device="cpu")
    c = ss.alloc_cache(2, 3, 1, 16, 64, "int4", device="cpu")
    assert (c.head_dim, c.struct.slot_stride, c.struct.scale_head_stride) == (64, 32, 64)
    i32 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ss.SSError):  # not on the device
        ss.ss_cache_append(c, 0, torch.zeros(4, 1, 64), torch.zeros(4, 1, 64), i32[None], i32, i32)


def test_plain_rows_round_trip():
    rng = np.random.default_rng(0)
    x = R.bf16(rng.standard_normal((50, 64)) * np.exp(rng.uniform(-4, 4, (50, 1))))
    n, s, m = R.quantise(x)
    assert np.array_equal(R.unpack(R.pack(n)), n)
    assert np.array_equal(R.bf16(s), s) and np.array_equal(R.bf16(m), m)
    assert (np.abs(n * s[:, None].astype(np.float64) + m[:, None] - x) <= s[:, None] * 0.5000001).all()
    assert (15 * s.astype(np.float64) + m >= x.max(-1)).all()
