"""Rotary positions and the 8-bit cache without a GPU: the frequencies, the
refusals of the entry points and of the binding, and the plain
implementations against other ways to say the same."""
import ctypes as C
import math

import numpy as np
import pytest

from speculative_verification_gb300 import build as ss_build
from speculative_verification_gb300 import ss
from tests import rope_ref as P
from tests.test_cache_abi import append_args, attention, attention_args, cache, pool

torch = pytest.importorskip("torch")
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    ss_build.build()
    return ss.load()


def eight(**kw):
    c = cache(format=2, slot_stride=64, k_scale=4096, v_scale=8192, scale_layer_stride=1 << 16, scale_page_stride=1 << 10,
              scale_head_stride=4)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_EIGHT = [dict(k_scale=None), dict(v_scale=None), dict(k_scale=4098), dict(v_scale=8194), dict(head_dim=8),
             dict(head_dim=72), dict(head_dim=144), dict(slot_stride=48), dict(slot_stride=72), dict(scale_head_stride=0),
             dict(scale_page_stride=(1 << 10) + 2), dict(page_size=32), dict(page_size=4), dict(format=3), dict(k=4100)]


def table(**kw):
    t = ss.ss_rope_table(4096, 64, 0, 1.0)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


BAD_TURNS = [dict(turns=None), dict(turns=4100), dict(rot_dim=0), dict(rot_dim=-2), dict(rot_dim=7), dict(rot_dim=66),
             dict(layout=2), dict(layout=-1), dict(magnitude=float("inf")), dict(magnitude=float("nan"))]


def rope_args(t=None, **kw):
    a = ss.ss_rope_args(C.pointer(t or table()), 2, 4, 8, 64, 4096, 4096, None, None, 8, 4, 4096, 4096, 512, 64, 512, 64,
                        4096, 4096, 256, 64, 256, 64, 4096)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def step_args(t=None, b=None, **kw):
    a = ss.ss_rope_append_args(C.pointer(t or table()), C.pointer(b or append_args()), None, None, 8, 4096, 4096, 512, 64,
                               512, 64)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_caches_of_8_bits_that_cannot_be(lib):
    ok = C.c_void_p(4096)
    for kw in BAD_EIGHT:
        c = eight(**kw)
        for rows in (lib.ss_cache_append, lib.ss_cache_read):
            assert rows(C.byref(append_args(c)), None) == INVALID, kw
        assert attention(lib, attention_args(c)) == INVALID, kw
        assert lib.ss_rope_append(C.byref(step_args(b=append_args(c))), None) == INVALID, kw
        assert lib.ss_pages_fork(C.byref(pool()), C.byref(c), 1, ok, ok, ok, ok, None) == INVALID, kw
        assert lib.ss_pages_compact(C.byref(pool()), C.byref(c), 1, None, ok, ok, 4, ok, None, C.c_void_p(8192), ok,
                                    None) == INVALID, kw
    # and one that can: the next check answers
    assert attention(lib, attention_args(eight()), size=0) == 4
    assert lib.ss_cache_append(C.byref(append_args(eight(), num_requests=0)), None) == 0
    assert lib.ss_cache_append(C.byref(append_args(eight(), max_tokens=1 << 28)), None) == UNSUPPORTED


def test_rope_refusals(lib):
    assert lib.ss_rope(None, None) == INVALID
    for kw in BAD_TURNS:
        assert lib.ss_rope(C.byref(rope_args(table(**kw))), None) == INVALID, kw
        assert lib.ss_rope_append(C.byref(step_args(table(**kw))), None) == INVALID, kw
    for kw in (dict(rope=None), dict(num_requests=-1), dict(num_requests=65536), dict(max_tokens=-1), dict(total_tokens=-1),
               dict(head_dim=0), dict(head_dim=68), dict(head_dim=136), dict(head_dim=56), dict(kv_len=None),
               dict(parents=4096, positions=4096), dict(num_heads=-1), dict(num_heads=65536), dict(num_kv_heads=-1),
               dict(q=4100), dict(q_out=None), dict(q_out=4104), dict(k=4098), dict(k_out=None), dict(k_out=4108),
               dict(q_token_stride=508), dict(q_head_stride=4), dict(q_out_token_stride=9), dict(q_out_head_stride=1),
               dict(k_token_stride=2), dict(k_head_stride=-1), dict(k_out_token_stride=4), dict(k_out_head_stride=12),
               dict(out_status=None), dict(token_offsets=None, total_tokens=1)):
        assert lib.ss_rope(C.byref(rope_args(**kw)), None) == INVALID, kw
    assert lib.ss_rope(C.byref(rope_args(num_requests=0)), None) == 0


def test_rope_append_refusals(lib):
    assert lib.ss_rope_append(None, None) == INVALID
    for kw in (dict(rope=None), dict(append=None), dict(parents=4096, positions=4096), dict(num_heads=-1),
               dict(num_heads=65536), dict(q=None), dict(q_out=None), dict(q=4104), dict(q_out=4100),
               dict(q_token_stride=4), dict(q_head_stride=7), dict(q_out_token_stride=-4), dict(q_out_head_stride=2)):
        assert lib.ss_rope_append(C.byref(step_args(**kw)), None) == INVALID, kw
    for kw in (dict(layer=2), dict(num_requests=-1), dict(kv_len=None), dict(out_status=None), dict(k=None),
               dict(token_stride=4), dict(token_offsets=None, total_tokens=1)):
        assert lib.ss_rope_append(C.byref(step_args(b=append_args(**kw))), None) == INVALID, kw
    # turns of more channels than the cache's heads have
    assert lib.ss_rope_append(C.byref(step_args(table(rot_dim=128))), None) == INVALID
    assert lib.ss_rope_append(C.byref(step_args(b=append_args(num_requests=0))), None) == 0


@pytest.mark.parametrize("kw", [dict(base=10000.0), dict(base=500000.0, scaling="linear", factor=4.0), dict(base=6.2832),
                                dict(base=500000.0, scaling="by_parts", factor=8.0, length=8192.0, low=1.0, high=4.0),
                                dict(base=10000.0, scaling="by_parts", factor=40.0, length=4096.0, low=1.0, high=32.0)])
@pytest.mark.parametrize("rot_dim", [2, 10, 64, 128])
def test_frequencies(lib, kw, rot_dim):
    rope = ss.Rope(128, rot_dim=rot_dim, device="cpu", **kw)
    got = [int(x) for x in rope.turns.numpy().view(np.uint64)]
    want = P.turns(rot_dim, **kw)
    assert len(got) == rot_dim // 2
    for a, b in zip(got, want):
        # pow and a handful of double operations, each off by a unit of 2^-53 at most a few times, and half a unit of
        # the fixed point
        assert abs(a / 2.0 ** 64 - float(b)) <= 2.0 ** -48 * float(b) + 2.0 ** -65 * 1.01


def test_frequencies_that_cannot_be(lib):
    out = (C.c_uint64 * 64)()
    good = dict(rot_dim=64, base=1e4, scaling=0, factor=1.0, length=1.0, low=1.0, high=4.0)

    def call(**kw):
        a = {**good, **kw}
        return lib.ss_rope_turns(a["rot_dim"], a["base"], a["scaling"], a["factor"], a["length"], a["low"], a["high"], out)

    assert call() == 0 and abs(out[0] / 2 ** 64 * 2 * math.pi - 1) < 1e-15
    before = list(out)
    inf, nan = float("inf"), float("nan")
    for kw in (dict(rot_dim=0), dict(rot_dim=130), dict(rot_dim=5), dict(base=0.0), dict(base=-1.0), dict(base=inf),
               dict(base=nan), dict(base=1e-9), dict(scaling=3), dict(scaling=-1), dict(scaling=1, factor=0.0),
               dict(scaling=1, factor=0.1), dict(scaling=1, factor=nan), dict(scaling=2, factor=2.0, length=0.0),
               dict(scaling=2, factor=2.0, low=4.0), dict(scaling=2, factor=2.0, low=-1.0), dict(scaling=2, high=inf),
               dict(scaling=2, length=nan)):
        assert call(**kw) == INVALID, kw
    assert list(out) == before  # nothing half done
    assert lib.ss_rope_turns(64, 1e4, 0, 1.0, 1.0, 1.0, 4.0, None) == INVALID
    for kw in (dict(layout="rows"), dict(scaling="log"), dict(rot_dim=130), dict(rot_dim=3), dict(rot_dim=0),
               dict(base=float("nan")), dict(turns=torch.zeros(64)), dict(turns=torch.zeros(63, dtype=torch.int64))):
        with pytest.raises(ss.SSError):
            ss.Rope(128, device="cpu", **kw)


def test_the_plain_rounding_is_the_types():
    g = np.random.default_rng(1)
    x = np.concatenate([g.standard_normal(4000) * np.exp2(g.integers(-12, 8, 4000)), [0.0, 2.0 ** -10, 3 * 2.0 ** -10, 448, 464]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn)
    assert np.array_equal(P.e4m3(x), want.float().numpy().astype(np.float64))
    assert np.array_equal(P.e4m3_of(want.view(torch.uint8).numpy()), P.e4m3(x))
    every = np.arange(256)
    back = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(P.e4m3_of(every), back.astype(np.float64), equal_nan=True)
    assert np.isnan(P.e4m3([np.inf, -np.inf, np.nan])).all()


def test_the_plain_scale():
    for top, want in ((448.0, 1.0), (449.0, 2.0), (0.0, 2.0 ** -100), (224.0, 0.5), (2.0 ** -120, 2.0 ** -100),
                      (3.3895e38, 2.0 ** 120), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8), (1.7578125, 2.0 ** -7)):
        assert P.scale_of(np.array([[-top, 0.0], [np.nan, np.inf]])) == want, top


def test_the_plain_rotation_is_a_rotation():
    g = np.random.default_rng(2)
    x = g.standard_normal((5, 3, 12))
    table = [int(float(t) * 2.0 ** 64) for t in P.turns(8, 100.0)]
    for layout in ("halves", "interleaved"):
        y = P.turn(x, [0, 3, 10 ** 6, -7, 2 ** 31 - 1], table, 8, layout, 2.0)
        assert np.array_equal(y[0], np.concatenate([2 * x[0, :, :8], x[0, :, 8:]], -1)) and np.array_equal(y[..., 8:], x[..., 8:])
        assert np.allclose((y[..., :8] ** 2).sum(-1), 4 * (x[..., :8] ** 2).sum(-1))
        # the product of two turned rows depends on the distance alone
        q, k = (np.stack([g.standard_normal((1, 12))] * 2) for _ in range(2))
        a, b = P.turn(q, [5, 105], table, 8, layout, 1.0), P.turn(k, [2, 102], table, 8, layout, 1.0)
        assert np.allclose((a[0, 0] * b[0, 0]).sum(), (a[1, 0] * b[1, 0]).sum())
    # pair (x, y) at a quarter turn becomes (-y, x)
    z = P.turn(np.array([[[1.0, 2.0, 3.0, 4.0]]]), [1], [2 ** 62, 2 ** 62], 4, "halves", 1.0)
    assert np.allclose(z, [[[-3.0, -4.0, 1.0, 2.0]]])


def test_the_plain_append_and_compact():
    g = np.random.default_rng(3)
    c = P.Cache8(g.integers(0, 120, (3, 2, 16, 4)), np.exp2(g.integers(-9, -6, (3, 2, 1))))
    before = c.n.copy()
    old = c.values(1, 0, slice(0, 3))
    new = g.standard_normal((4, 2, 4)) * 100
    c.append([1, 2], 3, new)
    s = c.s[1, 0, 0]
    assert 448 * s >= np.abs(new[:, 0]).max() and 224 * s < np.abs(np.concatenate([new[:, 0], old])).max()
    assert np.abs(c.values(1, 0, slice(3, 7)) - new[:, 0]).max() <= 2.0 ** -4 * np.abs(new).max()
    assert np.array_equal(c.n[1, :, 7:], before[1, :, 7:]) and np.array_equal(c.n[2], before[2])
    held = c.values(1, 1, slice(0, 7)).copy()
    c.compact([1, 2], 2, [2, 4])  # slots 4 and 6 to 3 and 4
    got = c.values(1, 1, slice(0, 5))
    want = held[[0, 1, 2, 4, 6]]
    assert np.abs(got - want).max() <= 2.0 ** -10 * c.s[1, 1, 0] * 8 + 2.0 ** -4 * np.abs(want).max()


# ------------------------------------------------------------ the binding --

from tests.test_cache_binding import Elsewhere, Host, calls, half, ints, moved, on, pools  # noqa: E402, F401


def eight_tensors(page=16):
    shape = (1, 4, 2, page)
    data = lambda: on(torch.zeros(*shape, 64, dtype=torch.uint8).view(torch.float8_e4m3fn))  # noqa: E731
    scale = lambda: on(torch.zeros(1, 4, 2, max(1, page // 16)))  # noqa: E731
    return dict(k=data(), v=data(), k_scale=scale(), v_scale=scale())


def a_rope(device_of=lambda t: t, dim=64):
    return ss.Rope(dim, turns=device_of(on(torch.zeros(dim // 2, dtype=torch.int64))))


def rope(t):
    a = dict(q=half(3, 4, 64), q_out=half(3, 4, 64), k=half(3, 2, 64), k_out=half(3, 2, 64), kv_len=ints(3), status=ints(3),
             token_offsets=ints(4), parents=ints(3))
    a.update(t)
    r = a.pop("rope", None) or a_rope()
    ss.ss_rope(r, *(a.pop(x) for x in ("q", "q_out", "k", "k_out", "kv_len", "status")), max_tokens=1, **a)


def step(t):
    a = dict(q=half(3, 4, 64), q_out=half(3, 4, 64), k=half(3, 2, 64), v=half(3, 2, 64), page_table=ints(3, 2), kv_len=ints(3),
             status=ints(3), token_offsets=ints(4), table_rows=ints(3), positions=ints(3))
    a.update(t)
    r, c = a.pop("rope", None) or a_rope(), a.pop("cache", None) or ss.KVCache(**eight_tensors())
    ss.ss_rope_append(r, c, 0, *(a.pop(x) for x in ("q", "q_out", "k", "v", "page_table", "kv_len", "status")), max_tokens=1, **a)


@pytest.mark.parametrize("call,name,arguments", [
    (rope, "ss_rope", "q q_out k k_out kv_len status token_offsets parents positions"),
    (step, "ss_rope_append", "q q_out k v page_table kv_len status token_offsets table_rows parents positions")])
def test_every_argument_is_asked_for_its_gpu(calls, call, name, arguments):  # noqa: F811
    call({})
    assert calls == [name]
    shapes = {"q": half(3, 4, 64), "q_out": half(3, 4, 64), "k": half(3, 2, 64), "k_out": half(3, 2, 64), "v": half(3, 2, 64),
              "page_table": ints(3, 2), "token_offsets": ints(4)}
    for x in arguments.split():
        for cls in (Host, Elsewhere):
            with pytest.raises(ss.SSError):
                call({x: moved(shapes.get(x, ints(3)), cls)})
    for cls in (Host, Elsewhere):
        with pytest.raises(ss.SSError):
            call({"rope": a_rope(lambda t: moved(t, cls))})
        if call is step:
            there = ss.KVCache(**{k: moved(t, cls) for k, t in eight_tensors().items()})
            with pytest.raises(ss.SSError):
                call({"cache": there})
    assert calls == [name]


def test_arguments_of_other_shapes_and_types(calls):  # noqa: F811
    for call, t in ((rope, dict(q=half(3, 4, 32))), (rope, dict(q_out=half(3, 5, 64))), (rope, dict(q_out=None)), (rope, dict(k=None)),
                    (rope, dict(q=half(3, 64, 4).transpose(1, 2))), (rope, dict(q=half(4, 4, 64), q_out=half(4, 4, 64))),
                    (rope, dict(parents=ints(4))), (rope, dict(kv_len=ints(2))), (rope, dict(token_offsets=ints(3))),
                    (rope, dict(q=half(3, 256))), (rope, dict(k=half(3, 2, 64).float())), (rope, dict(positions=half(3))),
                    (step, dict(rope=a_rope(dim=128))), (step, dict(q=half(2, 4, 64), q_out=half(2, 4, 64))),
                    (step, dict(v=half(3, 3, 64))), (step, dict(k=half(3, 2, 32), v=half(3, 2, 32))), (step, dict(q_out=None)),
                    (step, dict(page_table=ss.PagePool(page_size=32, **pools())))):
        with pytest.raises(ss.SSError):
            call(t)
    assert not calls
    rope(dict(q=None, q_out=None))
    rope(dict(k=None, k_out=None, kv_len=None, positions=ints(3), parents=None))
    step(dict(q=None, q_out=None, page_table=ss.PagePool(page_size=16, **pools())))
    assert calls == ["ss_rope", "ss_rope", "ss_rope_append"]


def test_caches_of_8_bits():
    for page in (8, 16, 64):
        c = ss.KVCache(**eight_tensors(page))
        assert c.format == "fp8" and c.struct.format == 2 and c.head_dim == 64 and c.struct.slot_stride == 64
        assert c.struct.scale_head_stride == 4 * max(1, page // 16)
    for kw in (dict(k_scale=on(torch.zeros(1, 4, 2, 2))), dict(k_scale=None), dict(v_scale=None), dict(v=half(1, 4, 2, 16, 64)),
               dict(k_scale=on(torch.zeros(1, 4, 2, 1, dtype=torch.float64))), dict(v_scale=moved(on(torch.zeros(1, 4, 2, 1)), Host)),
               dict(v_scale=on(torch.zeros(1, 2, 4, 1).transpose(1, 2)))):
        with pytest.raises(ss.SSError):
            ss.KVCache(**{**eight_tensors(), **kw})
    with pytest.raises(ss.SSError):
        ss.alloc_cache(1, 2, 2, 16, 64, "e4m3", device="cpu")
    c = ss.alloc_cache(2, 3, 2, 32, 48, "fp8", device="cpu")
    assert c.k.shape == (2, 3, 2, 32, 48) and c.v_scale.shape == (2, 3, 2, 2) and c.device == -1
