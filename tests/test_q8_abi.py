"""Refusals and sizes of the 8-bit cache's entry points, and its reference against itself (no GPU)."""

import ctypes

import numpy as np
import pytest

import q8_reference as R

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P, BIG = ctypes.c_void_p(256), 1 << 50


@pytest.fixture(scope="module")
def lib():
    from looped_transformer_kv_gb300 import build
    build.build()
    from looped_transformer_kv_gb300 import _lib
    return _lib


def _shape(**kw):
    from looped_transformer_kv_gb300 import rq
    a = dict(batch=2, n_q_heads=4, n_kv_heads=2, head_dim=128, n_loops=4, capacity=128, fmt="e4m3")
    fmt = kw.pop("format", None)
    a.update(kw)
    s = rq.make_q8_shape(**a)
    if fmt is not None:
        s.format = fmt
    return s


def _rope(lib, **kw):
    a = dict(table=256, positions=None, n_pos=128, rot_dim=64, interleaved=0)
    a.update(kw)
    return lib.RqRope(a["table"], a["positions"], a["n_pos"], a["rot_dim"], a["interleaved"])


def _call(lib, what, shape=None, paging=None, paged=False, **kw):
    """Status of a call with dummy pointers: every one of these is refused before any use."""
    a = dict(codes=256, scales=256, cache=True, x=P, strides=(8,) * 5, loop=0, loops=1, n_lens=None, n=2, ctx=P,
             max_ctx=64, window=0, sinks=0, rope=None, out=ctypes.c_void_p(1 << 40), ws=P, ws_bytes=BIG)
    a.update(kw)
    s = shape or _shape()
    c = lib.RqQ8Cache(a["codes"], a["scales"])
    k = 5 if what == "append" else 3
    st = None if a["strides"] is None else (ctypes.c_int64 * k)(*a["strides"][:k])
    rope = None if a["rope"] is None else ctypes.byref(a["rope"])
    head = [ctypes.byref(s), ctypes.byref(c) if a["cache"] else None]
    if paged:
        head.append(None if paging is None else ctypes.byref(paging))
    L = lib.lib()
    if what == "append":
        f = L.rq_paged_q8_append if paged else L.rq_q8_append
        return f(*head, a["x"], st, a["loop"], a["loops"], a["n_lens"], a["n"], a["ctx"], rope, None)
    f = L.rq_paged_q8_attention if paged else L.rq_q8_attention
    return f(*head, a["x"], st, a["loop"], a["n_lens"], a["n"], a["ctx"], a["max_ctx"], a["window"], a["sinks"],
             rope, a["out"], a["ws"], a["ws_bytes"], None)


BOTH = [(dict(cache=False), INVALID), (dict(codes=0), INVALID), (dict(scales=0), INVALID), (dict(codes=256 + 64), INVALID),
        (dict(scales=256 + 8), INVALID), (dict(x=None), INVALID), (dict(strides=None), INVALID), (dict(ctx=None), INVALID),
        (dict(n=-1), INVALID), (dict(loop=-1), INVALID), (dict(loop=4), INVALID), (dict(strides=(8, -1, 8, 8, 8)), INVALID),
        (dict(strides=(1 << 62, 1 << 62, 8, 8, 8)), INVALID), (dict(n=0), OK), (dict(n=0, x=None), OK)]


@pytest.mark.parametrize("what", ["append", "attention"])
@pytest.mark.parametrize("kw,status", BOTH)
def test_refusals(lib, what, kw, status):
    assert _call(lib, what, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(loops=0), INVALID), (dict(loop=2, loops=3), INVALID), (dict(loop=1 << 30, loops=1 << 30), INVALID)])
def test_append_refusals(lib, kw, status):
    assert _call(lib, "append", **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(out=None), INVALID), (dict(max_ctx=-1), INVALID), (dict(max_ctx=129), INVALID), (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID), (dict(n=1 << 22), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws_bytes=255), WORKSPACE),
    (dict(ws=ctypes.c_void_p(128)), WORKSPACE), (dict(out=ctypes.c_void_p(256 + 64)), INVALID),
    (dict(n=0, ws=None, ws_bytes=0), OK)])
def test_attention_refusals(lib, kw, status):
    assert _call(lib, "attention", **kw) == status


@pytest.mark.parametrize("what", ["append", "attention"])
@pytest.mark.parametrize("kw,status", [
    (dict(table=0), INVALID), (dict(table=264), INVALID), (dict(n_pos=0), INVALID), (dict(rot_dim=0), INVALID),
    (dict(rot_dim=144), INVALID), (dict(rot_dim=24), UNSUPPORTED), (dict(interleaved=2), INVALID)])
def test_rotation_refusals(lib, what, kw, status):
    assert _call(lib, what, rope=_rope(lib, **kw)) == status


@pytest.mark.parametrize("what", ["append", "attention"])
@pytest.mark.parametrize("bad,status", [
    (dict(head_dim=96), UNSUPPORTED), (dict(format=2), UNSUPPORTED), (dict(n_loops=17), UNSUPPORTED), (dict(n_loops=0), INVALID),
    (dict(n_q_heads=3), INVALID), (dict(capacity=100), INVALID), (dict(batch=0), INVALID), (dict(batch=65536), UNSUPPORTED),
    (dict(softmax_scale=-1.0), INVALID), (dict(softmax_scale=float("nan")), INVALID), (dict(softmax_scale=float("inf")), INVALID)])
def test_bad_shapes(lib, what, bad, status):
    s = _shape(**bad)
    assert _call(lib, what, shape=s) == status
    assert lib.lib().rq_q8_cache_bytes(ctypes.byref(s)) == 0
    assert lib.lib().rq_q8_workspace_bytes(ctypes.byref(s), 1, 0, 0, 0) == 0


@pytest.mark.parametrize("what", ["append", "attention"])
def test_paging_refusals(lib, what):
    def paging(table=256, max_pages=2, n_pages=9):
        g = lib.RqPaging()
        g.block_table, g.max_pages, g.n_pages = table, max_pages, n_pages
        return g

    assert _call(lib, what, paged=True) == INVALID
    for bad in (dict(table=None), dict(max_pages=3), dict(max_pages=0), dict(n_pages=0)):
        assert _call(lib, what, paged=True, paging=paging(**bad)) == INVALID
    assert _call(lib, what, paged=True, paging=paging(), n=0) == OK


def test_cache_bytes(lib):
    s = _shape(head_dim=64, n_loops=3, capacity=192)
    assert lib.lib().rq_q8_cache_bytes(ctypes.byref(s)) == 2 * 2 * 192 * 3 * 2 * 64
    assert lib.lib().rq_q8_paged_cache_bytes(ctypes.byref(s), 7) == 7 * 2 * 64 * 3 * 2 * 64
    assert lib.lib().rq_q8_paged_cache_bytes(ctypes.byref(s), 0) == 0


def test_a_workspace_serves_every_smaller_call(lib):
    size = lib.lib().rq_q8_workspace_bytes
    for heads, d in ((1, 64), (5, 128), (8, 128), (32, 64)):
        s = _shape(batch=3, n_q_heads=2 * heads, n_kv_heads=2, head_dim=d, capacity=1 << 15)
        by_n = [size(ctypes.byref(s), n, 20000, 0, 0) for n in (1, 2, 3, 4, 5, 8, 9, 16, 17, 33, 64, 65, 200, 257, 1025, 4096)]
        assert by_n == sorted(by_n) and by_n[0] > 0
        by_ctx = [size(ctypes.byref(s), 3, c, 0, 0) for c in (0, 1, 64, 65, 1000, 8192, 1 << 15)]
        assert by_ctx == sorted(by_ctx)
        by_n = [size(ctypes.byref(s), n, 20000, 300, 9) for n in (1, 16, 17, 33, 64, 65, 200, 257, 1025, 4096)]
        assert by_n == sorted(by_n)
        by_ctx = [size(ctypes.byref(s), 2000, c, w, 64) for w in (0, 500) for c in (0, 1, 64, 65, 1000, 8192, 1 << 15)]
        assert by_ctx[:7] == sorted(by_ctx[:7]) and by_ctx[7:] == sorted(by_ctx[7:])


def test_reference_codes_are_the_nearest():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(2000) * 40, rng.standard_normal(2000) * 0.01, [448, -448, 460, 0, 2.0 ** -10, 3 * 2.0 ** -10]])
    every = np.sort(R.E4M3[np.isfinite(R.E4M3)])
    y = R.nearest(x, "e4m3")
    assert (np.abs(y - x) <= np.abs(every[None] - x[:, None]).min(1) + 1e-15).all()
    by = R.byte_of(y, "e4m3")
    assert (R.value_of(by, "e4m3") == y).all()
    assert R.nearest(np.array([2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0]), "e4m3").tolist() == [0, 2.0 ** -8, 16.0, 20.0]   # ties to even
    assert R.nearest(np.array([0.5, 1.5, 127.2, -300]), "int8").tolist() == [0, 2, 127, -127]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_reference_exponent_is_the_least(fmt):
    rng = np.random.default_rng(1)
    top = R.MOST[fmt]
    for a in [*np.exp(rng.uniform(-60, 60, 200)), top, 2 * top, top / 1024, 1.0]:
        e = R.exponent(a, fmt)
        a16 = float(R.bf16(a))
        assert a16 <= top * 2.0 ** e and (e == R.LEAST or a16 > top * 2.0 ** (e - 1))
    assert R.exponent(0.0, fmt) == R.LEAST
