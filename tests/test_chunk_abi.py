"""Refusals of the chunk and eviction entry points, and their sizes (no GPU needed)."""

import ctypes

import pytest

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from looped_transformer_kv_gb300 import build
    build.build()
    from looped_transformer_kv_gb300 import _lib
    return _lib


def _shape(**kw):
    from looped_transformer_kv_gb300 import rq
    a = dict(batch=2, n_q_heads=4, n_kv_heads=2, head_dim=128, n_loops=4, capacity=128, res_bits=(2, 2, 2))
    a.update(kw)
    return rq.make_shape(**a)


def _cache(lib, at=256):
    c = lib.RqCache()
    c.data = at
    c.rot_signs[0] = c.rot_signs[1] = 16
    return c


P = ctypes.c_void_p(256)
BIG = 1 << 50


def _chunk(lib, shape=None, paging=None, paged=False, **kw):
    """Status of a call with dummy pointers: every one of these is refused before any use."""
    a = dict(cache=_cache(lib), q=P, qs=(8, 4, 1), loop=0, kv=P, ks=(1, 1, 1, 1, 1), n_lens=None, n=2,
             ctx=P, max_ctx=64, out=P, weights=None, window=0, ws=P, ws_bytes=BIG)
    a.update(kw)
    s = shape or _shape()
    qs = None if a["qs"] is None else (ctypes.c_int64 * 3)(*a["qs"])
    ks = None if a["ks"] is None else (ctypes.c_int64 * 5)(*a["ks"])
    c = None if a["cache"] is None else ctypes.byref(a["cache"])
    rest = (a["q"], qs, a["loop"], a["kv"], ks, a["n_lens"], a["n"], a["ctx"], a["max_ctx"], a["out"],
            a["weights"], a["window"], a["ws"], a["ws_bytes"], None)
    L = lib.lib()
    if paged:
        return L.rq_paged_chunk_attention(ctypes.byref(s), c, None if paging is None else ctypes.byref(paging), *rest)
    return L.rq_chunk_attention(ctypes.byref(s), c, *rest)


@pytest.mark.parametrize("kw,status", [
    (dict(cache=None), INVALID), (dict(q=None), INVALID), (dict(qs=None), INVALID),
    (dict(kv=None), INVALID), (dict(ks=None), INVALID), (dict(ctx=None), INVALID),
    (dict(out=None), INVALID), (dict(loop=-1), INVALID), (dict(loop=4), INVALID),
    (dict(n=-1), INVALID), (dict(max_ctx=-1), INVALID), (dict(max_ctx=129), INVALID),
    (dict(window=1), INVALID), (dict(weights=P), INVALID), (dict(weights=P, window=3), INVALID),
    (dict(weights=P, window=-1), INVALID), (dict(qs=(-1, 4, 1)), INVALID),
    (dict(ks=(1, 1, -1, 1, 1)), INVALID), (dict(qs=(1 << 62, 1 << 62, 1)), INVALID),
    (dict(n=1 << 30), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws_bytes=16), WORKSPACE),
    (dict(ws=ctypes.c_void_p(128)), WORKSPACE), (dict(n=0), OK), (dict(n=0, ws=None, ws_bytes=0), OK),
])
def test_chunk_refusals(lib, kw, status):
    assert _chunk(lib, **kw) == status


@pytest.mark.parametrize("bad,status", [
    (dict(head_dim=96), UNSUPPORTED), (dict(res_bits=(3, 2, 2)), UNSUPPORTED),
    (dict(n_q_heads=3), INVALID), (dict(capacity=100), INVALID),
])
def test_chunk_refuses_bad_shapes(lib, bad, status):
    assert _chunk(lib, shape=_shape(**bad)) == status
    assert lib.lib().rq_chunk_workspace_bytes(ctypes.byref(_shape(**bad)), 0, 1, 0, 0) == 0


@pytest.mark.parametrize("heads,n,status", [(1, 65535 * 256, OK), (1, 65535 * 256 + 1, UNSUPPORTED),
                                            (256, 65535, OK), (256, 65536, UNSUPPORTED)])
def test_most_rows_of_a_chunk(lib, heads, n, status):
    s = _shape(batch=1, n_kv_heads=1, n_q_heads=heads)
    size = lib.lib().rq_chunk_workspace_bytes(ctypes.byref(s), 0, n, 0, 0)
    assert (size > 0) == (status == OK)
    # (the call is refused either way: its workspace is too small)
    assert _chunk(lib, shape=s, n=n, max_ctx=0, ws_bytes=16) == (WORKSPACE if status == OK else status)


@pytest.mark.parametrize("apart", [0, 2, 2 * 2 * 4 * 128 * 2 - 2])
def test_chunk_output_over_its_inputs_is_refused(lib, apart):
    """Rows [2][2][4][128] each: out overlaps q, or kv_new, by at least one element."""
    at, far = (1 << 32), ctypes.c_void_p(1 << 40)
    strides = dict(qs=(2 * 4 * 128, 4 * 128, 128), ks=(0, 0, 0, 0, 0))
    for off in (apart, -apart):
        assert _chunk(lib, q=ctypes.c_void_p(at), kv=far, out=ctypes.c_void_p(at + off), **strides) == INVALID
    strides = dict(qs=(0, 0, 0), ks=(2 * 4 * 128, 4 * 128, 256, 0, 128))
    assert _chunk(lib, q=far, kv=ctypes.c_void_p(at), out=ctypes.c_void_p(at + apart), **strides) == INVALID


def test_chunk_paging_is_validated(lib):
    assert _chunk(lib, paged=True) == INVALID
    g = lib.RqPaging()
    g.block_table, g.max_pages, g.n_pages = 16, 1, 8            # capacity is not 64 * max_pages
    assert _chunk(lib, paging=g, paged=True) == INVALID
    g.max_pages = 2
    assert _chunk(lib, paging=g, paged=True, n=0) == OK


def test_chunk_workspace(lib):
    f = lambda *a: lib.lib().rq_chunk_workspace_bytes(ctypes.byref(_shape(capacity=4096)), *a)  # noqa: E731
    assert f(0, 1, 64, 0) > 256
    for n in (1, 8, 9, 100, 1000):
        assert f(0, n, 4096, 0) <= f(0, n, 4096, 1) <= f(0, n, 4096, n)
    for bad in ((-1, 1, 0, 0), (4, 1, 0, 0), (0, -1, 0, 0), (0, 1, 4097, 0), (0, 1, 0, 2)):
        assert f(*bad) == 0


def _select(lib, **kw):
    a = dict(w=P, B=2, H=2, cap=100, ctx=P, budget=10, first=2, last=3, keep=P, kept=P)
    a.update(kw)
    return lib.lib().rq_evict_select(a["w"], a["B"], a["H"], a["cap"], a["ctx"], a["budget"], a["first"],
                                     a["last"], a["keep"], a["kept"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), INVALID), (dict(ctx=None), INVALID), (dict(keep=None), INVALID),
    (dict(kept=None), INVALID), (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(cap=0), INVALID),
    (dict(budget=0), INVALID), (dict(first=-1), INVALID), (dict(last=-1), INVALID),
    (dict(first=8), INVALID), (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), INVALID),
    (dict(B=1 << 20, H=1 << 10), UNSUPPORTED), (dict(cap=2 ** 31 - 1), UNSUPPORTED),
    (dict(kept=P), INVALID), (dict(kept=ctypes.c_void_p(256 + 4)), INVALID),
])
def test_select_refusals(lib, kw, status):
    assert _select(lib, **kw) == status


def _compact(lib, paged=False, **kw):
    a = dict(s=_shape(), c=_cache(lib), ts=_shape(capacity=64), t=_cache(lib, 1 << 40), keep=P, budget=10,
             kept=P, w=None, tw=None, g=None, tg=None)
    a.update(kw)
    ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    tail = (a["keep"], a["budget"], a["kept"], a["w"], a["tw"], None)
    if paged:
        return lib.lib().rq_paged_evict_compact(ref(a["s"]), ref(a["c"]), ref(a["g"]), ref(a["ts"]),
                                                ref(a["t"]), ref(a["tg"]), *tail)
    return lib.lib().rq_evict_compact(ref(a["s"]), ref(a["c"]), ref(a["ts"]), ref(a["t"]), *tail)


@pytest.mark.parametrize("kw", [
    dict(keep=None), dict(kept=None), dict(budget=0), dict(ts=None), dict(t=None), dict(c=None),
    dict(w=P), dict(tw=P), "batch", "heads", "dim", "loops", "bits", "overlap", "weights overlap",
    "weights apart in place",
])
def test_compact_refusals(lib, kw):
    if isinstance(kw, str):
        kw = {
            "batch": dict(ts=_shape(batch=3)), "heads": dict(ts=_shape(n_kv_heads=4)),
            "dim": dict(ts=_shape(head_dim=64)), "loops": dict(ts=_shape(n_loops=3)),
            "bits": dict(ts=_shape(res_bits=(2, 4, 2))), "overlap": dict(t=_cache(lib, 256 + 4096)),
            "weights overlap": dict(w=P, tw=ctypes.c_void_p(256 + 64)),
            "weights apart in place": dict(ts=_shape(), t=_cache(lib), w=P, tw=ctypes.c_void_p(1 << 40)),
        }[kw]
    assert _compact(lib, **kw) == INVALID


def test_compact_paging_is_validated(lib):
    g = lib.RqPaging()
    g.block_table, g.max_pages, g.n_pages = 16, 2, 8
    assert _compact(lib, paged=True, g=g) == INVALID            # one of the two tables missing
    h = lib.RqPaging()
    h.block_table, h.max_pages, h.n_pages = 16, 2, 8            # to's capacity is one page
    assert _compact(lib, paged=True, g=g, tg=h) == INVALID


def test_compact_within_the_same_pages_under_another_plan_is_refused(lib):
    """One pool and one block table, but another capacity or page count: not in place, and the rows would
    move among the same pages unordered."""
    g = lib.RqPaging()
    g.block_table, g.max_pages, g.n_pages = 16, 2, 8
    h = lib.RqPaging()
    h.block_table, h.max_pages, h.n_pages = 16, 1, 8
    one = _cache(lib)
    for batch in (1, 2):
        s, ts = _shape(batch=batch), _shape(batch=batch, capacity=64)
        assert _compact(lib, paged=True, s=s, c=one, g=g, ts=ts, t=_cache(lib), tg=h) == INVALID
        assert _compact(lib, paged=True, s=ts, c=one, g=h, ts=s, t=_cache(lib), tg=g) == INVALID
        h2 = lib.RqPaging()
        h2.block_table, h2.max_pages, h2.n_pages = 16, 2, 9
        assert _compact(lib, paged=True, s=s, c=one, g=g, ts=s, t=_cache(lib), tg=h2) == INVALID


def _fits(lib, shape, loop, n, max_ctx, window, ws_bytes):
    """Would a call take this workspace?  (Its output lies over its queries, which is refused after the
    workspace was looked at: nothing is ever enqueued.)"""
    d, g = shape.head_dim, shape.n_q_heads
    status = _chunk(lib, shape=shape, loop=loop, n=n, max_ctx=max_ctx, window=window,
                    weights=P if window else None, qs=(n * g * d, g * d, d), ks=(0, 0, 0, 0, 0),
                    kv=ctypes.c_void_p(1 << 44), ws_bytes=ws_bytes)
    assert status in (INVALID, WORKSPACE)
    return status == INVALID


@pytest.mark.parametrize("seed", range(6))
def test_chunk_workspace_serves_every_smaller_call(lib, seed):
    """One workspace, made for the longest chunk, context and window, is enough for any shorter."""
    import random
    rng = random.Random(seed)
    for _ in range(40):
        H, heads, d = rng.choice([1, 2, 8, 16]), rng.choice([1, 1, 2, 4, 8, 16, 33, 128]), rng.choice([64, 128])
        bits = [rng.choice([2, 4]) for _ in range(rng.randint(0, 3))]
        s = _shape(batch=rng.choice([1, 2, 16, 300]), n_q_heads=H * heads, n_kv_heads=H, head_dim=d,
                   n_loops=len(bits) + 1, res_bits=bits, capacity=64 * rng.choice([2, 40, 512, 4096]))
        n = int(2 ** rng.uniform(0, 12))
        ctx = rng.choice([0, s.capacity, rng.randint(0, s.capacity)])
        w = rng.choice([0, 1, n, rng.randint(0, n)])
        loop = rng.randint(0, len(bits))
        size = lib.lib().rq_chunk_workspace_bytes(ctypes.byref(s), loop, n, ctx, w)
        assert size > 0 and _fits(lib, s, loop, n, ctx, w, size)
        for _ in range(40):
            n1 = rng.choice([1, n, rng.randint(1, n), min(n, max(1, 8 // heads)), min(n, max(1, 128 // heads))])
            ctx1 = rng.choice([0, ctx, rng.randint(0, ctx), min(ctx, n1 * 32), max(0, min(ctx, n1 * 32) - 1)])
            w1 = rng.choice([0, min(w, n1), rng.randint(0, min(w, n1))])
            assert _fits(lib, s, loop, n1, ctx1, w1, size), (n, ctx, w, n1, ctx1, w1, H, heads, d, s.batch)


def test_chunk_workspace_for_the_capacity_serves_every_context(lib):
    s = _shape(batch=1, n_q_heads=16, n_kv_heads=16, capacity=32768)
    for n in (1, 8, 64):
        size = lib.lib().rq_chunk_workspace_bytes(ctypes.byref(s), 0, n, 32768, 0)
        for ctx in range(0, 32769, 64):
            assert _fits(lib, s, 0, n, ctx, 0, size)
