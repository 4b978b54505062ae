"""The binding of the 8-bit cache refuses a shape or a paging that does not fit the cache (no GPU: the refusals
come before the library is called)."""

import pytest

torch = pytest.importorskip("torch")

SHAPE = dict(batch=2, n_q_heads=4, n_kv_heads=2, head_dim=64, n_loops=2, capacity=128, fmt="int8")


@pytest.fixture(scope="module")
def rq():
    from looped_transformer_kv_gb300 import build
    build.build()
    import looped_transformer_kv_gb300
    return looped_transformer_kv_gb300


class Called(Exception):
    """The checks were passed."""


def _call(rq, monkeypatch, what, cache, paging=None, **other):
    a = dict(SHAPE) | other
    shape = rq.make_q8_shape(**a)
    B, H, d, L = a["batch"], a["n_kv_heads"], a["head_dim"], a["n_loops"]
    ctx = torch.zeros(B, dtype=torch.int32)

    def device():
        raise Called

    monkeypatch.setattr(torch._C, "_cuda_getDevice", device, raising=False)
    paged = [] if paging is None else [paging]
    if what == "append":
        f = rq.q8_append if paging is None else rq.paged_q8_append
        f(shape, cache, *paged, torch.zeros(B, 1, 2, L, H, d, dtype=torch.bfloat16), 0, ctx)
    else:
        q = torch.zeros(B, 1, a["n_q_heads"], d, dtype=torch.bfloat16)
        f = rq.q8_attention if paging is None else rq.paged_q8_attention
        f(shape, cache, *paged, q, 0, ctx, 5, torch.empty_like(q), torch.empty(1 << 16, dtype=torch.uint8))


def _table(B=2, pages=2):
    return torch.zeros(B, pages, dtype=torch.int32)


@pytest.mark.parametrize("what", ["append", "attention"])
def test_shapes_that_do_not_fit(rq, monkeypatch, what):
    cache = rq.Q8Cache(rq.make_q8_shape(**SHAPE), device="cpu")
    for other in (dict(batch=3), dict(n_kv_heads=1), dict(n_kv_heads=4), dict(head_dim=128), dict(n_loops=3), dict(n_loops=1),
                  dict(capacity=192), dict(capacity=64), dict(fmt="e4m3")):
        with pytest.raises(AssertionError):
            _call(rq, monkeypatch, what, cache, **other)
    for other in (dict(), dict(n_q_heads=8), dict(batch=1), dict(softmax_scale=0.5)):
        with pytest.raises(Called):
            _call(rq, monkeypatch, what, cache, **other)


@pytest.mark.parametrize("what", ["append", "attention"])
def test_pagings_that_do_not_fit(rq, monkeypatch, what):
    shape = rq.make_q8_shape(**SHAPE)
    pool, plain = rq.Q8Cache(shape, device="cpu", n_pages=5), rq.Q8Cache(shape, device="cpu")
    for cache, paging, other in ((pool, None, {}), (plain, rq.make_paging(_table(), 4), {}), (pool, rq.make_paging(_table(), 6), {}),
                                 (pool, rq.make_paging(_table(1), 5), {}), (pool, rq.make_paging(_table(), 5), dict(n_loops=1)),
                                 (pool, rq.make_paging(_table(), 5), dict(head_dim=128)), (pool, rq.make_paging(_table(), 5), dict(fmt="e4m3"))):
        with pytest.raises(AssertionError):
            _call(rq, monkeypatch, what, cache, paging, **other)
    # a pool serves other batches and lengths than it was made with
    for paging, other in ((rq.make_paging(_table(), 5), {}), (rq.make_paging(_table(), 3), {}),
                          (rq.make_paging(_table(7, 40), 5), dict(batch=7, capacity=40 * 64))):
        with pytest.raises(Called):
            _call(rq, monkeypatch, what, pool, paging, **other)


def test_the_cache_goes_by_the_shape_it_was_made_with(rq, monkeypatch):
    shape = rq.make_q8_shape(**SHAPE)
    cache = rq.Q8Cache(shape, device="cpu")
    shape.capacity = 1 << 20
    with pytest.raises(AssertionError):
        _call(rq, monkeypatch, "append", cache, capacity=1 << 20)
