"""Chunk attention where its kernels meet: calls in a row, schedules of ragged batches, groups of
sequences, the ends of the states' range, on the GPU."""

import itertools

import numpy as np
import pytest

import chunk_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from looped_transformer_kv_gb300 import rq  # noqa: F401
    from test_gpu_chunk import Case, HALF16, HALFB


def test_window_calls_back_to_back():
    """Calls of every path on two streams, each CTA followed at once by another's: the first one's
    bits each time (a CTA leaves nothing in flight)."""
    cases = [Case(2, 8, 2, 128, (2,), [400, 333], 70, window=5), Case(1, 8, 2, 64, (4,), [500], 90, window=90),
             Case(2, 8, 2, 128, (2, 4), [129, 700], 8, [8, 3]), Case(1, 4, 2, 128, (2,), [300], 3, window=3)]
    want = []
    for c in cases:
        c.call()
        torch.cuda.synchronize()
        c.check()
        want.append((c.out.clone(), None if c.weights is None else c.weights.clone()))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for i, c in enumerate(cases):
            if c.weights is not None:
                c.weights.copy_(c.w0)
        torch.cuda.synchronize()
        for i, c in enumerate(cases):
            c.call(stream=streams[i % 2])
        torch.cuda.synchronize()
        for c, (out, weights) in zip(cases, want):
            assert c.error_word() == 0
            assert torch.equal(c.out.view(torch.int16), out.view(torch.int16))
            assert weights is None or torch.equal(c.weights, weights)


@pytest.mark.parametrize("B,Hq,H,d,n_new,max_ctx,ctx,lens", [
    (1, 32, 8, 128, 2048, 4096, [1450], [5]),
    (1, 16, 2, 128, 2048, 16384, [4000], [1]),
    (2, 32, 4, 64, 2048, 4096, [1400, 900], [3, 0]),
    (3, 16, 4, 128, 2048, 4096, [0, 2222, 129], [0, 40, 17]),
    (4, 32, 2, 128, 1024, 4096, [3000, 1, 0, 700], [1, 0, 700, 0]),
])
def test_short_tail_in_a_call_planned_for_long_chunks(B, Hq, H, d, n_new, max_ctx, ctx, lens):
    """Most row blocks of the plan have no rows: fewer key tiles than the CTAs that share them.  What
    the workspace held before does not matter."""
    c = Case(B, Hq, H, d, (2,), ctx, n_new, lens, max_ctx=max_ctx, seed=7)
    c.call()
    torch.cuda.synchronize()
    c.check()
    out = c.out.clone()
    for fill in (0x3F, 0x00, 0x48):                 # finite as fp32, fp16 and counts
        c.ws.fill_(fill)
        c.out.fill_(776.0)
        c.call()
        torch.cuda.synchronize()
        assert c.error_word() == 0 and torch.equal(c.out.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("fault", [None, "ctx", "negative", "n_len", "page"])
def test_fault_of_a_later_group_makes_every_output_nan(fault):
    """Operand images of one sequence take more than 2 GB (max_ctx 640,000, of which little is used),
    so each sequence is a group of its own; the last one's lengths or pages are wrong."""
    B, Hq, H, d, n, pages = 3, 32, 8, 128, 40, 10000
    g = torch.Generator().manual_seed(3)
    shape = rq.make_shape(B, Hq, H, d, 2, 64 * pages, (2,))
    table = torch.full((B, pages), -1, dtype=torch.int32)
    table[:, :3] = torch.arange(9).view(3, 3)
    ctx = torch.tensor([100, 0, 129], dtype=torch.int32)
    lens = torch.tensor([n, 7, n], dtype=torch.int32)
    if fault == "ctx":
        ctx[2] = 64 * pages - n + 1
    elif fault == "negative":
        ctx[2] = -1
    elif fault == "n_len":
        lens[2] = n + 1
    elif fault == "page":
        table[2, 2] = 9
    table = table.cuda()
    signs = torch.ones(2, H, d)
    cache = rq.PackedCache(shape, signs, n_pages=9)
    new = torch.randn(B, n, 2, 2, H, d, generator=g).bfloat16().cuda()
    paging = rq.make_paging(table, 9)
    good = table.clone()
    good[2, 2] = 8
    states = torch.randn(B, 192, 2, 2, H, d, generator=g).bfloat16().cuda()
    rq.paged_encode_append(shape, cache, rq.make_paging(good, 9), states)
    q = torch.randn(B, n, Hq, d, generator=g).bfloat16().cuda()
    out = torch.full_like(q, 776.0)
    need = rq.chunk_workspace_bytes(shape, 0, n, 64 * pages - n)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    rq.paged_chunk_attention(shape, cache, paging, q, 0, new, ctx.cuda(), 64 * pages - n, out, ws, n_lens=lens.cuda())
    torch.cuda.synchronize()
    word = int(ws[:4].view(torch.int32).item())
    if fault is None:
        assert word == 0 and torch.isfinite(out.float()).all()
    else:
        assert word != 0
        assert out[0].isnan().all() and out[1, :7].isnan().all() and out[2].isnan().all()
    assert (out[1, 7:] == 776.0).all()


# fp16 resolves 2^-24 below 2^-14: half a step, 2^-25, is what a rounding of a cached element costs at
# least.  The cache's own steps and offsets are stored with that resolution.
FLOOR16 = 2.0 ** -25


def scaled_case(cached, own, B, Hq, H, d, bits, ctx, n_new, lens=None, **kw):
    """Case with the cached states times `cached` and the chunk's times `own`."""
    c = Case(B, Hq, H, d, bits, ctx, n_new, lens, **kw)
    g = torch.Generator().manual_seed(11)
    L = len(bits) + 1
    x = torch.randn(B, max(ctx + [1]), 2, 1, H, d, generator=g)
    x = (x + 0.1 * torch.randn(*x.shape[:3], L, H, d, generator=g)) * cached
    for b in range(B):
        if ctx[b]:
            pos = torch.full((B, ctx[b]), -1, dtype=torch.int32)
            pos[b] = torch.arange(ctx[b])
            src = x[:, :ctx[b]].bfloat16().cuda()
            if c.paging is not None:
                rq.paged_encode_append(c.shape, c.cache, c.paging, src, positions=pos.cuda())
            else:
                rq.encode_append(c.shape, c.cache, src, positions=pos.cuda())
    c.new_host = (c.new_host.float() * own).bfloat16()
    c.new.copy_(c.new_host)
    return c


def check_small(c, least_weight=0.0, least_new=0.0):
    """Case.check, in which the roundings of cached elements cost at least FLOOR16: two of a reference
    element (times a, below 2), one of a residual level and thus sqrt(d) of a channel, one of a rebuilt
    element; that of a softmax weight least_weight of the row's largest, of an element beside larger ones
    least_new of the largest."""
    assert c.error_word() == 0
    G, d = c.Hq // c.H, c.d
    out = c.out.double().cpu().numpy()
    least = FLOOR16 * (5 + d ** 0.5)
    for b, h in itertools.product(range(c.B), range(c.H)):
        m, ctx = c.lens[b], c.ctx[b]
        if m == 0:
            continue
        ref, p, mag, v = c.reference(b, h)
        got = out[b, :m, h * G:(h + 1) * G]
        rec = c.records(b, h)
        rk, rv = (np.concatenate([R.residual_norms(rec, ctx, d, c.bits, c.loop, kv), np.zeros(m)]) for kv in (0, 1))
        q = c.q_host[b, :m, h * G:(h + 1) * G].double().numpy()
        e = HALF16 * (2 * mag + 4 * np.linalg.norm(q, axis=-1) * rk.max() * d ** -0.5)[..., None]
        e += (np.abs(q).sum(-1) * least * d ** -0.5)[..., None] * (ctx > 0)
        k = np.concatenate([R.rebuild(rec, ctx, d, c.bits, c.loop, 0, c.signs[0, h].numpy()),
                            c.new_host[b, :m, 0, c.loop, h].double().numpy()])
        e += (np.abs(q).sum(-1) * least_new * np.abs(k).max() * d ** -0.5)[..., None]
        pv = np.einsum("jgt,td->jgd", p, np.abs(v)) + least_new / HALF16 * np.abs(v).max()
        tol = pv * (np.expm1(2 * e) + 3 * HALF16 + 1e-5) + 3 * HALF16 * (p @ rv)[..., None]
        tol += (least_weight * p.max(-1))[..., None] * np.maximum(np.abs(v), 1).sum(0)
        tol += p[..., :ctx].sum(-1)[..., None] * least + HALFB * np.abs(ref) * 1.01 + 1e-38
        worst = (np.abs(got - ref) / tol).max()
        assert worst <= 1, (b, h, worst)


SMALL_STATES = [
    # B, Hq, H, d, bits, loop, ctx, n_new, lens: 8 rows and fewer; 9 to 128
    (2, 4, 2, 128, (2,), 0, [3, 200], 2, [2, 1]),
    (1, 8, 1, 64, (4, 2), 0, [70], 1, None),
    (2, 4, 1, 128, (2, 4), 0, [1, 130], 9, None),
    (1, 8, 1, 128, (4,), 0, [2], 8, None),
    (1, 16, 1, 64, (2,), 0, [5], 4, None),
    (2, 10, 2, 128, (2,), 1, [4, 65], 3, [3, 1]),
]


@pytest.mark.parametrize("scale", [1e-2, 1e-3, 1e-4, 1e-5])
@pytest.mark.parametrize("case", range(len(SMALL_STATES)))
def test_small_states(case, scale):
    B, Hq, H, d, bits, loop, ctx, n, lens = SMALL_STATES[case]
    c = scaled_case(scale, scale, B, Hq, H, d, bits, ctx, n, lens, loop=loop, paged=case % 2 == 0)
    c.call()
    torch.cuda.synchronize()
    check_small(c)
    if scale >= 1e-3:
        c.check()                                    # (one rounding relative to the states)


# A weight below 2^-14 has steps of 2^-24, and a row's largest lies at 2^7 at least (the maximum that
# weights refer to lags by up to 2^8 above that): half a step is 2^-32 of it.  With 8 rows and fewer the
# decode kernel multiplies codes (to 15 of the reference, to 15 of a residual, its rotation sqrt(d) of
# them) by fp16 pairs of weight x a x step, the largest weight at 2^0 at least: half a step is 2^-25 of a
# unit of the code.
LEAST_WEIGHT = 2.0 ** -32


@pytest.mark.parametrize("Hq,H,d,bits,n_new", [
    (4, 1, 128, (2,), 1), (2, 2, 64, (4,), 3),                     # 8 rows and fewer
    (8, 2, 128, (2,), 3), (4, 1, 64, (4, 2), 4), (8, 2, 128, (), 8),   # to 128
    (8, 2, 128, (2,), 40), (20, 4, 64, (4, 2), 40), (4, 1, 128, (), 70),   # more
])
def test_weights_far_below_the_largest(Hq, H, d, bits, n_new):
    """A first token that takes nearly all of the weight (the others: about 2^-29 of its own each) and
    whose value is zero: the output is what the small weights add up to."""
    B, ctx = 2, 64
    c = Case(B, Hq, H, d, bits, [ctx] * B, n_new, seed=d + n_new)
    g = torch.Generator().manual_seed(n_new)
    L = len(bits) + 1
    x = torch.randn(B, ctx, 2, 1, H, d, generator=g).expand(-1, -1, -1, L, -1, -1).clone()
    x += 0.1 * torch.randn(x.shape, generator=g)
    u = torch.randint(0, 2, (d,), generator=g) * 2.0 - 1
    x[:, :, 1] += 1
    x[:, 0, 0] = 40 / d ** 0.5 * u
    x[:, 0, 1] = 0
    rq.encode_append(c.shape, c.cache, x.bfloat16().cuda())
    c.q_host = (0.5 * u + 0.5 * torch.randn(c.q_host.shape, generator=g)).bfloat16()
    c.q.copy_(c.q_host)
    c.call()
    torch.cuda.synchronize()
    _, p, _, _ = c.reference(0, 0)
    assert np.median(p[..., 1:ctx]) < 2.0 ** -26 and np.median(p[..., 0]) > 0.999
    check_small(c, LEAST_WEIGHT if n_new * Hq // H > 8 else FLOOR16 * 15 * (1 + d ** 0.5))


SMALL_MANY = [
    # B, Hq, H, d, bits, loop, ctx, n_new, lens
    (1, 2, 2, 128, (2,), 0, [0], 200, None),
    (2, 8, 2, 128, (4, 2), 0, [0, 70], 40, [40, 33]),
    (1, 10, 2, 64, (2,), 1, [3], 65, None),
    (2, 4, 2, 64, (4,), 0, [0, 129], 129, [7, 129]),
]


# A tile's operands carry a power of two that takes its largest element to 2^-1 or more: half a step,
# 2^-25, is 2^-24 of it.
LEAST_NEW = 2.0 ** -24


@pytest.mark.parametrize("window", [0, 3])
@pytest.mark.parametrize("cached,own", [(1e-3, 1e-3), (1e-5, 1e-5), (1, 1e-5), (1e-3, 2e-8), (1e-4, 1e-20),
                                        (1e-20, 1e-12), (1, 6000)])
@pytest.mark.parametrize("case", range(len(SMALL_MANY)))
def test_many_rows_of_states_of_any_size(case, cached, own, window):
    """New states of any size that their bf16 has (6000: the largest near 25,000) keep one rounding of
    2^-11, or LEAST_NEW of the largest."""
    B, Hq, H, d, bits, loop, ctx, n, lens = SMALL_MANY[case]
    c = scaled_case(cached, own, B, Hq, H, d, bits, ctx, n, lens, loop=loop, window=window, paged=case % 2 == 1)
    if own > 1:
        c.q_host = (c.q_host.float() / 4000).bfloat16()       # (scores of a softmax still)
        c.q.copy_(c.q_host)
    c.call()
    torch.cuda.synchronize()
    check_small(c, least_new=LEAST_NEW)
    if window:
        c.check_weights()


@pytest.mark.parametrize("ctx", [0, 70])
@pytest.mark.parametrize("value", [float("nan"), float("-inf"), 7e4])
def test_token_out_of_range_among_small_states(ctx, value):
    """Its magnitude does not count for the tile's power of two: the rows before it keep their bits."""
    args = (1e-3, 1e-5, 1, 4, 2, 128, (2,), [ctx], 200)
    c, clean, at = scaled_case(*args), scaled_case(*args), 37
    for kv in (0, 1):
        c.new[0, at + 90 * kv, kv, 0, kv, 5 + kv] = value
    c.call()
    clean.call()
    torch.cuda.synchronize()
    assert c.error_word() == 0
    assert c.out[0, at:, :2].isnan().all() and c.out[0, at + 90:, 2:].isnan().all()
    c.out[0, at:, :2] = clean.out[0, at:, :2]
    c.out[0, at + 90:, 2:] = clean.out[0, at + 90:, 2:]
    check_small(c, least_new=LEAST_NEW)


def takes(c, size):
    """Would the call take a workspace of this size?  (Asked with the output over the queries, which is
    refused after the workspace: nothing runs.)"""
    with pytest.raises(rq._lib.RqError) as e:
        args = (c.q, c.loop, c.new, c.ctx_lens, c.max_ctx, c.q, c.ws[:size])
        kw = dict(n_lens=c.n_lens, weights=c.weights, window=c.window)
        if c.paging is not None:
            rq.paged_chunk_attention(c.shape, c.cache, c.paging, *args, **kw)
        else:
            rq.chunk_attention(c.shape, c.cache, *args, **kw)
    assert e.value.status in (1, 3)
    return e.value.status == 1


@pytest.mark.parametrize("B,Hq,H,d,bits,ctx,n_new,lens,window", [
    (1, 4, 2, 128, (2,), [5000], 2, None, 0),                 # the cache streamed, one split
    (2, 4, 2, 64, (4,), [3000, 70], 2, [1, 2], 2),
    (2, 8, 1, 128, (2,), [4000, 129], 4, [4, 3], 0),          # fused; streamed with a short workspace
    (1, 2, 1, 128, (2, 4), [5000], 64, None, 0),              # fused; tiles with a short workspace
    (3, 4, 2, 128, (2,), [300, 70, 0], 100, [100, 7, 64], 0),   # tiles, groups of fewer sequences
    (3, 12, 2, 64, (2,), [1000, 0, 129], 40, [40, 1, 33], 7),
    (1, 32, 2, 128, (2,), [4096], 2048, [300], 0),            # key tiles shared evenly; one CTA a block
])
def test_any_workspace_that_is_taken_does(B, Hq, H, d, bits, ctx, n_new, lens, window):
    c = Case(B, Hq, H, d, bits, ctx, n_new, lens, window=window, seed=5, paged=B == 2)
    most = c.ws.numel()
    low, high = 0, most                                       # refused, taken
    assert takes(c, high)
    while high - low > 1:
        mid = (low + high) // 2
        low, high = (low, mid) if takes(c, mid) else (mid, high)
    whole = c.ws
    for size in sorted({high, (high + most) // 2, max(high, most - 1), most}):
        whole.fill_(255)
        c.ws = whole[:size]
        c.out.fill_(776.0)
        if c.weights is not None:
            c.weights.copy_(c.w0)
        c.call()
        torch.cuda.synchronize()
        c.check()
        assert (whole[size:] == 255).all()


@pytest.mark.parametrize("n_new,ctxs", [(1, [[8000], [3000], [1]]), (64, [[1984], [4000], [2048], [0]])])
def test_workspace_for_the_capacity(n_new, ctxs):
    """One workspace for calls of every context, and of fewer tokens."""
    big = None
    for ctx in ctxs:
        for n in sorted({1, n_new}):
            c = Case(1, 2, 1, 128, (2,), ctx, n, cap=32768 + 64)
            if big is None:
                big = torch.empty(rq.chunk_workspace_bytes(c.shape, 0, n_new, 32768), dtype=torch.uint8, device="cuda")
            c.ws = big.fill_(255)
            c.call()
            torch.cuda.synchronize()
            c.check()
