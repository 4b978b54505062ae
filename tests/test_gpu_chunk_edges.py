"""Chunk attention where its kernels meet: calls in a row, schedules of ragged batches, groups of
sequences, the ends of the states' range, on the GPU."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from looped_transformer_kv_gb300 import rq  # noqa: F401
    from test_gpu_chunk import Case


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
