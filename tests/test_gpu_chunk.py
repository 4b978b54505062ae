"""Chunk attention over the packed cache against the 64-bit reference, on the GPU."""

import itertools

import numpy as np
import pytest

import chunk_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from looped_transformer_kv_gb300 import rq

# A score or output of the kernels differs from the 64-bit one by roundings only.  With more than 8
# rows the operands are fp16, one rounding half a step, 2^-11: a residual level r once, a rebuilt
# element or reference level at most twice, a rotated query once, a softmax weight once; the sums are
# fp32.  The rotation keeps norms and a ref = K - R^T r, so a score is off by at most
#   e = 2^-11 scale (2 sum|q k| + 4 |q| |r|)
# and a V element by 2^-11 (2 |v| + 3 |r|).  A weight is then within a factor exp(2 e) of its own and
# an output off by at most sum p|v| (exp(2 e) - 1 + 3 * 2^-11) + 3 * 2^-11 sum p |r_v|, and by half a
# bf16 step (2^-8 relative) of its result.  fp32 steps in sums of up to a few thousand terms stay
# below 1e-5 of sum p|v|.
HALF16, HALFB = 2.0 ** -11, 2.0 ** -8
# Collected weights come from scores in which each product carries at least 21 bits (two fp16
# parts) and fp32 sums of d terms: e = (2^-21 + d 2^-24) sum|q k| scale; twice that in a weight,
# fp32 exponentials and sums (1e-5 relative covers 64 additions and exp2's last bits).
W_PRODUCT = 2.0 ** -21


class Case:
    """A cache of encoded states, a chunk, and the reference results."""

    def __init__(self, B, Hq, H, d, bits, ctx, n_new, n_lens=None, window=0, seed=0, loop=0,
                 paged=False, cap=None, max_ctx=None, spread=False):
        g = torch.Generator().manual_seed(seed)
        self.B, self.Hq, self.H, self.d, self.bits, self.loop = B, Hq, H, d, tuple(bits), loop
        self.ctx, self.n_new, self.window = list(ctx), n_new, window
        self.lens = list(n_lens) if n_lens is not None else [n_new] * B
        L = len(bits) + 1
        self.max_ctx = max(self.ctx) if max_ctx is None else max_ctx
        self.cap = cap or -(-(max(self.ctx + [self.max_ctx]) + n_new) // 64) * 64
        self.signs = torch.randint(0, 2, (2, H, d), generator=g) * 2 - 1
        self.shape = rq.make_shape(B, Hq, H, d, L, self.cap, bits)
        base = torch.randn(B, self.cap, 2, 1, H, d, generator=g)
        base[..., 3] *= 8
        x = base * (0.8 + 0.4 * torch.rand(B, self.cap, 2, L, H, 1, generator=g))
        x += 0.1 * torch.randn(x.shape, generator=g)
        # slots behind the context hold NaN steps and offsets
        if paged:
            pages = self.cap // 64
            order = torch.randperm(B * pages + 3, generator=g)[:B * pages].int().view(B, pages)
            self.table = order.cuda()
            self.cache = rq.PackedCache(self.shape, self.signs, n_pages=B * pages + 3)
            self.paging = rq.make_paging(self.table, B * pages + 3)
        else:
            self.table, self.paging = None, None
            self.cache = rq.PackedCache(self.shape, self.signs)
        self.cache.data.fill_(255)
        kv = x.bfloat16().cuda()
        for b in range(B):
            if self.ctx[b] == 0:
                continue
            pos = torch.full((B, self.ctx[b]), -1, dtype=torch.int32)
            pos[b] = torch.arange(self.ctx[b])
            src = kv[:, :self.ctx[b]]
            if paged:
                rq.paged_encode_append(self.shape, self.cache, self.paging, src, positions=pos.cuda())
            else:
                rq.encode_append(self.shape, self.cache, src, positions=pos.cuda())
        new = torch.randn(B, n_new, 2, L, H, d, generator=g).bfloat16()
        q = torch.randn(B, n_new, Hq, d, generator=g).bfloat16()
        for b in range(B):      # behind a sequence's last token: NaN
            q[b, self.lens[b]:] = float("nan")
            new[b, self.lens[b]:] = float("nan")
        self.new_host, self.q_host = new, q
        if spread:              # strides of a fused projection's output, odd offsets
            buf = torch.full((B, n_new, 3 * Hq * d + 5), float("nan"), dtype=torch.bfloat16)
            self.q = buf.cuda()[:, :, 3:3 + Hq * d].view(B, n_new, Hq, d)
            self.q.copy_(q)
            wide = torch.full((B, n_new, 2, L, H, d + 1), float("nan"), dtype=torch.bfloat16)
            self.new = wide.cuda()[..., 1:]
            self.new.copy_(new)
        else:
            self.q, self.new = q.cuda(), new.cuda()
        self.ctx_lens = torch.tensor(self.ctx, dtype=torch.int32).cuda()
        self.n_lens = None if n_lens is None else torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.w0 = torch.rand(B, H, self.cap, generator=g)
        self.weights = self.w0.cuda() if window else None
        self.out = torch.full((B, n_new, Hq, d), 776.0, dtype=torch.bfloat16).cuda()
        need = rq.chunk_workspace_bytes(self.shape, loop, n_new, self.max_ctx, window)
        assert need > 0
        self.ws = torch.full((need,), 255, dtype=torch.uint8).cuda()

    def call(self, stream=None):
        args = (self.q, self.loop, self.new, self.ctx_lens, self.max_ctx, self.out, self.ws)
        kw = dict(n_lens=self.n_lens, weights=self.weights, window=self.window, stream=stream)
        if self.paging is not None:
            rq.paged_chunk_attention(self.shape, self.cache, self.paging, *args, **kw)
        else:
            rq.chunk_attention(self.shape, self.cache, *args, **kw)

    def error_word(self):
        return int(self.ws[:4].view(torch.int32).item())

    def records(self, b, h):
        data = self.cache.records()
        return (data[self.table[b].long(), h] if self.paging is not None else data[b, h]).cpu().numpy()

    def reference(self, b, h):
        m, ctx, G, d = self.lens[b], self.ctx[b], self.Hq // self.H, self.d
        rec = self.records(b, h)
        k, v = (np.concatenate([
            R.rebuild(rec, ctx, d, self.bits, self.loop, kv, self.signs[kv, h].numpy()),
            self.new_host[b, :m, kv, self.loop, h].double().numpy()]) for kv in (0, 1))
        q = self.q_host[b, :m, h * G:(h + 1) * G].double().numpy()
        return (*R.attend(q, k, v, ctx, d ** -0.5), v)

    def check(self):
        assert self.error_word() == 0
        G, d = self.Hq // self.H, self.d
        out = self.out.float().cpu().numpy().astype(np.float64)
        for b, h in itertools.product(range(self.B), range(self.H)):
            m, ctx = self.lens[b], self.ctx[b]
            assert (out[b, m:, h * G:(h + 1) * G] == 776.0).all()      # left as they were
            if m == 0:
                continue
            ref, p, mag, v = self.reference(b, h)
            got = out[b, :m, h * G:(h + 1) * G]
            pv = np.einsum("jgt,td->jgd", p, np.abs(v))
            rec = self.records(b, h)
            rk, rv = (np.concatenate([R.residual_norms(rec, ctx, d, self.bits, self.loop, kv), np.zeros(m)])
                      for kv in (0, 1))
            qn = np.linalg.norm(self.q_host[b, :m, h * G:(h + 1) * G].double().numpy(), axis=-1)
            e = HALF16 * (2 * mag + 4 * qn * rk.max() * d ** -0.5)[..., None]
            tol = pv * (np.expm1(2 * e) + 3 * HALF16 + 1e-5) + 3 * HALF16 * (p @ rv)[..., None]
            tol += HALFB * np.abs(ref) * 1.01 + 1e-30
            worst = (np.abs(got - ref) / tol).max()
            assert worst <= 1, (b, h, worst)
        if self.weights is not None:
            self.check_weights()

    def check_weights(self):
        got = self.weights.cpu().double().numpy()
        for b, h in itertools.product(range(self.B), range(self.H)):
            m, ctx = self.lens[b], self.ctx[b]
            want, tol = self.w0[b, h].double().numpy().copy(), np.zeros(self.cap)
            if m:
                _, p, mag, _ = self.reference(b, h)
                e = (W_PRODUCT + self.d * 2.0 ** -24) * mag[..., None]
                keep = slice(max(0, m - self.window), m)
                n = min(ctx + m, self.cap)
                add = p[keep].sum((0, 1))[:n]
                tol[:n] = (p[keep] * (np.expm1(2 * e[keep]) + 1e-5)).sum((0, 1))[:n]
                want[:n] += add
            tol += 2.0 ** -24 * want
            worst = (np.abs(got[b, h] - want) / np.maximum(tol, 1e-38))
            assert (np.abs(got[b, h] - want) <= tol).all(), (b, h, worst.max(), worst.argmax())


SMALL = [
    # B, Hq, H, d, bits, loop, ctx, n_new, n_lens
    (1, 2, 2, 128, (2,), 0, [1], 1, None),
    (1, 2, 2, 128, (2,), 1, [0], 1, None),
    (2, 2, 2, 128, (2, 2), 1, [65, 0], 1, [1, 0]),
    (1, 2, 2, 64, (2, 2, 2), 1, [256], 3, None),
    (2, 4, 1, 128, (4, 2), 0, [129, 64], 2, [2, 1]),
    (2, 8, 2, 64, (4,), 0, [63, 300], 5, [5, 2]),
    (1, 10, 2, 128, (), 0, [200], 4, None),
    (3, 4, 2, 128, (2,) * 7, 6, [0, 127, 128], 4, [4, 3, 1]),
]


@pytest.mark.parametrize("window", [0, 1, 2])
@pytest.mark.parametrize("case", range(len(SMALL)))
def test_few_rows(case, window):
    B, Hq, H, d, bits, loop, ctx, n, lens = SMALL[case]
    c = Case(B, Hq, H, d, bits, ctx, n, lens, window=min(window, n), seed=case, loop=loop,
             paged=case % 2 == 1)
    c.call()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("spread", [False, True])
def test_strides_do_not_matter(spread):
    c = Case(2, 6, 2, 128, (2,), [70, 5], 3, [3, 2], window=3, spread=spread)
    c.call()
    torch.cuda.synchronize()
    c.check()


def test_step_equals_decode_attention_and_collects_all_its_weight():
    # one new token: the same attention as rq_decode_attention with the token pending
    c = Case(3, 4, 4, 128, (2, 4), [200, 64, 1], 1, window=1)
    c.weights.zero_()
    c.call()
    want = torch.empty(3, 4, 1, 128, dtype=torch.bfloat16, device="cuda")
    pend = c.new[:, 0, :, 0:1].contiguous()                        # [B][2][1][H][d]
    ws = torch.empty(rq.decode_workspace_bytes(c.shape, 1, c.max_ctx), dtype=torch.uint8, device="cuda")
    rq.decode_attention(c.shape, c.cache, c.q.transpose(1, 2).contiguous(), 0, 1, pend, c.ctx_lens,
                        c.max_ctx, want, ws)
    torch.cuda.synchronize()
    diff = (c.out.transpose(1, 2).float() - want.float()).abs()
    assert (diff <= 2.0 ** -7 * want.float().abs() + 1e-6).all()   # one bf16 step apart at most
    total = c.weights.sum(-1).cpu()
    assert ((total - 1).abs() < 1e-5).all()


def test_chunk_weight_beyond_the_capacity_is_dropped():
    c = Case(1, 2, 1, 128, (2,), [62], 4, window=4, cap=64)
    c.call()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("n_new", [4, 20, 80])
@pytest.mark.parametrize("kv", [0, 1])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 1e5])
def test_token_out_of_range_reaches_its_own_and_later_rows_only(n_new, kv, value):
    c = Case(2, 4, 2, 128, (2,), [70, 10], n_new, seed=3)
    at = n_new // 2
    c.new[1, at, kv, 0, 1, 17] = value
    c.call()
    torch.cuda.synchronize()
    assert c.error_word() == 0
    got = c.out.float().cpu().clone()
    assert got[1, at:, 2:].isnan().all()
    # (the reference knows the chunk without it)
    clean = Case(2, 4, 2, 128, (2,), [70, 10], n_new, seed=3)
    clean.call()
    torch.cuda.synchronize()
    c.out[1, at:, 2:] = clean.out[1, at:, 2:]
    clean.out.copy_(c.out)
    clean.check()


@pytest.mark.parametrize("n_new", [2, 20, 70])
@pytest.mark.parametrize("fault", ["ctx", "negative", "n_len", "page"])
def test_bad_device_values_set_the_error_word(n_new, fault):
    c = Case(2, 2, 2, 128, (2,), [70, 100], n_new, [n_new, 1], paged=fault == "page", max_ctx=100)
    if fault == "ctx":
        c.ctx_lens[0] = 101
    elif fault == "negative":
        c.ctx_lens[0] = -1
    elif fault == "n_len":
        c.n_lens[1] = n_new + 1
    else:
        c.table[0, 1] = c.paging.n_pages
    c.call()
    torch.cuda.synchronize()
    assert c.error_word() != 0
    assert c.out[0].float().isnan().all()
    if fault == "page":                       # the table mended: an ordinary call again
        c.table[0, 1] = 0
        c.call()
        torch.cuda.synchronize()
        assert c.error_word() == 0


@pytest.mark.parametrize("n_new", [3, 90])
def test_captured_call_replays_with_new_lengths_on_another_stream(n_new):
    c = Case(2, 4, 2, 128, (2,), [200, 90], n_new, window=2, max_ctx=200)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.call()
    torch.cuda.synchronize()
    c.check()
    graph = torch.cuda.CUDAGraph()
    c.weights.copy_(c.w0)
    with torch.cuda.graph(graph):
        c.call()
    again = torch.cuda.CUDAGraph()            # a second graph on the same workspace
    with torch.cuda.graph(again):
        c.call()
    for lens in ([200, 90], [17, 64]):
        c.ctx = lens
        c.ctx_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        for g in (graph, again):
            c.weights.copy_(c.w0)
            c.out.fill_(776.0)
            g.replay()
            torch.cuda.synchronize()
            c.check()


def test_same_call_twice_gives_the_same_bits():
    c = Case(2, 8, 2, 128, (2,), [400, 333], 70, window=5)
    c.call()
    torch.cuda.synchronize()
    o, w = c.out.clone(), c.weights.clone()
    c.weights.copy_(c.w0)
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(o.view(torch.int16), c.out.view(torch.int16)) and torch.equal(w, c.weights)


def test_nothing_new_enqueues_nothing():
    c = Case(1, 2, 2, 128, (2,), [70], 1)
    q = c.q[:, :0]
    rq.chunk_attention(c.shape, c.cache, q, 0, c.new[:, :0], c.ctx_lens, 70, c.out[:, :0], c.ws)


MIDDLE = [
    # B, Hq, H, d, bits, loop, ctx, n_new, n_lens
    (1, 2, 2, 128, (2,), 0, [64], 9, None),
    (2, 8, 2, 128, (2, 4), 0, [129, 1], 8, [8, 3]),
    (2, 8, 2, 128, (4, 2), 0, [63, 0], 9, [9, 0]),
    (1, 4, 1, 128, (2, 2), 2, [200], 32, None),
    (2, 6, 2, 64, (2,), 0, [65, 640], 11, [1, 11]),
    (1, 16, 1, 64, (4,), 0, [300], 3, None),
    (1, 8, 2, 64, (), 0, [127], 7, None),
    (1, 8, 1, 128, (2,), 0, [3000], 16, None),
    (3, 128, 1, 128, (4,), 0, [100, 192, 7], 1, None),
    (1, 1, 1, 128, (2,), 0, [4096], 128, None),
    (2, 4, 2, 64, (4,), 0, [2080, 70], 64, [63, 64]),
]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("case", range(len(MIDDLE)))
def test_middle_rows(case, paged):
    B, Hq, H, d, bits, loop, ctx, n, lens = MIDDLE[case]
    c = Case(B, Hq, H, d, bits, ctx, n, lens, seed=case, loop=loop, paged=paged, spread=case == 2)
    c.call()
    torch.cuda.synchronize()
    c.check()


MANY = [
    # B, Hq, H, d, bits, loop, ctx, n_new, n_lens
    (1, 2, 2, 128, (2,), 0, [0], 33, None),
    (1, 4, 1, 128, (2,), 1, [64], 40, None),
    (2, 4, 2, 128, (4, 2), 0, [129, 1], 65, [65, 64]),
    (2, 2, 1, 64, (2,), 0, [200, 0], 129, [129, 7]),
    (1, 5, 1, 64, (4,), 0, [70], 52, None),
    (1, 8, 1, 128, (2, 2), 1, [257], 127, None),
    (1, 1, 1, 128, (2,), 0, [383], 257, None),
    (2, 20, 4, 128, (4,), 0, [100, 127], 13, [13, 0]),
    (1, 2, 2, 128, (2,), 0, [2000], 64, None),
]


@pytest.mark.parametrize("window", [0, 1, 40])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_many_rows(case, window):
    B, Hq, H, d, bits, loop, ctx, n, lens = MANY[case]
    c = Case(B, Hq, H, d, bits, ctx, n, lens, window=min(window, n), seed=case, loop=loop,
             paged=case % 2 == 0)
    c.call()
    torch.cuda.synchronize()
    c.check()


def check_on_gpu(c, b, h, cached):
    """Case.check with the 64-bit attention on the GPU; returns the weights its window should add.
    cached: (k, v, norms of k's and v's residuals) of the cached tokens."""
    G, d, m, n0 = c.Hq // c.H, c.d, c.lens[b], c.ctx[b]
    assert (c.out[b, m:, h * G:(h + 1) * G] == 776.0).all()
    k, v = (torch.cat([cached[kv].cuda(), c.new_host[b, :m, kv, c.loop, h].double().cuda()]) for kv in (0, 1))
    rk, rv = (torch.cat([cached[2 + kv], torch.zeros(m).double()]).cuda() for kv in (0, 1))
    late = torch.arange(n0 + m, device="cuda").view(1, -1) > n0 + torch.arange(m, device="cuda").view(-1, 1)
    added = torch.zeros(n0 + m, dtype=torch.float64, device="cuda")
    for g in range(G):
        q = c.q[b, :m, h * G + g].double()
        s = (q @ k.T * d ** -0.5).masked_fill(late, -float("inf"))
        p = torch.softmax(s, -1)
        added += p[max(0, m - c.window):].sum(0)
        ref, got = p @ v, c.out[b, :m, h * G + g].double()
        # the bound of Case.check, its largest score error over all keys
        mag = (q.abs() @ k.abs().T * d ** -0.5).amax(-1, keepdim=True)
        e = HALF16 * (2 * mag + 4 * q.norm(dim=-1, keepdim=True) * rk.max() * d ** -0.5)
        tol = (p @ v.abs()) * (torch.expm1(2 * e) + 3 * HALF16 + 1e-5) + 3 * HALF16 * (p @ rv)[:, None]
        tol += HALFB * ref.abs() * 1.01 + 1e-30
        assert ((got - ref).abs() <= tol).all(), (b, h, g, ((got - ref).abs() / tol).max().item())
    return added


def cached_rows(rec, n, d, bits, h, signs):
    return ([torch.from_numpy(R.rebuild(rec, n, d, bits, 0, kv, signs[kv, h].numpy())) for kv in (0, 1)] +
            [torch.from_numpy(R.residual_norms(rec, n, d, bits, 0, kv)) for kv in (0, 1)])


LONG = [(128, 16, [0, 130], [4096, 3001]), (64, 12, [257, 1], [4000, 4096])]


@pytest.mark.parametrize("d,Hq,ctx,lens", LONG)
def test_long_chunks_shared_evenly(d, Hq, ctx, lens):
    """Enough key tiles that the CTAs share them evenly, across row blocks."""
    B, H = 2, 2
    c = Case(B, Hq, H, d, (2,), ctx, 4096, lens, seed=d, window=3)
    c.call()
    torch.cuda.synchronize()
    assert c.error_word() == 0
    G = Hq // H
    for b, h in itertools.product(range(B), range(H)):
        end = ctx[b] + lens[b]
        added = check_on_gpu(c, b, h, cached_rows(c.records(b, h), ctx[b], d, c.bits, h, c.signs))
        got = c.weights[b, h].double() - c.w0[b, h].double().cuda()
        # (weights: fp32 additions to values below 1, 2^-24 each, and the scores' 21 bits)
        assert (got[:end] - added).abs().max().item() <= 2.0 ** -23 + 3 * G * 2e-4 * added.max().item()
        assert (got[end:] == 0).all()
    o, w = c.out.clone(), c.weights.clone()
    c.weights.copy_(c.w0)
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(o.view(torch.int16), c.out.view(torch.int16)) and torch.equal(w, c.weights)


def test_long_chunk_with_bad_lengths_is_nan():
    c = Case(2, 16, 2, 128, (2,), [0, 130], 4096, [4096, 3001])
    c.ctx_lens[1] = 131                        # max_ctx + 1
    c.call()
    torch.cuda.synchronize()
    assert c.error_word() != 0
    assert torch.isnan(c.out[0]).all() and torch.isnan(c.out[1, :3001]).all()
    assert (c.out[1, 3001:] == 776.0).all()


@pytest.mark.parametrize("n_new", [4096, 20, 2])
def test_batch_without_new_tokens(n_new):
    c = Case(2, 16, 2, 128, (2,), [70, 130], n_new, [0, 0], window=2)
    c.call()
    torch.cuda.synchronize()
    assert c.error_word() == 0 and (c.out == 776.0).all() and torch.equal(c.weights.cpu(), c.w0)


@pytest.mark.parametrize("n_new", [2, 8, 40])
def test_cache_of_more_than_4_gigabytes(n_new):
    """330 sequences with the same cached rows.  40 tokens: their images, more than 4 GB too, are made
    in three groups, which meet at sequences 127 and 254."""
    B, Hq, H, d, cap = 330, 16, 4, 128, 16384
    g = torch.Generator().manual_seed(n_new)
    ctx = torch.randint(0, 700, (B,), generator=g).tolist()
    lens = torch.randint(0, n_new + 1, (B,), generator=g).tolist()
    sampled = (0, 126, 127, 253, 254, 329)
    for b, x in zip(sampled, (cap, 100, cap - 1, 700, 0, cap - 130)):
        ctx[b], lens[b] = min(x, cap - n_new), n_new - b % 2
    one = Case(1, Hq, H, d, (2,), [cap - n_new], n_new, seed=1)      # its records go to every sequence
    c = Case.__new__(Case)
    c.Hq, c.H, c.d, c.ctx, c.lens, c.loop, c.window = Hq, H, d, ctx, lens, 0, 0
    shape = rq.make_shape(B, Hq, H, d, 2, cap, (2,))
    cache = rq.PackedCache(shape, one.signs, data=one.cache.data.repeat(B))
    assert cache.data.numel() > 2 ** 32
    q = torch.randn(B, n_new, Hq, d, generator=g).bfloat16()
    c.new_host = torch.randn(B, n_new, 2, 2, H, d, generator=g).bfloat16()
    for b in range(B):
        q[b, lens[b]:] = float("nan")
        c.new_host[b, lens[b]:] = float("nan")
    c.q, c.out = q.cuda(), torch.full(q.shape, 776.0, dtype=torch.bfloat16).cuda()
    c.ws = torch.full((rq.chunk_workspace_bytes(shape, 0, n_new, cap - n_new),), 255, dtype=torch.uint8).cuda()
    rq.chunk_attention(shape, cache, c.q, 0, c.new_host.cuda(), torch.tensor(ctx, dtype=torch.int32).cuda(),
                       cap - n_new, c.out, c.ws, n_lens=torch.tensor(lens, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert c.error_word() == 0
    for h in range(H):
        k, v, rk, rv = cached_rows(one.records(0, h), cap - n_new, d, (2,), h, one.signs)
        for b in sampled:
            check_on_gpu(c, b, h, (k[:ctx[b]], v[:ctx[b]], rk[:ctx[b]], rv[:ctx[b]]))
    out = c.out.float()
    for b in range(B):
        assert torch.isfinite(out[b, :lens[b]]).all() and (out[b, lens[b]:] == 776.0).all()


@pytest.mark.parametrize("n_new", [2, 20, 90])
def test_broadcast_inputs(n_new):
    """Strides of 0: one query for all heads, the same new states for all kv-heads and sequences."""
    c = Case(2, 4, 2, 128, (2,), [100, 300], n_new, window=1 if n_new == 90 else 0)
    c.q = c.q[:, :, :1].expand(-1, -1, 4, -1)
    c.new = c.new[:1, :, :, :, :1].expand(2, -1, -1, -1, 2, -1)
    c.q_host, c.new_host = c.q.cpu(), c.new.cpu()
    c.call()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("n_new", [2, 20, 90, 600])
def test_two_calls_at_once(n_new):
    """The same cache, two streams, a workspace each; one of the calls on another sequence length."""
    a = Case(1, 8, 2, 128, (2,), [900], n_new)
    b = Case(1, 8, 2, 128, (2,), [900], n_new, [n_new - 1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for c, s in zip((a, b), streams):
            c.call(stream=s)
    torch.cuda.synchronize()
    a.check()
    b.check()
