"""The 8-bit cache on the GPU: appending bit for bit, attention against the 64-bit reference."""

import itertools

import numpy as np
import pytest

import q8_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import looped_transformer_kv_gb300 as rq
    from looped_transformer_kv_gb300.rq import advance_ctx

MARK = 776.0      # what outputs hold before a call


def angles(n_pos, rot, base=10000.0):
    half = rot // 2
    a = np.arange(n_pos)[:, None] * base ** (-np.arange(half) / half)
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


class Case:
    """A cache, and new tokens for it.  Slots that hold no token are full of 0xff bytes (not a number
    as e4m3) under scales that are not numbers."""

    def __init__(self, B, Hq, H, d, fmt, ctx, n_new, n_lens=None, loops=1, loop=0, rot=0, interleaved=False,
                 window=0, sinks=0, paged=False, spread=False, max_ctx=None, cap=None, seed=0, positions=None,
                 scale=0.0, size=1.0, fill=True):
        rng = np.random.default_rng(seed)
        self.B, self.Hq, self.H, self.d, self.fmt, self.loops, self.loop = B, Hq, H, d, fmt, loops, loop
        self.ctx, self.n_new, self.window, self.sinks = list(ctx), n_new, window, sinks
        self.lens = list(n_lens) if n_lens is not None else [n_new] * B
        self.cap = cap or -(-(max(self.ctx) + n_new) // 64) * 64 or 64
        self.max_ctx = max(self.ctx) if max_ctx is None else max_ctx
        self.scale = scale or d ** -0.5
        self.shape = rq.make_q8_shape(B, Hq, H, d, loops, self.cap, fmt, scale)
        tiles = self.cap // 64
        self.codes = np.full((B, H, tiles, loops, 2, 64 * d), 255, np.uint8)
        self.scales = np.full((B, H, tiles, loops, 2, 4), np.nan, np.float32)
        old = rng.standard_normal((B, max(self.ctx + [1]), 2, loops, H, d)) * np.exp(0.5 * rng.standard_normal((B, max(self.ctx + [1]), 2, 1, 1, 1)))
        old[..., 3] *= 8
        old = torch.from_numpy((old * size).astype(np.float32)).bfloat16().float().numpy()
        if fill:
            for b, h, l in itertools.product(range(B), range(H), range(loops)):
                R.append(self.codes[b, h, :, l], self.scales[b, h, :, l], old[b, :self.ctx[b], :, l, h], 0, fmt)
        self.table_np = angles(max(self.cap, 1), rot) if rot else None
        self.interleaved = interleaved
        self.positions = positions
        if rot:
            pos = None if positions is None else torch.tensor(positions, dtype=torch.int32).cuda()
            self.rope = rq.make_rope(torch.from_numpy(self.table_np).cuda(), interleaved, pos)
        else:
            self.rope = None
        if paged:
            n_pages = B * tiles + 3
            self.table = torch.from_numpy(rng.permutation(n_pages)[:B * tiles].astype(np.int32).reshape(B, tiles)).cuda()
            self.paging = rq.make_paging(self.table, n_pages)
            self.cache = rq.Q8Cache(self.shape, n_pages=n_pages)
        else:
            self.table = self.paging = None
            self.cache = rq.Q8Cache(self.shape)
        self.cache.codes.fill_(255)
        self.cache.scales.fill_(float("nan"))
        self.put()
        kv = torch.from_numpy((rng.standard_normal((B, n_new, 2, loops, H, d)) * size).astype(np.float32)).bfloat16()
        q = torch.from_numpy(rng.standard_normal((B, n_new, Hq, d)).astype(np.float32)).bfloat16()
        for b in range(B):      # behind a sequence's last token: NaN
            kv[b, self.lens[b]:] = float("nan")
            q[b, self.lens[b]:] = float("nan")
        self.kv_host, self.q_host = kv, q
        if spread:              # strides of a fused projection's output, odd offsets
            buf = torch.full((B, n_new, 3 * Hq * d + 5), float("nan"), dtype=torch.bfloat16)
            self.q = buf.cuda()[:, :, 3:3 + Hq * d].view(B, n_new, Hq, d)
            self.q.copy_(q)
            wide = torch.full((B, n_new, 2, loops, H, d + 1), float("nan"), dtype=torch.bfloat16)
            self.kv = wide.cuda()[..., 1:]
            self.kv.copy_(kv)
        else:
            self.q, self.kv = q.cuda(), kv.cuda()
        self.ctx_lens = torch.tensor(self.ctx, dtype=torch.int32).cuda()
        self.n_lens = None if n_lens is None else torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.out = torch.full((B, n_new, Hq, d), MARK, dtype=torch.bfloat16).cuda()
        need = rq.q8_workspace_bytes(self.shape, n_new, self.max_ctx, window, sinks)
        assert need > 0
        self.ws = torch.full((need,), 255, dtype=torch.uint8).cuda()

    def put(self):
        """The host's cache to the GPU."""
        codes = torch.from_numpy(self.codes).view(*self.codes.shape[:-1], 64, self.d)
        scales = torch.from_numpy(self.scales)
        if self.paging is None:
            self.cache.codes.copy_(codes)
            self.cache.scales.copy_(scales)
        else:
            at = self.table.long().cpu()
            where = at >= 0
            self.cache.codes[at[where]] = codes.transpose(1, 2)[where].cuda()
            self.cache.scales[at[where]] = scales.transpose(1, 2)[where].cuda()

    def get(self):
        """The GPU's cache by sequence: codes [B][H][tiles][loops][2][64 d] and scales."""
        codes, scales = self.cache.codes.cpu(), self.cache.scales.cpu()
        if self.paging is not None:
            at = self.table.long().cpu()
            codes, scales = codes[at].transpose(1, 2), scales[at].transpose(1, 2)
        return codes.flatten(-2).numpy(), scales.numpy()

    def pos_of(self, b, m):
        return np.array(self.positions)[b, :m] if self.positions is not None else self.ctx[b] + np.arange(m)

    def append(self, stream=None, loop_begin=0, kv=None):
        args = (self.kv if kv is None else kv, loop_begin, self.ctx_lens)
        kw = dict(n_lens=self.n_lens, rope=self.rope, stream=stream)
        if self.paging is not None:
            rq.paged_q8_append(self.shape, self.cache, self.paging, *args, **kw)
        else:
            rq.q8_append(self.shape, self.cache, *args, **kw)

    def append_reference(self, loops=None):
        for b, h, l in itertools.product(range(self.B), range(self.H), loops or range(self.loops)):
            m = min(self.lens[b], self.cap - self.ctx[b])
            x = self.kv_host[b, :m, :, l, h].float().numpy().copy()
            x[:, 0] = R.rotate(x[:, 0], self.pos_of(b, m), self.table_np, self.interleaved)
            R.append(self.codes[b, h, :, l], self.scales[b, h, :, l], x, self.ctx[b], self.fmt)

    def same_cache(self):
        codes, scales = self.get()
        np.testing.assert_array_equal(scales, self.scales)
        np.testing.assert_array_equal(codes, self.codes)

    def attend(self, stream=None, **kw):
        args = (self.q, self.loop, self.ctx_lens, self.max_ctx, self.out, self.ws)
        kw = dict(n_lens=self.n_lens, window=self.window, n_sink=self.sinks, rope=self.rope, stream=stream) | kw
        if self.paging is not None:
            rq.paged_q8_attention(self.shape, self.cache, self.paging, *args, **kw)
        else:
            rq.q8_attention(self.shape, self.cache, *args, **kw)

    def error_word(self):
        return int(self.ws[:4].view(torch.int32).item())

    def check(self, skip=()):
        """Outputs against the reference over the cache that the GPU holds.

        Codes and, without rotation, queries enter the products exactly; a rotated query is rounded to
        fp16, half a step 2^-11 of each element.  The fp32 sums of d products and the scaling are off by
        at most (d + 8) 2^-23 of sum |q k|: a score by e = scale sum|q k| (2^-11 [rotated] + (d + 8) 2^-23).
        m's own rounding drops out (it is the same number in a row's weights and sum).  A weight is
        then within exp(2 e) of its own; rounded to fp16 (2^-11 of itself, or 2^-25 where the largest of
        its row under the largest V scale seen is 2^-1 or more: 2^-24 of V's largest scale times the
        largest code); 2^x and fp32 sums of T terms (chains of T / 16 products, then of a few parts)
        stay below (T / 16 + 64) 2^-23 of sum p|v|, once above and once below the line.  The result is
        rounded to bf16, 2^-8 of itself."""
        assert self.error_word() == 0
        codes, scales = self.get()
        out = self.out.float().cpu().numpy().astype(np.float64)
        G, d = self.Hq // self.H, self.d
        for b, h in itertools.product(range(self.B), range(self.H)):
            m, ctx = self.lens[b], self.ctx[b]
            rows = out[b, :, h * G:(h + 1) * G]
            assert (rows[m:] == MARK).all()                         # left as they were
            if m == 0 or b in skip:
                continue
            k, v = R.rows_of(codes[b, h, :, self.loop], scales[b, h, :, self.loop], ctx + m, d, self.fmt)
            q = self.q_host[b, :m, h * G:(h + 1) * G].float().numpy()
            q = np.stack([R.rotate(q[:, g], self.pos_of(b, m), self.table_np, self.interleaved) for g in range(G)], 1)
            q = q.astype(np.float64)
            lo = max(0, ctx + 1 - self.window) if self.window else 0
            unseen = np.arange(ctx + m) < lo
            unseen[:self.sinks] = False
            k[unseen] = v[unseen] = 0                                  # (may be gone)
            ref, p, mag = R.attend(q, k, v, ctx, self.scale, self.window, self.sinks)
            pv = np.einsum("jgt,td->jgd", p, np.abs(v))
            e = mag[..., None] * ((2.0 ** -11 if self.rope is not None else 0) + (d + 8) * 2.0 ** -23)
            T = ctx + m
            # (two weighted means of the same values are never further apart than 2 max|v|: that bounds the
            # first term where e is large, and keeps pv = 0 from meeting an infinite factor)
            tol = np.minimum(pv * np.expm1(np.minimum(2 * e, 60)) + 2 * np.abs(v).max() * (2 * e > 60), 2 * np.abs(v).max())
            tol += pv * (2.0 ** -11 + 2 * (T / 16 + 64) * 2.0 ** -23)
            tol += 2.0 ** -24 * (p > 0).sum(-1)[..., None] * np.abs(v).max() * p.max(-1)[..., None]
            tol += 2.0 ** -8 * np.abs(ref) * 1.01 + 1e-30
            worst = (np.abs(rows[:m] - ref) / tol).max()
            assert worst <= 1, (b, h, worst)


# ------------------------------------------------------------------------------------ appending

APPENDS = [
    # B, H, d, fmt, ctx, n_new, n_lens, more
    (1, 1, 64, "int8", [0], 1, None, {}),
    (1, 2, 128, "e4m3", [0], 1, None, dict(rot=128)),
    (3, 2, 128, "int8", [15, 16, 17], 1, None, dict(rot=64)),
    (3, 2, 64, "e4m3", [15, 16, 17], 2, None, dict(rot=16, interleaved=True)),
    (2, 3, 128, "e4m3", [63, 64], 130, None, dict(rot=128, interleaved=True, loops=3)),
    (2, 1, 64, "int8", [5, 200], 65, [64, 0], dict(rot=64, loops=2)),
    (4, 2, 128, "int8", [0, 3, 100, 31], 33, [33, 1, 17, 0], dict(rot=96, paged=True)),
    (4, 2, 64, "e4m3", [0, 3, 100, 31], 33, [33, 1, 17, 0], dict(rot=32, paged=True, spread=True)),
    (2, 5, 128, "e4m3", [1, 14], 20, None, dict(spread=True, loops=2)),
    (1, 1, 128, "e4m3", [40], 24, None, dict(cap=64)),
    (1, 1, 128, "int8", [40], 100, None, dict(cap=128)),          # the last ones fall off
    (1, 2, 64, "int8", [7], 9, None, dict(size=1e-20)),
    (1, 2, 128, "e4m3", [7], 9, None, dict(size=1e-33)),           # below the smallest scale's codes
    (1, 2, 128, "e4m3", [7], 9, None, dict(size=1e30, rot=128)),
    (2, 2, 64, "int8", [9, 70], 4, None, dict(rot=64, positions=[[0, 5, 2, 127], [7, 7, 7, 0]], cap=128)),
]


@pytest.mark.parametrize("B,H,d,fmt,ctx,n,lens,more", APPENDS)
def test_append(B, H, d, fmt, ctx, n, lens, more):
    c = Case(B, H, H, d, fmt, ctx, n, lens, **more)
    c.append()
    c.append_reference()
    c.same_cache()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
def test_append_token_by_token(fmt, d):
    """40 steps whose sizes grow and fall: scales rise inside blocks, older codes follow."""
    c = Case(2, 1, 1, d, fmt, [0, 11], 1, cap=64, rot=d)
    rng = np.random.default_rng(1)
    for step in range(40):
        kv = torch.from_numpy((rng.standard_normal((2, 1, 2, 1, 1, d)) * 4.0 ** rng.integers(-3, 4)).astype(np.float32)).bfloat16()
        c.kv_host = kv
        c.append(kv=kv.cuda())
        c.append_reference()
        c.same_cache()
        advance_ctx(c.ctx_lens, 1, c.cap)
        c.ctx = [x + 1 for x in c.ctx]


def test_append_again_leaves_the_same_bits():
    c = Case(2, 2, 2, 128, "int8", [9, 30], 20, rot=128)
    c.append()
    first = [t.clone() for t in c.cache.tensors()]
    c.append()
    assert torch.equal(first[0], c.cache.codes) and torch.equal(first[1].view(torch.int32), c.cache.scales.view(torch.int32))


def test_append_one_loop_of_several():
    c = Case(2, 2, 2, 64, "e4m3", [9, 30], 20, loops=3)
    c.append(loop_begin=1, kv=c.kv[:, :, :, 1:2])
    c.append_reference(loops=[1])
    c.same_cache()


def test_rotation_against_64_bits():
    """Products and a sum rounded one by one: off by at most 3 * 2^-24 (|x| + |y|), and the code by half
    a step more (int8: half the scale)."""
    c = Case(1, 1, 1, 128, "int8", [0], 200, rot=128)
    c.append()
    codes, scales = c.get()
    k, v = R.rows_of(codes[0, 0, :, 0], scales[0, 0, :, 0], 200, 128, "int8")
    x = c.kv_host[0, :, 0, 0, 0].double().numpy()
    z = (x[:, :64] + 1j * x[:, 64:]) * (c.table_np[:200, :, 0].astype(np.float64) + 1j * c.table_np[:200, :, 1])
    y = np.concatenate([z.real, z.imag], -1)
    step = np.repeat(scales[0, 0, :, 0, 0].reshape(-1)[:13], 16)[:200, None]
    size = np.abs(x[:, :64]) + np.abs(x[:, 64:])
    # (a magnitude that bf16 rounds down may lie 2^-8 of itself above the largest code)
    tol = step * 0.5 + 3 * 2.0 ** -24 * np.concatenate([size, size], -1) + 2.0 ** -8 * np.abs(y) * (np.abs(y) > 127 * step)
    assert (np.abs(k - y) <= tol).all()
    assert (np.abs(v - c.kv_host[0, :, 1, 0, 0].double().numpy()) <= np.repeat(scales[0, 0, :, 0, 1].reshape(-1)[:13], 16)[:200, None] * 0.5
            + 2.0 ** -8 * np.abs(v)).all()


def test_rows_that_are_not_finite_spoil_their_block_only():
    c = Case(1, 1, 1, 128, "e4m3", [0], 64, rot=128)
    c.kv_host[0, 20, 0, 0, 0, 5] = float("inf")
    c.kv_host[0, 40, 1, 0, 0, 5] = float("nan")
    c.append(kv=c.kv_host.cuda())
    with np.errstate(invalid="ignore"):
        c.append_reference()
    c.same_cache()
    assert np.isnan(c.scales[0, 0, 0, 0, 0, 1]) and np.isnan(c.scales[0, 0, 0, 0, 1, 2])
    assert np.isnan(c.scales).sum() == 2
    c.attend()
    out = c.out.float().cpu()
    assert torch.isfinite(out[0, :16]).all() and torch.isnan(out[0, 16:]).all()
    # a window that sees none of either block; a block begun anew
    w = Case(1, 1, 1, 128, "e4m3", [0], 64, rot=128, window=4)
    w.cache.codes.copy_(c.cache.codes)
    w.cache.scales.copy_(c.cache.scales)
    w.q.copy_(c.q)
    w.attend()
    bad = torch.isnan(w.out[0].float()).all(-1).all(-1).cpu()
    assert bad.tolist() == [16 <= j < 16 + 16 + 3 or 32 <= j < 32 + 16 + 3 for j in range(64)]
    assert torch.isfinite(w.out[0].float().cpu()[~bad]).all()


def test_positions_outside_the_table():
    pos = [[0, 1, 99999, 3] + [4] * 28]
    c = Case(1, 1, 1, 64, "int8", [0], 32, rot=64, positions=pos)
    c.append()
    assert torch.isnan(c.cache.scales[0, 0, 0, 0, 0, 0]) and torch.isfinite(c.cache.scales[0, 0, 0, 0, 1, :2]).all()
    d = Case(1, 1, 1, 64, "int8", [0], 32, rot=64)
    d.append()
    d.rope = c.rope
    d.attend()
    bad = torch.isnan(d.out[0].float()).all(-1).all(-1).cpu().tolist()
    assert bad == [j == 2 for j in range(32)] and d.error_word() == 0


def test_append_skips_bad_lengths_and_pages():
    c = Case(5, 1, 1, 64, "e4m3", [3, 3, 3, 3, 3], 70, [70, 5, 70, 70, 70], cap=128, paged=True)
    c.ctx_lens.copy_(torch.tensor([3, 3, -1, 128, 3], dtype=torch.int32))
    c.n_lens.copy_(torch.tensor([71, 5, 70, 70, 70], dtype=torch.int32))
    before = c.get()
    table = c.table.clone()
    c.table[4, 0] = -1
    c.append()
    c.table.copy_(table)
    codes, scales = c.get()
    for b in (0, 2, 3):
        np.testing.assert_array_equal(codes[b], before[0][b])
        np.testing.assert_array_equal(scales[b], before[1][b])
    np.testing.assert_array_equal(codes[4, :, 0], before[0][4, :, 0])
    c.append_reference()
    for b, tiles in ((1, slice(None)), (4, slice(1, 2))):
        np.testing.assert_array_equal(codes[b, :, tiles], c.codes[b, :, tiles])
        np.testing.assert_array_equal(scales[b, :, tiles], c.scales[b, :, tiles])


# ------------------------------------------------------------------------------------ attention

SHAPES = [
    # B, Hq, H, d, fmt, ctx, n_new, n_lens, more
    (1, 1, 1, 64, "e4m3", [0], 1, None, {}),
    (1, 2, 2, 64, "int8", [1], 1, None, {}),
    (3, 2, 2, 128, "e4m3", [14, 15, 16], 1, None, {}),
    (3, 4, 1, 128, "int8", [62, 63, 64], 1, None, dict(rot=128)),
    (2, 8, 2, 64, "e4m3", [300, 0], 1, [1, 0], dict(rot=32, interleaved=True)),
    (2, 5, 1, 128, "int8", [127, 500], 1, None, dict(loops=3, loop=1)),
    (2, 6, 2, 128, "e4m3", [100, 33], 2, [2, 1], dict(rot=64)),
    (1, 8, 1, 128, "int8", [700], 2, None, dict(paged=True)),
    (2, 16, 1, 64, "e4m3", [130, 65], 1, None, dict(paged=True, rot=64)),
    (1, 4, 1, 128, "e4m3", [250], 8, None, dict(spread=True, rot=128)),
    (2, 3, 3, 64, "int8", [90, 10], 17, [17, 3], dict(spread=True)),
    (1, 5, 1, 128, "int8", [60], 7, None, {}),
    (2, 2, 2, 128, "e4m3", [0, 0], 33, [33, 16], dict(rot=128)),
    (1, 8, 2, 64, "int8", [64], 65, None, dict(rot=64, interleaved=True)),
    (2, 4, 4, 128, "e4m3", [5, 70], 130, [130, 77], dict(paged=True)),
    (1, 3, 1, 128, "int8", [200], 257, None, dict(rot=96, loops=2, loop=1)),
    (1, 16, 2, 128, "e4m3", [1], 40, None, dict(scale=0.3)),
    (1, 2, 1, 128, "int8", [900], 1, None, dict(max_ctx=1000, cap=1024)),
    (2, 1, 1, 128, "e4m3", [0, 300], 34, [34, 1], {}),
    (1, 4, 1, 64, "e4m3", [63], 33, None, dict(rot=64)),
    (3, 8, 1, 128, "int8", [0, 500, 130], 70, [70, 0, 33], dict(rot=128, paged=True, spread=True)),
    (1, 1, 1, 128, "int8", [1000], 300, None, {}),
    (2, 2, 1, 64, "int8", [129, 128], 127, [127, 64], dict(rot=16, interleaved=True, loops=2, loop=1)),
    (1, 2, 1, 64, "e4m3", [40], 100, None, dict(size=1e-20)),
    (1, 2, 1, 128, "e4m3", [40], 100, None, dict(size=1e25)),
    (2, 8, 1, 128, "e4m3", [0, 300], 130, [130, 65], dict(paged=True, rot=128)),
    (1, 4, 1, 64, "int8", [100], 260, None, dict(rot=32)),
    (3, 3, 1, 64, "e4m3", [5, 0, 200], 400, [257, 0, 400], dict(loops=2, loop=1)),
    (1, 8, 2, 128, "int8", [700], 70, None, dict(spread=True, interleaved=True, rot=64)),
    (1, 2, 1, 64, "e4m3", [40], 3, None, dict(size=1e-20)),
    (1, 2, 1, 128, "int8", [40], 3, None, dict(size=1e-33)),
]


@pytest.mark.parametrize("B,Hq,H,d,fmt,ctx,n,lens,more", SHAPES)
def test_attention(B, Hq, H, d, fmt, ctx, n, lens, more):
    c = Case(B, Hq, H, d, fmt, ctx, n, lens, **more)
    c.append()
    c.attend()
    c.check()


WINDOWS = [(1, 0), (2, 1), (16, 0), (17, 4), (64, 64), (63, 130), (100, 16), (1000, 7), (1, 1000)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("n", [1, 5, 70, 200])
def test_window(window, sinks, n):
    """Window and sinks; the pages that no token sees are gone (entries of -1 and beyond the pool)."""
    fmt = "int8" if (window + n) % 2 else "e4m3"
    c = Case(2, 6, 2, 128 if n < 70 else 64, fmt, [333, 65], n, window=window, sinks=sinks, paged=True, rot=64)
    c.append()
    for b, ctx in enumerate(c.ctx):
        lo = max(0, ctx + 1 - window)
        for tile in range(c.cap // 64):
            seen = tile * 64 < ctx + n and (tile * 64 + 63 >= lo or tile * 64 < min(sinks, ctx + n))
            if not seen:
                page = int(c.table[b, tile])
                c.cache.codes[page] = 255
                c.cache.scales[page] = float("nan")
    keep = c.table.clone()
    for b, ctx in enumerate(c.ctx):
        lo = max(0, ctx + 1 - window)
        for tile in range(c.cap // 64):
            if not (tile * 64 < ctx + n and (tile * 64 + 63 >= lo or tile * 64 < min(sinks, ctx + n))):
                c.table[b, tile] = -1 if tile % 2 else 1 << 30
    c.attend()
    c.table.copy_(keep)
    c.check()


LONG = [
    # B, Hq, H, d, fmt, ctx, n_new, n_lens, more: units that several CTAs share
    (2, 2, 1, 128, "e4m3", [9000, 2111], 1, None, dict(rot=128, fill=False)),
    (1, 16, 2, 128, "int8", [7001], 2, None, dict(paged=True, fill=False)),
    (2, 8, 1, 64, "int8", [5000, 130], 4, [4, 3], dict(rot=64, fill=False)),
    (1, 4, 1, 128, "e4m3", [6000], 40, None, dict(rot=64, fill=False)),
    (2, 4, 1, 64, "e4m3", [100, 3000], 300, [300, 222], dict(paged=True, fill=False)),
    (1, 8, 1, 128, "int8", [3333], 200, None, dict(rot=128, window=1000, sinks=70, fill=False)),
    (1, 2, 1, 128, "e4m3", [20000], 3, None, dict(window=5000, sinks=200, fill=False, paged=True)),
]


def fill_cache(c, seed=0):
    """Random codes and scales (2^-6 .. 2^-3) in every slot of a case's cache, on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 127, c.cache.codes.shape, generator=g, device="cuda", dtype=torch.uint8)
    codes |= torch.randint(0, 2, codes.shape, generator=g, device="cuda", dtype=torch.uint8) << 7
    if c.fmt == "e4m3":        # below 16, no NaN
        codes &= 0xd7
    c.cache.codes.copy_(codes)
    c.cache.scales.copy_(2.0 ** torch.randint(-6, -2, c.cache.scales.shape, generator=g, device="cuda"))


@pytest.mark.parametrize("B,Hq,H,d,fmt,ctx,n,lens,more", LONG)
def test_long_contexts(B, Hq, H, d, fmt, ctx, n, lens, more):
    c = Case(B, Hq, H, d, fmt, ctx, n, lens, **more)
    fill_cache(c)
    c.append()
    c.attend()
    c.check()


def test_a_run_of_tokens_as_a_serving_loop_makes_it():
    """A prompt in two chunks, drafted tokens, single tokens: append, attend, advance, on one paged cache;
    every output against the reference over the cache as it is then."""
    c = Case(2, 8, 2, 128, "e4m3", [0, 0], 200, cap=512, rot=128, paged=True, max_ctx=400)
    rng = np.random.default_rng(3)
    for n in (200, 75, 5, 1, 1, 1):
        c.n_new, c.lens = n, [n, n]
        c.kv_host = torch.from_numpy(rng.standard_normal((2, n, 2, 1, 2, 128)).astype(np.float32)).bfloat16()
        c.q_host = torch.from_numpy(rng.standard_normal((2, n, 8, 128)).astype(np.float32)).bfloat16()
        c.q, c.out = c.q_host.cuda(), torch.full((2, n, 8, 128), MARK, dtype=torch.bfloat16, device="cuda")
        c.append(kv=c.kv_host.cuda())
        c.append_reference()
        c.same_cache()
        c.attend()
        c.check()
        advance_ctx(c.ctx_lens, n, c.cap)
        c.ctx = [x + n for x in c.ctx]
    assert c.ctx_lens.tolist() == [283, 283]


@pytest.mark.parametrize("n", [1, 3, 40, 300])
def test_bad_lengths_and_pages(n):
    """A sequence with bad lengths, and tokens that see a bad page, are NaN; the others are as ever."""
    def case():
        c = Case(4, 2, 2, 64, "e4m3", [130, 64, 200, 10], n, paged=True, max_ctx=200, cap=576)
        c.append()
        return c

    c = case()
    c.attend()
    c.check()
    clean = c.out.clone()
    for what, value, b in (("ctx", -1, 1), ("ctx", 201, 3), ("ctx", 577, 0), ("n", -1, 2), ("n", n + 1, 0)):
        d = case()
        lens = torch.full((4,), n, dtype=torch.int32).cuda()
        d.n_lens = lens
        (d.ctx_lens if what == "ctx" else lens)[b] = value
        d.attend()
        assert d.error_word() != 0
        assert torch.isnan(d.out[b].float()).all()
        others = [x for x in range(4) if x != b]
        assert torch.isfinite(d.out[others].float()).all()
        np.testing.assert_allclose(d.out[others].float().cpu(), clean[others].float().cpu(), rtol=2.0 ** -7, atol=1e-3)
    for bad in (-1, 1 << 30):
        d = case()
        d.table[2, 1] = bad           # slots 64..127 of sequence 2: all of its tokens see them
        d.attend()
        assert d.error_word() != 0 and torch.isnan(d.out[2].float()).all()
        assert torch.isfinite(d.out[[0, 1, 3]].float()).all()


def test_no_new_tokens():
    for n in (1, 40, 600):
        c = Case(3, 2, 1, 64, "int8", [5, 0, 70], n, [0, 0, 0], cap=704)
        c.append()
        c.same_cache()
        c.attend()
        torch.cuda.synchronize()
        assert c.error_word() == 0 and (c.out == MARK).all()
    c = Case(3, 2, 1, 64, "int8", [5, 0, 70], 1)
    rq.q8_append(c.shape, c.cache, c.kv[:, :0], 0, c.ctx_lens)
    rq.q8_attention(c.shape, c.cache, c.q[:, :0], 0, c.ctx_lens, 70, c.out[:, :0], c.ws)
    c.same_cache()


@pytest.mark.parametrize("n,heads", [(1, 1), (1, 3), (2, 1)])
def test_wide_batches(n, heads):
    """More sequences than a CTA cuts for itself, many of them without tokens."""
    B = 1500
    rng = np.random.default_rng(5)
    ctx = rng.integers(0, 150, B).tolist()
    lens = rng.integers(0, n + 1, B).tolist()
    c = Case(B, heads, 1, 64, "e4m3", ctx, n, lens, cap=192, fill=False)
    fill_cache(c)
    c.append()
    c.attend()
    c.check()


SHORT = [
    # B, Hq, H, d, fmt, longest, n_new, more
    (4, 8, 8, 128, "e4m3", 63, 1, {}),
    (40, 16, 16, 64, "int8", 380, 1, dict(rot=64)),
    (28, 16, 16, 128, "e4m3", 500, 1, dict(paged=True)),
    (40, 24, 24, 64, "e4m3", 200, 1, {}),
    (70, 16, 4, 64, "int8", 250, 4, dict(rot=32)),
    (90, 8, 2, 128, "e4m3", 300, 5, dict(paged=True, rot=128)),
    (40, 16, 2, 64, "int8", 120, 4, dict(spread=True)),
    (60, 4, 4, 64, "e4m3", 900, 1, dict(window=150, sinks=70, paged=True)),
    (60, 8, 4, 128, "int8", 700, 6, dict(window=33)),
]


@pytest.mark.parametrize("B,Hq,H,d,fmt,longest,n,more", SHORT)
def test_many_short_sequences(B, Hq, H, d, fmt, longest, n, more):
    """Contexts so short that no unit is divided, of all lengths, some without tokens."""
    rng = np.random.default_rng(B + n)
    ctx = rng.integers(0, longest + 1, B)
    ctx[B // 3] = longest
    ctx[: B // 4 : 5] = 0
    c = Case(B, Hq, H, d, fmt, ctx.tolist(), n, rng.integers(0, n + 1, B).tolist(), fill=False, **more)
    fill_cache(c)
    c.append()
    c.attend()
    c.check()


@pytest.mark.parametrize("n", [1, 4, 50, 300])
def test_blocks_of_very_different_sizes(n):
    """V's and K's scales from 2^-100 (zeros) over 2^-20 to 2^10 in one context."""
    c = Case(1, 2, 1, 128, "int8", [400], n, cap=704)
    rng = np.random.default_rng(9)
    rows = rng.standard_normal((400, 2, 128)).astype(np.float32)
    size = np.repeat(2.0 ** rng.integers(-20, 3, (25, 2)), 16, 0)[:400]
    size[rng.integers(0, 25, 4) * 16 + 3] *= 0
    rows *= size[:, :, None]
    rows[96:112, 1] = 0
    rows[200:, 1] *= 2.0 ** 8
    R.append(c.codes[0, 0, :, 0], c.scales[0, 0, :, 0], torch.from_numpy(rows).bfloat16().float().numpy(), 0, "int8")
    c.put()
    c.append()
    c.attend()
    c.check()


@pytest.mark.parametrize("n", [1, 50, 300])
def test_huge_scores_pick_one_slot(n):
    """Scores of 1e25: the weights are 0 and 1, and the output one value row."""
    c = Case(1, 1, 1, 128, "e4m3", [200], n, size=1e25, cap=512)
    c.append()
    c.attend()
    codes, scales = c.get()
    k, v = R.rows_of(codes[0, 0, :, 0], scales[0, 0, :, 0], 200 + n, 128, "e4m3")
    s = c.q_host[0, :, 0].double().numpy() @ k.T
    s[np.arange(200 + n)[None] > 200 + np.arange(n)[:, None]] = -np.inf
    best = s.argmax(1)
    # (rows whose two largest scores are closer than the fp32 sums' rounding may go either way)
    top = np.sort(s, 1)[:, -2:]
    sure = top[:, 1] - top[:, 0] > 2.0 ** -15 * np.abs(c.q_host[0, :, 0].double().numpy()).sum(1) * np.abs(k).max()
    assert sure.sum() >= n / 2
    out = c.out[0, :, 0].double().cpu().numpy()
    assert (np.abs(out - v[best])[sure] <= 2.0 ** -8 * np.abs(v[best])[sure] * 1.01 + 2.0 ** -10 * np.abs(v).max()).all()


def test_same_call_same_bits_and_any_larger_workspace():
    for n in (1, 5, 60, 400):
        c = Case(2, 4, 2, 64, "e4m3", [900, 333], n, rot=64, fill=False)
        fill_cache(c)
        c.append()
        c.attend()
        first = c.out.clone()
        c.ws = torch.full((rq.q8_workspace_bytes(c.shape, n + 700, c.max_ctx, 0, 0),), 255, dtype=torch.uint8).cuda()
        c.out.fill_(MARK)
        c.attend()
        assert torch.equal(first, c.out)
        c.check()


def test_unaligned_outputs_and_inputs():
    for n in (1, 20, 300):
        c = Case(1, 3, 1, 128, "int8", [77], n, spread=True, cap=384)
        buf = torch.full((n * 3 * 128 + 9,), MARK, dtype=torch.bfloat16, device="cuda")
        c.out = buf[5:5 + n * 3 * 128].view(1, n, 3, 128)
        c.append()
        c.attend()
        c.check()
        assert (buf[:5] == MARK).all() and (buf[-4:] == MARK).all()


def test_broadcast_queries():
    """Strides of 0: one query row for all heads and tokens."""
    c = Case(2, 4, 2, 64, "e4m3", [50, 9], 3)
    c.append()
    c.q = c.q[:1, :1, :1].expand(2, 3, 4, 64)
    c.q_host = c.q.cpu()
    c.attend()
    c.check()


def test_two_calls_at_once_on_side_streams():
    cases = [Case(2, 8, 2, 128, "e4m3", [3000, 900], n, rot=128, fill=False, seed=n) for n in (1, 30, 300)]
    for c in cases:
        fill_cache(c, c.n_new)
        c.append()
        c.attend()
    torch.cuda.synchronize()
    want = [c.out.clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for c in cases:
        c.out.fill_(MARK)
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cases, streams):
            c.append(stream=s)
            c.attend(stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert c.error_word() == 0 and torch.equal(c.out, w)


def test_a_captured_step_replayed():
    """Append, attend and advance in one graph: replays leave the same bits as eager steps."""
    def build():
        c = Case(2, 4, 2, 128, "int8", [60, 3], 1, rot=128, cap=256, max_ctx=255)
        return c

    eager, graphed = build(), build()

    def step(c):
        c.append()
        c.attend()
        advance_ctx(c.ctx_lens, 1, c.cap)

    outs = []
    for _ in range(40):
        step(eager)
        outs.append(eager.out.clone())
    graphed.append()      # (once before the capture: the same call again leaves the same bits)
    graphed.attend()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(graphed)
    for i in range(40):
        g.replay()
        assert torch.equal(graphed.out, outs[i]), i
    assert torch.equal(eager.cache.codes, graphed.cache.codes)
    assert eager.ctx_lens.tolist() == graphed.ctx_lens.tolist() == [100, 43]
    assert graphed.error_word() == 0


@pytest.mark.parametrize("n", [1, 20, 150, 300])
def test_captured_chunks(n):
    c = Case(2, 4, 1, 64, "e4m3", [500, 77], n, rot=64, cap=832, fill=False)
    fill_cache(c)
    c.append()
    c.attend()
    torch.cuda.synchronize()
    want = c.out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.append()
        c.attend()
        c.attend()
    c.out.fill_(MARK)
    for _ in range(3):
        g.replay()
    assert torch.equal(c.out, want) and c.error_word() == 0


def test_offsets_beyond_32_bits():
    """A cache of 5.4 GB (16 loops, 1,310,720 slots): the last slots, through a window, by each kernel."""
    L, cap = 16, 5 << 18
    shape = rq.make_q8_shape(1, 2, 2, 64, L, cap, "e4m3")
    cache = rq.Q8Cache(shape)
    assert cache.codes.numel() > 1 << 32
    cache.codes.fill_(255)
    for n in (1, 30, 600):
        ctx = cap - 700
        c = Case(1, 2, 2, 64, "e4m3", [40], n, rot=64, cap=704, window=30, positions=[list(range(n))])
        kv = torch.full((1, n, 2, L, 2, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        kv[:, :, :, L - 1] = c.kv[:, :, :, 0]
        lens = torch.tensor([ctx], dtype=torch.int32, device="cuda")
        rq.q8_append(shape, cache, kv[:, :, :, L - 1:], L - 1, lens, rope=c.rope)
        ws = torch.empty(rq.q8_workspace_bytes(shape, n, ctx, 30, 0), dtype=torch.uint8, device="cuda")
        out = torch.full((1, n, 2, 64), MARK, dtype=torch.bfloat16, device="cuda")
        # slots before the new ones hold nothing: a window of 1 sees a token's own slot
        rq.q8_attention(shape, cache, c.q, L - 1, lens, ctx, out, ws, window=1, rope=c.rope)
        t = ctx + np.arange(n)
        codes = cache.codes[0, :, ctx // 64:-(-(ctx + n) // 64), L - 1, 1].flatten(2).cpu().numpy()
        scales = cache.scales[0, :, ctx // 64:-(-(ctx + n) // 64), L - 1, 1].cpu().numpy()
        for h in (0, 1):
            v = np.stack([R.value_of(codes[h, x // 64 - ctx // 64, R.place(x, 64)], "e4m3") *
                          float(scales[h, x // 64 - ctx // 64, x % 64 // 16]) for x in t])
            got = out[0, :, h].float().cpu().numpy()
            assert (np.abs(got - v) <= 2.0 ** -8 * np.abs(v) + 2.0 ** -10 * np.abs(v) + 1e-30).all()
        assert int(ws[:4].view(torch.int32).item()) == 0
    del cache
    torch.cuda.empty_cache()


def test_sequences_in_groups():
    """Operand tiles of more than 2 GB: sequences are handled in groups; each as it is alone, and a bad
    length in any of them is told."""
    B, H, ctx, n = 9, 16, 30000, 520
    cap = 30592
    shape, one = (rq.make_q8_shape(b, H, H, 128, 1, cap, "int8") for b in (B, 1))
    cache = rq.Q8Cache(shape)
    g = torch.Generator(device="cuda").manual_seed(0)
    cache.codes.random_(generator=g)
    cache.scales.fill_(2.0 ** -7)
    q = torch.randn(B, n, H, 128, generator=g, device="cuda").bfloat16()
    lens = torch.tensor([ctx - 3000 * b for b in range(B)], dtype=torch.int32, device="cuda")
    need = rq.q8_workspace_bytes(shape, n, ctx, 0, 0)
    assert need > 2 << 30
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, MARK)
    rq.q8_attention(shape, cache, q, 0, lens, ctx, out, ws)
    assert int(ws[:4].view(torch.int32).item()) == 0
    for b in (0, 4, 8):
        alone = rq.Q8Cache(one, codes=cache.codes[b].reshape(-1), scales=cache.scales[b].reshape(-1))
        got = torch.full_like(q[:1], MARK)
        rq.q8_attention(one, alone, q[b:b + 1], 0, lens[b:b + 1].clone(), ctx, got, ws)
        # the same products; parts joined elsewhere (fp32), results rounded to bf16
        torch.testing.assert_close(out[b:b + 1].float(), got.float(), rtol=2.0 ** -7, atol=1e-4)
    for b in (0, 8):
        bad = lens.clone()
        bad[b] = ctx + 1
        rq.q8_attention(shape, cache, q, 0, bad, ctx, out, ws)
        assert int(ws[:4].view(torch.int32).item()) != 0
        assert torch.isnan(out[b].float()).all() and torch.isfinite(out[4].float()).all()
    del cache, ws
    torch.cuda.empty_cache()


def test_the_largest_windows_and_sinks():
    """Windows and sinks beyond any context: everything is seen."""
    for n in (1, 40):
        c = Case(1, 2, 1, 64, "e4m3", [300], n)
        c.append()
        c.attend()
        want = c.out.clone()
        for window, sinks in (((1 << 31) - 1, 0), ((1 << 31) - 1, (1 << 31) - 1), (1 << 30, 5), (1, (1 << 31) - 1)):
            c.ws = torch.empty(rq.q8_workspace_bytes(c.shape, n, c.max_ctx, window, sinks), dtype=torch.uint8, device="cuda")
            c.out.fill_(MARK)
            c.attend(window=window, n_sink=sinks)
            assert torch.equal(c.out, want), (n, window, sinks)


def test_zero_queries_and_zero_states():
    """Rows of zeros: equal weights, outputs the mean; a cache of zeros: zeros."""
    for n in (1, 9, 50):
        c = Case(1, 4, 1, 128, "int8", [100], n)
        c.append()
        c.q_host[:] = 0
        c.q = c.q_host.cuda()
        c.attend()
        c.check()
        z = Case(1, 4, 1, 128, "int8", [0], n)
        z.append(kv=torch.zeros_like(z.kv))
        assert (z.cache.scales[0, 0, 0, 0, :, 0] == 2.0 ** -100).all()
        z.attend()
        assert (z.out == 0).all()


def test_tensors_elsewhere_are_refused():
    c = Case(1, 2, 1, 64, "e4m3", [5], 2, rot=64)
    with pytest.raises(AssertionError):
        rq.q8_append(c.shape, c.cache, c.kv.cpu(), 0, c.ctx_lens)
    with pytest.raises(AssertionError):
        rq.q8_append(c.shape, c.cache, c.kv, 0, c.ctx_lens.cpu())
    with pytest.raises(AssertionError):
        rq.q8_append(c.shape, c.cache, c.kv, 0, c.ctx_lens, rope=rq.make_rope(torch.zeros(8, 32, 2)))
    for q, out, ws in ((c.q.cpu(), c.out, c.ws), (c.q, c.out.cpu(), c.ws), (c.q, c.out, c.ws.cpu())):
        with pytest.raises(AssertionError):
            rq.q8_attention(c.shape, c.cache, q, 0, c.ctx_lens, 5, out, ws)
