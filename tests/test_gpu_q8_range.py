"""The 8-bit cache's attention where blocks of slots, scores and rows lie far apart, against 64 bits."""

import numpy as np
import pytest

import q8_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_q8 import MARK, Case, fill_cache  # noqa: E402


@pytest.mark.parametrize("B,n,longest", [(60, 40, 600), (60, 100, 2500), (60, 300, 900), (12, 300, 6000)])
def test_row_tiles_without_rows(B, n, longest):
    """Many units of which one row tile has no rows: a CTA walks several, some in turn with full ones, and
    neither runs ahead of the other tile's products nor falls behind them."""
    rng = np.random.default_rng(n)
    ctx = rng.integers(0, longest, B)
    ctx[7] = longest
    c = Case(B, 4, 4, 64, "int8", ctx.tolist(), n, rng.integers(0, n + 1, B).tolist(), fill=False)
    fill_cache(c)
    c.append()
    for _ in range(3):
        c.out.fill_(MARK)
        c.attend()
    c.check()


class Hand(Case):
    """One sequence whose rows are given, the same for all H kv-heads: k, v [ctx + n][d], q [n][G][d].  (With
    one head a context is divided among CTAs, with many a CTA walks it.)"""

    def __init__(self, k, v, q, fmt, H=1, **more):
        n, G, d = q.shape
        ctx = len(k) - n
        super().__init__(1, G * H, H, d, fmt, [ctx], n, fill=False, **more)
        kv = torch.from_numpy(np.stack([k, v], 1).astype(np.float32)).bfloat16()
        R.append(self.codes[0, 0, :, 0], self.scales[0, 0, :, 0], kv[:ctx].float().numpy(), 0, fmt)
        self.codes[:], self.scales[:] = self.codes[:, :1], self.scales[:, :1]
        self.put()
        self.kv_host = kv[ctx:].view(1, n, 2, 1, 1, d).expand(1, n, 2, 1, H, d).contiguous()
        self.q_host = torch.from_numpy(np.concatenate([q] * H, 1).astype(np.float32)).bfloat16()[None].contiguous()
        self.kv, self.q = self.kv_host.cuda(), self.q_host.cuda()

    def run(self):
        self.append()
        self.attend()
        assert self.error_word() == 0
        return self


def close(c, tokens=slice(None)):
    """Outputs of a case of one sequence against the reference over the cache that the GPU holds.

    Everything goes by what a row sees and how much it weighs.  A score's error e: the fp32 sum of d products
    and its scaling, (d + 8) 2^-23 of its sum |q k|; the row's reference is subtracted, and the exponents of
    scales (at most 2^8 in all) added, in fp32: 2^-23 of the largest such sum among slots that matter, and
    2^-15.  A weight is off by expm1(e), and so is its share of the sum.  Times its block's scale it is
    rounded to fp16: 2^-11 of itself, or 2^-24 of the largest product of weight and scale that the row sees
    (which is 2^-1 or more in units where fp16's last half step is 2^-25); fp32 sums (T / 16 + 64) 2^-23,
    twice; the result 2^-8 of itself."""
    codes, scales = c.get()
    assert (codes == codes[:, :1]).all() and ((scales == scales[:, :1]) | np.isnan(scales)).all()
    G, d, m, ctx = c.Hq // c.H, c.d, c.n_new, c.ctx[0]
    T = ctx + m
    out = c.out.double().cpu().numpy().reshape(m, c.H, G, d)
    k, v = R.rows_of(codes[0, 0, :, 0], scales[0, 0, :, 0], T, d, c.fmt)
    q = c.q_host[0, :, :G].double().numpy()
    block = np.repeat(scales[0, 0, :, 0, 1].reshape(-1).astype(np.float64), 16)[:T]
    own, t = (ctx + np.arange(m))[:, None], np.arange(T)[None]
    seen = t <= own
    if c.window:
        seen &= (t > own - c.window) | (t < c.sinks)
    s = np.einsum("jgd,td->jgt", q, k) * c.scale
    s = np.where(seen[:, None], s, -np.inf)
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    ref = np.einsum("jgt,td->jgd", p, v)
    pv = np.einsum("jgt,td->jgd", p, np.abs(v))
    mag = np.einsum("jgd,td->jgt", np.abs(q), np.abs(k)) * c.scale * seen[:, None]
    best = np.where(p > 1e-9, mag, 0).max(-1, keepdims=True)
    u = p * np.expm1(np.minimum((mag + best) * (d + 8) * 2.0 ** -23 + 2.0 ** -15, 60))
    assert np.median(u[tokens].sum(-1)) < 2.0 ** -6                        # (the test means something)
    tol = 2 * (np.einsum("jgt,td->jgd", u, np.abs(v)) + np.abs(ref) * u.sum(-1)[..., None])
    tol += pv * (2.0 ** -11 + 2 * (T / 16 + 64) * 2.0 ** -23)
    most = (p * block).max(-1)[..., None]
    tol += 2.0 ** -24 * most * np.einsum("jt,td->jd", seen.astype(np.float64), np.abs(v) / block[:, None])[:, None]
    tol += 2.0 ** -8 * np.abs(ref) * 1.01 + 1e-37
    worst = (np.abs(out - ref[:, None]) / tol[:, None])[tokens].max()
    assert worst <= 1, worst


FEW = [(2, 1), (2, 4), (4, 4), (8, 4)]          # tokens, query heads: 2, 8, 16, 32 rows
MANY = [(40, 1), (64, 4), (300, 1)]
ONE = [(1, 1), (1, 8)]


def normal(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def slots_of(n, T=200):
    """A context for n new tokens of which the last begins a block of 16 slots."""
    return -(-(T + n) // 16) * 16 + 1


def aimed(seed, n, G, d):
    """Queries that lie along one direction, and the direction."""
    u = normal(seed, d)
    u /= np.linalg.norm(u)
    return 8 * u + 0.1 * normal(seed + 1, n, G, d), u


@pytest.mark.parametrize("far", [12, 30, 60, 100])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("H", [1, 128])
@pytest.mark.parametrize("n,G", FEW + MANY)
def test_the_last_token_s_large_value_changes_no_earlier_output(n, G, fmt, far, H):
    T, d = slots_of(n), 128 if n % 8 else 64
    k, v, q = normal(1, T, d) / 2, normal(2, T, d), normal(3, n, G, d)
    v[-1] *= 2.0 ** far
    close(Hand(k, v, q, fmt, H).run())


@pytest.mark.parametrize("far", [12, 30, 60, 100])
@pytest.mark.parametrize("H", [1, 128])
@pytest.mark.parametrize("n,G", FEW + MANY)
def test_a_large_value_that_left_the_window(n, G, far, H):
    """Only the first token's window reaches the slot; the other slots of its block are out of every window."""
    window, d = 289, 128 if n % 8 else 64
    ctx = 600 + 15 - (600 + 1 - window) % 16
    assert (ctx + 1 - window) % 16 == 15
    T = ctx + n
    k, v, q = normal(27, T, d) / 2, normal(28, T, d), normal(29, n, G, d)
    v[ctx + 1 - window] *= 2.0 ** far
    close(Hand(k, v, q, "e4m3" if far % 4 else "int8", H, window=window).run())


@pytest.mark.parametrize("far", [12, 30, 38])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("H", [1, 128])
@pytest.mark.parametrize("n,G", ONE + FEW + MANY)
def test_large_values_of_no_weight(n, G, fmt, far, H):
    """A block whose values are 2^far larger at weights of e^-60."""
    T, d = slots_of(n, 300), 128 if n % 8 else 64
    q, u = aimed(4, n, G, d)
    k, v = normal(5, T, d) / 4, normal(6, T, d)
    for block in (slice(32, 48), slice(192, 208)):
        k[block] = -60 * d ** 0.5 / 8 * u + normal(7, 16, d) / 4
        v[block] *= 2.0 ** far
    close(Hand(k, v, q, fmt, H).run())


@pytest.mark.parametrize("H", [1, 128])
@pytest.mark.parametrize("n,G", ONE + FEW + MANY)
def test_values_of_many_sizes(n, G, H):
    """Every block of values of another size, 2^-90 to 2^100, its weights such that each matters somewhere."""
    for seed in range(4):
        rng = np.random.default_rng(seed)
        T, d = slots_of(n, 700), 128
        q, u = aimed(8 + seed, n, G, d)
        far = np.repeat(rng.integers(-90, 101, T // 16 + 1), 16)[:T] if seed else np.repeat(rng.permutation(T // 16 + 1) % 40 * 5 - 90, 16)[:T]
        k = normal(9 + seed, T, d) / 4 - (far * np.log(2.0) * d ** 0.5 / 8)[:, None] * u / 2 ** (seed % 2)
        v = normal(10 + seed, T, d) * 2.0 ** far[:, None]
        close(Hand(k, v, q, "int8" if seed % 2 else "e4m3", H).run())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("H", [1, 128])
@pytest.mark.parametrize("n,G", ONE + FEW + MANY)
def test_scores_far_below_zero(n, G, fmt, H):
    """All scores near -1e32, one the largest by far: the output is its value row."""
    T, d = n + 150, 64
    q = np.zeros((n, G, d))
    q[:, :, 5] = 2.0 ** 50
    k = np.zeros((T, d))
    k[:, 5] = -2.0 ** 60 * (1.5 + np.arange(T) % 7 / 8)
    k[3, 5] = -2.0 ** 60
    c = Hand(k, normal(11, T, d), q, fmt, H).run()
    codes, scales = c.get()
    v = R.rows_of(codes[0, 0, :, 0], scales[0, 0, :, 0], T, d, fmt)[1][3]
    assert (np.abs(c.out[0].double().cpu().numpy() - v) <= 2.0 ** -8 * np.abs(v)).all()


SIZES = [(-90, -50, 0.0), (-80, -45, 0.0), (0, -50, 2.0 ** -80), (-60, -60, 2.0 ** -20), (-100, -100, 0.0), (100, -98, 0.0), (-98, 100, 0.0),
         (-105, 106, 0.0), (-112, 112, 0.0), (-118, 117, 0.0), (-30, 110, 2.0 ** -81), (110, -20, 2.0 ** -92)]


@pytest.mark.parametrize("qe,ke,scale", SIZES)
@pytest.mark.parametrize("n,G", ONE[:1] + FEW[1:] + MANY)
def test_sizes_of_queries_and_keys(n, G, qe, ke, scale):
    """Queries of 2^qe and keys of 2^ke, whose scores are moderate."""
    T, d = n + 280, 128 if n % 8 else 64
    k, v, q = normal(12, T, d) * 2.0 ** ke, normal(13, T, d), normal(14, n, G, d) * 2.0 ** qe
    close(Hand(k, v, q, "int8" if n % 3 else "e4m3", scale=scale).run())


@pytest.mark.parametrize("far", [20, 28, 34, 60, 110])
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("H", [1, 128])
@pytest.mark.parametrize("n,G", ONE + FEW + MANY)
def test_zeros_beside_large_values(n, G, first, far, H):
    """Slots of zero values keep their weight in the sum beside values of 2^far."""
    T, d = n + 512, 64
    k, v, q = normal(15, T, d) / 2, normal(16, T, d) * 2.0 ** far, normal(17, n, G, d)
    if first:
        v[:256] = 0
    else:
        v[128:384] = 0
    close(Hand(k, v, q, "int8" if far % 4 else "e4m3", H).run())


@pytest.mark.parametrize("far", [10, 16, 25, 30, 60])
@pytest.mark.parametrize("H", [1, 128])
@pytest.mark.parametrize("n,G", FEW + MANY)
def test_the_last_token_s_large_key_changes_no_earlier_output(n, G, far, H):
    T, d = slots_of(n), 128 if n % 8 else 64
    k, v, q = normal(18, T, d), normal(19, T, d), normal(20, n, G, d)
    k[-1] *= 2.0 ** far
    v[-1] *= 2.0 ** far
    close(Hand(k, v, q, "e4m3" if far % 4 else "int8", H).run(), slice(0, n - 1))


@pytest.mark.parametrize("far", [10, 16, 25, 30, 60])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("H", [1, 128])
@pytest.mark.parametrize("n,G", ONE + FEW + MANY)
def test_large_keys_of_no_weight(n, G, fmt, far, H):
    """A block of keys 2^far larger that point away from the queries: the other keys' scores decide."""
    T, d = slots_of(n, 300), 128 if n % 8 else 64
    q, u = aimed(21, n, G, d)
    k, v = normal(22, T, d), normal(23, T, d)
    for block in (slice(16, 32), slice(208, 224)):
        k[block] = -u * d ** 0.5 * 2.0 ** far
    close(Hand(k, v, q, fmt, H).run())


@pytest.mark.parametrize("T", [100, 3000])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("n,G", ONE + FEW + MANY)
def test_values_near_the_largest(n, G, fmt, T):
    """Values up to 3e38: a weighted mean is no larger."""
    T, d = T + n, 64
    k, v, q = normal(24, T, d) / 2, np.clip(normal(25, T, d), -1, 1) * 2.98e38, normal(26, n, G, d)
    v[:, :8] = np.abs(v[:, :8])
    close(Hand(k, v, q, fmt).run())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("n,Hq", [(5, 1), (5, 4), (40, 1)])
def test_a_bad_page_spoils_only_tokens_that_see_it(n, Hq, fmt):
    """Whatever lies in the pool's first page."""
    c = next(c for c in (Case(1, Hq, 1, 64, fmt, [62], n, paged=True, seed=s) for s in range(99)) if not (c.table == 0).any())
    c.append()
    c.attend()
    c.check()
    want = c.out.clone()
    c.cache.codes[0] = 255
    c.cache.scales[0] = 1.0
    c.table[0, 1] = -1
    c.attend()
    assert c.error_word() != 0
    assert torch.isnan(c.out[0, 2:].float()).all()
    # (the products are the same; a unit may be divided elsewhere)
    torch.testing.assert_close(c.out[0, :2].float(), want[0, :2].float(), rtol=2.0 ** -7, atol=1e-4)


@pytest.mark.parametrize("qe,ke", [(100, 60), (120, 118), (126, 2), (2, 118), (-110, -90)])
@pytest.mark.parametrize("n,G", ONE + FEW + MANY)
def test_queries_and_keys_without_a_common_channel(n, G, qe, ke):
    """Scores of exactly 0, whatever the sizes; some queries are zeros."""
    T, d = n + 100, 64
    k, v, q = normal(30, T, d) * 2.0 ** ke, normal(31, T, d), normal(32, n, G, d) * 2.0 ** qe
    k, q = np.clip(k, -3e38, 3e38), np.clip(q, -3e38, 3e38)
    k[:, ::2] = 0
    q[:, :, 1::2] = 0
    q[-16:, ::2] = 0
    close(Hand(k, v, q, "int8" if ke % 4 else "e4m3").run())
