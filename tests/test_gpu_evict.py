"""Eviction by accumulated attention weight, on the GPU: the choice of slots and the move of rows
against host references, exactly; then a run of prompt chunks, eviction and decode steps."""

import itertools

import numpy as np
import pytest

import chunk_reference as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from looped_transformer_kv_gb300 import rq


def _select(w, ctx, budget, first=0, last=0):
    B, H, _ = w.shape
    keep = torch.full((B, H, budget), -7, dtype=torch.int32, device="cuda")
    kept = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    rq.evict_select(w.cuda(), torch.tensor(ctx, dtype=torch.int32).cuda(), budget, keep, kept,
                    n_first=first, n_last=last)
    torch.cuda.synchronize()
    return keep.cpu().numpy(), kept.cpu().numpy()


def _check_select(w, ctx, budget, first=0, last=0):
    keep, kept = _select(w, ctx, budget, first, last)
    for b, n in enumerate(ctx):
        assert kept[b] == min(n, budget)
        for h in range(w.shape[1]):
            want = R.select(w[b, h].numpy(), n, min(n, budget), first, last)
            assert keep[b, h, :kept[b]].tolist() == want, (b, h)
            assert (keep[b, h, kept[b]:] == -7).all()


@pytest.mark.parametrize("ctx,budget,first,last", [
    ([1, 0, 2], 1, 0, 0), ([5, 3, 4], 3, 1, 1), ([33, 31, 32], 8, 0, 0), ([64, 64, 64], 64, 4, 4),
    ([511, 513, 700], 300, 4, 64), ([4097, 4000, 100], 1024, 0, 1024), ([1000, 999, 998], 999, 0, 0),
    ([9000, 9001, 8999], 1, 0, 0), ([9000, 1, 17], 40, 40, 0),
])
@pytest.mark.parametrize("kind", ["spread", "equal", "few"])
def test_select(ctx, budget, first, last, kind):
    g = torch.Generator().manual_seed(len(kind) + budget)
    cap = max(ctx) + 11
    w = torch.exp(3 * torch.randn(3, 2, cap, generator=g))
    if kind == "equal":
        w.fill_(0.25)
    elif kind == "few":      # many ties
        w = torch.randint(0, 3, w.shape, generator=g).float() * 0.5
    _check_select(w, ctx, budget, first, last)


def test_select_special_values():
    inf, nan = float("inf"), float("nan")
    row = [0.0, -0.0, 1.0, nan, inf, -1.0, -inf, 1.0, 5e-45, -nan, 0.0, 3e38]
    w = torch.tensor([[row * 3]])
    for budget in range(1, 36):
        _check_select(w, [36], budget)
        _check_select(w, [36], budget, min(2, budget), min(3, budget - min(2, budget)))


@pytest.mark.parametrize("n,heads", [(20000, 1), (70001, 2), (50000, 160), (400100, 1)])
def test_select_long_rows(n, heads):
    g = torch.Generator().manual_seed(n)
    w = (torch.randn(1, heads, n + 3, generator=g) * 64).round() / 64
    budget = n // 3
    keep, kept = _select(w, [n], budget, 3, 100)
    assert kept[0] == budget
    x = w[0, :, :n].numpy().astype(np.float64)
    x[:, :3] = x[:, n - 100:] = np.inf
    for h in range(0, heads, max(1, heads // 5)):
        want = np.sort(np.argsort(-x[h], kind="stable")[:budget])
        assert (keep[0, h] == want).all()


def test_select_marks_a_length_out_of_range():
    w = torch.rand(3, 1, 64)
    keep, kept = _select(w, [65, -1, 10], 5)
    assert kept.tolist() == [-1, -1, 5]
    assert (keep[:2] == -7).all()


# ---------------------------------------------------------------------------------- compact

def _cache(B, H, d, bits, cap, seed, paged=False, spare=3):
    """A cache of random bytes: the move looks at none of them."""
    g = torch.Generator().manual_seed(seed)
    shape = rq.make_shape(B, H, H, d, len(bits) + 1, cap, bits)
    signs = torch.ones(2, H, d)
    n_pages = B * (cap // 64) + spare if paged else None
    c = rq.PackedCache(shape, signs, n_pages=n_pages)
    c.data.copy_(torch.randint(0, 256, c.data.shape, generator=g, dtype=torch.uint8))
    table = paging = None
    if paged:
        table = torch.randperm(n_pages, generator=g)[:B * (cap // 64)].int().view(B, -1).cuda()
        paging = rq.make_paging(table, n_pages)
    return shape, c, table, paging


def _tokens(c, table, b, h, d, bits, rows):
    rec = c.records()
    rec = (rec[table[b].long(), h] if table is not None else rec[b, h]).cpu().numpy()
    return [R.token_bytes(rec[t // 64], t % 64, d, bits).tobytes() for t in rows]


COMPACT = [
    # d, bits, cap, to_cap, budget, kept
    (128, (2, 2, 2), 256, 128, 100, [100, 37]),
    (128, (), 128, 64, 64, [64, 0]),
    (64, (2, 4), 1280, 704, 700, [700, 65]),
    (128, (4, 2), 64, 64, 1, [1, 1]),
    (128, (2,) * 15, 192, 192, 192, [192, 130]),
    (64, (), 192, 128, 127, [127, 3]),
]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", range(len(COMPACT)))
def test_compact(case, in_place, paged):
    d, bits, cap, to_cap, budget, kept = COMPACT[case]
    B, H = 2, 3
    if in_place:
        to_cap = cap
    shape, src, table, paging = _cache(B, H, d, bits, cap, case, paged)
    w = torch.rand(B, H, cap).cuda()
    if in_place:
        to_shape, to, to_table, to_paging, to_w = shape, src, table, paging, w
    else:
        to_shape, to, to_table, to_paging = _cache(B, H, d, bits, to_cap, case + 50, paged)
        to_w = torch.rand(B, H, to_cap).cuda()
    rng = np.random.default_rng(case)
    keep = np.full((B, H, budget), 10 ** 6, np.int32)
    for b, h in itertools.product(range(B), range(H)):
        keep[b, h, :kept[b]] = np.sort(rng.choice(cap, kept[b], replace=False))
        if (b, h) == (0, 1):
            keep[b, h, :kept[b]] = np.arange(kept[b])     # nothing moves
    want, behind = {}, {}
    for b, h in itertools.product(range(B), range(H)):
        want[b, h] = _tokens(src, table, b, h, d, bits, keep[b, h, :kept[b]])
        behind[b, h] = _tokens(to, to_table, b, h, d, bits, range(kept[b], to_cap))
    w_old, pool_old = w.clone().cpu().numpy(), to.data.clone()
    args = (torch.from_numpy(keep).cuda(), torch.tensor(kept, dtype=torch.int32).cuda(), w, to_w)
    if paged:
        rq.paged_evict_compact(shape, src, paging, to_shape, to, to_paging, *args)
    else:
        rq.evict_compact(shape, src, to_shape, to, *args)
    torch.cuda.synchronize()
    got_w = to_w.cpu().numpy()
    for b, h in itertools.product(range(B), range(H)):
        assert _tokens(to, to_table, b, h, d, bits, range(kept[b])) == want[b, h], (b, h)
        assert _tokens(to, to_table, b, h, d, bits, range(kept[b], to_cap)) == behind[b, h], (b, h)
        assert (got_w[b, h, :kept[b]] == w_old[b, h, keep[b, h, :kept[b]]]).all()
        assert (got_w[b, h, kept[b]:] == 0).all()
    if paged:      # pages of no sequence are untouched
        free = torch.ones(to_paging.n_pages, dtype=torch.bool)
        free[to_table.cpu().long().view(-1)] = False
        old = pool_old.view(to_paging.n_pages, -1).cpu()
        assert torch.equal(to.data.view(to_paging.n_pages, -1).cpu()[free], old[free])


def test_compact_to_other_pages_of_one_pool():
    """Two sequences share their pages; each gets its own, in the same pool."""
    d, bits, H, cap, budget = 128, (2, 4), 2, 256, 100
    shape, pool, _, _ = _cache(2, H, d, bits, cap, 9, paged=True, spare=4)      # 12 pages
    table = torch.tensor([[3, 0, 7, 5]] * 2, dtype=torch.int32).cuda()
    to_table = torch.tensor([[1, 11], [8, 2]], dtype=torch.int32).cuda()
    to_shape = rq.make_shape(2, H, H, d, 3, 128, bits)
    rng = np.random.default_rng(9)
    keep = np.stack([[np.sort(rng.choice(cap, budget, replace=False)) for _ in range(H)] for _ in range(2)])
    want = {(b, h): _tokens(pool, table, b, h, d, bits, keep[b, h]) for b in range(2) for h in range(H)}
    old = pool.data.clone().view(12, -1)
    rq.paged_evict_compact(shape, pool, rq.make_paging(table, 12), to_shape, pool, rq.make_paging(to_table, 12),
                           torch.from_numpy(keep.astype(np.int32)).cuda(),
                           torch.tensor([budget, 65], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    for b, n in ((0, budget), (1, 65)):
        for h in range(H):
            assert _tokens(pool, to_table, b, h, d, bits, range(n)) == want[b, h][:n], (b, h)
    rest = [p for p in range(12) if p not in (1, 11, 8, 2)]
    assert torch.equal(pool.data.view(12, -1)[rest], old[rest])


@pytest.mark.parametrize("in_place", [False, True])
def test_entries_out_of_range_move_nothing(in_place):
    d, bits = 128, (2,)
    shape, src, table, paging = _cache(1, 1, d, bits, 128, 3, paged=True)
    to_shape, to, to_table, to_paging = (shape, src, table, paging) if in_place else \
        _cache(1, 1, d, bits, 128, 4, paged=True)
    keep = torch.tensor([[[5, 9, -1, 128, 2 ** 30, 100]]], dtype=torch.int32).cuda()
    before = _tokens(to, to_table, 0, 0, d, bits, range(128))
    want = _tokens(src, table, 0, 0, d, bits, [5, 9, 100])
    bad = table.clone()
    rq.paged_evict_compact(shape, src, paging, to_shape, to, to_paging, keep,
                           torch.tensor([6], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    got = _tokens(to, to_table, 0, 0, d, bits, range(128))
    assert got[:2] == want[:2] and got[5] == want[2]
    assert got[2:5] == before[2:5] and got[6:] == before[6:]
    bad[0, 0] = -5                            # a source page out of range: its rows stay
    paging = rq.make_paging(bad, paging.n_pages)
    shape2, to2, to2_table, to2_paging = _cache(1, 1, d, bits, 128, 5, paged=True)
    before = _tokens(to2, to2_table, 0, 0, d, bits, range(128))
    rq.paged_evict_compact(shape, src, paging, shape2, to2, to2_paging, keep,
                           torch.tensor([1000], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    got = _tokens(to2, to2_table, 0, 0, d, bits, range(128))
    assert got[:5] == before[:5] and got[5] == _tokens(src, table, 0, 0, d, bits, [100])[0]


# ---------------------------------------------------------------------------------- together

@pytest.mark.parametrize("Hq,H,bits", [(2, 2, (2, 2)), (8, 2, (4,))])
def test_prompt_eviction_and_decode(Hq, H, bits):
    """A prompt in chunks, its collected weights, eviction in place, then decode steps over what is
    left: every output against the 64-bit reference over the kept rows."""
    B, d, L, cap, budget = 2, 128, len(bits) + 1, 512, 150
    g = torch.Generator().manual_seed(5)
    signs = torch.randint(0, 2, (2, H, d), generator=g) * 2 - 1
    shape = rq.make_shape(B, Hq, H, d, L, cap, bits)
    cache = rq.PackedCache(shape, signs)
    weights = torch.zeros(B, H, cap, device="cuda")
    ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens, done = [300, 211], [0, 0]
    x = torch.randn(B, 320, 2, L, H, d, generator=g).bfloat16().cuda()
    q = torch.randn(B, 320, Hq, d, generator=g).bfloat16().cuda()
    step = 128
    ws = torch.empty(max(rq.chunk_workspace_bytes(shape, l, step, cap, step) for l in range(L)),
                     dtype=torch.uint8, device="cuda")
    for t in range(0, 300, step):
        n = torch.tensor([max(0, min(step, m - t)) for m in lens], dtype=torch.int32)
        xs, qs = x[:, t:t + step], q[:, t:t + step]
        xs = torch.nn.functional.pad(xs, (0,) * 9 + (step - xs.shape[1],))
        qs = torch.nn.functional.pad(qs, (0,) * 5 + (step - qs.shape[1],))
        out = torch.zeros_like(qs)
        for l in range(L):
            rq.chunk_attention(shape, cache, qs, l, xs, ctx, cap, out, ws, n_lens=n.cuda(),
                               weights=weights, window=step)
            assert int(ws[:4].view(torch.int32).item()) == 0
        pos = torch.where(torch.arange(step).view(1, -1) < n.view(-1, 1),
                          torch.tensor(done).view(-1, 1) + torch.arange(step), -1).int().cuda()
        rq.encode_append(shape, cache, xs.contiguous(), positions=pos)
        done = [a + int(m) for a, m in zip(done, n)]
        ctx.copy_(torch.tensor(done, dtype=torch.int32))
    total = weights.sum(-1).cpu()          # every query of every loop weighs 1
    want = torch.tensor(lens).float().view(B, 1) * L * (Hq // H)
    assert ((total / want - 1).abs() < 1e-4).all()
    keep = torch.zeros(B, H, budget, dtype=torch.int32, device="cuda")
    kept = torch.zeros(B, dtype=torch.int32, device="cuda")
    rec_old = cache.records().cpu().numpy().copy()
    rq.evict_select(weights, ctx, budget, keep, kept, n_first=4, n_last=32)
    rq.evict_compact(shape, cache, shape, cache, keep, kept, weights, weights)
    torch.cuda.synchronize()
    assert kept.tolist() == [150, 150]
    pend = torch.randn(B, 1, 2, L, H, d, generator=g).bfloat16()
    q1 = torch.randn(B, Hq, 1, d, generator=g).bfloat16()
    dws = torch.empty(rq.decode_workspace_bytes(shape, 1, cap), dtype=torch.uint8, device="cuda")
    for l in range(L):
        out = torch.empty(B, Hq, 1, d, dtype=torch.bfloat16, device="cuda")
        rq.decode_attention(shape, cache, q1.cuda(), l, 1, pend[:, 0, :, l:l + 1].contiguous().cuda(),
                            kept, cap, out, dws)
        torch.cuda.synchronize()
        for b, h in itertools.product(range(B), range(H)):
            rows = keep[b, h].cpu().numpy()
            k, v = (np.concatenate([
                R.rebuild(rec_old[b, h], lens[b], d, bits, l, kv, signs[kv, h].numpy())[rows],
                pend[b, :, kv, l, h].double().numpy()]) for kv in (0, 1))
            G = Hq // H
            ref, p, _ = R.attend(q1[b, h * G:(h + 1) * G, 0].double().numpy()[None], k, v, 150, d ** -0.5)
            got = out[b, h * G:(h + 1) * G, 0].float().cpu().numpy()
            # (rq_decode_attention's bound: 2e-3 beyond half a bf16 step)
            assert (np.abs(got - ref[0]) <= 2e-3 + 2.0 ** -8 * np.abs(ref[0])).all()


@pytest.mark.parametrize("cap", [48640, 48641, 49152, 97792, 98304])
def test_select_at_the_ends_of_what_shared_memory_holds(cap):
    """Rows about as long as the keys of one or two CTAs."""
    g = torch.Generator().manual_seed(cap)
    w = torch.randint(0, 5000, (1, 160, cap), generator=g).float()
    budget = cap // 2
    keep, kept = _select(w, [cap], budget, 2, 5)
    assert kept[0] == budget
    x = w[0].numpy().astype(np.float64)
    x[:, :2] = x[:, cap - 5:] = np.inf
    for h in (0, 77, 159):
        assert (keep[0, h] == np.sort(np.argsort(-x[h], kind="stable")[:budget])).all()
