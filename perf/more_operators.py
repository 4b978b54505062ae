"""Cases, plain forms and 64-bit definitions of the operators around the 8-bit cache.

Operators: appending new keys and values to a cache held in 8 bits, the position rotation applied
to the keys on the way (append); attention of one or several new tokens over that cache, queries
rotated on the way (attend); the same where a token sees the last `window` tokens and the `sinks`
first ones (window).

The cache: tiles of 64 slots, [B][Hkv][capacity/64] or [n_pages][Hkv].  Codes of a tile
[loops][2][64][d] bytes, K before V, the 16-byte chunk c of row t at chunk position
c ^ (t & 7) (d = 128) or c ^ (t / 2 & 3) (d = 64).  A scale, a power of two, for every block of 16
slots: [loops][2][4] fp32 a tile.  A code is e4m3 or int8, its value is code * scale.
"""

import math

import torch

own = False

TILE, BLOCK = 64, 16
MOST = {"e4m3": 448.0, "int8": 127.0}    # the largest code
LEAST = -100                             # exponent of the smallest scale


# ------------------------------------------------------------------------------ cases

def _append(name, batch, kv_heads, head_dim, fmt, loops, ctx, n_new, rot=0, interleaved=False,
            ragged=False, paged=False):
    return {"name": name, "op": "append", "batch": batch, "kv_heads": kv_heads, "head_dim": head_dim,
            "fmt": fmt, "loops": loops, "ctx": ctx, "n_new": n_new, "rot": rot,
            "interleaved": interleaved, "ragged": ragged, "paged": paged}


def _attend(name, batch, q_heads, kv_heads, head_dim, fmt, ctx, n_new, window=0, sinks=0, rot=0,
            interleaved=False, ragged=False, paged=False):
    return {"name": name, "op": "window" if window else "attend", "batch": batch, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "fmt": fmt, "loops": 1, "ctx": ctx,
            "n_new": n_new, "window": window, "sinks": sinks, "rot": rot, "interleaved": interleaved,
            "ragged": ragged, "paged": paged}


def listed():
    return [
        # the step of one sequence of the smallest model: latency
        _append("append_step_small", 1, 2, 64, "int8", 1, 250, 1, rot=64),
        # the step of a batch on a paged cache: most blocks are half full, some scales rise
        _append("append_step_paged", 64, 8, 128, "e4m3", 1, 1000, 1, rot=128, ragged=True, paged=True),
        # prompts of unequal lengths, four loops at once, half the channels rotated
        _append("append_prompt", 4, 16, 128, "int8", 4, 5, 1023, rot=64, interleaved=True, ragged=True),
        # a decode step of one sequence of the smallest model: latency
        _attend("decode_small", 1, 2, 2, 64, "e4m3", 256, 1),
        # a decode step of an ordinary batch, a query head for every kv-head
        _attend("decode_batch", 16, 16, 16, 128, "e4m3", 4096, 1, rot=128),
        # long contexts of unequal lengths on a paged cache, grouped-query heads
        _attend("decode_long_paged", 16, 32, 8, 128, "int8", 16384, 1, rot=128, ragged=True, paged=True),
        # verification of eight drafted tokens, grouped-query heads
        _attend("verify_gqa", 8, 32, 8, 128, "e4m3", 16384, 8),
        # prompts' first chunks, a padded batch of unequal ones
        _attend("first_chunk", 4, 16, 16, 128, "e4m3", 0, 1023, rot=128, ragged=True),
        # a long prompt's late chunk, grouped-query heads
        _attend("late_chunk", 1, 32, 8, 128, "int8", 14336, 2048, rot=128),
        # a decode step far beyond the window: pages between the sinks and the window are gone
        _attend("window_decode_paged", 64, 32, 8, 128, "e4m3", 30000, 1, window=4096, sinks=4, rot=128,
                ragged=True, paged=True),
        # a few rows of an odd shape: five query heads to a kv-head, short window, many sinks
        _attend("window_verify_odd", 3, 15, 3, 64, "int8", 3001, 17, window=1001, sinks=130, rot=32,
                interleaved=True),
        # a chunk of a prompt much longer than the window
        _attend("window_chunk", 2, 32, 8, 128, "e4m3", 20000, 2000, window=4096, sinks=64),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    most = max(_cost(c) for c in listed())
    while True:
        batch, kv, d = log(1, 64), rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([64, 128, 128])
        fmt, ragged, paged = rng.choice(["e4m3", "int8"]), rng.random() < 0.5, rng.random() < 0.4
        rot, turned = rng.choice([0, d // 2, d, d]), rng.random() < 0.3
        n, ctx = rng.choice([1, log(1, 64), log(1, 2048)]), rng.choice([0, log(1, 32768), log(64, 32768)])
        if rng.random() < 0.3:
            c = _append("", batch, kv, d, fmt, rng.randint(1, 4), min(ctx, 4096), n, rot, turned, ragged, paged)
        else:
            window = rng.choice([0, log(1, 8192)])
            c = _attend("", batch, kv * rng.choice([1, 1, 2, 4, 5, 8]), kv, d, fmt, ctx, n, window,
                        rng.choice([0, log(1, 256)]) if window else 0, rot, turned, ragged, paged)
        del c["name"]
        if _cost(c) <= most:
            return c


def _cost(c):
    # bytes, operations at 1/300 of a byte's price, and what the plain form makes of codes and scores
    w = work(c)
    cells = c["batch"] * c["kv_heads"] * c["head_dim"] * c["loops"] * 2
    if c["op"] == "append":
        return w["bytes"] + cells * (c["n_new"] + (c["ctx"] + c["n_new"]) / 4)
    seen = max(len(t) for t in _tiles(c)) * TILE
    return w["bytes"] + w["flops"] / 300 + 2 * cells * seen + c["batch"] * c["q_heads"] * c["n_new"] * seen


def _ctx_lens(c):
    """Cached tokens of each sequence before the new ones (part of the case, not of the seed)."""
    n = c["ctx"]
    return [n - (b * 2654435761 % (n // 3 + 1) if c["ragged"] and b else 0) for b in range(c["batch"])]


def _new_lens(c):
    """New tokens of each sequence."""
    n = c["n_new"]
    return [n - (b * 40503 % (n // 2 + 1) if c["ragged"] and b else 0) for b in range(c["batch"])]


def _sees(c, ctx, j):
    """Slot ranges [lo, hi) that new token j sees: the sinks apart from the window, and the window."""
    hi = ctx + j + 1
    lo = max(0, hi - c["window"]) if c["window"] else 0
    return (0, min(c["sinks"], lo)), (lo, hi)


def _tiles(c):
    """Tiles of 64 slots that some new token of each sequence sees."""
    found = []
    for ctx, n in zip(_ctx_lens(c), _new_lens(c)):
        (_, sink), (lo, _) = _sees(c, ctx, 0)
        sink = max(sink, min(c.get("sinks", 0), _sees(c, ctx, n - 1)[1][0]))
        found.append(sorted(set(range(-(-sink // TILE))) | set(range(lo // TILE, -(-(ctx + n) // TILE)))))
    return found


def work(case):
    c = case
    ctx, new, H, d = _ctx_lens(c), _new_lens(c), c["kv_heads"], c["head_dim"]
    if c["op"] == "append":
        turns = sum(new) * c["rot"] // 2 * 8 if c["rot"] else 0
        blocks = sum(-(-(x + n) // BLOCK) - x // BLOCK for x, n in zip(ctx, new))
        return {"bytes": 2 * c["loops"] * H * (3 * d * sum(new) + 4 * blocks) + turns,
                "flops": 2 * c["loops"] * H * d * sum(new) * 4}
    slots, pairs = 0, 0
    for x, n in zip(ctx, new):
        (_, s0), (lo, _) = _sees(c, x, 0)
        late = _sees(c, x, n - 1)[1][0]
        slots += x + n - lo + max(s0, min(c["sinks"], lo, late))
        for j in range(n):
            (_, s), (a, b) = _sees(c, x, j)
            pairs += b - a + s
    return {"bytes": H * slots * 2 * d + H * slots // BLOCK * 8 + sum(new) * c["q_heads"] * d * 4,
            "flops": 4 * d * c["q_heads"] * pairs}


# ------------------------------------------------------------------------------ inputs

def _exponent(amax, fmt):
    """The least e with amax <= MOST 2^e, at least LEAST; amax rounded to bf16 first, so that the
    last bits of a rotation decide nothing."""
    top, k = math.frexp(MOST[fmt])
    m, x = torch.frexp(amax.bfloat16().float())
    e = x - k + (m > top).to(x.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, LEAST)).clamp(min=LEAST)


def _round(x, fmt):
    """fp32 code units -> bytes (round to nearest, ties to even)."""
    if fmt == "int8":
        return x.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _units(codes, fmt):
    """Bytes -> fp32 code units."""
    return codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float()


def _chunk_places(d, device):
    """Stored position of each 16-byte chunk of each row of a tile: [64][d / 16]."""
    t = torch.arange(TILE, device=device).view(-1, 1)
    return torch.arange(d // 16, device=device).view(1, -1) ^ ((t & 7) if d == 128 else (t // 2 & 3))


def _swap(x, places):
    """Chunks of the rows [..., rows, d] moved between natural and stored order (its own inverse)."""
    y = x.unflatten(-1, (-1, 16))
    return y.gather(-2, places.unsqueeze(-1).expand(y.shape)).flatten(-2)


def _states(gen, shape, d, device):
    """Keys or values: two outlier channels of each head, sizes that differ by token."""
    B, H, T = shape
    scale = torch.ones(1, H, 1, d, device=device)
    scale.scatter_(3, torch.rand(1, H, 1, d, generator=gen, device=device).topk(2, 3).indices, 8.0)
    u = torch.exp(0.3 * torch.randn(B, H, T, 1, generator=gen, device=device))
    return torch.randn(B, H, T, d, generator=gen, device=device) * scale * u


def _fill(c, gen, tiles, device):
    """Tiles of one sequence, every slot filled: codes [tiles][H][L][2][64][d], scales [...][4]."""
    H, L, d, fmt = c["kv_heads"], c["loops"], c["head_dim"], c["fmt"]
    codes = torch.empty(tiles, H, L, 2, TILE, d, dtype=torch.uint8, device=device)
    scales = torch.empty(tiles, H, L, 2, TILE // BLOCK, device=device)
    places = _chunk_places(d, device)
    for l in range(L):
        for kv in (0, 1):
            x = _states(gen, (1, H, tiles * TILE), d, device).bfloat16().float().view(H, tiles, TILE // BLOCK, BLOCK, d)
            e = _exponent(x.abs().amax((-1, -2)), fmt)
            by = _round(torch.ldexp(x, -e[..., None, None]), fmt).view(H, tiles, TILE, d)
            codes[:, :, l, kv] = _swap(by, places).transpose(0, 1)
            scales[:, :, l, kv] = torch.ldexp(torch.ones((), device=device), e).transpose(0, 1)
    return codes, scales


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    B, H, L, d, n = c["batch"], c["kv_heads"], c["loops"], c["head_dim"], c["n_new"]
    ctx, new = _ctx_lens(c), _new_lens(c)
    cap = max(-(-(x + n) // TILE) for x in ctx) * TILE
    s = {"case": c, "cap": cap, "max_ctx": max(ctx),
         "ctx": torch.tensor(ctx, dtype=torch.int32, device=dev),
         "new": torch.tensor(new, dtype=torch.int32, device=dev), "places": _chunk_places(d, dev)}
    if c["op"] == "append":      # only the tile that takes the first new token holds older rows
        tiles = [sorted({x // TILE} | set(range(x // TILE, -(-(x + m) // TILE)))) for x, m in zip(ctx, new)]
    else:
        tiles = _tiles(c)
    # the tiles that hold something, one sequence after the other, in a pool or at their places
    n_pages = sum(len(t) for t in tiles) + 5
    if c["paged"]:
        order = torch.randperm(n_pages, generator=gen, device=dev)
        codes = torch.zeros(n_pages, H, L, 2, TILE, d, dtype=torch.uint8, device=dev)
        scales = torch.ones(n_pages, H, L, 2, TILE // BLOCK, device=dev)
        table = torch.full((B, cap // TILE), -1, dtype=torch.int32, device=dev)   # (-1: no page)
    else:
        codes = torch.zeros(B, H, cap // TILE, L, 2, TILE, d, dtype=torch.uint8, device=dev)
        scales = torch.ones(B, H, cap // TILE, L, 2, TILE // BLOCK, device=dev)
    at = 0
    for b, t in enumerate(tiles):
        held = torch.tensor(t, device=dev)
        x, y = _fill(c, gen, len(t), dev)
        if c["op"] == "append" and ctx[b] % TILE == 0:
            x.zero_()
        if c["paged"]:
            pages = order[at:at + len(t)]
            table[b, held] = pages.int()
            codes[pages], scales[pages] = x, y
        else:
            codes[b][:, held], scales[b][:, held] = x.transpose(0, 1), y.transpose(0, 1)
        at += len(t)
    s["codes"], s["scales"] = codes, scales
    if c["paged"]:
        s["table"], s["n_pages"] = table, n_pages
    if c["rot"]:
        half = c["rot"] // 2
        angle = torch.arange(cap, dtype=torch.float64, device=dev).view(-1, 1) * \
            10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        s["rope"] = torch.stack([angle.cos(), angle.sin()], -1).float()            # [cap][rot / 2][2]
    if c["op"] == "append":
        x = torch.stack([_states(gen, (B, H, n * L), d, dev) for _ in range(2)], 1)
        s["kv_new"] = x.view(B, 2, H, n, L, d).permute(0, 3, 1, 4, 2, 5).contiguous().bfloat16()
        return s
    s["q"] = torch.randn(B, n, c["q_heads"], d, generator=gen, device=dev).bfloat16()
    s["out"] = torch.zeros(B, n, c["q_heads"], d, dtype=torch.bfloat16, device=dev)
    most = max(len(t) for t in tiles)                    # constants of the plain form: tiles it gathers
    s["tiles"] = torch.tensor([t + [-1] * (most - len(t)) for t in tiles], device=dev)
    return s


# ------------------------------------------------------------------------------ one pass

def run(state):
    s = state
    if own:
        return _own_append(s) if s["case"]["op"] == "append" else _own_attend(s)
    return _plain_append(s) if s["case"]["op"] == "append" else _plain_attend(s)


def _handles(s):
    """The shape, cache and rotation handles that a program keeps for its buffers."""
    import looped_transformer_kv_gb300 as rq
    c = s["case"]
    shape = rq.make_q8_shape(c["batch"], c.get("q_heads", c["kv_heads"]), c["kv_heads"], c["head_dim"],
                             c["loops"], s["cap"], c["fmt"])
    cache = rq.Q8Cache(shape, n_pages=s["n_pages"] if c["paged"] else None, codes=s["codes"].view(-1),
                       scales=s["scales"].view(-1))
    rope = rq.make_rope(s["rope"], interleaved=c["interleaved"]) if c["rot"] else None
    paging = rq.make_paging(s["table"], s["n_pages"]) if c["paged"] else None
    if c["op"] != "append":
        need = rq.q8_workspace_bytes(shape, c["n_new"], s["max_ctx"], c["window"], c["sinks"])
        s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    s["handle"] = shape, cache, rope, paging
    return s["handle"]


def _own_append(s):
    import looped_transformer_kv_gb300 as rq
    c = s["case"]
    shape, cache, rope, paging = s.get("handle") or _handles(s)
    more = {"n_lens": s["new"] if c["ragged"] else None, "rope": rope}
    if c["paged"]:
        rq.paged_q8_append(shape, cache, paging, s["kv_new"], 0, s["ctx"], **more)
    else:
        rq.q8_append(shape, cache, s["kv_new"], 0, s["ctx"], **more)
    return _held(s)


def _own_attend(s):
    import looped_transformer_kv_gb300 as rq
    c = s["case"]
    shape, cache, rope, paging = s.get("handle") or _handles(s)
    args = (s["q"], 0, s["ctx"], s["max_ctx"], s["out"], s["ws"])
    more = {"n_lens": s["new"] if c["ragged"] else None, "window": c["window"], "n_sink": c["sinks"], "rope": rope}
    if c["paged"]:
        rq.paged_q8_attention(shape, cache, paging, *args, **more)
    else:
        rq.q8_attention(shape, cache, *args, **more)
    return s["out"]


def _held(s):
    """The cache as the numbers it holds."""
    kind = torch.int8 if s["case"]["fmt"] == "int8" else torch.float8_e4m3fn
    return {"codes": s["codes"].view(kind), "scales": s["scales"]}


# ------------------------------------------------------------------------------ plain forms

def _turn(x, table, pos, c):
    """The first `rot` channels of x [..., d] rotated by the angles of pos [...]; products and sums
    rounded one by one."""
    r = c["rot"]
    if not r:
        return x
    cs = table[pos]
    co, si = cs[..., 0], cs[..., 1]
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * co - b * si, b * co + a * si], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * co - b * si, b * co + a * si], -1)
    return torch.cat([y, x[..., r:]], -1)


def _plain_append(s):
    c = s["case"]
    B, H, L, d, n, fmt = c["batch"], c["kv_heads"], c["loops"], c["head_dim"], c["n_new"], c["fmt"]
    dev = s["codes"].device
    most = (n + 2 * BLOCK - 2) // BLOCK                                     # blocks that n tokens may touch
    ctx, new = s["ctx"].long(), s["new"].long()
    blocks = ctx.view(B, 1) // BLOCK + torch.arange(most, device=dev)       # [B][most]
    used = blocks * BLOCK < (ctx + new).view(B, 1)
    b, k = used.nonzero(as_tuple=True)                                      # the touched blocks, one list
    blk = blocks[b, k]
    slot = blk.view(-1, 1) * BLOCK + torch.arange(BLOCK, device=dev)        # [m][16]
    j = slot - ctx[b].view(-1, 1)
    fresh = (j >= 0) & (j < new[b].view(-1, 1))
    src = s["kv_new"][b.view(-1, 1), j.clamp(0, n - 1)].float()             # [m][16][2][L][H][d]
    pos = slot.clamp(max=s["cap"] - 1).view(*slot.shape, 1, 1).expand(*slot.shape, L, H)
    src[:, :, 0] = _turn(src[:, :, 0], s.get("rope"), pos, c)
    src = src.permute(0, 4, 3, 2, 1, 5)                                     # [m][H][L][2][16][d]
    src = torch.where(fresh.view(-1, 1, 1, 1, BLOCK, 1), src, torch.zeros_like(src))
    tile, part = blk // (TILE // BLOCK), blk % (TILE // BLOCK)
    if c["paged"]:
        codes, scales, where = s["codes"], s["scales"], (s["table"][b, tile].long(),)
    else:
        codes, scales, where = s["codes"].transpose(1, 2), s["scales"].transpose(1, 2), (b, tile)
    codes = codes.unflatten(-2, (TILE // BLOCK, BLOCK))                     # [..][H][L][2][4][16][d]
    m = torch.arange(len(b), device=dev)
    was, was_scale = codes[where][m, :, :, :, part], scales[where][m, ..., part]
    places = s["places"].view(TILE // BLOCK, BLOCK, -1)[part].view(-1, 1, 1, 1, BLOCK, d // 16)
    places = places.expand(*was.shape[:-1], d // 16)
    old = (j < 0).view(-1, 1, 1, 1, BLOCK, 1)
    had = (j[:, 0] < 0).view(-1, 1, 1, 1)
    e_new = _exponent(src.abs().amax((-1, -2)), fmt)
    e_old = torch.frexp(was_scale)[1] - 1
    e = torch.where(had, torch.maximum(e_old, e_new), e_new)
    x = torch.ldexp(src, -e[..., None, None])
    kept = torch.ldexp(_units(_swap(was, places), fmt), (e_old - e)[..., None, None])
    by = _round(torch.where(old, kept, x), fmt)
    live = old | fresh.view(-1, 1, 1, 1, BLOCK, 1)
    by = torch.where(live, _swap(by, places), was)
    at = (where[0].view(-1, 1, 1, 1), torch.arange(H, device=dev).view(1, -1, 1, 1)) if c["paged"] else \
        (where[0].view(-1, 1, 1, 1), where[1].view(-1, 1, 1, 1), torch.arange(H, device=dev).view(1, -1, 1, 1))
    at += (torch.arange(L, device=dev).view(1, 1, -1, 1), torch.arange(2, device=dev).view(1, 1, 1, -1),
           part.view(-1, 1, 1, 1))
    codes[at] = by
    scales[at] = torch.ldexp(torch.ones((), device=dev), e)
    return _held(s)


def _gather(s, kv):
    """K or V of the tiles that are seen, 32 bits: [B][H][tiles * 64][d]."""
    c, t = s["case"], s["tiles"].clamp(min=0)
    b = torch.arange(c["batch"], device=t.device).view(-1, 1)
    if c["paged"]:
        at = s["table"][b, t].long().clamp(min=0)
        codes, scales = s["codes"][at, :, 0, kv], s["scales"][at, :, 0, kv]
    else:
        codes, scales = s["codes"].transpose(1, 2)[b, t, :, 0, kv], s["scales"].transpose(1, 2)[b, t, :, 0, kv]
    x = _units(_swap(codes.transpose(1, 2), s["places"].view(1, 1, 1, TILE, -1)
                     .expand(codes.shape[0], codes.shape[2], codes.shape[1], -1, -1)), c["fmt"])
    x = x.unflatten(-2, (TILE // BLOCK, BLOCK)) * scales.transpose(1, 2)[..., None, None]
    return x.flatten(2, 4)


def _plain_attend(s):
    c = s["case"]
    B, H, d, n = c["batch"], c["kv_heads"], c["head_dim"], c["n_new"]
    G, dev = c["q_heads"] // H, s["q"].device
    j = torch.arange(n, device=dev)
    at = s["ctx"].long().view(B, 1) + j                                     # slot of each new token
    q = _turn(s["q"].float(), s.get("rope"), at.clamp(max=s["cap"] - 1).unsqueeze(-1).expand(B, n, H * G), c)
    q = q.view(B, n, H, G, d).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, d)
    t = s["tiles"]
    slot = (t.unsqueeze(-1) * TILE + torch.arange(TILE, device=dev)).flatten(1).unsqueeze(1)   # [B][1][T]
    there = t.repeat_interleave(TILE, 1).unsqueeze(1) >= 0
    T = slot.shape[-1]
    mask = there & (slot <= at.unsqueeze(-1))                               # [B][n][T]
    if c["window"]:
        mask &= (slot > at.unsqueeze(-1) - c["window"]) | (slot < c["sinks"])
    k = _gather(s, 0)
    x = (q @ k.transpose(2, 3)).view(B, H, G, n, T).mul_(1 / math.sqrt(d))
    del k
    x.masked_fill_(~mask.view(B, 1, 1, n, T), -math.inf)
    x -= x.amax(-1, keepdim=True)
    p = x.exp_()
    p /= p.sum(-1, keepdim=True)
    out = (p.view(B, H, G * n, T) @ _gather(s, 1)).view(B, H, G, n, d).permute(0, 3, 1, 2, 4).reshape(B, n, H * G, d)
    valid = j.view(1, n) < s["new"].view(B, 1)
    s["out"].copy_(torch.where(valid.view(B, n, 1, 1), out.bfloat16(), s["out"]))
    return s["out"]


# ------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """What run returns, from the definitions in 64 bits, each element found by its address."""
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)


def _exact_turn(s, x, pos, c):
    """Rotation of the rows x [..., m, d] at the positions pos [m], by complex numbers."""
    r = c["rot"]
    if not r:
        return x
    w = torch.view_as_complex(s["rope"][pos].double().contiguous())         # [m][r / 2]
    i = torch.arange(r, device=x.device)
    first, second = (i[0::2], i[1::2]) if c["interleaved"] else (i[:r // 2], i[r // 2:])
    z = torch.complex(x[..., first], x[..., second]) * w
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _byte_at(t, ch, d):
    """Place of channel ch of slot t of its tile among the tile's bytes of one loop and K or V."""
    r = t % TILE
    turn = r % 8 if d == 128 else r // 2 % 4
    return r * d + ((ch // 16) ^ turn) * 16 + ch % 16


def _exact_append(s):
    c = s["case"]
    d, L, H, fmt = c["head_dim"], c["loops"], c["kv_heads"], c["fmt"]
    codes = _units(s["codes"], fmt).double()
    scales = s["scales"].double()
    ch = torch.arange(d, device=codes.device)
    for b, (ctx, m) in enumerate(zip(_ctx_lens(c), _new_lens(c))):
        x = s["kv_new"][b, :m].double().permute(1, 2, 3, 0, 4).contiguous()  # [2][L][H][m][d]
        x[0] = _exact_turn(s, x[0], torch.arange(ctx, ctx + m, device=x.device), c)
        for k in range(ctx // BLOCK, -(-(ctx + m) // BLOCK)):
            t = torch.arange(max(ctx, k * BLOCK), min(ctx + m, (k + 1) * BLOCK), device=x.device)
            before = torch.arange(k * BLOCK, max(k * BLOCK, min(ctx, (k + 1) * BLOCK)), device=x.device)
            tile, part = k // 4, k % 4
            if c["paged"]:
                page = int(s["table"][b, tile])
                tile_codes, tile_scales = codes[page], scales[page]
            else:
                tile_codes, tile_scales = codes[b, :, tile], scales[b, :, tile]
            rows = x[:, :, :, t - ctx].permute(2, 1, 0, 3, 4)                # [H][L][2][t][d]
            biggest = _to_bf16(rows.abs().amax((-1, -2)))
            e = torch.ceil(torch.log2(biggest.clamp(min=1e-300) / MOST[fmt]))
            e -= (biggest <= MOST[fmt] * torch.exp2(e - 1)).double()         # (the logarithm may be a bit off)
            e += (biggest > MOST[fmt] * torch.exp2(e)).double()
            e = e.clamp(min=LEAST)
            if len(before):
                e = torch.maximum(e, torch.log2(tile_scales[..., part]))
            step = torch.exp2(e)
            flat = tile_codes.flatten(-2).clone()                            # [H][L][2][64 d]
            if len(before):
                at = _byte_at(before.view(-1, 1), ch.view(1, -1), d).flatten()
                flat[..., at] = _nearest(flat[..., at] * (tile_scales[..., part] / step).unsqueeze(-1), fmt)
            at = _byte_at(t.view(-1, 1), ch.view(1, -1), d).flatten()
            flat[..., at] = _nearest(rows.flatten(-2) / step.unsqueeze(-1), fmt)
            tile_codes.copy_(flat.view(tile_codes.shape))
            tile_scales[..., part] = step
    return {"codes": codes, "scales": scales}


def _nearest(x, fmt):
    """The nearest number that a code can hold, ties to even."""
    if fmt == "int8":
        return x.round().clamp(-127, 127)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return ((x / step).round() * step).clamp(-448, 448)


def _to_bf16(x):
    """The nearest number of 8 significant bits, ties to even."""
    m, e = torch.frexp(x)
    return torch.ldexp((m * 256).round() / 256, e)


def _exact_attend(s):
    c = s["case"]
    H, d = c["kv_heads"], c["head_dim"]
    G, dev = c["q_heads"] // H, s["q"].device
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    ch = torch.arange(d, device=dev)
    for b, (ctx, m) in enumerate(zip(_ctx_lens(c), _new_lens(c))):
        at = ctx + torch.arange(m, device=dev)
        q = _exact_turn(s, s["q"][b, :m].double().transpose(0, 1), at, c)    # [Hq][m][d]
        (_, sink), (lo, _) = _sees(c, ctx, 0)
        sink = min(c["sinks"], _sees(c, ctx, m - 1)[1][0]) if c["window"] else 0
        t = torch.cat([torch.arange(min(sink, lo), device=dev), torch.arange(lo, ctx + m, device=dev)])
        unseen = t.view(1, -1) > at.view(-1, 1)
        if c["window"]:
            unseen |= (t.view(1, -1) <= at.view(-1, 1) - c["window"]) & (t.view(1, -1) >= c["sinks"])
        byte = _byte_at(t.view(-1, 1), ch.view(1, -1), d)
        for h in range(H):
            rows = []
            for kv in (0, 1):
                if c["paged"]:
                    page = s["table"][b].long()[t // TILE]
                    codes, scale = s["codes"][:, h, 0, kv], s["scales"][:, h, 0, kv]
                else:
                    page, codes, scale = t // TILE, s["codes"][b, h, :, 0, kv], s["scales"][b, h, :, 0, kv]
                x = _units(codes.flatten(1)[page.view(-1, 1), byte], c["fmt"]).double()
                rows.append(x * scale[page, t % TILE // BLOCK].double().view(-1, 1))
            for g in range(G):
                x = q[h * G + g] @ rows[0].T / math.sqrt(d)
                x[unseen] = -math.inf
                out[b, :m, h * G + g] = torch.softmax(x, -1) @ rows[1]
    return out
