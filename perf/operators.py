"""Cases, plain forms and 64-bit definitions of the serving operators around the packed cache.

Operators: attention of several new tokens per sequence over the packed cache (chunk), the
choice of the cache slots to keep by accumulated attention weight (select), and the move of
their rows to the front of a cache (compact).

The packed cache is made here in plain torch, in the layout that include/rq.h states: tile
records [B][Hkv][capacity/64] (or [n_pages][Hkv]) of 64-row sections.
"""

import math

import numpy as np
import torch

own = False

TILE = 64
GROUP = 32


# ------------------------------------------------------------------------------ cases

def _chunk(name, batch, q_heads, kv_heads, head_dim, res_bits, loop, ctx, n_new, window=0,
           ragged=False, paged=False):
    return {"name": name, "op": "chunk", "batch": batch, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "res_bits": res_bits, "loop": loop, "ctx": ctx, "n_new": n_new,
            "window": window, "ragged": ragged, "paged": paged}


def _select(name, batch, kv_heads, ctx, budget, first, last, ragged=False):
    return {"name": name, "op": "select", "batch": batch, "kv_heads": kv_heads, "ctx": ctx,
            "budget": budget, "first": first, "last": last, "ragged": ragged}


def _compact(name, batch, kv_heads, head_dim, res_bits, ctx, budget, ragged=False):
    return {"name": name, "op": "compact", "batch": batch, "kv_heads": kv_heads,
            "head_dim": head_dim, "res_bits": res_bits, "ctx": ctx, "budget": budget,
            "ragged": ragged}


def listed():
    return [
        # three drafted tokens on the smallest model of the configurations: latency
        _chunk("chunk_draft_small", 1, 2, 2, 64, "222", 1, 256, 3),
        # one decode step of one loop that also collects the attention weights
        _chunk("chunk_step_weights", 16, 16, 16, 128, "222", 0, 4096, 1, window=1),
        # the same over long contexts of a paged cache, lengths differing by sequence
        _chunk("chunk_step_long_paged", 16, 16, 16, 128, "2", 0, 32768, 1, window=1, ragged=True,
               paged=True),
        # verification of eight drafted tokens, grouped-query heads
        _chunk("chunk_verify_gqa", 8, 32, 8, 128, "2222222", 2, 16384, 8),
        # a prompt's first chunk, padded batch of unequal prompts, the final loop (no residual)
        _chunk("chunk_first_ragged", 4, 16, 16, 128, "222", 3, 0, 1023, ragged=True),
        # a middle chunk whose last tokens vote on what to keep; 4-bit residuals
        _chunk("chunk_window_4bit", 2, 16, 16, 128, "422", 0, 6000, 509, window=32),
        # a long prompt's late chunk, grouped-query heads
        _chunk("chunk_prompt_gqa", 1, 32, 8, 128, "2222222", 2, 14336, 2048),
        # eviction for one short sequence: latency
        _select("select_small", 1, 2, 256, 128, 4, 32),
        # a batch of long sequences of unequal lengths
        _select("select_large", 32, 8, 16384, 4096, 4, 256, ragged=True),
        # moving the rows of one short sequence, and of a batch
        _compact("compact_small", 1, 8, 128, "2222222", 1000, 500),
        _compact("compact_large", 16, 16, 128, "222", 4096, 2048, ragged=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["chunk", "chunk", "chunk", "select", "compact"])
        batch, kv = log(1, 32), rng.choice([1, 2, 3, 4, 8, 16])
        bits = "".join(rng.choice("224") for _ in range(rng.randint(0, 7)))
        if op == "chunk":
            n = log(1, 2048)
            c = _chunk("", batch, kv * rng.choice([1, 1, 2, 4, 5, 8]), kv, rng.choice([64, 128, 128]),
                       bits, rng.randint(0, len(bits)), rng.choice([0, log(1, 32768), log(64, 32768)]),
                       n, rng.choice([0, 0, min(n, log(1, 64))]), rng.random() < 0.5,
                       rng.random() < 0.3)
        elif op == "select":
            ctx = log(2, 65536)
            budget = rng.randint(1, ctx)
            last = rng.randint(0, budget // 2)
            c = _select("", batch, kv, ctx, budget, rng.randint(0, min(8, budget - last)), last,
                        rng.random() < 0.5)
        else:
            ctx = log(2, 16384)
            c = _compact("", batch, kv, rng.choice([64, 128, 128]), bits, ctx, rng.randint(1, ctx),
                         rng.random() < 0.5)
        del c["name"]
        if _cost(c) <= most:
            return c


def _cost(c):
    w = work(c)
    # bytes, operations at 1/300 of a byte's price, and the floats of the plain form's scores
    plain = 0
    if c["op"] == "chunk":
        plain = 4 * c["batch"] * c["q_heads"] * c["n_new"] * (c["ctx"] + c["n_new"])
    return w["bytes"] + w["flops"] / 300 + plain / 4


def _ctx_lens(c):
    """Cached tokens of each sequence (part of the case, not of the seed)."""
    n = c["ctx"]
    return [n - (b * 2654435761 % (n // 3 + 1) if c["ragged"] and b else 0) for b in range(c["batch"])]


def _new_lens(c):
    """New tokens of each sequence."""
    n = c["n_new"]
    return [n - (b * 40503 % (n // 2 + 1) if c["ragged"] and b else 0) for b in range(c["batch"])]


def _bits(c):
    return [int(x) for x in c["res_bits"]]


def _row_bytes(d, bits=None):
    """Bytes of one token of one kv-head, K and V: the reference, or one loop's residual."""
    ng = d // GROUP
    return 2 * (d // 2 + 4 * ng) if bits is None else 2 * (d * bits // 8 + 4 * ng + 2)


def work(case):
    c = case
    ctx = _ctx_lens(c)
    if c["op"] == "select":
        kept = sum(min(x, c["budget"]) for x in ctx)
        return {"bytes": 4 * c["kv_heads"] * (sum(ctx) + kept), "flops": 0}
    d, H, bits = c["head_dim"], c["kv_heads"], _bits(c)
    if c["op"] == "compact":
        kept = sum(min(x, c["budget"]) for x in ctx)
        row = _row_bytes(d) + sum(_row_bytes(d, b) for b in bits)
        return {"bytes": H * kept * (2 * row + 4 + 8), "flops": 0}
    row = _row_bytes(d) + (_row_bytes(d, bits[c["loop"]]) if c["loop"] < len(bits) else 0)
    new = _new_lens(c)
    total = H * row * sum(ctx)
    total += sum(new) * (2 * 2 * c["q_heads"] * d + 2 * 2 * H * d)
    if c["window"]:
        total += 8 * H * (sum(ctx) + sum(new))
    pairs = sum(n * x + n * (n + 1) // 2 for n, x in zip(new, ctx))
    return {"bytes": total, "flops": 4 * d * c["q_heads"] * pairs}


# ------------------------------------------------------------------------------ inputs

def _sections(d, bits):
    """(offset in a record, row bytes) of each kind of rows; loop None is the reference."""
    ng, at, found = d // GROUP, 0, {}
    for loop in [None] + list(range(len(bits))):
        rb = d // 2 if loop is None else d * bits[loop] // 8
        for kv in (0, 1):
            for kind, n in (("codes", rb), ("meta", 4 * ng)) + ((("a", 2),) if loop is not None else ()):
                found[loop, kv, kind] = (at, n)
                at += TILE * n
    return found, at


def _swizzle(units):
    """Position of 16-bit unit u of a V row in token pair p: [32][units]."""
    p = torch.arange(TILE // 2).view(-1, 1)
    x = 8 * (p % 4) if units == 32 else 8 * (p // 2 % 2) if units == 16 else 0 * p
    return torch.arange(units).view(1, -1) ^ x


def _pack_k(codes, b):
    """codes [..., 64, d] -> stored bytes [..., 64, d b / 8], words group-interleaved."""
    by = _to_bytes(codes, b)
    ng = codes.shape[-1] // GROUP
    return by.unflatten(-1, (ng, b, 4)).transpose(-3, -2).flatten(-3)


def _pack_v(codes, b):
    """codes [..., 64, d] -> stored bytes [..., 64 * d b / 8], in token pairs."""
    by = _to_bytes(codes, b)
    units = by.shape[-1] // 2
    x = by.unflatten(-1, (units, 2)).unflatten(-3, (TILE // 2, 2)).transpose(-3, -2)   # pair, u, parity
    at = _swizzle(units).to(codes.device)
    out = torch.empty_like(x)
    out.scatter_(-3, at.view(*at.shape, 1, 1).expand(x.shape), x)
    return out.flatten(-4)


def _to_bytes(codes, b):
    x = codes.to(torch.uint8).unflatten(-1, (-1, 8 // b))
    out = torch.zeros_like(x[..., 0])
    for k in range(8 // b):
        out |= x[..., k] << (k * b)
    return out


def _hadamard(d, device, dtype=torch.float32):
    h = torch.ones(1, 1, dtype=dtype, device=device)
    while h.shape[0] < d:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _quantise(x, b):
    g = x.unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    step, off = ((hi - lo) / (2 ** b - 1)).half().float(), lo.half().float()
    codes = torch.where(step > 0, (g - off) / step, torch.zeros_like(g)).round().clamp(0, 2 ** b - 1)
    return codes.flatten(-2), torch.cat([step, off], -1).half().flatten(-2), (codes * step + off).flatten(-2)


def _states(gen, scale, shape, L, u):
    """Loop states u_l * base + N(0, 0.1^2): [..., L, d]."""
    dev = scale.device
    base = torch.randn(shape, generator=gen, device=dev) * scale
    x = base.unsqueeze(-2) * u
    return x + 0.1 * torch.randn(x.shape, generator=gen, device=dev)


def _fill(c, gen, scale, signs, cap, ctx):
    """Tile records of one sequence: [Hkv][cap/64][record bytes], every slot below ctx encoded."""
    d, H, bits, dev = c["head_dim"], c["kv_heads"], _bits(c), scale.device
    at, rec = _sections(d, bits)
    tiles = cap // TILE
    data = torch.zeros(H, tiles, rec, dtype=torch.uint8, device=dev)
    L, used = len(bits) + 1, -(-ctx // TILE)
    had = _hadamard(d, dev) / math.sqrt(d)
    for t0 in range(0, used, 128):
        n = min(128, used - t0)
        u = 0.8 + 0.4 * torch.rand(H, n, TILE, L, 1, generator=gen, device=dev)

        def put(loop, kv, kind, rows):
            o, w = at[loop, kv, kind]
            data[:, t0:t0 + n, o:o + TILE * w] = rows.reshape(H, n, TILE * w)

        for kv in (0, 1):
            x = _states(gen, scale[kv].view(H, 1, 1, d), (H, n, TILE, d), L, u)
            pack = _pack_v if kv else _pack_k
            codes, meta, ref = _quantise(x[..., L - 1, :], 4)
            put(None, kv, "codes", pack(codes, 4))
            put(None, kv, "meta", meta.contiguous().view(torch.uint8))
            for l, b in enumerate(bits):
                y = x[..., l, :]
                a = ((y * ref).sum(-1) / (ref * ref).sum(-1)).half()
                r = (y - a.float().unsqueeze(-1) * ref) * signs[kv].view(H, 1, 1, d)
                codes, meta, _ = _quantise(r @ had.T, b)
                put(l, kv, "codes", pack(codes, b))
                put(l, kv, "meta", meta.contiguous().view(torch.uint8))
                put(l, kv, "a", a.contiguous().view(torch.uint8))
    return data


def _cache(c, gen, dev, cap, lens):
    """Packed cache of the batch [B][Hkv][cap/64][record] and the rotation signs [2][Hkv][d]."""
    d, H = c["head_dim"], c["kv_heads"]
    signs = torch.randint(0, 2, (2, H, d), generator=gen, device=dev).float() * 2 - 1
    scale = torch.ones(2, H, d, device=dev)     # two outlier channels of each head, x8
    scale.scatter_(2, torch.rand(2, H, d, generator=gen, device=dev).topk(2, 2).indices, 8.0)
    return torch.stack([_fill(c, gen, scale, signs, cap, n) for n in lens]), signs, scale


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    B, H, lens = c["batch"], c["kv_heads"], _ctx_lens(c)
    s = {"case": c, "ctx": torch.tensor(lens, dtype=torch.int32, device=dev)}
    cap = -(-max(lens + [1]) // TILE) * TILE
    if c["op"] != "select":     # constants of the layout that the plain forms use
        s["had"] = _hadamard(c["head_dim"], dev)
        s["turn"] = {u: _swizzle(u).to(dev) for u in (8, 16, 32)}
    if c["op"] != "chunk":
        # weights as attention leaves them: most slots near nothing, a few collect most, and
        # slots that no query has weighted yet are equal
        w = torch.exp(2.5 * torch.randn(B, H, cap, generator=gen, device=dev) - 6)
        s["weights"] = w * (torch.rand(B, H, cap, generator=gen, device=dev) > 0.05)
        s["kept"] = torch.zeros(B, dtype=torch.int32, device=dev)
        if c["op"] == "select":
            s["keep"] = torch.zeros(B, H, c["budget"], dtype=torch.int32, device=dev)
            return s
        s["kept"] = s["ctx"].clamp(max=c["budget"])
        s["keep"] = _some_slots(gen, s["weights"], lens, c["budget"])
        s["cap"], s["to_cap"] = cap, -(-c["budget"] // TILE) * TILE
        s["data"], s["signs"], _ = _cache(c, gen, dev, cap, lens)
        s["to"] = torch.zeros(B, H, s["to_cap"] // TILE, s["data"].shape[-1], dtype=torch.uint8, device=dev)
        s["to_weights"] = torch.zeros(B, H, s["to_cap"], device=dev)
        return s
    d, n, L = c["head_dim"], c["n_new"], len(c["res_bits"]) + 1
    cap = -(-(max(lens) + n) // TILE) * TILE
    s["cap"], s["max_ctx"] = cap, max(lens)
    s["data"], s["signs"], scale = _cache(c, gen, dev, cap, lens)
    u = 0.8 + 0.4 * torch.rand(B, n, 2, H, L, 1, generator=gen, device=dev)
    x = _states(gen, scale, (B, n, 2, H, d), L, u)
    s["kv_new"] = x.transpose(3, 4).contiguous().bfloat16()                 # [B][n][2][L][H][d]
    s["q"] = torch.randn(B, n, c["q_heads"], d, generator=gen, device=dev).bfloat16()
    s["new"] = torch.tensor(_new_lens(c), dtype=torch.int32, device=dev)
    s["out"] = torch.zeros(B, n, c["q_heads"], d, dtype=torch.bfloat16, device=dev)
    if c["window"]:
        s["weights"] = torch.rand(B, H, cap, generator=gen, device=dev)
    if c["paged"]:
        pages = cap // TILE
        order = torch.randperm(B * pages + 7, generator=gen, device=dev)[:B * pages]
        pool = torch.zeros(B * pages + 7, H, s["data"].shape[-1], dtype=torch.uint8, device=dev)
        pool[order] = s["data"].transpose(1, 2).flatten(0, 1)
        s["data"], s["table"] = pool, order.to(torch.int32).view(B, pages)
    return s


def _some_slots(gen, weights, lens, budget):
    """An ascending choice of slots for each (sequence, head), as a selection leaves it."""
    B, H, cap = weights.shape
    keep = torch.zeros(B, H, budget, dtype=torch.int32, device=weights.device)
    for b, n in enumerate(lens):
        k = min(n, budget)
        keep[b, :, :k] = weights[b, :, :n].topk(k, -1).indices.sort(-1).values.int()
    return keep


# ------------------------------------------------------------------------------ one pass

def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        return {"chunk": _own_chunk, "select": _own_select, "compact": _own_compact}[op](s)
    return {"chunk": _plain_chunk, "select": _plain_select, "compact": _plain_compact}[op](s)


def _handles(s, key, cap, data):
    """The shape and cache handle that a program keeps for a cache buffer."""
    import looped_transformer_kv_gb300 as rq
    c = s["case"]
    shape = rq.make_shape(c["batch"], c.get("q_heads", c["kv_heads"]), c["kv_heads"], c["head_dim"],
                          len(c["res_bits"]) + 1, cap, _bits(c))
    n_pages = data.shape[0] if c.get("paged") else None
    s[key] = shape, rq.PackedCache(shape, s["signs"], n_pages=n_pages, data=data.view(-1))
    return s[key]


def _own_chunk(s):
    import looped_transformer_kv_gb300 as rq
    c = s["case"]
    shape, cache = s.get("handle") or _handles(s, "handle", s["cap"], s["data"])
    if "ws" not in s:
        need = rq.chunk_workspace_bytes(shape, c["loop"], c["n_new"], s["max_ctx"], c["window"])
        s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        s["paging"] = rq.make_paging(s["table"], s["data"].shape[0]) if c["paged"] else None
    args = (s["q"], c["loop"], s["kv_new"], s["ctx"], s["max_ctx"], s["out"], s["ws"])
    more = {"n_lens": s["new"] if c["ragged"] else None, "weights": s.get("weights"), "window": c["window"]}
    if c["paged"]:
        rq.paged_chunk_attention(shape, cache, s["paging"], *args, **more)
    else:
        rq.chunk_attention(shape, cache, *args, **more)
    return {"out": s["out"], "weights": s["weights"]} if c["window"] else s["out"]


def _own_select(s):
    import looped_transformer_kv_gb300 as rq
    c = s["case"]
    rq.evict_select(s["weights"], s["ctx"], c["budget"], s["keep"], s["kept"], n_first=c["first"],
                    n_last=c["last"])
    return {"keep": s["keep"], "kept": s["kept"]}


def _own_compact(s):
    import looped_transformer_kv_gb300 as rq
    shape, cache = s.get("handle") or _handles(s, "handle", s["cap"], s["data"])
    to_shape, to_cache = s.get("to_handle") or _handles(s, "to_handle", s["to_cap"], s["to"])
    rq.evict_compact(shape, cache, to_shape, to_cache, s["keep"], s["kept"], weights=s["weights"],
                     to_weights=s["to_weights"])
    return {"cache": s["to"], "weights": s["to_weights"]}


# ------------------------------------------------------------------------------ plain forms

def _codes(by, b):
    x = torch.stack([(by >> (k * b)) & (2 ** b - 1) for k in range(8 // b)], -1)
    return x.flatten(-2).float()


def _rows(s, data, loop, kv, T):
    """Dequantised rows [B][H][T][d] of one kind of section and the a rows (None: reference)."""
    d, bits = s["case"]["head_dim"], _bits(s["case"])
    at, _ = _sections(d, bits)
    b, ng = 4 if loop is None else bits[loop], d // GROUP
    data = data[:, :, :T // TILE]

    def rows(kind):
        o, w = at[loop, kv, kind]
        return data[..., o:o + TILE * w].unflatten(-1, (TILE, w))

    by = rows("codes")
    if kv == 0:
        by = by.unflatten(-1, (b, ng, 4)).transpose(-3, -2).flatten(-3)
    else:
        units = d * b // 16
        x = by.flatten(-2).unflatten(-1, (TILE // 2, units, 2, 2))
        pos = s["turn"][units]
        x = x.gather(-3, pos.view(*pos.shape, 1, 1).expand(x.shape))
        by = x.transpose(-3, -2).flatten(-2).flatten(-3, -2)
    meta = rows("meta").contiguous().view(torch.float16).float().unflatten(-1, (ng, 2))
    x = _codes(by, b).unflatten(-1, (ng, GROUP)) * meta[..., :1] + meta[..., 1:]
    x = x.flatten(-2).flatten(2, 3)
    a = None if loop is None else rows("a").contiguous().view(torch.float16).float().flatten(2, 4)
    return x, a


def _rebuild(s, kv, T):
    """K or V of the call's loop for the first T slots, 32 bits: [B][H][T][d]."""
    c, data = s["case"], s["data"]
    if c["paged"]:
        data = data[s["table"].long()].transpose(1, 2)
    ref, _ = _rows(s, data, None, kv, T)
    if c["loop"] == len(c["res_bits"]):
        return ref
    res, a = _rows(s, data, c["loop"], kv, T)
    d = c["head_dim"]
    back = (res @ s["had"]) / math.sqrt(d) * s["signs"][kv].view(1, -1, 1, d)
    return ref * a.unsqueeze(-1) + back


def _plain_chunk(s):
    c = s["case"]
    B, H, d, n = c["batch"], c["kv_heads"], c["head_dim"], c["n_new"]
    G = c["q_heads"] // H
    T = -(-s["max_ctx"] // TILE) * TILE
    dev = s["q"].device
    new = s["kv_new"][:, :, :, c["loop"]].float()                            # [B][n][2][H][d]
    k = torch.cat([_rebuild(s, 0, T), new[:, :, 0].transpose(1, 2)], 2)
    v = torch.cat([_rebuild(s, 1, T), new[:, :, 1].transpose(1, 2)], 2)
    q = s["q"].float().view(B, n, H, G, d).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, d)
    j = torch.arange(n, device=dev)
    old = torch.arange(T, device=dev).view(1, 1, -1) < s["ctx"].view(B, 1, 1)
    fresh = (j.view(1, 1, n) <= j.view(1, n, 1)) & (j.view(1, 1, n) < s["new"].view(B, 1, 1))
    mask = torch.cat([old.expand(B, n, T), fresh.expand(B, n, n)], 2)
    x = (q @ k.transpose(2, 3)).view(B, H, G, n, T + n) / math.sqrt(d)
    x = x.masked_fill(~mask.view(B, 1, 1, n, T + n), -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    del x
    p /= p.sum(-1, keepdim=True)
    out = (p.view(B, H, G * n, T + n) @ v).view(B, H, G, n, d).permute(0, 3, 1, 2, 4).reshape(B, n, H * G, d)
    valid = j.view(1, n) < s["new"].view(B, 1)
    s["out"].copy_(torch.where(valid.view(B, n, 1, 1), out.bfloat16(), s["out"]))
    if not c["window"]:
        return s["out"]
    voted = valid & (j.view(1, n) >= s["new"].view(B, 1) - c["window"])
    w = (p * voted.view(B, 1, 1, n, 1)).sum((2, 3))                          # [B][H][T + n]
    slot = torch.cat([torch.arange(T, device=dev).expand(B, T), s["ctx"].long().view(B, 1) + j], 1)
    s["weights"].scatter_add_(2, slot.clamp(max=s["cap"] - 1).view(B, 1, -1).expand(B, H, -1),
                              w * (slot < s["cap"]).view(B, 1, -1))
    return {"out": s["out"], "weights": s["weights"]}


def _plain_select(s):
    c, w = s["case"], s["weights"]
    cap, K = w.shape[2], c["budget"]
    t = torch.arange(cap, device=w.device).view(1, 1, -1)
    n = s["ctx"].view(-1, 1, 1)
    # held slots before all weights, slots behind the context after them
    held = (t < c["first"]) | (t >= n - c["last"])
    key = torch.where(t < n, torch.where(held, math.inf, w), -math.inf)
    order = key.sort(dim=-1, descending=True, stable=True).indices
    chosen = torch.zeros_like(order, dtype=torch.bool)
    chosen.scatter_(2, order[..., :K], True)
    chosen &= t < n
    rank = chosen.cumsum(-1) - 1
    row = s["keep"].view(-1, K)
    at = torch.arange(row.shape[0], device=w.device).view(-1, 1).expand(-1, cap)
    hit = chosen.view(-1, cap)
    row[at[hit], rank.view(-1, cap)[hit]] = t.expand(chosen.shape).reshape(-1, cap)[hit].int()
    s["kept"].copy_(s["ctx"].clamp(max=K))
    return {"keep": s["keep"], "kept": s["kept"]}


def _plain_compact(s):
    c = s["case"]
    d, bits = c["head_dim"], _bits(c)
    at, _ = _sections(d, bits)
    B, H, K = s["keep"].shape
    T = s["to_cap"]
    keep = torch.zeros(B, H, T, dtype=torch.long, device=s["keep"].device)
    keep[..., :K] = s["keep"]
    live = torch.arange(T, device=keep.device).view(1, 1, T) < s["kept"].view(B, 1, 1)
    keep *= live
    for (loop, kv, kind), (o, w) in at.items():
        def rows(x):
            x = x[..., o:o + TILE * w]
            if kind != "codes" or kv == 0:
                return x.reshape(B, H, -1, w)
            units = w // 2
            x = x.unflatten(-1, (TILE // 2, units, 2, 2))
            pos = s["turn"][units]
            x = x.gather(-3, pos.view(*pos.shape, 1, 1).expand(x.shape))
            return x.transpose(-3, -2).reshape(B, H, -1, w)

        src, old = rows(s["data"]), rows(s["to"])
        new = src.gather(2, keep.unsqueeze(-1).expand(B, H, T, w))
        new = torch.where(live.unsqueeze(-1), new, old).view(B, H, T // TILE, TILE, w)
        if kind == "codes" and kv == 1:
            x = new.unflatten(-1, (w // 2, 2)).unflatten(-3, (TILE // 2, 2)).transpose(-3, -2)
            pos = s["turn"][w // 2]
            new = torch.empty_like(x).scatter_(-3, pos.view(*pos.shape, 1, 1).expand(x.shape), x)
        s["to"][..., o:o + TILE * w] = new.reshape(B, H, T // TILE, TILE * w)
    moved = s["weights"].gather(2, keep) * live
    s["to_weights"].copy_(moved)
    return {"cache": s["to"], "weights": s["to_weights"]}


# ------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """What run returns, from the definitions in 64 bits: one (sequence, head) at a time, each
    element found by its address in the record."""
    c = case
    s = prepare(c, seed)
    if c["op"] == "select":
        return _exact_select(s)
    if c["op"] == "compact":
        got = torch.zeros(s["to_weights"].shape, dtype=torch.float64, device=s["keep"].device)
        for b, n in enumerate(s["kept"].tolist()):
            for h in range(c["kv_heads"]):
                got[b, h, :n] = s["weights"][b, h].double()[s["keep"][b, h, :n].long()]
        return {"cache": None, "weights": got}
    B, H, d, n = c["batch"], c["kv_heads"], c["head_dim"], c["n_new"]
    G = c["q_heads"] // H
    out = torch.zeros(B, n, c["q_heads"], d, dtype=torch.float64, device=s["q"].device)
    acc = s["weights"].double() if c["window"] else None
    for b, (ctx, m) in enumerate(zip(_ctx_lens(c), _new_lens(c))):
        for h in range(H):
            k, v = (torch.cat([_exact_rows(s, b, h, kv, ctx), s["kv_new"][b, :m, kv, c["loop"], h].double()])
                    for kv in (0, 1))
            late = torch.arange(ctx + m, device=k.device).view(1, -1) > ctx + torch.arange(m, device=k.device).view(-1, 1)
            for g in range(G):
                x = s["q"][b, :m, h * G + g].double() @ k.T / math.sqrt(d)
                x[late] = -math.inf
                p = torch.softmax(x, -1)
                out[b, :m, h * G + g] = p @ v
                if acc is not None:
                    acc[b, h, :ctx + m] += p[max(0, m - c["window"]):].sum(0)[:acc.shape[2]]
    return {"out": out, "weights": acc} if c["window"] else out


def _exact_rows(s, b, h, kv, T):
    c = s["case"]
    d, bits, dev = c["head_dim"], _bits(c), s["q"].device
    at, rec = _sections(d, bits)
    t = torch.arange(T, device=dev)
    page = s["table"][b].long() if c["paged"] else None
    unit = s["data"][page, h] if c["paged"] else s["data"][b, h]             # [tiles][rec]
    flat, base, r = unit.reshape(-1), t // TILE * rec, t % TILE
    ch = torch.arange(d, device=dev)

    def half(addr):
        return (flat[addr].long() | flat[addr + 1].long() << 8).to(torch.int32).to(torch.int16).view(torch.float16).double()

    def level(loop):
        w = 4 if loop is None else bits[loop]
        o, rb = at[loop, kv, "codes"]
        byte = ch * w // 8
        if kv == 0:
            word = byte // 4
            a = (base + o + r * rb).view(-1, 1) + ((word % w) * (d // 32) + word // w) * 4 + byte % 4
        else:
            pair = (r // 2).view(-1, 1)
            turn = 8 * (pair % 4) if rb == 64 else 8 * (pair // 2 % 2) if rb == 32 else 0 * pair
            a = (base + o).view(-1, 1) + pair * 2 * rb + ((byte // 2) ^ turn) * 4 + (r % 2).view(-1, 1) * 2 + byte % 2
        code = (flat[a].long() >> (ch * w % 8)) & (2 ** w - 1)
        o, mb = at[loop, kv, "meta"]
        m = (base + o + r * mb).view(-1, 1) + ch // GROUP * 4
        return code.double() * half(m) + half(m + 2)

    x = level(None)
    if c["loop"] < len(bits):
        o, _ = at[c["loop"], kv, "a"]
        y = level(c["loop"])
        k = torch.arange(d)
        ones = torch.tensor([[bin(i & j).count("1") % 2 for j in k.tolist()] for i in k.tolist()], device=dev)
        x = x * half(base + o + 2 * r).view(-1, 1) + (y @ (1.0 - 2.0 * ones.double())) / math.sqrt(d) * s["signs"][kv, h].double()
    return x


def _exact_select(s):
    c = s["case"]
    w = s["weights"].cpu().numpy()
    keep = np.zeros(s["keep"].shape, dtype=np.int64)
    kept = np.zeros(c["batch"], dtype=np.int64)
    for b, n in enumerate(_ctx_lens(c)):
        k = kept[b] = min(n, c["budget"])
        for h in range(c["kv_heads"]):
            rest = np.arange(min(c["first"], n), max(min(c["first"], n), n - c["last"]))
            held = np.setdiff1d(np.arange(n), rest)
            best = rest[np.lexsort((rest, -w[b, h, rest].astype(np.float64)))][:max(0, k - len(held))]
            keep[b, h, :k] = np.sort(np.concatenate([held, best]))[:k]
    return {"keep": torch.from_numpy(keep).int(), "kept": torch.from_numpy(kept).int()}
