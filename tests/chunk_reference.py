"""64-bit references of the chunk and eviction operators, on the host.

The cache is read back byte by byte at the addresses include/rq.h gives (no code shared with the
library or its binding), rebuilt in float64, and attended by the textbook formula."""

import numpy as np

TILE, GROUP = 64, 32


def row_layout(d, bits):
    """{(loop or None, kv, kind): (offset in a record, row bytes)} and the record's bytes."""
    ng, at, out = d // GROUP, 0, {}
    for loop in [None] + list(range(len(bits))):
        rb = d // 2 if loop is None else d * bits[loop] // 8
        for kv in (0, 1):
            kinds = [("codes", rb), ("meta", 4 * ng)] + ([("a", 2)] if loop is not None else [])
            for kind, n in kinds:
                out[loop, kv, kind] = (at, n)
                at += TILE * n
    return out, at


def _swz(pair, units):
    return 8 * (pair % 4) if units == 32 else 8 * (pair // 2 % 2) if units == 16 else 0


def token_bytes(rec, t, d, bits):
    """Every stored byte of token row t (0..63) of one record, in natural order."""
    lay, _ = row_layout(d, bits)
    out = []
    for (loop, kv, kind), (o, n) in lay.items():
        if kind != "codes":
            out.append(rec[o + t * n:o + (t + 1) * n])
            continue
        b = 4 if loop is None else bits[loop]
        k = np.arange(n)
        if kv == 0:
            w = k // 4
            idx = o + t * n + ((w % b) * (d // 32) + w // b) * 4 + k % 4
        else:
            p = t // 2
            idx = o + p * 2 * n + ((k // 2) ^ _swz(p, n // 2)) * 4 + (t % 2) * 2 + k % 2
        out.append(rec[idx])
    return np.concatenate(out)


def _level(rec, t, d, bits, loop, kv):
    lay, _ = row_layout(d, bits)
    b = 4 if loop is None else bits[loop]
    o, n = lay[loop, kv, "codes"]
    i = np.arange(d)
    k = i * b // 8
    if kv == 0:
        w = k // 4
        idx = o + t * n + ((w % b) * (d // 32) + w // b) * 4 + k % 4
    else:
        p = t // 2
        idx = o + p * 2 * n + ((k // 2) ^ _swz(p, n // 2)) * 4 + (t % 2) * 2 + k % 2
    code = (rec[idx].astype(np.int64) >> (i * b % 8)) & (2 ** b - 1)
    o, n = lay[loop, kv, "meta"]
    meta = rec[o + t * n:o + (t + 1) * n].copy().view(np.float16).astype(np.float64).reshape(-1, 2)
    return code * np.repeat(meta[:, 0], GROUP) + np.repeat(meta[:, 1], GROUP)


def hadamard(d):
    h = np.ones((1, 1))
    while len(h) < d:
        h = np.block([[h, h], [h, -h]])
    return h


def rebuild(records, n, d, bits, loop, kv, signs):
    """K or V of `loop` for tokens 0..n-1 of one (sequence, head): records [tiles][rec] -> [n][d]."""
    out = np.zeros((n, d))
    lay, _ = row_layout(d, bits)
    had = hadamard(d) / np.sqrt(d)
    for t in range(n):
        rec, r = records[t // TILE], t % TILE
        x = _level(rec, r, d, bits, None, kv)
        if loop < len(bits):
            o, _ = lay[loop, kv, "a"]
            a = float(rec[o + 2 * r:o + 2 * r + 2].copy().view(np.float16)[0])
            x = a * x + (_level(rec, r, d, bits, loop, kv) @ had) * signs
        out[t] = x
    return out


def residual_norms(records, n, d, bits, loop, kv):
    """Euclidean norm of each token's residual levels (0 for the final loop)."""
    if loop == len(bits):
        return np.zeros(n)
    return np.array([np.linalg.norm(_level(records[t // TILE], t % TILE, d, bits, loop, kv)) for t in range(n)])


def attend(q, k, v, ctx, scale):
    """q [m][G][d], k, v [ctx + m][d]: causal over the chunk.  Outputs [m][G][d], weights
    [m][G][ctx + m] and the largest sum |q k| * scale of each row."""
    m = q.shape[0]
    s = np.einsum("jgd,td->jgt", q, k) * scale
    s[np.broadcast_to((np.arange(ctx + m)[None, :] > ctx + np.arange(m)[:, None])[:, None], s.shape)] = -np.inf
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    mag = (np.einsum("jgd,td->jgt", np.abs(q), np.abs(k)) * scale).max(-1)
    return np.einsum("jgt,td->jgd", p, v), p, mag


def select(w, n, budget, first, last):
    """Kept slots of one row, ascending."""
    key = [(1, 0.0) if t < first or t >= n - last else (0, np.inf) if np.isnan(w[t]) else (-1, float(w[t]))
           for t in range(n)]
    order = sorted(range(n), key=lambda t: (-key[t][0], -key[t][1], t))
    return sorted(order[:budget])
