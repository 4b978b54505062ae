"""64-bit references of the 8-bit cache's operators, on the host: bytes at the addresses that
include/rq_q8.h gives, no code shared with the library or its binding."""

import numpy as np

MOST = {"e4m3": 448.0, "int8": 127.0}
LEAST = -100


def _e4m3_table():
    x = np.zeros(256)
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        x[b] = (-v if b & 128 else v) if b & 127 != 127 else np.nan
    return x


E4M3 = _e4m3_table()


def bf16(x):
    """The nearest bf16 numbers (ties to even), of non-negative finite x."""
    m, e = np.frexp(np.asarray(x, np.float64))
    return np.ldexp(np.rint(m * 256) / 256, e)


def nearest(x, fmt):
    """Codes' values nearest to x (ties to even), saturated."""
    if fmt == "int8":
        return np.clip(np.rint(x), -127, 127)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -20))), -6) - 3)
    return np.clip(np.rint(x / step) * step, -448, 448)


def byte_of(x, fmt):
    """Bytes of code values."""
    if fmt == "int8":
        return x.astype(np.int8).view(np.uint8)
    pos = E4M3[:127]
    at = np.searchsorted(pos, np.abs(x))
    assert (pos[at] == np.abs(x)).all()
    return (at | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def value_of(by, fmt):
    return by.view(np.int8).astype(np.float64) if fmt == "int8" else E4M3[by]


def place(t, d):
    """Byte places of slot t's channels in a tile's [64][d] bytes."""
    r = t % 64
    turn = r % 8 if d == 128 else r // 2 % 4
    ch = np.arange(d)
    return r * d + ((ch // 16) ^ turn) * 16 + ch % 16


def exponent(amax, fmt):
    a = float(bf16(amax))
    if a == 0:
        return LEAST
    e = int(np.floor(np.log2(a))) - 12
    while a > MOST[fmt] * 2.0 ** e:
        e += 1
    return max(e, LEAST)


def rotate(x, pos, table, interleaved):
    """x fp32 [..., d] rotated in fp32, products and sums rounded one by one."""
    if table is None:
        return x
    x = x.astype(np.float32)
    half = table.shape[1]
    co, si = table[pos, :, 0], table[pos, :, 1]
    y = x.copy()
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y[..., a] = x[..., a] * co - x[..., b] * si
    y[..., b] = x[..., b] * co + x[..., a] * si
    assert y.dtype == np.float32
    return y


def append(codes, scales, kv, ctx, fmt):
    """Codes [tiles][2][64 d] and scales [tiles][2][4] of one (sequence, head, loop) after new rows kv
    [n][2][d] (rotated, fp32) went to the slots from ctx on; in place."""
    n, _, d = kv.shape
    for which in (0, 1):
        for k in range(ctx // 16, -(-(ctx + n) // 16) if n else 0):
            tile, part = k // 4, k % 4
            new = range(max(ctx, 16 * k), min(ctx + n, 16 * k + 16))
            old = range(16 * k, max(16 * k, min(ctx, 16 * k + 16)))
            rows = kv[new.start - ctx:new.stop - ctx, which].astype(np.float64)
            was = float(scales[tile, which, part])
            bad = not np.isfinite(rows).all() or (len(old) > 0 and np.isnan(was))
            if bad:
                scales[tile, which, part] = np.nan
                for t in new:
                    codes[tile, which, place(t, d)] = 0
                continue
            e = exponent(np.abs(rows).max(), fmt)
            if len(old):
                e0 = int(np.log2(was))
                e = max(e, e0)
                for t in old:
                    p = place(t, d)
                    codes[tile, which, p] = byte_of(nearest(value_of(codes[tile, which, p], fmt) * 2.0 ** (e0 - e), fmt), fmt)
            scales[tile, which, part] = 2.0 ** e
            for t, row in zip(new, rows):
                codes[tile, which, place(t, d)] = byte_of(nearest(row * 2.0 ** -e, fmt), fmt)


def rows_of(codes, scales, n, d, fmt):
    """Values [2][n][d] of the first n slots, from codes [tiles][2][64 d] and scales [tiles][2][4]."""
    t = np.arange(n)
    at = np.stack([place(x, d) for x in range(64)])[t % 64]                  # [n][d]
    out = np.zeros((2, n, d))
    for which in (0, 1):
        by = np.take_along_axis(codes[t // 64, which], at, 1)
        out[which] = value_of(by, fmt) * scales[t // 64, which, t % 64 // 16].astype(np.float64)[:, None]
    return out


def attend(q, k, v, ctx, scale, window=0, sinks=0):
    """q [m][G][d], k, v [ctx + m][d].  Outputs [m][G][d], weights [m][G][T], and the largest
    sum |q k| * scale of each row."""
    m, T = q.shape[0], k.shape[0]
    s = np.einsum("jgd,td->jgt", q, k) * scale
    own, t = (ctx + np.arange(m))[:, None], np.arange(T)[None, :]
    seen = t <= own
    if window:
        seen &= (t > own - window) | (t < sinks)
    s = np.where(seen[:, None], s, -np.inf)
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    mag = (np.einsum("jgd,td->jgt", np.abs(q), np.abs(k)) * scale * seen[:, None]).max(-1)
    return np.einsum("jgt,td->jgd", p, np.where(seen.any(0)[:, None], v, 0)), p, mag
