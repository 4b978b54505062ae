"""Thin PyTorch binding of librq: argument marshalling only.

Every step of encode and decode attention runs in the library's CUDA kernels; PyTorch
provides device memory and the current stream.  Names follow the C ABI (include/rq.h, include/rq_q8.h).
"""

import ctypes

import torch

from . import _lib
from ._lib import (RQ_MAX_LOOPS, RqCache, RqPaging, RqQ8Cache, RqQ8Shape, RqRope, RqShape,
                   RqSynthParams, check)

GROUP = 32


def _ptr(t):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _raw_stream(stream):
    """The same as a number, without a Stream object (4 us of a small call)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def make_shape(batch, n_q_heads, n_kv_heads, head_dim, n_loops, capacity, res_bits,
               softmax_scale=0.0, group=GROUP):
    """rq_shape for one layer; res_bits lists the residual bits of loops 0..L-2."""
    s = RqShape()
    s.batch, s.n_q_heads, s.n_kv_heads = batch, n_q_heads, n_kv_heads
    s.head_dim, s.n_loops, s.group, s.capacity = head_dim, n_loops, group, capacity
    for l, b in enumerate(res_bits):
        s.res_bits[l] = int(b)
    s.softmax_scale = float(softmax_scale)
    return s


def res_bits_of(shape):
    return [int(shape.res_bits[l]) for l in range(shape.n_loops - 1)]


PAGE = 64   # tokens per page of a paged cache


class PackedCache:
    """One layer's packed cache in device memory: the tile records of include/rq.h in one
    buffer (256-byte aligned), [B][Hkv][capacity/64] records, or [n_pages][Hkv] in paged
    form, plus the rotation signs.  record_bytes() is rq_record_bytes; section(...) gives the
    byte range of one kind of row inside a record (for reading the cache back).  data: an
    existing uint8 buffer of exactly the cache's bytes to use instead of a new one (kept alive
    here)."""

    def __init__(self, shape, rot_signs, device="cuda", n_pages=None, data=None):
        B, H, cap, d = shape.batch, shape.n_kv_heads, shape.capacity, shape.head_dim
        self.n_pages = n_pages
        self.shape = shape
        self.rec = int(_lib.lib().rq_record_bytes(ctypes.byref(shape)))
        assert self.rec > 0
        n_rec = (n_pages * H) if n_pages is not None else (B * H * (cap // PAGE))
        if data is None:
            data = torch.empty(n_rec * self.rec, dtype=torch.uint8, device=device)
        assert data.dtype == torch.uint8 and data.is_contiguous() and data.numel() == n_rec * self.rec
        self.data = data.view(-1)
        self.rot_signs = rot_signs.to(device=data.device, dtype=torch.int8).contiguous()  # [2][H][d]
        assert tuple(self.rot_signs.shape) == (2, H, d)
        c = RqCache()
        c.data = self.data.data_ptr()
        for kv in range(2):
            c.rot_signs[kv] = self.rot_signs[kv].data_ptr()
        self.struct = c

    def records(self):
        """The records as [B][Hkv][capacity/64][rec] (or [n_pages][Hkv][rec] when paged)."""
        s = self.shape
        if self.n_pages is not None:
            return self.data.view(self.n_pages, s.n_kv_heads, self.rec)
        return self.data.view(s.batch, s.n_kv_heads, s.capacity // PAGE, self.rec)

    def section(self, kind, kv, loop=None):
        """(byte offset in a record, row bytes) of one kind of 64 rows: kind in 'codes',
        'meta', 'alpha'; loop None = the reference section."""
        d = self.shape.head_dim
        ng = d // GROUP
        if loop is None:
            base = kv * PAGE * (d // 2 + 4 * ng)
            return {"codes": (base, d // 2), "meta": (base + PAGE * d // 2, 4 * ng)}[kind]
        bits = res_bits_of(self.shape)
        off = PAGE * (d + 8 * ng)
        for b in bits[:loop]:
            off += PAGE * (2 * (d * b // 8) + 8 * ng + 4)
        rb = d * bits[loop] // 8
        base = off + kv * PAGE * (rb + 4 * ng + 2)
        return {"codes": (base, rb), "meta": (base + PAGE * rb, 4 * ng),
                "alpha": (base + PAGE * (rb + 4 * ng), 2)}[kind]

    def tensors(self):
        return [self.data]

    def nbytes(self):
        return self.data.numel()


def cache_bytes(shape):
    return int(_lib.lib().rq_cache_bytes(ctypes.byref(shape)))


def advance_ctx(ctx_lens, n, capacity, stream=None):
    """rq_advance_ctx: ctx_lens[b] += n on the device (capped at capacity)."""
    assert ctx_lens.dtype == torch.int32 and ctx_lens.is_contiguous()
    check("rq_advance_ctx", _lib.lib().rq_advance_ctx(_ptr(ctx_lens), ctx_lens.numel(), int(n),
                                                      int(capacity), _stream(stream)))


def paged_cache_bytes(shape, n_pages):
    return int(_lib.lib().rq_paged_cache_bytes(ctypes.byref(shape), int(n_pages)))


def make_paging(block_table, n_pages):
    """rq_paging for a device int32 block table [B][max_pages] (kept alive by the caller)."""
    assert block_table.dtype == torch.int32 and block_table.dim() == 2
    assert block_table.is_contiguous()
    g = RqPaging()
    g.block_table = block_table.data_ptr()
    g.max_pages = block_table.shape[1]
    g.n_pages = int(n_pages)
    g.sequences, g.device = block_table.shape[0], block_table.get_device()
    return g


def paged_encode_append(shape, cache, paging, kv_new, positions=None, pos_begin=0, stream=None):
    """rq_paged_encode_append; kv_new as in encode_append."""
    assert kv_new.dtype == torch.bfloat16 and kv_new.dim() == 6 and kv_new.stride(5) == 1
    st = (ctypes.c_int64 * 5)(*[kv_new.stride(i) for i in range(5)])
    check("rq_paged_encode_append", _lib.lib().rq_paged_encode_append(
        ctypes.byref(shape), ctypes.byref(cache.struct), ctypes.byref(paging), _ptr(kv_new), st,
        _ptr(positions), int(pos_begin), int(kv_new.shape[1]), _stream(stream)))


def paged_decode_attention(shape, cache, paging, q, loop_begin, loop_count, pending_kv,
                           ctx_lens, max_ctx, out, ws, stream=None):
    check("rq_paged_decode_attention", _lib.lib().rq_paged_decode_attention(
        ctypes.byref(shape), ctypes.byref(cache.struct), ctypes.byref(paging), _ptr(q),
        int(loop_begin), int(loop_count), _ptr(pending_kv), _ptr(ctx_lens), int(max_ctx),
        _ptr(out), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def encode_append(shape, cache, kv_new, positions=None, pos_begin=0, stream=None):
    """kv_new: bf16 [B][n_new][2][L][Hkv][d] (any strides, channel stride 1)."""
    assert kv_new.dtype == torch.bfloat16 and kv_new.dim() == 6 and kv_new.stride(5) == 1
    st = (ctypes.c_int64 * 5)(*[kv_new.stride(i) for i in range(5)])
    n_new = kv_new.shape[1]
    check("rq_encode_append", _lib.lib().rq_encode_append(
        ctypes.byref(shape), ctypes.byref(cache.struct), _ptr(kv_new), st, _ptr(positions),
        int(pos_begin), int(n_new), _stream(stream)))


def ablation_encode_append(shape, cache, kv_new, alpha_mode, positions=None, pos_begin=0,
                           stream=None):
    """rq_ablation_encode_append (include/rq_ablation.h): a_l fixed by alpha_mode
    (0 least squares, 1 one, 2 zero)."""
    assert kv_new.dtype == torch.bfloat16 and kv_new.dim() == 6 and kv_new.stride(5) == 1
    st = (ctypes.c_int64 * 5)(*[kv_new.stride(i) for i in range(5)])
    check("rq_ablation_encode_append", _lib.lib().rq_ablation_encode_append(
        ctypes.byref(shape), ctypes.byref(cache.struct), _ptr(kv_new), st, _ptr(positions),
        int(pos_begin), int(kv_new.shape[1]), int(alpha_mode), _stream(stream)))


def ablation_decode_attention(shape, cache, mode, q, loop, pending_kv, ctx_lens, max_ctx, out, ws,
                              stream=None):
    """rq_ablation_decode_attention: per-loop decode of residual loop `loop` over a cache
    encoded with a = 1 (mode 1) or a = 0 (mode 2)."""
    check("rq_ablation_decode_attention", _lib.lib().rq_ablation_decode_attention(
        ctypes.byref(shape), ctypes.byref(cache.struct), int(mode), _ptr(q), int(loop),
        _ptr(pending_kv), _ptr(ctx_lens), int(max_ctx), _ptr(out), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def decode_workspace_bytes(shape, loop_count, max_ctx):
    return int(_lib.lib().rq_decode_workspace_bytes(ctypes.byref(shape), int(loop_count),
                                                    int(max_ctx)))


def decode_attention(shape, cache, q, loop_begin, loop_count, pending_kv, ctx_lens, max_ctx,
                     out, ws, stream=None):
    check("rq_decode_attention", _lib.lib().rq_decode_attention(
        ctypes.byref(shape), ctypes.byref(cache.struct), _ptr(q), int(loop_begin),
        int(loop_count), _ptr(pending_kv), _ptr(ctx_lens), int(max_ctx), _ptr(out), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def decode_attention_noalloc(shape, cache, q, loop_begin, loop_count, pending_kv, ctx_lens,
                             max_ctx, out, stream=None):
    """rq_decode_attention_noalloc: the library's fixed scratch array instead of a workspace."""
    check("rq_decode_attention_noalloc", _lib.lib().rq_decode_attention_noalloc(
        ctypes.byref(shape), ctypes.byref(cache.struct), _ptr(q), int(loop_begin),
        int(loop_count), _ptr(pending_kv), _ptr(ctx_lens), int(max_ctx), _ptr(out),
        _stream(stream)))


def test_decode_attention_wait_runs_out(shape, cache, q, loop_begin, loop_count, pending_kv,
                                        ctx_lens, max_ctx, out, ws, wait_limit_ns, stream=None):
    """rq_test_decode_attention_wait_runs_out (test hook, include/rq_test.h)."""
    check("rq_test_decode_attention_wait_runs_out",
          _lib.lib().rq_test_decode_attention_wait_runs_out(
              ctypes.byref(shape), ctypes.byref(cache.struct), _ptr(q), int(loop_begin),
              int(loop_count), _ptr(pending_kv), _ptr(ctx_lens), int(max_ctx), _ptr(out), _ptr(ws),
              ws.numel() * ws.element_size(), int(wait_limit_ns), _stream(stream)))


def noalloc_scratch_bytes():
    return int(_lib.lib().rq_decode_noalloc_scratch_bytes())


def bf16_decode_attention(shape, k, v, q, loop_begin, loop_count, pending_kv, ctx_lens, max_ctx,
                          out, ws, stream=None):
    check("rq_bf16_decode_attention", _lib.lib().rq_bf16_decode_attention(
        ctypes.byref(shape), _ptr(k), _ptr(v), _ptr(q), int(loop_begin), int(loop_count),
        _ptr(pending_kv), _ptr(ctx_lens), int(max_ctx), _ptr(out), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def _f32(t):
    assert t is None or (t.dtype == torch.float32 and t.is_contiguous())
    return _ptr(t)


def _i32(t):
    assert t is None or (t.dtype == torch.int32 and t.is_contiguous())
    return _ptr(t)


def chunk_workspace_bytes(shape, loop, n_new, max_ctx, window=0):
    """rq_chunk_workspace_bytes: workspace of chunk_attention / paged_chunk_attention calls of this
    shape and loop with at most these n_new, max_ctx and window."""
    return int(_lib.lib().rq_chunk_workspace_bytes(ctypes.byref(shape), int(loop), int(n_new),
                                                   int(max_ctx), int(window)))


_I3, _I5 = ctypes.c_int64 * 3, ctypes.c_int64 * 5


def _chunk_args(shape, q, loop, kv_new, ctx_lens, max_ctx, out, ws, n_lens, weights, window, stream):
    B, n, Hq, d = q.shape
    H = shape.n_kv_heads
    assert q.dtype == kv_new.dtype == out.dtype == torch.bfloat16
    assert B == shape.batch and Hq == shape.n_q_heads and d == shape.head_dim
    assert kv_new.shape == (B, n, 2, shape.n_loops, H, d)
    qs, ks = q.stride(), kv_new.stride()
    assert n == 0 or qs[3] == ks[5] == 1
    assert out.is_contiguous() and out.shape == q.shape
    assert ctx_lens.numel() == B and (n_lens is None or n_lens.numel() == B)
    assert weights is None or weights.shape == (B, H, shape.capacity)
    return (q.data_ptr(), _I3(*qs[:3]), loop, kv_new.data_ptr(), _I5(*ks[:5]), _i32(n_lens), n,
            _i32(ctx_lens), max_ctx, out.data_ptr(), _f32(weights), window, ws.data_ptr(),
            ws.numel() * ws.element_size(), _stream(stream))


def chunk_attention(shape, cache, q, loop, kv_new, ctx_lens, max_ctx, out, ws, n_lens=None,
                    weights=None, window=0, stream=None):
    """rq_chunk_attention: q, out bf16 [B][n][Hq][d] (q any strides, channel stride 1), kv_new as
    in encode_append, n_lens int32 [B]; weights fp32 [B][Hkv][capacity] collects the softmax
    weights of each sequence's last `window` tokens."""
    check("rq_chunk_attention", _lib.lib().rq_chunk_attention(
        ctypes.byref(shape), ctypes.byref(cache.struct),
        *_chunk_args(shape, q, loop, kv_new, ctx_lens, max_ctx, out, ws, n_lens, weights, window,
                     stream)))


def paged_chunk_attention(shape, cache, paging, q, loop, kv_new, ctx_lens, max_ctx, out, ws,
                          n_lens=None, weights=None, window=0, stream=None):
    """rq_paged_chunk_attention; the other arguments as in chunk_attention."""
    check("rq_paged_chunk_attention", _lib.lib().rq_paged_chunk_attention(
        ctypes.byref(shape), ctypes.byref(cache.struct), ctypes.byref(paging),
        *_chunk_args(shape, q, loop, kv_new, ctx_lens, max_ctx, out, ws, n_lens, weights, window,
                     stream)))


def evict_select(weights, ctx_lens, budget, keep, kept_lens, n_first=0, n_last=0, stream=None):
    """rq_evict_select: weights fp32 [B][Hkv][capacity]; keep int32 [B][Hkv][budget] takes the kept
    slots, ascending, kept_lens int32 [B] their number."""
    B, H, cap = weights.shape
    assert tuple(keep.shape) == (B, H, budget) and ctx_lens.numel() == B and kept_lens.numel() == B
    check("rq_evict_select", _lib.lib().rq_evict_select(
        _f32(weights), B, H, cap, _i32(ctx_lens), int(budget), int(n_first), int(n_last),
        _i32(keep), _i32(kept_lens), _stream(stream)))


def _compact_args(shape, to_shape, keep, kept_lens, weights, to_weights, stream):
    B, H = shape.batch, shape.n_kv_heads
    assert tuple(keep.shape[:2]) == (B, H) and keep.dim() == 3 and kept_lens.numel() == B
    assert weights is None or tuple(weights.shape) == (B, H, shape.capacity)
    assert to_weights is None or tuple(to_weights.shape) == (B, H, to_shape.capacity)
    return (_i32(keep), int(keep.shape[2]), _i32(kept_lens), _f32(weights), _f32(to_weights),
            _stream(stream))


def evict_compact(shape, cache, to_shape, to_cache, keep, kept_lens, weights=None, to_weights=None,
                  stream=None):
    """rq_evict_compact: row keep[b][h][t] of cache becomes row t of to_cache (which may be the
    same cache), its weights alike."""
    check("rq_evict_compact", _lib.lib().rq_evict_compact(
        ctypes.byref(shape), ctypes.byref(cache.struct), ctypes.byref(to_shape),
        ctypes.byref(to_cache.struct),
        *_compact_args(shape, to_shape, keep, kept_lens, weights, to_weights, stream)))


def paged_evict_compact(shape, cache, paging, to_shape, to_cache, to_paging, keep, kept_lens,
                        weights=None, to_weights=None, stream=None):
    """rq_paged_evict_compact; the other arguments as in evict_compact."""
    check("rq_paged_evict_compact", _lib.lib().rq_paged_evict_compact(
        ctypes.byref(shape), ctypes.byref(cache.struct), ctypes.byref(paging),
        ctypes.byref(to_shape), ctypes.byref(to_cache.struct), ctypes.byref(to_paging),
        *_compact_args(shape, to_shape, keep, kept_lens, weights, to_weights, stream)))


Q8_FORMATS = {"e4m3": 0, "int8": 1}


def make_q8_shape(batch, n_q_heads, n_kv_heads, head_dim, n_loops, capacity, fmt="e4m3",
                  softmax_scale=0.0):
    """rq_q8_shape of one layer's 8-bit cache; fmt "e4m3" or "int8"."""
    return RqQ8Shape(batch, n_q_heads, n_kv_heads, head_dim, n_loops, capacity, Q8_FORMATS[fmt],
                     float(softmax_scale))


def q8_cache_bytes(shape):
    return int(_lib.lib().rq_q8_cache_bytes(ctypes.byref(shape)))


def q8_paged_cache_bytes(shape, n_pages):
    return int(_lib.lib().rq_q8_paged_cache_bytes(ctypes.byref(shape), int(n_pages)))


class Q8Cache:
    """One layer's 8-bit cache in device memory (include/rq_q8.h): codes uint8, 128-byte aligned,
    [B][Hkv][capacity/64][loops][2][64][d], or [n_pages][Hkv]... in paged form, and scales fp32
    [...][loops][2][4].  codes, scales: existing buffers of exactly these sizes to use instead of
    new ones (kept alive here).  rows() gives the numbers that a cache holds."""

    def __init__(self, shape, device="cuda", n_pages=None, codes=None, scales=None):
        B, H, tiles, d, L = shape.batch, shape.n_kv_heads, shape.capacity // PAGE, shape.head_dim, shape.n_loops
        self.shape, self.n_pages, self.key = shape, n_pages, bytes(shape)
        lead = (B, H, tiles) if n_pages is None else (n_pages, H)
        full = (*lead, L, 2, PAGE, d)
        n = q8_cache_bytes(shape) if n_pages is None else q8_paged_cache_bytes(shape, n_pages)
        assert n > 0
        if codes is None:
            codes = torch.zeros(n, dtype=torch.uint8, device=device)
        if scales is None:
            scales = torch.ones(n // (4 * d * 4), dtype=torch.float32, device=codes.device)
        assert codes.dtype == torch.uint8 and codes.is_contiguous() and codes.numel() == n
        assert scales.dtype == torch.float32 and scales.is_contiguous() and scales.numel() * 16 * d == n
        self.codes, self.scales = codes.view(full), scales.view(*lead, L, 2, 4)
        self.struct = RqQ8Cache(self.codes.data_ptr(), self.scales.data_ptr())

    def rows(self):
        """The values in natural order, fp32 [...][loops][2][64][d] (to look at; nothing calls it)."""
        s = self.shape
        t = torch.arange(PAGE, device=self.codes.device).view(-1, 1)
        c = torch.arange(s.head_dim // 16, device=self.codes.device).view(1, -1)
        at = c ^ ((t & 7) if s.head_dim == 128 else (t // 2 & 3))
        x = self.codes.unflatten(-1, (-1, 16))
        x = x.gather(-2, at.unsqueeze(-1).expand(x.shape)).flatten(-2)
        x = x.view(torch.int8 if s.format == Q8_FORMATS["int8"] else torch.float8_e4m3fn).float()
        return (x.unflatten(-2, (4, 16)) * self.scales[..., None, None]).flatten(-3, -2)

    def tensors(self):
        return [self.codes, self.scales]

    def nbytes(self):
        return self.codes.numel() + 4 * self.scales.numel()


def make_rope(table, interleaved=False, positions=None):
    """rq_rope: table fp32 [n_pos][rot_dim/2][2] (cos, sin), positions int32 [B][n_new] or None (a
    token's slot); the tensors are kept alive by the handle."""
    assert table.dtype == torch.float32 and table.is_contiguous() and table.dim() == 3 and table.shape[2] == 2
    assert positions is None or (positions.dtype == torch.int32 and positions.is_contiguous())
    r = RqRope(table.data_ptr(), None if positions is None else positions.data_ptr(), table.shape[0],
               2 * table.shape[1], int(interleaved))
    r.tensors = (table, positions)
    return r


def _rope(rope, B, n, dev):
    if rope is None:
        return None
    table, positions = rope.tensors
    assert table.get_device() == dev
    assert positions is None or (positions.shape == (B, n) and positions.get_device() == dev)
    return ctypes.byref(rope)


def _lens(t, B, dev):
    """Address of an int32 [B] tensor, or None."""
    if t is None:
        return None
    assert t.dtype == torch.int32 and t.numel() == B and t.is_contiguous() and t.get_device() == dev
    return t.data_ptr()


def _q8_fits(shape, cache, paging):
    """The library sees bare pointers: what a call of this shape reads and writes lies in the cache."""
    if paging is None:
        assert cache.n_pages is None, "a paged cache in a contiguous call"
    else:
        assert cache.n_pages is not None, "a contiguous cache in a paged call"
        assert paging.n_pages <= cache.n_pages, "more pages than the cache has"
        assert paging.sequences >= shape.batch, "fewer block-table rows than sequences"
    if bytes(shape) == cache.key:
        return
    own = RqQ8Shape.from_buffer_copy(cache.key)
    assert ((shape.n_kv_heads, shape.head_dim, shape.n_loops, shape.format) ==
            (own.n_kv_heads, own.head_dim, own.n_loops, own.format)), "another layout than the cache's"
    # (a pool serves any batch and any length; a contiguous cache its first sequences)
    assert paging is not None or (shape.capacity == own.capacity and shape.batch <= own.batch), "a larger shape than the cache's"


def _q8_append_args(shape, cache, paging, kv_new, loop_begin, ctx_lens, n_lens, rope, stream):
    _q8_fits(shape, cache, paging)
    B, n, two, loops, H, d = kv_new.shape
    dev = torch._C._cuda_getDevice()      # every tensor lies on the current device
    assert paging is None or paging.device == dev
    assert kv_new.get_device() == cache.codes.get_device() == cache.scales.get_device() == dev
    s0, s1, s2, s3, s4, s5 = kv_new.stride()
    assert kv_new.dtype == torch.bfloat16 and (B, two, H, d) == (shape.batch, 2, shape.n_kv_heads, shape.head_dim)
    assert s5 == 1 or kv_new.numel() == 0
    return (kv_new.data_ptr(), _I5(s0, s1, s2, s3, s4), loop_begin, loops, _lens(n_lens, B, dev), n,
            _lens(ctx_lens, B, dev), _rope(rope, B, n, dev), _raw_stream(stream))


def q8_append(shape, cache, kv_new, loop_begin, ctx_lens, n_lens=None, rope=None, stream=None):
    """rq_q8_append: kv_new bf16 [B][n][2][loops][Hkv][d] (any strides, channel stride 1) goes to the
    slots from ctx_lens[b] on, of the loops from loop_begin on; n_lens int32 [B]; rope from make_rope."""
    check("rq_q8_append", _lib.lib().rq_q8_append(
        ctypes.byref(shape), ctypes.byref(cache.struct),
        *_q8_append_args(shape, cache, None, kv_new, loop_begin, ctx_lens, n_lens, rope, stream)))


def paged_q8_append(shape, cache, paging, kv_new, loop_begin, ctx_lens, n_lens=None, rope=None,
                    stream=None):
    """rq_paged_q8_append; the other arguments as in q8_append."""
    check("rq_paged_q8_append", _lib.lib().rq_paged_q8_append(
        ctypes.byref(shape), ctypes.byref(cache.struct), ctypes.byref(paging),
        *_q8_append_args(shape, cache, paging, kv_new, loop_begin, ctx_lens, n_lens, rope, stream)))


def q8_workspace_bytes(shape, n_new, max_ctx, window=0, n_sink=0):
    """rq_q8_workspace_bytes: workspace of q8_attention / paged_q8_attention calls of this shape with
    at most these n_new and max_ctx."""
    return int(_lib.lib().rq_q8_workspace_bytes(ctypes.byref(shape), int(n_new), int(max_ctx),
                                                int(window), int(n_sink)))


def _q8_attention_args(shape, cache, paging, q, loop, ctx_lens, max_ctx, out, ws, n_lens, window, n_sink, rope, stream):
    _q8_fits(shape, cache, paging)
    B, n, Hq, d = q.shape
    dev = torch._C._cuda_getDevice()
    assert paging is None or paging.device == dev
    assert (q.get_device() == out.get_device() == ws.get_device() == cache.codes.get_device() ==
            cache.scales.get_device() == dev)
    s0, s1, s2, s3 = q.stride()
    assert q.dtype == out.dtype == torch.bfloat16
    assert (B, Hq, d) == (shape.batch, shape.n_q_heads, shape.head_dim)
    assert s3 == 1 or q.numel() == 0
    assert out.shape == q.shape and out.is_contiguous() and ws.is_contiguous()
    return (q.data_ptr(), _I3(s0, s1, s2), loop, _lens(n_lens, B, dev), n, _lens(ctx_lens, B, dev), max_ctx, window,
            n_sink, _rope(rope, B, n, dev), out.data_ptr(), ws.data_ptr(), ws.nbytes, _raw_stream(stream))


def q8_attention(shape, cache, q, loop, ctx_lens, max_ctx, out, ws, n_lens=None, window=0, n_sink=0,
                 rope=None, stream=None):
    """rq_q8_attention: q, out bf16 [B][n][Hq][d] (q any strides, channel stride 1) of the n tokens
    that q8_append stored from ctx_lens[b] on; window 0: all slots up to a token's own, else its last
    `window` and the first n_sink."""
    check("rq_q8_attention", _lib.lib().rq_q8_attention(
        ctypes.byref(shape), ctypes.byref(cache.struct),
        *_q8_attention_args(shape, cache, None, q, loop, ctx_lens, max_ctx, out, ws, n_lens, window, n_sink, rope,
                            stream)))


def paged_q8_attention(shape, cache, paging, q, loop, ctx_lens, max_ctx, out, ws, n_lens=None, window=0,
                       n_sink=0, rope=None, stream=None):
    """rq_paged_q8_attention; the other arguments as in q8_attention."""
    check("rq_paged_q8_attention", _lib.lib().rq_paged_q8_attention(
        ctypes.byref(shape), ctypes.byref(cache.struct), ctypes.byref(paging),
        *_q8_attention_args(shape, cache, paging, q, loop, ctx_lens, max_ctx, out, ws, n_lens, window, n_sink, rope,
                            stream)))


def synth_params(seed, layer, head_dim, n_kv_heads, dist, sigma, outlier_mult, outlier_table):
    """rq_synth_params; outlier_table: device int32 [Hkv][2][n] (kept alive by the caller)."""
    p = RqSynthParams()
    p.seed, p.layer, p.head_dim, p.n_kv_heads, p.dist = seed, layer, head_dim, n_kv_heads, dist
    for l, s in enumerate(sigma):
        p.sigma[l] = float(s)
    p.outlier_mult = float(outlier_mult)
    p.n_outliers = int(outlier_table.shape[-1]) if outlier_table is not None else 0
    p.outlier_table = outlier_table.data_ptr() if outlier_table is not None else None
    return p


def synth_states(params, out, strides, b0, nb, t0, nt, l0, nl, stream=None):
    st = (ctypes.c_int64 * 5)(*strides)
    check("rq_synth_states", _lib.lib().rq_synth_states(
        ctypes.byref(params), _ptr(out), st, b0, nb, t0, nt, l0, nl, _stream(stream)))


def synth_queries(params, out, n_q_heads, b0, nb, l0, nl, step=0, stream=None):
    check("rq_synth_queries", _lib.lib().rq_synth_queries(
        ctypes.byref(params), _ptr(out), n_q_heads, b0, nb, l0, nl, step, _stream(stream)))
