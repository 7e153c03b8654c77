"""Rotary positions, the paged FP8 cache and attention over it: the part of a
decoder layer between its Q/K/V and output projections.

    cache = kv_cache(pages, kv_heads, page_size, head_dim)
    table = rope_table(positions, rot_dim)
    q = kv_append(cache, k, v, block_table, kv_lens, table=table, q=q)
    out = kv_attention(q, cache, block_table, kv_lens)

Marshalling only, as in the rest of the package: shapes, types and devices
are checked here, everything else by the C entry points (include/w8a16.h,
which defines the operators and the cache's layout).  Calls run on the
current (or given) torch stream, take the memory of their outputs there, and
do not synchronise.
"""

from __future__ import annotations

import ctypes
from contextlib import nullcontext
from typing import NamedTuple, Optional

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_ORDERS = {"split": 0, "turns": 1, "own": 2}
ROPE_MAX_AXES = 4
ROPE_SCALINGS = {None: 0, "linear": 1, "base": 2, "bands": 3}
KV_BLOCK = 16
KV_KERNEL_ROWS = 1
KV_KERNEL_TILE = 2

_vp, _u32, _i64, _u64 = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_int64, ctypes.c_uint64


class RopeConfig(ctypes.Structure):
    """w8a16_rope_config_t"""
    _fields_ = [(n, ctypes.c_double) for n in ("base", "factor", "original", "low_turns",
                                               "high_turns", "magnitude")] + [("scaling", _u32)]


class KVCacheDesc(ctypes.Structure):
    """w8a16_kv_cache_t"""
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp),
                ("k_page_stride", _u64), ("v_page_stride", _u64),
                ("k_scale_page_stride", _u64), ("v_scale_page_stride", _u64),
                ("pages", _u32), ("page_size", _u32), ("kv_heads", _u32), ("head_dim", _u32)]


class KVSeqs(ctypes.Structure):
    """w8a16_kv_seqs_t"""
    _fields_ = [("block_table", _vp), ("kv_lens", _vp), ("cu_seqlens", _vp),
                ("block_table_stride", _u32), ("block_table_width", _u32), ("seqs", _u32),
                ("tokens", _u32), ("max_new", _u32)]


class KVAppendArgs(ctypes.Structure):
    """w8a16_kv_append_args_t"""
    _fields_ = [("k", _vp), ("v", _vp), ("q", _vp), ("q_out", _vp)] + \
        [(n, _i64) for n in ("k_token_stride", "k_head_stride", "v_token_stride", "v_head_stride",
                             "q_token_stride", "q_head_stride", "q_out_token_stride",
                             "q_out_head_stride")] + \
        [("table", _vp), ("table_positions", _u32), ("rot_dim", _u32), ("layout", _u32),
         ("dtype", _u32), ("q_heads", _u32)]


class Axes(ctypes.Structure):
    """w8a16_axes_t"""
    _fields_ = [("positions", _vp), ("axis_stride", _i64), ("count", _u32), ("order", _u32),
                ("pairs", _u32 * ROPE_MAX_AXES), ("table_pairs", _u32)]


class KVPlan(ctypes.Structure):
    """w8a16_kv_plan_t"""
    _fields_ = [("kernel", _u32), ("row_blocks", _u32), ("waves", _u32), ("row_tiles", _u32), ("chunk_tiles", _u32),
                ("chunks", _u32), ("grid", _u32), ("workspace_bytes", _u64)]

    def as_dict(self) -> dict:
        return {name: int(getattr(self, name)) for name, _ in self._fields_}


class KVAttentionArgs(ctypes.Structure):
    """w8a16_kv_attention_args_t"""
    _fields_ = [("q", _vp), ("out", _vp), ("lse", _vp),
                ("q_token_stride", _i64), ("q_head_stride", _i64),
                ("out_token_stride", _i64), ("out_head_stride", _i64),
                ("plan", ctypes.POINTER(KVPlan)), ("scale", ctypes.c_float),
                ("q_heads", _u32), ("dtype", _u32), ("causal", _u32), ("window", _u32),
                ("max_kv", _u32)]


class KVSpan(ctypes.Structure):
    """w8a16_kv_span_t"""
    _fields_ = [("sinks", _u32), ("shared", _u32)]


def declare(lib) -> None:
    """Argument types of the entry points."""
    ptr = ctypes.POINTER
    lib.w8a16_rope_table.argtypes = [ptr(RopeConfig), _vp, _u32, _u32, _vp]
    lib.w8a16_rope.argtypes = [_vp, _i64, _i64, _vp, _i64, _i64, _u32, _u32, _u32, _u32, _vp, _u32,
                               _u32, _vp, _u32, _u32, _vp]
    lib.w8a16_rope_axes.argtypes = [_vp, _i64, _i64, _vp, _i64, _i64, _u32, _u32, _u32, _u32, _vp, _u32,
                                    ptr(Axes), _u32, _u32, _vp]
    lib.w8a16_kv_append_axes.argtypes = [ptr(KVCacheDesc), ptr(KVSeqs), ptr(KVAppendArgs), ptr(Axes), _vp]
    lib.w8a16_kv_append.argtypes = [ptr(KVCacheDesc), ptr(KVSeqs), ptr(KVAppendArgs), _vp]
    lib.w8a16_kv_attention.argtypes = [ptr(KVCacheDesc), ptr(KVSeqs), ptr(KVAttentionArgs), _vp]
    lib.w8a16_kv_attention_span.argtypes = [ptr(KVCacheDesc), ptr(KVSeqs), ptr(KVAttentionArgs), ptr(KVSpan),
                                            _vp]
    lib.w8a16_plan_kv_shared.argtypes = [_u32] * 9 + [ptr(KVPlan)] * 2
    lib.w8a16_plan_kv_attention.argtypes = [_u32] * 8 + [ptr(KVPlan)]
    for name in ("w8a16_rope_table", "w8a16_rope", "w8a16_rope_axes", "w8a16_kv_append",
                 "w8a16_kv_append_axes", "w8a16_kv_attention", "w8a16_kv_attention_span",
                 "w8a16_plan_kv_shared", "w8a16_plan_kv_attention"):
        getattr(lib, name).restype = ctypes.c_int


_state = None
_codes = _scale_bytes = ()     # torch types of a cache's codes and scale bytes


def _setup():
    """(library, torch, dtype codes, raise function, raw stream of a device
    index), resolved once."""
    global _state, _codes, _scale_bytes
    if _state is None:
        import torch

        from . import _raise_if, library
        # what current_stream(device).cuda_stream returns, an order of
        # magnitude faster (0.06 against 1.8 us of a call's 8)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda index: torch.cuda.current_stream(index).cuda_stream)
        _codes = (torch.uint8, torch.float8_e4m3fn)
        _scale_bytes = (torch.uint8, torch.float8_e8m0fnu)
        _state = (library(), torch,
                  {torch.bfloat16: 1, torch.float16: 2, torch.float32: 3}, _raise_if, raw)
    return _state


class KVCache(NamedTuple):
    """Codes (uint8 or float8_e4m3fn) and scale bytes (uint8 or
    float8_e8m0fnu) of a paged FP8 cache:
    k [pages, kv_heads, page_size, head_dim], v [pages, kv_heads,
    page_size / 16, head_dim, 16], k_scale and v_scale [pages, kv_heads,
    page_size / 16].  Only the page axis may be strided."""
    k: "torch.Tensor"            # noqa: F821
    v: "torch.Tensor"            # noqa: F821
    k_scale: "torch.Tensor"      # noqa: F821
    v_scale: "torch.Tensor"      # noqa: F821


def kv_cache(pages: int, kv_heads: int, page_size: int, head_dim: int, device="cuda") -> KVCache:
    """A new, empty cache (scale bytes 0: a block that was never written
    gives NaN if it is read)."""
    import torch
    blocks = page_size // KV_BLOCK
    if page_size < KV_BLOCK or page_size % KV_BLOCK or page_size > 1024:
        raise ValueError("page_size must be a multiple of 16 in 16..1024")

    def zeros(*shape):
        return torch.zeros(shape, dtype=torch.uint8, device=device)
    return KVCache(zeros(pages, kv_heads, page_size, head_dim),
                   zeros(pages, kv_heads, blocks, head_dim, KV_BLOCK),
                   zeros(pages, kv_heads, blocks), zeros(pages, kv_heads, blocks))


def _page_stride(name, t, inside):
    """Page stride of a cache tensor whose pages are contiguous inside."""
    st, want = t.stride(), 1
    for n, have in zip(reversed(t.shape[1:]), reversed(st[1:])):
        if n > 1 and have != want:
            raise ValueError("the inside of a %s page must be contiguous" % name)
        want *= n
    return max(st[0], inside) if t.shape[0] < 2 else st[0]


def _cache_desc(cache) -> KVCacheDesc:
    k, v, ks, vs = cache
    pages, heads, page, dim = k.shape
    blocks = page // KV_BLOCK
    if v.shape != (pages, heads, blocks, dim, KV_BLOCK) or ks.shape != (pages, heads, blocks) or \
            vs.shape != ks.shape:
        raise ValueError("cache must be k [pages, heads, page, dim], v [pages, heads, page/16, dim, "
                         "16] and scales [pages, heads, page/16]")
    if k.dtype not in _codes or v.dtype not in _codes or ks.dtype not in _scale_bytes or \
            vs.dtype not in _scale_bytes:
        raise ValueError("cache codes must be uint8 or float8_e4m3fn, its scales uint8 or float8_e8m0fnu")
    if not (k.is_cuda and v.is_cuda and ks.is_cuda and vs.is_cuda):
        raise ValueError("cache must be GPU tensors")
    codes, bytes_ = heads * page * dim, heads * blocks
    return KVCacheDesc(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(),
                       codes if k.is_contiguous() else _page_stride("k", k, codes),
                       codes if v.is_contiguous() else _page_stride("v", v, codes),
                       bytes_ if ks.is_contiguous() else _page_stride("k_scale", ks, bytes_),
                       bytes_ if vs.is_contiguous() else _page_stride("v_scale", vs, bytes_),
                       pages, page, heads, dim)


def _seqs_desc(i32, block_table, kv_lens, cu_seqlens, tokens, max_new) -> KVSeqs:
    if block_table.dtype != i32 or kv_lens.dtype != i32 or kv_lens.dim() != 1:
        raise ValueError("block_table must be int32 [seqs, pages] and kv_lens int32 [seqs]")
    seqs = kv_lens.shape[0]
    rows, width = block_table.shape
    if rows != seqs or not (block_table.is_cuda and kv_lens.is_cuda):
        raise ValueError("block_table and kv_lens must be GPU tensors of the same sequences")
    pitch = width
    if not block_table.is_contiguous():
        pitch = block_table.stride(0) if seqs > 1 else width
        if width > 1 and block_table.stride(1) != 1:
            raise ValueError("block_table rows must be contiguous")
    if not kv_lens.is_contiguous():
        raise ValueError("kv_lens must be contiguous")
    cu = 0
    if cu_seqlens is not None:
        if cu_seqlens.dtype != i32 or cu_seqlens.shape != (seqs + 1,) or \
                not cu_seqlens.is_contiguous() or not cu_seqlens.is_cuda:
            raise ValueError("cu_seqlens must be a contiguous int32 GPU tensor [seqs + 1]")
        cu = cu_seqlens.data_ptr()
        if max_new is None:
            max_new = tokens
    elif max_new is None:
        max_new = tokens // max(1, seqs)
    return KVSeqs(block_table.data_ptr(), kv_lens.data_ptr(), cu, pitch, width, seqs, tokens, max_new)


def _rows(name, t, tokens, heads, dim, dtype):
    """Token and head strides of a [tokens, heads, dim] operand."""
    if t.shape != (tokens, heads, dim) or t.dtype != dtype or not t.is_cuda:
        raise ValueError("%s must be a %s GPU tensor [%d, %d, %d]" % (name, dtype, tokens, heads, dim))
    st, sh, sd = t.stride()
    if sd != 1 and dim > 1:
        raise ValueError("%s needs a unit stride along head_dim" % name)
    return st, sh


def _on(torch, stream):
    """Where a call makes its outputs: on the stream that will write them (the
    current stream's memory might still be written by work that is to come
    there)."""
    return nullcontext() if stream is None else torch.cuda.stream(stream)


def _like(torch, t, stream):
    """A new contiguous tensor of t's shape and type."""
    if stream is not None:
        with _on(torch, stream):
            return _like(torch, t, None)
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def rope_table(positions: int, rot_dim: int, *, base: float = 10000.0, scaling: Optional[str] = None,
               factor: float = 1.0, original: float = 0.0, low_turns: float = 1.0,
               high_turns: float = 4.0, magnitude: float = 1.0, out=None, device="cuda", stream=None):
    """float32 [positions, rot_dim / 2, 2]: (cos, sin) of every position and
    pair, times `magnitude`.  scaling: None, "linear", "base" or "bands"
    (w8a16_rope_scaling in include/w8a16.h)."""
    lib, torch, _, check, raw = _setup()
    if scaling not in ROPE_SCALINGS:
        raise ValueError("scaling must be None, 'linear', 'base' or 'bands'")
    shape = (positions, rot_dim // 2, 2)
    if out is None:
        with _on(torch, stream):
            out = torch.empty(shape, dtype=torch.float32, device=device)
    if out.dtype != torch.float32 or out.shape != shape or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("out must be a contiguous float32 GPU tensor [positions, rot_dim/2, 2]")
    cfg = RopeConfig(base, factor, original, low_turns, high_turns, magnitude, ROPE_SCALINGS[scaling])
    check(lib.w8a16_rope_table(cfg, out.data_ptr(), positions, rot_dim,
                               raw(out.get_device()) if stream is None else stream.cuda_stream))
    return out


def _check_table(f32, table):
    if table.dtype != f32 or table.dim() != 3 or table.shape[2] != 2 or \
            not table.is_contiguous() or not table.is_cuda:
        raise ValueError("table must be a contiguous float32 GPU tensor [positions, rot_dim/2, 2]")
    positions, pairs, _ = table.shape
    return table.data_ptr(), positions, 2 * pairs


def _axes(i32, positions, tokens, sections, order, table_pairs) -> Axes:
    """Positions of several axes; sections: pairs of each."""
    if order not in ROPE_ORDERS:
        raise ValueError("order must be 'split', 'turns' or 'own'")
    count = len(sections)
    if not 0 < count <= ROPE_MAX_AXES or min(sections) < 0:
        raise ValueError("sections must be the pairs of 1 to %d axes" % ROPE_MAX_AXES)
    if positions is None or positions.dtype != i32 or positions.shape != (count, tokens) or \
            not positions.is_cuda or (tokens > 1 and positions.stride(1) != 1):
        raise ValueError("positions must be an int32 GPU tensor [%d, %d] with a unit stride along tokens" %
                         (count, tokens))
    return Axes(positions.data_ptr(), positions.stride(0), count, ROPE_ORDERS[order],
                (_u32 * ROPE_MAX_AXES)(*sections), table_pairs)


def rope(x, table, positions, out=None, *, layout: str = "half", inverse: bool = False, sections=None,
         order: str = "split", stream=None):
    """x [tokens, heads, head_dim] (bfloat16, float16 or float32) with the
    first 2 * table.shape[1] elements of each head rotated to `positions`
    (int32 [tokens]).  inverse=True rotates back, which is also the gradient:
    dx = rope(dy, ..., inverse=True).  out may be x.  Returns out.

    sections: pairs of each of up to four axes (a picture's frame, row and
    column); positions is then int32 [axes, tokens] and the first
    2 * sum(sections) elements are rotated.  order: "split" (the first
    sections[0] pairs are axis 0's, and so on), "turns" (pair i is axis
    i % axes's while that one has pairs left, else axis 0's) or "own" (as
    split, each axis starting again at the table's first column); the table has
    sum(sections) pairs, in "own" at least max(sections)."""
    lib, torch, dtypes, check, raw = _setup()
    dtype = x.dtype
    if x.dim() != 3 or dtype not in dtypes:
        raise ValueError("x must be bfloat16, float16 or float32 [tokens, heads, head_dim]")
    tokens, heads, dim = x.shape
    xt, xh = _rows("x", x, tokens, heads, dim, dtype)
    if out is None:
        out = _like(torch, x, stream)
        yt, yh = heads * dim, dim
    else:
        yt, yh = _rows("out", out, tokens, heads, dim, dtype)
    if layout not in ROPE_LAYOUTS:
        raise ValueError("layout must be 'half' or 'interleaved'")
    tp, tn, rot = _check_table(torch.float32, table)
    if sections is not None:
        st = lib.w8a16_rope_axes(x.data_ptr(), xt, xh, out.data_ptr(), yt, yh, dtypes[dtype], tokens, heads,
                                 dim, tp, tn,
                                 _axes(torch.int32, positions, tokens, sections, order, table.shape[1]),
                                 ROPE_LAYOUTS[layout], inverse,
                                 raw(x.get_device()) if stream is None else stream.cuda_stream)
        if st:
            check(st)
        return out
    if positions.shape != (tokens,) or positions.dtype != torch.int32 or \
            not positions.is_contiguous() or not positions.is_cuda:
        raise ValueError("positions must be a contiguous int32 GPU tensor [tokens]")
    st = lib.w8a16_rope(x.data_ptr(), xt, xh, out.data_ptr(), yt, yh, dtypes[dtype], tokens, heads, dim,
                        tp, tn, rot, positions.data_ptr(), ROPE_LAYOUTS[layout], inverse,
                        raw(x.get_device()) if stream is None else stream.cuda_stream)
    if st:
        check(st)
    return out


def kv_append(cache, k, v, block_table, kv_lens, *, cu_seqlens=None, max_new: Optional[int] = None,
              table=None, layout: str = "half", q=None, q_out=None, positions=None, sections=None,
              order: str = "split", stream=None):
    """Append the new tokens' keys and values (k, v [tokens, kv_heads,
    head_dim]) to `cache`, keys rotated by `table` if given; with q [tokens,
    q_heads, head_dim] also rotate the queries, in the same launch.

    kv_lens int32 [seqs]: tokens each sequence holds with the new ones
    counted.  block_table int32 [seqs, pages].  cu_seqlens int32 [seqs + 1]:
    offsets of the sequences' new tokens; None: tokens / seqs each.  max_new:
    at least the most new tokens of one sequence (None: all tokens; a closer
    bound launches less).  sections, positions (int32 [axes, tokens]) and
    order: rotate by positions of several axes, as rope does, in place of each
    token's place in its sequence.  Returns q_out (None without q)."""
    lib, torch, dtypes, check, raw = _setup()
    dtype = k.dtype
    if k.dim() != 3 or dtype not in dtypes:
        raise ValueError("k must be bfloat16, float16 or float32 [tokens, kv_heads, head_dim]")
    tokens, heads, dim = k.shape
    desc = _cache_desc(cache)
    if heads != desc.kv_heads or dim != desc.head_dim:
        raise ValueError("k must have the cache's heads and head_dim")
    kt, kh = _rows("k", k, tokens, heads, dim, dtype)
    vt, vh = _rows("v", v, tokens, heads, dim, dtype)
    if layout not in ROPE_LAYOUTS:
        raise ValueError("layout must be 'half' or 'interleaved'")
    tp = tn = rot = qp = op = hq = qt = qh = ot = oh = 0
    if table is not None:
        tp, tn, rot = _check_table(torch.float32, table)
    if q is not None:
        hq = q.shape[1] if q.dim() == 3 else 0
        qt, qh = _rows("q", q, tokens, hq, dim, dtype)
        if q_out is None:
            q_out = _like(torch, q, stream)
            ot, oh = hq * dim, dim
        else:
            ot, oh = _rows("q_out", q_out, tokens, hq, dim, dtype)
        qp, op = q.data_ptr(), q_out.data_ptr()
    else:
        q_out = None
    seqs = _seqs_desc(torch.int32, block_table, kv_lens, cu_seqlens, tokens, max_new)
    axes = None
    if sections is not None:
        if table is None:
            raise ValueError("positions of several axes need a table")
        axes = _axes(torch.int32, positions, tokens, sections, order, table.shape[1])
        rot = 2 * sum(sections)
    elif positions is not None:
        raise ValueError("positions need sections")
    args = KVAppendArgs(k.data_ptr(), v.data_ptr(), qp, op, kt, kh, vt, vh, qt, qh, ot, oh, tp, tn, rot,
                        ROPE_LAYOUTS[layout], dtypes[dtype], hq)
    queue = raw(k.get_device()) if stream is None else stream.cuda_stream
    if axes is None:
        st = lib.w8a16_kv_append(desc, seqs, args, queue)
    else:
        st = lib.w8a16_kv_append_axes(desc, seqs, args, axes, queue)
    if st:
        check(st)
    return q_out


def kv_attention(q, cache, block_table, kv_lens, out=None, *, cu_seqlens=None,
                 max_new: Optional[int] = None, max_kv: Optional[int] = None,
                 scale: Optional[float] = None, causal: bool = True, window: int = 0, sinks: int = 0,
                 shared: int = 0, return_lse: bool = False, plan_: Optional[KVPlan] = None, stream=None):
    """Attention of the new tokens' queries q [tokens, q_heads, head_dim]
    (bfloat16 or float16) over `cache`.  block_table, kv_lens, cu_seqlens and
    max_new as for kv_append (which has stored the new tokens before);
    max_kv: at least the largest of kv_lens, for the launch's shape (None:
    what the block table can hold).  scale: None for 1 / sqrt(head_dim).
    window: keys a query sees at most, itself counted (0: all).  sinks: the
    first tokens that stay visible behind a window.  shared: tokens that all
    sequences start with, on the same pages (the block table's rows agree on
    them): whole pages of them are read once for the batch where that pays;
    results are the same up to the order of additions.  Returns
    out, or (out, lse) with lse float32 [tokens, q_heads]."""
    lib, torch, dtypes, check, raw = _setup()
    desc = _cache_desc(cache)
    dim, dtype = desc.head_dim, q.dtype
    if q.dim() != 3 or dtype not in dtypes:
        raise ValueError("q must be bfloat16 or float16 [tokens, q_heads, head_dim]")
    tokens, heads, _ = q.shape
    qt, qh = _rows("q", q, tokens, heads, dim, dtype)
    if out is None:
        out = _like(torch, q, stream)
        ot, oh = heads * dim, dim
    else:
        ot, oh = _rows("out", out, tokens, heads, dim, dtype)
    lse, lp = None, 0
    if return_lse:
        with _on(torch, stream):
            lse = q.new_empty((tokens, heads), dtype=torch.float32)
        lp = lse.data_ptr()
    if window < 0 or sinks < 0 or shared < 0:
        raise ValueError("window, sinks and shared must not be negative")
    seqs = _seqs_desc(torch.int32, block_table, kv_lens, cu_seqlens, tokens, max_new)
    args = KVAttentionArgs(q.data_ptr(), out.data_ptr(), lp, qt, qh, ot, oh,
                           None if plan_ is None else ctypes.pointer(plan_),
                           dim ** -0.5 if scale is None else scale, heads, dtypes[dtype], causal,
                           window, max_kv or 0)
    queue = raw(q.get_device()) if stream is None else stream.cuda_stream
    if sinks or shared:
        st = lib.w8a16_kv_attention_span(desc, seqs, args, KVSpan(min(sinks, 1 << 30), min(shared, 1 << 30)), queue)
    else:
        st = lib.w8a16_kv_attention(desc, seqs, args, queue)
    if st:
        check(st)
    return (out, lse) if return_lse else out


def plan_kv_attention(seqs: int, max_new: int, max_kv: int, q_heads: int, kv_heads: int,
                      head_dim: int, window: int = 0, cu_count: int = 0) -> KVPlan:
    """Default plan of kv_attention (no GPU call)."""
    from . import _raise_if, library
    p = KVPlan()
    _raise_if(library().w8a16_plan_kv_attention(seqs, max_new, max_kv, q_heads, kv_heads, head_dim,
                                                window, cu_count, ctypes.byref(p)))
    return p


def plan_kv_shared(seqs: int, tokens: int, max_new: int, max_kv: int, shared: int, q_heads: int,
                   kv_heads: int, head_dim: int, cu_count: int = 0):
    """Default plans of kv_attention over a shared part of whole pages: (the
    pass over it, the pass over the sequences' own keys), or (None, plan)
    where one pass over everything is as fast (no GPU call)."""
    from . import _raise_if, library
    first, own = KVPlan(), KVPlan()
    _raise_if(library().w8a16_plan_kv_shared(seqs, tokens, max_new, max_kv, shared, q_heads, kv_heads,
                                             head_dim, cu_count, ctypes.byref(first), ctypes.byref(own)))
    return (first if first.grid else None), own
