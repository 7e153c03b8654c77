"""Rotary positions, the paged FP8 cache and attention over it: the part of a
decoder layer between its Q/K/V and output projections.

    cache = kv_cache(pages, kv_heads, page_size, head_dim)
    table = rope_table(positions, rot_dim)
    q = kv_append(cache, k, v, block_table, kv_lens, table=table, q=q)
    out = kv_attention(q, cache, block_table, kv_lens)

Marshalling only, as in the rest of the package: shapes, types and devices
are checked here, everything else by the C entry points (include/w8a16.h,
which defines the operators and the cache's layout).  Calls run on the
current (or given) torch stream and do not synchronise.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
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


class KVPlan(ctypes.Structure):
    """w8a16_kv_plan_t"""
    _fields_ = [("kernel", _u32), ("row_blocks", _u32), ("row_tiles", _u32), ("chunk_tiles", _u32),
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


def declare(lib) -> None:
    """Argument types of the entry points."""
    ptr = ctypes.POINTER
    lib.w8a16_rope_table.argtypes = [ptr(RopeConfig), _vp, _u32, _u32, _vp]
    lib.w8a16_rope.argtypes = [_vp, _i64, _i64, _vp, _i64, _i64, _u32, _u32, _u32, _u32, _vp, _u32,
                               _u32, _vp, _u32, _u32, _vp]
    lib.w8a16_kv_append.argtypes = [ptr(KVCacheDesc), ptr(KVSeqs), ptr(KVAppendArgs), _vp]
    lib.w8a16_kv_attention.argtypes = [ptr(KVCacheDesc), ptr(KVSeqs), ptr(KVAttentionArgs), _vp]
    lib.w8a16_plan_kv_attention.argtypes = [_u32] * 8 + [ptr(KVPlan)]
    for name in ("w8a16_rope_table", "w8a16_rope", "w8a16_kv_append", "w8a16_kv_attention",
                 "w8a16_plan_kv_attention"):
        getattr(lib, name).restype = ctypes.c_int


_state = None


def _setup():
    """(library, torch, dtype codes, raise function), resolved once."""
    global _state
    if _state is None:
        import torch

        from . import _raise_if, library
        _state = (library(), torch,
                  {torch.bfloat16: 1, torch.float16: 2, torch.float32: 3}, _raise_if)
    return _state


def _stream(torch, t, stream):
    return (torch.cuda.current_stream(t.device) if stream is None else stream).cuda_stream


class KVCache(NamedTuple):
    """Codes and scale bytes of a paged FP8 cache (uint8 or float8 tensors):
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


def _cache_desc(cache) -> KVCacheDesc:
    k, v, ks, vs = cache
    pages, heads, page, dim = k.shape
    kst, vst, ksst, vsst = k.stride(), v.stride(), ks.stride(), vs.stride()
    blocks = page // KV_BLOCK
    if tuple(v.shape) != (pages, heads, blocks, dim, KV_BLOCK) or \
            tuple(ks.shape) != (pages, heads, blocks) or tuple(vs.shape) != (pages, heads, blocks):
        raise ValueError("cache must be k [pages, heads, page, dim], v [pages, heads, page/16, dim, "
                         "16] and scales [pages, heads, page/16]")
    if kst[1:] != (page * dim, dim, 1) or vst[1:] != (page * dim, dim * KV_BLOCK, KV_BLOCK, 1) or \
            ksst[1:] != (blocks, 1) or vsst[1:] != (blocks, 1):
        raise ValueError("the inside of a cache page must be contiguous")
    if k.element_size() + v.element_size() + ks.element_size() + vs.element_size() != 4:
        raise ValueError("cache tensors must be uint8 or float8")
    if not (k.is_cuda and v.is_cuda and ks.is_cuda and vs.is_cuda):
        raise ValueError("cache must be GPU tensors")
    return KVCacheDesc(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), kst[0], vst[0],
                       ksst[0], vsst[0], pages, page, heads, dim)


def _seqs_desc(torch, block_table, kv_lens, cu_seqlens, tokens, max_new) -> KVSeqs:
    i32 = torch.int32
    seqs = kv_lens.shape[0]
    if block_table.dtype != i32 or kv_lens.dtype != i32 or kv_lens.dim() != 1 or \
            block_table.dim() != 2 or block_table.shape[0] != seqs:
        raise ValueError("block_table must be int32 [seqs, pages] and kv_lens int32 [seqs]")
    if not (block_table.is_cuda and kv_lens.is_cuda):
        raise ValueError("block_table and kv_lens must be GPU tensors")
    width = block_table.shape[1]
    if (width > 1 and block_table.stride(1) != 1) or not kv_lens.is_contiguous():
        raise ValueError("block_table rows and kv_lens must be contiguous")
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
    return KVSeqs(block_table.data_ptr(), kv_lens.data_ptr(), cu,
                  max(block_table.stride(0), width) if seqs < 2 else block_table.stride(0), width,
                  seqs, tokens, max_new)


def _rows(name, t, heads, dim, dtype):
    """Token and head strides of a [tokens, heads, dim] operand."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim or t.dtype != dtype:
        raise ValueError("%s must be %s [tokens, %d, %d]" % (name, dtype, heads, dim))
    s = t.stride()
    if s[2] != 1:
        raise ValueError("%s needs a unit stride along head_dim" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    return s[0], s[1]


def rope_table(positions: int, rot_dim: int, *, base: float = 10000.0, scaling: Optional[str] = None,
               factor: float = 1.0, original: float = 0.0, low_turns: float = 1.0,
               high_turns: float = 4.0, magnitude: float = 1.0, out=None, device="cuda", stream=None):
    """float32 [positions, rot_dim / 2, 2]: (cos, sin) of every position and
    pair, times `magnitude`.  scaling: None, "linear", "base" or "bands"
    (w8a16_rope_scaling in include/w8a16.h)."""
    lib, torch, _, check = _setup()
    if scaling not in ROPE_SCALINGS:
        raise ValueError("scaling must be None, 'linear', 'base' or 'bands'")
    shape = (positions, rot_dim // 2, 2)
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=device)
    if out.dtype != torch.float32 or tuple(out.shape) != shape or not out.is_contiguous() or \
            not out.is_cuda:
        raise ValueError("out must be a contiguous float32 GPU tensor [positions, rot_dim/2, 2]")
    cfg = RopeConfig(base, factor, original, low_turns, high_turns, magnitude, ROPE_SCALINGS[scaling])
    check(lib.w8a16_rope_table(cfg, out.data_ptr(), positions, rot_dim, _stream(torch, out, stream)))
    return out


def _check_table(torch, table, dim):
    if table.dim() != 3 or table.shape[2] != 2 or table.dtype != torch.float32 or \
            not table.is_contiguous() or not table.is_cuda:
        raise ValueError("table must be a contiguous float32 GPU tensor [positions, rot_dim/2, 2]")
    return table.data_ptr(), table.shape[0], 2 * table.shape[1]


def rope(x, table, positions, out=None, *, layout: str = "half", inverse: bool = False, stream=None):
    """x [tokens, heads, head_dim] (bfloat16, float16 or float32) with the
    first 2 * table.shape[1] elements of each head rotated to `positions`
    (int32 [tokens]).  inverse=True rotates back, which is also the gradient:
    dx = rope(dy, ..., inverse=True).  out may be x.  Returns out."""
    lib, torch, dtypes, check = _setup()
    if x.dim() != 3 or x.dtype not in dtypes:
        raise ValueError("x must be bfloat16, float16 or float32 [tokens, heads, head_dim]")
    tokens, heads, dim = x.shape
    xt, xh = _rows("x", x, heads, dim, x.dtype)
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=x.dtype, device=x.device)
    yt, yh = _rows("out", out, heads, dim, x.dtype)
    if out.shape[0] != tokens or positions.shape != (tokens,) or positions.dtype != torch.int32 or \
            not positions.is_contiguous() or not positions.is_cuda:
        raise ValueError("out must have x's shape and positions be a contiguous int32 GPU tensor [tokens]")
    if layout not in ROPE_LAYOUTS:
        raise ValueError("layout must be 'half' or 'interleaved'")
    tp, tn, rot = _check_table(torch, table, dim)
    st = lib.w8a16_rope(x.data_ptr(), xt, xh, out.data_ptr(), yt, yh, dtypes[x.dtype], tokens, heads,
                        dim, tp, tn, rot, positions.data_ptr(), ROPE_LAYOUTS[layout], inverse,
                        _stream(torch, x, stream))
    if st:
        check(st)
    return out


def kv_append(cache, k, v, block_table, kv_lens, *, cu_seqlens=None, max_new: Optional[int] = None,
              table=None, layout: str = "half", q=None, q_out=None, stream=None):
    """Append the new tokens' keys and values (k, v [tokens, kv_heads,
    head_dim]) to `cache`, keys rotated by `table` if given; with q [tokens,
    q_heads, head_dim] also rotate the queries, in the same launch.

    kv_lens int32 [seqs]: tokens each sequence holds with the new ones
    counted.  block_table int32 [seqs, pages].  cu_seqlens int32 [seqs + 1]:
    offsets of the sequences' new tokens; None: tokens / seqs each.  max_new:
    at least the most new tokens of one sequence (None: all tokens; a closer
    bound launches less).  Returns q_out (None without q)."""
    lib, torch, dtypes, check = _setup()
    if k.dim() != 3 or k.dtype not in dtypes:
        raise ValueError("k must be bfloat16, float16 or float32 [tokens, kv_heads, head_dim]")
    tokens, heads, dim = k.shape
    dtype = k.dtype
    desc = _cache_desc(cache)
    if heads != desc.kv_heads or dim != desc.head_dim:
        raise ValueError("k must have the cache's heads and head_dim")
    kt, kh = _rows("k", k, heads, dim, dtype)
    vt, vh = _rows("v", v, heads, dim, dtype)
    if v.shape[0] != tokens:
        raise ValueError("k and v must have the same tokens")
    if layout not in ROPE_LAYOUTS:
        raise ValueError("layout must be 'half' or 'interleaved'")
    args = KVAppendArgs(k.data_ptr(), v.data_ptr(), None, None, kt, kh, vt, vh)
    args.dtype = dtypes[dtype]
    if table is not None:
        args.table, args.table_positions, args.rot_dim = _check_table(torch, table, dim)
        args.layout = ROPE_LAYOUTS[layout]
    if q is not None:
        hq = q.shape[1] if q.dim() == 3 else 0
        args.q_token_stride, args.q_head_stride = _rows("q", q, hq, dim, dtype)
        if q_out is None:
            q_out = torch.empty((tokens, hq, dim), dtype=dtype, device=q.device)
        args.q_out_token_stride, args.q_out_head_stride = _rows("q_out", q_out, hq, dim, dtype)
        if q.shape[0] != tokens or q_out.shape[0] != tokens:
            raise ValueError("q and q_out must have k's tokens")
        args.q, args.q_out, args.q_heads = q.data_ptr(), q_out.data_ptr(), hq
    seqs = _seqs_desc(torch, block_table, kv_lens, cu_seqlens, tokens, max_new)
    st = lib.w8a16_kv_append(desc, seqs, args, _stream(torch, k, stream))
    if st:
        check(st)
    return q_out if q is not None else None


def kv_attention(q, cache, block_table, kv_lens, out=None, *, cu_seqlens=None,
                 max_new: Optional[int] = None, max_kv: Optional[int] = None,
                 scale: Optional[float] = None, causal: bool = True, window: int = 0,
                 return_lse: bool = False, plan_: Optional[KVPlan] = None, stream=None):
    """Attention of the new tokens' queries q [tokens, q_heads, head_dim]
    (bfloat16 or float16) over `cache`.  block_table, kv_lens, cu_seqlens and
    max_new as for kv_append (which has stored the new tokens before);
    max_kv: at least the largest of kv_lens, for the launch's shape (None:
    what the block table can hold).  scale: None for 1 / sqrt(head_dim).
    window: keys a query sees at most, itself counted (0: all).  Returns
    out, or (out, lse) with lse float32 [tokens, q_heads]."""
    lib, torch, dtypes, check = _setup()
    desc = _cache_desc(cache)
    dim = desc.head_dim
    if q.dim() != 3:
        raise ValueError("q must be [tokens, q_heads, head_dim]")
    tokens, heads = q.shape[0], q.shape[1]
    dtype = q.dtype
    if dtype not in dtypes:
        raise ValueError("q must be bfloat16 or float16")
    qt, qh = _rows("q", q, heads, dim, dtype)
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=dtype, device=q.device)
    elif out.shape[0] != tokens:
        raise ValueError("out must have q's tokens")
    ot, oh = _rows("out", out, heads, dim, dtype)
    lse = torch.empty((tokens, heads), dtype=torch.float32, device=q.device) if return_lse else None
    if window < 0:
        raise ValueError("window must not be negative")
    seqs = _seqs_desc(torch, block_table, kv_lens, cu_seqlens, tokens, max_new)
    args = KVAttentionArgs(q.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(),
                           qt, qh, ot, oh, None if plan_ is None else ctypes.pointer(plan_),
                           dim ** -0.5 if scale is None else scale, heads, dtypes[dtype], causal,
                           window, max_kv or 0)
    st = lib.w8a16_kv_attention(desc, seqs, args, _stream(torch, q, stream))
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
