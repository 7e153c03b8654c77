"""Rotary positions, the paged FP8 cache and attention over it: the part of a
decoder layer between its Q/K/V and output projections.

    cache = kv_cache(pages, kv_heads, page_size, head_dim)
    table = rope_table(positions, rot_dim)
    q = kv_append(cache, k, v, block_table, kv_lens, table=table, q=q)
    out = kv_attention(q, cache, block_table, kv_lens)

Marshalling only, as in the rest of the package: shapes, types and devices
are checked by the native part of the binding (csrc/binding.cpp), everything
else by the C entry points (include/w8a16.h, which defines the operators and
the cache's layout).  Calls run on their tensors' device, on the current (or
given) torch stream, take the memory of their outputs there, and do not
synchronise.
"""

from __future__ import annotations

import ctypes
from contextlib import nullcontext
from typing import NamedTuple, Optional

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
    lib.w8a16_plan_kv_sinks.argtypes = [_u32] * 9 + [ptr(KVPlan)]
    for name in ("w8a16_rope_table", "w8a16_rope", "w8a16_rope_axes", "w8a16_kv_append",
                 "w8a16_kv_append_axes", "w8a16_kv_attention", "w8a16_kv_attention_span",
                 "w8a16_plan_kv_shared", "w8a16_plan_kv_sinks", "w8a16_plan_kv_attention"):
        getattr(lib, name).restype = ctypes.c_int


_state = None
_fast = None       # (native binding, raw stream of a device index, current device index, raise function)


def _setup():
    """(library, torch, raise function, raw stream of a device index),
    resolved once, and the native binding's entry points."""
    global _state, _fast
    if _state is None:
        import torch

        from . import _raise_if, library
        lib = library()
        again = "; run python -m block_scaled_fp8_w8a16_amd.build"
        try:
            from . import _binding
        except ImportError as e:
            raise ImportError("_binding.so cannot be loaded (%s)%s" % (e, again)) from e
        if _binding.torch_version != str(torch.__version__):
            raise ImportError("_binding.so is built for torch %s, this is %s%s" %
                              (_binding.torch_version, torch.__version__, again))
        # what current_stream(device).cuda_stream returns, an order of
        # magnitude faster (0.06 against 1.8 us)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda index: torch.cuda.current_stream(index).cuda_stream)
        current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _binding.bind(*(ctypes.cast(getattr(lib, "w8a16_" + name), _vp).value
                        for name in ("rope", "rope_axes", "kv_append", "kv_append_axes", "kv_attention",
                                     "kv_attention_span", "gemm_epilogue")))
        _fast = (_binding, raw, current, _raise_if)
        _state = (lib, torch, _raise_if, raw)
    return _state


def _run(name, x, stream, *args):
    """Native entry point `name` on the given stream, or the current one of
    x's device."""
    if _fast is None:
        _setup()
    binding, raw, current, check = _fast
    index = x.get_device()
    if stream is None and (index < 0 or index == current()):
        r = getattr(binding, name)(*args, raw(index) if index >= 0 else 0)
    else:
        # outputs are made on the stream that will write them (the current
        # stream's memory might still be written by work that is to come there)
        import torch
        with torch.cuda.device(index) if stream is None else torch.cuda.stream(stream):
            r = getattr(binding, name)(*args, raw(index) if stream is None else stream.cuda_stream)
    if r.__class__ is int:
        check(r)
    return r


def _on(torch, stream):
    """Where a call makes its outputs."""
    return nullcontext() if stream is None else torch.cuda.stream(stream)


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


def rope_table(positions: int, rot_dim: int, *, base: float = 10000.0, scaling: Optional[str] = None,
               factor: float = 1.0, original: float = 0.0, low_turns: float = 1.0,
               high_turns: float = 4.0, magnitude: float = 1.0, out=None, device="cuda", stream=None):
    """float32 [positions, rot_dim / 2, 2]: (cos, sin) of every position and
    pair, times `magnitude`.  scaling: None, "linear", "base" or "bands"
    (w8a16_rope_scaling in include/w8a16.h)."""
    lib, torch, check, raw = _setup()
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
    return _run("rope", x, stream, x, table, positions, out, layout, inverse, sections, order)


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
    return _run("kv_append", k, stream, cache, k, v, block_table, kv_lens, cu_seqlens, max_new, table, layout,
                q, q_out, positions, sections, order)


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
    return _run("kv_attention", q, stream, q, cache, block_table, kv_lens, out, cu_seqlens, max_new, max_kv,
                scale, causal, window, sinks, shared, return_lse,
                0 if plan_ is None else ctypes.addressof(plan_))


def plan_kv_attention(seqs: int, max_new: int, max_kv: int, q_heads: int, kv_heads: int,
                      head_dim: int, window: int = 0, cu_count: int = 0, sinks: int = 0) -> KVPlan:
    """Default plan of kv_attention (no GPU call)."""
    from . import _raise_if, library
    p = KVPlan()
    _raise_if(library().w8a16_plan_kv_sinks(seqs, max_new, max_kv, q_heads, kv_heads, head_dim, window, sinks,
                                            cu_count, ctypes.byref(p)))
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
