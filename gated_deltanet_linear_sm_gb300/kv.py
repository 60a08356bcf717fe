"""Python binding of the paged key-value cache and the attention over it
(include/gdnspec.h): argument marshalling only, as in binding.py.

Every call has a prepared form, as in ops.py.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import binding
from .binding import _STATE_DTYPES, GdnError
from .ops import _BF16, _F32, _I32, _VP, PreparedOp, PreparedScan, _cuda, _dense, _int32, _ptr, _rows, _shape, _typed

E4M3, I8 = 3, 4
_CACHE_DTYPES = {torch.bfloat16: binding.BF16, torch.float16: binding.F16, torch.float8_e4m3fn: E4M3, torch.int8: I8}


class gdn_kv_dims(ctypes.Structure):
    """Mirror of gdn_kv_dims in include/gdnspec.h."""

    _fields_ = [
        ("batch", ctypes.c_int32), ("num_tokens", ctypes.c_int32), ("H_q", ctypes.c_int32), ("H_kv", ctypes.c_int32),
        ("D", ctypes.c_int32), ("page_size", ctypes.c_int32), ("table_cols", ctypes.c_int32), ("max_T", ctypes.c_int32),
        ("window", ctypes.c_int32), ("reserved", ctypes.c_int32), ("num_pages", ctypes.c_int64),
        ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
        ("scale_page_stride", ctypes.c_int64), ("scale_token_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64),
        ("table_stride", ctypes.c_int64), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64), ("z_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64),
    ]


binding.EXPORTS.update({
    "gdn_kv_write": (ctypes.c_int, [_VP] * 10 + [ctypes.POINTER(gdn_kv_dims), ctypes.c_int, _VP, _VP]),
    "gdn_kv_read": (ctypes.c_int, [_VP] * 9 + [ctypes.POINTER(gdn_kv_dims), ctypes.c_int, ctypes.c_int, _VP, _VP]),
    "gdn_attn_decode": (ctypes.c_int, [_VP] * 12 + [ctypes.c_int64, ctypes.POINTER(gdn_kv_dims), ctypes.c_float, ctypes.c_int,
                                                    _VP, _VP]),
    "gdn_attn_decode_workspace": (ctypes.c_int64, [ctypes.POINTER(gdn_kv_dims), ctypes.c_int]),
})


def _strides(t, other, name, axes):
    """Strides of the first `axes` axes of t, in elements: those of an axis with one entry do not matter and count as
    the other tensor's (0 where it has one entry too); places must not overlap."""
    strides = []
    for a in range(axes):
        s = t.stride(a) if t.shape[a] > 1 else 0
        if other is not None and s != (other.stride(a) if other.shape[a] > 1 else 0):
            raise ValueError(f"{name}: k and v must have the same strides; got {tuple(t.stride())}, {tuple(other.stride())}")
        strides.append(s)
    width = math.prod(t.shape[axes:])
    for s, n in sorted((s, n) for s, n in zip(strides, t.shape) if n > 1):
        if s < width:
            raise ValueError(f"{name}: rows overlap (shape {tuple(t.shape)}, strides {tuple(t.stride())})")
        width = s * (n - 1) + width
    # an axis with one entry: any stride that the kernels' alignment takes
    return [s if s else width for s in strides]


def _cache_shapes(k_cache, v_cache, k_scale, v_scale, page_table, B):
    """Sizes, and what goes by the cache's type; devices and layouts come later (_cache_dims)."""
    _shape(v_cache, "v_cache", tuple(k_cache.shape))
    pages, page, G, D = k_cache.shape
    _shape(page_table, "page_table", (B, None))
    if pages < 1 or page < 1 or G < 1 or page_table.shape[1] < 1:
        raise ValueError(f"expected a cache of at least one page and a page_table [B, at least 1]; got {tuple(k_cache.shape)}, "
                         f"{tuple(page_table.shape)}")
    if D not in (64, 128, 192, 256):
        raise ValueError(f"expected a head dim of 64, 128, 192 or 256; got {D}")
    if k_cache.dtype not in _CACHE_DTYPES:
        raise TypeError(f"k_cache: dtype {k_cache.dtype} not in bf16 / fp16 / float8_e4m3fn / int8")
    small = k_cache.dtype.itemsize == 1
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if (t is not None) != small:
            raise ValueError(f"expected {n} with an 8-bit cache and not with another; got {t if t is None else tuple(t.shape)} with "
                             f"{k_cache.dtype}")
        if small:
            _shape(t, n, (pages, page, G))
    _int32(sequences=B, page_size=page, heads=G, pages_of_a_sequence=page_table.shape[1])


def _cache_dims(k_cache, v_cache, k_scale, v_scale, page_table, dev) -> gdn_kv_dims:
    """Sizes and strides of a cache; the other sizes are left for the caller."""
    _typed(dev, k_cache.dtype, k_cache=k_cache, v_cache=v_cache)
    _typed(dev, _F32, k_scale=k_scale, v_scale=v_scale)
    _typed(dev, _I32, page_table=page_table)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.stride(3) != 1:
            raise ValueError(f"{n}: the elements of a row must be contiguous")
    d = gdn_kv_dims()
    d.num_pages, d.page_size, d.H_kv, d.D = k_cache.shape
    d.H_q, d.max_T = d.H_kv, 1
    d.page_stride, d.token_stride, d.head_stride = _strides(k_cache, v_cache, "k_cache", 3)
    if k_scale is not None:
        d.scale_page_stride, d.scale_token_stride, d.scale_head_stride = _strides(k_scale, v_scale, "k_scale", 3)
    d.batch, d.table_cols = page_table.shape
    d.table_stride = _rows(page_table, "page_table")
    return d


def _sequences(cu_seqlens):
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError(f"expected cu_seqlens [B+1]; got {tuple(cu_seqlens.shape)}")
    return cu_seqlens.shape[0] - 1


# ---- gdn_kv_write ----------------------------------------------------------------


def prepare_kv_write(k, v, k_cache, v_cache, page_table, kv_lens, cu_seqlens, *, k_scale=None, v_scale=None,
                     spec_token_indx=None, status=None) -> PreparedOp:
    """A prepared gdn_kv_write call (see there)."""
    B = _sequences(cu_seqlens)
    _shape(k_cache, "k_cache", (None, None, None, None))
    _shape(k, "k", (None, *k_cache.shape[2:]))
    _shape(v, "v", tuple(k.shape))
    _shape(kv_lens, "kv_lens", (B,))
    _int32(rows=k.shape[0])
    _cache_shapes(k_cache, v_cache, k_scale, v_scale, page_table, B)
    dev = k.device
    _cuda(dev, "gdn_kv_write")
    _typed(dev, _BF16, k=k, v=v)
    d = _cache_dims(k_cache, v_cache, k_scale, v_scale, page_table, dev)
    _dense(dev, kv_lens=kv_lens, cu_seqlens=cu_seqlens, spec_token_indx=spec_token_indx, status=status)
    d.num_tokens = k.shape[0]
    d.k_stride, d.v_stride = _rows(k, "k"), _rows(v, "v")
    return PreparedOp("gdn_kv_write",
                      [_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(page_table),
                       _ptr(kv_lens), _ptr(cu_seqlens), _ptr(spec_token_indx), d, _CACHE_DTYPES[k_cache.dtype], _ptr(status)],
                      dev, (k, v, k_cache, v_cache, k_scale, v_scale, page_table, kv_lens, cu_seqlens, spec_token_indx, status))


def gdn_kv_write(k, v, k_cache, v_cache, page_table, kv_lens, cu_seqlens, *, k_scale=None, v_scale=None,
                 spec_token_indx=None, status=None, stream=None):
    """Rows of keys and values into a paged cache (see include/gdnspec.h): k, v
    [N, H_kv, D] bf16 (rows may be strided); k_cache, v_cache [pages, page_size,
    H_kv, D] bf16 / fp16 / float8_e4m3fn / int8 of the same strides (any order of
    the first three axes), the 8-bit ones with k_scale, v_scale [pages, page_size,
    H_kv] fp32; page_table [B, columns], kv_lens [B] (positions before these rows)
    and cu_seqlens [B+1] int32.  Writes the caches and scales."""
    prepare_kv_write(k, v, k_cache, v_cache, page_table, kv_lens, cu_seqlens, k_scale=k_scale, v_scale=v_scale,
                     spec_token_indx=spec_token_indx, status=status)(stream)


# ---- gdn_kv_read -----------------------------------------------------------------


def prepare_kv_read(k_cache, v_cache, page_table, kv_begin, cu_seqlens, k, v, *, k_scale=None, v_scale=None,
                    status=None) -> PreparedOp:
    """A prepared gdn_kv_read call (see there)."""
    B = _sequences(cu_seqlens)
    _shape(k_cache, "k_cache", (None, None, None, None))
    _shape(k, "k", (None, *k_cache.shape[2:]))
    _shape(v, "v", tuple(k.shape))
    if kv_begin is not None:
        _shape(kv_begin, "kv_begin", (B,))
    _int32(rows=k.shape[0])
    _cache_shapes(k_cache, v_cache, k_scale, v_scale, page_table, B)
    dev = k.device
    _cuda(dev, "gdn_kv_read")
    if k.dtype not in _STATE_DTYPES:
        raise TypeError(f"k: dtype {k.dtype} not in fp32 / bf16 / fp16")
    _typed(dev, k.dtype, v=v)
    d = _cache_dims(k_cache, v_cache, k_scale, v_scale, page_table, dev)
    _dense(dev, kv_begin=kv_begin, cu_seqlens=cu_seqlens, status=status)
    d.num_tokens = k.shape[0]
    d.k_stride, d.v_stride = _rows(k, "k"), _rows(v, "v")
    return PreparedOp("gdn_kv_read",
                      [_ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(page_table), _ptr(kv_begin),
                       _ptr(cu_seqlens), _ptr(k), _ptr(v), d, _CACHE_DTYPES[k_cache.dtype], _STATE_DTYPES[k.dtype], _ptr(status)],
                      dev, (k_cache, v_cache, k_scale, v_scale, page_table, kv_begin, cu_seqlens, k, v, status))


def gdn_kv_read(k_cache, v_cache, page_table, kv_begin, cu_seqlens, k, v, *, k_scale=None, v_scale=None, status=None,
                stream=None):
    """Cached rows back as dense ones (see include/gdnspec.h): positions
    kv_begin[i] + t of sequence i (kv_begin int32 [B], or None: from 0) to rows
    cu_seqlens[i] + t of k and v [N, H_kv, D], fp32 / bf16 / fp16 (rows may be
    strided); the cache as for gdn_kv_write.  Returns (k, v)."""
    prepare_kv_read(k_cache, v_cache, page_table, kv_begin, cu_seqlens, k, v, k_scale=k_scale, v_scale=v_scale,
                    status=status)(stream)
    return k, v


# ---- gdn_attn_decode --------------------------------------------------------------


def prepare_attn_decode(q, k_cache, v_cache, page_table, kv_lens, cu_seqlens, out, *, max_T, k_scale=None, v_scale=None, z=None,
                        scale=None, window=0, spec_token_indx=None, workspace=None, status=None) -> PreparedOp:
    """A prepared gdn_attn_decode call (see there).  Without ``workspace`` each
    of its launches takes one (PreparedScan); with it, calls on two streams or
    from two graphs must not run at the same time."""
    B = _sequences(cu_seqlens)
    _shape(k_cache, "k_cache", (None, None, None, None))
    _shape(q, "q", (None, None, k_cache.shape[3]))
    _shape(out, "out", tuple(q.shape))
    if z is not None:
        _shape(z, "z", tuple(q.shape))
    N, H, D = q.shape
    G = k_cache.shape[2]
    if G < 1 or H < 1 or H % G != 0:
        raise ValueError(f"expected q [N, H, D] with H a multiple of the cache's heads; got H={H}, {G} heads")
    _shape(kv_lens, "kv_lens", (B,))
    _int32(rows=N, heads_of_q=H, max_T=max_T, window=window)
    _cache_shapes(k_cache, v_cache, k_scale, v_scale, page_table, B)
    dev = q.device
    _cuda(dev, "gdn_attn_decode")
    _typed(dev, _BF16, q=q, z=z, out=out)
    d = _cache_dims(k_cache, v_cache, k_scale, v_scale, page_table, dev)
    _dense(dev, kv_lens=kv_lens, cu_seqlens=cu_seqlens, spec_token_indx=spec_token_indx, status=status)
    d.num_tokens, d.H_q, d.max_T, d.window = N, H, max_T, window
    d.q_stride, d.out_stride = _rows(q, "q"), _rows(out, "out")
    d.z_stride = _rows(z, "z") if z is not None else 0
    kind = _CACHE_DTYPES[k_cache.dtype]
    need = attn_decode_workspace(d, k_cache.dtype, dev)
    if workspace is not None:
        _typed(dev, torch.uint8, contiguous=True, workspace=workspace)
        if workspace.numel() < need:
            raise ValueError(f"expected workspace of at least {need} bytes; got {workspace.numel()}")
    args = [_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(page_table), _ptr(kv_lens),
            _ptr(cu_seqlens), _ptr(spec_token_indx), _ptr(z), _ptr(out), _ptr(workspace), need, d,
            1.0 / math.sqrt(D) if scale is None else float(scale), kind, _ptr(status)]
    keep = (q, k_cache, v_cache, k_scale, v_scale, page_table, kv_lens, cu_seqlens, spec_token_indx, z, out, workspace, status)
    if need == 0 or workspace is not None:
        return PreparedOp("gdn_attn_decode", args, dev, keep)
    return PreparedScan("gdn_attn_decode", args, dev, keep, at=11, nbytes=need)


def attn_decode_workspace(dims, cache_dtype, device=None) -> int:
    """Bytes of workspace that gdn_attn_decode needs for these gdn_kv_dims and a
    cache of this torch dtype on the device (default: the current one).  Raises
    GdnError for invalid sizes."""
    with torch.cuda.device(device):
        need = int(binding.load_library().gdn_attn_decode_workspace(ctypes.byref(dims), _CACHE_DTYPES[cache_dtype]))
    if need < 0:
        raise GdnError(2, "invalid sizes of the attention over the cache")
    return need


def gdn_attn_decode(q, k_cache, v_cache, page_table, kv_lens, cu_seqlens, out, *, max_T, k_scale=None, v_scale=None, z=None,
                    scale=None, window=0, spec_token_indx=None, workspace=None, status=None, stream=None):
    """The attention of one to eight tokens of each sequence over its cached keys
    and values, the step's own among them (see include/gdnspec.h): q, out and z
    (a sigmoid gate, or None) [N, H_q, D] bf16 (rows may be strided); the cache
    and its tables as for gdn_kv_write, kv_lens the positions before the step's;
    ``max_T`` bounds every sequence's tokens; ``scale`` of the scores (default
    D^-0.5); ``window``: positions that a token sees, itself included (0: all).
    ``workspace``: uint8, at least what attn_decode_workspace asks for, used by
    this call alone until it has run (default: each launch takes one on its
    stream).  Returns ``out``."""
    prepare_attn_decode(q, k_cache, v_cache, page_table, kv_lens, cu_seqlens, out, max_T=max_T, k_scale=k_scale,
                        v_scale=v_scale, z=z, scale=scale, window=window, spec_token_indx=spec_token_indx, workspace=workspace,
                        status=status)(stream)
    return out
