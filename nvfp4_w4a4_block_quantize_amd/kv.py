"""Python binding of the paged FP8 KV cache (include/nvfp4_kv.h), part of the
package's namespace:

  nvfp4_kv_block_table(cached_lens, new_lens, page_size, free_pages,
                       free_used, block_table, slot_map)
                -> (seq_lens, token_starts, first_pages, free_used_out)
  nvfp4_rope(q, k, positions, inv_freq, axes)       -> (q_out, k_out)
  nvfp4_kv_cache_write(k, v, k_scale, v_scale,
                       slot_map, k_cache, v_cache)  -> (k_cache, v_cache)
  nvfp4_paged_attention(q, k_cache, v_cache, k_scale, v_scale,
                        block_table, seq_lens)      -> out
  nvfp4_paged_attention_workspace(q_heads, kv_heads, head_dim) -> bytes

As in the rest of the binding, only arguments are marshalled here: the kernels
do the work, on torch's current stream of the tensors' device unless a stream is
given, and there is no fallback.  Several of these calls a layer and token are
short ones, so the tensors are checked and read in a small native module
(csrc/kv_bind.cpp) that calls the same C functions.
"""
from __future__ import annotations

import ctypes

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_F32 = ctypes.c_float
# every symbol include/nvfp4_kv.h declares, with (restype, argtypes)
KV_SIGNATURES = {
    "nvfp4_kv_block_table": (_I32, [_I64, _P, _P, _I64, _P, _I64, _P, _P, _I64, _I64, _P, _I64, _P, _P, _P, _P, _P]),
    "nvfp4_rope": (_I32, [_I64, _I64, _I64, _I32, _I32, _P, _I64, _I64, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64,
                          _P, _P, _I64, _I64, _I64, _I64, _I64, _P]),
    "nvfp4_kv_cache_write": (_I32, [_I64, _I64, _I64, _I32, _P, _I64, _I64, _P, _I64, _I64, _P, _P, _P, _P, _P, _I64,
                                    _I64, _P]),
    "nvfp4_paged_attention": (_I32, [_I64, _I64, _I64, _I64, _I32, _P, _I64, _I64, _P, _P, _I64, _I64, _P, _P, _P,
                                     _I64, _I64, _P, _F32, _I64, _P, _I64, _I64, _P, _P, _I64, _P]),
    "nvfp4_paged_attention_workspace": (_I32, [_I64, _I64, _I64, _P]),
}

_bind = _nv = _torch = None  # the native module, the package and torch, once something is called


def _load():
    global _bind, _nv, _torch
    import nvfp4_w4a4_block_quantize_amd as nv

    _torch = nv._torch()
    nv.load_library()  # raises if nothing is built
    try:
        from . import _kv_bind
    except ModuleNotFoundError:
        raise RuntimeError("_kv_bind.so is missing: it is built where PyTorch is installed "
                           "(python -c 'import __graft_entry__ as g; g.build()')") from None
    _nv, _bind = nv, _kv_bind


def _new(shape, dtype, like, stream):
    """A tensor to fill on `stream`: the allocator knows it by the stream that it is used on."""
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=like.device)
    with _torch.cuda.stream(stream):
        return _torch.empty(shape, dtype=dtype, device=like.device)


def nvfp4_kv_block_table(cached_lens, new_lens, page_size: int, free_pages, free_used, block_table, slot_map,
                         seq_lens=None, token_starts=None, first_pages=None, free_used_out=None, stream=None):
    """Pages for the requests' new tokens, from the free list into the rows of
    block_table, and a slot for every new token into slot_map.

    cached_lens, new_lens int32 [n]; free_pages int32 [any]; free_used int32 [1];
    block_table int32 [n, max_pages]; slot_map int32 [room for the new tokens].
    seq_lens may be cached_lens and free_used_out may be free_used (updated in
    place).  Returns (seq_lens, token_starts, first_pages, free_used_out).
    """
    if _bind is None:
        _load()
    if seq_lens is None:
        seq_lens = _new(cached_lens.shape, _torch.int32, cached_lens, stream)
    if token_starts is None:
        token_starts = _new((cached_lens.numel() + 1,), _torch.int32, cached_lens, stream)
    if first_pages is None:
        first_pages = _new(cached_lens.shape, _torch.int32, cached_lens, stream)
    if free_used_out is None:
        free_used_out = _new((1,), _torch.int32, cached_lens, stream)
    status = _bind.block_table(cached_lens, new_lens, page_size, free_pages, free_used, block_table, slot_map,
                               seq_lens, token_starts, first_pages, free_used_out,
                               None if stream is None else stream.cuda_stream)
    if status:
        _nv._check("nvfp4_kv_block_table", status)
    return seq_lens, token_starts, first_pages, free_used_out


def nvfp4_rope(q, k, positions, inv_freq, axes, adjacent: bool = False, q_out=None, k_out=None, stream=None):
    """Rotary positions on q [tokens, q_heads, head_dim] and k [tokens, k_heads,
    head_dim] (or None): pair i turns by positions[axes[i], token] * inv_freq[i].

    positions int32 [n_axes, tokens], of text one row expanded to all axes;
    inv_freq float32 and axes int32 [rot_dim / 2].  adjacent pairs elements 2i
    and 2i + 1 instead of i and i + rot_dim / 2.  Pass q (k) itself as q_out
    (k_out) to turn in place.
    Returns (q_out, k_out).
    """
    if _bind is None:
        _load()
    if q_out is None:
        q_out = _new(q.shape, q.dtype, q, stream)
    if k_out is None and k is not None:
        k_out = _new(k.shape, k.dtype, k, stream)
    status = _bind.rope(q, k, positions, inv_freq, axes, adjacent, q_out, k_out,
                        None if stream is None else stream.cuda_stream)
    if status:
        _nv._check("nvfp4_rope", status)
    return q_out, k_out


def nvfp4_kv_cache_write(k, v, k_scale, v_scale, slot_map, k_cache, v_cache, stream=None):
    """Quantise the rows of k and v [tokens, kv_heads, head_dim] to E4M3 with
    their static scales, into the cache at their slots (int32 [tokens]; a slot
    outside the cache leaves its token out).  Caches: uint8 [num_pages, kv_heads,
    page_size, head_dim].  Returns (k_cache, v_cache)."""
    if _bind is None:
        _load()
    status = _bind.cache_write(k, v, k_scale, v_scale, slot_map, k_cache, v_cache,
                               None if stream is None else stream.cuda_stream)
    if status:
        _nv._check("nvfp4_kv_cache_write", status)
    return k_cache, v_cache


def nvfp4_paged_attention_workspace(q_heads: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of workspace that nvfp4_paged_attention wants for these heads."""
    if _bind is None:
        _load()
    out = ctypes.c_int64(0)
    _nv._check("nvfp4_paged_attention_workspace",
               _nv.load_library().nvfp4_paged_attention_workspace(q_heads, kv_heads, head_dim, ctypes.addressof(out)))
    return out.value


def nvfp4_paged_attention(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, softmax_scale=None,
                          window: int = 0, out=None, lse=None, workspace=None, stream=None):
    """Attention of one new token per sequence, q [n, q_heads, head_dim], over
    its seq_lens[i] cached tokens (the last `window` of them, 0: all).

    softmax_scale defaults to head_dim ** -0.5.  lse: float32 [n, q_heads] to
    fill, or None.  workspace: a byte tensor of at least
    nvfp4_paged_attention_workspace() bytes that no other running call uses;
    by default one comes from torch's allocator for this call.  Returns out.
    """
    if _bind is None:
        _load()
    if out is None:
        out = _new(q.shape, q.dtype, q, stream)
    if softmax_scale is None:
        softmax_scale = q.shape[-1] ** -0.5
    if workspace is None:
        if not q.is_cuda:
            raise ValueError("nvfp4_paged_attention needs GPU tensors")
        size = nvfp4_paged_attention_workspace(q.shape[1], k_cache.shape[1], q.shape[-1])
        workspace = _new((size,), _torch.uint8, q, stream)
    status = _bind.paged_attention(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, softmax_scale, window,
                                   out, lse, workspace, None if stream is None else stream.cuda_stream)
    if status:
        _nv._check("nvfp4_paged_attention", status)
    return out
