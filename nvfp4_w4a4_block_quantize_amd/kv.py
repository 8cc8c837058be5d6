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
given, and there is no fallback.
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


_nv = _torch = _int32 = None  # the package and torch, once something is called
_device = _raw_stream = None  # torch's current device, and its current stream on one
_fns = {}


def _load():
    global _nv, _torch, _int32, _device, _raw_stream
    import nvfp4_w4a4_block_quantize_amd as nv

    _torch = nv._torch()
    _int32 = _torch.int32
    # the accessors below torch's own skip its per-call initialisation check: a GPU tensor is at hand
    _device = getattr(_torch._C, "_cuda_getDevice", _torch.cuda.current_device)
    _raw_stream = getattr(_torch._C, "_cuda_getCurrentRawStream",
                          lambda index: _torch.cuda.current_stream(index).cuda_stream)
    _nv = nv


def _call(name, like, stream, args):
    """One C call on `like`'s device: on `stream`, else on torch's current stream there."""
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(_nv.load_library(), name)
    index = like.get_device()
    if index < 0:
        raise ValueError(f"{name} needs GPU tensors")
    queue = _raw_stream(index) if stream is None else stream.cuda_stream
    if index == _device():
        status = fn(*args, queue)
    else:
        with _torch.cuda.device(index):
            status = fn(*args, queue)
    if status:
        _nv._check(name, status)


def _ints(t, n, name, index):
    """The address of a dense int32 tensor [n] on device `index`."""
    if t.dtype is _int32 and t.numel() == n and t.dim() == 1 and t.is_contiguous() and t.get_device() == index:
        return t.data_ptr()
    if t.dtype is not _int32:
        raise ValueError(f"{name} must be int32, got {t.dtype}")
    if tuple(t.shape) != (n,):
        raise ValueError(f"{name} must have shape {(n,)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise _elsewhere(t, name, index)


def _elsewhere(t, name, index):
    return ValueError(f"{name} is on {t.device}, expected {'cpu' if index < 0 else f'cuda:{index}'}")


def _scale(t, name, index):
    """The address of a one-element float32 tensor on device `index`."""
    if t.dtype is not _torch.float32 or t.numel() != 1:
        _nv._scalar_f32(t, name)
    if t.get_device() != index:
        raise _elsewhere(t, name, index)
    return t.data_ptr()


def _new(shape, dtype, like, stream):
    """A tensor to fill on `stream`: the allocator knows it by the stream that it is used on."""
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=like.device)
    with _torch.cuda.stream(stream):
        return _torch.empty(shape, dtype=dtype, device=like.device)


def _table(t, rows, index):
    """A block table, int32 with unit column stride: (address, columns, row stride)."""
    shape = t.shape
    if t.dtype is not _int32 or len(shape) != 2 or shape[0] != rows:
        raise ValueError(f"block_table must be int32 [{rows}, pages], got {t.dtype} {tuple(shape)}")
    ld, unit = t.stride()
    if unit != 1 and shape[1] != 1:
        raise ValueError("block_table must have unit column stride")
    if t.get_device() != index:
        raise _elsewhere(t, "block_table", index)
    return t.data_ptr(), shape[1], ld if rows > 1 else shape[1]


def _heads(t, name, shape, dtype, index):
    """[tokens, heads, head_dim] of `shape` and `dtype` on device `index`, with any
    strides between heads and tokens: (address, token stride, head stride).  The
    stride of an axis of one is free."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if len(shape) != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {tuple(shape)}")
    if t.get_device() != index:
        raise _elsewhere(t, name, index)
    token, head, unit = t.stride()
    if unit != 1 and shape[2] != 1:
        raise ValueError(f"{name} must have unit stride along head_dim")
    if shape[1] == 1:
        head = shape[2]
    return t.data_ptr(), token if shape[0] > 1 else shape[1] * head, head


def _cache(k_cache, v_cache, index):
    """Two [num_pages, kv_heads, page_size, head_dim] byte tensors: (addresses, shape)."""
    shape, u8 = k_cache.shape, _torch.uint8
    if len(shape) != 4:
        raise ValueError(f"k_cache must be [num_pages, kv_heads, page_size, head_dim], got {tuple(shape)}")
    if k_cache.dtype is not u8 or not k_cache.is_contiguous():
        _nv._bytes_arg(k_cache, shape, "k_cache")
    if v_cache.dtype is not u8 or v_cache.shape != shape or not v_cache.is_contiguous():
        _nv._bytes_arg(v_cache, shape, "v_cache")
    if k_cache.get_device() != index or v_cache.get_device() != index:
        raise _elsewhere(k_cache if k_cache.get_device() != index else v_cache, "k_cache or v_cache", index)
    return k_cache.data_ptr(), v_cache.data_ptr(), shape


def nvfp4_kv_block_table(cached_lens, new_lens, page_size: int, free_pages, free_used, block_table, slot_map,
                         seq_lens=None, token_starts=None, first_pages=None, free_used_out=None, stream=None):
    """Pages for the requests' new tokens, from the free list into the rows of
    block_table, and a slot for every new token into slot_map.

    cached_lens, new_lens int32 [n]; free_pages int32 [any]; free_used int32 [1];
    block_table int32 [n, max_pages]; slot_map int32 [room for the new tokens].
    seq_lens may be cached_lens and free_used_out may be free_used (updated in
    place).  Returns (seq_lens, token_starts, first_pages, free_used_out).
    """
    if _nv is None:
        _load()
    n = cached_lens.numel() if cached_lens.dim() == 1 else -1
    if n < 0 or free_pages.dim() != 1 or slot_map.dim() != 1:
        raise ValueError("cached_lens, free_pages and slot_map must be 1-D")
    if seq_lens is None:
        seq_lens = _new((n,), _int32, cached_lens, stream)
    if token_starts is None:
        token_starts = _new((n + 1,), _int32, cached_lens, stream)
    if first_pages is None:
        first_pages = _new((n,), _int32, cached_lens, stream)
    if free_used_out is None:
        free_used_out = _new((1,), _int32, cached_lens, stream)
    index = cached_lens.get_device()
    table, max_pages, ld = _table(block_table, n, index)
    n_free, tokens = free_pages.numel(), slot_map.numel()
    _call("nvfp4_kv_block_table", cached_lens, stream,
          (n, _ints(cached_lens, n, "cached_lens", index), _ints(new_lens, n, "new_lens", index), page_size,
           _ints(free_pages, n_free, "free_pages", index), n_free, _ints(free_used, 1, "free_used", index), table,
           max_pages, ld, _ints(slot_map, tokens, "slot_map", index), tokens,
           _ints(seq_lens, n, "seq_lens", index), _ints(token_starts, n + 1, "token_starts", index),
           _ints(first_pages, n, "first_pages", index), _ints(free_used_out, 1, "free_used_out", index)))
    return seq_lens, token_starts, first_pages, free_used_out


def nvfp4_rope(q, k, positions, inv_freq, axes, adjacent: bool = False, q_out=None, k_out=None, stream=None):
    """Rotary positions on q [tokens, q_heads, head_dim] and k [tokens, k_heads,
    head_dim] (or None): pair i turns by positions[axes[i], token] * inv_freq[i].

    positions int32 [n_axes, tokens]; inv_freq float32 and axes int32
    [rot_dim / 2].  adjacent pairs elements 2i and 2i + 1 instead of i and
    i + rot_dim / 2.  Pass q (k) itself as q_out (k_out) to turn in place.
    Returns (q_out, k_out).
    """
    if _nv is None:
        _load()
    if q_out is None:
        q_out = _new(q.shape, q.dtype, q, stream)
    shape, dtype, index = q.shape, q.dtype, q.get_device()
    pq, q_token, q_head = _heads(q, "q", shape, dtype, index)
    po, o_token, o_head = _heads(q_out, "q_out", shape, dtype, index)
    tokens, q_heads, dim = shape
    pos_shape = positions.shape
    if len(pos_shape) != 2 or positions.dtype is not _int32 or pos_shape[1] != tokens:
        raise ValueError(f"positions must be int32 [axes, {tokens}], got {positions.dtype} {tuple(pos_shape)}")
    ld_pos, unit = positions.stride()
    if unit != 1 and tokens != 1:
        raise ValueError("positions must have unit stride along tokens")
    if inv_freq.dim() != 1 or inv_freq.dtype is not _torch.float32 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be float32 [rot_dim / 2], contiguous")
    for t, name in ((positions, "positions"), (inv_freq, "inv_freq")):
        if t.get_device() != index:
            raise _elsewhere(t, name, index)
    pairs, n_axes = inv_freq.shape[0], pos_shape[0]
    keys = (None, None, 0, 0, 0, 0, 0)
    if k is not None:
        k_shape = k.shape
        if k.dtype is not dtype or len(k_shape) != 3 or k_shape[0] != tokens or k_shape[2] != dim:
            raise ValueError(f"k must be {dtype} [{tokens}, heads, {dim}], got {k.dtype} {tuple(k_shape)}")
        if k_out is None:
            k_out = _new(k_shape, dtype, k, stream)
        pk, k_token, k_head = _heads(k, "k", k_shape, dtype, index)
        pko, ko_token, ko_head = _heads(k_out, "k_out", k_shape, dtype, index)
        keys = (pk, pko, k_shape[1], k_token, k_head, ko_token, ko_head)
    elif k_out is not None:
        raise ValueError("k_out without k")
    _call("nvfp4_rope", q, stream,
          (tokens, dim, 2 * pairs, _nv._dtype_code(dtype), int(adjacent), positions.data_ptr(), n_axes,
           ld_pos if n_axes > 1 else tokens, inv_freq.data_ptr(), _ints(axes, pairs, "axes", index), pq, po, q_heads,
           q_token, q_head, o_token, o_head, *keys))
    return q_out, k_out


def nvfp4_kv_cache_write(k, v, k_scale, v_scale, slot_map, k_cache, v_cache, stream=None):
    """Quantise the rows of k and v [tokens, kv_heads, head_dim] to E4M3 with
    their static scales, into the cache at their slots (int32 [tokens]; a slot
    outside the cache leaves its token out).  Caches: uint8 [num_pages, kv_heads,
    page_size, head_dim].  Returns (k_cache, v_cache)."""
    if _nv is None:
        _load()
    shape, dtype, index = k.shape, k.dtype, k.get_device()
    pk, k_token, k_head = _heads(k, "k", shape, dtype, index)
    pv, v_token, v_head = _heads(v, "v", shape, dtype, index)
    tokens, heads, dim = shape
    ck, cv, (pages, kv_heads, page_size, d) = _cache(k_cache, v_cache, index)
    if kv_heads != heads or d != dim:
        raise ValueError(f"k_cache must be [pages, {heads}, page_size, {dim}], got {tuple(k_cache.shape)}")
    _call("nvfp4_kv_cache_write", k, stream,
          (tokens, heads, dim, _nv._dtype_code(dtype), pk, k_token, k_head, pv, v_token, v_head,
           _scale(k_scale, "k_scale", index), _scale(v_scale, "v_scale", index),
           _ints(slot_map, tokens, "slot_map", index),
           ck, cv, pages, page_size))
    return k_cache, v_cache


def nvfp4_paged_attention_workspace(q_heads: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of workspace that nvfp4_paged_attention wants for these heads on the current device."""
    if _nv is None:
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
    if _nv is None:
        _load()
    if out is None:
        out = _new(q.shape, q.dtype, q, stream)
    shape, dtype, index = q.shape, q.dtype, q.get_device()
    pq, q_token, q_head = _heads(q, "q", shape, dtype, index)
    po, o_token, o_head = _heads(out, "out", shape, dtype, index)
    n, heads, dim = shape
    ck, cv, (pages, kv_heads, page_size, d) = _cache(k_cache, v_cache, index)
    if d != dim:
        raise ValueError(f"k_cache has head_dim {d}, q has {dim}")
    table, max_pages, ld = _table(block_table, n, index)
    if lse is not None:
        if lse.dtype is not _torch.float32 or lse.shape != (n, heads) or not lse.is_contiguous():
            raise ValueError(f"lse must be float32 [{n}, {heads}], contiguous")
        if lse.get_device() != index:
            raise _elsewhere(lse, "lse", index)
    if workspace is None:
        if index < 0:
            raise ValueError("nvfp4_paged_attention needs GPU tensors")
        with _torch.cuda.device(q.device):
            size = nvfp4_paged_attention_workspace(heads, kv_heads, dim)
        workspace = _new((size,), _torch.uint8, q, stream)
    elif workspace.dtype is not _torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    elif workspace.get_device() != index:
        raise _elsewhere(workspace, "workspace", index)
    _call("nvfp4_paged_attention", q, stream,
          (n, heads, kv_heads, dim, _nv._dtype_code(dtype), pq, q_token, q_head, ck, cv, pages, page_size,
           _scale(k_scale, "k_scale", index), _scale(v_scale, "v_scale", index), table, max_pages, ld,
           _ints(seq_lens, n, "seq_lens", index), dim ** -0.5 if softmax_scale is None else softmax_scale, window, po,
           o_token, o_head, None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel()))
    return out
