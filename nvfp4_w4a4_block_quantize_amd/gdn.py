"""Python binding of the gated delta layer (include/nvfp4_gdn.h), part of the
package's namespace:

  nvfp4_causal_conv(x, weight, state, slots, token_starts)      -> out
  nvfp4_causal_conv_step(x, weight, state, slots)               -> out
  nvfp4_gated_delta_chunked(q, k, v, a, b, a_log, dt_bias,
                            state, slots, token_starts)         -> out
  nvfp4_gated_delta_step(q, k, v, a, b, a_log, dt_bias,
                         state, slots)                          -> out
  nvfp4_gated_delta_workspace(tokens, n_seqs, k_heads, v_heads,
                              head_k, head_v, dtype)            -> bytes
  nvfp4_group_norm(x, weight)                                   -> out

As in the rest of the binding, only arguments are marshalled here: the kernels
do the work, on torch's current stream of the tensors' device unless a stream is
given, and there is no fallback.  Tensors are checked and read in the native
module that the paged KV cache's binding has too (csrc/gdn_bind.cpp).

States are read in `state` and written in `state_out`, by default `state` itself.
"""
from __future__ import annotations

import ctypes

from . import kv

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_F32 = ctypes.c_float
_CONV = [_I64, _I64, _I64, _I32, _P, _I64, _P, _P, _I32]
_DELTA = [_I64, _I64, _I64, _I64, _I64, _I32, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _P, _I64, _P, _P, _F32, _F32]
# every symbol include/nvfp4_gdn.h declares, with (restype, argtypes)
GDN_SIGNATURES = {
    "nvfp4_causal_conv": (_I32, [*_CONV, _I64, _P, _P, _P, _P, _P, _I64, _P, _I64, _P]),
    "nvfp4_causal_conv_step": (_I32, [*_CONV, _P, _P, _P, _I64, _P, _I64, _P]),
    "nvfp4_gated_delta_chunked": (_I32, [*_DELTA, _I64, _P, _P, _P, _P, _P, _I64, _P, _I64, _I64, _P, _I64, _P]),
    "nvfp4_gated_delta_workspace": (_I32, [_I64, _I64, _I64, _I64, _I64, _I64, _I32, _P]),
    "nvfp4_gated_delta_step": (_I32, [*_DELTA, _P, _P, _P, _I64, _P, _I64, _I64, _P]),
    "nvfp4_group_norm": (_I32, [_I64, _I64, _I64, _I32, _P, _I64, _I64, _P, _I64, _P, _P, _I64, _I64, _I32, _I32, _F32, _P, _I64, _I64,
                                _P]),
}
ACTIVATIONS = {"none": 0, None: 0, "silu": 1}


def _act(name) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be 'none' or 'silu', got {name!r}")
    return ACTIVATIONS[name]


def _pointer(stream):
    return None if stream is None else stream.cuda_stream


def nvfp4_causal_conv(x, weight, state, slots, token_starts, cached_lens=None, bias=None, activation="silu", state_out=None, out=None,
                      stream=None):
    """Causal depthwise convolution of ragged prompts: x [tokens, channels], rows of
    any stride; weight float32 [channels, width], width 2 to 4.

    Sequence r has the rows token_starts[r] to token_starts[r + 1] - 1 (int32
    [n + 1]) and starts from the inputs in state[slots[r]] ([num_slots, width - 1,
    channels] of x's dtype), or from zeros where cached_lens (int32 [n]) is given and
    not positive.  Rows of no sequence stay as they were.  Returns out.
    """
    if kv._bind is None:
        kv._load()
    if out is None:
        out = kv._new(x.shape, x.dtype, x, stream)
    status = kv._bind.causal_conv(x, weight, bias, _act(activation), state, state if state_out is None else state_out, slots, token_starts,
                                  cached_lens, out, _pointer(stream))
    if status:
        kv._nv._check("nvfp4_causal_conv", status)
    return out


def nvfp4_causal_conv_step(x, weight, state, slots, bias=None, activation="silu", state_out=None, out=None, stream=None):
    """The same for one new token a sequence: x [n, channels], row r of the sequence
    in slot slots[r]; a slot that the state does not have (-1) leaves its row out."""
    if kv._bind is None:
        kv._load()
    if out is None:
        out = kv._new(x.shape, x.dtype, x, stream)
    status = kv._bind.causal_conv_step(x, weight, bias, _act(activation), state, state if state_out is None else state_out, slots, out,
                                       _pointer(stream))
    if status:
        kv._nv._check("nvfp4_causal_conv_step", status)
    return out


def nvfp4_gated_delta_workspace(tokens: int, n_seqs: int, k_heads: int, v_heads: int, head_k: int, head_v: int, dtype) -> int:
    """Bytes of workspace that nvfp4_gated_delta_chunked wants for calls of up to these many tokens and sequences."""
    if kv._bind is None:
        kv._load()
    size = ctypes.c_int64(0)
    kv._nv._check("nvfp4_gated_delta_workspace",
                  kv._nv.load_library().nvfp4_gated_delta_workspace(tokens, n_seqs, k_heads, v_heads, head_k, head_v,
                                                                    kv._nv._dtype_code(dtype), ctypes.addressof(size)))
    return size.value


def nvfp4_gated_delta_chunked(q, k, v, a, b, a_log, dt_bias, state, slots, token_starts, cached_lens=None, scale=None, eps: float = 1e-6,
                              state_out=None, out=None, workspace=None, stream=None):
    """The gated delta rule over ragged prompts: q, k [tokens, k_heads, head_k] (not
    normalised yet), v [tokens, v_heads, head_v], a and b [tokens, v_heads] (the
    projected forget gate and write strength), a_log and dt_bias float32 [v_heads].

    Sequences are given as to nvfp4_causal_conv; state is float32 [num_slots,
    v_heads, head_k, head_v].  scale defaults to head_k ** -0.5.  workspace: a byte
    tensor of at least nvfp4_gated_delta_workspace() bytes that no other running call
    uses; by default one comes from torch's allocator for this call.  Returns out,
    shaped like v.
    """
    if kv._bind is None:
        kv._load()
    if q.dim() != 3 or v.dim() != 3 or slots.dim() != 1:  # sizes are read from them here
        raise ValueError(f"q and v must be [tokens, heads, head_dim] and slots [n], got {tuple(q.shape)}, {tuple(v.shape)}, {tuple(slots.shape)}")
    if out is None:
        out = kv._new(v.shape, v.dtype, v, stream)
    if scale is None:
        scale = q.shape[-1] ** -0.5
    if workspace is None:
        if not q.is_cuda:
            raise ValueError("nvfp4_gated_delta_chunked needs GPU tensors")
        size = nvfp4_gated_delta_workspace(q.shape[0], slots.shape[0], q.shape[1], v.shape[1], q.shape[2], v.shape[2], q.dtype)
        workspace = kv._new((size,), kv._torch.uint8, q, stream)
    status = kv._bind.gated_delta_chunked(q, k, v, a, b, a_log, dt_bias, state, state if state_out is None else state_out, scale, eps, out,
                                          slots, token_starts, cached_lens, workspace, _pointer(stream))
    if status:
        kv._nv._check("nvfp4_gated_delta_chunked", status)
    return out


def nvfp4_gated_delta_step(q, k, v, a, b, a_log, dt_bias, state, slots, scale=None, eps: float = 1e-6, state_out=None, out=None,
                           stream=None):
    """The same rule for one new token a sequence: row r of q, k, v, a and b belongs
    to the sequence in slot slots[r]; a slot that the state does not have (-1) leaves
    its row out.  Returns out, shaped like v."""
    if kv._bind is None:
        kv._load()
    if q.dim() != 3:
        raise ValueError(f"q must be [tokens, heads, head_dim], got {tuple(q.shape)}")
    if out is None:
        out = kv._new(v.shape, v.dtype, v, stream)
    status = kv._bind.gated_delta_step(q, k, v, a, b, a_log, dt_bias, state, state if state_out is None else state_out,
                                       q.shape[-1] ** -0.5 if scale is None else scale, eps, out, slots, _pointer(stream))
    if status:
        kv._nv._check("nvfp4_gated_delta_step", status)
    return out


def nvfp4_group_norm(x, weight, bias=None, gate=None, activation="silu", centred: bool = False, eps: float = 1e-6, out=None, stream=None):
    """Each group of x [tokens, groups, group_dim] over the root of its mean square
    (centred: its mean taken off first), times weight plus bias (float32 [group_dim],
    shared by the groups, or [groups, group_dim]), times act(gate); without a gate,
    act of that.  out may be x or gate.  Returns out.
    """
    if kv._bind is None:
        kv._load()
    if out is None:
        out = kv._new(x.shape, x.dtype, x, stream)
    status = kv._bind.group_norm(x, weight, bias, gate, _act(activation), centred, eps, out, _pointer(stream))
    if status:
        kv._nv._check("nvfp4_group_norm", status)
    return out
