"""A full-attention layer served beside Gated DeltaNet layers
(include/gdn_attention.h) for torch CUDA tensors: argument marshalling only,
compiled where a call is short (csrc/gdn_binding.cpp).

`kv_append` normalises and rotates a step's queries and keys and puts keys and
values into a paged cache, `PagedAttention.attend` runs causal attention over the
pages. Offsets, positions, slots and block tables are those of `slot_map`. Devices,
streams and what a call allocates are as in prefill.py.
"""
from __future__ import annotations

import ctypes

import torch

from . import _native
from ._native import GDN_OK, GdnError
from .prefill import _INT_MAX, _empty, _stream

__all__ = ["PagedAttention", "kv_append"]


def kv_append(q, k, v, token_pos, slots, inv_freq, k_cache, v_cache, *, q_norm_w=None, k_norm_w=None, norm_eps=1e-6,
              interleaved=False, q_out=None, error=None, stream=None):
    """Norms and rotation of queries and keys, keys and values into the cache
    (gdn_kv_append). q [T, Hq * d] (None: keys and values alone), k, v [T, Hkv * d]
    (views of the projection's rows will do), token_pos int32 and slots int64 [T],
    inv_freq f32 [rotary_dim / 2] (None: no rotation); k_cache, v_cache [slots, Hkv, d],
    updated; norm weights bf16 [d] or None. q_out may be q; error: int32 [1], optional.
    Returns q_out."""
    if stream is not None:
        if q is not None and q_out is None:
            q_out = _empty(q.shape, q.dtype, q, stream)
        stream = _stream(stream)
    r = _native.calls().kv_append(stream, q, k, v, token_pos, slots, inv_freq, k_cache, v_cache, q_norm_w, k_norm_w, norm_eps,
                                  interleaved, q_out, error)
    if r.__class__ is int:
        raise GdnError("gdn_kv_append", r)
    return r


class PagedAttention:
    """Causal attention over a paged cache, bound to one workspace on one device.
    max_tokens and max_seqs bound one call; scale None: head_dim ** -0.5. Making it waits for
    its stream, so that calls on other streams find the workspace cleared. The handle may be
    dropped while its calls run; a graph that captured them needs it for as long as it is
    replayed."""

    def __init__(self, num_q_heads, num_kv_heads, head_dim, block_size, *, max_tokens: int, max_seqs: int, scale=None,
                 stream=None):
        L = _native.lib()
        sizes = (num_q_heads, num_kv_heads, head_dim, block_size, max_tokens, max_seqs)
        if max(sizes) > _INT_MAX or min(sizes) < 0:
            raise GdnError("gdn_attn_create", _native.GDN_ERR_ARG)
        self.cfg = _native.AttnConfig(num_q_heads=num_q_heads, num_kv_heads=num_kv_heads, head_dim=head_dim,
                                      block_size=block_size, max_tokens=max_tokens, max_seqs=max_seqs,
                                      scale=float(head_dim) ** -0.5 if scale is None and head_dim else scale or 0.0)
        n = L.gdn_attn_workspace_bytes(ctypes.byref(self.cfg))
        if n == 0:
            raise GdnError("gdn_attn_workspace_bytes", _native.GDN_ERR_UNSUPPORTED)
        with torch.cuda.stream(stream):  # None: the current one
            self.workspace = torch.empty(n, dtype=torch.uint8, device="cuda")
        self._home = _stream(stream)  # the stream whose memory it is
        self._heads, self._d, self._block, self._columns = num_kv_heads, head_dim, block_size, num_q_heads * head_dim
        h = ctypes.c_void_p()
        st = L.gdn_attn_create(ctypes.byref(self.cfg), self.workspace.data_ptr(), n, self._home, ctypes.byref(h))
        if st != GDN_OK:
            raise GdnError("gdn_attn_create", st)
        self._h = h
        with torch.cuda.stream(stream):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            _native.lib().gdn_attn_destroy(h)
            self._h = None

    def _on(self, stream):
        """The stream of a call, as a number. The workspace is kept until what runs there is
        done, also past the handle's end."""
        st = _stream(stream)
        if st != self._home:
            self.workspace.record_stream(stream if stream is not None else torch.cuda.current_stream())
        return st

    def attend(self, q, k_cache, v_cache, block_table, cu_seqlens, context_lens, gate=None, out=None, max_len=None,
               stream=None):
        """softmax(scale q k^T) v of every request's new tokens over its context and
        themselves, times sigmoid(gate) if given (gdn_attn_paged). q, gate, out
        [T, Hq * d], k_cache, v_cache [slots, Hkv, d] (slots a multiple of the block
        size), block_table int32 [S, blocks], cu_seqlens [S + 1], context_lens [S]. max_len:
        no request has more new tokens (None: no better bound than T, with which single tokens
        take the chunks' form, up to half as long again). Returns out."""
        if stream is not None:
            if out is None:
                out = _empty(q.shape, q.dtype, q, stream)
            stream = self._on(stream)
        r = _native.calls().attend(stream, self._h.value, self.workspace, self._home, self._heads, self._d, self._block, self._columns,
                                   q, k_cache, v_cache, block_table, cu_seqlens, context_lens, gate, out, max_len)
        if r.__class__ is int:
            raise GdnError("gdn_attn_paged", r)
        return r

    def check(self, stream=None):
        """(status, detail word) of the sticky device error word; synchronises."""
        d = ctypes.c_uint32()
        st = _native.lib().gdn_attn_check(self._h, self._on(stream), ctypes.byref(d))
        return st, d.value

    def reset(self, stream=None):
        st = _native.lib().gdn_attn_reset(self._h, self._on(stream))
        if st != GDN_OK:
            raise GdnError("gdn_attn_reset", st)
