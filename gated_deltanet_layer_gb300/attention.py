"""A full-attention layer served beside Gated DeltaNet layers
(include/gdn_attention.h) for torch CUDA tensors: argument marshalling only.

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
from .prefill import _INT_MAX, _bf16, _dense, _empty, _i32, _rows, _stream
from . import prefill as _p

__all__ = ["PagedAttention", "kv_append"]


def _cache(t, name):
    """A [slots, heads, head_dim] bf16 CUDA tensor whose slots' rows are packed: its sizes and slot stride."""
    if t.dtype is not _bf16 or not t.is_cuda or t.dim() != 3 or (_p._several and t.get_device() != _p._device()):
        raise ValueError(f"{name} must be a [slots, heads, head_dim] bf16 CUDA tensor on the current device")
    (n, h, d), (ld, a, b) = t.shape, t.stride()
    if n > _INT_MAX or (n and ((b != 1 and d > 1) or (a != d and h > 1) or (ld < h * d and n > 1))):
        raise ValueError(f"the heads of a slot of {name} must be packed, and its slots must not overlap")
    return n, h, d, ld if n > 1 else -(-h * d // 8) * 8


def kv_append(q, k, v, token_pos, slots, inv_freq, k_cache, v_cache, *, q_norm_w=None, k_norm_w=None, norm_eps=1e-6,
              interleaved=False, q_out=None, error=None, stream=None):
    """Norms and rotation of queries and keys, keys and values into the cache
    (gdn_kv_append). q [T, Hq * d] (None: keys and values alone), k, v [T, Hkv * d]
    (views of the projection's rows will do), token_pos int32 and slots int64 [T],
    inv_freq f32 [rotary_dim / 2] (None: no rotation); k_cache, v_cache [slots, Hkv, d],
    updated; norm weights bf16 [d] or None. q_out may be q; error: int32 [1], optional.
    Returns q_out."""
    n, heads, d, ldkc = _cache(k_cache, "k_cache")
    nv, hv, dv, ldvc = _cache(v_cache, "v_cache")
    ldk, ldv = _rows(k, "k"), _rows(v, "v")
    T, cols = k.shape
    if nv != n or hv != heads or dv != d:
        raise ValueError("k_cache and v_cache have different sizes")
    if cols != heads * d or v.shape != (T, cols):
        raise ValueError(f"k and v must be [tokens, {heads * d}]")
    if T > _INT_MAX:
        raise GdnError("gdn_kv_append", _native.GDN_ERR_UNSUPPORTED)
    qp, ldq, qo, ldqo, hq = None, 0, None, 0, 0
    if q is not None:
        ldq, qp = _rows(q, "q"), q.data_ptr()
        rows, cols = q.shape
        hq = cols // d if d else 0
        if rows != T or hq * d != cols or hq == 0:
            raise ValueError(f"q must be [tokens, heads * {d}]")
        if q_out is None:
            q_out, ldqo = _empty((T, cols), _bf16, q, stream), cols
        else:
            ldqo = _rows(q_out, "q_out")
            if q_out.shape != (T, cols):
                raise ValueError("q_out must have q's shape")
        qo = q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    freq, rotary = None, 0
    if inv_freq is not None:
        rotary = inv_freq.numel()
        freq = _dense(inv_freq, "inv_freq", torch.float32, rotary)
        rotary *= 2
    st = _native.lib().gdn_kv_append(
        T, hq, heads, d, qp, ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, _dense(token_pos, "token_pos", _i32, T),
        _dense(slots, "slots", torch.int64, T), n, freq, rotary, interleaved,
        None if q_norm_w is None else _dense(q_norm_w, "q_norm_w", _bf16, d),
        None if k_norm_w is None else _dense(k_norm_w, "k_norm_w", _bf16, d), norm_eps, qo, ldqo, k_cache.data_ptr(), ldkc,
        v_cache.data_ptr(), ldvc, None if error is None else _dense(error, "error", _i32, 1), _stream(stream))
    if st != GDN_OK:
        raise GdnError("gdn_kv_append", st)
    return q_out


class PagedAttention:
    """Causal attention over a paged cache, bound to one workspace on one device.
    max_tokens and max_seqs bound one call; scale None: head_dim ** -0.5. The handle may be
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
        no request has more new tokens (None: no better bound than T). Returns out."""
        ldq, (T, cols) = _rows(q, "q"), q.shape
        n, heads, d, ldk = _cache(k_cache, "k_cache")
        nv, hv, dv, ldv = _cache(v_cache, "v_cache")
        if heads != self._heads or d != self._d or hv != heads or dv != d or nv != n or n % self._block:
            raise ValueError(f"k_cache and v_cache must be [slots, {self._heads}, {self._d}], whole blocks of {self._block} slots")
        if cols != self._columns:
            raise ValueError(f"q must be [tokens, {self._columns}]")
        S, wide = block_table.shape
        if max_len is None or max_len > T:
            max_len = T
        if T > _INT_MAX or S >= _INT_MAX or wide > _INT_MAX or max_len < 0:
            raise GdnError("gdn_attn_paged", _native.GDN_ERR_ARG)
        gp, ldg = None, 0
        if gate is not None:
            gp, ldg = gate.data_ptr(), _rows(gate, "gate")
            if gate.shape != (T, cols):
                raise ValueError("gate must have q's shape")
        if out is None:
            out, ldo = _empty((T, cols), _bf16, q, stream), cols
        else:
            ldo = _rows(out, "out")
            if out.shape != (T, cols):
                raise ValueError("out must have q's shape")
        st = _native.lib().gdn_attn_paged(
            self._h, S, T, max_len, q.data_ptr(), ldq, k_cache.data_ptr(), ldk, v_cache.data_ptr(), ldv, n // self._block,
            _dense(block_table, "block_table", _i32, S * wide), wide, _dense(cu_seqlens, "cu_seqlens", _i32, S + 1),
            _dense(context_lens, "context_lens", _i32, S), gp, ldg, out.data_ptr(), ldo, self._on(stream))
        if st != GDN_OK:
            raise GdnError("gdn_attn_paged", st)
        return out

    def check(self, stream=None):
        """(status, detail word) of the sticky device error word; synchronises."""
        d = ctypes.c_uint32()
        st = _native.lib().gdn_attn_check(self._h, self._on(stream), ctypes.byref(d))
        return st, d.value

    def reset(self, stream=None):
        st = _native.lib().gdn_attn_reset(self._h, self._on(stream))
        if st != GDN_OK:
            raise GdnError("gdn_attn_reset", st)
