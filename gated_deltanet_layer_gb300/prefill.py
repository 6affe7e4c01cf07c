"""The prompt side of a Gated DeltaNet layer (include/gdn_prefill.h) for torch
CUDA tensors: argument marshalling only, as for the decode step.

`slot_map` turns request lengths into offsets, block tables and slots,
`linear` runs a projection with its epilogue, and `GdnPrefill` the conv and the
gated delta rule over ragged prompts; the states they leave are those
`GdnDecode.step` continues from.
"""
from __future__ import annotations

import ctypes
from collections import namedtuple

import torch

from . import _native
from ._native import (GDN_ACT_GELU_TANH, GDN_ACT_NONE, GDN_ACT_SILU, GDN_OK, GDN_STATE_BF16, GDN_STATE_F32, GdnError)

__all__ = ["GdnPrefill", "SlotMap", "linear", "linear_check", "slot_map"]

ACTIVATIONS = {None: GDN_ACT_NONE, "none": GDN_ACT_NONE, "silu": GDN_ACT_SILU, "gelu": GDN_ACT_GELU_TANH}

SlotMap = namedtuple("SlotMap", "cu_seqlens token_seq token_pos slots free_count")

_bf16, _i32 = torch.bfloat16, torch.int32


def _stream(stream, device):
    return (stream if stream is not None else torch.cuda.current_stream(device)).cuda_stream


def _rows(t, name, dtype=_bf16):
    """A [rows, columns] CUDA tensor with packed columns; its row stride."""
    if t.dim() != 2 or t.dtype is not dtype or not t.is_cuda:
        raise ValueError(f"{name} must be a two-dimensional {dtype} CUDA tensor")
    rows, ld = t.shape[0], t.stride(0)
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"the columns of {name} must be packed")
    if rows <= 1 or ld < t.shape[1]:
        if rows > 1:
            raise ValueError(f"the rows of {name} must not overlap")
        return -(-t.shape[1] // 8) * 8  # a single row's stride does not matter
    return ld


def _dense(t, name, dtype, shape=None):
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous() or (shape is not None and tuple(t.shape) != shape):
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor" + (f" of shape {shape}" if shape else ""))
    return t.data_ptr()


def linear(x, w, bias=None, activation=None, residual=None, out=None, stream=None):
    """out = act(x w^T + bias) + residual: x [M, K], w [N, K], bias [N],
    residual and out [M, N], bf16, rows at any stride that is a multiple of 8
    (x, w). activation: None, "silu" or "gelu" (tanh form). out may be
    residual. Returns out."""
    ldx, ldw = _rows(x, "x"), _rows(w, "w")
    (M, K), N = x.shape, w.shape[0]
    if w.shape[1] != K:
        raise ValueError("x and w have different inner sizes")
    if out is None:
        out = torch.empty((M, N), dtype=_bf16, device=x.device)
    elif out.shape != (M, N):
        raise ValueError("out must be [M, N]")
    ldr = 0
    if residual is not None:
        if residual.shape != (M, N):
            raise ValueError("residual must be [M, N]")
        ldr = _rows(residual, "residual")
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    st = _native.lib().gdn_linear(
        M, N, K, x.data_ptr(), ldx, w.data_ptr(), ldw, None if bias is None else _dense(bias, "bias", _bf16, (N,)),
        ACTIVATIONS[activation], None if residual is None else residual.data_ptr(), ldr, out.data_ptr(),
        _rows(out, "out"), _stream(stream, x.device))
    if st != GDN_OK:
        raise GdnError("gdn_linear", st)
    return out


def linear_check(stream=None):
    """(status, detail word) of the device's gdn_linear calls; synchronises
    and clears the word."""
    d = ctypes.c_uint32()
    st = _native.lib().gdn_linear_check(_stream(stream, None), ctypes.byref(d))
    return st, d.value


def slot_map(new_lens, context_lens, block_size, block_table, free_list, free_count, tokens, *, out=None, error=None,
             stream=None):
    """Offsets, block tables and slots of a ragged step (gdn_slot_map).
    new_lens, context_lens [R], block_table [R, max_blocks] (updated),
    free_list [F], free_count [1], int32; tokens: rows of the step (at least
    the sum of new_lens). `out`: a SlotMap to write into (its free_count not
    this call's); error: int32 [1], optional. Returns a SlotMap of int32
    cu_seqlens [R + 1], token_seq [tokens], token_pos [tokens], int64 slots
    [tokens] and int32 free_count [1]."""
    R, dev = new_lens.shape[0], new_lens.device
    if block_table.dim() != 2 or block_table.shape[0] != R:
        raise ValueError("block_table must be [requests, max_blocks]")
    if out is None:
        i = torch.empty(R + 2 + 2 * tokens, dtype=_i32, device=dev)
        cu, seq, pos, left = i.split((R + 1, tokens, tokens, 1))
        out = SlotMap(cu, seq, pos, torch.empty(tokens, dtype=torch.int64, device=dev), left)
    st = _native.lib().gdn_slot_map(
        R, tokens, _dense(new_lens, "new_lens", _i32), _dense(context_lens, "context_lens", _i32, (R,)), block_size,
        block_table.shape[1], _dense(block_table, "block_table", _i32), _dense(free_list, "free_list", _i32),
        free_list.numel(), _dense(free_count, "free_count", _i32, (1,)), _dense(out.free_count, "free_count", _i32, (1,)),
        _dense(out.cu_seqlens, "cu_seqlens", _i32, (R + 1,)), _dense(out.token_seq, "token_seq", _i32, (tokens,)),
        _dense(out.token_pos, "token_pos", _i32, (tokens,)), _dense(out.slots, "slots", torch.int64, (tokens,)),
        None if error is None else _dense(error, "error", _i32, (1,)), _stream(stream, dev))
    if st != GDN_OK:
        raise GdnError("gdn_slot_map", st)
    return out


class GdnPrefill:
    """The conv and the gated delta rule of one GDN layer shape over ragged
    prompts, bound to one workspace on one device. `shape` has the fields of
    workloads.LayerShape; max_tokens and max_seqs bound one call."""

    def __init__(self, shape, *, max_tokens: int, max_seqs: int, stream=None):
        L = _native.lib()
        self.shape = shape
        self.cfg = _native.PrefillConfig(
            num_k_heads=shape.num_k_heads, num_v_heads=shape.num_v_heads, head_k_dim=shape.head_k_dim,
            head_v_dim=shape.head_v_dim, conv_kernel=shape.conv_kernel, num_slots=shape.num_slots,
            max_tokens=max_tokens, max_seqs=max_seqs,
            ssm_dtype=GDN_STATE_BF16 if shape.ssm_dtype == "bf16" else GDN_STATE_F32,
            gated_norm_eps=shape.gated_norm_eps, l2_eps=shape.l2_eps,
            q_scale=shape.q_scale if shape.q_scale is not None else float(shape.head_k_dim) ** -0.5)
        n = L.gdn_prefill_workspace_bytes(ctypes.byref(self.cfg))
        if n == 0:
            raise GdnError("gdn_prefill_workspace_bytes", _native.GDN_ERR_UNSUPPORTED)
        self.workspace = torch.empty(n, dtype=torch.uint8, device="cuda")
        self._channels = 2 * shape.num_k_heads * shape.head_k_dim + shape.num_v_heads * shape.head_v_dim
        self._columns = shape.num_v_heads * shape.head_v_dim
        self._state = (torch.bfloat16 if shape.ssm_dtype == "bf16" else torch.float32,
                       (shape.num_slots, shape.num_v_heads, shape.head_v_dim, shape.head_k_dim))
        h = ctypes.c_void_p()
        st = L.gdn_prefill_create(ctypes.byref(self.cfg), self.workspace.data_ptr(), n,
                                  _stream(stream, self.workspace.device), ctypes.byref(h))
        if st != GDN_OK:
            raise GdnError("gdn_prefill_create", st)
        self._h = h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            _native.lib().gdn_prefill_destroy(h)
            self._h = None

    def _out(self, out, like, cols):
        if out is None:
            return torch.empty((like.shape[0], cols), dtype=_bf16, device=like.device)
        if out.shape != (like.shape[0], cols):
            raise ValueError(f"out must be [tokens, {cols}]")
        return out

    def conv(self, x, conv_w, cu_seqlens, state_in, state_out, conv_state, out=None, stream=None):
        """Causal conv1d + SiLU over the rows x [tokens, C] (a view of the
        projection's rows will do); sequences are cu_seqlens [S + 1], their
        slots state_in and state_out [S]. conv_state [slots, C, 3] is updated.
        Returns out [tokens, C]."""
        C, S = self._channels, state_in.shape[0]
        if x.shape[1] != C:
            raise ValueError(f"x must be [tokens, {C}]")
        out = self._out(out, x, C)
        st = _native.lib().gdn_prefill_conv(
            self._h, S, x.shape[0], x.data_ptr(), _rows(x, "x"), _dense(conv_w, "conv_w", _bf16, (C, 4)),
            _dense(cu_seqlens, "cu_seqlens", _i32, (S + 1,)), _dense(state_in, "state_in", _i32),
            _dense(state_out, "state_out", _i32, (S,)),
            _dense(conv_state, "conv_state", _bf16, (self.shape.num_slots, C, 3)), out.data_ptr(), _rows(out, "out"),
            _stream(stream, x.device))
        if st != GDN_OK:
            raise GdnError("gdn_prefill_conv", st)
        return out

    def delta(self, qkv, ba, weights: dict, cu_seqlens, state_in, state_out, ssm_state, z=None, out=None, max_len=None,
              stream=None):
        """The gated delta rule over the conv's rows qkv [tokens, C] and the
        projection's ba [tokens, 2 Hv]; `weights` holds A_log, dt_bias and, with
        the gate z [tokens, Hv*dv], gated_norm_w. ssm_state is updated. max_len:
        no sequence is longer (None: no better bound than the rows). Returns
        core [tokens, Hv*dv]."""
        C, S, Hv = self._channels, state_in.shape[0], self.shape.num_v_heads
        T = qkv.shape[0]
        if qkv.shape[1] != C or ba.shape != (T, 2 * Hv) or (z is not None and z.shape != (T, self._columns)):
            raise ValueError("qkv, ba and z must be [tokens, C], [tokens, 2 Hv] and [tokens, Hv*dv]")
        out = self._out(out, qkv, self._columns)
        st = _native.lib().gdn_prefill_delta(
            self._h, S, T, T if max_len is None else max_len, qkv.data_ptr(), _rows(qkv, "qkv"),
            None if z is None else z.data_ptr(), 0 if z is None else _rows(z, "z"), ba.data_ptr(), _rows(ba, "ba"),
            _dense(weights["A_log"], "A_log", torch.float32, (Hv,)), _dense(weights["dt_bias"], "dt_bias", _bf16, (Hv,)),
            None if z is None else _dense(weights["gated_norm_w"], "gated_norm_w", _bf16, (self.shape.head_v_dim,)),
            _dense(cu_seqlens, "cu_seqlens", _i32, (S + 1,)), _dense(state_in, "state_in", _i32),
            _dense(state_out, "state_out", _i32, (S,)), _dense(ssm_state, "ssm_state", *self._state), out.data_ptr(),
            _rows(out, "out"), _stream(stream, qkv.device))
        if st != GDN_OK:
            raise GdnError("gdn_prefill_delta", st)
        return out

    def check(self, stream=None):
        """(status, detail word) of the sticky device error word; synchronises."""
        d = ctypes.c_uint32()
        st = _native.lib().gdn_prefill_check(self._h, _stream(stream, self.workspace.device), ctypes.byref(d))
        return st, d.value

    def reset(self, stream=None):
        st = _native.lib().gdn_prefill_reset(self._h, _stream(stream, self.workspace.device))
        if st != GDN_OK:
            raise GdnError("gdn_prefill_reset", st)
