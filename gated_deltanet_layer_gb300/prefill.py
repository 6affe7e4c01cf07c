"""The prompt side of a Gated DeltaNet layer (include/gdn_prefill.h) for torch
CUDA tensors: argument marshalling only, as for the decode step.

`slot_map` turns request lengths into offsets, block tables and slots,
`linear` runs a projection with its epilogue, and `GdnPrefill` the conv and the
gated delta rule over ragged prompts; the states they leave are those
`GdnDecode.step` continues from. Every call runs on the current device, where
its tensors must be, and on the current stream, or on `stream`; what it
allocates is allocated there, and tensors of another stream are the caller's to
order and to keep (Tensor.record_stream).
"""
from __future__ import annotations

import ctypes
from collections import namedtuple

import torch

from . import _native
from ._native import (GDN_ACT_GELU_TANH, GDN_ACT_NONE, GDN_ACT_SILU, GDN_OK, GDN_STATE_BF16, GDN_STATE_F32,
                      GdnError)

__all__ = ["GdnPrefill", "SlotMap", "linear", "linear_check", "slot_map"]

ACTIVATIONS = {None: GDN_ACT_NONE, "none": GDN_ACT_NONE, "silu": GDN_ACT_SILU, "gelu": GDN_ACT_GELU_TANH}

SlotMap = namedtuple("SlotMap", "cu_seqlens token_seq token_pos slots free_count")

_bf16, _i32 = torch.bfloat16, torch.int32
_INT_MAX = 2**31 - 1  # sizes cross the C ABI as int32, and ctypes would cut what is larger


# The calling thread's current stream as a number, without building a Stream object.
_raw_stream = torch._C._cuda_getCurrentRawStream


# The calling thread's current device, where the library launches.
_device = torch._C._cuda_getDevice
# Whether this process sees several devices (2: not known yet); with one there is no other to
# be on, and asking each tensor for its own takes 2 us a call.
_several = 2


def _stream(stream):
    """The stream of a call, as a number; one of the current device."""
    global _several
    if _several == 2:
        _several = torch.cuda.device_count() > 1
    if stream is None:
        return _raw_stream(_device())
    if _several and stream.device_index != _device():
        raise ValueError("the stream must be one of the current device")
    return stream.cuda_stream


def _empty(size, dtype, like, stream):
    """A new tensor on like's device, in the memory of the stream that writes it first."""
    if stream is None:
        return torch.empty(size, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(size, dtype=dtype, device=like.device)


def _rows(t, name):
    """A [rows, columns] bf16 CUDA tensor with packed columns; its row stride."""
    if t.dtype is not _bf16 or not t.is_cuda or t.dim() != 2 or (_several and t.get_device() != _device()):
        raise ValueError(f"{name} must be a two-dimensional bf16 CUDA tensor on the current device")
    (rows, cols), (ld, unit) = t.shape, t.stride()
    if unit != 1 and cols > 1 and rows:
        raise ValueError(f"the columns of {name} must be packed")
    if rows > 1 and ld >= cols:
        return ld
    if rows > 1:
        raise ValueError(f"the rows of {name} must not overlap")
    return -(-cols // 8) * 8  # the stride of one row, or none, does not matter


def _dense(t, name, dtype, n):
    """The address of a contiguous CUDA tensor of n values."""
    if (t.dtype is not dtype or not t.is_cuda or not t.is_contiguous() or t.numel() != n
            or (_several and t.get_device() != _device())):
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of {n} values on the current device")
    return t.data_ptr()


def linear(x, w, bias=None, activation=None, residual=None, out=None, stream=None):
    """out = act(x w^T + bias) + residual: x [M, K], w [N, K], bias [N],
    residual and out [M, N], bf16, rows at any stride that is a multiple of 8
    (x, w). activation: None, "silu" or "gelu" (tanh form). out may be
    residual. Returns out."""
    ldx, ldw = _rows(x, "x"), _rows(w, "w")
    (M, K), (N, inner) = x.shape, w.shape
    if inner != K:
        raise ValueError("x and w have different inner sizes")
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    if M > _INT_MAX or N > _INT_MAX or K > _INT_MAX:
        raise GdnError("gdn_linear", _native.GDN_ERR_UNSUPPORTED)
    if out is None:
        out, ldo = _empty((M, N), _bf16, x, stream), N
    else:
        ldo = _rows(out, "out")
        if out.shape != (M, N):
            raise ValueError("out must be [M, N]")
    r, ldr = None, 0
    if residual is not None:
        r, ldr = residual.data_ptr(), _rows(residual, "residual")
        if residual.shape != (M, N):
            raise ValueError("residual must be [M, N]")
    st = _native.lib().gdn_linear(
        M, N, K, x.data_ptr(), ldx, w.data_ptr(), ldw, None if bias is None else _dense(bias, "bias", _bf16, N),
        ACTIVATIONS[activation], r, ldr, out.data_ptr(), ldo, _stream(stream))
    if st != GDN_OK:
        raise GdnError("gdn_linear", st)
    return out


def linear_check(stream=None):
    """(status, detail word) of the device's gdn_linear calls; synchronises
    and clears the word."""
    d = ctypes.c_uint32()
    s = _stream(stream) if stream is not None else torch.cuda.current_stream().cuda_stream
    st = _native.lib().gdn_linear_check(s, ctypes.byref(d))
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
    R, wide = block_table.shape
    n = R + 1
    if not 0 < block_size <= _INT_MAX or not 0 <= tokens <= _INT_MAX or max(R, wide, free_list.numel()) > _INT_MAX:
        raise GdnError("gdn_slot_map", _native.GDN_ERR_ARG)
    if out is None:
        # one allocation; the rows' arrays on 16 bytes
        up = -(-tokens // 4) * 4
        i = _empty(2 * up + n + 1, _i32, new_lens, stream)
        a, b, c, d = i.split_with_sizes((up, up, n, 1))
        if up != tokens:
            a, b = a[:tokens], b[:tokens]
        out = SlotMap(c, a, b, _empty(tokens, torch.int64, new_lens, stream), d)
        seq = i.data_ptr()
        pos = seq + 4 * up
        cu = pos + 4 * up
        left, slots = cu + 4 * n, out.slots.data_ptr()
    else:
        cu, seq, pos = (_dense(t, "out", _i32, m) for t, m in zip(out, (n, tokens, tokens)))
        slots, left = _dense(out.slots, "slots", torch.int64, tokens), _dense(out.free_count, "free_count", _i32, 1)
    st = _native.lib().gdn_slot_map(
        R, tokens, _dense(new_lens, "new_lens", _i32, R), _dense(context_lens, "context_lens", _i32, R), block_size, wide,
        _dense(block_table, "block_table", _i32, R * wide), _dense(free_list, "free_list", _i32, free_list.numel()),
        free_list.numel(), _dense(free_count, "free_count", _i32, 1), left, cu, seq, pos, slots,
        None if error is None else _dense(error, "error", _i32, 1), _stream(stream))
    if st != GDN_OK:
        raise GdnError("gdn_slot_map", st)
    return out


class GdnPrefill:
    """The conv and the gated delta rule of one GDN layer shape over ragged
    prompts, bound to one workspace on one device. `shape` has the fields of
    workloads.LayerShape; max_tokens and max_seqs bound one call. The handle may be
    dropped while its calls run; a graph that captured them needs it for as long
    as it is replayed."""

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
        sizes = (shape.num_k_heads, shape.num_v_heads, shape.head_k_dim, shape.head_v_dim, shape.conv_kernel,
                 shape.num_slots, max_tokens, max_seqs)
        if max(sizes) > _INT_MAX or min(sizes) < 0:
            raise GdnError("gdn_prefill_create", _native.GDN_ERR_ARG)
        n = L.gdn_prefill_workspace_bytes(ctypes.byref(self.cfg))
        if n == 0:
            raise GdnError("gdn_prefill_workspace_bytes", _native.GDN_ERR_UNSUPPORTED)
        with torch.cuda.stream(stream):  # None: the current one
            self.workspace = torch.empty(n, dtype=torch.uint8, device="cuda")
        self._home = _stream(stream)  # the stream whose memory it is
        self._channels = 2 * shape.num_k_heads * shape.head_k_dim + shape.num_v_heads * shape.head_v_dim
        self._columns = shape.num_v_heads * shape.head_v_dim
        self._state = torch.bfloat16 if shape.ssm_dtype == "bf16" else torch.float32
        self._state_values = shape.num_slots * self._columns * shape.head_k_dim
        self._conv_values = shape.num_slots * self._channels * 3
        h = ctypes.c_void_p()
        st = L.gdn_prefill_create(ctypes.byref(self.cfg), self.workspace.data_ptr(), n, self._home, ctypes.byref(h))
        if st != GDN_OK:
            raise GdnError("gdn_prefill_create", st)
        self._h = h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            _native.lib().gdn_prefill_destroy(h)
            self._h = None

    def _on(self, stream):
        """The stream of a call, as a number. The workspace is kept until what runs there is
        done, also past the handle's end."""
        st = _stream(stream)
        if st != self._home:
            self.workspace.record_stream(stream if stream is not None else torch.cuda.current_stream())
        return st

    def _out(self, out, like, cols, stream):
        """The output and its row stride."""
        if out is None:
            return _empty((like.shape[0], cols), _bf16, like, stream), cols
        if out.shape != (like.shape[0], cols):
            raise ValueError(f"out must be [tokens, {cols}]")
        return out, _rows(out, "out")

    def conv(self, x, conv_w, cu_seqlens, state_in, state_out, conv_state, out=None, stream=None):
        """Causal conv1d + SiLU over the rows x [tokens, C] (a view of the
        projection's rows will do); sequences are cu_seqlens [S + 1], their
        slots state_in and state_out [S]. conv_state [slots, C, 3] is updated.
        Returns out [tokens, C]."""
        C, S = self._channels, state_in.shape[0]
        ldx = _rows(x, "x")
        T, cols = x.shape
        if cols != C:
            raise ValueError(f"x must be [tokens, {C}]")
        if T > _INT_MAX or S >= _INT_MAX:
            raise GdnError("gdn_prefill_conv", _native.GDN_ERR_ARG)
        out, ldo = self._out(out, x, C, stream)
        st = _native.lib().gdn_prefill_conv(
            self._h, S, T, x.data_ptr(), ldx, _dense(conv_w, "conv_w", _bf16, 4 * C),
            _dense(cu_seqlens, "cu_seqlens", _i32, S + 1), _dense(state_in, "state_in", _i32, S),
            _dense(state_out, "state_out", _i32, S), _dense(conv_state, "conv_state", _bf16, self._conv_values),
            out.data_ptr(), ldo, self._on(stream))
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
        S, Hv, T = state_in.shape[0], self.shape.num_v_heads, qkv.shape[0]
        ldqkv, ldba, zp, ldz, norm = _rows(qkv, "qkv"), _rows(ba, "ba"), None, 0, None
        if qkv.shape[1] != self._channels or ba.shape != (T, 2 * Hv):
            raise ValueError("qkv and ba must be [tokens, C] and [tokens, 2 Hv]")
        if max_len is None or max_len > T:
            max_len = T
        if T > _INT_MAX or S >= _INT_MAX or max_len < 0:
            raise GdnError("gdn_prefill_delta", _native.GDN_ERR_ARG)
        if z is not None:
            zp, ldz = z.data_ptr(), _rows(z, "z")
            if z.shape != (T, self._columns):
                raise ValueError("z must be [tokens, Hv*dv]")
            norm = _dense(weights["gated_norm_w"], "gated_norm_w", _bf16, self.shape.head_v_dim)
        out, ldo = self._out(out, qkv, self._columns, stream)
        st = _native.lib().gdn_prefill_delta(
            self._h, S, T, max_len, qkv.data_ptr(), ldqkv, zp, ldz, ba.data_ptr(), ldba,
            _dense(weights["A_log"], "A_log", torch.float32, Hv), _dense(weights["dt_bias"], "dt_bias", _bf16, Hv), norm,
            _dense(cu_seqlens, "cu_seqlens", _i32, S + 1), _dense(state_in, "state_in", _i32, S),
            _dense(state_out, "state_out", _i32, S), _dense(ssm_state, "ssm_state", self._state, self._state_values),
            out.data_ptr(), ldo, self._on(stream))
        if st != GDN_OK:
            raise GdnError("gdn_prefill_delta", st)
        return out

    def check(self, stream=None):
        """(status, detail word) of the sticky device error word; synchronises."""
        d = ctypes.c_uint32()
        st = _native.lib().gdn_prefill_check(self._h, self._on(stream), ctypes.byref(d))
        return st, d.value

    def reset(self, stream=None):
        st = _native.lib().gdn_prefill_reset(self._h, self._on(stream))
        if st != GDN_OK:
            raise GdnError("gdn_prefill_reset", st)
