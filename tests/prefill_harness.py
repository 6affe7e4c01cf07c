"""Plain 64-bit implementations of the prompt-side operators and seeded ragged
batches for their tests. Nothing here is shared with the kernels.

Tolerances (set from the arithmetic, before any run):
  bf16 outputs  one rounding to bf16 is at most 2^-9 of the value; twice that
                is allowed, beside an absolute part for what comes before it.
  conv          that absolute part: four f32 products and an f32 SiLU, 2^-20
                of sum |w x|.
  linear        sums of K products in f32, in groups of 16 or less with one
                rounding (or cut) each: (K / 16 + 16) 2^-23 of sum |x w|, times
                1.2 for the steepest activation.
  delta core    intermediate values may be kept in 11 bits where only the
                output sees them: 2^-8 of the row's root mean square, per value
                head (the gated form: of |w silu(z)|, its scale).
  delta state   f32 sums over the sequence: 2e-5 in the 2-norm of a value
                head's state, relative to the larger of the final and the
                starting state and the values' norm; a bf16 state one
                rounding more, 2^-8 of the value.
"""
from __future__ import annotations

import numpy as np
import torch

from gated_deltanet_layer_gb300 import workloads as WL

SMALL = WL.LayerShape("small", hidden=256, num_k_heads=2, num_v_heads=4, head_k_dim=64, head_v_dim=64, num_slots=24)
WIDE = WL.LayerShape("wide", hidden=256, num_k_heads=2, num_v_heads=6, head_k_dim=128, head_v_dim=128, num_slots=24)


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def silu(x):
    with np.errstate(over="ignore"):
        return x / (1.0 + np.exp(-x))


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


class Batch:
    """A ragged batch of conv / delta inputs on the device. pad: sequences that
    are padding; extra: pad rows past the last sequence; fresh: sequences that
    start from zero; share: all the others start from the first one's slot;
    same: state_out is state_in. Rows nobody may read hold NaN."""

    def __init__(self, shape, lens, seed, *, pad=(), extra=0, fresh=(), share=False, same=False, stride=0, a_log=None,
                 keys=None, beta=None, values=1.0):
        rng = np.random.default_rng(seed)
        self.shape, self.lens = shape, list(lens)
        S, T = len(lens), int(sum(lens)) + extra
        self.T, self.S = T, S
        Hk, Hv, d, C = shape.num_k_heads, shape.num_v_heads, shape.head_k_dim, shape.conv_channels
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        slots = rng.permutation(np.arange(1, shape.num_slots))
        assert 2 * S < shape.num_slots
        self.first = slots[:S].astype(np.int32)
        self.last = slots[S:2 * S].astype(np.int32)
        if same:
            self.last = self.first.copy()
        if share:
            self.first[:] = self.first[0]
        for s in fresh:
            self.first[s] = 0 if s % 2 else -1
        for s in pad:
            self.last[s] = 0 if s % 2 else -3
        x = rng.standard_normal((T, C)).astype(np.float32)
        x[:, 2 * Hk * d:] *= values
        if keys is not None:
            x[:, Hk * d:2 * Hk * d] = keys(rng, T, Hk * d)
        self.x = x
        self.z = rng.standard_normal((T, Hv * d)).astype(np.float32)
        ba = rng.standard_normal((T, 2 * Hv)).astype(np.float32) * 1.5
        if beta is not None:
            ba[:, :Hv] = beta
        self.ba = ba
        for r in [(self.cu[s], self.cu[s + 1]) for s in pad] + [(self.cu[S], T)]:
            for t in (self.x, self.z, self.ba):
                t[r[0]:r[1]] = np.nan
        self.conv_w = rng.standard_normal((C, 4)) * 0.4
        self.A_log = (rng.uniform(-2, 0, Hv) if a_log is None else np.full(Hv, a_log)).astype(np.float32)
        self.dt_bias, self.gnorm = rng.standard_normal(Hv) * 0.5, 1 + 0.1 * rng.standard_normal(d)
        conv = rng.standard_normal((shape.num_slots, C, 3))
        ssm = rng.standard_normal((shape.num_slots, Hv, d, d)) * 0.1
        conv[0] = ssm[0] = np.nan
        used = set(self.first.tolist()) | set(self.last.tolist())
        for i in range(shape.num_slots):
            if i not in used:
                conv[i] = ssm[i] = np.nan  # a slot nobody reads
        def rows(a):
            t = bf16(a).cuda()
            if stride:
                wide = torch.full((t.shape[0], t.shape[1] + stride), float("nan"), dtype=t.dtype, device="cuda")
                wide[:, :t.shape[1]] = t
                return wide[:, :t.shape[1]]
            return t
        self.dx, self.dz, self.dba = rows(self.x), rows(self.z), rows(self.ba)
        self.dw = bf16(self.conv_w).cuda()
        self.dconv = bf16(conv).cuda()
        self.dssm = (bf16(ssm) if shape.ssm_dtype == "bf16" else torch.from_numpy(ssm.astype(np.float32))).cuda()
        self.weights = {"A_log": torch.from_numpy(self.A_log).cuda(), "dt_bias": bf16(self.dt_bias).cuda(),
                        "gated_norm_w": bf16(self.gnorm).cuda()}
        self.dcu, self.dfirst, self.dlast = (torch.from_numpy(a).cuda() for a in (self.cu, self.first, self.last))
        self.conv0, self.ssm0 = f64(self.dconv), f64(self.dssm)

    def live(self):
        return [s for s in range(self.S) if self.last[s] > 0]

    def rows_of(self, s):
        return slice(int(self.cu[s]), int(self.cu[s + 1]))


def conv_reference(b):
    """(out, scale of the sums, new conv pool)."""
    x, w = f64(b.dx), f64(b.dw)
    out, scale, pool = np.zeros(x.shape), np.zeros(x.shape), b.conv0.copy()
    for s in b.live():
        old = b.conv0[b.first[s]].T if b.first[s] > 0 else np.zeros((3, x.shape[1]))
        line = np.concatenate([old, x[b.rows_of(s)]])
        for i in range(b.lens[s]):
            taps = line[i:i + 4].T * w
            out[b.cu[s] + i] = silu(taps.sum(1))
            scale[b.cu[s] + i] = np.abs(taps).sum(1)
        pool[b.last[s]] = line[-3:].T
    return out, scale, pool


def delta_reference(b, gated):
    """(core, absolute scale of core, new state pool, norm of each state's sums)."""
    sh = b.shape
    Hk, Hv, d, G = sh.num_k_heads, sh.num_v_heads, sh.head_k_dim, sh.group
    x, z, ba = f64(b.dx), f64(b.dz), f64(b.dba)
    rate, shift, gw = np.exp(f64(b.weights["A_log"])), f64(b.weights["dt_bias"]), f64(b.weights["gated_norm_w"])
    core, scale, pool, norm = np.zeros((b.T, Hv, d)), np.zeros((b.T, Hv, d)), b.ssm0.copy(), {}
    for s in b.live():
        S = b.ssm0[b.first[s]].copy() if b.first[s] > 0 else np.zeros((Hv, d, d))
        most = np.sqrt((S * S).sum((1, 2)))
        for t in range(int(b.cu[s]), int(b.cu[s + 1])):
            q, k, v = (x[t, i:j].reshape(-1, d) for i, j in ((0, Hk * d), (Hk * d, 2 * Hk * d), (2 * Hk * d, None)))
            q = np.repeat(q / np.sqrt((q * q).sum(1, keepdims=True) + sh.l2_eps) * sh.scale_q, G, 0)
            k = np.repeat(k / np.sqrt((k * k).sum(1, keepdims=True) + sh.l2_eps), G, 0)
            beta = 1 / (1 + np.exp(-ba[t, :Hv]))
            decay = np.exp(-rate * np.logaddexp(0, ba[t, Hv:] + shift))
            S *= decay[:, None, None]
            u = beta[:, None] * (v - np.einsum("hvk,hk->hv", S, k))
            S += u[:, :, None] * k[:, None, :]
            o = np.einsum("hvk,hk->hv", S, q)
            rms = np.sqrt((o * o).mean(1, keepdims=True))
            if gated:
                gate = gw * silu(z[t].reshape(Hv, d))
                core[t] = o / np.sqrt(rms * rms + sh.gated_norm_eps) * gate
                scale[t] = np.abs(gate) * (rms / np.sqrt(rms * rms + sh.gated_norm_eps))
            else:
                core[t], scale[t] = o, rms
            most = np.maximum(most, np.maximum(np.sqrt((S * S).sum((1, 2))), np.sqrt((v * v).sum(1))))
        pool[b.last[s]] = S
        norm[s] = most
    return core.reshape(b.T, Hv * d), scale.reshape(b.T, Hv * d), pool, norm


def check_delta(b, core, gated, *, core_tol=2.0 ** -8, state_tol=2e-5):
    want, scale, pool, norm = delta_reference(b, gated)
    got, ssm = f64(core), f64(b.dssm)
    assert np.isfinite(got).all()
    off = np.abs(got - want) - (2.0 ** -8 * np.abs(want) + core_tol * scale + 1e-30)
    assert off.max(initial=-1) <= 0, f"core off by {off.max()} more than allowed"
    for s in b.live():
        d = np.abs(ssm[b.last[s]] - pool[b.last[s]])
        if b.shape.ssm_dtype == "bf16":
            d = np.maximum(0, d - 2.0 ** -8 * np.abs(pool[b.last[s]]))
        err = np.sqrt((d * d).sum((1, 2)))
        assert (err <= state_tol * norm[s] + 1e-30).all(), f"state of sequence {s}: {(err / norm[s]).max():.3g}"
    kept = [i for i in range(b.shape.num_slots) if i not in {int(b.last[s]) for s in b.live()}]
    np.testing.assert_array_equal(ssm[kept], b.ssm0[kept])


def slot_map_reference(new, ctx, B, table, free, count, tokens):
    """(cu, token_seq, token_pos, slots, blocks left, table, anything wrong), request by request."""
    table = table.copy()
    R, wide = table.shape
    cu = np.zeros(R + 1, np.int64)
    seq, pos, slots = (np.full(tokens, -1, np.int64) for _ in range(3))
    left, short, wrong = min(max(int(count), 0), len(free)), False, False
    for r in range(R):
        n, c = max(int(new[r]), 0), max(int(ctx[r]), 0)
        have, want = -(-c // B), -(-(c + n) // B)
        ok = new[r] >= 0 and ctx[r] >= 0 and want <= wide and c + n < 2 ** 31
        if ok and want > have:
            if short or want - have > left:
                short, ok = True, False
            else:
                for i in range(have, want):
                    left -= 1
                    table[r, i] = free[left]
        wrong = wrong or not ok
        cu[r + 1] = cu[r] + n
        for i in range(min(n, max(0, tokens - int(cu[r])))):
            t = cu[r] + i
            seq[t], pos[t] = r, min(c + i, 2 ** 31 - 1)
            slots[t] = int(table[r, (c + i) // B]) * B + (c + i) % B if ok else -1
    wrong = wrong or cu[R] > tokens
    return np.minimum(cu, tokens), seq, pos, slots, left, table, wrong
