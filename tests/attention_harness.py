"""Plain 64-bit implementations of the attention layer's operators and of the
projections with 4-bit weights, and seeded batches for their tests. Nothing here
is shared with the kernels.

Tolerances (set from the arithmetic, before any run; a rounding to bf16 is at most
2^-8 of the value, one to f32 2^-24, a tensor core's f32 addition cuts at 2^-23):
  append    2^-8 |y| for the rounding. Before it: cosines and sines are within 2^-22,
            a head's norm within 2^-19 of its value, a product and a sum or two more:
            2^-18 (|a| + |b|) of the pair's values.
  attend    2^-8 |o| for the rounding, 2^-8 A with A = sum p |v| for the weights', and what
            comes before: a score is a sum of d products in steps of 16, so off by at most
            (d / 16 + 16) 2^-23 of sum |q k|, times scale, which is a weight's relative error
            (twice: the sum of weights has it too); the sums over L keys (L / 16 + 64) 2^-23
            of A; the exponentials and the gate 2^-20.
            All together, errors of roundings have no common sign: the 2-norm of a call's error is below
            2^-8 of the outputs' (each rounding's mean square is a third of its largest).
  w4        2^-8 |y| for the rounding. A weight without its scale has at most 8 bits, so products
            are exact: (G / 16 + 16) 2^-23 of sum |x w| for the sums within the groups, (K / G +
            16) 2^-23 for the groups' sums in f32. Times 1.2 for the steepest activation.
"""
from __future__ import annotations

import numpy as np
import torch


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def ints(a, dtype=np.int32):
    return torch.from_numpy(np.asarray(a, dtype=dtype)).cuda()


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def strided(t, extra):
    """t's rows inside wider rows of NaN."""
    if not extra:
        return t.cuda()
    wide = torch.full((*t.shape[:1], int(np.prod(t.shape[1:])) + extra), float("nan"), dtype=t.dtype)
    wide[:, :wide.shape[1] - extra] = t.reshape(t.shape[0], -1)
    return wide.cuda()[:, :wide.shape[1] - extra].view(t.shape) if t.dim() == 2 else \
        wide.cuda()[:, :wide.shape[1] - extra].unflatten(1, t.shape[1:])


class Pages:
    """Requests of (context, new tokens) with pages anywhere in a pool. Slots that no request
    has, table entries that no request needs, and pad rows hold what nobody may read."""

    def __init__(self, heads, d, block, requests, seed, *, gate=False, extra=0, stride=0, q_std=2.0, blocks=None):
        rng = np.random.default_rng(seed)
        self.Hq, self.Hkv = heads
        self.G, self.d, self.block = heads[0] // heads[1], d, block
        self.ctx = np.array([c for c, _ in requests], np.int64)
        self.new = np.array([n for _, n in requests], np.int64)
        self.S, self.T = len(requests), int(self.new.sum()) + extra
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int64)
        need = -(-(self.ctx + self.new) // block)
        pages = int(need.sum()) + 3 if blocks is None else blocks
        order = rng.permutation(pages)
        self.table = np.full((self.S, max(1, int(need.max(initial=0))) + 1), 1 << 30, np.int64)
        at = 0
        for s in range(self.S):
            self.table[s, :need[s]] = order[at:at + need[s]]
            at += int(need[s])
        self.pages = pages
        cache = np.full((2, pages * block, self.Hkv, d), np.nan, np.float32)
        for s in range(self.S):
            sl = self.slots(s)
            cache[:, sl] = rng.standard_normal((2, len(sl), self.Hkv, d))
        cols = self.Hq * d
        q = rng.standard_normal((self.T, cols)).astype(np.float32) * q_std
        z = rng.standard_normal((self.T, cols)).astype(np.float32) * 2
        q[int(self.cu[-1]):] = np.nan
        z[int(self.cu[-1]):] = np.nan
        self.q, self.z = strided(bf16(q), stride), strided(bf16(z), stride) if gate else None
        self.k, self.v = strided(bf16(cache[0]), stride), strided(bf16(cache[1]), stride)
        self.dtable, self.dcu, self.dctx = ints(self.table), ints(self.cu), ints(self.ctx)
        self.scale = d ** -0.5

    def slots(self, s):
        p = np.arange(int(self.ctx[s] + self.new[s]))
        return self.table[s][p // self.block] * self.block + p % self.block

    def handle(self, **kw):
        from gated_deltanet_layer_gb300 import PagedAttention
        return PagedAttention(self.Hq, self.Hkv, self.d, self.block, max_tokens=max(1, self.T), max_seqs=max(1, self.S), **kw)

    def call(self, h, **kw):
        kw.setdefault("max_len", int(self.new.max(initial=0)))
        return h.attend(self.q, self.k, self.v, self.dtable, self.dcu, self.dctx, gate=self.z, **kw)

    def reference(self, padding=()):
        """(outputs, tolerance of each)."""
        q, k, v = f64(self.q).reshape(self.T, self.Hq, self.d), f64(self.k), f64(self.v)
        out, tol = np.zeros(q.shape), np.zeros(q.shape)
        for s in range(self.S):
            if s in padding or self.new[s] == 0:
                continue
            sl, n, c = self.slots(s), int(self.new[s]), int(self.ctx[s])
            rows = slice(int(self.cu[s]), int(self.cu[s + 1]))
            hidden = np.arange(len(sl))[None, :] > c + np.arange(n)[:, None]
            for h in range(self.Hq):
                kk, vv, qq = k[sl, h // self.G], v[sl, h // self.G], q[rows, h]
                with np.errstate(invalid="ignore", over="ignore"):
                    x = np.where(hidden, -np.inf, qq @ kk.T * self.scale)
                    size = np.where(hidden, 0, np.abs(qq) @ np.abs(kk).T * self.scale).max(1)
                    p = np.exp(x - x.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                # 0 x NaN: what a row does not see has no part in it
                seen = [np.nonzero(~m)[0] for m in hidden]
                if np.isfinite(vv).all():
                    o, a = p @ vv, p @ np.abs(vv)
                else:
                    with np.errstate(invalid="ignore"):
                        o = np.stack([p[i, j] @ vv[j] for i, j in enumerate(seen)])
                        a = np.stack([p[i, j] @ np.abs(vv[j]) for i, j in enumerate(seen)])
                before = 2 * (self.d / 16 + 16) * 2.0 ** -23 * size[:, None] + (len(sl) / 16 + 64) * 2.0 ** -23 + 2.0 ** -20
                out[rows, h] = o
                tol[rows, h] = 2.0 ** -8 * np.abs(o) * 1.01 + (2.0 ** -8 + before) * a
        if self.z is not None:
            g = sigmoid(f64(self.z).reshape(q.shape))
            g[int(self.cu[-1]):] = 0
            out, tol = out * g, tol * g
        return out.reshape(self.T, -1), tol.reshape(self.T, -1)


def check(got, want, tol, norm=True):
    got = f64(got)
    bad = ~np.isfinite(want)
    assert not np.isfinite(got[bad]).any(), "a value that is not finite was lost"
    ok = ~bad
    err = np.abs(got[ok] - want[ok])
    assert np.isfinite(got[ok]).all(), f"{(~np.isfinite(got[ok])).sum()} values are not finite"
    over = err > tol[ok] + 1e-30
    assert not over.any(), f"{over.sum()} of {over.size} off, worst {np.max(err - tol[ok])}, error {err.max()}"
    if norm and err.size:
        assert np.linalg.norm(err) <= 2.0 ** -8 * np.linalg.norm(want[ok]) + 1e-30


def append_reference(q, k, v, pos, slots, freq, kc, vc, qw, kw, eps, interleaved, d):
    """(q', cache of keys, of values, their tolerances), 64 bits."""
    r = 0 if freq is None else 2 * len(freq)

    def turned(x, w):
        x = x.reshape(x.shape[0], -1, d)
        if w is not None:
            x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1 + w)
        y, size = x.copy(), np.abs(x)
        if r:
            a = pos[:, None].astype(np.float64) * freq
            c, s = np.cos(a)[:, None], np.sin(a)[:, None]
            one, two = ((slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r)))
            y[..., one] = x[..., one] * c - x[..., two] * s
            y[..., two] = x[..., two] * c + x[..., one] * s
            both = np.abs(x[..., one]) + np.abs(x[..., two])
            size[..., one] = size[..., two] = both
        return y, 2.0 ** -8 * np.abs(y) * 1.01 + 2.0 ** -18 * size

    live = slots >= 0
    out = None
    if q is not None:
        y, tol = turned(q, qw)
        out = np.where(live[:, None], y.reshape(len(pos), -1), 0), np.where(live[:, None], tol.reshape(len(pos), -1), 0)
    y, tol = turned(k, kw)
    kc, vc = kc.copy(), vc.copy()
    ktol = np.zeros(kc.shape)
    kc[slots[live]], ktol[slots[live]] = y[live], tol[live]
    vc[slots[live]] = v.reshape(len(pos), -1, d)[live]
    return out, (kc, ktol), vc


E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def w4_weights(codes, scales, zeros):
    """([N, K] weights, [N, groups] scales), 64 bits."""
    c = codes.cpu().numpy()
    c = np.stack([c & 15, c >> 4], -1).reshape(c.shape[0], -1)
    g = c.shape[1] // scales.shape[1]
    if scales.dtype == torch.uint8:
        s = np.exp2(scales.cpu().numpy().astype(np.float64) - 127)
        return E2M1[c] * np.repeat(s, g, 1), s
    s = f64(scales)
    z = 8.0 if zeros is None else np.repeat(zeros.cpu().numpy().astype(np.float64), g, 1)
    return (c - z) * np.repeat(s, g, 1), s


def w4_reference(x, codes, scales, zeros, bias, act, residual):
    """(outputs, tolerance), 64 bits."""
    w, s = w4_weights(codes, scales, zeros)
    x = f64(x)
    K, groups = x.shape[1], s.shape[1]
    G = K // groups
    with np.errstate(invalid="ignore"):
        y = x @ w.T
        size = np.abs(x) @ np.abs(w).T
        before = (groups + 16) * 2.0 ** -23 * size
        before += (G / 16 + 16) * 2.0 ** -23 * size
    if bias is not None:
        y = y + f64(bias)
    if act == "silu":
        y = y * sigmoid(y)
    elif act == "gelu":
        y = 0.5 * y * (1 + np.tanh(0.7978845608028654 * (y + 0.044715 * y ** 3)))
    if residual is not None:
        y = y + f64(residual)
    return y, 2.0 ** -8 * np.abs(y) * 1.01 + 1.2 * before + 2.0 ** -20
