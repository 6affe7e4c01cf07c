"""The attention layer's operators together, as a server runs them, and what a single call's
tests leave out: long joins, many heads, caches past 32 bits, two handles at once."""
import os
import sys

import numpy as np
import pytest
import torch

import attention_harness as H

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def run(p, **kw):
    h = p.handle()
    out = p.call(h, **kw)
    assert h.check() == (0, 0)
    return out


# ------------------------------------------------------------------- a server's steps

@pytest.mark.parametrize("head_dim,rotary,block,lens", [(64, 32, 16, (37, 1, 130, 64)), (128, 128, 24, (5, 300, 0, 17)),
                                                        (256, 64, 1, (90, 33, 2))])
def test_prompts_then_decode(head_dim, rotary, block, lens):
    """Every operator's output against the 64-bit one of the inputs that it had."""
    import serve_attention_layer as E
    L = E.Layer(hidden=256, q_heads=6, kv_heads=2, head_dim=head_dim, rotary=rotary, block=block)
    R = len(lens)
    w = E.make_weights(L, 3)
    need = sum(-(-(n + 8) // block) for n in lens)
    s = E.Server(L, w, blocks=need + 5, max_blocks=-(-(max(lens) + 8) // block), requests=R, max_tokens=sum(lens) + 1)
    rng = np.random.default_rng(head_dim)
    q, kv = L.q_heads * head_dim, L.kv_heads * head_dim
    for new in (lens, [1] * R, [1] * R, [3, 2, 1, 2][:R]):
        x = H.bf16(rng.standard_normal((sum(new), L.hidden))).cuda()
        ctx = s.context.cpu().numpy().astype(np.int64)
        k0, v0 = H.f64(s.k), H.f64(s.v)
        y, d = s.step(x, H.ints(new), max(new))
        s.check()
        rows = H.f64(d["rows"])
        H.check(d["rows"], *H.w4_reference(x, *w["proj"], None, None, None), norm=False)
        m = d["map"]
        pos, slots = m.token_pos.cpu().numpy(), m.slots.cpu().numpy()
        want = np.concatenate([c + np.arange(n) for c, n in zip(ctx, new)])
        assert np.array_equal(pos, want) and len(set(slots.tolist())) == len(slots)
        out, (wk, tk), wv = H.append_reference(rows[:, :q], rows[:, q:q + kv], rows[:, q + kv:q + 2 * kv], pos, slots,
                                               H.f64(w["freq"]), k0, v0, H.f64(w["q_norm"]), H.f64(w["k_norm"]), 1e-6, False,
                                               head_dim)
        H.check(d["turned"], *out)
        H.check(s.k, wk, tk)
        assert np.array_equal(H.f64(s.v), wv)
        p = H.Pages((L.q_heads, L.kv_heads), head_dim, block, [(1, 1)], 0)
        p.S, p.T, p.ctx, p.new = R, sum(new), ctx, np.asarray(new)
        p.cu, p.table = np.concatenate([[0], np.cumsum(new)]), s.table.cpu().numpy().astype(np.int64)
        p.q, p.k, p.v, p.z = d["turned"], s.k, s.v, d["rows"][:, q + 2 * kv:]
        H.check(d["core"], *p.reference(), norm=False)
        H.check(y, *H.w4_reference(d["core"], *w["out"], None, None, x), norm=False)


def test_example_runs():
    import serve_attention_layer as E
    outs, server = E.main(steps=3)
    assert [o.shape[0] for o in outs] == [232, 4, 4, 4] and server.context.tolist() == [40, 4, 133, 67]
    assert all(torch.isfinite(o.float()).all() for o in outs)


# ------------------------------------------------------------------- shapes of work

@pytest.mark.parametrize("heads,d,n", [((8, 1), 64, 1), ((8, 1), 128, 1), ((6, 1), 256, 1), ((8, 1), 64, 4), ((10, 1), 128, 5),
                                       ((6, 1), 256, 7), ((20, 1), 128, 40)])
def test_one_long_context(heads, d, n):
    """A request that all CTAs share: more parts than are joined at once, keys split between row tiles."""
    p = H.Pages(heads, d, 32, [(40000, n)], seed=d + n)
    H.check(run(p), *p.reference())


@pytest.mark.parametrize("heads,d,requests", [((128, 1), 64, [(300, 5), (10, 1)]), ((65, 1), 128, [(200, 3), (700, 2)]),
                                              ((136, 1), 64, [(100, 3), (40, 1)]), ((300, 2), 128, [(130, 2)]),
                                              ((33, 1), 256, [(500, 9)])])
def test_many_heads_of_a_key(heads, d, requests):
    p = H.Pages(heads, d, 16, requests, seed=d, gate=True)
    H.check(run(p), *p.reference())


def test_hidden_keys_where_keys_are_split():
    """NaN in values that later tokens alone see, in a task whose keys are split between row tiles."""
    for heads, d, ctx, n in (((8, 2), 64, 1000, 6), ((10, 2), 128, 900, 5), ((12, 2), 256, 700, 4)):
        p = H.Pages(heads, d, 16, [(ctx, n), (ctx - 130, n)], seed=d)
        for s in range(2):
            at = p.slots(s)
            p.v[int(at[-1]), 0, 3] = float("nan")
            p.v[int(at[-2]), 1, d - 2] = float("-inf")
        want, tol = p.reference()
        got, ok = H.f64(run(p)), np.isfinite(want)
        assert ok.any() and not ok.all() and not np.isfinite(got[~ok]).any()
        assert np.isfinite(got[ok]).all() and (np.abs(got[ok] - want[ok]) <= tol[ok]).all()


@pytest.mark.parametrize("n", [1, 40])
def test_cache_past_32_bits(n):
    """Blocks beyond the first 4 GiB of each cache, for the append and both forms of the attention."""
    from gated_deltanet_layer_gb300 import kv_append
    d, heads, block = 256, 8, 16
    blocks = (1 << 32) // (block * heads * d * 2) + 40
    p = H.Pages((16, heads), d, block, [(70, n), (33, n)], seed=n)
    far = p.table.copy()
    shift = blocks - p.pages
    far[p.table < p.pages] += shift
    big = [torch.empty(blocks * block, heads, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for b, small in zip(big, (p.k, p.v)):
        b[shift * block:] = small
    # the new tokens' own keys and values go in through the append, unturned
    slots = np.concatenate([p.slots(s)[-n:] for s in range(p.S)])
    kv = [t[torch.from_numpy(slots).cuda()].reshape(len(slots), -1).clone() for t in (p.k, p.v)]
    for b in big:
        b[torch.from_numpy(slots + shift * block).cuda()] = float("nan")
    kv_append(None, *kv, H.ints(np.zeros(len(slots))), H.ints(slots + shift * block, np.int64), None, *big)
    h = p.handle()
    out = h.attend(p.q, *big, H.ints(far), p.dcu, p.dctx, max_len=n)
    assert h.check() == (0, 0)
    H.check(out, *p.reference())


def test_two_handles_at_once():
    """Two handles on two streams, decode steps beside a prompt's chunks, many of them under way."""
    a = H.Pages((8, 2), 128, 16, [(3000, 1), (500, 1), (40, 1)], seed=1)
    b = H.Pages((8, 2), 128, 16, [(600, 200), (0, 77)], seed=2)
    want = [p.reference() for p in (a, b)]
    hs, outs = [p.handle() for p in (a, b)], [[], []]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(8):
        for i, p in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                outs[i].append(p.call(hs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        H.check(outs[i][0], *want[i])
        assert all(torch.equal(o, outs[i][0]) for o in outs[i]) and hs[i].check() == (0, 0)


def test_refused_with_a_handle():
    """What the call refuses on a handle that is whole, before any launch."""
    from gated_deltanet_layer_gb300 import GdnError, PagedAttention
    p = H.Pages((8, 2), 128, 16, [(20, 3)], seed=1)
    h = p.handle()
    for bad in (dict(out=p.q), dict(max_len=-1)):
        with pytest.raises(GdnError):
            p.call(h, **bad)
    for name, t in (("q", p.q.float()), ("k", p.k[:-1]), ("v", p.v[:16]), ("q", p.q[:, :-8]), ("dcu", p.dcu[:-1]),
                    ("dctx", p.dctx.long()), ("dtable", p.dtable.cpu())):
        keep = getattr(p, name)
        setattr(p, name, t)
        with pytest.raises(ValueError):
            p.call(h)
        setattr(p, name, keep)
    small = PagedAttention(8, 2, 128, 16, max_tokens=2, max_seqs=1)
    with pytest.raises(GdnError):
        p.call(small)
    H.check(p.call(h), *p.reference())


@pytest.mark.parametrize("heads,d,block,requests", [
    ((40, 8), 128, 32, [(500 + 97 * i, 4) for i in range(24)]),
    ((64, 8), 64, 16, [(0, 700), (600, 33), (0, 500), (900, 16), (1000, 32), (77, 300), (520, 40), (700, 9)]),
    ((64, 8), 128, 16, [(0, 600), (640, 20), (0, 333), (800, 32), (515, 3), (33, 64), (1200, 17)]),
    ((24, 4), 256, 64, [(300 + 41 * i, 3 + 2 * i) for i in range(24)]),
    ((16, 16), 64, 16, [(512 + 64 * i, 30 + i) for i in range(12)])])
def test_many_tasks(heads, d, block, requests):
    """Many tasks a CTA, whole and in parts, some of them split between row tiles, right after one another."""
    p = H.Pages(heads, d, block, requests, seed=d + len(requests))
    h = p.handle()
    outs = [p.call(h) for _ in range(4)]
    assert h.check() == (0, 0)
    H.check(outs[0], *p.reference())
    assert all(torch.equal(o, outs[0]) for o in outs[1:])


@pytest.mark.parametrize("heads,d", [((24, 4), 256), ((40, 8), 128), ((64, 8), 64)])
def test_rows_that_are_none(heads, d):
    """What stands in the place of a row tile's rows that are none changes no bit of the others: pad rows, and
    what another call has left in shared memory."""
    outs = []
    for big in (0.0, 300.0):
        other = H.Pages(heads, d, 16, [(0, 300)], seed=9, q_std=1.0 + big)
        other.call(other.handle())
        p = H.Pages(heads, d, 16, [(700, 37), (90, 301)], seed=d, extra=40)
        p.q[int(p.cu[-1]):] = big
        outs.append(p.call(p.handle())[:int(p.cu[-1])])
    assert torch.equal(*outs)
