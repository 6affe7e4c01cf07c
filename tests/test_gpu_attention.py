"""Paged attention and the append to its cache on the GPU, against 64-bit
implementations."""
import numpy as np
import pytest
import torch

import attention_harness as H

pytestmark = pytest.mark.gpu


def run(p, **kw):
    h = p.handle()
    out = p.call(h, **kw)
    assert h.check() == (0, 0)
    return out


# ------------------------------------------------------------------- attend

SINGLE = [
    # heads, head size, block, requests of (context, new tokens)
    ((8, 2), 64, 16, [(0, 1)]),
    ((8, 2), 64, 16, [(129, 1)]),
    ((8, 1), 128, 1, [(1, 1), (63, 1), (64, 1), (127, 1), (128, 1)]),
    ((6, 2), 128, 24, [(500, 1), (0, 1), (1000, 1)]),
    ((4, 4), 64, 64, [(300, 1), (5, 1), (2000, 1), (77, 1)]),
    ((12, 2), 256, 32, [(700, 1), (31, 1)]),
    ((16, 1), 256, 256, [(3000, 1)]),
    ((5, 1), 128, 16, [(9000, 1)]),
    ((16, 16), 128, 16, [(100, 1), (1, 0), (200, 1)]),
]
FEW = [
    ((8, 2), 64, 16, [(100, 4), (0, 4), (33, 4)]),
    ((6, 2), 128, 24, [(500, 5), (0, 5), (1001, 5)]),
    ((4, 4), 256, 32, [(64, 8), (63, 8), (1, 8)]),
    ((3, 1), 64, 7, [(1, 2), (2, 3), (3, 1), (0, 0), (60, 5)]),
    ((16, 1), 128, 64, [(2500, 2), (100, 2)]),
]
CHUNK = [
    ((8, 2), 64, 16, [(0, 300)]),
    ((4, 2), 128, 16, [(0, 129), (70, 130), (0, 1), (40, 0), (513, 33)]),
    ((5, 1), 128, 24, [(1000, 257), (3, 64)]),
    ((6, 1), 256, 64, [(0, 200), (333, 100)]),
    ((2, 2), 256, 1, [(5, 140)]),
    ((24, 1), 64, 16, [(10, 17)]),
    ((20, 1), 128, 32, [(0, 40), (1, 1), (127, 1), (2000, 3)]),
    ((1, 1), 128, 128, [(0, 700), (0, 128), (0, 127), (129, 1)]),
]


@pytest.mark.parametrize("heads,d,block,requests", SINGLE + FEW + CHUNK)
@pytest.mark.parametrize("gate", [False, True])
def test_attend(heads, d, block, requests, gate):
    p = H.Pages(heads, d, block, requests, seed=len(requests) + d + block, gate=gate)
    H.check(run(p), *p.reference())


@pytest.mark.parametrize("heads,d,block,requests", [SINGLE[3], FEW[1], CHUNK[1], CHUNK[3]])
def test_strides_pad_rows_and_bound(heads, d, block, requests):
    """Rows and slots inside wider ones, pad rows past the last request, and no bound on the lengths."""
    p = H.Pages(heads, d, block, requests, seed=5, gate=True, extra=9, stride=24)
    want = p.reference()
    out = torch.full((p.T, p.q.shape[1] + 40), 7.0, dtype=torch.bfloat16, device="cuda")
    h = p.handle()
    got = p.call(h, out=out[:, 8:8 + p.q.shape[1]], max_len=None)
    H.check(got, *want)
    assert (got[int(p.cu[-1]):] == 0).all() and h.check() == (0, 0)
    assert (out[:, :8] == 7).all() and (out[:, 8 + p.q.shape[1]:] == 7).all()


@pytest.mark.parametrize("n,longest", [(257, 40), (1100, 9)])
def test_many_requests(n, longest):
    """More requests than every CTA plans for itself."""
    rng = np.random.default_rng(n)
    p = H.Pages((4, 2), 64, 8, [(int(rng.integers(0, longest)), int(rng.integers(0, 3))) for _ in range(n)], seed=n, extra=2)
    H.check(run(p), *p.reference())


def test_one_handle_many_calls():
    """Calls one right after the other, of different forms and sizes, do not see each other, and a call
    repeated gives the same bits."""
    sets = [SINGLE[3], FEW[1], ((6, 2), 128, 24, [(4000, 1)]), ((6, 2), 128, 24, [(200, 90), (0, 300)])]
    ps = [H.Pages(*c, seed=i) for i, c in enumerate(sets)]
    from gated_deltanet_layer_gb300 import PagedAttention
    h = PagedAttention(6, 2, 128, 24, max_tokens=400, max_seqs=8)
    first = [p.call(h) for p in ps]
    again = [[p.call(h) for p in ps] for _ in range(3)]
    for p, a in zip(ps, first):
        H.check(a, *p.reference())
    for turn in again:
        assert all(torch.equal(a, b) for a, b in zip(first, turn))
    assert h.check() == (0, 0)


@pytest.mark.parametrize("heads,d,block,requests", [((8, 2), 64, 16, [(40, 6), (0, 3)]), ((6, 2), 128, 24, [(30, 4)]),
                                                    ((4, 1), 256, 32, [(17, 4), (60, 8)]), ((8, 2), 128, 16, [(100, 150)]),
                                                    ((4, 2), 256, 16, [(100, 70)]), ((8, 2), 64, 16, [(0, 200)])])
def test_hidden_keys_have_no_part(heads, d, block, requests):
    """NaN and infinities in keys and values that later tokens alone see."""
    p = H.Pages(heads, d, block, requests, seed=3)
    for s in range(p.S):
        at = p.slots(s)
        n = int(p.new[s])
        p.k[int(at[-1]), 0] = float("nan")
        p.v[int(at[-1]), :, 5] = float("inf")
        p.v[int(at[-(n // 2)]), p.Hkv - 1, d - 1] = float("nan")
        p.k[int(at[-2]), p.Hkv - 1, 3] = float("-inf")
    want, tol = p.reference()
    got = H.f64(run(p))
    ok = np.isfinite(want)
    assert ok.any() and not ok.all()
    assert not np.isfinite(got[~ok]).any()
    assert np.isfinite(got[ok]).all() and (np.abs(got[ok] - want[ok]) <= tol[ok]).all()


def test_seen_keys_that_are_not_finite():
    """A context's NaN reaches its request's rows alone; scores of minus infinity have no weight."""
    p = H.Pages((4, 2), 128, 16, [(200, 3), (100, 3), (50, 3)], seed=8)
    at = p.slots(0)
    p.v[int(at[7]), 0, 11] = float("nan")
    at = p.slots(1)
    p.q[3:6] = p.q[3:6].abs()
    p.k[int(at[20]), 1] = float("-inf")
    p.v[int(at[20]), 1] = 1e4
    want, tol = p.reference()
    got = H.f64(run(p))
    ok = np.isfinite(want)
    assert not np.isfinite(got[~ok]).any() and (np.abs(got[ok] - want[ok]) <= tol[ok]).all()


def test_large_scores():
    """Scores of some thousands: one key takes all the weight; equal keys share it."""
    p = H.Pages((4, 1), 64, 16, [(300, 2), (600, 70)], seed=4, q_std=400.0)
    H.check(run(p), *p.reference(), norm=False)
    p = H.Pages((4, 1), 64, 16, [(300, 2), (600, 70)], seed=4, q_std=0.0)
    H.check(run(p), *p.reference(), norm=False)


def test_shared_blocks():
    """Requests whose contexts begin in the same blocks."""
    p = H.Pages((6, 2), 128, 16, [(64, 1), (70, 1), (64, 1)], seed=6)
    p.table[1, :4] = p.table[0, :4]
    p.table[2, :4] = p.table[0, :4]
    p.dtable = H.ints(p.table)
    H.check(run(p), *p.reference())


def word(what, who):
    return (5 << 24) | (what << 16) | who


@pytest.mark.parametrize("n", [1, 3, 60])
def test_index_errors(n):
    """What is wrong with a request is recorded, the request is padding, and the others go on."""
    requests = [(100, n), (64, n), (200, n)]
    p = H.Pages((8, 2), 128, 16, requests, seed=7)
    want = p.reference(padding=(1,))
    h = p.handle()
    for ctx in (-1, p.table.shape[1] * 16 - n + 1, 2**31 - 1):
        dctx = p.dctx.clone()
        dctx[1] = ctx
        out = h.attend(p.q, p.k, p.v, p.dtable, p.dcu, dctx, max_len=n)
        H.check(out, *want)
        assert h.check() == (5, word(5, 1))
        h.reset()
    cu = p.dcu.clone()
    cu[2] = n - 1  # goes back: the second request has no rows, and the third would have one of the first's
    out = h.attend(p.q, p.k, p.v, p.dtable, cu, p.dctx, max_len=3 * n)
    assert h.check() == (5, word(2, 1))
    H.check(out, *p.reference(padding=(1, 2)))
    h.reset()
    cu = p.dcu.clone()
    cu[0] = 1
    out = h.attend(p.q, p.k, p.v, p.dtable, cu, p.dctx, max_len=3 * n)
    assert h.check() == (5, word(2, 0)) and (out[:n] == 0).all()
    w = p.reference(padding=(0,))
    H.check(out, *w)
    h.reset()


def test_longer_than_the_bound():
    p = H.Pages((8, 2), 128, 16, [(100, 1), (64, 2), (200, 1)], seed=7)
    h = p.handle()
    out = p.call(h, max_len=1)
    assert h.check() == (5, word(3, 1))
    H.check(out, *p.reference(padding=(1,)))


@pytest.mark.parametrize("n", [1, 60])
@pytest.mark.parametrize("bad", [-1, 1 << 30, -2**31])
def test_bad_block(n, bad):
    """A block outside the cache is read as zeros and recorded."""
    p = H.Pages((8, 2), 128, 16, [(100, n), (64, n)], seed=9)
    p.dtable[1, 2] = bad
    h = p.handle()
    out = p.call(h)
    assert h.check() == (5, word(1, 1))
    good, p.table[1, 2] = p.table[1, 2].copy(), p.pages  # one more block, of zeros
    for name in ("k", "v"):
        t = getattr(p, name)
        setattr(p, name, torch.cat([t, torch.zeros(16, *t.shape[1:], dtype=t.dtype, device="cuda")]))
    H.check(out, *p.reference())


def test_nothing_to_do():
    p = H.Pages((8, 2), 64, 16, [(5, 0), (0, 0)], seed=1, extra=3)
    assert (run(p) == 0).all()
    from gated_deltanet_layer_gb300 import PagedAttention
    h = PagedAttention(8, 2, 64, 16, max_tokens=4, max_seqs=2)
    e = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")
    q = torch.empty(0, 512, dtype=torch.bfloat16, device="cuda")
    assert h.attend(q, p.k, p.v, e(0, 3), torch.zeros(1, dtype=torch.int32, device="cuda"), e(0)).shape == (0, 512)


@pytest.mark.parametrize("heads,d,block,requests", [SINGLE[3], CHUNK[1]])
def test_graph_and_stream(heads, d, block, requests):
    """Captured once, replayed with other contents in the same memory; and on another stream."""
    p = H.Pages(heads, d, block, requests, seed=21)
    other = H.Pages(heads, d, block, requests, seed=22)
    h, out = p.handle(), torch.empty_like(p.q)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        p.call(h, out=out)
    side.synchronize()
    H.check(out, *p.reference())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.call(h, out=out)
    for a, b in ((p.q, other.q), (p.k, other.k), (p.v, other.v), (p.dtable, other.dtable)):
        a.copy_(b)
    for _ in range(2):
        out.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        H.check(out, *other.reference())
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    H.check(p.call(h, stream=st), *other.reference())
    assert h.check(st) == (0, 0)


# ------------------------------------------------------------------- append

def append_case(heads, d, rotary, T, block, seed, *, norms, interleaved, far=1000, pads=(), stride=0, in_place=False, q=True,
                turn=1.0):
    from gated_deltanet_layer_gb300 import kv_append
    rng = np.random.default_rng(seed)
    hq, hkv = heads
    rows = H.bf16(rng.standard_normal((T, (hq + 2 * hkv) * d + stride)) * 2).cuda()
    a, b = hq * d, hkv * d
    qs, ks, vs = rows[:, :a], rows[:, a:a + b], rows[:, a + b:a + 2 * b]
    pos = rng.integers(0, far, T)
    n = T * 2 + 5
    slots = rng.permutation(n)[:T]
    slots[list(pads)] = -1 - np.arange(len(pads))
    freq = torch.from_numpy((1e6 ** (-np.arange(0, rotary, 2) / rotary)).astype(np.float32)).cuda() * turn if rotary else None
    qw, kw = ((H.bf16(rng.standard_normal(d) * 0.2).cuda() for _ in range(2)) if norms else (None, None))
    kc, vc = (H.strided(H.bf16(rng.standard_normal((n, hkv, d))), stride) for _ in range(2))
    want, (wk, tk), wv = H.append_reference(H.f64(qs) if q else None, H.f64(ks), H.f64(vs), pos, slots,
                                            None if freq is None else H.f64(freq), H.f64(kc), H.f64(vc),
                                            H.f64(qw) if norms else None, H.f64(kw) if norms else None, 1e-6, interleaved, d)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = kv_append(qs if q else None, ks, vs, H.ints(pos), H.ints(slots, np.int64), freq, kc, vc, q_norm_w=qw, k_norm_w=kw,
                    interleaved=interleaved, q_out=qs if in_place else None, error=err)
    if q:
        H.check(got, *want)
    H.check(kc, wk, tk)
    assert np.array_equal(H.f64(vc), wv) and err.item() == 0


@pytest.mark.parametrize("heads,d,rotary,T", [((8, 1), 128, 128, 1), ((8, 2), 64, 64, 5), ((6, 2), 256, 64, 37),
                                              ((3, 3), 128, 48, 130), ((40, 8), 128, 128, 700), ((2, 1), 256, 256, 3),
                                              ((4, 2), 64, 0, 9), ((5, 5), 64, 16, 2000)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norms", [False, True])
def test_append(heads, d, rotary, T, interleaved, norms):
    append_case(heads, d, rotary, T, 16, T + d, norms=norms, interleaved=interleaved, pads=(0,) if T > 4 else (),
                stride=8 * (T % 3))


@pytest.mark.parametrize("far", [1 << 20, 1 << 24, 2**31 - 1])
def test_append_far_positions(far):
    append_case((4, 2), 128, 128, 64, 16, 3, norms=False, interleaved=False, far=far)


def test_append_in_place_and_keys_alone():
    append_case((4, 2), 128, 64, 33, 16, 4, norms=True, interleaved=False, in_place=True, pads=(3, 30))
    append_case((4, 2), 256, 64, 33, 16, 5, norms=True, interleaved=True, q=False)


def test_append_bad_slot():
    from gated_deltanet_layer_gb300 import kv_append
    q = torch.ones(3, 128, dtype=torch.bfloat16, device="cuda")
    kc, vc = (torch.zeros(8, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = kv_append(q, q[:, :64], q[:, 64:], H.ints([0, 1, 2]), H.ints([7, 8, 2**62], np.int64), None, kc, vc, error=err)
    assert err.item() in (word(1, 1), word(1, 2))
    assert (out[0] == 1).all() and (out[1:] == 0).all()
    assert (kc[7] == 1).all() and (kc[:7] == 0).all() and (vc[7] == 1).all() and (vc[:7] == 0).all()
    err.fill_(77)  # a word that is set stays
    kv_append(None, q[:, :64], q[:, 64:], H.ints([0, 1, 2]), H.ints([7, 8, 9], np.int64), None, kc, vc, error=err)
    assert err.item() == 77


@pytest.mark.parametrize("turn,far", [(-1.0, 1 << 31), (-2.0 ** -30, 1 << 31), (2.0 ** -30, 1 << 31), (2.0 ** 38, 1000), (-2.0 ** 20, 1000)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_frequencies(turn, far, interleaved):
    append_case((4, 2), 64, 64, 50, 16, 77, norms=True, interleaved=interleaved, far=far, turn=turn)


def test_append_on_a_stream():
    from gated_deltanet_layer_gb300 import kv_append
    rng = np.random.default_rng(4)
    q, k, v = (H.bf16(rng.standard_normal((9, c))).cuda() for c in (512, 128, 128))
    pos, slots = H.ints(np.arange(9)), H.ints(np.arange(9)[::-1].copy(), np.int64)
    freq = torch.full((32,), 0.5, device="cuda")
    outs = []
    for st in (None, torch.cuda.Stream()):
        kc, vc = torch.zeros(10, 1, 128, dtype=torch.bfloat16, device="cuda"), torch.ones(10, 1, 128, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        out = kv_append(q, k, v, pos, slots, freq, kc, vc, interleaved=True, stream=st)
        torch.cuda.synchronize()
        outs.append((out, kc, vc))
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and outs[0][0].shape == q.shape
    assert kv_append(None, k, v, pos, slots, freq, *outs[0][1:]) is None
