"""Paged attention at the ends of its ranges, on the GPU."""
import numpy as np
import pytest
import torch

import attention_harness as H

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_len", [0, 1, 40])
@pytest.mark.parametrize("requests", [0, 3, 200])
def test_pad_rows_alone(requests, max_len):
    """No request has a new token, or there is none: nothing to share out, and every row is zero."""
    from gated_deltanet_layer_gb300 import PagedAttention
    h = PagedAttention(8, 2, 128, 16, max_tokens=40, max_seqs=200)
    kv = torch.full((160, 2, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = torch.full((40, 1024), float("nan"), dtype=torch.bfloat16, device="cuda")
    ints = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    for _ in range(3):
        out = h.attend(q, kv, kv.clone(), ints(requests, 4), ints(requests + 1), ints(requests), max_len=max_len)
        assert (out == 0).all()
    assert h.check() == (0, 0)


@pytest.mark.parametrize("heads,d,block", [((8, 2), 64, 16), ((8, 2), 128, 32), ((12, 3), 256, 16)])
def test_pieces_and_boxes_in_turn(heads, d, block):
    """Many short requests a CTA, whose last keys come in pieces and the others in boxes: each place of the ring has both in
    turn. Every call has the first one's bits."""
    rng = np.random.default_rng(d)
    p = H.Pages(heads, d, block, [(int(c), 1) for c in rng.integers(0, 700, 400)], seed=d)
    h = p.handle()
    outs = [p.call(h) for _ in range(10)]
    assert h.check() == (0, 0)
    H.check(outs[0], *p.reference())
    assert all(torch.equal(o, outs[0]) for o in outs[1:])


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", [16, 33, 60, 100])
@pytest.mark.parametrize("heads,d,requests", [((8, 2), 64, [(130, 1), (700, 1)]), ((8, 2), 64, [(100, 60), (0, 130)]),
                                              ((8, 2), 128, [(100, 60), (0, 130)]), ((10, 2), 128, [(900, 5), (33, 5)]),
                                              ((6, 1), 256, [(300, 1), (600, 2)]), ((6, 1), 256, [(70, 90), (300, 20)])])
def test_scores_of_any_size(heads, d, requests, size, sign):
    """Scores of 2^size times a whole number from 1 to 100, or of minus that, times the scale: the largest one's keys have all the
    weight, in equal parts. They are exact in f32 but for the scale's rounding, which equal ones have alike, and what is
    between two of them leaves the smaller no weight; so a row's error is the roundings of weights (1, or what the sum
    divides out again) and of the output, and the sums'."""
    p = H.Pages(heads, d, 16, requests, seed=d + size)
    rng = np.random.default_rng(size)
    q = np.zeros((p.T, p.Hq, d))
    q[:, :, 1] = 2.0 ** (size // 2)
    k = H.f64(p.k)
    k[:, :, 1] = sign * rng.integers(1, 101, k.shape[:2]) * 2.0 ** (size - size // 2)
    p.q, p.k = H.bf16(q.reshape(p.T, -1)).cuda(), H.bf16(k).cuda()
    k, v = H.f64(p.k), H.f64(p.v)
    h = p.handle()
    got = H.f64(p.call(h)).reshape(p.T, p.Hq, d)
    assert h.check() == (0, 0)
    for s in range(p.S):
        at = p.slots(s)
        for t in range(int(p.new[s])):
            seen = at[:int(p.ctx[s]) + t + 1]
            for head in range(p.Hkv):
                best = k[seen, head, 1] == k[seen, head, 1].max()
                o, a = v[seen[best], head].mean(0), np.abs(v[seen[best], head]).mean(0)
                tol = 2.0 ** -8 * np.abs(o) * 1.01 + (2.0 ** -8 + (len(at) / 16 + 64) * 2.0 ** -23 + 2.0 ** -20) * a
                rows = got[int(p.cu[s]) + t, head * p.G:(head + 1) * p.G]
                assert (np.abs(rows - o) <= tol).all()


@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-30])
@pytest.mark.parametrize("size", [126, 70, 62, 20, -20, -38, -45, -60, -126, -133])
@pytest.mark.parametrize("heads,d,rotary", [((4, 2), 64, 64), ((6, 1), 128, 48), ((3, 3), 256, 64)])
def test_norms_of_any_size(heads, d, rotary, size, eps):
    """Heads of values about 2^size, beside ordinary ones, through the norms, all of which are defined (no head is zero)."""
    from gated_deltanet_layer_gb300 import kv_append
    rng = np.random.default_rng(d)
    (hq, hkv), T = heads, 21
    x = rng.standard_normal((T, hq + 2 * hkv, d)).clip(-2.9, 2.9)
    x[rng.random(x.shape[:2]) < 0.5] *= 2.0 ** size
    x[:, :, 0] = np.where(x[:, :, 0] == 0, 1, x[:, :, 0])
    rows = H.bf16(x.reshape(T, -1))
    zero = (rows.view(T, -1, d) == 0).all(-1).any()
    assert not zero
    rows = rows.cuda()
    a, b = hq * d, hkv * d
    qs, ks, vs = rows[:, :a], rows[:, a:a + b], rows[:, a + b:]
    pos, slots = rng.integers(0, 1000, T), rng.permutation(T + 3)[:T]
    freq = torch.from_numpy((1e4 ** (-np.arange(0, rotary, 2) / rotary)).astype(np.float32)).cuda()
    qw, kw = (H.bf16(rng.standard_normal(d) * 0.2).cuda() for _ in range(2))
    for q_norm, k_norm in ((qw, kw), (None, kw), (qw, None)):
        kc, vc = (torch.zeros(T + 3, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        # each side by itself: the other is taken as it is
        want = [H.append_reference(H.f64(qs), H.f64(ks), H.f64(vs), pos, slots, H.f64(freq), H.f64(kc), H.f64(vc), n, n, float(np.float32(eps)), False, d)
                for n in (None if q_norm is None else H.f64(qw), None if k_norm is None else H.f64(kw))]
        got = kv_append(qs, ks, vs, H.ints(pos), H.ints(slots, np.int64), freq, kc, vc, q_norm_w=q_norm, k_norm_w=k_norm,
                        norm_eps=eps)
        for y, (w, tol) in ((got, want[0][0]), (kc, want[1][1])):
            # turned as they are, the largest may pass bf16's range; the smallest are rounded to whole subnormals
            ok = np.abs(w) < 3.3e38
            assert (np.abs(H.f64(y)[ok] - w[ok]) <= tol[ok] + 2.0 ** -134).all()
        assert torch.equal(vc[H.ints(slots).long()].reshape(T, -1), vs)


@pytest.mark.parametrize("heads,d,requests", [((8, 2), 128, [(3000, 1), (9000, 1)]), ((8, 2), 64, [(2000, 60)])])
def test_made_on_a_busy_stream(heads, d, requests):
    """A handle made on a stream that is busy, in memory that held something else, and called on another stream at once."""
    p = H.Pages(heads, d, 16, requests, seed=3)
    want = p.reference()
    first = p.handle()
    size = first.workspace.numel()
    del first
    busy, other = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(busy):
        torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(200_000_000)
        h = p.handle()
    out = p.call(h, stream=other)
    other.synchronize()
    assert h.check(other) == (0, 0)
    H.check(out, *want)


@pytest.mark.parametrize("given", [False, True])
def test_made_within_a_capture(given):
    """Making a handle while its stream captures waits for nothing; its clearing is a part of the graph."""
    p = H.Pages((8, 2), 128, 16, [(3000, 1), (200, 1)], seed=4)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    p.call(p.handle())  # what a first call loads is there
    torch.cuda.synchronize()
    out = torch.empty_like(p.q)
    with torch.cuda.graph(g, stream=side):
        if given:
            with torch.cuda.stream(torch.cuda.Stream()):  # another one is current, and does not capture
                h = p.handle(stream=side)
        else:
            h = p.handle()
        p.call(h, out=out)
    for _ in range(3):
        out.fill_(5)
        g.replay()
        torch.cuda.synchronize()
        H.check(out, *p.reference())


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_captured(interleaved):
    """An append in a graph, replayed with other rows, positions and slots in the same memory, pad rows among them."""
    from gated_deltanet_layer_gb300 import kv_append
    rng, (hq, hkv, d), T = np.random.default_rng(5), (6, 2, 128), 19
    freq = torch.from_numpy((1e4 ** (-np.arange(0, d, 2) / d)).astype(np.float32)).cuda()
    qw, kw = (H.bf16(rng.standard_normal(d) * 0.2).cuda() for _ in range(2))
    rows = torch.empty(T, (hq + 2 * hkv) * d, dtype=torch.bfloat16, device="cuda")
    pos, slots = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(T, dtype=torch.int64, device="cuda")
    kc, vc = (torch.zeros(40, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    err, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty(T, hq * d, dtype=torch.bfloat16, device="cuda")

    def call():
        q, k, v = rows.split([hq * d, hkv * d, hkv * d], 1)
        return kv_append(q, k, v, pos, slots, freq, kc, vc, q_norm_w=qw, k_norm_w=kw, interleaved=interleaved, q_out=out, error=err)

    def fill():
        rows.copy_(H.bf16(rng.standard_normal(tuple(rows.shape))))
        pos.copy_(torch.from_numpy(rng.integers(0, 2**31 - 1, T).astype(np.int32)))
        at = rng.permutation(40)[:T]
        at[rng.integers(0, T, 3)] = -1
        slots.copy_(torch.from_numpy(at))
    fill()
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(4):
        fill()
        q, k, v = (H.f64(t) for t in rows.split([hq * d, hkv * d, hkv * d], 1))
        want, (wk, tk), wv = H.append_reference(q, k, v, pos.cpu().numpy(), slots.cpu().numpy(), H.f64(freq), H.f64(kc), H.f64(vc),
                                                H.f64(qw), H.f64(kw), 1e-6, interleaved, d)
        g.replay()
        torch.cuda.synchronize()
        H.check(out, *want)
        H.check(kc, wk, tk)
        assert np.array_equal(H.f64(vc), wv) and err.item() == 0
