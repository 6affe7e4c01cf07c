"""The prompt-side operators on the GPU against plain 64-bit implementations
(tests/prefill_harness.py, which derives the tolerances)."""
import numpy as np
import pytest
import torch

from gated_deltanet_layer_gb300 import (GdnDecode, GdnError, GdnPrefill, _native, linear, linear_check, slot_map,
                                        workloads as WL)
import prefill_harness as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def handle(b, **kw):
    return GdnPrefill(b.shape, max_tokens=max(b.T, 1), max_seqs=max(b.S, 1), **kw)


# ------------------------------------------------------------------ conv

LENS = [[1], [3], [2, 0, 1, 5], [64], [65, 63], [0, 1, 130, 64, 2, 0], [191, 7]]


@pytest.mark.parametrize("shape", [P.SMALL, P.WIDE], ids=lambda s: s.name)
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("how", ["apart", "same", "share", "strided"])
def test_conv(shape, lens, how):
    b = P.Batch(shape, lens, 5, same=how == "same", share=how == "share", stride=24 if how == "strided" else 0,
                fresh=[1] if len(lens) > 1 else [], pad=[2] if len(lens) > 2 else [], extra=3 if how == "strided" else 0)
    want, scale, pool = P.conv_reference(b)
    h = handle(b)
    got = P.f64(h.conv(b.dx, b.dw, b.dcu, b.dfirst, b.dlast, b.dconv))
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * scale).all()
    np.testing.assert_array_equal(P.f64(b.dconv), pool)
    assert h.check()[0] == 0


# ------------------------------------------------------------------ delta

@pytest.mark.parametrize("shape", [P.SMALL, P.WIDE], ids=lambda s: s.name)
@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("lens", LENS + [[1, 1, 0, 1, 1]], ids=str)
def test_delta(shape, state, gated, lens):
    b = P.Batch(shape.with_(ssm_dtype=state), lens, 7, fresh=[1] if len(lens) > 1 else [],
                pad=[2] if len(lens) > 2 else [])
    h = handle(b)
    core = h.delta(b.dx, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, b.dssm, z=b.dz if gated else None, max_len=max(lens))
    P.check_delta(b, core, gated)
    assert h.check()[0] == 0


@pytest.mark.parametrize("how", ["same", "share", "strided"])
@pytest.mark.parametrize("shape", [P.SMALL, P.WIDE], ids=lambda s: s.name)
def test_delta_slots_and_strides(shape, how):
    b = P.Batch(shape, [70, 1, 9, 128, 0], 8, same=how == "same", share=how == "share", pad=[2],
                stride=16 if how == "strided" else 0, extra=70 if how == "strided" else 0)
    h = handle(b)
    core = h.delta(b.dx, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, b.dssm, z=b.dz)
    P.check_delta(b, core, True)
    assert h.check()[0] == 0


def _one_key(rng, T, n):
    return np.tile(rng.standard_normal((1, n)), (T, 1))


def _alternating(rng, T, n):
    return _one_key(rng, T, n) * np.where(np.arange(T) % 2, -1.0, 1.0)[:, None]


def _zeros(rng, T, n):
    return np.where(rng.random((T, 1)) < 0.5, 0.0, rng.standard_normal((T, n)))


def _wide_range(rng, T, n):
    return rng.standard_normal((T, n)) * 10.0 ** rng.uniform(-6, 6, (T, 1))


def _one_large(rng, T, n):
    k = rng.standard_normal((T, n)) * 1e-4
    k[:, ::64] = 1.0
    return k


@pytest.mark.parametrize("keys", [_one_key, _alternating, _zeros, _wide_range, _one_large])
@pytest.mark.parametrize("a_log", [-8.0, 0.0, 4.0], ids=["keeps", "decays", "forgets"])
@pytest.mark.parametrize("beta", [-30.0, 30.0, None], ids=["beta0", "beta1", "beta"])
def test_delta_keys_and_gates(keys, a_log, beta):
    """Keys that repeat, vanish or span many magnitudes; gates at their ends."""
    b = P.Batch(P.WIDE, [150, 64, 5], 9, keys=keys, a_log=a_log, beta=beta)
    core = handle(b).delta(b.dx, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, b.dssm)
    P.check_delta(b, core, False)


@pytest.mark.parametrize("values", [1e-12, 1e-3, 1e4, 1e12])
def test_delta_value_magnitudes(values):
    b = P.Batch(P.SMALL, [130, 3], 10, values=values, fresh=[0, 1])
    core = handle(b).delta(b.dx, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, b.dssm)
    P.check_delta(b, core, False)


def test_delta_long_sequence():
    b = P.Batch(P.SMALL, [1500], 11)
    core = handle(b).delta(b.dx, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, b.dssm, z=b.dz)
    P.check_delta(b, core, True)


def test_delta_of_a_sequence_does_not_depend_on_its_neighbours():
    lens = [130, 1, 77, 20]
    b = P.Batch(P.WIDE, lens, 12)
    start = b.dssm.clone()
    core = handle(b).delta(b.dx, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, b.dssm, z=b.dz)
    for s, n in enumerate(lens):
        rows, ssm = b.rows_of(s), start.clone()
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        alone = handle(b).delta(b.dx[rows], b.dba[rows], b.weights, cu, b.dfirst[s:s + 1], b.dlast[s:s + 1], ssm,
                                z=b.dz[rows])
        assert torch.equal(alone.view(torch.int16), core[rows].view(torch.int16))
        assert torch.equal(ssm[b.last[s]], b.dssm[b.last[s]])


def test_a_prompt_in_pieces_is_the_prompt():
    """Continuing from the stored f32 state gives what the whole prompt gives."""
    b = P.Batch(P.WIDE, [200], 13, same=True)
    ssm, conv = b.dssm.clone(), b.dconv.clone()
    h = handle(b)
    y = h.conv(b.dx, b.dw, b.dcu, b.dfirst, b.dlast, b.dconv)
    core = h.delta(y, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, b.dssm)
    at = 0
    for n in (2, 64, 1, 100, 33):
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        rows = slice(at, at + n)
        yp = h.conv(b.dx[rows], b.dw, cu, b.dfirst, b.dlast, conv)
        assert torch.equal(yp, y[rows])
        cp = h.delta(yp, b.dba[rows], b.weights, cu, b.dfirst, b.dlast, ssm)
        rms = P.f64(core[rows]).reshape(n, -1, 128)
        rms = np.sqrt((rms * rms).mean(2, keepdims=True))
        off = np.abs(P.f64(cp) - P.f64(core[rows])).reshape(n, -1, 128)
        assert (off <= 2.0 ** -7 * np.abs(P.f64(core[rows])).reshape(n, -1, 128) + 2.0 ** -7 * rms).all()
        at += n
    assert torch.equal(conv[b.last[0]], b.dconv[b.last[0]])
    d = P.f64(ssm[b.last[0]]) - P.f64(b.dssm[b.last[0]])
    assert np.linalg.norm(d) <= 4e-5 * np.linalg.norm(P.f64(b.dssm[b.last[0]]))


def test_prefill_index_errors_pad_their_sequence_only():
    b = P.Batch(P.SMALL, [5, 66, 9], 14)
    first, last = b.dfirst.clone(), b.dlast.clone()
    h = handle(b)
    last[1] = b.shape.num_slots
    core = h.delta(b.dx, b.dba, b.weights, b.dcu, first, last, b.dssm)
    assert h.check() == (_native.GDN_ERR_INDEX, (5 << 24) | (1 << 16) | 1)
    b.last[1] = 0
    P.check_delta(b, core, False)
    h.reset()
    assert h.check() == (0, 0)
    h.delta(b.dx, b.dba, b.weights, b.dcu, first, b.dlast, b.dssm, max_len=64)
    assert h.check() == (_native.GDN_ERR_INDEX, (5 << 24) | (3 << 16) | 1)
    h.reset()
    cu = b.dcu.clone()
    cu[2] = 4  # offsets that go back
    conv = b.dconv.clone()
    h.conv(b.dx, b.dw, cu, first, b.dlast, conv)
    assert h.check() == (_native.GDN_ERR_INDEX, (5 << 24) | (2 << 16) | 1)
    assert torch.equal(conv[b.last[1]].view(torch.int16), b.dconv[b.last[1]].view(torch.int16))
    h.reset()
    cu = b.dcu.clone()
    cu[3] = b.T + 1
    h.conv(b.dx, b.dw, cu, first, b.dlast, conv)
    assert h.check() == (_native.GDN_ERR_INDEX, (5 << 24) | (2 << 16) | 2)


@pytest.mark.parametrize("start", [1, 64, 130])
def test_prefill_offsets_that_do_not_start_at_0(start):
    """The first sequence is an error and padding; the others are not affected, and rows
    before the first offset are not taken for a sequence's."""
    b = P.Batch(P.SMALL, [200, 66, 9], 14)
    cu = b.dcu.clone()
    cu[0] = start
    h = handle(b)
    b.last[0] = 0
    core = torch.zeros_like(b.dz)
    h.delta(b.dx, b.dba, b.weights, cu, b.dfirst, b.dlast, b.dssm, out=core)
    assert h.check() == (_native.GDN_ERR_INDEX, (5 << 24) | (2 << 16))
    P.check_delta(b, core, False)
    h.reset()
    y = torch.zeros_like(b.dx)
    h.conv(b.dx, b.dw, cu, b.dfirst, b.dlast, b.dconv, out=y)
    assert h.check() == (_native.GDN_ERR_INDEX, (5 << 24) | (2 << 16))
    want, scale, pool = P.conv_reference(b)
    got = P.f64(y)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * scale).all()
    np.testing.assert_array_equal(P.f64(b.dconv), pool)


def test_outputs_belong_to_the_stream_that_writes_them():
    """An output that a call on a stream of its own makes is that stream's memory: what
    is free on the current stream alone is not taken for it."""
    x, w = torch.ones(300, 64, device="cuda").bfloat16(), torch.ones(520, 64, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    free = torch.empty(300, 520, dtype=torch.bfloat16, device="cuda")
    was = free.data_ptr()
    del free
    y = linear(x, w, stream=side)
    assert y.data_ptr() != was
    torch.cuda.synchronize()
    assert (y == 64).all()


def test_prefill_graph_replay_and_another_stream():
    b = P.Batch(P.WIDE, [70, 1, 129], 15)
    h = handle(b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, core = torch.empty_like(b.dx), torch.empty_like(b.dz)
    def both():
        h.conv(b.dx, b.dw, b.dcu, b.dfirst, b.dlast, b.dconv, out=y)
        h.delta(y, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, b.dssm, z=b.dz, out=core)
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    want = core.clone(), b.dssm.clone(), b.dconv.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for _ in range(3):
        core.zero_()
        y.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(core, want[0])
    live = b.dlast.long()
    assert torch.equal(b.dssm[live], want[1][live]) and torch.equal(b.dconv[live], want[2][live])


def test_prefill_then_decode():
    """A prompt through the prompt-side operators leaves the states that decode
    steps over the same tokens leave, and the next decode step agrees. Both
    round the projections to bf16; the prompt side also rounds the conv's
    output and an f32 sum may round the other way, so the bars are the decode
    step's own (cosine 0.9999; states within 1e-2 of their largest value)."""
    shape = WL.TINY
    n = 70
    rng = torch.Generator().manual_seed(3)
    w = {k: (v.cuda() if v is not None else None) for k, v in WL.make_weights(shape, 31, conv_std=0.4).items()}
    st = WL.make_state(shape, 32)
    x = torch.randn(n + 1, shape.hidden, generator=rng).to(torch.bfloat16).cuda()
    slot = torch.tensor([3], dtype=torch.int32, device="cuda")
    conv_a, ssm_a = st["conv_state"].cuda(), st["ssm_state"].cuda()
    conv_b, ssm_b = conv_a.clone(), ssm_a.clone()
    layer, cores = GdnDecode(shape), []
    for t in range(n + 1):
        if t == n:
            conv_n, ssm_n = conv_a[3].clone(), ssm_a[3].clone()
        core, _ = layer.step(x[t:t + 1], None, w, slot, conv_a, ssm_a)
        cores.append(core.clone())
    h = GdnPrefill(shape, max_tokens=n, max_seqs=1)
    r = x[:n].float()
    xn = (r * torch.rsqrt((r * r).mean(1, keepdim=True) + shape.norm_eps) * (1 + w["input_norm_w"].float())).to(torch.bfloat16)
    qkvz, ba = linear(xn, w["qkvz"]), linear(xn, w["ba"])
    C = shape.conv_channels
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    y = h.conv(qkvz[:, :C], w["conv_w"], cu, slot, slot, conv_b)
    core = h.delta(y, ba, w, cu, slot, slot, ssm_b, z=qkvz[:, C:])
    last, _ = layer.step(x[n:], None, w, slot, conv_b.clone(), ssm_b.clone())
    cos = lambda a, b: torch.nn.functional.cosine_similarity(a.double().flatten(), b.double().flatten(), 0).item()
    assert cos(core, torch.cat(cores[:n])) >= 0.9999
    assert cos(last, cores[n]) >= 0.9999
    assert (ssm_b[3] - ssm_n).abs().max() <= 1e-2 * ssm_n.abs().max()
    assert (conv_b[3].float() - conv_n.float()).abs().max() <= 2.0 ** -7 * conv_n.abs().max()


# ------------------------------------------------------------------ linear

def _linear_reference(x, w, bias, act, residual):
    xd, wd = P.f64(x), P.f64(w)
    y, scale = xd @ wd.T, np.abs(xd) @ np.abs(wd).T
    if bias is not None:
        y = y + P.f64(bias)
        scale = scale + np.abs(P.f64(bias))
    if act == "silu":
        y = P.silu(y)
    elif act == "gelu":
        y = 0.5 * y * (1 + np.tanh(np.sqrt(2 / np.pi) * (y + 0.044715 * y ** 3)))
    return (y + P.f64(residual) if residual is not None else y), scale


def _linear_case(M, N, K, act=None, bias=False, residual=False, stride=0, seed=1, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    def mat(r, c, s):
        t = torch.full((r, c + s), float("nan"), dtype=torch.bfloat16, device="cuda")
        t[:, :c] = torch.randn(r, c, generator=g, device="cuda")
        return t[:, :c]
    up = lambda n: -n % 8
    x, w = mat(M, K, up(K) + 8 * stride), mat(N, K, up(K) + 8 * stride)
    b = torch.randn(N, generator=g, device="cuda").to(torch.bfloat16) if bias else None
    r = mat(M, N, stride) if residual else None
    got = linear(x, w, bias=b, activation=act, residual=r, **kw)
    want, scale = _linear_reference(x, w, b, act, r)
    off = np.abs(P.f64(got) - want) - (2.0 ** -8 * np.abs(want) + 1.2 * (K / 16 + 16) * 2.0 ** -23 * scale)
    assert off.max() <= 0, off.max()
    assert linear_check() == (0, 0)


@pytest.mark.parametrize("M", [1, 2, 5, 16, 17, 64, 65, 128, 129, 300])
@pytest.mark.parametrize("N,K", [(1, 8), (7, 1), (128, 64), (130, 72), (257, 1000), (512, 513), (1024, 2048)])
def test_linear_sizes(M, N, K):
    _linear_case(M, N, K)


@pytest.mark.parametrize("act", [None, "silu", "gelu"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,N,K", [(3, 136, 520), (200, 333, 200), (700, 640, 128)])
def test_linear_epilogue(act, bias, residual, M, N, K):
    _linear_case(M, N, K, act, bias, residual)
    _linear_case(M, N, K, act, bias, residual, stride=3, seed=2)


@pytest.mark.parametrize("M,N,K", [(1, 8192, 8192), (33, 2560, 4096), (1000, 1500, 8192), (4097, 2049, 264)])
def test_linear_large(M, N, K):
    _linear_case(M, N, K, bias=True, residual=True)


def test_linear_adds_in_place():
    g = torch.Generator(device="cuda").manual_seed(4)
    for M in (4, 150):
        x, w, r = (torch.randn(a, b, generator=g, device="cuda").to(torch.bfloat16) for a, b in ((M, 96), (77, 96), (M, 77)))
        want = linear(x, w, residual=r.clone())
        assert linear(x, w, residual=r, out=r) is r
        assert torch.equal(r, want)


def test_linear_keeps_infinities_and_nan_in_their_row_and_column():
    for M in (6, 140):
        x, w = torch.ones(M, 200, dtype=torch.bfloat16, device="cuda"), torch.ones(150, 200, dtype=torch.bfloat16, device="cuda")
        x[3, 7], w[140, 199], x[5, 0] = float("nan"), float("inf"), float("-inf")
        y = linear(x, w)
        assert y[3].isnan().all() and (y[5, :140] == float("-inf")).all() and y[5, 140].isnan()
        keep = [i for i in range(M) if i not in (3, 5)]
        assert (y[keep, 140] == float("inf")).all() and (y[keep][:, :140] == 200).all() and (y[keep][:, 141:] == 200).all()


# ------------------------------------------------------------------ slot_map

def _slots_case(new, ctx, B, wide, pool, count, tokens, seed=1, errors=None):
    rng = np.random.default_rng(seed)
    R = len(new)
    table = rng.integers(1, 1 << 20, (R, wide)).astype(np.int32)
    free = rng.permutation(pool).astype(np.int32) + 5
    want = P.slot_map_reference(new, ctx, B, table, free, count, tokens)
    dev = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32).cuda()
    dtable, error = dev(table).reshape(R, wide), torch.zeros(1, dtype=torch.int32, device="cuda")
    m = slot_map(dev(new), dev(ctx), B, dtable, dev(free), dev([count]), tokens, error=error)
    for got, ref in zip((*m, dtable), want):
        np.testing.assert_array_equal(got.cpu().numpy(), ref)
    assert (int(error) != 0) == want[6]
    if errors is not None:
        assert (int(error) >> 24, (int(error) >> 16) & 255) == (5, errors)


@pytest.mark.parametrize("B", [1, 3, 16, 1 << 20])
@pytest.mark.parametrize("R,top", [(1, 1), (1, 3000), (7, 1), (33, 40), (1023, 3), (1025, 9), (3000, 5)])
def test_slot_map(B, R, top):
    rng = np.random.default_rng(R + top)
    new, ctx = rng.integers(0, top + 1, R), rng.integers(0, 50, R)
    wide = -(-(top + 50) // B)
    need = int((-(-(new + ctx) // B) - -(-ctx // B)).sum())
    _slots_case(new, ctx, B, wide, need + 4, need + 2, int(new.sum()) + 3)


def test_slot_map_ends():
    _slots_case([], [], 4, 3, 5, 4, 6)
    _slots_case([0, 0], [0, 3], 4, 3, 0, 0, 0)
    _slots_case([0, 4], [5, 0], 1, 5, 4, 4, 4)


def test_slot_map_refuses_what_does_not_fit():
    _slots_case([5, 60, 0, 4, 1], [0, 0, 9, 3, 0], 4, 20, 30, 6, 70, errors=2)   # the free list is short
    _slots_case([5, -2, 3], [0, 0, 0], 4, 5, 30, 30, 9, errors=1)                # a negative length
    _slots_case([5, 2, 3], [0, -7, 0], 4, 5, 30, 30, 10, errors=1)
    _slots_case([5, 200, 3], [0, 0, 0], 4, 5, 30, 30, 208, errors=1)             # more blocks than the table holds
    _slots_case([5, 6, 3], [0, 0, 0], 4, 5, 30, 30, 9, errors=3)                 # more tokens than rows
    _slots_case([5, 6], [0, 0], 4, 5, 3, -4, 11, errors=2)                       # counts outside the list
    _slots_case([5, 6], [0, 0], 4, 5, 3, 999, 11, errors=2)
    _slots_case([2 ** 31 - 1] * 3, [2 ** 31 - 1] * 3, 1 << 20, 4096, 9000, 9000, 50, errors=1)  # positions past 32 bits
    _slots_case([2 ** 31 - 1] * 3, [0] * 3, 1 << 20, 4096, 9000, 9000, 50, errors=3)  # sums past 32 bits


def test_slot_map_slots_pass_32_bits():
    new = [3, 2]
    table = torch.tensor([[1 << 20, 0], [2 ** 31 - 1, 0]], dtype=torch.int32, device="cuda")
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    m = slot_map(i(*new), i(7, 4095), 4096, table, i(2 ** 31 - 2), i(1), 5)
    assert m.slots.tolist() == [(1 << 32) + 7, (1 << 32) + 8, (1 << 32) + 9, (2 ** 31 - 1) * 4096 + 4095, (2 ** 31 - 2) * 4096]


def test_slots_for_a_verify_step():
    """A block size of 1 gives a verify step's state slots."""
    table = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    m = slot_map(i(3, 3), i(0, 2), 1, table, i(4, 5, 6, 7, 8, 9), i(6), 6)
    assert m.slots.tolist() == [9, 8, 7, 6, 5, 4] and int(m.free_count) == 0


# ------------------------------------------------------------------ ends and accidents

@pytest.mark.parametrize("lens,extra", [([0], 0), ([0, 0, 0], 0), ([], 5), ([0, 9], 70)], ids=str)
def test_prefill_of_nothing(lens, extra):
    b = P.Batch(P.SMALL, lens, 16, extra=extra)
    h = handle(b)
    y = h.conv(b.dx, b.dw, b.dcu, b.dfirst, b.dlast, b.dconv)
    np.testing.assert_array_equal(P.f64(b.dconv), P.conv_reference(b)[2])
    core = h.delta(b.dx, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, b.dssm, z=b.dz)
    P.check_delta(b, core, True)
    used = int(b.cu[-1])
    assert not y[used:].any() and not core[used:].any()


def test_prefill_of_many_sequences():
    rng = np.random.default_rng(17)
    lens = [int(n) for n in rng.choice([0, 1, 2, 8, 9, 20, 70], 150)]
    b = P.Batch(P.SMALL.with_(num_slots=310), lens, 17, pad=[3, 40], fresh=range(0, 150, 7))
    h = handle(b)
    want, scale, pool = P.conv_reference(b)
    got = P.f64(h.conv(b.dx, b.dw, b.dcu, b.dfirst, b.dlast, b.dconv))
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * scale).all()
    np.testing.assert_array_equal(P.f64(b.dconv), pool)
    P.check_delta(b, h.delta(b.dx, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, b.dssm, z=b.dz), True)
    assert h.check()[0] == 0


@pytest.mark.parametrize("what", ["v", "k", "q", "b", "a"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [0, 13, 70, 149])
def test_delta_of_values_that_are_not_finite(what, value, at):
    """Nothing before such a token changes, nor any row of the state that the
    token's value is not part of."""
    b = P.Batch(P.WIDE, [150, 30], 18)
    sh = b.shape
    Hk, Hv, d = sh.num_k_heads, sh.num_v_heads, sh.head_k_dim
    good = handle(b).delta(b.dx, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, b.dssm.clone(), z=None).view(-1, Hv, d).clone()
    dx, dba, ssm = b.dx.clone(), b.dba.clone(), b.dssm.clone()
    ref = b.dssm.clone()
    handle(b).delta(b.dx, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, ref)
    head, row = 4, 77
    hit = torch.zeros(Hv, d, dtype=torch.bool, device="cuda")  # state rows the value is part of
    if what == "v":
        dx[at, 2 * Hk * d + head * d + row] = value
        hit[head, row] = True
    elif what in "qk":
        dx[at, (Hk * d if what == "k" else 0) + (head // sh.group) * d + 5] = value
        hit[head // sh.group * sh.group:(head // sh.group + 1) * sh.group] = True
    else:
        dba[at, (Hv if what == "a" else 0) + head] = value
        hit[head] = True
    core = handle(b).delta(dx, dba, b.weights, b.dcu, b.dfirst, b.dlast, ssm).view(-1, Hv, d)
    same = lambda a, c: torch.equal(a.contiguous().view(torch.int16), c.contiguous().view(torch.int16))
    before = at // 64 * 64  # whole chunks before the token's; the rest of its chunk within the usual bounds
    assert same(core[:before], good[:before]) and same(core[150:], good[150:])
    want, scale, _, _ = P.delta_reference(b, False)
    off = np.abs(P.f64(core).reshape(180, -1) - want)[:at] - 2.0 ** -8 * (np.abs(want) + scale)[:at]
    assert off.max(initial=-1) <= 0
    if what in "ab" and value == float("inf"):  # gates at their ends: beta 1, e^g 0
        assert core.isfinite().all() and ssm[b.last[0]].isfinite().all()
        return
    assert torch.allclose(core[:150, ~hit].float(), good[:150, ~hit].float(), rtol=2.0 ** -7, atol=1e-6)
    assert not core[at, hit].isfinite().any()
    if what == "q":
        assert same(core[at + 1:150], good[at + 1:150]) and torch.equal(ssm[b.last[0]], ref[b.last[0]])
    else:
        assert not core[at:150, hit].isfinite().any() and not ssm[b.last[0]][hit].isfinite().any()
        err = (ssm[b.last[0]] - ref[b.last[0]])[~hit].double().norm() / ref[b.last[0]][~hit].double().norm()
        assert err <= 2e-5


def test_delta_of_a_state_that_is_not_finite():
    for n in (3, 100):
        b = P.Batch(P.WIDE, [n], 19)
        ref, ssm = b.dssm.clone(), b.dssm.clone()
        good = handle(b).delta(b.dx, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, ref)
        ssm[b.first[0], 2, 50, 3] = float("nan")
        core = handle(b).delta(b.dx, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, ssm)
        bad = 2 * 128 + 50
        assert not core[:, bad].isfinite().any() and not ssm[b.last[0], 2, 50].isfinite().all()
        keep = torch.arange(core.shape[1], device="cuda") != bad
        assert torch.equal(core[:, keep], good[:, keep])
        ssm[b.last[0], 2, 50] = ref[b.last[0], 2, 50]
        assert torch.equal(ssm[b.last[0]], ref[b.last[0]])


def test_python_refusals():
    b = P.Batch(P.SMALL, [5, 66], 20)
    h = handle(b)
    conv = lambda **k: h.conv(**{**dict(x=b.dx, conv_w=b.dw, cu_seqlens=b.dcu, state_in=b.dfirst, state_out=b.dlast,
                                        conv_state=b.dconv), **k})
    delta = lambda **k: h.delta(**{**dict(qkv=b.dx, ba=b.dba, weights=b.weights, cu_seqlens=b.dcu, state_in=b.dfirst,
                                          state_out=b.dlast, ssm_state=b.dssm, z=b.dz), **k})
    for call in (lambda: conv(x=b.dx.float()), lambda: conv(x=b.dx[:, 1:]), lambda: conv(x=b.dx.cpu()),
                 lambda: conv(x=b.dx.T), lambda: conv(cu_seqlens=b.dcu[:2]), lambda: conv(state_out=b.dlast.long()),
                 lambda: conv(conv_state=b.dconv[1:]), lambda: delta(z=b.dz[:, 1:]), lambda: delta(ba=b.dba[1:]),
                 lambda: delta(ssm_state=b.dssm.half()), lambda: delta(out=torch.empty_like(b.dx)),
                 lambda: linear(b.dx, b.dx[:, 8:]), lambda: linear(b.dx, b.dx, activation="relu"),
                 lambda: linear(b.dx, b.dx, bias=b.dx[0])):
        with pytest.raises(ValueError):
            call()
    wide = torch.zeros(71, b.dx.shape[1] + 8, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: conv(x=wide[:, 1:1 + b.dx.shape[1]]), lambda: conv(out=b.dx),
                 lambda: delta(qkv=wide[:, 4:4 + b.dx.shape[1]]), lambda: linear(wide[:, 1:65], wide[:, 8:72])):
        with pytest.raises(GdnError) as e:
            call()
        assert e.value.code == _native.GDN_ERR_ARG
    big = P.Batch(P.SMALL, [99], 21)
    with pytest.raises(GdnError):  # more rows than the handle was made for
        h.conv(big.dx, big.dw, big.dcu, big.dfirst, big.dlast, big.dconv)


def test_example_runs():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "prefill_then_decode.py")
    spec = importlib.util.spec_from_file_location("prefill_then_decode", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    y, cores, conv, ssm, slots, m = ex.main("tiny", 3)
    assert y.shape == (232, WL.TINY.hidden) and y.isfinite().all()
    assert m.cu_seqlens.tolist() == [0, 37, 38, 168, 232] and len(set(slots.tolist())) == 4 and min(slots.tolist()) >= 1
    assert int(m.free_count) == WL.TINY.num_slots - 1 - 4
    for core in cores:
        assert core.isfinite().all() and core.abs().sum(1).min() > 0
    idle = [i for i in range(WL.TINY.num_slots) if i not in slots.tolist()]
    assert not ssm[idle].any() and not conv[idle].any()
