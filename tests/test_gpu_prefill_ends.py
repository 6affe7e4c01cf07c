"""The prompt-side operators where their arguments come to an end of what they may be
(tests/prefill_harness.py derives the tolerances)."""
import numpy as np
import pytest
import torch

from gated_deltanet_layer_gb300 import GdnError, GdnPrefill, _native, linear, prefill, slot_map, workloads as WL
import prefill_harness as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def handle(b, **kw):
    return GdnPrefill(b.shape, max_tokens=max(b.T, 1), max_seqs=max(b.S, 1), **kw)


def delta(h, b, gated=False, **kw):
    return h.delta(b.dx, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, b.dssm, z=b.dz if gated else None, **kw)


# ------------------------------------------------------------------ the norms' constants

@pytest.mark.parametrize("shape", [P.SMALL, P.WIDE], ids=lambda s: s.name)
@pytest.mark.parametrize("n", [13, 15, 16, 20, 48, 50, 63, 64, 70, 130])
def test_delta_without_l2_eps(shape, n):
    """x / sqrt(sum x^2) is an ordinary number for every token; the rows past a
    chunk's last token are nobody's."""
    b = P.Batch(shape.with_(l2_eps=0.0), [n, 3], 30)
    h = handle(b)
    P.check_delta(b, delta(h, b, True), True)
    assert h.check()[0] == 0


@pytest.mark.parametrize("kw", [dict(l2_eps=0.25), dict(q_scale=-3.0), dict(gated_norm_eps=0.5),
                                dict(l2_eps=0.0, q_scale=1.0, gated_norm_eps=0.0)], ids=str)
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_delta_of_other_constants(kw, gated):
    b = P.Batch(P.WIDE.with_(**kw), [70, 5], 31)
    P.check_delta(b, delta(handle(b), b, gated), gated)


@pytest.mark.parametrize("what", ["k", "q"])
@pytest.mark.parametrize("n,at", [(12, 0), (12, 7), (100, 0), (100, 5), (100, 40), (100, 63), (100, 70)])
def test_delta_of_a_zero_row_without_l2_eps(what, n, at):
    """0 / sqrt(0) is not a number: a zero q's outputs are lost, a zero key's state and
    outputs from its token on, and nothing else, in either form."""
    b = P.Batch(P.WIDE.with_(l2_eps=0.0), [n, 30], 32)
    sh = b.shape
    d = sh.head_k_dim
    head = (sh.num_k_heads if what == "k" else 0) + 1  # the second key head's
    b.dx[at, head * d:(head + 1) * d] = 0
    with np.errstate(invalid="ignore"):
        want, scale, pool, norm = P.delta_reference(b, False)
    got = P.f64(delta(handle(b), b))
    there = np.isfinite(want)
    assert not there[at].all() and there[:at].all() and there[n:].all()
    np.testing.assert_array_equal(np.isfinite(got), there)
    off = np.abs(got - want)[there] - 2.0 ** -8 * (np.abs(want) + scale)[there]
    assert off.max() <= 0
    for s in (0, 1):
        state, ref = P.f64(b.dssm)[b.last[s]], pool[b.last[s]]
        np.testing.assert_array_equal(np.isfinite(state), np.isfinite(ref))
        for head in range(sh.num_v_heads):
            if np.isfinite(ref[head]).all():
                assert np.linalg.norm(state[head] - ref[head]) <= 2e-5 * norm[s][head]


# ------------------------------------------------------------------ offsets that are not in order

LINE = WL.LayerShape("line", hidden=64, num_k_heads=1, num_v_heads=1, head_k_dim=64, head_v_dim=64, num_slots=10010)
EVEN = [100 * s for s in range(41)]


def _with(offsets, at, value):
    return offsets[:at] + [value] + offsets[at + 1:]


def _long():
    n = np.random.default_rng(33).choice([0, 1, 1, 2, 20, 70], 5000)
    return np.concatenate([[0], np.cumsum(n)]).tolist()


# offsets, rows, sequences that stay as they are, sequences that are to blame
OFFSETS = {
    "goes back over a chunk": ([0, 130, 5, 200], 200, [0], [1]),
    "goes back by one token": ([0, 130, 129, 200], 200, [0], [1]),
    "owns no chunk place": ([0, 70, 4, 80], 80, [0], [1]),
    "past the rows": ([0, 10, 5000, 60, 70], 100, [0, 3], [1, 2]),
    "past the rows, chunks": ([0, 100, 5000, 300, 430], 450, [0, 3], [1, 2]),
    "the last": ([0, 70, 140, 0], 150, [0, 1], [2]),
    "the first": ([3, 70, 140], 150, [1], [0]),
    "the first below 0": ([-3, 70, 140], 150, [1], [0]),
    "all": ([-5, 300, 7, 2 ** 31 - 1, -2 ** 31], 120, [], [0, 1, 2, 3]),
    "one of 40, past": (_with(EVEN, 4, 4001), 4000, [s for s in range(40) if s not in (3, 4)], [3, 4]),
    "one of 40, far past": (_with(EVEN, 31, 2 ** 31 - 1), 4000, [s for s in range(40) if s not in (30, 31)], [30, 31]),
    "one of 40, below 0": (_with(EVEN, 33, -1), 4000, [s for s in range(40) if s not in (32, 33)], [32, 33]),
    # the nineteenth's rows reach over those of the fifteen that follow
    "one of 40, too far": (_with(EVEN, 20, 3500), 4000, [*range(20), *range(35, 40)], [20]),
    "one of 128": (_with([20 * s for s in range(129)], 64, 5), 2600, [s for s in range(128) if s not in (63, 64)], [63]),
    "the last but one of 128": (_with([20 * s for s in range(129)], 127, 2580), 2600, list(range(127)), [127]),
    "one of 129": (_with([20 * s for s in range(130)], 65, 2601), 2600, [s for s in range(129) if s not in (64, 65)], [64, 65]),
    "one of 5000": (_with(_long(), 777, 5), None, [s for s in range(5000) if s not in (776, 777)], [776]),
    "none of 5000": (_long(), None, list(range(5000)), []),
}


def _bad_batch(name):
    """A batch with these offsets. The sequences that they make padding have slots all the
    same, which are not to be touched; rows that no other sequence owns hold NaN."""
    cu, T, good, blamed = OFFSETS[name]
    S = len(cu) - 1
    T = T if T is not None else max(cu) + 9
    b = P.Batch(LINE if S > 100 else P.SMALL.with_(num_slots=2 * S + 4), [T] + [0] * (S - 1), 34)
    b.cu = np.array(cu, np.int64)
    b.lens = [cu[s + 1] - cu[s] if s in set(good) else 0 for s in range(S)]
    b.dcu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    owned = np.zeros(T, bool)
    for s in good:
        owned[cu[s]:cu[s + 1]] = True
    for t in (b.dx, b.dz, b.dba):
        t[torch.from_numpy(~owned).cuda()] = float("nan")
    b.last = np.where(np.isin(np.arange(S), good), b.last, 0)  # of the references; b.dlast keeps the slots
    h = handle(b)
    h.workspace[4096:] = 255  # nothing that an earlier call may have left
    return b, h, blamed


def _check_blame(h, blamed):
    status, word = h.check()
    if not blamed:
        assert status == 0
    else:
        assert status == _native.GDN_ERR_INDEX and word >> 16 == (5 << 8 | 2) and word & 0xffff in blamed


@pytest.mark.parametrize("name", OFFSETS)
def test_conv_of_bad_offsets(name):
    b, h, blamed = _bad_batch(name)
    out = torch.full_like(b.dx, float("nan"))
    h.conv(b.dx, b.dw, b.dcu, b.dfirst, b.dlast, b.dconv, out=out)
    _check_blame(h, blamed)
    want, scale, pool = P.conv_reference(b)
    got = P.f64(out)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * scale).all()
    np.testing.assert_array_equal(P.f64(b.dconv), pool)


@pytest.mark.parametrize("name", OFFSETS)
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_delta_of_bad_offsets(name, gated):
    b, h, blamed = _bad_batch(name)
    core = delta(h, b, gated, out=torch.full_like(b.dz, float("nan")))
    _check_blame(h, blamed)
    P.check_delta(b, core, gated)


# ------------------------------------------------------------------ rows of other magnitudes

@pytest.mark.parametrize("shape", [P.SMALL, P.WIDE], ids=lambda s: s.name)
@pytest.mark.parametrize("how", ["small", "large"])
@pytest.mark.parametrize("fresh", [False, True])
def test_delta_rows_do_not_share_their_precision(shape, how, fresh):
    """A row of the state needs no other row, so the bounds of a head's state and of its
    outputs hold for each of its rows by itself, however large the others are: the state's
    2e-5 of the row's own norms, the outputs' 2^-8 of what |S| |q| allows."""
    b = P.Batch(shape, [130, 70, 9], 35, fresh=[0, 1, 2] if fresh else [])
    Hk, Hv, d = shape.num_k_heads, shape.num_v_heads, shape.head_k_dim
    # rows of 1, 2^-13, 2^-26 and 2^-40 side by side, or one row of 2^40 among them
    f = 2.0 ** torch.tensor([0, -13, -26, -40] if how == "small" else [0, 0, 0, 0]).repeat(Hv * d // 4)
    if how == "large":
        f[5::d] = 2.0 ** 40
    f = f.cuda()
    b.dx[:, 2 * Hk * d:] *= f.to(torch.bfloat16)
    b.dssm *= f.view(1, Hv, d, 1)
    b.ssm0 = P.f64(b.dssm)
    core, ssm = P.f64(delta(handle(b), b)).reshape(b.T, Hv, d), P.f64(b.dssm)
    assert np.isfinite(core).all()
    x, ba = P.f64(b.dx), P.f64(b.dba)
    rate, shift = np.exp(P.f64(b.weights["A_log"])), P.f64(b.weights["dt_bias"])
    for s in range(b.S):
        S = b.ssm0[b.first[s]].copy() if b.first[s] > 0 else np.zeros((Hv, d, d))
        most = np.sqrt((S * S).sum(2))
        for t in range(int(b.cu[s]), int(b.cu[s + 1])):
            q, k, v = (x[t, i:j].reshape(-1, d) for i, j in ((0, Hk * d), (Hk * d, 2 * Hk * d), (2 * Hk * d, None)))
            q = np.repeat(q / np.sqrt((q * q).sum(1, keepdims=True) + shape.l2_eps) * shape.scale_q, shape.group, 0)
            k = np.repeat(k / np.sqrt((k * k).sum(1, keepdims=True) + shape.l2_eps), shape.group, 0)
            beta = 1 / (1 + np.exp(-ba[t, :Hv]))
            S *= np.exp(-rate * np.logaddexp(0, ba[t, Hv:] + shift))[:, None, None]
            S += (beta[:, None] * (v - np.einsum("hvk,hk->hv", S, k)))[:, :, None] * k[:, None, :]
            most = np.maximum(most, np.maximum(np.sqrt((S * S).sum(2)), np.abs(v)))
            o = np.einsum("hvk,hk->hv", S, q)
            off = np.abs(core[t] - o) - 2.0 ** -8 * (np.abs(o) + np.sqrt((S * S).sum(2)) * np.sqrt((q * q).sum(1))[:, None])
            assert off.max() <= 0
        d2 = ssm[b.last[s]] - S
        err = np.sqrt((d2 * d2).sum(2)) / most
        assert err.max() <= 2e-5, f"state rows of sequence {s}: {err.max():.3g}"


# ------------------------------------------------------------------ streams

@pytest.mark.parametrize("given", [True, False], ids=["given", "current"])
@pytest.mark.parametrize("call", ["conv", "delta"])
def test_workspace_outlives_a_dropped_handle(call, given):
    """A handle dropped while its call runs on another stream leaves its workspace to
    that call: the stream that it was made on does not get the memory before."""
    b = P.Batch(P.SMALL, [100, 3], 36)
    side = torch.cuda.Stream()
    out = torch.empty_like(b.dx if call == "conv" else b.dz)

    def run(h, **kw):
        if call == "conv":
            h.conv(b.dx, b.dw, b.dcu, b.dfirst, b.dlast, b.dconv, out=out, **kw)
        else:
            h.delta(b.dx, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, b.dssm, out=out, **kw)

    run(handle(b))  # a kernel's first launch waits for the device
    h = GdnPrefill(b.shape, max_tokens=5000, max_seqs=2)
    torch.cuda.synchronize()
    where, size = h.workspace.data_ptr(), h.workspace.numel()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # what comes next on this stream is not done for a tenth of a second
    with torch.cuda.stream(None if given else side):
        run(h, stream=side if given else None)
    del h
    held = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(3)]
    assert not side.query() and where not in [t.data_ptr() for t in held]
    torch.cuda.synchronize()
    assert out.isfinite().all()


# ------------------------------------------------------------------ devices

def test_tensors_of_another_device_are_refused(monkeypatch):
    """Kernels run on the current device. What belongs to another one (here: everything,
    once the binding is told of several devices, 1 the current one) is an error, not a launch."""
    b = P.Batch(P.SMALL, [20, 3], 37)
    h = handle(b)
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    lens, ctx, table, free, count = i(3, 3), i(0, 2), torch.zeros(2, 8, dtype=torch.int32, device="cuda"), i(4, 5, 6, 7, 8), i(5)
    own = torch.cuda.Stream()
    conv, ssm = b.dconv.clone(), b.dssm.clone()
    monkeypatch.setattr(prefill, "_device", lambda: 1)
    monkeypatch.setattr(prefill, "_several", True)
    for call in (lambda: linear(b.dx, b.dx), lambda: slot_map(lens, ctx, 1, table, free, count, 6),
                 lambda: h.conv(b.dx, b.dw, b.dcu, b.dfirst, b.dlast, b.dconv), lambda: delta(h, b)):
        with pytest.raises(ValueError, match="current device"):
            call()
    with pytest.raises(ValueError, match="current device"):
        prefill._stream(own)
    monkeypatch.undo()
    torch.cuda.synchronize()
    same = lambda a, c: torch.equal(a.view(torch.uint8), c.view(torch.uint8))
    assert same(conv, b.dconv) and same(ssm, b.dssm) and not table.any()


# ------------------------------------------------------------------ sizes past 32 bits

def test_sizes_past_32_bits_are_refused():
    """Sizes are 32 bits at the C ABI. A larger one is an error, not what is left of it."""
    long = torch.empty(1, 2 ** 32 + 8, dtype=torch.bfloat16, device="cuda")
    for x, w in ((long, long), (long[:, :1], long.T), (long.T, long[:, :1])):
        with pytest.raises(GdnError) as e:
            linear(x, w)
        assert e.value.code == _native.GDN_ERR_UNSUPPORTED
    del long, x, w
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    table = torch.zeros(1, 8, dtype=torch.int32, device="cuda")
    for block, tokens in ((2 ** 32 + 4, 3), (4, 2 ** 32 + 3), (-2 ** 32 + 4, 3), (0, 3)):
        with pytest.raises(GdnError) as e:
            slot_map(i(3), i(0), block, table, i(4, 5), i(2), tokens)
        assert e.value.code == _native.GDN_ERR_ARG and not table.any()
    for kw in (dict(max_tokens=2 ** 32 + 64), dict(max_seqs=2 ** 32 + 2)):
        with pytest.raises(GdnError):
            GdnPrefill(P.SMALL, **{**dict(max_tokens=64, max_seqs=2), **kw})


@pytest.mark.parametrize("most", [2 ** 31, 2 ** 32, 2 ** 40, 2 ** 32 + 5])
def test_any_bound_of_the_lengths_will_do(most):
    """max_len is an upper bound, however large."""
    b = P.Batch(P.SMALL, [20, 3], 38)
    h = handle(b)
    P.check_delta(b, delta(h, b, max_len=most), False)
    assert h.check()[0] == 0
    for below in (-1, -2 ** 32):
        with pytest.raises(GdnError):
            delta(h, b, max_len=below)


@pytest.mark.parametrize("tokens", [0, 300000])
def test_slot_map_of_two_billion_blocks(tokens):
    """A request of 2^31 - 1 new blocks: every one of them is written, by one CTA or many."""
    n = 2 ** 31 - 1
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    free = torch.arange(n, dtype=torch.int32, device="cuda")
    table = torch.full((1, n), -1, dtype=torch.int32, device="cuda")
    error = i(0)
    m = slot_map(i(n), i(0), 1, table, free, i(n), tokens, error=error)
    assert int(m.free_count) == 0 and int(error) == (5 << 24 | 3 << 16)  # more tokens than rows
    step = 1 << 28
    for at in range(0, n, step):
        end = min(n, at + step)
        assert torch.equal(table[0, at:end], torch.arange(n - 1 - at, n - 1 - end, -1, dtype=torch.int32, device="cuda"))
    assert torch.equal(m.slots, torch.arange(n - 1, n - 1 - tokens, -1, device="cuda"))


# ------------------------------------------------------------------ states near the largest float

@pytest.mark.parametrize("n", [9, 100, 700])
def test_delta_forgets_a_state_near_the_largest_float(n):
    """A finite state however large, once it is forgotten, leaves nothing behind."""
    b = P.Batch(P.SMALL, [n, 70], 39, a_log=6.0)
    b.dssm[b.first[0]] *= 1 / b.dssm[b.first[0]].abs().max()
    b.dssm[b.first[0]] *= 2e38
    assert b.dssm[b.first[0]].isfinite().all()
    b.ssm0 = P.f64(b.dssm)
    b.dba[:, b.shape.num_v_heads:] = 3.0  # e^g is 0 in f32 from the first token on
    core = delta(handle(b), b)
    fresh = P.Batch(P.SMALL, [n, 70], 39, a_log=6.0, fresh=[0])
    fresh.dba[:, b.shape.num_v_heads:] = 3.0
    want = delta(handle(fresh), fresh)
    rows = P.f64(want).reshape(b.T, -1, 64)
    rms = np.sqrt((rows * rows).mean(2, keepdims=True))
    off = np.abs(P.f64(core).reshape(rows.shape) - rows)
    assert (off <= 2.0 ** -8 * np.abs(rows) + 2.0 ** -8 * rms).all()
    s, f = P.f64(b.dssm)[b.last[0]], P.f64(fresh.dssm)[fresh.last[0]]
    assert np.linalg.norm(s - f) <= 2e-5 * np.linalg.norm(f)


# ------------------------------------------------------------------ outputs beside inputs

@pytest.mark.parametrize("M", [5, 300])
def test_linear_writes_beside_its_inputs(M):
    """x, the residual and the output as columns of the same rows."""
    g = torch.Generator(device="cuda").manual_seed(46)
    K, N = 64, 77
    rows = torch.randn(M, 64 + 2 * N + 6, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(N, K, generator=g, device="cuda").to(torch.bfloat16)
    before = rows.clone()
    want = linear(rows[:, :K].clone(), w, residual=rows[:, K:K + N].clone())
    out = rows[:, K + N:K + 2 * N]
    assert linear(rows[:, :K], w, residual=rows[:, K:K + N], out=out) is out
    assert torch.equal(out, want) and torch.equal(rows[:, :K + N], before[:, :K + N])
    assert torch.equal(rows[:, K + 2 * N:], before[:, K + 2 * N:])


def test_prefill_writes_beside_its_inputs():
    """The conv's outputs beside its inputs, and the delta rule's in the q | k | v columns of
    the projection's rows, beside z: the conv is the last to read those."""
    b = P.Batch(P.SMALL, [70, 5], 47)
    C, cols = b.shape.conv_channels, b.shape.num_v_heads * 64
    h = handle(b)
    conv, ssm = b.dconv.clone(), b.dssm.clone()
    y = h.conv(b.dx, b.dw, b.dcu, b.dfirst, b.dlast, conv)
    want = h.delta(y, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, ssm, z=b.dz)
    rows = torch.cat([b.dx, torch.zeros_like(b.dx), b.dz], 1)
    beside = h.conv(rows[:, :C], b.dw, b.dcu, b.dfirst, b.dlast, b.dconv, out=rows[:, C:2 * C])
    assert torch.equal(beside, y) and torch.equal(rows[:, :C], b.dx)
    core = h.delta(beside, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, b.dssm, z=rows[:, 2 * C:], out=rows[:, :cols])
    live = b.dlast.long()
    assert torch.equal(core, want) and torch.equal(rows[:, 2 * C:], b.dz) and torch.equal(b.dssm[live], ssm[live])


@pytest.mark.parametrize("shift", [-1, 1, 63, -63])
def test_outputs_over_inputs_are_refused(shift):
    rows = torch.zeros(9, 320, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(GdnError) as e:
        linear(rows[:, 128:192], w, out=rows[:, 128 + shift:192 + shift])
    assert e.value.code == _native.GDN_ERR_ARG
    flat = rows.view(-1)
    with pytest.raises(GdnError):  # the output's rows run on into x's of the next row
        linear(rows[1:5, :64], w, out=torch.as_strided(flat, (4, 64), (320, 1), 300))
