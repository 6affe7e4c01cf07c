"""The prompt-side operators where their sizes choose between forms: tile widths, passes over
a key head's value heads, the order of many sequences, long sequences
(tests/prefill_harness.py derives the tolerances but one, below)."""
import numpy as np
import pytest
import torch

from gated_deltanet_layer_gb300 import GdnPrefill, linear, linear_check, workloads as WL
import prefill_harness as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__ as g
    g.build()


def run(b, gated, max_len=None):
    h = GdnPrefill(b.shape, max_tokens=max(b.T, 1), max_seqs=max(b.S, 1))
    core = h.delta(b.dx, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, b.dssm, z=b.dz if gated else None, max_len=max_len)
    assert h.check()[0] == 0
    return core


def shape(Hk, Hv, d, slots=24, state="f32"):
    return WL.LayerShape(f"{Hk}x{Hv}x{d}", hidden=256, num_k_heads=Hk, num_v_heads=Hv, head_k_dim=d, head_v_dim=d,
                         num_slots=slots, ssm_dtype=state)


# ------------------------------------------------------------------ value heads of a key head

@pytest.mark.parametrize("Hk,Hv", [(3, 3), (1, 4), (1, 5), (2, 12), (1, 8)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("state", ["f32", "bf16"])
def test_delta_value_heads_of_a_key_head(Hk, Hv, d, state):
    """One to eight of them, four at a time."""
    b = P.Batch(shape(Hk, Hv, d, state=state), [150, 64, 20, 3], 40, pad=[2])
    P.check_delta(b, run(b, True), True)


@pytest.mark.parametrize("what", ["k", "v", "b"])
def test_delta_of_nan_in_a_later_pass(what):
    """What one value head holds stays there, in the second pass over a key head's as well."""
    b = P.Batch(shape(1, 8, 128), [100], 41)
    good = run(b, False).view(100, 8, 128).clone()
    b = P.Batch(shape(1, 8, 128), [100], 41)
    if what == "k":
        b.dx[70, 128 + 3] = float("nan")
    elif what == "v":
        b.dx[70, 2 * 128 + 6 * 128 + 9] = float("nan")
    else:
        b.dba[70, 6] = float("nan")
    core = run(b, False).view(100, 8, 128)
    hit = torch.zeros(8, 128, dtype=torch.bool, device="cuda")
    if what == "v":
        hit[6, 9] = True
    else:
        hit[slice(None) if what == "k" else 6] = True
    assert core[:70].isfinite().all() and not core[70:, hit].isfinite().any()
    assert torch.allclose(core[70:, ~hit].float(), good[70:, ~hit].float(), rtol=2.0 ** -7, atol=1e-6)


# ------------------------------------------------------------------ many sequences, long ones

@pytest.mark.parametrize("Hk,Hv,d,S", [(2, 4, 64, 39), (2, 4, 64, 60), (1, 2, 64, 128), (1, 2, 64, 129), (2, 6, 128, 30)])
@pytest.mark.parametrize("state", ["f32", "bf16"])
def test_delta_of_many_sequences(Hk, Hv, d, S, state):
    """Lengths that repeat and differ, empty ones and padding among them; the longest ones
    start first where they are more than one wave."""
    rng = np.random.default_rng(42 + S)
    lens = [int(n) for n in rng.choice([0, 1, 14, 15, 20, 20, 64, 65, 100, 130], S)]
    b = P.Batch(shape(Hk, Hv, d, 2 * S + 4, state), lens, 42, pad=[3, S // 2], fresh=range(0, S, 5), extra=9)
    P.check_delta(b, run(b, True), True)


@pytest.mark.parametrize("lens", [[1100], [600, 700, 64]], ids=str)
@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("a_log", [None, -8.0], ids=["decays", "keeps"])
def test_delta_long_sequences_of_large_heads(lens, state, gated, a_log):
    """More than eight chunks of heads of 128: the rows' norms are measured on the way."""
    b = P.Batch(P.WIDE.with_(ssm_dtype=state), lens, 43, a_log=a_log)
    P.check_delta(b, run(b, gated), gated)


# In a chunk S, R, T and U enter their products as two f16 terms each, 2^-23 off at most (half
# of the last of 22 bits), k as it is; T R leaves out lo x lo (2^-24), and the rest is sums in
# f32. So a chunk adds no more than 8 x 2^-23 of the row's norms to the state, and what it
# adds decays with the state: of inputs without cancellation, 1e-6.
@pytest.mark.parametrize("shape,lens", [(P.SMALL, [1500]), (P.WIDE, [1100, 130, 64, 20]), (P.WIDE, [14, 9, 1])], ids=str)
def test_delta_state_of_ordinary_inputs(shape, lens):
    b = P.Batch(shape, lens, 44)
    P.check_delta(b, run(b, False), False, state_tol=1e-6)


# ------------------------------------------------------------------ linear: tiles of 256 columns

@pytest.mark.parametrize("M,N,K", [(4097, 1024, 200), (8192, 257, 136), (8192, 2560, 512), (6000, 3001, 264)])
@pytest.mark.parametrize("act,bias,residual", [(None, False, False), ("silu", True, True), ("gelu", True, False)])
def test_linear_wide_tiles(M, N, K, act, bias, residual):
    """Sizes whose tiles are 256 columns wide, of one round and of several."""
    g = torch.Generator(device="cuda").manual_seed(45)
    mat = lambda r, c: torch.randn(r, c, generator=g, device="cuda").to(torch.bfloat16)
    x, w = mat(M, K), mat(N, K)
    c, r = mat(1, N)[0] if bias else None, mat(M, N) if residual else None
    got = linear(x, w, bias=c, activation=act, residual=r)
    y, scale = x.double() @ w.double().T, x.double().abs() @ w.double().abs().T
    if bias:
        y, scale = y + c.double(), scale + c.double().abs()
    if act == "silu":
        y = y * torch.sigmoid(y)
    elif act == "gelu":
        y = 0.5 * y * (1 + torch.tanh((2 / np.pi) ** 0.5 * (y + 0.044715 * y ** 3)))
    if residual:
        y = y + r.double()
    off = (got.double() - y).abs() - (2.0 ** -8 * y.abs() + 1.2 * (K / 16 + 16) * 2.0 ** -23 * scale)
    assert off.max() <= 0
    assert linear_check() == (0, 0)


# ------------------------------------------------------------------ one handle, call after call

@pytest.mark.parametrize("S", [40, 200])
@pytest.mark.parametrize("graph", [False, True], ids=["calls", "graph"])
def test_calls_of_one_handle_do_not_see_each_other(S, graph):
    """Calls of different offsets and slots, one right after the other on one handle, give
    what each gives by itself: nothing of a call before is left in the workspace."""
    sh = shape(1, 4, 64, 2 * S + 4)
    batches = []
    for seed in (50, 51, 52):
        rng = np.random.default_rng(seed)
        lens = [int(n) for n in rng.choice([0, 1, 14, 15, 20, 64, 65, 130], S)]
        batches.append(P.Batch(sh, lens, seed, pad=[seed - 45], fresh=range(0, S, 7), extra=3))
    most = max(b.T for b in batches)
    make = lambda: GdnPrefill(sh, max_tokens=most, max_seqs=S)

    def call(h, b, y, core):
        h.conv(b.dx, b.dw, b.dcu, b.dfirst, b.dlast, b.dconv, out=y)
        h.delta(b.dx, b.dba, b.weights, b.dcu, b.dfirst, b.dlast, b.dssm, z=b.dz, out=core)

    outs = lambda b: (torch.zeros_like(b.dx), torch.zeros_like(b.dz))
    want = []
    for b in batches:
        o = outs(b)
        call(make(), b, *o)  # first and last slots are apart, so a call again gives the same
        want.append((*o, b.dconv.clone(), b.dssm.clone()))
    torch.cuda.synchronize()
    h, got = make(), [outs(b) for b in batches]

    def several():
        for _ in range(4):
            for b, o in zip(batches, got):
                call(h, b, *o)

    if graph:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            several()
        torch.cuda.synchronize()
        for o in got:
            o[0].zero_(), o[1].zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            several()
        g.replay()
    else:
        several()
    torch.cuda.synchronize()
    assert h.check()[0] == 0
    same = lambda a, c: torch.equal(a.view(torch.uint8), c.view(torch.uint8))
    for b, o, w in zip(batches, got, want):
        assert same(o[0], w[0]) and same(o[1], w[1]) and same(b.dconv, w[2]) and same(b.dssm, w[3])
