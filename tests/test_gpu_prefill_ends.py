"""The prompt-side operators where their arguments come to an end of what they may be
(tests/prefill_harness.py derives the tolerances)."""
import numpy as np
import pytest
import torch

from gated_deltanet_layer_gb300 import GdnPrefill
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
