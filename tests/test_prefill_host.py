"""Host-only checks of the prompt side's C ABI: argument errors come back before
any launch. No kernel runs here (no GPU is needed)."""
import ctypes

import numpy as np
import pytest

from gated_deltanet_layer_gb300 import _native, build as B
import prefill_harness as H

ARG, UNSUPPORTED = _native.GDN_ERR_ARG, _native.GDN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _native.lib()


def config(**kw):
    c = _native.PrefillConfig(num_k_heads=2, num_v_heads=8, head_k_dim=128, head_v_dim=128, conv_kernel=4, num_slots=32,
                              max_tokens=100, max_seqs=4, ssm_dtype=0, gated_norm_eps=1e-6, l2_eps=1e-6, q_scale=0.1)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("field,value,status", [
    ("num_k_heads", 0, ARG), ("num_slots", 0, ARG), ("max_tokens", 0, ARG), ("max_seqs", 0, ARG), ("ssm_dtype", 2, ARG),
    ("l2_eps", -1.0, ARG), ("gated_norm_eps", float("nan"), ARG), ("q_scale", float("nan"), ARG),
    ("conv_kernel", 3, UNSUPPORTED), ("head_k_dim", 96, UNSUPPORTED), ("head_v_dim", 64, UNSUPPORTED),
    ("num_k_heads", 3, UNSUPPORTED), ("max_tokens", 1 << 25, UNSUPPORTED), ("max_seqs", 1 << 17, UNSUPPORTED),
    ("max_seqs", 1 << 16, UNSUPPORTED),
])
def test_config_refused(lib, field, value, status):
    c, h = config(**{field: value}), ctypes.c_void_p()
    assert lib.gdn_prefill_workspace_bytes(ctypes.byref(c)) == 0
    assert lib.gdn_prefill_create(ctypes.byref(c), 4096, 1 << 40, None, ctypes.byref(h)) == status
    assert not h.value


def test_create_argument_errors(lib):
    c, h = config(), ctypes.c_void_p()
    n = lib.gdn_prefill_workspace_bytes(ctypes.byref(c))
    assert n > 0
    for ws, size in ((None, n), (4096 + 16, n), (4096, n - 1)):
        assert lib.gdn_prefill_create(ctypes.byref(c), ws, size, None, ctypes.byref(h)) == ARG
    assert lib.gdn_prefill_create(ctypes.byref(c), 4096, n, None, None) == ARG
    assert lib.gdn_prefill_create(None, 4096, n, None, ctypes.byref(h)) == ARG
    assert lib.gdn_prefill_check(None, None, None) == ARG
    assert lib.gdn_prefill_reset(None, None) == ARG
    assert lib.gdn_prefill_conv(None, 1, 1, 16, 8, 16, 16, 16, 16, 16, 16, 8, None) == ARG
    assert lib.gdn_prefill_delta(None, 1, 1, 1, 16, 8, None, 0, 16, 8, 16, 16, 16, 16, 16, 16, 16, 16, 8, None) == ARG
    lib.gdn_prefill_destroy(None)


# Placeholder device addresses, far apart; every case below has one defect and
# fails on the host, so none is ever used.
A = [0x10_0000_0000 * i for i in range(1, 9)]


def linear_args(**kw):
    a = dict(rows=5, cols=7, inner=9, x=A[0], ldx=16, w=A[1], ldw=16, bias=A[2], act=0, residual=A[3], ldr=7, out=A[4], ldo=7)
    a.update(kw)
    return (*a.values(), None)


@pytest.mark.parametrize("defect", [
    dict(rows=-1), dict(cols=-1), dict(inner=0), dict(act=3), dict(act=-1), dict(x=None), dict(w=None), dict(out=None),
    dict(x=A[0] + 2), dict(w=A[1] + 8), dict(ldx=12), dict(ldw=20), dict(ldx=8), dict(ldw=8), dict(ldo=6), dict(ldr=6),
    dict(bias=A[2] + 1), dict(out=A[0]), dict(out=A[1] + 2), dict(out=A[3] + 2), dict(out=A[3], ldo=8),
], ids=str)
def test_linear_refuses(lib, defect):
    assert lib.gdn_linear(*linear_args(**defect)) == ARG


@pytest.mark.parametrize("edge", [dict(rows=2**31 - 1), dict(cols=2**31 - 1, ldo=2**31, ldr=2**31, residual=None),
                                  dict(inner=2**31 - 1, ldx=2**31, ldw=2**31), dict(ldx=2**38)], ids=str)
def test_linear_beyond_a_tile_map(lib, edge):
    assert lib.gdn_linear(*linear_args(**edge)) == UNSUPPORTED


def test_linear_of_nothing(lib):
    assert lib.gdn_linear(*linear_args(rows=0)) == 0
    assert lib.gdn_linear(*linear_args(cols=0)) == 0


def slot_args(**kw):
    a = dict(requests=3, tokens=9, new=A[0], ctx=A[1], block=4, wide=5, table=A[2], free=A[3], cap=8, count=A[4],
             left=A[4] + 64, cu=A[5], seq=A[6], pos=A[6] + 4096, slots=A[7], error=A[7] + 4096)
    a.update(kw)
    return (*a.values(), None)


@pytest.mark.parametrize("defect", [
    dict(requests=-1), dict(tokens=-1), dict(block=0), dict(wide=-1), dict(cap=-1), dict(new=None), dict(ctx=None),
    dict(table=None), dict(free=None), dict(count=None), dict(left=None), dict(cu=None), dict(seq=None), dict(pos=None),
    dict(slots=None), dict(slots=A[7] + 4), dict(new=A[0] + 2), dict(left=A[4]), dict(seq=A[0]), dict(pos=A[6] + 8),
    dict(error=A[7] + 64),
], ids=str)
def test_slot_map_refuses(lib, defect):
    assert lib.gdn_slot_map(*slot_args(**defect)) == ARG


def test_slot_map_reference_by_hand():
    """The tests' own plain form, against a case worked by hand: blocks of 4,
    contexts of 3 and 4 tokens, 2 and 1 new ones."""
    table = np.array([[7, -1], [8, -1]])
    cu, seq, pos, slots, left, table, wrong = H.slot_map_reference([2, 1], [3, 4], 4, table, [20, 21, 22], 3, 4)
    assert cu.tolist() == [0, 2, 3] and seq.tolist() == [0, 0, 1, -1] and pos.tolist() == [3, 4, 4, -1]
    assert slots.tolist() == [31, 88, 84, -1] and left == 1 and table.tolist() == [[7, 22], [8, 21]] and not wrong
