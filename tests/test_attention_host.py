"""Host-only checks of the attention layer's C ABI and of the projections with
4-bit weights: argument errors come back before any launch. No kernel runs here
(no GPU is needed)."""
import ctypes

import pytest
import torch

from gated_deltanet_layer_gb300 import GdnError, PagedAttention, _native, build as B, kv_append, linear_w4

ARG, UNSUPPORTED = _native.GDN_ERR_ARG, _native.GDN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _native.lib()


def config(**kw):
    c = _native.AttnConfig(num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, max_tokens=100, max_seqs=4, scale=0.1)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("field,value,status", [
    ("num_q_heads", 0, ARG), ("num_kv_heads", 0, ARG), ("head_dim", -1, ARG), ("block_size", 0, ARG), ("max_tokens", 0, ARG),
    ("max_seqs", 0, ARG), ("scale", float("nan"), ARG), ("head_dim", 96, UNSUPPORTED), ("num_q_heads", 9, UNSUPPORTED),
    ("num_q_heads", 2048, UNSUPPORTED), ("max_tokens", 1 << 25, UNSUPPORTED), ("max_seqs", 1 << 16, UNSUPPORTED),
])
def test_config_refused(lib, field, value, status):
    c, h = config(**{field: value}), ctypes.c_void_p()
    assert lib.gdn_attn_workspace_bytes(ctypes.byref(c)) == 0
    assert lib.gdn_attn_create(ctypes.byref(c), 4096, 1 << 40, None, ctypes.byref(h)) == status
    assert not h.value


def test_rows_past_32_bits_refused(lib):
    c = config(num_q_heads=1024, num_kv_heads=1, max_tokens=1 << 24)
    assert lib.gdn_attn_workspace_bytes(ctypes.byref(c)) == 0


def test_create_argument_errors(lib):
    c, h = config(), ctypes.c_void_p()
    n = lib.gdn_attn_workspace_bytes(ctypes.byref(c))
    assert n > 0
    for ws, size in ((None, n), (4096 + 16, n), (4096, n - 1)):
        assert lib.gdn_attn_create(ctypes.byref(c), ws, size, None, ctypes.byref(h)) == ARG
    assert lib.gdn_attn_create(ctypes.byref(c), 4096, n, None, None) == ARG
    assert lib.gdn_attn_create(None, 4096, n, None, ctypes.byref(h)) == ARG
    assert lib.gdn_attn_check(None, None, None) == ARG
    assert lib.gdn_attn_reset(None, None) == ARG
    assert lib.gdn_attn_paged(None, 1, 1, 1, 16, 1024, 16, 256, 16, 256, 1, 16, 1, 16, 16, None, 0, 16, 1024, None) == ARG
    lib.gdn_attn_destroy(None)


# Placeholder device addresses, far apart; every case below has one defect and
# fails on the host, so none is ever used.
A = [0x10_0000_0000 * i for i in range(1, 16)]

APPEND = dict(tokens=4, num_q_heads=8, num_kv_heads=2, head_dim=128, q=A[0], ldq=1024, k=A[1], ldk=256, v=A[2], ldv=256,
              token_pos=A[3], slots=A[4], num_slots=64, inv_freq=A[5], rotary_dim=128, interleaved=0, q_norm_w=A[6],
              k_norm_w=A[7], norm_eps=1e-6, q_out=A[8], ldqo=1024, k_cache=A[9], ldkc=256, v_cache=A[10], ldvc=256,
              error=A[11], stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), ARG), (dict(num_q_heads=0), ARG), (dict(num_kv_heads=0), ARG), (dict(num_slots=-1), ARG),
    (dict(rotary_dim=-16), ARG), (dict(rotary_dim=144), ARG), (dict(inv_freq=None), ARG), (dict(norm_eps=-1.0), ARG),
    (dict(norm_eps=float("nan")), ARG), (dict(q=None), ARG), (dict(q_out=None), ARG), (dict(ldq=1016), ARG),
    (dict(ldq=1025), ARG), (dict(ldqo=1000), ARG), (dict(ldk=248), ARG), (dict(ldv=260), ARG), (dict(ldkc=0), ARG),
    (dict(ldvc=255), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(token_pos=None), ARG), (dict(slots=None), ARG),
    (dict(k_cache=None), ARG), (dict(v_cache=None), ARG), (dict(q=A[0] + 8), ARG), (dict(k=A[1] + 2), ARG),
    (dict(q_norm_w=A[6] + 2), ARG), (dict(k_cache=A[9] + 4), ARG), (dict(token_pos=A[3] + 2), ARG),
    (dict(slots=A[4] + 4), ARG), (dict(error=A[11] + 1), ARG), (dict(inv_freq=A[5] + 2), ARG),
    (dict(head_dim=96, rotary_dim=96), UNSUPPORTED), (dict(rotary_dim=24), UNSUPPORTED), (dict(num_q_heads=1 << 17, ldq=1 << 24, ldqo=1 << 24), UNSUPPORTED),
    # overlaps
    (dict(q_out=A[0] + 16), ARG), (dict(q_out=A[0], ldqo=1032), ARG), (dict(q_out=A[1]), ARG), (dict(k_cache=A[1]), ARG),
    (dict(v_cache=A[9]), ARG), (dict(v_cache=A[0]), ARG), (dict(error=A[4]), ARG), (dict(q_out=A[9]), ARG),
    (dict(k_cache=A[6] - 32), ARG), (dict(v_cache=A[5]), ARG),
])
def test_append_refused(lib, change, status):
    assert lib.gdn_kv_append(*{**APPEND, **change}.values()) == status


def test_append_of_nothing(lib):
    assert lib.gdn_kv_append(*{**APPEND, "tokens": 0}.values()) == 0


PAGED = dict(seqs=2, tokens=6, max_len=3, q=A[0], ldq=1024, k=A[1], ldk=256, v=A[2], ldv=256, num_blocks=8, table=A[3],
             max_blocks=4, cu=A[4], ctx=A[5], gate=A[6], ldg=1024, out=A[7], ldo=1024, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(seqs=-1), ARG), (dict(seqs=5), ARG), (dict(tokens=-1), ARG), (dict(tokens=101), ARG), (dict(max_len=-1), ARG),
    (dict(num_blocks=-1), ARG), (dict(max_blocks=-1), ARG), (dict(cu=None), ARG), (dict(ctx=None), ARG), (dict(table=None), ARG),
    (dict(q=None), ARG), (dict(out=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(cu=A[4] + 2), ARG),
    (dict(ctx=A[5] + 1), ARG), (dict(table=A[3] + 2), ARG), (dict(q=A[0] + 8), ARG), (dict(out=A[7] + 2), ARG),
    (dict(gate=A[6] + 4), ARG), (dict(k=A[1] + 8), ARG), (dict(ldq=1016), ARG), (dict(ldq=1028), ARG), (dict(ldo=512), ARG),
    (dict(ldg=1000), ARG), (dict(ldk=248), ARG), (dict(ldv=257), ARG), (dict(num_blocks=1 << 27), UNSUPPORTED),
    (dict(ldq=1 << 38), UNSUPPORTED), (dict(ldk=1 << 38), UNSUPPORTED), (dict(ldv=1 << 38), UNSUPPORTED),
    # overlaps
    (dict(out=A[0]), ARG), (dict(out=A[1] + 4096), ARG), (dict(out=A[2]), ARG), (dict(out=A[6] + 512), ARG),
    (dict(out=A[4] - 1024), ARG),
])
def test_paged_refused(lib, change, status):
    # a handle needs a device to be made; it holds host state only, its config first, and every
    # check here comes before anything else of it is used
    c = config()
    h = ctypes.create_string_buffer(256)
    ctypes.memmove(h, ctypes.byref(c), ctypes.sizeof(c))
    assert lib.gdn_attn_paged(h, *{**PAGED, **change}.values()) == status


W4 = dict(rows=4, cols=100, inner=256, x=A[0], ldx=256, format=0, group=64, codes=A[1], scales=A[2], zeros=A[3], bias=A[4],
          act=0, residual=A[5], ldr=100, out=A[6], ldo=100, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), ARG), (dict(cols=-1), ARG), (dict(inner=0), ARG), (dict(act=3), ARG), (dict(format=2), ARG),
    (dict(format=1, group=32), ARG), (dict(format=1, group=64, zeros=None), UNSUPPORTED), (dict(group=16), UNSUPPORTED),
    (dict(group=256), UNSUPPORTED), (dict(inner=224, ldx=224), UNSUPPORTED), (dict(x=None), ARG), (dict(codes=None), ARG),
    (dict(scales=None), ARG), (dict(out=None), ARG), (dict(x=A[0] + 8), ARG), (dict(codes=A[1] + 8), ARG),
    (dict(scales=A[2] + 1), ARG), (dict(bias=A[4] + 1), ARG), (dict(residual=A[5] + 1), ARG), (dict(out=A[6] + 1), ARG),
    (dict(ldx=248), ARG), (dict(ldx=257), ARG), (dict(ldo=99), ARG), (dict(ldr=99), ARG), (dict(rows=1 << 21), UNSUPPORTED),
    (dict(cols=1 << 29, ldo=1 << 29, ldr=1 << 29), UNSUPPORTED),
    # overlaps
    (dict(out=A[0]), ARG), (dict(out=A[1]), ARG), (dict(out=A[2]), ARG), (dict(out=A[3]), ARG), (dict(out=A[4]), ARG),
    (dict(out=A[5] + 2), ARG), (dict(out=A[5], ldo=104), ARG),
])
def test_w4_refused(lib, change, status):
    assert lib.gdn_linear_w4(*{**W4, **change}.values()) == status


def test_w4_of_nothing(lib):
    assert lib.gdn_linear_w4(*{**W4, "rows": 0}.values()) == 0
    assert lib.gdn_linear_w4(*{**W4, "cols": 0}.values()) == 0


def test_python_refusals(lib):
    """What the binding refuses before it calls the library."""
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not on a device
        linear_w4(b(2, 64), torch.zeros(8, 32, dtype=torch.uint8), b(8, 2))
    with pytest.raises(ValueError):
        kv_append(b(2, 128), b(2, 64), b(2, 64), torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64), None,
                  b(8, 1, 64), b(8, 1, 64))
    for bad in (dict(head_dim=96), dict(num_q_heads=7), dict(max_tokens=1 << 25), dict(block_size=0), dict(max_seqs=-1),
                dict(max_tokens=1 << 40)):
        a = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, max_tokens=10, max_seqs=2)
        a.update(bad)
        with pytest.raises(GdnError):
            PagedAttention(a.pop("num_q_heads"), a.pop("num_kv_heads"), a.pop("head_dim"), a.pop("block_size"), **a)


def test_calls_from_python_refused(lib):
    """The compiled binding's own checks: types first, whatever comes after."""
    x, f = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(4)
    with pytest.raises(TypeError):
        kv_append(x, x, x, f, f, None, [1], x)
    with pytest.raises(ValueError):
        kv_append(x, x, x, f, f, None, x.view(2, 1, 64), x.view(2, 1, 64))  # not on a device
    with pytest.raises(TypeError):
        linear_w4(None, f, f)
    with pytest.raises(ValueError):
        linear_w4(x, f, f)
    with pytest.raises(ValueError):
        linear_w4(x, f, f, activation="relu")
    with pytest.raises(TypeError):
        _native.calls().linear_w4(None, x)


@pytest.mark.parametrize("scale", [float("inf"), -float("inf"), 3e38])
def test_scale_that_is_not_finite_refused(lib, scale):
    """3e38 is not, once it has taken up the logarithm's base."""
    c, h = config(scale=scale), ctypes.c_void_p()
    assert lib.gdn_attn_workspace_bytes(ctypes.byref(c)) == 0
    assert lib.gdn_attn_create(ctypes.byref(c), 4096, 1 << 40, None, ctypes.byref(h)) == ARG


@pytest.mark.parametrize("scale", [0.0, -0.1, -3e37, 1e-45])
def test_finite_scales_taken(lib, scale):
    assert lib.gdn_attn_workspace_bytes(ctypes.byref(config(scale=scale))) > 0


def test_built_again_for_another_torch(lib, monkeypatch):
    """The binding is bound to the torch that it was built against, whatever the sources' times."""
    assert B.up_to_date()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1")
        assert not B.up_to_date()
    with monkeypatch.context() as m:
        m.setattr(torch.version, "git_version", "0")
        assert not B.up_to_date()
    assert B.up_to_date()
