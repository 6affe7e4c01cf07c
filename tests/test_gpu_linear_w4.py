"""Projections with 4-bit weights on the GPU, against a 64-bit implementation."""
import numpy as np
import pytest
import torch

import attention_harness as H

pytestmark = pytest.mark.gpu


def weights(rng, N, K, group, zeros):
    codes = torch.from_numpy(rng.integers(0, 256, (N, K // 2)).astype(np.uint8)).cuda()
    if group == "mx":
        return codes, torch.from_numpy(rng.integers(117, 126, (N, K // 32)).astype(np.uint8)).cuda(), None
    z = torch.from_numpy(rng.integers(0, 16, (N, K // group)).astype(np.uint8)).cuda() if zeros else None
    return codes, H.bf16(rng.uniform(-0.01, 0.02, (N, K // group))).cuda(), z


def case(M, N, K, group, seed, *, zeros=False, bias=False, act=None, residual=False, stride=0, scale=None):
    from gated_deltanet_layer_gb300 import linear_w4
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K))
    if scale is not None:
        x = x * scale(rng, M, K)
    x = H.strided(H.bf16(x), stride)
    codes, scales, z = weights(rng, N, K, group, zeros)
    b = H.bf16(rng.standard_normal(N)).cuda() if bias else None
    r = H.strided(H.bf16(rng.standard_normal((M, N))), 3 if stride else 0) if residual else None
    want = H.w4_reference(x, codes, scales, z, b, act, r)
    got = linear_w4(x, codes, scales, zeros=z, bias=b, activation=act, residual=r)
    H.check(got, *want, norm=False)
    return x, codes, scales, z, got


@pytest.mark.parametrize("group", ["mx", 32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 16, 128), (1, 1, 256), (2, 129, 1024), (5, 300, 2176), (8, 1000, 512), (9, 257, 1152),
                                   (16, 128, 4096), (17, 130, 640), (32, 500, 1408), (33, 64, 2048), (64, 640, 1280),
                                   (65, 70, 384), (200, 33, 256)])
def test_shapes(group, M, N, K):
    case(M, N, K, group, M + N + K, zeros=True)


@pytest.mark.parametrize("K", [32, 64, 96, 160, 1056, 8160])
def test_inner_sizes(K):
    case(3, 40, K, 32, K, zeros=True)
    case(3, 40, K, "mx", K)


@pytest.mark.parametrize("act", [None, "silu", "gelu"])
@pytest.mark.parametrize("bias,residual", [(True, False), (False, True), (True, True)])
def test_epilogue(act, bias, residual):
    case(7, 203, 640, 64, 5, bias=bias, act=act, residual=residual, stride=16)
    case(40, 77, 320, "mx", 6, bias=bias, act=act, residual=residual)


def test_wide():
    """Columns enough that a CTA has many groups of them and few shares of the inner size."""
    case(4, 20000, 2304, 128, 1, zeros=True)
    case(30, 6000, 2304, 32, 2)


def test_scales_of_rows():
    """Rows of very different sizes, and values of very different sizes in a row."""
    case(8, 64, 1024, 128, 3, zeros=True, scale=lambda r, M, K: np.exp2(r.integers(-60, 60, (M, 1))))
    case(8, 64, 1024, "mx", 4, scale=lambda r, M, K: np.exp2(r.integers(-60, 60, (M, 1)).astype(float)))
    case(5, 64, 512, 32, 5, scale=lambda r, M, K: np.exp2(r.integers(-12, 1, (M, K)).astype(float)))


def test_zero_rows_and_values_that_are_not_finite():
    from gated_deltanet_layer_gb300 import linear_w4
    rng = np.random.default_rng(9)
    for group in ("mx", 32, 128):
        codes, scales, z = weights(rng, 100, 512, group, True)
        x = H.bf16(rng.standard_normal((6, 512))).cuda()
        x[2] = 0
        base = linear_w4(x, codes, scales, zeros=z)
        assert (base[2] == 0).all()
        x[1, 40], x[4, 7] = float("nan"), float("inf")
        got = linear_w4(x, codes, scales, zeros=z)
        rest = [0, 2, 3, 5]
        assert torch.equal(got[rest], base[rest])
        assert not torch.isfinite(got[1].float()).any()
        assert not torch.isfinite(got[4].float())[H.w4_weights(codes, scales, z)[0][:, 7] != 0].any()
    codes, scales, _ = weights(rng, 100, 512, "mx", False)
    x = H.bf16(rng.standard_normal((6, 512))).cuda()
    base = linear_w4(x, codes, scales)
    scales[17, 3] = 255
    got = linear_w4(x, codes, scales)
    assert torch.isnan(got[:, 17]).all()
    rest = [n for n in range(100) if n != 17]
    assert torch.equal(got[:, rest], base[:, rest])


def test_extreme_scales():
    """e8m0 from end to end: 2^-127 and 2^127."""
    from gated_deltanet_layer_gb300 import linear_w4
    codes = torch.full((2, 16), 0x22, dtype=torch.uint8, device="cuda")  # ones
    scales = torch.tensor([[0], [254]], dtype=torch.uint8, device="cuda")
    x = torch.zeros(1, 32, dtype=torch.bfloat16, device="cuda")
    x[0, 0] = 1.0
    got = linear_w4(x, codes, scales).double().cpu()
    assert got[0, 0] == 2.0 ** -127 and got[0, 1] == 2.0 ** 127


def test_residual_in_place_stream_and_graph():
    from gated_deltanet_layer_gb300 import linear_w4
    x, codes, scales, z, base = case(12, 300, 1024, 64, 11, zeros=True)
    r = torch.randn_like(base)
    want = linear_w4(x, codes, scales, zeros=z, residual=r)
    assert linear_w4(x, codes, scales, zeros=z, residual=r, out=r) is r and torch.equal(r, want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = linear_w4(x, codes, scales, zeros=z, stream=st)
    st.synchronize()
    assert torch.equal(got, base)
    out = torch.empty_like(base)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        linear_w4(x, codes, scales, zeros=z, out=out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, base)


@pytest.mark.parametrize("group", ["mx", 32, 128])
@pytest.mark.parametrize("M,N,K", [(12, 2500, 1408), (16, 5000, 256), (20, 4000, 640), (33, 2500, 1152), (64, 4900, 384),
                                   (1, 30000, 512), (40, 5000, 128)])
def test_passes(group, M, N, K):
    """Enough columns that rows are taken 16 or 32 at a time, and CTAs have several groups of them."""
    case(M, N, K, group, M + K, zeros=True)
