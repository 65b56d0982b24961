"""Products with MXFP8 activations and the routed experts on operands whose fp32 sums are exact
(mx8_exact.py): results and the experts' h bit for bit, by every way that a call can take.
Each test prints the case it runs (flushed) before touching the GPU.
"""
import numpy as np
import pytest
import torch

import mx8_exact as ex
from oracle import mx4_oracle as mx4, mx8_oracle as mx
from test_gpu_mx4 import DT, awq, say  # noqa: F401
from test_gpu_mx8 import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("case", range(len(ex.LAYERS)))
def test_experts_h(awq, case, dt):
    """The 8-bit h of every pair, shown by a down product of single ones: the definition's, whatever
    the way and Y's type."""
    say("experts' h", *ex.LAYERS[case], dt)
    layer = ex.Layer(*ex.LAYERS[case], case, True)
    Y = awq.mx4_experts(*dev(*layer.arrays()), dtype=DT[dt])
    off = layer.check(Y.cpu().double().numpy(), dt)
    say("err/bound", off)
    assert off <= 1


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("case", range(len(ex.LAYERS)))
def test_experts_sums(awq, case, dt):
    say("experts' sums", *ex.LAYERS[case], dt)
    layer = ex.Layer(*ex.LAYERS[case], 100 + case, False)
    Y = awq.mx4_experts(*dev(*layer.arrays()), dtype=DT[dt])
    off = layer.check(Y.cpu().double().numpy(), dt, ex.some_tokens(layer.shape[0], 8))
    say("err/bound", off)
    assert off <= 1


# where a way ends and the next begins: 8, 16 and 17 pairs, 24 an expert, whole and half tiles; the sort's
# second way (more than 16384 pairs)
BORDERS = [(M, E, k, H, I) for M, E, k in [(8, 6, 1), (9, 6, 1), (16, 6, 1), (17, 6, 1), (4, 9, 5), (71, 6, 2), (72, 6, 2), (23, 1, 1), (24, 1, 1),
                                           (128, 1, 1), (129, 1, 1), (256, 1, 1), (257, 1, 1), (385, 1, 1)]
           for H, I in [(96, 4128), (4128, 96)]] + [(5500, 5, 3, 64, 96), (8200, 3, 2, 96, 64)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(BORDERS)))
def test_experts_where_ways_meet(awq, case, dt):
    say("experts, borders of the ways", *BORDERS[case], dt)
    some = ex.some_tokens(BORDERS[case][0], 4)
    for show in (True, False):
        layer = ex.Layer(*BORDERS[case], 200 + case, show)
        Y = awq.mx4_experts(*dev(*layer.arrays()), dtype=DT[dt])
        off = layer.check(Y.cpu().double().numpy(), dt, some)
        say("err/bound", show, off)
        assert off <= 1


# M, out, in: up to 16 tokens by two, four, eight waves a row tile; small tiles; large ones, whole and half
GEMM = [(1, 70, 32), (1, 300, 4096), (4, 20490, 160), (16, 10250, 608), (15, 1000, 14336), (17, 130, 1024), (33, 65, 32),
        (70, 500, 2080), (40, 2000, 4128), (128, 4100, 160), (250, 4090, 1184), (1000, 700, 1056), (2050, 4097, 256), (2050, 4097, 1312)]


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,out,n", GEMM)
def test_gemm_a8(awq, M, out, n, dt):
    """Without large products nothing is cut off: the exact sums, rounded to Y's type."""
    say("gemm_a8, exact sums", M, out, n, dt)
    r = np.random.default_rng(M + n)
    xc, xs = ex.tokens(r, M, n, 0)
    c, s = ex.rows(r, (out,), n)
    Y = awq.mx4_gemm_a8(*dev(xc, xs, c, s), dtype=DT[dt]).cpu()
    want = torch.from_numpy(ex.sums(mx.dequantize(xc, xs), mx4.dequantize(c, s))).to(DT[dt])
    assert torch.equal(Y, want)


@pytest.mark.parametrize("M,out,n", GEMM)
def test_gemm_a8_fp32_keeps_small_products_beside_large(awq, M, out, n):
    say("gemm_a8, fp32, large products", M, out, n)
    r = np.random.default_rng(M + n)
    xc, xs = ex.tokens(r, M, n)
    c, s = ex.rows(r, (out,), n)
    Y = awq.mx4_gemm_a8(*dev(xc, xs, c, s), dtype=torch.float32).cpu()
    want = torch.from_numpy(ex.sums(mx.dequantize(xc, xs), mx4.dequantize(c, s))).float()
    say("wrong", float((Y != want).float().mean()))
    assert torch.equal(Y, want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gemm_a8_small_tiles_with_weights_beyond_32_bits(awq, dt):
    """32 tokens take the small tiles; the last rows against a call on those alone."""
    say("small tiles beyond 2^32 bytes", dt)
    M, out, n, last = 32, 540672, 16384, 32768
    c, s, xc, xs = (torch.randint(lo, hi, shape, dtype=torch.uint8, device="cuda") for lo, hi, shape in
                    [(0, 256, (out, n // 2)), (112, 120, (out, n // 32)), (0, 127, (M, n)), (112, 120, (M, n // 32))])
    Y = awq.mx4_gemm_a8(xc, xs, c, s, dtype=DT[dt])
    Z = awq.mx4_gemm_a8(xc, xs, c[-last:].contiguous(), s[-last:].contiguous(), dtype=DT[dt])
    assert torch.equal(Y[:, -last:], Z) and bool(torch.isfinite(Z).all()) and bool((Z != 0).any())
