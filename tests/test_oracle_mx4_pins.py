"""Hand-worked values of the MXFP4 oracle (CPU)."""
import numpy as np
import pytest

from oracle import mx4_oracle as mx

INF, NAN = float("inf"), float("nan")


def block(*first):
    v = np.zeros((1, 32), np.float32)
    v[0, :len(first)] = first
    return v


def codes_of(c):
    return np.stack((c & 15, c >> 4), -1).reshape(c.shape[0], -1)


def test_every_magnitude_and_sign_in_place():
    mags = [0, .5, 1, 1.5, 2, 3, 4, 6]
    v = np.array([mags + [-m for m in mags[1:]] + [-0.0] + [0] * 16], np.float32)
    c, s = mx.quantize(v)
    assert s.tolist() == [[127]]                       # largest 6: floor(log2 6) - 2 = 0
    assert codes_of(c)[0].tolist() == list(range(8)) + [9, 10, 11, 12, 13, 14, 15, 8] + [0] * 16
    assert c[0, 0] == 0x10                             # columns 0, 1 = codes 0, 1: the even one in the low half
    assert np.array_equal(mx.dequantize(c, s), v.astype(np.float64))


@pytest.mark.parametrize("x,want", [(0.25, 0), (0.26, .5), (0.75, 1), (0.74, .5), (1.25, 1), (1.26, 1.5), (1.75, 2),
                                    (1.74, 1.5), (2.5, 2), (2.51, 3), (3.5, 4), (3.49, 3), (5, 4), (5.01, 6), (7.9, 6)])
def test_rounding_to_nearest_ties_to_the_even_code(x, want):
    c, s = mx.quantize(block(4.0, x, -x))
    assert s[0, 0] == 127
    assert mx.dequantize(c, s)[0, 1:3].tolist() == [want, -want]


@pytest.mark.parametrize("top,byte", [(1.0, 125), (7.99, 127), (8.0, 128), (2.0 ** -126, 0), (2.0 ** -124, 1),
                                      (2.0 ** -149, 0), (0.0, 0), (3.4e38, 252)])
def test_scale_byte(top, byte):
    c, s = mx.quantize(block(0.0, top))
    assert s[0, 0] == byte


def test_nan_and_infinite_blocks_stand_alone():
    for bad in (NAN, INF, -INF):
        v = np.concatenate((block(1.0, bad), block(1.0)), 1)
        c, s = mx.quantize(v)
        assert s[0].tolist() == [255, 125] and not c[0, :16].any()
        d = mx.dequantize(c, s)
        assert np.isnan(d[0, :32]).all() and d[0, 32] == 1.0 and not d[0, 33:].any()


def test_column_scales_multiply_before_the_rounding():
    v = block(3.0, 1.0)
    s = np.ones(32, np.float32)
    s[0] = 2.0
    c, sc = mx.quantize(v, s)
    assert sc[0, 0] == 127 and mx.dequantize(c, sc)[0, :2].tolist() == [6.0, 1.0]


def test_error_bound():
    """Below the saturation (|v| <= 6 2^e) a value is off by at most one unit 2^e."""
    v = np.random.default_rng(3).standard_normal((64, 256)).astype(np.float32)
    c, s = mx.quantize(v)
    d, unit = mx.dequantize(c, s), np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, 1)
    assert (np.abs(d - v) <= np.where(np.abs(v) <= 6 * unit, 1.0, 2.0) * unit).all()


def test_product_by_hand():
    c, s = mx.quantize(np.concatenate((block(1.0, -2.0), block(0.5)), 1))
    x = np.zeros((1, 64))
    x[0, 0], x[0, 1], x[0, 32] = 10, 1, 4
    assert mx.gemm(x, c, s).tolist() == [[10.0]]       # 10 - 2 + 2


def test_routing_by_hand():
    x = np.array([[1.0, 0.0]])
    router = np.log(np.array([[1.0, 1], [4, 1], [4, 1], [1, 1]]))
    ids, w, _ = mx.route(x, router, 2, True)
    assert ids.tolist() == [[1, 2]]                    # equal logits: the lower expert first
    assert np.allclose(w, [[0.5, 0.5]])
    _, w, _ = mx.route(x, router, 3, False)
    assert np.allclose(w, [[0.4, 0.4, 0.1]])


def test_moe_by_hand():
    """One expert routed: y = Wd (silu(Wg x) * (Wu x))."""
    gate, up, down = block(2.0), block(0.0, 3.0), block(1.0)
    gu = np.zeros((2, 64, 32), np.float32)
    gu[1, 0], gu[1, 32] = gate[0], up[0]               # intermediate column 0 of expert 1
    dn = np.zeros((2, 32, 32), np.float32)
    dn[1, 5] = down[0]
    q = [[mx.quantize(m) for m in a] for a in (gu, dn)]
    gc, gs, dc, ds = (np.stack([t[i] for t in l]) for l in q for i in (0, 1))
    x = np.zeros((1, 32))
    x[0, 0], x[0, 1] = 1.0, 2.0
    router = np.zeros((2, 32))
    router[1, 0] = 5.0
    y = mx.moe(x, router, gc, gs, dc, ds, 1, True)
    want = np.zeros((1, 32))
    want[0, 5] = 2.0 / (1 + np.exp(-2.0)) * 6.0
    assert np.allclose(y, want, rtol=1e-15)
