"""The checks of experts on exact sums (mx8_exact.py) accept the definition's results, rounded, and reject
those of contractions that leave out their last 32 columns, of an h that is not rounded to
8 bits, and of gate and up products that are cut off below 2^-13 of the largest of eight."""
import numpy as np
import pytest
import torch

import mx8_exact as ex
from oracle import mx4_oracle as mx4, mx8_oracle as mx

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def cut_sums(x, xs, w, ws):
    """x w^T with every product cut off, towards zero, below 2^-13 of the power of two of its eight's largest."""
    out = np.zeros((len(x), len(w)))
    ew = ex.of_eights(ex.exponents(w, ws, 1.0))
    for m, e in enumerate(ex.of_eights(ex.exponents(x, xs, 2.0 ** -6))):
        step = np.ldexp(1.0, (e + ew).max(-1, keepdims=True) - 13)
        out[m] = (np.trunc(ex.of_eights(x[m]) * ex.of_eights(w) / step) * step).sum((-1, -2))
    return out


def output(layer, some, fault=None):
    """The rows `some` of the layer's output as a kernel with `fault` would write them."""
    M, E, k, H, I = layer.shape
    Y = np.zeros((M, H))
    x, xs = mx.dequantize(layer.xc, layer.xs), layer.xs
    for e, t, j in layer.experts(some):
        t = some[t]
        w, ws, wd = mx4.dequantize(layer.gu[e], layer.gus[e]), layer.gus[e], mx4.dequantize(layer.dn[e], layer.dns[e])
        n = H - 32 if fault == "columns of gate and up" else H
        both = cut_sums(x[t], xs[t], w, ws) if fault == "cut" else x[t, :n] @ w[:, :n].T
        h = both[:, :I] / (1 + np.exp(-both[:, :I])) * both[:, I:]
        h = h if fault == "rounding of h" else ex.rounded(h)[0]
        n = I - 32 if fault == "columns of down" else I
        Y[t] += layer.w[t, j][:, None].astype(np.float64) * (h[:, :n] @ wd[:, :n].T)
    return Y


def rounded_to(Y, dt):
    return torch.from_numpy(Y).to(DT[dt]).double().numpy()


@pytest.mark.parametrize("case", range(len(ex.LAYERS)))
def test_checks_tell_right_from_wrong(case):
    some = ex.some_tokens(ex.LAYERS[case][0], 3)[:3]
    I, H = ex.LAYERS[case][4], ex.LAYERS[case][3]
    for show in (True, False):
        layer = ex.Layer(*ex.LAYERS[case], case, show)
        Y = output(layer, some)
        for dt in DT:
            assert layer.check(rounded_to(Y, dt), dt, some) <= 1, (show, dt)
        for fault in ["columns of gate and up", "columns of down", "rounding of h", "cut"]:
            if fault == "columns of gate and up" and H == 32 or not show and fault in ("rounding of h", "cut"):
                continue                               # nothing left; h's own matter
            Y = output(layer, some, fault)
            for dt in DT:
                assert layer.check(rounded_to(Y, dt), dt, some) > 1, (show, fault, dt)


def test_sums_are_exact_in_any_order():
    """fp32 partial sums in three orders: all the exact one."""
    r = np.random.default_rng(1)
    x, w = mx.dequantize(*ex.tokens(r, 3, 2080)), mx4.dequantize(*ex.rows(r, (40,), 2080))
    want = ex.sums(x, w)
    p = (x[:, None] * w[None]).astype(np.float32)
    for order in (np.arange(2080), np.arange(2080)[::-1], r.permutation(2080)):
        assert np.array_equal(np.cumsum(p[..., order], -1, dtype=np.float32)[..., -1], want)
