"""MXFP4 (microscaled 4-bit floating point) in numpy, fp64: the plain statement
of awq_mx4_quantize, the products and the mixture-of-experts layer.

Test infrastructure only; shares nothing with the HIP library. Arrays: codes
uint8 (rows, in / 2), scales uint8 (rows, in / 32), values fp64."""
import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(W, s=None):
    """W fp32 (rows, in), s fp32 (in) or None -> (codes, scales)."""
    v = np.asarray(W, np.float32)
    if s is not None:
        with np.errstate(over="ignore", invalid="ignore"):
            v = v * np.asarray(s, np.float32)[None, :]          # fp32 products
    rows, n = v.shape
    b = v.reshape(rows, n // 32, 32).astype(np.float64)
    bad = ~np.isfinite(b).all(2)
    a = np.abs(np.where(bad[..., None], 0.0, b))
    top = a.max(2)
    m, ex = np.frexp(top)                                       # top = m 2^ex, m in [0.5, 1)
    e = np.where(top == 0, -127, np.clip(ex - 1 - 2, -127, 127))
    x = np.ldexp(a, -e[..., None])
    # nearest magnitude; of two equally near ones that with the even index
    code = np.zeros(x.shape, np.int64)
    best = np.abs(x - MAGNITUDES[0])
    for i in range(1, 8):
        d = np.abs(x - MAGNITUDES[i])
        take = (d < best) | ((d == best) & (i % 2 == 0))
        code[take] = i
        best = np.minimum(best, d)
    code += 8 * np.signbit(b)
    code[bad] = 0
    scale = np.where(bad, 255, e + 127).astype(np.uint8)
    code = code.reshape(rows, n // 2, 2)
    return (code[..., 0] + 16 * code[..., 1]).astype(np.uint8), scale


def dequantize(codes, scales):
    """The values, fp64 (..., in); NaN where the scale is 255."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1).astype(np.int64)
    v = np.where(c >= 8, -1.0, 1.0) * MAGNITUDES[c & 7]
    f = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(f, 32, axis=-1)


def gemm(X, codes, scales):
    return np.asarray(X, np.float64) @ dequantize(codes, scales).T


def route(X, router, top_k, renorm):
    """(ids (M, k), weights (M, k), logits (M, E)), fp64; equal logits: the lowest expert."""
    logits = np.asarray(X, np.float64) @ np.asarray(router, np.float64).T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top_k]
    p = np.exp(logits - logits.max(1, keepdims=True))
    w = np.take_along_axis(p / p.sum(1, keepdims=True), ids, 1)
    if renorm:
        w = w / w.sum(1, keepdims=True)
    return ids, w, logits


def moe(X, router, gu, gus, dn, dns, top_k, renorm):
    """The layer's output (M, hidden), fp64."""
    X = np.asarray(X, np.float64)
    inter = dn.shape[2] * 2
    ids, w, _ = route(X, router, top_k, renorm)
    y = np.zeros_like(X)
    for e in np.unique(ids):
        tok, slot = np.nonzero(ids == e)
        gate_up = gemm(X[tok], gu[e], gus[e])
        g, u = gate_up[:, :inter], gate_up[:, inter:]
        h = g / (1 + np.exp(-g)) * u * w[tok, slot][:, None]
        y[tok] += gemm(h, dn[e], dns[e])
    return y
