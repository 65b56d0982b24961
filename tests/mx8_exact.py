"""Operands whose products any order of fp32 sums adds up exactly, and what they pin.

Activations: codes of +-2^-6, 2^-5, 2^-4 under 2^-1 or 1 and, in `pairs` pairs of a row, a
large code (256 to 448) and its negative in two eights (columns 8 i ... 8 i + 7) of one block;
weights: any e2m1 code under 2^-1 or 1, 6 at columns 8 i. Every product is a multiple of
2^-9 (2^-6 * 0.5 under 2^-2) and, as `sums` asserts, all of a sum's magnitudes together are below
2^15: every partial sum has at most 24 bits, so an fp32 sum is the exact one. The large
products cancel, but products of eight columns that are cut off 2^13 below the largest of
them lose the small ones beside it (2^-3 and below beside 448 * 6): sums go wrong by about
their own size, unless the parts are multiplied apart.

Experts on such tokens: gate and up are exact, h = silu(gate) up is off by less than 16 u |h| (exp, sum,
division, product) and its 8-bit value therefore the oracle's, or next to a border one of two.
`chosen` makes a down product that shows h's values themselves.
"""
import numpy as np

from oracle import mx4_oracle as mx4, mx8_oracle as mx

U = 2.0 ** -24
EPS = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def tokens(r, M, n, pairs=5):
    """(codes, scales) of M rows."""
    small = mx.e4m3_codes(np.exp2(r.integers(-6, -3, (M, n)).astype(float)))
    codes = (small + 128 * r.integers(0, 2, (M, n))).astype(np.uint8)
    large = mx.e4m3_codes(np.array([256.0, 288.0, 320.0, 352.0, 384.0, 416.0, 448.0]))
    for m in range(M):
        for b in r.permutation(n // 32)[:pairs]:
            i, j = r.permutation(4)[:2]
            c = r.choice(large)
            codes[m, 32 * b + 8 * i], codes[m, 32 * b + 8 * j] = c, c + 128
    return codes, r.integers(126, 128, (M, n // 32)).astype(np.uint8)


def rows(r, shape, n):
    """(codes, scales) of weights (*shape, n)."""
    codes = r.integers(0, 256, (*shape, n // 2)).astype(np.uint8)
    codes[..., ::4] = codes[..., ::4] & 0xF0 | 7
    return codes, r.integers(126, 128, (*shape, n // 32)).astype(np.uint8)


def sums(x, w):
    """x w^T of values that meet the conditions."""
    for a, step in ((x, 2.0 ** -7), (w, 2.0 ** -2)):
        assert np.array_equal(a, np.rint(a / step) * step)
    assert (np.abs(x) @ np.abs(w).T).max() < 2.0 ** 15
    return x @ w.T


def chosen(r, E, H, I):
    """A down product (codes, scales) with one 1 in every row, and the columns (E, H) that it
    chooses: the first and last blocks' among them."""
    at = np.empty((E, H), int)
    for e in range(E):
        order = np.r_[0, I - 1, 31, I - 32, r.permutation(I)]
        order = order[np.sort(np.unique(order, return_index=True)[1])]         # each once, in this order
        at[e] = r.permutation(np.resize(order, H))
    codes = np.zeros((E, H, I // 2), np.uint8)
    np.put_along_axis(codes, at[..., None] // 2, (2 << 4 * (at[..., None] % 2)).astype(np.uint8), 2)
    return codes, np.full((E, H, I // 32), 127, np.uint8), at


def routing(r, M, E, k):
    return np.argsort(r.random((M, E)) + 0.3 * r.random(E), 1)[:, :k].astype(np.int32)


def rounded(h):
    """(values, scale bytes) of h (rows, inter) as MXFP8."""
    c, s = mx.quantize(h.astype(np.float32))
    return mx.dequantize(c, s), s


def hidden_rows(gate, up):
    """(q, dq, bytes): the 8-bit values of h, how far another that rounding allows may lie
    (0 where none does), the larger of the allowed scale bytes."""
    with np.errstate(over="ignore"):
        h = gate / (1 + np.exp(-gate)) * up
    q, s = rounded(h)
    ends = [rounded(h * (1 + sign * 16 * U)) for sign in (-1, 1)]
    # only the largest or only another value of the block may move
    ends += [(scaled(h * (1 + sign * 16 * U), b), b) for sign in (-1, 1) for b in (ends[0][1], ends[1][1])]
    return q, np.max([np.abs(v - q) for v, _ in ends], 0), np.max([b for _, b in ends], 0)


def scaled(h, byte):
    """h rounded to e4m3 under given scale bytes (cut off at 448)."""
    f = np.repeat(np.ldexp(1.0, byte.astype(int) - 127), 32, axis=-1)
    return mx.VALUES[mx.e4m3_codes(np.clip(h / f, -448, 448))] * f


def exponents(v, scale, least):
    """floor(log2 |v|), of values below `least` times their scale that of the latter."""
    f = np.repeat(np.ldexp(least, scale.astype(int) - 127), 32, axis=-1)
    return np.frexp(np.maximum(np.abs(v), f))[1] - 1


def of_eights(e):
    return e.reshape(*e.shape[:-1], -1, 8)


def cut(q, qs, w, ws):
    """The most that cutting products off costs the sums q w^T: 2^-13 P for every product of an
    eight with bits below that, P the power of two of the largest product by its operands'
    exponents (those below 2^-6 and 1 of their scales count as that)."""
    ew, nw = of_eights(exponents(w, ws, 1.0)), of_eights(w != 0)
    out = np.zeros((len(q), len(w)))
    for m, (ex, nx) in enumerate(zip(of_eights(exponents(q, qs, 2.0 ** -6)), of_eights(q != 0))):
        e = ex + ew                                     # (rows, eights, 8); 3 and 1 fraction bits
        top = e.max(-1, keepdims=True)
        lost = nx & nw & (e - 4 < top - 13)
        out[m] = (lost.sum(-1) * np.ldexp(1.0, top[..., 0] - 13)).sum(-1)
    return out


def cut_chosen(q, qs):
    """The same of a single value q times 1 beside zeros."""
    e = of_eights(exponents(q, qs, 2.0 ** -6))
    top = e.max(-1, keepdims=True)
    return np.where(of_eights(q != 0) & (e - 3 < top - 13), np.ldexp(1.0, top - 13), 0.0).reshape(q.shape)


class Layer:
    """A layer of experts, its tokens and routing, and the exact gate and up of every pair.
    show: down chooses single values of h, and of each token one choice has the weight 1."""

    def __init__(self, M, E, k, H, I, seed, show):
        r = np.random.default_rng(seed)
        self.shape, self.show = (M, E, k, H, I), show
        self.xc, self.xs = tokens(r, M, H)
        self.gu, self.gus = rows(r, (E, 2 * I), H)
        self.ids = routing(r, M, E, k)
        if show:
            self.dn, self.dns, self.at = chosen(r, E, H, I)
            self.w = np.zeros((M, k), np.float32)
            self.w[np.arange(M), r.integers(0, k, M)] = 1
        else:
            self.dn = r.integers(0, 256, (E, H, I // 2)).astype(np.uint8)
            self.dns = r.integers(121, 124, (E, H, I // 32)).astype(np.uint8)
            self.w = r.uniform(0.1, 1.0, (M, k)).astype(np.float32)

    def arrays(self):
        return self.xc, self.xs, self.ids, self.w, self.gu, self.gus, self.dn, self.dns

    def experts(self, some):
        """(expert, places in `some`, choices) of the pairs of the tokens `some` that count."""
        for e in range(self.shape[1]):
            t, j = np.nonzero((self.ids[some] == e) & (self.w[some] != 0))
            if len(t):
                yield e, t, j

    def gate_up(self, e, some):
        both = sums(mx.dequantize(self.xc[some], self.xs[some]), mx4.dequantize(self.gu[e], self.gus[e]))
        return both[:, :self.shape[4]], both[:, self.shape[4]:]

    def check(self, Y, dt, some=None):
        """Y (tokens, hidden), fp64, against the definition: the largest error over its bound. With
        `show` the values of h, as they are (0 off) in fp32; else sums of fp32, what the cut costs
        where Y has 16 bits, and Y's rounding."""
        M, E, k, H, I = self.shape
        some = np.arange(M) if some is None else np.asarray(some)
        want, bound, terms = (np.zeros((len(some), H)) for _ in range(3))
        for e, t, j in self.experts(some):
            q, dq, byte = hidden_rows(*self.gate_up(e, some[t]))
            if self.show:
                want[t] += q[:, self.at[e]]
                bound[t] += dq[:, self.at[e]]
                if dt != "f32":
                    bound[t] += cut_chosen(q + np.where(q < 0, -dq, dq), byte)[:, self.at[e]]
                continue
            Wd, p = mx4.dequantize(self.dn[e], self.dns[e]), self.w[some[t], j].astype(np.float64)[:, None]
            size = (np.abs(q) + dq) @ np.abs(Wd).T
            want[t] += p * (q @ Wd.T)
            terms[t] += p * size
            bound[t] += p * (dq @ np.abs(Wd).T + (I + 16) * (U * size + 2.0 ** -149))
            if dt != "f32":
                bound[t] += p * cut(q + np.where(q < 0, -dq, dq), byte, Wd, self.dns[e])
        bound += (k + 2) * U * terms
        if dt != "f32":
            bound = bound * (1 + EPS[dt]) + EPS[dt] * np.abs(want) + (2.0 ** -25 if dt == "f16" else 0.0)
        err = np.abs(np.asarray(Y, np.float64)[some] - want)
        return float((err / np.maximum(bound, 1e-300)).max())


LAYERS = [  # M, experts, k, hidden, inter: unsorted pairs; streams; large tiles, whole, half, and both
    (1, 8, 2, 256, 512), (2, 64, 8, 2048, 96), (4, 6, 2, 4096, 160), (3, 9, 5, 96, 320), (4, 3, 2, 96, 4128),
    (5, 3, 2, 96, 4128), (33, 48, 4, 1056, 352), (17, 5, 1, 640, 1152), (60, 8, 2, 4096, 96), (9, 6, 2, 32, 64),
    (64, 2, 1, 128, 64), (100, 3, 2, 4096, 224), (700, 4, 2, 1120, 416), (385, 1, 1, 96, 2592), (513, 9, 4, 96, 608)]


def some_tokens(M, n=12):
    return np.unique(np.r_[0, M // 2, M - 1, np.random.default_rng(M).integers(0, M, n)])
