"""MXFP4 on the GPU at the ends of its ranges: scale bytes from 0 to 254, subnormal
weights and activations, blocks that fp16 cannot hold in the experts' weights.

Bounds as in test_gpu_mx4.py. Where products or sums fall below fp32's normal
numbers a rounding is off by at most a step of its subnormals, 2^-149, instead of
2^-24 of the sum: (n + 16) (u S + 2^-149). The matrix instructions align products by
their operands' exponents and a subnormal operand has that of the smallest normal
number: there S counts the operand as that number.
Each test prints the case it runs (flushed) before touching the GPU.
"""
import numpy as np
import pytest
import torch

from oracle import mx4_oracle as mx
from test_gpu_mx4 import EPS, NAN, U, awq, host, moe_reference, moe_routings, say, store  # noqa: F401

pytestmark = pytest.mark.gpu


def dev(*arrays):
    return [torch.from_numpy(a).cuda() for a in arrays]


def far(Y, want, S, n):
    """Error over bound of an fp32 product."""
    return np.abs(host(Y).astype(np.float64) - want) / ((n + 16) * (U * S + 2.0 ** -149))


def product(X32, Wd):
    X = X32.astype(np.float64)
    return X @ Wd.T, np.abs(X) @ np.abs(Wd).T


# split, gemv with two and four waves a tile, mid of each size, tile
SHAPES = [(1, 130, 672), (9, 130, 672), (3, 20490, 96), (7, 10250, 160), (40, 130, 672), (300, 1030, 672),
          (1030, 4100, 352)]


# bytes of a third of the rows each, exponents of the activations
ENDS = [([(0, 1), (0, 19), (0, 120)], (0, 11)),            # subnormal weights under large activations
        ([(0, 19), (221, 252), (0, 252)], (-24, -9))]      # small to subnormal (in fp16) ones under all weights


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("end", range(2))
@pytest.mark.parametrize("M,out,n", SHAPES)
def test_gemm_ends_of_the_scale_range(awq, M, out, n, end, dt):
    say("ends", M, out, n, end, dt)
    r = np.random.default_rng(21)
    c = r.integers(0, 256, (out, n // 2)).astype(np.uint8)
    thirds, (x0, x1) = ENDS[end]
    lo, hi = np.array(thirds)[np.arange(out) % 3].T
    s = r.integers(lo[:, None], hi[:, None] + 1, (out, n // 32)).astype(np.uint8)
    X = r.standard_normal((M, n)) * np.exp2(r.integers(x0, x1 + 1, (1, n)))
    X[:, ::7] = 0.0
    Xd, X32 = store(X, dt)
    want, S = product(X32, mx.dequantize(c, s))
    Y = awq.mx4_gemm(Xd, *dev(c, s), y_f32=True)
    worst = far(Y, want, S, n)
    say("max err/bound", float(worst.max()))
    assert (S < 2.0 ** 127).all() and (worst <= 1).all()


@pytest.mark.parametrize("M,out,n", SHAPES)
def test_gemm_a4_ends_of_the_scale_range(awq, M, out, n):
    """Both operands under all bytes below 255: tiny activations meet the largest
    weights, values of 2^128 and more among them."""
    say("a4 ends", M, out, n)
    r = np.random.default_rng(22)
    xc, c = (r.integers(0, 256, (k, n // 2)).astype(np.uint8) for k in (M, out))
    lo, hi = np.array([[0, 20], [221, 255], [0, 255]])[np.arange(out) % 3].T
    s = r.integers(lo[:, None], hi[:, None], (out, n // 32)).astype(np.uint8)
    xs = r.integers(0, 110, (M, n // 32)).astype(np.uint8)
    Xq, Wd = mx.dequantize(xc, xs), mx.dequantize(c, s)
    want, S = Xq @ Wd.T, np.abs(Xq) @ np.abs(Wd).T
    worst = far(awq.mx4_gemm_a4(*dev(xc, xs, c, s), dtype=torch.float32), want, S, n)
    say("max err/bound", float(worst.max()))
    assert (S < 2.0 ** 127).all() and (worst <= 1).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,out,n", SHAPES)
def test_gemm_bytes_253_and_254(awq, M, out, n, dt):
    """Codes below 2^128 under them are as good as any; larger values make their own
    row infinite or NaN and no other."""
    say("253, 254", M, out, n, dt)
    r = np.random.default_rng(23)
    c = r.integers(0, 256, (out, n // 2)).astype(np.uint8)
    s = r.integers(100, 150, (out, n // 32)).astype(np.uint8)
    s[::5, 0], c[::5, :16] = 253, 0x5D                     # -3 and 3 at most
    s[1::5, 1], c[1::5, 16:32] = 254, 0x3A                 # 1.5 at most
    s[2::5, 2], c[2::5, 40] = 253, 0x60                    # 4: 2^128
    s[3::5, 0], c[3::5, 3] = 254, 0x04                     # 2: 2^128
    X = r.standard_normal((M, n))
    X[:, :96] *= 2.0 ** -14
    X[:, 96:] *= 2.0 ** -4
    X[:, 6], X[:, 80:82] = 2.0 ** -14, 2.0 ** -14
    Xd, X32 = store(X, dt)
    want, S = product(X32, mx.dequantize(c, s))
    Y = awq.mx4_gemm(Xd, *dev(c, s), y_f32=True)
    worst = far(Y, want, S, n)
    large = np.isin(np.arange(out) % 5, (2, 3))
    say("max err/bound", float(worst[:, ~large].max()))
    assert (S < 2.0 ** 127).all() and (worst[:, ~large] <= 1).all()
    assert not np.isfinite(host(Y)[:, large]).any()


@pytest.mark.parametrize("M,out,n", SHAPES)
@pytest.mark.parametrize("lo,hi", [(114, 140), (113, 140), (114, 141), (104, 140), (103, 140), (104, 141)])
def test_gemm_f16_at_its_borders(awq, M, out, n, lo, hi):
    """fp16 holds weights under bytes 104 to 140, from 114 on as normal numbers, and is
    used for these: the ends of both ranges in every row, and one step past either
    end; activations are subnormal but in the last columns."""
    say("fp16 borders", M, out, n, lo, hi)
    r = np.random.default_rng(24)
    c = r.integers(0, 256, (out, n // 2)).astype(np.uint8)
    s = r.integers(lo, hi + 1, (out, n // 32)).astype(np.uint8)
    s[:, 0], s[:, 1] = lo, hi
    X = r.standard_normal((M, n)) * np.exp2(r.integers(-22, -15, (M, n)))
    X[:, -32:] *= 2.0 ** 10
    Xd, X32 = store(X, "f16")
    assert (np.abs(X32[:, :-32]) < 2.0 ** -13).all() and (X32[:, :-32] != 0).any()
    want, S = product(X32, mx.dequantize(c, s))
    worst = far(awq.mx4_gemm(Xd, *dev(c, s), y_f32=True), want, S, n)
    say("max err/bound", float(worst.max()))
    assert (worst <= 1).all()


@pytest.mark.parametrize("dt,tiny,bits,lo,hi", [("f16", 2.0 ** -14, 10, 114, 140), ("bf16", 2.0 ** -126, 7, 190, 250)])
@pytest.mark.parametrize("M,out,n", SHAPES + [(2, 130, 64)])
def test_gemm_subnormal_activations(awq, M, out, n, dt, tiny, bits, lo, hi):
    """Nothing but subnormal activations, from the largest to the smallest. The first
    token has the smallest alone: in the first 32 columns, and in one behind them,
    where the weights of each row are larger by another power of two."""
    say("subnormal activations", M, out, n, dt)
    r = np.random.default_rng(27)
    c = r.integers(0, 256, (out, n // 2)).astype(np.uint8)
    s = r.integers(lo, hi + 1, (out, n // 32)).astype(np.uint8)
    s[:, 0], s[:, 1] = lo + np.arange(out) % (hi - lo + 1), hi
    c[:, :16], c[:, 16] = 0x33, 0x11                       # 1.5 in the first block, 0.5 in the column
    k = np.maximum(r.integers(1, 2 ** bits, (M, n)) >> r.integers(0, bits, (M, 1)), 1) * r.choice([-1, 1], (M, n))
    k[0] = 0
    k[0, :32] = k[0, 32] = 1
    Xd, X32 = store(k * (tiny * 2.0 ** -bits), dt)
    assert (X32 == k * (tiny * 2.0 ** -bits)).all()
    Wd = mx.dequantize(c, s)
    want, S = product(X32, Wd)
    raised = np.where(X32 == 0, 0.0, np.maximum(np.abs(X32), tiny)) @ np.abs(Wd).T
    Y = awq.mx4_gemm(Xd, *dev(c, s), y_f32=True)
    say("max err/bound", float(far(Y, want, raised, n).max()), "with S itself", float(far(Y, want, S, n).max()))
    assert (far(Y, want, raised, n) <= 1).all()


@pytest.mark.parametrize("M,out,n", SHAPES)
def test_gemm_f16_subnormal_weights(awq, M, out, n):
    """Rows whose weights would all be subnormal in fp16, down to its smallest, under
    large activations (the matrix instruction would lose bits of them); others of
    larger ones."""
    say("fp16 subnormal", M, out, n)
    r = np.random.default_rng(26)
    c = r.integers(0, 256, (out, n // 2)).astype(np.uint8)
    lo, hi = np.array([[104, 104], [104, 113], [112, 116]])[np.arange(out) % 3].T
    s = r.integers(lo[:, None], hi[:, None] + 1, (out, n // 32)).astype(np.uint8)
    X = r.standard_normal((M, n)) * np.exp2(r.integers(0, 12, (1, n)))
    Xd, X32 = store(X, "f16")
    want, S = product(X32, mx.dequantize(c, s))
    worst = far(awq.mx4_gemm(Xd, *dev(c, s), y_f32=True), want, S, n)
    say("max err/bound", float(worst.max()))
    assert (worst <= 1).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("wide", [False, True])
def test_gemm_activations_in_several_stretches(awq, dt, wide):
    """16 tokens of 4128 columns do not fit the LDS of the kernel for many rows at once."""
    M, out, n = 16, 20490, 4128
    say("stretches", M, out, n, dt, wide)
    r = np.random.default_rng(25)
    c = r.integers(0, 256, (out, n // 2)).astype(np.uint8)
    s = r.integers(115, 135, (out, n // 32)).astype(np.uint8)
    if wide:
        s[:, -1] = 80
    Xd, X32 = store(r.standard_normal((M, n)), dt)
    rows = np.r_[0:70, 10200:10270, 20420:20490]
    want, S = product(X32, mx.dequantize(c[rows], s[rows]))
    Y = awq.mx4_gemm(Xd, *dev(c, s), y_f32=True)
    worst = far(Y[:, torch.from_numpy(rows).cuda()], want, S, n)
    say("max err/bound", float(worst.max()))
    assert (worst <= 1).all() and bool(torch.isfinite(Y).all())


# ---- mixture of experts ---------------------------------------------------------


def experts(r, E, hidden, inter):
    """Random codes of every expert, values around 0.04 (codes and scales of gate/up and down)."""
    gc = r.integers(0, 256, (E, 2 * inter, hidden // 2)).astype(np.uint8)
    dc = r.integers(0, 256, (E, hidden, inter // 2)).astype(np.uint8)
    gs = r.integers(119, 122, (E, 2 * inter, hidden // 32)).astype(np.uint8)
    ds = r.integers(119, 122, (E, hidden, inter // 32)).astype(np.uint8)
    return gc, gs, dc, ds


def check_moe(awq, X, X32, R, R32, w, k, renorm, dt):
    refs = [moe_reference(X32, R32, *w, ids, renorm, dt) for ids in moe_routings(X32, R32, k)]
    wd = dev(*w)
    Y = awq.mx4_moe(X, R, *wd, k, renorm=renorm)
    got = Y.float().cpu().numpy()
    lost = np.isnan(refs[0][0]).any(1)                     # tokens that meet a NaN
    ratio = [(np.abs(got - want) / bound)[~lost].max(1) for want, bound in refs]
    worst = np.min(ratio, axis=0)
    say("max err/bound", float(worst.max()), "NaN tokens", int(lost.sum()))
    assert (worst <= 1).all()
    assert torch.equal(Y.nan_to_num(7.0), awq.mx4_moe(X, R, *wd, k, renorm=renorm).nan_to_num(7.0))
    return got, lost


# one wave a tile of `up` to eight, with and without a launch for the routing, tokens
# in one stretch of columns and in several
WIDE = [(3, 4, 2, 544, 64), (8, 1, 1, 4128, 96), (16, 2, 1, 4128, 96), (64, 2, 2, 2112, 1248), (64, 2, 2, 2112, 2464),
        (64, 2, 2, 2112, 3296)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,E,k,hidden,inter", WIDE)
def test_moe_blocks_that_fp16_cannot_hold(awq, M, E, k, hidden, inter, dt):
    """Gate and up blocks below fp16's range, under large activations, and above it,
    under tiny ones, that weigh as much as the others; far smaller ones, and blocks of zeros."""
    say("moe wide", M, E, k, hidden, inter, dt)
    r = np.random.default_rng(31)
    gc, gs, dc, ds = experts(r, E, hidden, inter)
    gs[:, :, 1], gs[:, 2::5, 2] = 120 - 13, 60
    gs[:, 1::7, 3] = 121 + 21
    gs[:, 3::5, 4], gc[:, 3::5, 64:80] = 0, 0
    ds[:, ::3, 0], ds[:, 1::3, -1] = 60, 150
    dc[:, 1::3, -16:] &= 0x99                              # 0.5 at most, under 2^23
    x = r.standard_normal((M, hidden))
    x[:, 32:64] *= 2.0 ** 13
    x[:, 96:128] *= 2.0 ** -18                             # subnormal in fp16
    X, X32 = store(x, dt)
    router = r.standard_normal((E, hidden)) * 1.5 / hidden ** 0.5
    router[:, 32:64] *= 2.0 ** -13
    R, R32 = store(router, dt)
    if dt == "f16":                                        # keep the results in its range
        ds[:, 1::3, -1] = 125
    check_moe(awq, X, X32, R, R32, (gc, gs, dc, ds), k, True, dt)


@pytest.mark.parametrize("M,E,k,hidden,inter", WIDE)
def test_moe_f16_subnormal_weights(awq, M, E, k, hidden, inter):
    """Gate and up weights that would be subnormal in fp16, under large activations."""
    say("moe subnormal", M, E, k, hidden, inter)
    r = np.random.default_rng(35)
    gc, gs, dc, ds = experts(r, E, hidden, inter)
    gs -= 13                                               # 106 to 108
    gs[:, ::5, 0] = 104
    X, X32 = store(r.standard_normal((M, hidden)) * 2.0 ** 13, "f16")
    R, R32 = store(r.standard_normal((E, hidden)) * 1.5 * 2.0 ** -13 / hidden ** 0.5, "f16")
    check_moe(awq, X, X32, R, R32, (gc, gs, dc, ds), k, True, "f16")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,E,k,hidden,inter", [(4, 8, 2, 544, 64), (30, 8, 2, 2112, 96)])
@pytest.mark.parametrize("wide", [False, True])
def test_moe_zero_and_nan_blocks(awq, M, E, k, hidden, inter, dt, wide):
    """Blocks of zeros everywhere and of NaN in two experts, with and without blocks that fp16 cannot hold."""
    say("moe zeros and NaN", M, E, k, hidden, inter, dt, wide)
    r = np.random.default_rng(32)
    gc, gs, dc, ds = experts(r, E, hidden, inter)
    gs[:, ::3, 0], gc[:, ::3, :16] = 0, 0
    ds[:, 1::3, 1], dc[:, 1::3, 16:32] = 0, 0
    gs[2, 5, -1], gc[2, 5, -16:] = 255, 0
    ds[6, :, 0], dc[6, :, :16] = 255, 0
    if wide:
        gs[:, ::4, 2] = 90
    X, X32 = store(r.standard_normal((M, hidden)), dt)
    R, R32 = store(r.standard_normal((E, hidden)) * 1.5 / hidden ** 0.5, dt)
    got, lost = check_moe(awq, X, X32, R, R32, (gc, gs, dc, ds), k, False, dt)
    assert lost.any() and not lost.all()
    assert np.isnan(got[lost]).all() and np.isfinite(got[~lost]).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,E,k,hidden,inter", [(1, 8, 8, 1024, 4096), (1, 8, 8, 2048, 4064), (2, 16, 4, 96, 4096),
                                                (4, 8, 2, 544, 4096)])
def test_moe_down_in_two_parts_for_few_tokens(awq, M, E, k, hidden, inter, dt):
    """64 units of 512 columns, as many as the narrow form takes: two blocks share them.
    All values are positive and the experts weigh alike, so that one unit is a 64th of
    the result and its bound a 400th."""
    say("moe two parts", M, E, k, hidden, inter, dt)
    r = np.random.default_rng(33)
    gc, gs, dc, ds = experts(r, E, hidden, inter)
    X, X32 = store(np.abs(r.standard_normal((M, hidden))) * 0.25, dt)
    R, R32 = store(r.standard_normal((E, hidden)) * 0.15 / hidden ** 0.5, dt)
    check_moe(awq, X, X32, R, R32, (gc & 0x77, gs, dc & 0x77, ds), k, True, dt)


def test_moe_byte_254_stays_with_its_tokens(awq):
    """A value of 2^128 and more counts as an infinity: the expert's tokens alone meet it."""
    say("moe 254")
    M, E, k, hidden, inter = 20, 6, 2, 96, 64
    r = np.random.default_rng(34)
    gc, gs, dc, ds = experts(r, E, hidden, inter)
    ds[3, :, 1], dc[3, :, 20] = 254, 0x77
    X, X32 = store(r.standard_normal((M, hidden)), "bf16")
    R, R32 = store(r.standard_normal((E, hidden)) * 1.5 / hidden ** 0.5, "bf16")
    ids = mx.route(X32, R32, k, True)[0]
    Y = awq.mx4_moe(X, R, *dev(gc, gs, dc, ds), k).float().cpu().numpy()
    hit = (ids == 3).any(1)
    assert hit.any() and not hit.all()
    assert not np.isfinite(Y[hit]).any() and np.isfinite(Y[~hit]).all()


@pytest.mark.parametrize("M", [3, 20])
def test_moe_nan_logit_without_renorm(awq, M):
    """A NaN among a token's logits: its softmax is NaN; renormalised weights leave it out."""
    say("moe nan logit", M)
    E, k, hidden, inter = 6, 2, 96, 64
    r = np.random.default_rng(36)
    w = dev(*experts(r, E, hidden, inter))
    X, X32 = store(r.standard_normal((M, hidden)), "f16")
    R, _ = store(r.standard_normal((E, hidden)) * 1.5 / hidden ** 0.5, "f16")
    R[4, 7] = NAN
    assert bool(awq.mx4_moe(X, R, *w, k, renorm=False).isnan().all())
    assert bool(awq.mx4_moe(X, R, *w, k, renorm=True).isfinite().all())


# ---- long operands ----------------------------------------------------------------


def codes_on_gpu(rows, n, seed, lo=119, hi=122):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randint(0, 256, (*rows, n // 2), dtype=torch.uint8, device="cuda", generator=g)
    return c, torch.randint(lo, hi, (*rows, n // 32), dtype=torch.uint8, device="cuda", generator=g)


@pytest.mark.parametrize("rows,n", [(262141, 32), (300001, 64), (65535 * 4 + 4, 288)])
def test_quantize_with_s_of_many_rows(awq, rows, n):
    """More rows than the grid has blocks of four for."""
    say("quantize many rows", rows, n)
    r = np.random.default_rng(41)
    W, W32 = store(r.standard_normal((rows, n)), "bf16")
    s = np.exp(r.uniform(-1.5, 1.5, n)).astype(np.float32)
    c, sc = awq.mx4_quantize(W, s=torch.from_numpy(s).cuda())
    pick = np.r_[0:2000, rows // 2:rows // 2 + 2000, rows - 2000:rows]
    want_c, want_s = mx.quantize(W32[pick], s)
    at = torch.from_numpy(pick).cuda()
    assert np.array_equal(host(c[at]), want_c) and np.array_equal(host(sc[at]), want_s)
    again, sc2 = awq.mx4_quantize(W * torch.from_numpy(s).cuda())      # fp32 products, no s
    assert torch.equal(c, again) and torch.equal(sc, sc2)


@pytest.mark.parametrize("with_s", [False, True])
def test_quantize_and_back_beyond_32_bits(awq, with_s):
    rows, n = 1040500, 4128                                # 2^32 values and more
    say("quantize long", rows, n, with_s)
    W = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    W.normal_(generator=torch.Generator(device="cuda").manual_seed(5))
    s = torch.rand(n, device="cuda") + 0.5 if with_s else None
    c, sc = awq.mx4_quantize(W, s=s)
    v = awq.mx4_dequantize(c, sc)
    for at in (slice(0, 50), slice(rows // 2 - 25, rows // 2 + 25), slice(rows - 50, rows)):
        want_c, want_s = mx.quantize(host(W[at].float()), None if s is None else host(s))
        assert np.array_equal(host(c[at]), want_c) and np.array_equal(host(sc[at]), want_s)
        assert np.array_equal(host(v[at].double()), mx.dequantize(want_c, want_s))


@pytest.mark.parametrize("M", [1, 5, 40])
def test_products_of_weights_beyond_32_bits(awq, M):
    out, n = 2080900, 4128                                 # 4.3 GB of codes
    say("long weights", M, out, n)
    c, s = codes_on_gpu((out,), n, 6)
    X, X32 = store(np.random.default_rng(42).standard_normal((M, n)), "bf16")
    xc, xs = awq.mx4_quantize(X)
    Y, Y4 = awq.mx4_gemm(X, c, s, y_f32=True), awq.mx4_gemm_a4(xc, xs, c, s, dtype=torch.float32)
    for at in (slice(0, 70), slice(out // 2, out // 2 + 70), slice(out - 70, out)):
        Wd = mx.dequantize(host(c[at]), host(s[at]))
        assert (far(Y[:, at], *product(X32, Wd), n) <= 1).all()
        assert (far(Y4[:, at], *product(mx.dequantize(host(xc), host(xs)), Wd), n) <= 1).all()


def test_products_of_activations_beyond_32_bits(awq):
    M, out, n = 2097120, 70, 4128                          # as many tokens as a call takes
    say("long activations", M, out, n)
    X = torch.empty(M, n, dtype=torch.bfloat16, device="cuda")
    X.normal_(generator=torch.Generator(device="cuda").manual_seed(7))
    c, s = codes_on_gpu((out,), n, 8)
    xc, xs = awq.mx4_quantize(X)
    Y, Y4 = awq.mx4_gemm(X, c, s, y_f32=True), awq.mx4_gemm_a4(xc, xs, c, s, dtype=torch.float32)
    Wd = mx.dequantize(host(c), host(s))
    for at in (slice(0, 150), slice(M // 2, M // 2 + 150), slice(M - 150, M)):
        assert (far(Y[at], *product(host(X[at].float()), Wd), n) <= 1).all()
        assert (far(Y4[at], *product(mx.dequantize(host(xc[at]), host(xs[at])), Wd), n) <= 1).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M", [1, 20])
def test_moe_weights_beyond_32_bits(awq, M, dt):
    """256 experts of 4.3 GB of gate and up codes; the last three alone have positive logits."""
    E, k, hidden, inter = 256, 2, 16416, 1024
    say("moe long", M, dt)
    r = np.random.default_rng(43)
    w = (*codes_on_gpu((E, 2 * inter), hidden, 9), *codes_on_gpu((E, hidden), inter, 10))
    X, X32 = store(np.abs(r.standard_normal((M, hidden))) * 0.25, dt)
    router = np.zeros((E, hidden))
    router[-3:] = np.abs(r.standard_normal((3, hidden))) * 4 / hidden
    R, R32 = store(router, dt)
    Y = awq.mx4_moe(X, R, *w, k).float().cpu().numpy()
    last = [host(t[-3:]) for t in w]
    refs = [moe_reference(X32, R32[-3:], *last, ids, True, dt) for ids in moe_routings(X32, R32[-3:], k)]
    worst = np.min([(np.abs(Y - want) / bound).max(1) for want, bound in refs], axis=0)
    say("max err/bound", float(worst.max()))
    assert (worst <= 1).all()
