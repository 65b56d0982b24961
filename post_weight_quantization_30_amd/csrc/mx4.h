// mx4.h -- device pieces shared by the MXFP4 kernels of libawq.so.
//
// An MXFP4 matrix (rows, in): every 32 consecutive columns of a row are a
// block of e2m1 codes (16 bytes, column 2i in the low half of byte i) and one
// e8m0 byte: value = e2m1(code) * 2^(byte - 127), byte 255 = NaN. A row has
// nb = in / 32 blocks, so its codes are 16 nb bytes and its scales nb bytes.
//
// The products below read both operands in whole blocks: in a 16-row matrix
// tile lane (r, c) = (lane % 16, lane / 16) holds block 4u + c of row r in
// step u. The sum over columns does not depend on the order in which both
// operands present them, so no operand is rearranged: a lane's block is one
// 16-byte load of codes and, for 16-bit activations, 64 contiguous bytes.
#pragma once

#include <type_traits>

#include "awq_internal.h"

namespace awq {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kMxBlock = 32;

// The activations of a product: 16-bit values, or MXFP4 like the weights.
struct Mx4Act {};

template <typename TX> struct XFrag {                 // one block of one row, one lane
    typename Vec8<TX>::type v[4];
};
template <> struct XFrag<Mx4Act> {
    u32x4 q;
    uint32_t s;
};

// 2^(byte - 127) as the conversion instructions take it: they read the
// exponent field only, 0 as 2^-127 and 255 as NaN.
__device__ __forceinline__ float mx4_scale(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

// The eight codes of one word as bf16 (exact for every scale: three
// significand bits at most, and bf16 reaches 2^-133).
__device__ __forceinline__ bf16x8 mx4_to_bf16(uint32_t w, float s)
{
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The eight codes of one word as fp16: exact where mx4_fits_f16(byte).
__device__ __forceinline__ f16x8 mx4_to_f16(uint32_t w, float s)
{
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 0);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 1);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 2);
    const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 3);
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// fp16 holds 0.5 * 2^E .. 6 * 2^E as normal numbers for E in [-13, 13].
__device__ __forceinline__ bool mx4_fits_f16(uint32_t byte) { return byte - 114u <= 26u; }

// fp16 values as the exact sum of two bf16 parts (11 significand bits = 8 + 3;
// an infinity stays in the first part).
__device__ __forceinline__ void split_f16(const f16x8 &x, bf16x8 &hi, bf16x8 &lo)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float f = static_cast<float>(x[i]);
        const float h = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, f) & 0xFFFF0000u);
        hi[i] = static_cast<bf16>(h);
        lo[i] = static_cast<bf16>(f == h ? 0.0f : f - h);
    }
}

__device__ __forceinline__ f32x4 mx4_mfma(const bf16x8 &a, const bf16x8 &b, const f32x4 &c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mx4_mfma(const f16x8 &a, const f16x8 &b, const f32x4 &c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
// Both operands MXFP4: 128 columns, a lane's block and its scale byte (the
// low byte of each scale register).
__device__ __forceinline__ f32x4 mx4_mfma(const u32x4 &a, uint32_t sa, const u32x4 &b, uint32_t sb, const f32x4 &c)
{
    const i32x8 a8 = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 b8 = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// What one wave loads at a time: U steps of 128 columns of 16 NT weight rows
// and 16 MT activation rows.
template <typename TX, int MT, int NT, int U> struct Mx4Item {
    u32x4 w[NT][U];
    uint32_t ws[NT][U];
    XFrag<TX> x[MT][U];
};

// A lane's rows: pointers to the starts of their codes, scales and activations.
template <typename TX, int MT, int NT> struct Mx4Rows {
    const uint8_t *w[NT], *ws[NT];
    const void *x[MT];
    const uint8_t *xs[MT];         // activation scales (MXFP4 activations only)
};

// Loads the item whose first block is b0. Blocks past the row's end load its
// last block: compute drops them.
template <typename TX, int MT, int NT, int U>
__device__ __forceinline__ void mx4_load(Mx4Item<TX, MT, NT, U> &it, const Mx4Rows<TX, MT, NT> &rows, int b0, int nb,
                                         int c)
{
#pragma unroll
    for (int u = 0; u < U; ++u) {
        int b = b0 + 4 * u + c;
        b = b < nb ? b : nb - 1;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            it.w[nt][u] = *reinterpret_cast<const u32x4 *>(rows.w[nt] + (int64_t)b * 16);
            it.ws[nt][u] = rows.ws[nt][b];
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            if constexpr (std::is_same<TX, Mx4Act>::value) {
                it.x[mt][u].q = *reinterpret_cast<const u32x4 *>((const uint8_t *)rows.x[mt] + (int64_t)b * 16);
                it.x[mt][u].s = rows.xs[mt][b];
            } else {
                const TX *p = (const TX *)rows.x[mt] + (int64_t)b * 32;
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    it.x[mt][u].v[s] = load8(p + 8 * s);
            }
        }
    }
}

// acc += the item's products. A lane whose block lies past the row's end
// multiplies zeros (its weights are then finite: scale 1). WIDE is for fp16
// activations under scales that fp16 cannot hold: weights in bf16, activations
// as two bf16 parts. The plain form reports such scales in `bad`.
template <bool WIDE, typename TX, int MT, int NT, int U>
__device__ __forceinline__ void mx4_compute(Mx4Item<TX, MT, NT, U> &it, f32x4 (&acc)[MT][NT], int b0, int nb, int c,
                                            bool &bad)
{
    if (b0 + 4 * U > nb) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (b0 + 4 * u + c < nb)
                continue;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                it.ws[nt][u] = 127;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if constexpr (std::is_same<TX, Mx4Act>::value) {
                    it.x[mt][u].q = u32x4{0, 0, 0, 0};
                    it.x[mt][u].s = 127;
                } else {
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        it.x[mt][u].v[s] = typename Vec8<TX>::type{};
                }
            }
        }
    }
    if constexpr (std::is_same<TX, Mx4Act>::value) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    acc[mt][nt] = mx4_mfma(it.x[mt][u].q, it.x[mt][u].s, it.w[nt][u], it.ws[nt][u], acc[mt][nt]);
    } else if constexpr (!WIDE) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float s = mx4_scale(it.ws[nt][u]);
                if constexpr (std::is_same<TX, f16>::value)
                    bad = bad || !mx4_fits_f16(it.ws[nt][u]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    typename Vec8<TX>::type w;
                    if constexpr (std::is_same<TX, f16>::value)
                        w = mx4_to_f16(it.w[nt][u][k], s);
                    else
                        w = mx4_to_bf16(it.w[nt][u][k], s);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        acc[mt][nt] = mx4_mfma(it.x[mt][u].v[k], w, acc[mt][nt]);
                }
            }
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    __builtin_amdgcn_sched_barrier(0);       // one split at a time: registers
                    bf16x8 hi, lo;
                    split_f16(it.x[mt][u].v[k], hi, lo);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const bf16x8 w = mx4_to_bf16(it.w[nt][u][k], mx4_scale(it.ws[nt][u]));
                        acc[mt][nt] = mx4_mfma(hi, w, acc[mt][nt]);
                        acc[mt][nt] = mx4_mfma(lo, w, acc[mt][nt]);
                    }
                }
    }
}

template <int MT, int NT> __device__ __forceinline__ void mx4_zero(f32x4 (&acc)[MT][NT])
{
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            acc[mt][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// One wave's share of a contraction: the items that begin at blocks first,
// first + step, ... of the rows, each in flight while the one before it is
// multiplied. fp16 activations: where a scale turns out not to fit, all of it
// once more in the wide form (real weights never need it, so the hot loop
// carries no branch and no registers for it).
template <typename TX, int MT, int NT, int U>
__device__ __forceinline__ void mx4_wave(const Mx4Rows<TX, MT, NT> &rows, f32x4 (&acc)[MT][NT], int first, int step,
                                         int nb, int c)
{
    mx4_zero(acc);
    if (first >= nb)
        return;
    Mx4Item<TX, MT, NT, U> a, b;
    bool bad = false;
    int i = first;
    mx4_load(a, rows, i, nb, c);
    while (true) {
        if (i + step < nb)
            mx4_load(b, rows, i + step, nb, c);
        mx4_compute<false>(a, acc, i, nb, c, bad);
        i += step;
        if (i >= nb)
            break;
        if (i + step < nb)
            mx4_load(a, rows, i + step, nb, c);
        mx4_compute<false>(b, acc, i, nb, c, bad);
        i += step;
        if (i >= nb)
            break;
    }
    if constexpr (std::is_same<TX, f16>::value) {
        if (__any(bad)) {
            mx4_zero(acc);
#pragma unroll 1
            for (i = first; i < nb; i += step) {
                mx4_load(a, rows, i, nb, c);
                mx4_compute<true>(a, acc, i, nb, c, bad);
            }
        }
    }
}

}  // namespace awq
