// mx8.h -- device pieces shared by the MXFP8 kernels of libawq.so.
//
// An MXFP8 matrix (rows, in): every 32 consecutive columns of a row are a block
// of e4m3 codes (32 bytes) and one e8m0 byte: value = e4m3(code) * 2^(byte - 127),
// byte 255 = NaN. A row has nb = in / 32 blocks, so its codes are 32 nb bytes and
// its scales nb bytes.
//
// The scaled matrix instructions take an e4m3 operand in two halves of 16 bytes:
// lane group c of a 16-row tile (128 columns a step) holds columns 16 c ... of the
// first 64 and 16 c ... of the second 64, lane group h of a 32-row tile (64
// columns) columns 16 h ... of either half of 32, where an e2m1 operand is the one
// block c or h (found by one-hot operands). The scale in lane group c is that of
// block c for both.
#pragma once

#include "mx4.h"

namespace awq {

// A's exponent field f and fraction give the byte max(f - 8 + (fraction > 0.75), 0):
// the least E with A 2^-E <= 448 = 1.75 * 2^8. The field 255 is an infinity or NaN.
__device__ __forceinline__ uint32_t mx8_byte(uint32_t a)
{
    const uint32_t field = (a + 0x1FFFFFu) >> 23;
    return a >= 0x7F800000u ? 255u : field > 8 ? field - 8 : 0;
}

// 2^(byte - 127) of any byte below 255 as a factor (0: a subnormal).
__device__ __forceinline__ float mx8_factor(uint32_t byte)
{
    return __builtin_bit_cast(float, byte == 0 ? 0x00400000u : byte << 23);
}

// Four values as e4m3 codes under 2^(byte - 127) (nearest even; none beyond 448).
__device__ __forceinline__ uint32_t mx8_codes4(float a, float b, float c, float d, float s)
{
    typedef short i16x2 __attribute__((ext_vector_type(2)));
    i16x2 q = {0, 0};
    q = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(q, a, b, s, false);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(q, c, d, s, true);
    return __builtin_bit_cast(uint32_t, q);
}

__device__ __forceinline__ uint32_t mx8_abs(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Eight values of a thread, four neighbouring lanes one block: chunk of 8 codes,
// one scale byte from the first of the four lanes.
__device__ __forceinline__ void mx8_quantize8(const float (&v)[8], uint8_t *codes, uint8_t *scales, int64_t chunk)
{
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        a = umax(a, mx8_abs(v[i]));
#pragma unroll
    for (int off = 1; off <= 2; off <<= 1)
        a = umax(a, (uint32_t)__shfl_xor((int)a, off));
    const uint32_t byte = mx8_byte(a);
    u32x2 q = {0, 0};
    if (byte != 255) {
        const float s = mx8_factor(byte);
        q = u32x2{mx8_codes4(v[0], v[1], v[2], v[3], s), mx8_codes4(v[4], v[5], v[6], v[7], s)};
    }
    reinterpret_cast<u32x2 *>(codes)[chunk] = q;
    if ((chunk & 3) == 0)
        scales[chunk >> 2] = (uint8_t)byte;
}

// Scaled products with e4m3 activations `x` and e2m1 weights `w`; byte S of the
// scale registers. 16 tokens x 16 rows over 128 columns: acc[i] of lane (r, c) is
// token 4 c + i, row r.
template <int S>
__device__ __forceinline__ f32x4 mfma16_a8(const i32x8 &x, uint32_t sx, const u32x4 &w, uint32_t sw, const f32x4 &acc)
{
    const i32x8 w8 = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, w8, acc, 0, 4, S, (int)sx, S, (int)sw);
}

// Of four codes those from 2 on, zeros in the others' places: bit 6 is the upper one of the
// exponent's four.
__device__ __forceinline__ uint32_t mx8_upper(uint32_t v)
{
    const uint32_t m = v >> 6 & 0x01010101u;
    return v & ((m << 8) - m);
}

// The two parts of an operand whose products of eight columns all fit (see mx8_stream.h).
__device__ __forceinline__ void mx8_parts(const i32x8 &x, i32x8 &high, i32x8 &low)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        high[i] = (int)mx8_upper((uint32_t)x[i]);
        low[i] = x[i] ^ high[i];
    }
}

__device__ __forceinline__ i32x8 join(const u32x4 &a, const u32x4 &b)
{
    return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

}  // namespace awq
