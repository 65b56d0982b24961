// mx4.h -- device pieces shared by the MXFP4 kernels of libawq.so.
//
// An MXFP4 matrix (rows, in): every 32 consecutive columns of a row are a
// block of e2m1 codes (16 bytes, column 2i in the low half of byte i) and one
// e8m0 byte: value = e2m1(code) * 2^(byte - 127), byte 255 = NaN. A row has
// nb = in / 32 blocks, so its codes are 16 nb bytes and its scales nb bytes.
//
// The products read weights in whole blocks: in a 16-row matrix tile lane
// (r, c) = (lane % 16, lane / 16) loads block 4u + c of row r, 16 bytes. The
// matrix step for 32 columns wants columns 8c ... 8c + 7 of one block in lane
// c: the four words of four lanes are transposed (transpose4), so that step s
// is block 4u + s for weights and 16-bit activations alike, and a load of
// activations is 64 contiguous bytes a row. With the words left where they
// are, lane c would want block 4u + c of the activations: a load would touch
// twice the cache lines for 16 bytes each, which held a decode product of 16
// tokens at a third of the speed.
#pragma once

#include <type_traits>

#include "awq_internal.h"

namespace awq {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kMxBlock = 32;

// 2^(byte - 127) as the conversion instructions take it: they read the
// exponent field only, 0 as 2^-127 and 255 as NaN.
__device__ __forceinline__ float mx4_scale(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

// The eight codes of one word as bf16: exact below 2^128 (two significand bits,
// and bf16 reaches down to 2^-133; the matrix instructions take its subnormals).
// 4 and 6 under byte 253 and 2 to 6 under byte 254 become infinities.
__device__ __forceinline__ bf16x8 mx4_to_bf16(uint32_t w, float s)
{
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The eight codes of one word as fp16: exact where F16Range holds the block to fit.
__device__ __forceinline__ f16x8 mx4_to_f16(uint32_t w, float s)
{
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 0);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 1);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 2);
    const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 3);
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// fp16 holds 0.5 * 2^E .. 6 * 2^E as normal numbers for E in [-13, 13]: whether
// the blocks seen are such, by the largest byte - 114 of those that hold anything
// but zeros. (A block of zeros has byte 0, a block of NaN 255, and the conversion
// makes NaN of that whatever the codes.) Subnormal fp16 weights, exact down to
// E = -23, would not do: the matrix instruction aligns their products as those of
// 2^-14, and 3 tokens x 20490 rows of 96 columns under E = -23 to -14 came out
// wrong by 270 * 2^-24 of sum |x w|.
struct F16Range {
    uint32_t worst = 0;
    __device__ __forceinline__ void see(const u32x4 &block, uint32_t byte)
    {
        const uint32_t over = ((block[0] | block[1] | block[2] | block[3]) & 0x77777777u) ? byte - 114u : 0;
        worst = worst > over ? worst : over;
    }
    __device__ __forceinline__ bool exceeded() const { return worst > 26; }
};

// fp16 values as the exact sum of two bf16 parts (11 significand bits = 8 + 3;
// an infinity stays in the first part). A weight of 2^128 or more is an infinity
// here: with a second part of zero it gives NaN.
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

// Word s of lane c <-> word c of lane s, for the four lanes (r, 0..3) of every
// row: two swaps of half waves, two of quarter waves.
__device__ __forceinline__ void transpose4(u32x4 &w)
{
    typedef uint32_t pair __attribute__((ext_vector_type(2)));
    const pair a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    const pair b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    const pair c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const pair d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    w = u32x4{c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ f32x4 mx4_mfma(const bf16x8 &a, const bf16x8 &b, const f32x4 &c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mx4_mfma(const f16x8 &a, const f16x8 &b, const f32x4 &c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
// The scale bytes of blocks b .. b + 3 of a row (127 for those past its end).
__device__ __forceinline__ uint32_t mx4_scales4(const uint8_t *row, int b, int nb)
{
    uint32_t v;
    if (b + 4 <= nb) {
        __builtin_memcpy(&v, row + b, 4);              // at any alignment
    } else {
        v = 0x7F7F7F7Fu;
        for (int i = 0; b + i < nb; ++i)
            v = (v & ~(0xFFu << (8 * i))) | (uint32_t)row[b + i] << (8 * i);
    }
    return v;
}

template <int MT, int NT> __device__ __forceinline__ void mx4_zero(f32x4 (&acc)[MT][NT])
{
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            acc[mt][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// ---------------------------------------------------------------------------
// The direct form, for few rows: a wave's share of a contraction, operands
// straight from memory to registers. A lane's rows: the starts of its codes,
// scales and activations.
template <typename TX> struct Mx4Rows {
    const uint8_t *w, *ws;
    const TX *x;
};
template <typename TX, int U> struct Mx4Item {         // U steps of 128 columns of 16 rows and 16 tokens
    u32x4 w[U];
    uint32_t ws[U];                                    // the four blocks' scale bytes
    typename Vec8<TX>::type x[U][4];
};

// Loads the item whose first block is b0. Blocks past the row's end load its
// last block: compute leaves them out.
template <typename TX, int U>
__device__ __forceinline__ void mx4_load(Mx4Item<TX, U> &it, const Mx4Rows<TX> &rows, int b0, int nb, int c)
{
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int b4 = b0 + 4 * u, b = b4 + c < nb ? b4 + c : nb - 1;
        it.w[u] = *reinterpret_cast<const u32x4 *>(rows.w + (int64_t)b * 16);
        it.ws[u] = mx4_scales4(rows.ws, b4, nb);
#pragma unroll
        for (int s = 0; s < 4; ++s)
            it.x[u][s] = load8(rows.x + (int64_t)(b4 + s < nb ? b4 + s : nb - 1) * 32 + 8 * c);
    }
}

// acc += the item's products. WIDE is for fp16 activations under scales that
// fp16 cannot hold: weights in bf16, activations as two bf16 parts. The plain
// form notes the scales it meets in `range`.
template <bool WIDE, typename TX, int U>
__device__ __forceinline__ void mx4_compute(Mx4Item<TX, U> &it, f32x4 &acc, int b0, int nb, int c, F16Range &range)
{
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if constexpr (std::is_same<TX, f16>::value && !WIDE)
            range.see(it.w[u], it.ws[u] >> (8 * c) & 0xFFu);
        transpose4(it.w[u]);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (b0 + 4 * u + s >= nb)
                break;
            const uint32_t byte = it.ws[u] >> (8 * s) & 0xFFu;
            if constexpr (WIDE) {
                __builtin_amdgcn_sched_barrier(0);           // one split at a time: registers
                bf16x8 hi, lo;
                split_f16(it.x[u][s], hi, lo);
                const bf16x8 w = mx4_to_bf16(it.w[u][s], mx4_scale(byte));
                acc = mx4_mfma(hi, w, acc);
                acc = mx4_mfma(lo, w, acc);
            } else if constexpr (std::is_same<TX, f16>::value) {
                acc = mx4_mfma(it.x[u][s], mx4_to_f16(it.w[u][s], mx4_scale(byte)), acc);
            } else {
                acc = mx4_mfma(it.x[u][s], mx4_to_bf16(it.w[u][s], mx4_scale(byte)), acc);
            }
        }
    }
}

// The items that begin at blocks first, first + step, ... of the rows, each in
// flight while the one before it is multiplied. fp16 activations: where a scale
// turns out not to fit, all of it once more in the wide form, so that the hot
// loop carries no branch for it.
template <int U, typename TX>
__device__ __forceinline__ void mx4_wave(const Mx4Rows<TX> &rows, f32x4 &acc, int first, int step, int nb, int c)
{
    acc = f32x4{0.f, 0.f, 0.f, 0.f};
    if (first >= nb)
        return;
    Mx4Item<TX, U> a, b;
    F16Range range;
    int i = first;
    mx4_load(a, rows, i, nb, c);
    while (true) {
        if (i + step < nb)
            mx4_load(b, rows, i + step, nb, c);
        mx4_compute<false>(a, acc, i, nb, c, range);
        i += step;
        if (i >= nb)
            break;
        if (i + step < nb)
            mx4_load(a, rows, i + step, nb, c);
        mx4_compute<false>(b, acc, i, nb, c, range);
        i += step;
        if (i >= nb)
            break;
    }
    if constexpr (std::is_same<TX, f16>::value) {
        if (__any(range.exceeded())) {
            acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
            for (i = first; i < nb; i += step) {
                mx4_load(a, rows, i, nb, c);
                mx4_compute<true>(a, acc, i, nb, c, range);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The streaming form, for few tokens: the activations of a stretch of columns
// lie in LDS and every wave runs its own stream of weights through registers.
// An item is 512 columns of 16 NT rows: four 16-byte loads of codes and one of
// scales a lane and row tile.
constexpr int kStreamBlocks = 16;              // blocks of 32 columns in an item

template <int NT> struct StreamItem {
    u32x4 w[NT][4], s[NT];
};

// A wave's 16 NT rows: scalar bases of the row tiles and one offset a lane (in
// is at most 2^23 columns: 16 rows stay below 2^32 bytes).
template <int NT> struct StreamRows {
    const uint8_t *w[NT], *s[NT];
    uint32_t wo, so;
    // row r of the tile (or any other row of it), lane quarter c
    __device__ __forceinline__ void lane(uint32_t row, int c, int nb)
    {
        so = row * (uint32_t)nb;
        wo = so * 16 + c * 16;
    }
};

// Words u of the item that begins at block b0; blocks past the rows' end load
// the last one.
template <int NT>
__device__ __forceinline__ void stream_load_w(u32x4 (&w)[NT][4], int u, const StreamRows<NT> &rows, int b0, int nb,
                                              int c)
{
    const int b4 = b0 + 4 * u, back = b4 + c < nb ? 0 : b4 + c - (nb - 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const uint8_t *const p = rows.w[nt] + (int64_t)b4 * 16;
        if (b4 + 4 <= nb)
            w[nt][u] = *reinterpret_cast<const u32x4 *>(p + rows.wo);
        else
            w[nt][u] = *reinterpret_cast<const u32x4 *>(p - back * 16 + (int64_t)rows.wo);
    }
}

template <int NT>
__device__ __forceinline__ void stream_load_s(u32x4 (&s)[NT], const StreamRows<NT> &rows, int b0, int nb)
{
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        if (b0 + kStreamBlocks <= nb)
            __builtin_memcpy(&s[nt], rows.s[nt] + b0 + rows.so, 16);
        else
#pragma unroll
            for (int u = 0; u < 4; ++u)
                s[nt][u] = mx4_scales4(rows.s[nt] + rows.so, b0 + 4 * u, nb);
}

template <int NT>
__device__ __forceinline__ void stream_load(StreamItem<NT> &it, const StreamRows<NT> &rows, int b0, int nb, int c)
{
    stream_load_s(it.s, rows, b0, nb);
#pragma unroll
    for (int u = 0; u < 4; ++u)
        stream_load_w(it.w, u, rows, b0, nb, c);
}

// acc += the item's products; x[mt] is the lane's activation row in LDS at the
// item's first column, plus 8 c columns. `blocks` of the item exist. ROLL: the
// item of `next` at block next_b0 takes its place, load by load as registers are
// used up (next_b0 < 0: none). One register set then keeps a wave's stream
// going; with two row tiles a wave two sets that change places are faster.
template <bool WIDE, bool ROLL, typename TX, int MT, int NT>
__device__ __forceinline__ void stream_compute(StreamItem<NT> &it, const TX *const (&x)[MT], f32x4 (&acc)[MT][NT],
                                               int blocks, const StreamRows<NT> &next, int next_b0, int nb, int c,
                                               F16Range &range)
{
    typedef typename Vec8<TX>::type vec;
    u32x4 sn[NT];
    if (ROLL && next_b0 >= 0)
        stream_load_s(sn, next, next_b0, nb);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        __builtin_amdgcn_sched_barrier(0);             // one step's activations in registers at a time
        u32x4 wu[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            wu[nt] = it.w[nt][u];
            if constexpr (std::is_same<TX, f16>::value && !WIDE)
                range.see(wu[nt], it.s[nt][u] >> (8 * c) & 0xFFu);
            transpose4(wu[nt]);
        }
        if (ROLL && next_b0 >= 0)
            stream_load_w(it.w, u, next, next_b0, nb, c);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (4 * u + s >= blocks)
                break;
            vec w[NT];
            bf16x8 wide[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint32_t byte = it.s[nt][u] >> (8 * s) & 0xFFu;
                if constexpr (WIDE) {
                    wide[nt] = mx4_to_bf16(wu[nt][s], mx4_scale(byte));
                } else if constexpr (std::is_same<TX, f16>::value) {
                    w[nt] = mx4_to_f16(wu[nt][s], mx4_scale(byte));
                } else {
                    w[nt] = mx4_to_bf16(wu[nt][s], mx4_scale(byte));
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const vec xv = load8(x[mt] + (4 * u + s) * 32);
                if constexpr (WIDE) {
                    __builtin_amdgcn_sched_barrier(0);
                    bf16x8 hi, lo;
                    split_f16(xv, hi, lo);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        acc[mt][nt] = mx4_mfma(hi, wide[nt], acc[mt][nt]);
                        acc[mt][nt] = mx4_mfma(lo, wide[nt], acc[mt][nt]);
                    }
                } else {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        acc[mt][nt] = mx4_mfma(xv, w[nt], acc[mt][nt]);
                }
            }
        }
    }
    if (ROLL && next_b0 >= 0)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            it.s[nt] = sn[nt];
}

// LDS for activations: rows of kc blocks, padded by 16 bytes (eight rows' pieces
// of 16 bytes then lie on distinct banks of 32; the counters still show 0.3 to
// 0.4 conflict cycles a busy one), kStreamLds bytes without the padding. kc for
// `rows` rows (64 at most): a whole number of items, all columns at most.
constexpr int kStreamLds = 64 * 1024;
__host__ __device__ inline int stream_chunk(int rows, int nb)
{
    const int fit = kStreamLds / (rows * 64 * kStreamBlocks) * kStreamBlocks;
    const int all = (nb + kStreamBlocks - 1) / kStreamBlocks * kStreamBlocks;
    return fit < all ? fit : all;
}

}  // namespace awq
