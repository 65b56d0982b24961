// k_mx4.hip -- rows to MXFP4 and back.
//
// Block of 32 values v (fp32; v = fp32(W s) with column scales), A = max |v|:
//   E = clamp(floor(log2 A) - 2, -127, 127), byte = E + 127
//   code = sign, and |v| 2^-E rounded to nearest even among 0 .5 1 1.5 2 3 4 6
// A's exponent field is floor(log2 A) + 127 (0 for subnormals, where E clamps
// to -127 all the same), so byte = max(field - 2, 0), and the field 255 of an
// infinity or NaN is the byte of a NaN block. The conversion instruction
// multiplies by a power of two, which is exact, rounds once to nearest even
// and saturates at 6.
//
// All are bound by HBM, one load of 16 bytes (fp32: 32) a thread four times in
// flight. 28672x4096, 2 bytes a value there and 0.53 here: quantize 53 us (5.6
// TB/s), with s 52, dequantize 51; fp32: 99, 99 and 97 us (5.4 TB/s); a copy of
// 2 GiB runs at 4.7 (both directions), a plain read at 6.1. 2048x4096 takes 6 to
// 7 us, of which a launch is 2-3. With s a block's 256 threads take one stretch of
// 2048 columns and those past the row idle: just above a multiple of 2048 and far
// below it s costs time (28672 rows of 2080 fp16 39 us, without s 29; of 256 8.2,
// 6.7; of 32 7.2, 3.3). Medians of graph replays over 600 MB of inputs in turn.
#include "mx4.h"

namespace awq {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 4;            // chunks of 8 values a thread has in flight

// One thread holds 8 values, four neighbouring lanes one block.
__device__ __forceinline__ void quantize8(const float (&v)[8], uint8_t *codes, uint8_t *scales, int64_t chunk)
{
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t m = __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu;
        a = a > m ? a : m;
    }
#pragma unroll
    for (int off = 1; off <= 2; off <<= 1) {
        const uint32_t o = __shfl_xor(a, off);
        a = a > o ? a : o;
    }
    const uint32_t field = a >> 23;
    const uint32_t byte = field == 255 ? 255 : field > 2 ? field - 2 : 0;
    const float s = __builtin_bit_cast(float, byte == 0 ? 0x00400000u : byte << 23);   // 2^E
    uint32_t q = 0;
    if (byte != 255) {
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], s, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], s, 1);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], s, 2);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], s, 3);
    }
    reinterpret_cast<uint32_t *>(codes)[chunk] = q;
    if ((chunk & 3) == 0)
        scales[chunk >> 2] = (uint8_t)byte;
}

// Without column scales the matrix is one long list of blocks.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_mx4_quantize(const T *__restrict__ W, int64_t chunks,
                                                           uint8_t *__restrict__ codes, uint8_t *__restrict__ scales)
{
    const int64_t first = (int64_t)blockIdx.x * (kThreads * kPer) + threadIdx.x;
    typename Vec8<T>::type x[kPer];
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        const int64_t ch = first + p * kThreads;
        x[p] = load8(W + (ch < chunks ? ch : chunks - 1) * 8);
    }
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        const int64_t ch = first + p * kThreads;
        if (ch < chunks) {         // chunks is a multiple of 4: a block's four lanes agree
            float v[8];
            widen8<T>(x[p], v);
            quantize8(v, codes, scales, ch);
        }
    }
}

// With column scales: a thread keeps the scales of its 8 columns and walks
// down rows.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_mx4_quantize_s(const T *__restrict__ W, const float *__restrict__ s,
                                                             int64_t rows, int64_t cpr, int64_t rows_per_block,
                                                             uint8_t *__restrict__ codes, uint8_t *__restrict__ scales)
{
    const int64_t col = (int64_t)blockIdx.x * kThreads + threadIdx.x;     // chunk within the row
    if (col >= cpr)
        return;
    const f32x8 sv = load8(s + col * 8);
    const int64_t r0 = (int64_t)blockIdx.y * rows_per_block;
    const int64_t r1 = r0 + rows_per_block < rows ? r0 + rows_per_block : rows;
    for (int64_t r = r0; r < r1; r += kPer) {
        typename Vec8<T>::type x[kPer];
#pragma unroll
        for (int p = 0; p < kPer; ++p)
            x[p] = load8(W + ((r + p < r1 ? r + p : r1 - 1) * cpr + col) * 8);
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            if (r + p >= r1)
                break;
            float v[8];
            widen8<T>(x[p], v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = opaque(v[i]) * sv[i];
            quantize8(v, codes, scales, (r + p) * cpr + col);
        }
    }
}

// The values that a thread makes of one load of codes, 16 bytes, so that lanes
// store whole lines (fp32 by 32 bytes a lane: 121 us where this takes 97).
template <typename T> struct Piece {
    typedef uint32_t word;
    static __device__ __forceinline__ typename Vec8<T>::type make(word w, float s)
    {
        if constexpr (std::is_same<T, f16>::value)
            return mx4_to_f16(w, s);
        else
            return mx4_to_bf16(w, s);
    }
};
template <> struct Piece<float> {
    typedef uint16_t word;
    static __device__ __forceinline__ f32x4 make(word w, float s)
    {
        const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4((uint32_t)w, s, 0);
        const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4((uint32_t)w, s, 1);
        return f32x4{a[0], a[1], b[0], b[1]};
    }
};

template <typename T>
__global__ __launch_bounds__(kThreads) void k_mx4_dequantize(const typename Piece<T>::word *__restrict__ codes,
                                                             const uint8_t *__restrict__ scales, int64_t pieces,
                                                             T *__restrict__ out)
{
    constexpr int V = 16 / sizeof(T), kEach = 32 / V;  // kEach: 32 values a thread
    typedef decltype(Piece<T>::make(0, 0.f)) vec;
    const int64_t first = (int64_t)blockIdx.x * (kThreads * kEach) + threadIdx.x;
    typename Piece<T>::word w[kEach];
    uint8_t b[kEach];
#pragma unroll
    for (int p = 0; p < kEach; ++p) {
        const int64_t at = first + p * kThreads < pieces ? first + p * kThreads : pieces - 1;
        w[p] = codes[at];
        b[p] = scales[at / (32 / V)];
    }
#pragma unroll
    for (int p = 0; p < kEach; ++p) {
        const int64_t at = first + p * kThreads;
        if (at < pieces)
            reinterpret_cast<vec *>(out)[at] = Piece<T>::make(w[p], mx4_scale(b[p]));
    }
}

template <typename T>
hipError_t quantize(const void *W, int64_t rows, int64_t in, const float *s, uint8_t *codes, uint8_t *scales,
                    hipStream_t st)
{
    const int64_t cpr = in / 8;
    if (!s) {
        const int64_t chunks = rows * cpr, blocks = (chunks + kThreads * kPer - 1) / (kThreads * kPer);
        k_mx4_quantize<T><<<dim3((uint32_t)blocks), kThreads, 0, st>>>((const T *)W, chunks, codes, scales);
    } else {
        const int64_t xb = (cpr + kThreads - 1) / kThreads;
        // rows per block: one round of loads, and within the grid's 65535
        const int64_t rpb = rows <= 65535 * kPer ? kPer : (rows + 65534) / 65535;
        k_mx4_quantize_s<T><<<dim3((uint32_t)xb, (uint32_t)((rows + rpb - 1) / rpb)), kThreads, 0, st>>>(
            (const T *)W, s, rows, cpr, rpb, codes, scales);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx4_quantize(const void *W, int dtype, int64_t rows, int64_t in, const float *s, uint8_t *codes,
                               uint8_t *scales, hipStream_t st)
{
    switch (dtype) {
    case AWQ_F32: return quantize<float>(W, rows, in, s, codes, scales, st);
    case AWQ_F16: return quantize<f16>(W, rows, in, s, codes, scales, st);
    default: return quantize<bf16>(W, rows, in, s, codes, scales, st);
    }
}

hipError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t in, void *out,
                                 int dtype, hipStream_t st)
{
    auto run = [&](auto *to) {
        typedef typename std::remove_pointer<decltype(to)>::type T;
        typedef typename Piece<T>::word word;
        const int64_t values = rows * in;
        k_mx4_dequantize<T><<<dim3((uint32_t)((values + kThreads * 32 - 1) / (kThreads * 32))), kThreads, 0, st>>>(
            (const word *)codes, scales, values / (int64_t)(16 / sizeof(T)), to);
    };
    if (dtype == AWQ_F32)
        run((float *)out);
    else if (dtype == AWQ_F16)
        run((f16 *)out);
    else
        run((bf16 *)out);
    return hipGetLastError();
}

}  // namespace awq
