// k_mx4_gemm.hip -- products with MXFP4 weights, Y[m][n] = sum_k X[m][k] W[n][k].
//
// Weights enter the matrix instructions as values: bf16 and fp16 hold
// e2m1 * 2^E exactly (fp16 for E in [-13, 13]; elsewhere the fp16 activations
// go as two exact bf16 parts), so the only roundings are those of the fp32
// sums. With MXFP4 activations the scaled matrix instruction takes codes and
// scale bytes as they are.
#include "mx4.h"

namespace awq {

namespace {

template <typename TX, typename TY>
__device__ __forceinline__ void store_tile(TY *Y, int64_t m, int64_t n, int64_t M, int64_t out, const f32x4 &v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (m + i < M && n < out)
            Y[(m + i) * out + n] = static_cast<TY>(v[i]);
}

// Block: 16 MT tokens x 16 NT rows, the columns split over the waves in items
// of 128 U; each wave's next item is in flight while it multiplies the
// current one. The waves' sums are added in wave order through LDS.
template <typename TX, typename TY, int MT, int NT, int U, int W>
__global__ __launch_bounds__(64 * W) void k_mx4_gemm_split(const void *__restrict__ X, const uint8_t *__restrict__ xs,
                                                           int64_t M, int nb, const uint8_t *__restrict__ codes,
                                                           const uint8_t *__restrict__ scales, int64_t out,
                                                           TY *__restrict__ Y)
{
    constexpr bool kAct4 = std::is_same<TX, Mx4Act>::value;
    constexpr int TILES = MT * NT, TG = TILES < 4 ? TILES : 4;
    __shared__ f32x4 red[W * TG * 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, c = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * NT), m0 = (int64_t)blockIdx.y * (16 * MT);

    // rows past the ends load the last row: their results are not stored
    Mx4Rows<TX, MT, NT> rows;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        int64_t n = n0 + 16 * nt + r;
        n = n < out ? n : out - 1;
        rows.w[nt] = codes + n * nb * 16;
        rows.ws[nt] = scales + n * nb;
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        int64_t m = m0 + 16 * mt + r;
        m = m < M ? m : M - 1;
        if constexpr (kAct4) {
            rows.x[mt] = (const uint8_t *)X + m * nb * 16;
            rows.xs[mt] = xs + m * nb;
        } else {
            rows.x[mt] = (const uint16_t *)X + m * nb * 32;
            rows.xs[mt] = nullptr;
        }
    }

    f32x4 acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            acc[mt][nt] = f32x4{0.f, 0.f, 0.f, 0.f};

    Mx4Item<TX, MT, NT, U> a, b;
    int i = wave * (4 * U);
    const int step = W * (4 * U);
    if (i < nb) {
        mx4_load(a, rows, i, nb, c);
        while (true) {
            if (i + step < nb)
                mx4_load(b, rows, i + step, nb, c);
            mx4_compute(a, acc, i, nb, c);
            i += step;
            if (i >= nb)
                break;
            if (i + step < nb)
                mx4_load(a, rows, i + step, nb, c);
            mx4_compute(b, acc, i, nb, c);
            i += step;
            if (i >= nb)
                break;
        }
    }

#pragma unroll
    for (int t0 = 0; t0 < TILES; t0 += TG) {
        if (t0)
            __syncthreads();
#pragma unroll
        for (int t = 0; t < TG; ++t)
            red[(wave * TG + t) * 64 + lane] = acc[(t0 + t) / NT][(t0 + t) % NT];
        __syncthreads();
        for (int idx = threadIdx.x; idx < TG * 64; idx += 64 * W) {
            f32x4 sum = red[idx];
#pragma unroll
            for (int w = 1; w < W; ++w)
                sum += red[w * TG * 64 + idx];
            const int t = t0 + idx / 64, l = idx & 63;
            store_tile<TX, TY>(Y, m0 + 16 * (t / NT) + 4 * (l >> 4), n0 + 16 * (t % NT) + (l & 15), M, out, sum);
        }
    }
}

template <typename TX, typename TY, int MT, int NT, int U>
hipError_t split(const void *X, const uint8_t *xs, int64_t M, int nb, const uint8_t *codes, const uint8_t *scales,
                 int64_t out, void *Y, hipStream_t st)
{
    const dim3 grid((uint32_t)((out + 16 * NT - 1) / (16 * NT)), (uint32_t)((M + 16 * MT - 1) / (16 * MT)));
    k_mx4_gemm_split<TX, TY, MT, NT, U, 8><<<grid, 512, 0, st>>>(X, xs, M, nb, codes, scales, out, (TY *)Y);
    return hipGetLastError();
}

template <typename TX, typename TY>
hipError_t gemm(const void *X, const uint8_t *xs, int64_t M, int nb, const uint8_t *codes, const uint8_t *scales,
                int64_t out, void *Y, hipStream_t st)
{
    if (M <= 16)
        return split<TX, TY, 1, 1, 4>(X, xs, M, nb, codes, scales, out, Y, st);
    if constexpr (std::is_same<TX, Mx4Act>::value)
        return split<TX, TY, 4, 4, 1>(X, xs, M, nb, codes, scales, out, Y, st);
    else
        return split<TX, TY, 4, 2, 1>(X, xs, M, nb, codes, scales, out, Y, st);
}

}  // namespace

hipError_t launch_mx4_gemm(const void *X, int dtype, int64_t M, int64_t in, const uint8_t *codes, const uint8_t *scales,
                           int64_t out, void *Y, bool yf32, hipStream_t st)
{
    const int nb = (int)(in / kMxBlock);
    if (dtype == AWQ_F16)
        return yf32 ? gemm<f16, float>(X, nullptr, M, nb, codes, scales, out, Y, st)
                    : gemm<f16, f16>(X, nullptr, M, nb, codes, scales, out, Y, st);
    return yf32 ? gemm<bf16, float>(X, nullptr, M, nb, codes, scales, out, Y, st)
                : gemm<bf16, bf16>(X, nullptr, M, nb, codes, scales, out, Y, st);
}

hipError_t launch_mx4_gemm_a4(const uint8_t *xcodes, const uint8_t *xscales, int64_t M, int64_t in,
                              const uint8_t *codes, const uint8_t *scales, int64_t out, void *Y, int y_dtype,
                              hipStream_t st)
{
    const int nb = (int)(in / kMxBlock);
    switch (y_dtype) {
    case AWQ_F32: return gemm<Mx4Act, float>(xcodes, xscales, M, nb, codes, scales, out, Y, st);
    case AWQ_F16: return gemm<Mx4Act, f16>(xcodes, xscales, M, nb, codes, scales, out, Y, st);
    default: return gemm<Mx4Act, bf16>(xcodes, xscales, M, nb, codes, scales, out, Y, st);
    }
}

}  // namespace awq
