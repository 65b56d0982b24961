// k_mx8_gemm.hip -- products of MXFP8 activations with MXFP4 weights, Y[m][n] = sum_k X[m][k] W[n][k].
//
// The scaled matrix instructions take both operands as they are stored, codes and
// scale bytes, so the only roundings are those of the fp32 sums. What the matrix cores cut off
// products of eight columns (see mx8_stream.h) lies far below a 16-bit Y's rounding, but
// not below that of an fp32 Y: for that one activations go in two parts.
#include "mx8_mid.h"
#include "mx8_stream.h"

namespace awq {

namespace {

template <typename TY> constexpr bool kExact = std::is_same<TY, float>::value;

// Up to 16 tokens (see mx8_stream.h). Block: 8 / S row tiles of 16, S waves a tile. Bound by
// the latency of a wave's weights, of which it has one item of 4 KB on its way at a time (64 KB a
// unit) and four in turn: 4 tokens x 28672x4096 17.9 us, 3.5 TB/s, fp32 Y 18.5; small
// layers by that of a launch too (1 token x 4096x4096 5.2 us, of which a launch is 2-3).
template <typename TY, int S>
__global__ __launch_bounds__(512, 4) void k_mx8_gemm_stream(const uint8_t *__restrict__ xcodes,
                                                            const uint8_t *__restrict__ xscales, int M, int nb,
                                                            const uint8_t *__restrict__ codes,
                                                            const uint8_t *__restrict__ scales, int64_t out,
                                                            TY *__restrict__ Y)
{
    __shared__ __align__(16) union { StreamLds in; f32x4 red[8][64]; } lds;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, c = lane >> 4;
    const int64_t n0 = ((int64_t)blockIdx.x * (8 / S) + wave / S) * 16, n = n0 + r < out ? n0 + r : out - 1;
    f32x4 acc;
    stream_contract<kExact<TY>, S>(acc, lds.in, xcodes, xscales, [](int m) { return m; }, M, codes + n * nb * 16, scales + n * nb, wave % S, nb);
    __syncthreads();                                   // the waves' sums in wave order
    lds.red[wave][lane] = acc;
    __syncthreads();
    if (wave % S)
        return;
#pragma unroll
    for (int k = 1; k < S; ++k)
        acc += lds.red[wave + k][lane];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (4 * c + i < M && n0 + r < out)
            Y[(int64_t)(4 * c + i) * out + n0 + r] = static_cast<TY>(acc[i]);
}

// Few tokens or few tiles (see mx8_mid.h): 32 x 32 NT. Bound by what a unit's load path takes
// (64 bytes a cycle, half of it for the weights' 64-byte rows) and by each wave's chain of
// wait, LDS reads and products: 64 tokens x 4096x4096 8.3 us, 256 tokens 15 us, 570 TFLOP/s, fp32 Y
// 9.5 and 16.8.
template <typename TY, int NT>
__global__ __launch_bounds__(kMidThreads) void k_mx8_gemm_mid(const uint8_t *__restrict__ xcodes,
                                                              const uint8_t *__restrict__ xscales, int64_t M, int nb,
                                                              const uint8_t *__restrict__ codes,
                                                              const uint8_t *__restrict__ scales, int64_t out,
                                                              TY *__restrict__ Y)
{
    __shared__ __align__(16) Mid8<NT> lds;
    int64_t m0, n0;
    if (!tile_of_block((M + 31) / 32, (out + 32 * NT - 1) / (32 * NT), m0, n0))
        return;
    m0 *= 32;
    n0 *= 32 * NT;
    mid8_contract<kExact<TY>>(
        lds, xcodes + m0 * nb * 32, xscales + m0 * nb, [&](int m) { return m0 + m < M ? m : (int)(M - 1 - m0); },
        codes + n0 * nb * 16, scales + n0 * nb, [&](int n) { return n0 + n < out ? n : (int)(out - 1 - n0); }, nb);
    // wave q: registers 4 q ... of every tile, tokens 8 q + 4 h ...
    const int lane = threadIdx.x & 63, q = threadIdx.x >> 6, r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int b = 0; b < NT; ++b) {
        const f32x4 s = mid8_sum(lds, b, lane, q);
        const int64_t m = m0 + 8 * q + 4 * h, n = n0 + 32 * b + r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (m + i < M && n < out)
                Y[(m + i) * out + n] = static_cast<TY>(s[i]);
    }
}

// Many tokens: tiles of 256 x 256 (see mx8_tile.h), those of a last round that fills at
// most half of the chip cut in two. Bound by the matrix cores (60 % busy) and the loads that
// their phases wait for: 2048 tokens x 28672x4096 203 us, 2370 TFLOP/s, 8192 tokens 2510; with
// an fp32 Y, twice the matrix instructions, 366 us.
template <typename TY, int MT>
__device__ __forceinline__ void tile(Tile8<MT> &lds, int64_t m0, int64_t n0, const uint8_t *xcodes,
                                     const uint8_t *xscales, int64_t M, int nb, const uint8_t *codes,
                                     const uint8_t *scales, int64_t out, TY *Y)
{
    constexpr int BM = Tile8<MT>::BM, BN = Tile8<MT>::BN;
    // rows past the ends load the last row: their results are not stored
    const int tid = threadIdx.x, mlast = (int)(M - 1 - m0 < BM - 1 ? M - 1 - m0 : BM - 1);
    const int nlast = (int)(out - 1 - n0 < BN - 1 ? out - 1 - n0 : BN - 1);
    auto xrow = [&](int m) { return m0 + (m < mlast ? m : mlast); };
    auto wrow = [&](int n) { return n0 + (n < nlast ? n : nlast); };
    uint32_t xo[MT], wo[2];                            // in is at most 2^23 columns
#pragma unroll
    for (int i = 0; i < MT; ++i)
        xo[i] = (uint32_t)(xrow(tile8_xrow() + 64 * i) - m0) * (uint32_t)nb * 32 + tile8_xchunk() * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        wo[i] = (uint32_t)(wrow(tile8_wrow() + 128 * i) - n0) * (uint32_t)nb * 16 + tile8_wchunk() * 16;
    const uint8_t *const sp = tid < BM ? xscales + xrow(tid) * nb : scales + wrow(tid - BM) * nb;
    const bool words = (((uintptr_t)xscales | (uintptr_t)scales | (uintptr_t)nb) & 3) == 0;
    f32x16 acc[MT][2];
    tile8_contract<false, kExact<TY>, MT>(lds, acc, xcodes + m0 * nb * 32, xo, codes + n0 * nb * 16, wo, sp, words, nb);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    store_tiles<TY, MT>(Y, acc, reinterpret_cast<float *>(lds.x) + 2048 * wave, m0 + 32 * MT * (wave >> 2),
                        n0 + 64 * (wave & 3), M, out, tid & 63);
}

// The tiles of an XCD (a contiguous range, as in tile_of_block) that are whole, of `chunk`.
__host__ __device__ inline int64_t whole_tiles(int64_t chunk) { return chunk % 32 <= 16 ? chunk / 32 * 32 : chunk; }

template <typename TY>
__global__ __launch_bounds__(512, 2) void k_mx8_gemm_tile(const uint8_t *__restrict__ xcodes,
                                                          const uint8_t *__restrict__ xscales, int64_t M, int nb,
                                                          const uint8_t *__restrict__ codes,
                                                          const uint8_t *__restrict__ scales, int64_t out,
                                                          TY *__restrict__ Y)
{
    __shared__ __align__(16) union { Tile8<4> four; Tile8<2> two; } lds;
    const int64_t tm = (M + 255) / 256, tn = (out + 255) / 256, tiles = tm * tn, chunk = (tiles + 7) / 8;
    const int64_t whole = whole_tiles(chunk), i = blockIdx.x >> 3, in_xcd = i < whole ? i : whole + (i - whole) / 2;
    const int64_t t = (blockIdx.x & 7) * chunk + in_xcd;
    if (in_xcd >= chunk || t >= tiles)
        return;
    const int64_t band = t / (4 * tn), first = band * 4, in_band = t - band * 4 * tn;      // see tile_of_block
    const int64_t h = tm - first < 4 ? tm - first : 4;
    int64_t m0 = (first + in_band % h) * 256;
    const int64_t n0 = in_band / h * 256;
    if (i < whole) {
        tile<TY, 4>(lds.four, m0, n0, xcodes, xscales, M, nb, codes, scales, out, Y);
    } else {
        m0 += (i - whole) % 2 * 128;
        if (m0 < M)
            tile<TY, 2>(lds.two, m0, n0, xcodes, xscales, M, nb, codes, scales, out, Y);
    }
}

template <typename TY>
hipError_t gemm_a8(const uint8_t *xc, const uint8_t *xs, int64_t M, int nb, const uint8_t *codes, const uint8_t *scales,
                   int64_t out, TY *Y, hipStream_t st)
{
    auto mid = [&]<int NT>() {
        k_mx8_gemm_mid<TY, NT><<<tile_grid(tiles_of(M, 32) * tiles_of(out, 32 * NT)), kMidThreads, 0, st>>>(
            xc, xs, M, nb, codes, scales, out, Y);
    };
    auto stream = [&]<int S>() {
        k_mx8_gemm_stream<TY, S><<<(uint32_t)tiles_of(out, 16 * (8 / S)), 512, 0, st>>>(xc, xs, (int)M, nb, codes, scales,
                                                                                       out, Y);
    };
    if (M <= 16) {
        // Waves a row tile: enough blocks for the chip (600 MB of weights in turn, us by S = 2,
        // 4, 8: 4 tokens x 28672x4096 17.9, 18.8, 21.3; x 12288x4096 11.4, 10.8, 11.6; x
        // 4096x14336 28.4, 17.7, 12.6; 1 token x 4096x4096 8.4, 6.2, 5.2; by k_mx8_gemm_mid
        // 20.2, 13.0, 25.0 and 7.5)
        const int64_t tiles = tiles_of(out, 16);
        if (tiles >= 1280)
            stream.template operator()<2>();
        else if (tiles >= 640)
            stream.template operator()<4>();
        else
            stream.template operator()<8>();
        return hipGetLastError();
    }
    // Blocks of 32 x 64, two on a unit at a time, or large tiles: 4096 columns take 15 us for
    // each 512 of the small (256 x 4096 rows 15, tiles 28; 512 x 4096 26, 29; 64 x 28672 35,
    // 33), 30 for one round of half tiles and 55 for each of whole ones; in two parts, for
    // which the large tiles' matrix cores need twice as long, 50 and 92 (512 x 4096 small
    // 30, tiles 50; 1024 x 4096 54, 53; 64 x 28672 38, 54; 128 x 28672 60, 54). Small blocks of
    // 32 x 32 where no unit has more than one (64 x 4096 rows 8.3 us, by 32 x 64 10.8).
    constexpr int half = kExact<TY> ? 50 : 30, round = kExact<TY> ? 92 : 55;
    const int64_t small = tiles_of(M, 32) * tiles_of(out, 64), large = tiles_of(M, 256) * tiles_of(out, 256);
    if (15 * tiles_of(small, 512) >= (2 * large <= 256 ? half : round * tiles_of(large, 256))) {
        const int64_t chunk = tiles_of(large, 8), whole = whole_tiles(chunk);
        k_mx8_gemm_tile<TY><<<(uint32_t)(8 * (2 * chunk - whole)), 512, 0, st>>>(xc, xs, M, nb, codes, scales, out, Y);
    } else if (tiles_of(M, 32) * tiles_of(out, 32) <= 256) {
        mid.template operator()<1>();
    } else {
        mid.template operator()<2>();
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx4_gemm_a8(const uint8_t *xcodes, const uint8_t *xscales, int64_t M, int64_t in,
                              const uint8_t *codes, const uint8_t *scales, int64_t out, void *Y, int y_dtype,
                              hipStream_t st)
{
    const int nb = (int)(in / kMxBlock);
    switch (y_dtype) {
    case AWQ_F32: return gemm_a8(xcodes, xscales, M, nb, codes, scales, out, (float *)Y, st);
    case AWQ_F16: return gemm_a8(xcodes, xscales, M, nb, codes, scales, out, (f16 *)Y, st);
    default: return gemm_a8(xcodes, xscales, M, nb, codes, scales, out, (bf16 *)Y, st);
    }
}

}  // namespace awq
