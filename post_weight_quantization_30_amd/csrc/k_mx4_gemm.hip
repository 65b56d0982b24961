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
    mx4_wave<TX, MT, NT, U>(rows, acc, wave * (4 * U), W * (4 * U), nb, c);

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

// ---------------------------------------------------------------------------
// Up to 16 tokens of 16-bit activations, more row tiles than the chip has
// units for a whole block each. Block: 8 / S row tiles of 16, all columns, S
// waves a tile; the activations go through LDS in chunks of kc blocks that all
// waves share. Every wave streams its own weights (see StreamItem), the next
// item in flight also across the chunks' barriers.
template <typename TX, typename TY, int S>
__global__ __launch_bounds__(512, 4) void k_mx4_gemv(const TX *__restrict__ X, int M, int nb, int kc,
                                                     const uint8_t *__restrict__ codes,
                                                     const uint8_t *__restrict__ scales, int64_t out,
                                                     TY *__restrict__ Y)
{
    __shared__ __align__(16) uint8_t lds[kStreamLds + 16 * 16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, c = lane >> 4, part = wave % S;
    const int64_t n0 = ((int64_t)blockIdx.x * (8 / S) + wave / S) * 16;
    const int64_t first = n0 < out ? n0 : out - 1;         // rows past the end load the last one: not stored
    StreamRows<1> rows = {{codes + first * nb * 16}, {scales + first * nb}};
    rows.lane((uint32_t)(first + r < out ? r : out - 1 - first), c, nb);
    const int stride = kc * 64 + 16, row = (r < M ? r : M - 1) * stride + c * 16;
    const int items = (nb + kStreamBlocks - 1) / kStreamBlocks, per = kc / kStreamBlocks;
    bool bad = false;
    f32x4 acc[1][1];

    auto stage = [&](int i0) {                             // columns of items i0 ... i0 + per - 1
        const int b0 = i0 * kStreamBlocks, len = (b0 + kc < nb ? kc : nb - b0) * 4;
        for (int m = wave; m < M; m += 8)
            for (int j = lane; j < len; j += 64)
                *reinterpret_cast<u32x4 *>(lds + m * stride + j * 16) =
                    *reinterpret_cast<const u32x4 *>(X + ((int64_t)m * nb + b0) * 32 + j * 8);
    };
    auto contract = [&]<bool WIDE>() {
        acc[0][0] = f32x4{0.f, 0.f, 0.f, 0.f};
        StreamItem<1> it;
        int i = part;                                      // the wave's items: part, part + S, ...
        if (i < items)
            stream_load(it, rows, i * kStreamBlocks, nb, c);
#pragma unroll 1
        for (int i0 = 0; i0 < items; i0 += per) {
            if (i0)
                __syncthreads();
            stage(i0);
            __syncthreads();
            const int end = i0 + per < items ? i0 + per : items;
#pragma unroll 1
            for (; i < end; i += S) {
                const TX *const x[1] = {(const TX *)(lds + row + (i - i0) * kStreamBlocks * 64)};
                stream_compute<WIDE, true>(it, x, acc, nb - i * kStreamBlocks, 1, rows,
                                     i + S < items ? (i + S) * kStreamBlocks : -1, nb, c, bad);
            }
        }
    };
    contract.template operator()<false>();
    if constexpr (std::is_same<TX, f16>::value)
        if (__syncthreads_or(bad))                         // scales that fp16 cannot hold
            contract.template operator()<true>();
    if constexpr (S > 1) {
        f32x4 *const red = reinterpret_cast<f32x4 *>(lds);
        __syncthreads();
        red[threadIdx.x] = acc[0][0];
        __syncthreads();
        if (part)
            return;
#pragma unroll
        for (int k = 1; k < S; ++k)
            acc[0][0] += red[threadIdx.x + 64 * k];
    }
    store_tile<TX, TY>(Y, 4 * c, n0 + r, M, out, acc[0][0]);
}

template <typename TX, typename TY, int S>
hipError_t gemv(const void *X, int M, int nb, const uint8_t *codes, const uint8_t *scales, int64_t out, void *Y,
                hipStream_t st)
{
    const int64_t tiles = (out + 15) / 16;
    k_mx4_gemv<TX, TY, S><<<dim3((uint32_t)((tiles + 8 / S - 1) / (8 / S))), 512, 0, st>>>(
        (const TX *)X, M, nb, stream_chunk(M, nb), codes, scales, out, (TY *)Y);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Many tokens: 32x32 matrix tiles.

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16 mfma32(const bf16x8 &a, const bf16x8 &b, const f32x16 &c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma32(const f16x8 &a, const f16x8 &b, const f32x16 &c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
// Both operands MXFP4, 64 columns; byte S of the scale registers.
template <int S>
__device__ __forceinline__ f32x16 mfma32(const u32x4 &a, uint32_t sa, const u32x4 &b, uint32_t sb, const f32x16 &c)
{
    const i32x8 a8 = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 b8 = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, S, (int)sa, S, (int)sb);
}

// Tile of this block: the blocks of one XCD (every eighth) walk a contiguous
// range of tiles, 16 token tiles by one row tile at a time, so that what they
// read together stays in that XCD's L2.
__device__ __forceinline__ bool tile_of_block(int64_t tm, int64_t tn, int64_t &m, int64_t &n)
{
    const int64_t tiles = tm * tn, chunk = (tiles + 7) / 8;
    const int64_t t = (blockIdx.x & 7) * chunk + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= chunk || t >= tiles)
        return false;
    const int64_t band = t / (16 * tn), first = band * 16, in_band = t - band * 16 * tn;
    const int64_t h = tm - first < 16 ? tm - first : 16;
    m = first + in_band % h;
    n = in_band / h;
    return true;
}

// The results of a wave's MT x NT tiles, tile (a, b) at token m0 + 32 a, row
// n0 + 32 b: register i of lane (r, h) is token 8 (i / 4) + 4 h + i % 4, row r.
template <typename TY, int MT, int NT>
__device__ __forceinline__ void store_tiles(TY *__restrict__ Y, const f32x16 (&acc)[MT][NT], int64_t m0, int64_t n0,
                                            int64_t M, int64_t out, int r, int h)
{
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int b = 0; b < NT; ++b) {
            const int64_t n = n0 + 32 * b + r;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int64_t m = m0 + 32 * a + 8 * (i / 4) + 4 * h + i % 4;
                if (m < M && n < out)
                    Y[m * out + n] = static_cast<TY>(acc[a][b][i]);
            }
        }
}

// 16-bit activations. Block: 128 tokens x 256 rows, 4 waves of 128 x 64. A
// step is 64 columns: 128 bytes of every activation row go to LDS as eight
// 16-byte chunks, chunk q of row m at position q ^ (m & 7), so that the eight
// rows which one 128-byte LDS cycle serves lie on distinct banks. Weights go
// from memory straight to the registers of the wave that multiplies them: no
// other wave has its rows, and one conversion there serves all 128 tokens.
// Step k + 1 is fetched while step k is multiplied; two LDS buffers, one
// barrier a step.
// Lane (r, h) = (lane % 32, lane / 32) of a 32-row tile holds in k-step s of 4
// columns 32 h + 8 s ... of the step: chunk 4 h + s of an activation row, word
// s of block h of a weight row.
template <typename TX, typename TY>
__global__ __launch_bounds__(256, 2) void k_mx4_gemm_tile(const TX *__restrict__ X, int64_t M, int nb,
                                                          const uint8_t *__restrict__ codes,
                                                          const uint8_t *__restrict__ scales, int64_t out,
                                                          TY *__restrict__ Y)
{
    typedef typename Vec8<TX>::type vec;
    constexpr int MT = 4, NT = 2, BM = 128, BN = 256;
    constexpr int CH = BM * 8 / 256;                   // activation chunks a thread moves in a step
    __shared__ __align__(16) u32x4 lds[2][BM * 8];

    int64_t m0, n0;
    if (!tile_of_block((M + BM - 1) / BM, (out + BN - 1) / BN, m0, n0))
        return;
    m0 *= BM;
    n0 *= BN;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, h = lane >> 5;
    const int xrow = nb * 64;                          // bytes of an activation row
    const int steps = (nb + 1) / 2, full = nb / 2;

    // Addresses are a scalar base (this tile, this step) and a 32-bit offset a
    // lane (rows have at most 2^23 columns). Rows past the ends load the last
    // row: their results are not stored.
    const uint8_t *const xbase = (const uint8_t *)X + m0 * xrow;
    const uint8_t *const wbase = codes + n0 * nb * 16, *const wsbase = scales + n0 * nb;
    const uint32_t mlast = (uint32_t)(M - 1 - m0 < BM - 1 ? M - 1 - m0 : BM - 1);
    const uint32_t nlast = (uint32_t)(out - 1 - n0 < BN - 1 ? out - 1 - n0 : BN - 1);
    uint32_t xo[CH], wo[NT], wso[NT];
    int xdst[CH];
    const int xq = threadIdx.x & 7;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const uint32_t row = (threadIdx.x + i * 256) >> 3;
        xdst[i] = row * 8 + (xq ^ (row & 7));
        xo[i] = (row < mlast ? row : mlast) * (uint32_t)xrow + xq * 16;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        uint32_t n = 64 * wave + 32 * t + r;
        n = n < nlast ? n : nlast;
        wo[t] = n * (uint32_t)nb * 16 + h * 16;
        wso[t] = n * (uint32_t)nb + h;
    }

    f32x16 acc[MT][NT];
    u32x4 xr[CH], w[NT], wnext[NT];
    uint32_t ws[NT], wsnext[NT];
    bool bad = false;

    // An odd last block: the step's second half loads the row's last block
    // instead; zeros (under scale 1) take its place on the way to use.
    auto fetch = [&](int k) {
        const bool end = k >= full;
        const uint32_t xback = end && xq >= 4 ? 64 : 0, wback = end && h ? 1 : 0;
        const uint8_t *const px = xbase + (int64_t)k * 128, *const pw = wbase + (int64_t)k * 32;
        const uint8_t *const ps = wsbase + k * 2;
#pragma unroll
        for (int i = 0; i < CH; ++i)
            xr[i] = *reinterpret_cast<const u32x4 *>(px + (xo[i] - xback));
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            wnext[t] = *reinterpret_cast<const u32x4 *>(pw + (wo[t] - 16 * wback));
            wsnext[t] = ps[wso[t] - wback];
        }
    };
    auto stash = [&](int k) {
        if (k >= full && xq >= 4)
#pragma unroll
            for (int i = 0; i < CH; ++i)
                xr[i] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < CH; ++i)
            lds[k & 1][xdst[i]] = xr[i];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            w[t] = wnext[t];
            ws[t] = k >= full && h ? 127 : wsnext[t];
        }
    };
    auto xfrag = [&](int k, int t, int s) -> u32x4 {
        const int row = 32 * t + r;
        return lds[k & 1][row * 8 + ((4 * h + s) ^ (row & 7))];
    };
    auto contract = [&]<bool WIDE>() {
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < NT; ++b)
                acc[a][b] = f32x16{};
        fetch(0);
        stash(0);
        __syncthreads();
        for (int k = 0; k < steps; ++k) {
            if (k + 1 < steps)
                fetch(k + 1);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if constexpr (!WIDE) {
                    vec wv[NT];
#pragma unroll
                    for (int b = 0; b < NT; ++b) {
                        if constexpr (std::is_same<TX, f16>::value) {
                            wv[b] = mx4_to_f16(w[b][s], mx4_scale(ws[b]));
                            bad = bad || !mx4_fits_f16(ws[b]);
                        } else {
                            wv[b] = mx4_to_bf16(w[b][s], mx4_scale(ws[b]));
                        }
                    }
#pragma unroll
                    for (int a = 0; a < MT; ++a) {
                        const vec x = __builtin_bit_cast(vec, xfrag(k, a, s));
#pragma unroll
                        for (int b = 0; b < NT; ++b)
                            acc[a][b] = mfma32(x, wv[b], acc[a][b]);
                    }
                } else {
                    __builtin_amdgcn_sched_barrier(0);
                    bf16x8 wv[NT];
#pragma unroll
                    for (int b = 0; b < NT; ++b)
                        wv[b] = mx4_to_bf16(w[b][s], mx4_scale(ws[b]));
#pragma unroll
                    for (int a = 0; a < MT; ++a) {
                        bf16x8 hi, lo;
                        split_f16(__builtin_bit_cast(f16x8, xfrag(k, a, s)), hi, lo);
#pragma unroll
                        for (int b = 0; b < NT; ++b) {
                            acc[a][b] = mfma32(hi, wv[b], acc[a][b]);
                            acc[a][b] = mfma32(lo, wv[b], acc[a][b]);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
            if (k + 1 < steps)
                stash(k + 1);
            __syncthreads();
        }
    };
    contract.template operator()<false>();
    // fp16 activations under scales that fp16 cannot hold: all of it once more
    // in the wide form (weights in bf16, activations as two bf16 parts)
    if constexpr (std::is_same<TX, f16>::value)
        if (__syncthreads_or(bad))
            contract.template operator()<true>();
    store_tiles<TY, MT, NT>(Y, acc, m0, n0 + 64 * wave, M, out, r, h);
}

// 16-bit activations, too few 128 x 256 tiles for the chip. Block: 32 MT tokens
// x 64 rows, 8 waves: two of 32 rows each in four groups that take the steps of
// 64 columns in turn, each with its own LDS buffers (laid out as above); the
// groups' sums meet in LDS. 64 x 64 tiles keep all units busy from about 200
// tokens x 4000 rows on, and a token's row is read in whole 128-byte lines
// (read in matrix order, 64 bytes of 16 rows at a time, it kept the load units
// busy for twice as long as everything else took).
template <typename TX, typename TY, int MT>
__global__ __launch_bounds__(512, 4) void k_mx4_gemm_mid(const TX *__restrict__ X, int64_t M, int nb,
                                                         const uint8_t *__restrict__ codes,
                                                         const uint8_t *__restrict__ scales, int64_t out,
                                                         TY *__restrict__ Y)
{
    typedef typename Vec8<TX>::type vec;
    constexpr int BM = 32 * MT, BN = 64, G = 4;
    constexpr int CH = BM * 8 / 128;                   // activation chunks a thread moves in a step
    __shared__ __align__(16) u32x4 lds[2][G][BM * 8];

    int64_t m0, n0;
    if (!tile_of_block((M + BM - 1) / BM, (out + BN - 1) / BN, m0, n0))
        return;
    m0 *= BM;
    n0 *= BN;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, h = lane >> 5, group = wave >> 1, wn = wave & 1, gt = threadIdx.x & 127;
    const int xrow = nb * 64;                          // bytes of an activation row
    const int steps = (nb + 1) / 2, full = nb / 2;

    const uint8_t *const xbase = (const uint8_t *)X + m0 * xrow;
    const uint8_t *const wbase = codes + n0 * nb * 16, *const wsbase = scales + n0 * nb;
    const uint32_t mlast = (uint32_t)(M - 1 - m0 < BM - 1 ? M - 1 - m0 : BM - 1);
    const uint32_t nlast = (uint32_t)(out - 1 - n0 < BN - 1 ? out - 1 - n0 : BN - 1);
    uint32_t xo[CH];
    int xdst[CH];
    const int xq = gt & 7;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const uint32_t row = (gt + i * 128) >> 3;
        xdst[i] = row * 8 + (xq ^ (row & 7));
        xo[i] = (row < mlast ? row : mlast) * (uint32_t)xrow + xq * 16;
    }
    const uint32_t wr = 32 * wn + r, wrow = wr < nlast ? wr : nlast;
    const uint32_t wo = wrow * (uint32_t)nb * 16 + h * 16, wso = wrow * (uint32_t)nb + h;

    f32x16 acc[MT];
    u32x4 xr[CH], w, wnext;
    uint32_t ws, wsnext;
    bool bad = false;

    // steps past the last one are fetched as that one and dropped; for an odd
    // last block see k_mx4_gemm_tile
    auto fetch = [&](int k) {
        k = k < steps ? k : steps - 1;
        const bool end = k >= full;
        const uint32_t xback = end && xq >= 4 ? 64 : 0, wback = end && h ? 1 : 0;
        const uint8_t *const px = xbase + (int64_t)k * 128, *const pw = wbase + (int64_t)k * 32;
        const uint8_t *const ps = wsbase + k * 2;
#pragma unroll
        for (int i = 0; i < CH; ++i)
            xr[i] = *reinterpret_cast<const u32x4 *>(px + (xo[i] - xback));
        wnext = *reinterpret_cast<const u32x4 *>(pw + (wo - 16 * wback));
        wsnext = ps[wso - wback];
    };
    auto stash = [&](int k, int buf) {
        if (k >= full && xq >= 4)
#pragma unroll
            for (int i = 0; i < CH; ++i)
                xr[i] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < CH; ++i)
            lds[buf][group][xdst[i]] = xr[i];
        w = wnext;
        ws = k >= full && h ? 127 : wsnext;
    };
    auto contract = [&]<bool WIDE>() {
#pragma unroll
        for (int a = 0; a < MT; ++a)
            acc[a] = f32x16{};
        fetch(group);
        stash(group, 0);
        __syncthreads();
        int buf = 0;
        for (int k0 = 0; k0 < steps; k0 += G, buf ^= 1) {
            const int k = k0 + group;
            const bool more = k0 + G < steps;
            if (more)
                fetch(k + G);
            if (k < steps) {
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    vec wv;
                    bf16x8 wide;
                    if constexpr (WIDE) {
                        wide = mx4_to_bf16(w[s], mx4_scale(ws));
                    } else if constexpr (std::is_same<TX, f16>::value) {
                        wv = mx4_to_f16(w[s], mx4_scale(ws));
                        bad = bad || !mx4_fits_f16(ws);
                    } else {
                        wv = mx4_to_bf16(w[s], mx4_scale(ws));
                    }
#pragma unroll
                    for (int a = 0; a < MT; ++a) {
                        const int row = 32 * a + r;
                        const u32x4 x = lds[buf][group][row * 8 + ((4 * h + s) ^ (row & 7))];
                        if constexpr (WIDE) {
                            bf16x8 hi, lo;
                            split_f16(__builtin_bit_cast(f16x8, x), hi, lo);
                            acc[a] = mfma32(hi, wide, acc[a]);
                            acc[a] = mfma32(lo, wide, acc[a]);
                        } else {
                            acc[a] = mfma32(__builtin_bit_cast(vec, x), wv, acc[a]);
                        }
                    }
                }
            }
            if (more)
                stash(k + G, buf ^ 1);
            __syncthreads();
        }
    };
    contract.template operator()<false>();
    if constexpr (std::is_same<TX, f16>::value)
        if (__syncthreads_or(bad))                     // scales that fp16 cannot hold
            contract.template operator()<true>();

    // the groups' sums, added in group order
    float *const red = reinterpret_cast<float *>(lds);         // [G][BM][BN]
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            red[(group * BM + 32 * a + 8 * (i / 4) + 4 * h + i % 4) * BN + 32 * wn + r] = acc[a][i];
    __syncthreads();
    const int n = threadIdx.x & (BN - 1);
#pragma unroll
    for (int q = 0; q < BM / 8; ++q) {
        const int m = (threadIdx.x >> 6) + 8 * q;
        float sum = red[m * BN + n];
#pragma unroll
        for (int g = 1; g < G; ++g)
            sum += red[(g * BM + m) * BN + n];
        if (m0 + m < M && n0 + n < out)
            Y[(m0 + m) * out + n0 + n] = static_cast<TY>(sum);
    }
}

// MXFP4 activations. Block: 256 x 256, 4 waves of 128 x 128 (256 accumulator
// registers each, one wave a SIMD). Both operands through LDS: a step is 128
// columns, per row four 16-byte blocks and four scale bytes. Block q of row m
// lies at position q ^ (m / 2 & 3) of the row's 64 bytes: eight rows at a time
// fall on distinct banks. Three buffers: while step k is multiplied, k + 1 is
// complete and k + 2 is on its way, so one barrier a step suffices and the
// first operands of the next step can be read before it.
// Lane (r, h) holds in k-step s of 2 block 2 s + h of its row.
template <typename TY>
__global__ __launch_bounds__(256, 1) void k_mx4_gemm_tile4(const uint8_t *__restrict__ xcodes,
                                                           const uint8_t *__restrict__ xscales, int64_t M, int nb,
                                                           const uint8_t *__restrict__ codes,
                                                           const uint8_t *__restrict__ scales, int64_t out,
                                                           TY *__restrict__ Y)
{
    constexpr int MT = 4, NT = 4, B = 256, ST = 3;
    __shared__ __align__(16) u32x4 lx[ST][B * 4], lw[ST][B * 4];
    __shared__ uint32_t lxs[ST][B], lws[ST][B];

    int64_t m0, n0;
    if (!tile_of_block((M + B - 1) / B, (out + B - 1) / B, m0, n0))
        return;
    m0 *= B;
    n0 *= B;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, h = lane >> 5, wm = wave >> 1, wn = wave & 1;
    const int steps = (nb + 3) / 4, full = nb / 4;

    const uint8_t *const xbase = xcodes + m0 * nb * 16, *const xsbase = xscales + m0 * nb;
    const uint8_t *const wbase = codes + n0 * nb * 16, *const wsbase = scales + n0 * nb;
    const uint32_t mlast = (uint32_t)(M - 1 - m0 < B - 1 ? M - 1 - m0 : B - 1);
    const uint32_t nlast = (uint32_t)(out - 1 - n0 < B - 1 ? out - 1 - n0 : B - 1);
    const int q = threadIdx.x & 3;
    uint32_t xo[4], wo[4];
    int dst[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t row = (threadIdx.x + i * 256) >> 2;
        dst[i] = row * 4 + (q ^ (row >> 1 & 3));
        xo[i] = (row < mlast ? row : mlast) * (uint32_t)nb * 16 + q * 16;
        wo[i] = (row < nlast ? row : nlast) * (uint32_t)nb * 16 + q * 16;
    }
    const uint32_t srow = threadIdx.x;                 // the row whose scales this thread moves
    const uint32_t xso = (srow < mlast ? srow : mlast) * (uint32_t)nb, wso = (srow < nlast ? srow : nlast) * (uint32_t)nb;

    u32x4 xr[4], wr[4];
    uint32_t xsr, wsr;
    // The last step of a row that ends inside it: zeros under scale 1 past the end.
    auto fetch = [&](int k) {
        const uint8_t *const px = xbase + (int64_t)k * 64, *const pw = wbase + (int64_t)k * 64;
        const uint8_t *const pxs = xsbase + k * 4, *const pws = wsbase + k * 4;
        if (k < full) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xr[i] = *reinterpret_cast<const u32x4 *>(px + xo[i]);
                wr[i] = *reinterpret_cast<const u32x4 *>(pw + wo[i]);
            }
            __builtin_memcpy(&xsr, pxs + xso, 4);
            __builtin_memcpy(&wsr, pws + wso, 4);
        } else {
            const int valid = nb - 4 * k;              // 1 .. 3 blocks
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xr[i] = wr[i] = u32x4{0, 0, 0, 0};
                if (q < valid) {
                    xr[i] = *reinterpret_cast<const u32x4 *>(px + xo[i]);
                    wr[i] = *reinterpret_cast<const u32x4 *>(pw + wo[i]);
                }
            }
            xsr = wsr = 0x7F7F7F7Fu;
            for (int i = 0; i < valid; ++i) {
                xsr = (xsr & ~(0xFFu << (8 * i))) | (uint32_t)pxs[xso + i] << (8 * i);
                wsr = (wsr & ~(0xFFu << (8 * i))) | (uint32_t)pws[wso + i] << (8 * i);
            }
        }
    };
    auto stash = [&](int buf) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lx[buf][dst[i]] = xr[i];
            lw[buf][dst[i]] = wr[i];
        }
        lxs[buf][srow] = xsr;
        lws[buf][srow] = wsr;
    };

    f32x16 acc[MT][NT];
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int b = 0; b < NT; ++b)
            acc[a][b] = f32x16{};
    // this lane's rows: 128 wm + 32 a + r and 128 wn + 32 b + r; the swizzle
    // depends on r alone
    const int xr0 = (128 * wm + r) * 4, wr0 = (128 * wn + r) * 4, swz = r >> 1 & 3;

    fetch(0);
    stash(0);
    if (steps > 1)
        fetch(1);
    __syncthreads();
    int cur = 0, nxt = 1;
    for (int k = 0; k < steps; ++k) {
        // step k + 1 (in registers) goes to its buffer, step k + 2 on its way
        if (k + 1 < steps)
            stash(nxt);
        if (k + 2 < steps)
            fetch(k + 2);
        uint32_t sa[MT], sb[NT];
#pragma unroll
        for (int a = 0; a < MT; ++a)
            sa[a] = lxs[cur][128 * wm + 32 * a + r] >> (8 * h);
#pragma unroll
        for (int b = 0; b < NT; ++b)
            sb[b] = lws[cur][128 * wn + 32 * b + r] >> (8 * h);
        u32x4 x[2][MT], w[2][NT];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int p = (2 * s + h) ^ swz;
#pragma unroll
            for (int a = 0; a < MT; ++a)
                x[s][a] = lx[cur][xr0 + 128 * a + p];
#pragma unroll
            for (int b = 0; b < NT; ++b)
                w[s][b] = lw[cur][wr0 + 128 * b + p];
        }
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < NT; ++b)
                acc[a][b] = mfma32<0>(x[0][a], sa[a], w[0][b], sb[b], acc[a][b]);
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < NT; ++b)
                acc[a][b] = mfma32<2>(x[1][a], sa[a], w[1][b], sb[b], acc[a][b]);
        __syncthreads();
        cur = nxt;
        nxt = nxt == ST - 1 ? 0 : nxt + 1;
    }
    store_tiles<TY, MT, NT>(Y, acc, m0 + 128 * wm, n0 + 128 * wn, M, out, r, h);
}

inline int64_t tiles_of(int64_t n, int64_t size) { return (n + size - 1) / size; }
// Whole multiples of 8: see tile_of_block.
inline uint32_t tile_grid(int64_t tiles) { return (uint32_t)((tiles + 7) / 8 * 8); }

template <typename TX, typename TY>
hipError_t gemm(const void *X, const uint8_t *xs, int64_t M, int nb, const uint8_t *codes, const uint8_t *scales,
                int64_t out, void *Y, hipStream_t st)
{
    if constexpr (!std::is_same<TX, Mx4Act>::value) {
        // Enough row tiles for more than a block's worth a unit: few waves a
        // tile (28672 rows of 4096, 4 tokens: S = 1, 2, 4, 8 take 16.4, 15.7,
        // 17.9, 21.1 us; 12288 rows, 2 tokens: 14.4, 10.3, 9.7, 10.9).
        const int64_t tiles = (out + 15) / 16;
        if (M <= 16 && tiles >= 640) {
            if (tiles >= 1280)
                return gemv<TX, TY, 2>(X, (int)M, nb, codes, scales, out, Y, st);
            return gemv<TX, TY, 4>(X, (int)M, nb, codes, scales, out, Y, st);
        }
    }
    if (M <= 16)
        return split<TX, TY, 1, 1, 4>(X, xs, M, nb, codes, scales, out, Y, st);
    if constexpr (std::is_same<TX, Mx4Act>::value) {
        if (tiles_of(M, 256) * tiles_of(out, 256) >= 64) {
            k_mx4_gemm_tile4<TY><<<tile_grid(tiles_of(M, 256) * tiles_of(out, 256)), 256, 0, st>>>(
                (const uint8_t *)X, xs, M, nb, codes, scales, out, (TY *)Y);
            return hipGetLastError();
        }
        return split<TX, TY, 4, 4, 1>(X, xs, M, nb, codes, scales, out, Y, st);
    } else {
        const TX *const x = (const TX *)X;
        TY *const y = (TY *)Y;
        if (tiles_of(M, 128) * tiles_of(out, 256) >= 200)
            k_mx4_gemm_tile<TX, TY><<<tile_grid(tiles_of(M, 128) * tiles_of(out, 256)), 256, 0, st>>>(
                x, M, nb, codes, scales, out, y);
        else if (M <= 32)
            k_mx4_gemm_mid<TX, TY, 1><<<tile_grid(tiles_of(M, 32) * tiles_of(out, 64)), 512, 0, st>>>(
                x, M, nb, codes, scales, out, y);
        else
            k_mx4_gemm_mid<TX, TY, 2><<<tile_grid(tiles_of(M, 64) * tiles_of(out, 64)), 512, 0, st>>>(
                x, M, nb, codes, scales, out, y);
        return hipGetLastError();
    }
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
