// k_mx4_gemm.hip -- products with MXFP4 weights, Y[m][n] = sum_k X[m][k] W[n][k].
//
// Weights enter the matrix instructions as values: bf16 and fp16 hold
// e2m1 * 2^E exactly (fp16 for E in [-13, 13]; elsewhere the fp16 activations
// go as two exact bf16 parts), so the only roundings are those of the fp32
// sums. With MXFP4 activations the scaled matrix instruction takes codes and
// scale bytes as they are. bf16 and fp16 tokens cost about the same (fp16 7 % more
// in `tile`) unless an fp16 product meets such scales: then its share of the work
// is done a second time, at half the rate (blocks of zeros do not count). One
// block of weights below 2^-11, and not 0, in one row of 64 takes 4 tokens x
// 28672x4096 from 20 to 49 us, 64 x 4096x4096 from 10.8 to 21.5, 203 x 4097x4064
// from 22 to 51, 2048 x 28672x4096 from 432 to 1342; in one row of 4096 these take
// 47, 21, 38 and 604. The second pass shares the first one's registers: of the
// fp16 kernels `tile` spills 8 a lane for it, `mid` of 64 x 64 with one buffer 6.
//
// What the forms reach (bf16 unless said; medians of graph replays, 600 MB of
// weights in turn, so that they come from HBM and not from the 256 MB cache
// before it; the choices below were measured with 25 to 310 MB in turn, unless
// they say otherwise):
//   split   1 token    x 4096x4096     5.0 us (a launch alone is 2-3)
//   gemv    4 tokens   x 28672x4096   19 us, 3.3 TB/s
//   mid     64 tokens  x 4096x4096     9.4 us
//   mid     256 tokens x 4096x4096    17.8 us, 480 TFLOP/s
//   tile    2048 tokens x 28672x4096  395 us, 1220 TFLOP/s
//   mid4    1 token    x 4096x4096     5.6 us
//   mid4    4 tokens   x 28672x4096   14.8 us, 4.2 TB/s
//   mid4    256 tokens x 4096x4096    10.5 us, 820 TFLOP/s
//   tile4   2048 tokens x 28672x4096  162 us, 2970 TFLOP/s
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

// Up to 16 tokens, 16-bit activations, few rows. Block: 16 rows, the columns
// split over W waves in items of 128 U, each wave's next item in flight while it
// multiplies the current one. The waves' sums are added in wave order through
// LDS. Bound by latency: 4096x4096 is one item a wave, all of it loaded at once
// and nothing in flight behind it (1 token 5.0 us, 16 tokens 7.8); with many
// tokens by the loads of their rows (4096x14336: 1 token 13.6 us, 16 tokens 23.0).
template <typename TX, typename TY, int U, int W>
__global__ __launch_bounds__(64 * W) void k_mx4_gemm_split(const TX *__restrict__ X, int M, int nb,
                                                           const uint8_t *__restrict__ codes,
                                                           const uint8_t *__restrict__ scales, int64_t out,
                                                           TY *__restrict__ Y)
{
    __shared__ f32x4 red[W * 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, c = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16, n = n0 + r < out ? n0 + r : out - 1;
    const Mx4Rows<TX> rows = {codes + n * nb * 16, scales + n * nb, X + (int64_t)(r < M ? r : M - 1) * nb * 32};
    f32x4 acc;
    mx4_wave<U>(rows, acc, wave * (4 * U), W * (4 * U), nb, c);
    red[wave * 64 + lane] = acc;
    __syncthreads();
    if (wave)
        return;
#pragma unroll
    for (int w = 1; w < W; ++w)
        acc += red[w * 64 + lane];
    store_tile<TX, TY>(Y, 4 * c, n0 + r, M, out, acc);
}

template <typename TX, typename TY, int U, int W>
hipError_t split(const TX *X, int M, int nb, const uint8_t *codes, const uint8_t *scales, int64_t out, TY *Y,
                 hipStream_t st)
{
    k_mx4_gemm_split<TX, TY, U, W><<<dim3((uint32_t)((out + 15) / 16)), 64 * W, 0, st>>>(X, M, nb, codes, scales, out,
                                                                                        Y);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Up to 16 tokens of 16-bit activations, more row tiles than the chip has
// units for a whole block each. Block: 8 / S row tiles of 16, all columns, S
// waves a tile; the activations go through LDS in chunks of kc blocks that all
// waves share. Every wave streams its own weights (see StreamItem), the next
// item in flight also across the chunks' barriers. Bound by how much the waves
// have in flight: 4 tokens x 28672x4096 (62 MB from HBM) 19 us, 3.3 TB/s, where a
// plain read of as much takes 11.6 us, 5.6 TB/s; with the weights partly in the
// last-level cache 16 us.
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
    F16Range range;
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
                stream_compute<WIDE, true>(it, x, acc, nb - i * kStreamBlocks, rows,
                                     i + S < items ? (i + S) * kStreamBlocks : -1, nb, c, range);
            }
        }
    };
    contract.template operator()<false>();
    if constexpr (std::is_same<TX, f16>::value)
        if (__syncthreads_or(range.exceeded()))          // scales that fp16 cannot hold
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
hipError_t gemv(const TX *X, int M, int nb, const uint8_t *codes, const uint8_t *scales, int64_t out, TY *Y,
                hipStream_t st)
{
    const int64_t tiles = (out + 15) / 16;
    k_mx4_gemv<TX, TY, S><<<dim3((uint32_t)((tiles + 8 / S - 1) / (8 / S))), 512, 0, st>>>(
        X, M, nb, stream_chunk(M, nb), codes, scales, out, Y);
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
// range of tiles, 4 token tiles by one row tile at a time, so that what they
// read together stays in that XCD's L2 (the 64 tiles that an XCD has in work read
// 13 MB then; by 16 token tiles 18: 2048 x 28672x4096 16-bit 405 us, 420).
__device__ __forceinline__ bool tile_of_block(int64_t tm, int64_t tn, int64_t &m, int64_t &n)
{
    const int64_t tiles = tm * tn, chunk = (tiles + 7) / 8;
    const int64_t t = (blockIdx.x & 7) * chunk + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= chunk || t >= tiles)
        return false;
    const int64_t band = t / (4 * tn), first = band * 4, in_band = t - band * 4 * tn;
    const int64_t h = tm - first < 4 ? tm - first : 4;
    m = first + in_band % h;
    n = in_band / h;
    return true;
}

// The results of a wave's MT x 2 tiles, tile (a, b) at token m0 + 32 a, row
// n0 + 32 b: register i of lane (r, h) is token 8 (i / 4) + 4 h + i % 4, row r.
// They go through 8 KB of the wave's own LDS, 32 tokens at a time, and out in
// 16-byte pieces, 64 rows of a token together: a store of single values in the
// matrix layout keeps the store unit busy for as long as a 16-byte one.
template <typename TY, int MT>
__device__ __forceinline__ void store_tiles(TY *__restrict__ Y, const f32x16 (&acc)[MT][2], float *lds, int64_t m0,
                                            int64_t n0, int64_t M, int64_t out, int lane)
{
    constexpr int V = 16 / sizeof(TY);                 // values a piece
    typedef TY piece __attribute__((ext_vector_type(V)));
    const int r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int a = 0; a < MT; ++a) {
        // value (t, n) at 64 t + (n ^ (8 (t & 4))): lane halves, 4 tokens apart, use different banks
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int t = 8 * (i / 4) + 4 * h + i % 4;
                lds[64 * t + ((32 * b + r) ^ (8 * (t & 4)))] = acc[a][b][i];
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int k = 0; k < 32 * 64 / V / 64; ++k) {
            const int p = lane + 64 * k, t = p / (64 / V), n = p % (64 / V) * V;
            piece v;
#pragma unroll
            for (int e = 0; e < V; ++e)
                v[e] = static_cast<TY>(lds[64 * t + ((n ^ (8 * (t & 4))) + e)]);
            const int64_t m = m0 + 32 * a + t;
            TY *const y = Y + m * out + n0 + n;
            if (m < M) {
                if (n0 + n + V <= out)
                    __builtin_memcpy(y, &v, 16);       // at any alignment
                else
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (n0 + n + e < out)
                            y[e] = v[e];
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// Eight scale bytes of a row from block b0 on, 127 for those past its end.
__device__ __forceinline__ u32x2 load_scales8(const uint8_t *row, int b0, int nb)
{
    u32x2 v;
    if (b0 + 8 <= nb)
        __builtin_memcpy(&v, row + b0, 8);             // at any alignment
    else
        v = u32x2{mx4_scales4(row, b0, nb), mx4_scales4(row, b0 + 4, nb)};
    return v;
}

// The products below stage both operands through LDS, rows of eight 16-byte
// chunks, chunk q of row m at position q ^ (m & 7): equal chunks of eight
// consecutive rows then lie on distinct banks of 32. Conflicts remain, 0.16 to 0.37
// cycles for every busy LDS cycle (2048 tokens x 28672x4096: 0.37 `tile`, 0.33
// `tile4`); where they come from has not been measured. A load unit takes 64
// cycles for a load whose neighbouring lanes lie in different rows, as a matrix
// operand wants them, whatever its width, and 19 where eight lanes cover 128
// bytes (measured): weights read straight into operand registers, and scales a
// byte or a word at a time, bounded these kernels by their loads.
__device__ __forceinline__ int swizzled(int row, int q) { return row * 8 + (q ^ (row & 7)); }

// 16-bit activations. Block: 128 tokens x 256 rows, 4 waves of 128 x 64. A
// step is 64 columns, 128 bytes of an activation row; weights come by the 256
// columns (128 bytes of codes, 8 of scales) into one buffer that four steps
// use. What comes next is on its way to registers meanwhile; activations have
// two buffers, so a step costs one barrier, and a fourth one more. Weights are
// converted by the wave that multiplies them (no other one has its rows), once
// for 128 tokens. 2048 tokens x 28672x4096: 395 us, 1220 TFLOP/s (8192 tokens:
// 1260), the matrix units busy for 57 % of it, LDS for 46 %; a dense bf16 library
// product of the shape takes 368 us.
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
    constexpr int CX = BM * 8 / 256, CW = BN * 8 / 256;        // chunks a thread moves
    __shared__ __align__(16) u32x4 lx[2][BM * 8], lw[BN * 8];
    __shared__ u32x2 lws[BN];

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
    const int q = threadIdx.x & 7, row0 = threadIdx.x >> 3;    // this thread's chunk of rows row0 + 32 i
    uint32_t xo[CX], wo[CW];
#pragma unroll
    for (int i = 0; i < CX; ++i) {
        const uint32_t row = row0 + 32 * i;
        xo[i] = (row < mlast ? row : mlast) * (uint32_t)xrow + q * 16;
    }
#pragma unroll
    for (int i = 0; i < CW; ++i) {
        const uint32_t row = row0 + 32 * i;
        wo[i] = (row < nlast ? row : nlast) * (uint32_t)nb * 16 + q * 16;
    }
    const uint32_t wso = (threadIdx.x < nlast ? threadIdx.x : nlast) * (uint32_t)nb;
    const int dst = swizzled(row0, q);                 // rows 32 apart: 256 chunks apart, swizzled alike

    f32x16 acc[MT][NT];
    u32x4 xr[CX], wr[CW];
    u32x2 wsr, ws[NT];
    F16Range range;

    // Past a row's end (in its last step or stretch) the last chunk there is is
    // loaded instead; zeros take its place among the activations, 127 (2^0)
    // among the scales.
    auto fetch_x = [&](int k) {
        const uint32_t back = k >= full && q >= 4 ? 64 : 0;
        const uint8_t *const p = xbase + (int64_t)k * 128;
#pragma unroll
        for (int i = 0; i < CX; ++i)
            xr[i] = *reinterpret_cast<const u32x4 *>(p + (xo[i] - back));
    };
    auto stash_x = [&](int k) {
        if (k >= full && q >= 4)
#pragma unroll
            for (int i = 0; i < CX; ++i)
                xr[i] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < CX; ++i)
            lx[k & 1][dst + 256 * i] = xr[i];
    };
    auto fetch_w = [&](int j) {                        // columns 256 j ...
        const int over = 8 * j + q - (nb - 1);
        const uint32_t back = over > 0 ? over * 16 : 0;
        const uint8_t *const p = wbase + (int64_t)j * 128;
#pragma unroll
        for (int i = 0; i < CW; ++i)
            wr[i] = *reinterpret_cast<const u32x4 *>(p + (wo[i] - back));
        wsr = load_scales8(wsbase + wso, 8 * j, nb);
    };
    auto stash_w = [&] {
#pragma unroll
        for (int i = 0; i < CW; ++i)
            lw[dst + 256 * i] = wr[i];
        lws[threadIdx.x] = wsr;
    };
    auto contract = [&]<bool WIDE>() {
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < NT; ++b)
                acc[a][b] = f32x16{};
        fetch_w(0);
        fetch_x(0);
        stash_w();
        stash_x(0);
        __syncthreads();
        for (int k = 0; k < steps; ++k) {
            const int part = k & 3;
            if (part == 0) {
                if (k + 4 < steps)
                    fetch_w(k / 4 + 1);
#pragma unroll
                for (int b = 0; b < NT; ++b)
                    ws[b] = lws[64 * wave + 32 * b + r];
            }
            if (k + 1 < steps)
                fetch_x(k + 1);
            u32x4 w[NT];
            uint32_t byte[NT];
#pragma unroll
            for (int b = 0; b < NT; ++b) {
                w[b] = lw[swizzled(64 * wave + 32 * b + r, 2 * part + h)];
                byte[b] = (part & 2 ? ws[b][1] : ws[b][0]) >> (16 * (part & 1) + 8 * h) & 0xFFu;
                if constexpr (std::is_same<TX, f16>::value && !WIDE)
                    range.see(w[b], byte[b]);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if constexpr (!WIDE) {
                    vec wv[NT];
#pragma unroll
                    for (int b = 0; b < NT; ++b) {
                        if constexpr (std::is_same<TX, f16>::value)
                            wv[b] = mx4_to_f16(w[b][s], mx4_scale(byte[b]));
                        else
                            wv[b] = mx4_to_bf16(w[b][s], mx4_scale(byte[b]));
                    }
#pragma unroll
                    for (int a = 0; a < MT; ++a) {
                        const vec x = __builtin_bit_cast(vec, lx[k & 1][swizzled(32 * a + r, 4 * h + s)]);
#pragma unroll
                        for (int b = 0; b < NT; ++b)
                            acc[a][b] = mfma32(x, wv[b], acc[a][b]);
                    }
                } else {
                    __builtin_amdgcn_sched_barrier(0);
                    bf16x8 wv[NT];
#pragma unroll
                    for (int b = 0; b < NT; ++b)
                        wv[b] = mx4_to_bf16(w[b][s], mx4_scale(byte[b]));
#pragma unroll
                    for (int a = 0; a < MT; ++a) {
                        bf16x8 hi, lo;
                        split_f16(__builtin_bit_cast(f16x8, lx[k & 1][swizzled(32 * a + r, 4 * h + s)]), hi, lo);
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
                stash_x(k + 1);
            __syncthreads();
            if (part == 3 && k + 1 < steps) {          // everyone has read the last of the weights
                stash_w();
                __syncthreads();
            }
        }
    };
    contract.template operator()<false>();
    // fp16 activations under scales that fp16 cannot hold: all of it once more
    // in the wide form (weights in bf16, activations as two bf16 parts)
    if constexpr (std::is_same<TX, f16>::value)
        if (__syncthreads_or(range.exceeded()))
            contract.template operator()<true>();
    // every wave is past its last read of the operands
    store_tiles<TY, MT>(Y, acc, reinterpret_cast<float *>(lx) + 2048 * wave, m0, n0 + 64 * wave, M, out, lane);
}

// The sums of G groups of 8 / G waves (32 rows each) to Y, added in a fixed
// order: the upper half of the groups to the lower, until two are left.
template <int G, typename TY, int MT>
__device__ __forceinline__ void add_groups(float (&red)[G / 2][32 * MT][256 / G], f32x16 (&acc)[MT], int group, int wn,
                                           int r, int h, TY *__restrict__ Y, int64_t m0, int64_t n0, int64_t M,
                                           int64_t out)
{
    constexpr int BN = 256 / G;
    auto put = [&](int g) {
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                red[g][32 * a + 8 * (i / 4) + 4 * h + i % 4][32 * wn + r] = acc[a][i];
    };
#pragma unroll
    for (int n = G / 2; n >= 2; n /= 2) {
        if (group >= n && group < 2 * n)
            put(group - n);
        __syncthreads();
        if (group < n)
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[a][i] += red[group][32 * a + 8 * (i / 4) + 4 * h + i % 4][32 * wn + r];
        __syncthreads();
    }
    if (group < 2)
        put(group);
    __syncthreads();
    const int n = threadIdx.x % BN;
#pragma unroll
    for (int i = 0; i < 32 * MT * BN / 512; ++i) {
        const int m = threadIdx.x / BN + 512 / BN * i;
        const float sum = red[0][m][n] + red[1][m][n];
        if (m0 + m < M && n0 + n < out)
            Y[(m0 + m) * out + n0 + n] = static_cast<TY>(sum);
    }
}

// 16-bit activations, too few 128 x 256 tiles for the chip. Block: 32 MT tokens
// x 256 / G rows, 8 waves: G groups of 32 rows a wave. A round is 64 G columns,
// of which each group takes 64; the groups' sums meet in LDS. Such shapes leave
// one block or two on a unit, so a round's loads go out two rounds ahead. BUF
// LDS buffers: two need one barrier a round, one leaves room for a second block.
// A round's loads and its LDS accesses, about 500 cycles each for 32 x 64, are
// what bounds it, and waits where they do not overlap (203 tokens x 4097x4064
// 21 us, 320 TFLOP/s; 64 tokens x 4096x14336 27 us).
template <typename TX, typename TY, int MT, int G, int BUF>
__global__ __launch_bounds__(512, BUF == 2 && MT * G == 8 ? 2 : 4) void k_mx4_gemm_mid(
    const TX *__restrict__ X, int64_t M, int nb, const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
    int64_t out, TY *__restrict__ Y)
{
    typedef typename Vec8<TX>::type vec;
    constexpr int BM = 32 * MT, BN = 256 / G, GT = 512 / G;     // GT: threads of a group
    constexpr int CX = BM * 8 / GT;                    // activation chunks a thread moves in a round
    union Lds {
        struct {
            u32x4 x[G][BM * 8], w[G / 4][BN * 8];     // of a weight row 8 chunks each
            u32x2 ws[G / 4][BN];
        } in[BUF];
        float red[G / 2][BM][BN];
    };
    __shared__ __align__(16) Lds lds;

    int64_t m0, n0;
    if (!tile_of_block((M + BM - 1) / BM, (out + BN - 1) / BN, m0, n0))
        return;
    m0 *= BM;
    n0 *= BN;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, h = lane >> 5, group = wave / (8 / G), wn = wave % (8 / G);
    const int xrow = nb * 64;                          // bytes of an activation row
    const int rounds = (nb + 2 * G - 1) / (2 * G);

    // addresses and row ends as in k_mx4_gemm_tile
    const uint8_t *const xbase = (const uint8_t *)X + m0 * xrow;
    const uint8_t *const wbase = codes + n0 * nb * 16, *const wsbase = scales + n0 * nb;
    const uint32_t mlast = (uint32_t)(M - 1 - m0 < BM - 1 ? M - 1 - m0 : BM - 1);
    const uint32_t nlast = (uint32_t)(out - 1 - n0 < BN - 1 ? out - 1 - n0 : BN - 1);
    const int q = threadIdx.x & 7, xrow0 = threadIdx.x % GT >> 3;
    const int wq = threadIdx.x % (2 * G);              // chunk of weight row wrow
    const uint32_t wrow = threadIdx.x / (2 * G), wsrow = threadIdx.x % BN;
    const int wshalf = threadIdx.x / BN;               // below G / 4: eight scales of row wsrow
    uint32_t xo[CX];
#pragma unroll
    for (int i = 0; i < CX; ++i) {
        const uint32_t row = xrow0 + GT / 8 * i;
        xo[i] = (row < mlast ? row : mlast) * (uint32_t)xrow + q * 16;
    }
    const uint32_t wo = (wrow < nlast ? wrow : nlast) * (uint32_t)nb * 16 + wq * 16;
    const uint32_t wso = (wsrow < nlast ? wsrow : nlast) * (uint32_t)nb;

    f32x16 acc[MT];
    struct Round {
        u32x4 x[CX], w;
        u32x2 ws;
    } even, odd;
    F16Range range;

    auto fetch = [&](Round &to, int j) {
        if (j >= rounds)
            return;
        const int b0 = 2 * G * j, xb = b0 + 2 * group + (q >> 2);      // xb: its block of the row
        const int xover = (xb - (nb - 1)) * 64;
        const int wover = (b0 + wq - (nb - 1)) * 16;
        const uint8_t *const px = xbase + (int64_t)b0 * 64 + group * 128, *const pw = wbase + (int64_t)b0 * 16;
#pragma unroll
        for (int i = 0; i < CX; ++i)
            to.x[i] = *reinterpret_cast<const u32x4 *>(px + ((int64_t)xo[i] - (xover > 0 ? xover : 0)));
        to.w = *reinterpret_cast<const u32x4 *>(pw + ((int64_t)wo - (wover > 0 ? wover : 0)));
        if (wshalf < G / 4)
            to.ws = load_scales8(wsbase + wso, b0 + 8 * wshalf, nb);
    };
    auto stash = [&](Round &from, int j) {
        if (j >= rounds)
            return;
        auto &in = lds.in[j % BUF];
        if (2 * G * j + 2 * group + (q >> 2) >= nb)
#pragma unroll
            for (int i = 0; i < CX; ++i)
                from.x[i] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < CX; ++i)
            in.x[group][swizzled(xrow0 + GT / 8 * i, q)] = from.x[i];
        in.w[wq >> 3][swizzled(wrow, wq & 7)] = from.w;
        if (wshalf < G / 4)
            in.ws[wshalf][wsrow] = from.ws;
    };
    auto contract = [&]<bool WIDE>() {
#pragma unroll
        for (int a = 0; a < MT; ++a)
            acc[a] = f32x16{};
        auto round = [&](Round &next, int j) {         // next: round j + 1 (one buffer: j)
            if constexpr (BUF == 1) {
                stash(next, j);
                __syncthreads();
                fetch(next, j + 2);
            }
            auto &in = lds.in[j % BUF];
            const u32x4 w = in.w[group >> 2][swizzled(32 * wn + r, 2 * (group & 3) + h)];
            const u32x2 ws = in.ws[group >> 2][32 * wn + r];
            const uint32_t byte = (group & 2 ? ws[1] : ws[0]) >> (16 * (group & 1) + 8 * h) & 0xFFu;
            if constexpr (std::is_same<TX, f16>::value && !WIDE)
                range.see(w, byte);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                vec wv;
                bf16x8 wide;
                if constexpr (WIDE)
                    wide = mx4_to_bf16(w[s], mx4_scale(byte));
                else if constexpr (std::is_same<TX, f16>::value)
                    wv = mx4_to_f16(w[s], mx4_scale(byte));
                else
                    wv = mx4_to_bf16(w[s], mx4_scale(byte));
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    const u32x4 x = in.x[group][swizzled(32 * a + r, 4 * h + s)];
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
            if constexpr (BUF == 2) {
                stash(next, j + 1);
                fetch(next, j + 3);
            }
            __syncthreads();
        };
        fetch(even, 0);
        fetch(odd, 1);
        if constexpr (BUF == 2) {
            stash(even, 0);
            fetch(even, 2);
            __syncthreads();
        }
        for (int j = 0; j < rounds; j += 2) {
            round(BUF == 2 ? odd : even, j);
            if (j + 1 < rounds)
                round(BUF == 2 ? even : odd, j + 1);
        }
    };
    contract.template operator()<false>();
    if constexpr (std::is_same<TX, f16>::value)
        if (__syncthreads_or(range.exceeded()))                     // scales that fp16 cannot hold
            contract.template operator()<true>();

    add_groups<G, TY, MT>(lds.red, acc, group, wn, r, h, Y, m0, n0, M, out);
}

// The scale bytes h, h + 2, h + 4, h + 6 of eight: those of lane (r, h)'s blocks
// in four k-steps, one register.
__device__ __forceinline__ uint32_t own_scales(const u32x2 &s, int h)
{
    return __builtin_amdgcn_perm(s[1], s[0], 0x06040200u + 0x01010101u * (uint32_t)h);
}

// MXFP4 activations. Block: 256 x 256, 8 waves of 128 x 64. A stage is 256
// columns, 128 bytes of codes of every row, in one of two LDS buffers; scales
// come by four stages, 32 bytes of a row, into one of two halves (a load of
// scales costs a load unit the same whatever its width). What comes next is on
// its way to registers meanwhile. (Four waves of 128 x 128 read a third less from
// LDS, but alone on their SIMDs they wait for it: 181 us.) 2048 tokens x 28672x4096: 162
// us, 2970 TFLOP/s. A stage is 2048 cycles of the matrix units and 2500 of LDS,
// which overlap in part (3700).
// Lane (r, h) holds in k-step s of 4 block 2 s + h of its row.
template <typename TY>
__global__ __launch_bounds__(512, 2) void k_mx4_gemm_tile4(const uint8_t *__restrict__ xcodes,
                                                           const uint8_t *__restrict__ xscales, int64_t M, int nb,
                                                           const uint8_t *__restrict__ codes,
                                                           const uint8_t *__restrict__ scales, int64_t out,
                                                           TY *__restrict__ Y)
{
    constexpr int MT = 4, NT = 2, B = 256, CH = 4;
    __shared__ __align__(16) u32x4 lx[2][B * 8], lw[2][B * 8];
    __shared__ u32x2 ls[8][2 * B];                     // scales of stage k at k & 7: activation rows, then weight rows

    int64_t m0, n0;
    if (!tile_of_block((M + B - 1) / B, (out + B - 1) / B, m0, n0))
        return;
    m0 *= B;
    n0 *= B;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, h = lane >> 5, wm = wave >> 2, wn = wave & 3;
    const int stages = (nb + 7) / 8;

    // addresses as in k_mx4_gemm_tile
    const uint8_t *const xbase = xcodes + m0 * nb * 16, *const xsbase = xscales + m0 * nb;
    const uint8_t *const wbase = codes + n0 * nb * 16, *const wsbase = scales + n0 * nb;
    const uint32_t mlast = (uint32_t)(M - 1 - m0 < B - 1 ? M - 1 - m0 : B - 1);
    const uint32_t nlast = (uint32_t)(out - 1 - n0 < B - 1 ? out - 1 - n0 : B - 1);
    const int q = threadIdx.x & 7, row0 = threadIdx.x >> 3;    // this thread's chunk of rows row0 + 64 i
    uint32_t xo[CH], wo[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const uint32_t row = row0 + 64 * i;
        xo[i] = (row < mlast ? row : mlast) * (uint32_t)nb * 16 + q * 16;
        wo[i] = (row < nlast ? row : nlast) * (uint32_t)nb * 16 + q * 16;
    }
    // the row whose scales this thread moves
    const uint32_t srow = threadIdx.x & (B - 1), slast = threadIdx.x < B ? mlast : nlast;
    const uint8_t *const sp = (threadIdx.x < B ? xsbase : wsbase) + (srow < slast ? srow : slast) * (uint32_t)nb;
    const int dst = swizzled(row0, q);

    u32x4 xr[CH], wr[CH];
    u32x2 sr[4];
    // past a row's end its last chunk is loaded; zeros, under scale 1, take its place
    auto fetch = [&](int k) {
        const int over = 8 * k + q - (nb - 1);
        const uint32_t back = over > 0 ? over * 16 : 0;
        const uint8_t *const px = xbase + (int64_t)k * 128, *const pw = wbase + (int64_t)k * 128;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            xr[i] = *reinterpret_cast<const u32x4 *>(px + (int64_t)(xo[i] - back));
            wr[i] = *reinterpret_cast<const u32x4 *>(pw + (int64_t)(wo[i] - back));
        }
    };
    auto fetch_s = [&](int k) {                        // of stages k ... k + 3
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sr[i] = load_scales8(sp, 8 * (k + i), nb);
    };
    auto stash_s = [&](int k) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            ls[(k & 4) + i][threadIdx.x] = sr[i];
    };
    auto stash = [&](int k) {
        if (8 * k + q >= nb)
#pragma unroll
            for (int i = 0; i < CH; ++i)
                xr[i] = wr[i] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            lx[k & 1][dst + 512 * i] = xr[i];
            lw[k & 1][dst + 512 * i] = wr[i];
        }
    };

    f32x16 acc[MT][NT];
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int b = 0; b < NT; ++b)
            acc[a][b] = f32x16{};

    // k-step s + 1's operands are read while k-step s is multiplied, and the last
    // k-step of a stage is multiplied behind the barrier, while the first
    // operands of the next stage are on their way.
    uint32_t sa[MT], sb[NT];
    u32x4 x[2][MT], w[2][NT];
    auto read_s = [&](int k) {
#pragma unroll
        for (int a = 0; a < MT; ++a)
            sa[a] = own_scales(ls[k & 7][128 * wm + 32 * a + r], h);
#pragma unroll
        for (int b = 0; b < NT; ++b)
            sb[b] = own_scales(ls[k & 7][B + 64 * wn + 32 * b + r], h);
    };
    auto read = [&](int k, int s) {
#pragma unroll
        for (int a = 0; a < MT; ++a)
            x[s & 1][a] = lx[k & 1][swizzled(128 * wm + 32 * a + r, 2 * s + h)];
#pragma unroll
        for (int b = 0; b < NT; ++b)
            w[s & 1][b] = lw[k & 1][swizzled(64 * wn + 32 * b + r, 2 * s + h)];
        asm volatile("" ::: "memory");                 // in this order: two sets of operands, no more
        __builtin_amdgcn_sched_barrier(0);
    };
    auto multiply = [&]<int S>() {
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < NT; ++b)
                acc[a][b] = mfma32<S>(x[S & 1][a], sa[a], w[S & 1][b], sb[b], acc[a][b]);
        // here, not after all reads of the stage (the products have no place of
        // their own among the memory accesses)
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < NT; ++b)
                asm volatile("" : "+v"(acc[a][b])::"memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    fetch(0);
    fetch_s(0);
    stash(0);
    stash_s(0);
    if (1 < stages)
        fetch(1);
    __syncthreads();
    read_s(0);
    read(0, 0);
#pragma unroll 1
    for (int k = 0; k < stages; ++k) {
        if ((k & 3) == 1 && (k | 3) + 1 < stages)
            fetch_s((k | 3) + 1);
        read(k, 1);
        multiply.template operator()<0>();
        read(k, 2);
        multiply.template operator()<1>();
        read(k, 3);
        if (k + 1 < stages) {
            stash(k + 1);
            if ((k & 3) == 3)
                stash_s(k + 1);
            if (k + 2 < stages)
                fetch(k + 2);
        }
        multiply.template operator()<2>();
        __syncthreads();
        if (k + 1 < stages)
            read(k + 1, 0);
        multiply.template operator()<3>();
        if (k + 1 < stages)
            read_s(k + 1);
    }
    // every wave is past its last read of the operands
    store_tiles<TY, MT>(Y, acc, reinterpret_cast<float *>(lx) + 2048 * wave, m0 + 128 * wm, n0 + 64 * wn, M, out, lane);
}

// MXFP4 activations, too few 256 x 256 tiles for the chip, or few tokens. Block:
// 32 MT tokens x 256 / G rows, 8 waves: G groups of 32 rows a wave. A round is
// 256 G columns, of which each group takes 256; the groups' sums meet in LDS.
// 256 tokens x 4096x4096 10.5 us (four rounds: latency), 256 tokens x 4096x14336
// 35 us, 855 TFLOP/s (28.7 with the weights in the last-level cache): bound by a
// round's loads and LDS accesses one after the other. (A second buffer and loads
// two rounds ahead: 11.1 and, from the cache, 27.1 us.) Up to 16 tokens too, by
// tiles of 32 (1 and 16 tokens: 4096x4096 5.6 and 5.8 us, 28672x4096 14.7 and 15.8).
template <typename TY, int MT, int G>
__global__ __launch_bounds__(512, 4) void k_mx4_gemm_mid4(const uint8_t *__restrict__ xcodes,
                                                          const uint8_t *__restrict__ xscales, int64_t M, int nb,
                                                          const uint8_t *__restrict__ codes,
                                                          const uint8_t *__restrict__ scales, int64_t out,
                                                          TY *__restrict__ Y)
{
    constexpr int BM = 32 * MT, BN = 256 / G, GT = 512 / G, CX = BM * 8 / GT, CW = BN * 8 / GT;
    static_assert(BM + BN <= GT);                      // a thread moves one row's scales
    union Lds {
        struct {
            u32x4 x[G][BM * 8], w[G][BN * 8];
            u32x2 xs[G][BM], ws[G][BN];
        } in;
        float red[G / 2][BM][BN];
    };
    __shared__ __align__(16) Lds lds;

    int64_t m0, n0;
    if (!tile_of_block((M + BM - 1) / BM, (out + BN - 1) / BN, m0, n0))
        return;
    m0 *= BM;
    n0 *= BN;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, h = lane >> 5, group = wave / (8 / G), wn = wave % (8 / G);
    const int rounds = (nb + 8 * G - 1) / (8 * G);

    // addresses as in k_mx4_gemm_tile; a group's threads move its columns
    const uint8_t *const xbase = xcodes + m0 * nb * 16, *const xsbase = xscales + m0 * nb;
    const uint8_t *const wbase = codes + n0 * nb * 16, *const wsbase = scales + n0 * nb;
    const uint32_t mlast = (uint32_t)(M - 1 - m0 < BM - 1 ? M - 1 - m0 : BM - 1);
    const uint32_t nlast = (uint32_t)(out - 1 - n0 < BN - 1 ? out - 1 - n0 : BN - 1);
    const int gt = threadIdx.x % GT, q = gt & 7, row0 = gt >> 3;       // chunk q of rows row0 + GT / 8 i
    uint32_t xo[CX], wo[CW];
#pragma unroll
    for (int i = 0; i < CX; ++i) {
        const uint32_t row = row0 + GT / 8 * i;
        xo[i] = (row < mlast ? row : mlast) * (uint32_t)nb * 16 + q * 16;
    }
#pragma unroll
    for (int i = 0; i < CW; ++i) {
        const uint32_t row = row0 + GT / 8 * i;
        wo[i] = (row < nlast ? row : nlast) * (uint32_t)nb * 16 + q * 16;
    }
    // scales: the group's first BN threads a weight row each, the others an activation row
    const uint32_t wso = ((uint32_t)gt < nlast ? (uint32_t)gt : nlast) * (uint32_t)nb;
    const uint32_t xso = ((uint32_t)(gt - BN) < mlast ? (uint32_t)(gt - BN) : mlast) * (uint32_t)nb;

    f32x16 acc[MT];
#pragma unroll
    for (int a = 0; a < MT; ++a)
        acc[a] = f32x16{};
    u32x4 xr[CX], wr[CW];
    u32x2 sr;
    auto fetch = [&](int j) {                          // zeros, under scale 1, past a row's end
        const int b0 = 8 * G * j + 8 * group;             // the group's first block
        const uint8_t *const px = xbase + (int64_t)b0 * 16, *const pw = wbase + (int64_t)b0 * 16;
        if (b0 + 8 <= nb) {
#pragma unroll
            for (int i = 0; i < CX; ++i)
                xr[i] = *reinterpret_cast<const u32x4 *>(px + xo[i]);
#pragma unroll
            for (int i = 0; i < CW; ++i)
                wr[i] = *reinterpret_cast<const u32x4 *>(pw + wo[i]);
        } else {
#pragma unroll
            for (int i = 0; i < CX; ++i) {
                xr[i] = u32x4{0, 0, 0, 0};
                if (b0 + q < nb)
                    xr[i] = *reinterpret_cast<const u32x4 *>(px + xo[i]);
            }
#pragma unroll
            for (int i = 0; i < CW; ++i) {
                wr[i] = u32x4{0, 0, 0, 0};
                if (b0 + q < nb)
                    wr[i] = *reinterpret_cast<const u32x4 *>(pw + wo[i]);
            }
        }
        if (gt < BN)
            sr = load_scales8(wsbase + wso, b0, nb);
        else if (gt < BN + BM)
            sr = load_scales8(xsbase + xso, b0, nb);
    };
    fetch(0);
    for (int j = 0; j < rounds; ++j) {
        if (j)
            __syncthreads();
#pragma unroll
        for (int i = 0; i < CX; ++i)
            lds.in.x[group][swizzled(row0 + GT / 8 * i, q)] = xr[i];
#pragma unroll
        for (int i = 0; i < CW; ++i)
            lds.in.w[group][swizzled(row0 + GT / 8 * i, q)] = wr[i];
        if (gt < BN)
            lds.in.ws[group][gt] = sr;
        else if (gt < BN + BM)
            lds.in.xs[group][gt - BN] = sr;
        __syncthreads();
        if (j + 1 < rounds)
            fetch(j + 1);
        uint32_t sa[MT];
#pragma unroll
        for (int a = 0; a < MT; ++a)
            sa[a] = own_scales(lds.in.xs[group][32 * a + r], h);
        const uint32_t sb = own_scales(lds.in.ws[group][32 * wn + r], h);
        auto kstep = [&]<int S>() {
            const u32x4 w = lds.in.w[group][swizzled(32 * wn + r, 2 * S + h)];
#pragma unroll
            for (int a = 0; a < MT; ++a)
                acc[a] = mfma32<S>(lds.in.x[group][swizzled(32 * a + r, 2 * S + h)], sa[a], w, sb, acc[a]);
        };
        kstep.template operator()<0>();
        kstep.template operator()<1>();
        kstep.template operator()<2>();
        kstep.template operator()<3>();
    }
    __syncthreads();
    add_groups<G, TY, MT>(lds.red, acc, group, wn, r, h, Y, m0, n0, M, out);
}

inline int64_t tiles_of(int64_t n, int64_t size) { return (n + size - 1) / size; }
// Whole multiples of 8: see tile_of_block.
inline uint32_t tile_grid(int64_t tiles) { return (uint32_t)((tiles + 7) / 8 * 8); }

// The tiles of the kernels for mid sizes. 32 tokens x 32 rows where that makes no
// more than a block a unit (16-bit, 64 x 4096x4096: 9.7 us, 64 x 64 tiles 12.4;
// 64 x 4096x14336: 23, 34; 128 x 4096x4096, 512 such blocks: 17.0, and 12.8 by
// 32 x 64). Else 64 tokens x 64 rows or 32: a block's time is about 1 to 0.6,
// and a unit does its blocks one after another.
template <typename F> void mid_shape(int64_t M, int64_t out, F run)
{
    const int64_t n = tiles_of(out, 64);
    const int64_t two = tiles_of(tiles_of(M, 64) * n, 256), one = tiles_of(tiles_of(M, 32) * n, 256);
    if (tiles_of(M, 32) * tiles_of(out, 32) <= 256)
        run.template operator()<1, 8>(tile_grid(tiles_of(M, 32) * tiles_of(out, 32)));
    else if (M > 32 && two * 10 <= one * 6)
        run.template operator()<2, 4>(tile_grid(tiles_of(M, 64) * n));
    else
        run.template operator()<1, 4>(tile_grid(tiles_of(M, 32) * n));
}

template <typename TX, typename TY>
hipError_t gemm(const TX *X, int64_t M, int nb, const uint8_t *codes, const uint8_t *scales, int64_t out, TY *Y,
                hipStream_t st)
{
    if (M <= 16) {
        // Enough row tiles for more than a block's worth a unit: few waves a
        // tile (600 MB in turn, 4 tokens, gemv with S = 1, 2, 4, 8, then split, us:
        // 28672 rows of 4096 20.4, 17.7, 20.7, 25.2, 33.1; 12288 rows 18.6, 12.7,
        // 11.3, 12.9, 15.4). Fewer rows: split (4096x4096, 1, 4, 16 tokens 5.0, 5.8,
        // 7.8, gemv with S = 8 6.5, 6.7, 10.3; 4096x14336 13.5, 15.4, 22.6, gemv 19.8,
        // 20.7, 37.9). Above 16 tokens `mid`, whose time hardly depends on the
        // tokens: 4096x4096 8.7, 4096x14336 25.5, 28672x4096 20.9 at 16 tokens, gemv
        // 20.1. In between it is not the best everywhere: 8192x4096, from 4 tokens on
        // split takes 10.8 to 14.9 where `mid` takes 10.0 and gemv, to 8 tokens, 9.5.
        const int64_t tiles = tiles_of(out, 16);
        if (tiles >= 1280)
            return gemv<TX, TY, 2>(X, (int)M, nb, codes, scales, out, Y, st);
        if (tiles >= 640)
            return gemv<TX, TY, 4>(X, (int)M, nb, codes, scales, out, Y, st);
        return split<TX, TY, 4, 8>(X, (int)M, nb, codes, scales, out, Y, st);
    }
    // 128 x 256 tiles or 64 x 64 ones: 4096 columns take 31 us for up to 512 of
    // the small tiles and each further 512; large ones 80 us for up to 256 (one
    // a unit), 100 for each 512 (1024 x 4096 rows: 60 us small, 80 large; 2048 x
    // 4096: 120, 79)
    const int64_t large = tiles_of(M, 128) * tiles_of(out, 256);
    const int64_t small = tiles_of(tiles_of(M, 64) * tiles_of(out, 64), 512);
    if ((large <= 256 ? 80 : 100 * tiles_of(large, 512)) < 31 * small)
        k_mx4_gemm_tile<TX, TY><<<tile_grid(large), 256, 0, st>>>(X, M, nb, codes, scales, out, Y);
    else
        mid_shape(M, out, [&]<int MT, int G>(uint32_t blocks) {
            // two blocks a unit against one with two buffers (4096 columns: 512
            // blocks 30 us, 33; 256 blocks 19.6, 17.8)
            if constexpr (MT == 2)
                if (blocks > 256) {
                    k_mx4_gemm_mid<TX, TY, MT, G, 1><<<blocks, 512, 0, st>>>(X, M, nb, codes, scales, out, Y);
                    return;
                }
            k_mx4_gemm_mid<TX, TY, MT, G, 2><<<blocks, 512, 0, st>>>(X, M, nb, codes, scales, out, Y);
        });
    return hipGetLastError();
}

template <typename TY>
hipError_t gemm_a4(const uint8_t *xc, const uint8_t *xs, int64_t M, int nb, const uint8_t *codes, const uint8_t *scales,
                   int64_t out, TY *Y, hipStream_t st)
{
    // 256 x 256 tiles or 64 x 64 ones: 4096 columns take 36 us for each 256 of the
    // large, 13 for each 512 of the small (1024 x 4096 rows: 28 us small, 35
    // large; 2048 x 4096: 52, 36)
    if (3 * tiles_of(tiles_of(M, 256) * tiles_of(out, 256), 256) < tiles_of(tiles_of(M, 64) * tiles_of(out, 64), 512))
        k_mx4_gemm_tile4<TY><<<tile_grid(tiles_of(M, 256) * tiles_of(out, 256)), 512, 0, st>>>(xc, xs, M, nb, codes,
                                                                                             scales, out, Y);
    else
        mid_shape(M, out, [&]<int MT, int G>(uint32_t blocks) {
            k_mx4_gemm_mid4<TY, MT, G><<<blocks, 512, 0, st>>>(xc, xs, M, nb, codes, scales, out, Y);
        });
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx4_gemm(const void *X, int dtype, int64_t M, int64_t in, const uint8_t *codes, const uint8_t *scales,
                           int64_t out, void *Y, bool yf32, hipStream_t st)
{
    const int nb = (int)(in / kMxBlock);
    if (dtype == AWQ_F16)
        return yf32 ? gemm((const f16 *)X, M, nb, codes, scales, out, (float *)Y, st)
                    : gemm((const f16 *)X, M, nb, codes, scales, out, (f16 *)Y, st);
    return yf32 ? gemm((const bf16 *)X, M, nb, codes, scales, out, (float *)Y, st)
                : gemm((const bf16 *)X, M, nb, codes, scales, out, (bf16 *)Y, st);
}

hipError_t launch_mx4_gemm_a4(const uint8_t *xcodes, const uint8_t *xscales, int64_t M, int64_t in,
                              const uint8_t *codes, const uint8_t *scales, int64_t out, void *Y, int y_dtype,
                              hipStream_t st)
{
    const int nb = (int)(in / kMxBlock);
    switch (y_dtype) {
    case AWQ_F32: return gemm_a4(xcodes, xscales, M, nb, codes, scales, out, (float *)Y, st);
    case AWQ_F16: return gemm_a4(xcodes, xscales, M, nb, codes, scales, out, (f16 *)Y, st);
    default: return gemm_a4(xcodes, xscales, M, nb, codes, scales, out, (bf16 *)Y, st);
    }
}

}  // namespace awq
