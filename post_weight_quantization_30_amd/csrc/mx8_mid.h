// mx8_mid.h -- products of MXFP8 activations and MXFP4 weights with too few large tiles for
// the chip.
//
// Block: 32 tokens x 32 NT weight rows, four waves that share the columns: wave p takes
// stages p, p + 4, ... of 128 columns. Each wave has its own ring of two stages in LDS,
// 128 bytes of every activation row and 64 of every weight row, loaded from memory without
// registers, and waits for nobody; the waves' sums meet in LDS at the end, in wave order.
// Scales are staged for 128 blocks of columns at a time by the whole block.
// EXACT: the activations in the two parts of mx8_stream.h, twice the matrix instructions.
// LDS places as in mx8_tile.h.
#pragma once

#include "mx8_tile.h"

namespace awq {

constexpr int kMidWaves = 4, kMidThreads = 64 * kMidWaves;
constexpr int kMidBlocks = 128, kMidStride = kMidBlocks + 4;   // scale bytes of a row, and with padding: 33 banks

// (256 tokens x 4096x4096, 512 blocks, 14.7 us by two stages; three or four leave a unit one
// block: 20.3, 20.7. 64 tokens, 256 blocks: 8.4, 8.6, 8.7.)
constexpr int kMidRing = 2;

template <int NT> struct Mid8 {
    static constexpr int BM = 32, BN = 32 * NT;
    struct Stage {
        u32x4 x[BM * 8], w[BN * 4];
    };
    union {
        Stage ring[kMidWaves][kMidRing];
        f32x16 sums[kMidWaves][NT][64];
    };
    uint32_t s[(BM + BN) * kMidStride / 4];
};

// The sums of all waves over the block's tokens and weight rows, in lds.sums[0 ... 3]. xrow(m),
// wrow(n): row indices, 0 <= m < 32, 0 <= n < 32 NT, every one of rows that exist, within
// 2^32 bytes of codes. All waves have written theirs when this returns.
template <bool EXACT, int NT, typename XRow, typename WRow>
__device__ __forceinline__ void mid8_contract(Mid8<NT> &lds, const uint8_t *xc, const uint8_t *xs, XRow xrow,
                                              const uint8_t *wc, const uint8_t *ws, WRow wrow, int nb)
{
    typedef Mid8<NT> Mid;
    constexpr int BM = Mid::BM, BN = Mid::BN, LOADS = 4 + 2 * NT;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 31, h = lane >> 5, stages = (nb + 3) / 4;

    // Load j of a stage's activations: rows 8 j + lane / 8, chunks as in mx8_tile.h (the
    // swizzle of odd j differs in its upper bit); of its weights rows 16 j + lane / 4. All
    // offsets from the operands' starts are below 2^32.
    const int xq = (lane & 7) ^ (lane >> 4), wq = (lane & 3) ^ (lane >> 4 & 3);
    uint32_t xo[4], wo[2 * NT];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        xo[j] = (uint32_t)xrow(8 * j + (lane >> 3)) * (uint32_t)nb * 32 + (xq ^ (j & 1) * 4) * 16;
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j)
        wo[j] = (uint32_t)wrow(16 * j + (lane >> 2)) * (uint32_t)nb * 16 + wq * 16;
    const uint32_t at0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)&lds.ring[0][0] +
                         wave * (kMidRing * (uint32_t)sizeof(typename Mid::Stage));
    xc = scalar(xc);
    wc = scalar(wc);
    auto fetch = [&](int k, int slot) {
        const uint32_t to = at0 + slot * (uint32_t)sizeof(typename Mid::Stage), to_w = to + (uint32_t)sizeof(Mid::Stage::x);
        const uint8_t *const px = xc + (int64_t)k * 128, *const pw = wc + (int64_t)k * 64;
        if (4 * k + 4 <= nb) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                load_to_lds(px, xo[j], to + j * 1024);
#pragma unroll
            for (int j = 0; j < 2 * NT; ++j)
                load_to_lds(pw, wo[j], to_w + j * 1024);
        } else {                                       // past the rows' end zeros, and the last weights
            const int over = 4 * k + wq - (nb - 1);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                load_to_lds(4 * k + ((xq ^ (j & 1) * 4) >> 1) >= nb ? reinterpret_cast<const uint8_t *>(&kTile8Zeros)
                                                                    : px + xo[j], to + j * 1024);
#pragma unroll
            for (int j = 0; j < 2 * NT; ++j)
                load_to_lds(pw, wo[j] - (over > 0 ? over * 16 : 0), to_w + j * 1024);
        }
    };
    auto stage_scales = [&](int b0) {
        const int words = (nb - b0 < kMidBlocks ? nb - b0 + 3 : kMidBlocks) / 4;
        for (int i = tid; i < (BM + BN) * 32; i += kMidThreads) {
            const int row = i >> 5, w = i & 31;
            if (w < words) {
                const uint8_t *const p = row < BM ? xs + (int64_t)xrow(row) * nb : ws + (int64_t)wrow(row - BM) * nb;
                lds.s[row * (kMidStride / 4) + w] = mx4_scales4(p, b0 + 4 * w, nb);
            }
        }
    };

    f32x16 acc[NT];
#pragma unroll
    for (int b = 0; b < NT; ++b)
        acc[b] = f32x16{};
    auto multiply = [&]<int S>(const typename Mid::Stage &in, uint32_t sx, const uint32_t (&sw)[NT]) {
        const u32x4 *const row = &in.x[r * 8];
        const int swz = r >> 1 & 7;
        const i32x8 x = join(row[(4 * S + h) ^ swz], row[(4 * S + 2 + h) ^ swz]);
        i32x8 high = x, low;
        if constexpr (EXACT)
            mx8_parts(x, high, low);
#pragma unroll
        for (int b = 0; b < NT; ++b) {
            const u32x4 w = in.w[(32 * b + r) * 4 + ((2 * S + h) ^ (r >> 2 & 3))];
            acc[b] = mfma32_a8<false, 2 * S>(high, sx, w, sw[b], acc[b]);
            if constexpr (EXACT)
                acc[b] = mfma32_a8<false, 2 * S>(low, sx, w, sw[b], acc[b]);
        }
    };
    // Stages of one chunk of scales: k = first ... end - 1, the wave's own among them; what is
    // loaded ahead may lie in the next chunk.
    int k = wave, slot = 0, ahead = wave;              // ahead: the next stage to load
#pragma unroll
    for (int j = 0; j < kMidRing; ++j, ahead += kMidWaves)
        if (ahead < stages)
            fetch(ahead, j);
    for (int k0 = 0; k0 < stages; k0 += kMidBlocks / 4) {
        const int end = k0 + kMidBlocks / 4 < stages ? k0 + kMidBlocks / 4 : stages;
        if (k0)
            __syncthreads();
        stage_scales(4 * k0);
        __syncthreads();
#pragma unroll 1
        for (; k < end; k += kMidWaves) {
            // stage k has come; the one behind it may be on its way
            if (ahead - kMidWaves < stages)
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kMidRing - 1) * LOADS) : "memory");
            else
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            const typename Mid::Stage &in = lds.ring[wave][slot];
            const uint32_t sx = lds.s[r * (kMidStride / 4) + (k - k0)] >> (8 * h);
            uint32_t sw[NT];
#pragma unroll
            for (int b = 0; b < NT; ++b)
                sw[b] = lds.s[(BM + 32 * b + r) * (kMidStride / 4) + (k - k0)] >> (8 * h);
            multiply.template operator()<0>(in, sx, sw);
            multiply.template operator()<1>(in, sx, sw);
            if (ahead < stages) {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");     // all of the stage has been read
                fetch(ahead, slot);
            }
            ahead += kMidWaves;
            slot = slot == kMidRing - 1 ? 0 : slot + 1;
        }
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < NT; ++b)
        lds.sums[wave][b][lane] = acc[b];
    __syncthreads();
}

// Registers 4 q ... 4 q + 3 of tile t, lane `lane`, over the waves.
template <int NT>
__device__ __forceinline__ f32x4 mid8_sum(const Mid8<NT> &lds, int t, int lane, int q)
{
    f32x4 s = reinterpret_cast<const f32x4 *>(&lds.sums[0][t][lane])[q];
#pragma unroll
    for (int w = 1; w < kMidWaves; ++w)
        s += reinterpret_cast<const f32x4 *>(&lds.sums[w][t][lane])[q];
    return s;
}

}  // namespace awq
