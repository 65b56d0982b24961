// mx8_tile.h -- the large tile of products of MXFP8 activations and MXFP4 weights,
// shared by the plain product and the routed experts.
//
// Block: 64 MT tokens x 256 weight rows, 8 waves (two a SIMD) of 32 MT x 64. A stage is
// 128 columns: 128 bytes of an activation row, 64 of a weight row, in one of three LDS
// buffers that memory is loaded to without registers, two stages ahead; scales come by
// four stages, 16 bytes of a row (a load of scales, whose lanes lie in different rows,
// costs a load unit the same whatever its width).
//
// LDS is read 256 bytes a cycle where the 16 lanes that it serves together touch all 64
// banks, 128 where two of them meet (measured, ds_read_b128: 4.9 and 8.5 units). Of
// activation rows of 128 bytes 16 rows are served together: chunk q of row m lies at
// q ^ (m / 2 & 7), so that the eight pairs of rows differ; of weight rows of 64 bytes, four
// to 256 bytes, at q ^ (m / 4 & 3).
// Lane (r, h) holds in k-step s (64 columns) chunks 4 s + h and 4 s + 2 + h of an
// activation row and chunk 2 s + h of a weight row (see mx8.h).
#pragma once

#include "mx8.h"
#include "mx_tiles.h"

namespace awq {

// 32 tokens x 32 rows over 64 columns. Tokens are the rows of the matrix instruction:
// acc[i] of lane (r, h) is token 8 (i / 4) + 4 h + i % 4, row r; TURNED: the other way.
template <bool TURNED, int S>
__device__ __forceinline__ f32x16 mfma32_a8(const i32x8 &x, uint32_t sx, const u32x4 &w, uint32_t sw, const f32x16 &acc)
{
    const i32x8 w8 = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
    if constexpr (TURNED)
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w8, x, acc, 4, 0, S, (int)sw, S, (int)sx);
    else
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, w8, acc, 0, 4, S, (int)sx, S, (int)sw);
}

// Scale bytes of 16 blocks of a row from block b on, 127 for those past its end.
__device__ __forceinline__ u32x4 load_scales16(const uint8_t *row, int b, int nb)
{
    u32x4 v;
    if (b + 16 <= nb)
        __builtin_memcpy(&v, row + b, 16);             // at any alignment
    else
        v = u32x4{mx4_scales4(row, b, nb), mx4_scales4(row, b + 4, nb), mx4_scales4(row, b + 8, nb),
                  mx4_scales4(row, b + 12, nb)};
    return v;
}

template <int MT> struct Tile8 {
    static constexpr int BM = 64 * MT, BN = 256, kBuf = 3;
    // scale bytes of four stages: activation rows, then weight rows
    u32x4 s[2][BM + BN];
    u32x4 x[kBuf][BM * 8], w[kBuf][BN * 4];
};

// What stands for the activations past a row's end.
static __device__ const u32x4 kTile8Zeros = {0, 0, 0, 0};

// 16 bytes a lane from memory to LDS, lane i's to `to` + 16 i, without registers on the
// way. In flight until a wait for the vector memory counter that the compiler knows
// nothing of: those are written out below. The LDS address goes in m0, as an operand: the
// compiler sets it, and knows what the register holds. (One wait state between the two.)
__device__ __forceinline__ void load_to_lds(const uint8_t *from, uint32_t to)
{
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "{m0}"(to) : "memory");
}
__device__ __forceinline__ void load_to_lds(const uint8_t *base, uint32_t off, uint32_t to)
{
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(to) : "memory");
}

// A pointer that is the same in all lanes, in scalar registers.
__device__ __forceinline__ const uint8_t *scalar(const uint8_t *p)
{
    const uint64_t v = (uint64_t)p;
    return (const uint8_t *)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 |
                             (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}

// The rows and chunks that a thread moves: activation rows tile8_xrow() + 64 i, chunk
// tile8_xchunk() of each eight, weight rows tile8_wrow() + 128 i, chunk tile8_wchunk() of
// each four. (A wave fills 1024 bytes of LDS in lane order; the swizzle is in which chunk
// a lane fetches.)
__device__ __forceinline__ int tile8_xrow() { return threadIdx.x >> 3; }
__device__ __forceinline__ int tile8_xchunk() { return (threadIdx.x & 7) ^ (threadIdx.x >> 4 & 7); }
__device__ __forceinline__ int tile8_wrow() { return threadIdx.x >> 2; }
__device__ __forceinline__ int tile8_wchunk() { return (threadIdx.x & 3) ^ (threadIdx.x >> 4 & 3); }

// acc = the wave's products. xbase + xo[i]: the first chunk of this thread's i-th activation
// row; wbase + wo[i]: of its weight row; sp: the scales of activation row threadIdx.x, or of
// weight row threadIdx.x - BM; EXACT: in the two parts of mx8_stream.h, twice the matrix
// instructions; `words`: all rows' scales begin at multiples of 4 bytes.
// Every wave is past its last read of the operands when this returns.
template <bool TURNED, bool EXACT, int MT>
__device__ __forceinline__ void tile8_contract(Tile8<MT> &lds, f32x16 (&acc)[MT][2], const uint8_t *xbase,
                                               const uint32_t (&xo)[MT], const uint8_t *wbase, const uint32_t (&wo)[2], const uint8_t *sp, bool words,
                                               int nb)
{
    constexpr int BM = Tile8<MT>::BM, BN = Tile8<MT>::BN, BUF = Tile8<MT>::kBuf;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 31, h = lane >> 5, wm = wave >> 2, wn = wave & 3;
    const int stages = (nb + 3) / 4, xq = tile8_xchunk() >> 1, wq = tile8_wchunk();
    const bool has_s = tid < BM + BN;
    const uint8_t *const base = reinterpret_cast<const uint8_t *>(&lds);
    const uint32_t at0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)base;
    constexpr uint32_t X0 = 2 * (BM + BN) * 16, W0 = X0 + BUF * BM * 128;

    // Load D of the MT + 2 of stage k. FULL: all of the stage's columns exist.
    xbase = scalar(xbase);
    wbase = scalar(wbase);
    auto fetch = [&]<int D, bool FULL>(int k, int buf) {
        if constexpr (D < MT) {
            const uint32_t to = at0 + X0 + buf * (BM * 128) + wave * 1024 + D * 8192;
            const uint8_t *const p = xbase + (int64_t)k * 128;
            if constexpr (FULL)
                load_to_lds(p, xo[D], to);
            else                                       // past the rows' end zeros
                load_to_lds(4 * k + xq >= nb ? reinterpret_cast<const uint8_t *>(&kTile8Zeros) : p + xo[D], to);
        } else {
            const int over = FULL ? 0 : 4 * k + wq - (nb - 1);   // past the rows' end their last block
            load_to_lds(wbase + (int64_t)k * 64, wo[D - MT] - (over > 0 ? over * 16 : 0),
                        at0 + W0 + buf * (BN * 64) + wave * 1024 + (D - MT) * 8192);
        }
    };
    auto fetch_all = [&](int k, int buf) {
        fetch.template operator()<0, false>(k, buf);
        fetch.template operator()<1, false>(k, buf);
        fetch.template operator()<2, false>(k, buf);
        fetch.template operator()<3, false>(k, buf);
        if constexpr (MT == 4) {
            fetch.template operator()<4, false>(k, buf);
            fetch.template operator()<5, false>(k, buf);
        }
    };
    // Scales of stages k ... k + 3. Through registers only where they must: the compiler's
    // wait for them is one for all loads on their way, which held a K of 14336 up by a
    // seventh.
    u32x4 sr;
    auto straight = [&](int k) { return words && 4 * k + 16 <= nb; };
    auto fetch_s = [&](int k) {
        if (!has_s)
            return;
        if (straight(k))
            load_to_lds(sp + 4 * k, at0 + (k >> 2 & 1) * ((BM + BN) * 16) + wave * 1024);
        else
            sr = load_scales16(sp, 4 * k, nb);
    };
    auto stash_s = [&](int k) {
        if (has_s && !straight(k))
            lds.s[k >> 2 & 1][tid] = sr;
    };

    i32x8 x[MT];
    u32x4 w[2];
    // a stage's four scale bytes, turned down by h: bytes 0 and 2 belong to the k-steps'
    // blocks of this lane, where the matrix instructions take them (reading them at that
    // byte is slow: LDS takes four times as long for words at odd addresses)
    uint32_t sx[MT], sw[2];
    // Rows 32 apart keep their swizzle: one address for each chunk, the rest are constants.
    uint32_t xa[2][2], wa[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
            xa[s][half] = X0 + (32 * MT * wm + r) * 128 + ((4 * s + 2 * half + h) ^ (r >> 1 & 7)) * 16;
        wa[s] = W0 + (64 * wn + r) * 64 + ((2 * s + h) ^ (r >> 2 & 3)) * 16;
    }
    const uint32_t sa = 4 * (32 * MT * wm + r), sb = 4 * (BM + 64 * wn + r);
    auto read = [&]<int S>(int k, int buf) {           // operands of k-step S
        auto chunk = [&](uint32_t at) { return *reinterpret_cast<const u32x4 *>(base + at); };
        const uint32_t xb = buf * (BM * 128), wb = buf * (BN * 64);
        if constexpr (S == 0) {
            const uint32_t *const at = reinterpret_cast<const uint32_t *>(lds.s[k >> 2 & 1]) + (k & 3);
#pragma unroll
            for (int a = 0; a < MT; ++a)
                sx[a] = at[sa + 128 * a];
#pragma unroll
            for (int b = 0; b < 2; ++b)
                sw[b] = at[sb + 128 * b];
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
            w[b] = chunk(wa[S] + wb + b * 2048);
#pragma unroll
        for (int a = 0; a < MT; ++a)
            x[a] = join(chunk(xa[S][0] + xb + a * 4096), chunk(xa[S][1] + xb + a * 4096));
    };
    auto barrier = [] {                                // waits are written out before it
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    auto multiply = [&]<int S>() {
        if constexpr (S == 0) {
#pragma unroll
            for (int a = 0; a < MT; ++a)
                sx[a] >>= 8 * h;
#pragma unroll
            for (int b = 0; b < 2; ++b)
                sw[b] >>= 8 * h;
        }
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if constexpr (EXACT) {
                    i32x8 high, low;
                    mx8_parts(x[a], high, low);
                    acc[a][b] = mfma32_a8<TURNED, 2 * S>(high, sx[a], w[b], sw[b], acc[a][b]);
                    acc[a][b] = mfma32_a8<TURNED, 2 * S>(low, sx[a], w[b], sw[b], acc[a][b]);
                } else {
                    acc[a][b] = mfma32_a8<TURNED, 2 * S>(x[a], sx[a], w[b], sw[b], acc[a][b]);
                }
#pragma unroll
        for (int a = 0; a < MT; ++a)                   // here, not behind the next reads
#pragma unroll
            for (int b = 0; b < 2; ++b)
                asm volatile("" : "+v"(acc[a][b])::"memory");
        __builtin_amdgcn_sched_barrier(0);
    };

#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
            acc[a][b] = f32x16{};
    fetch_s(0);
    stash_s(0);
    fetch_all(0, 0);
    if (1 < stages)
        fetch_all(1, 1);
    if (1 < stages)
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(MT + 2) : "memory");
    else
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    // Two groups of waves, one on each SIMD, half a k-step apart: while one multiplies the
    // other reads its operands. In phases from the start of the first group's stage k on,
    // first | second group:  R(k,0) | M(k-1,1),  M(k,0) | R(k,0),  R(k,1) | M(k,0),  M(k,1) | R(k,1).
    // Stage k - 1's buffer is free from the first of these on and takes stage k + 2, whose
    // loads go out in the reading phases (all in one multiplying phase: 5 % slower, the load
    // unit holds the waves up), and each group waits for its part before it leaves its last
    // reading phase of stage k + 1.
    if (wm)
        barrier();
    int buf = 0, next = 1, free = 2;                   // buffers of stages k, k + 1 and k + 2
    constexpr int HALF = (MT + 2) / 2;
    // FULL: stages k + 1 and k + 2 exist, with all their columns. Stage k + 2's buffer was
    // stage k - 1's, which all waves are past.
    auto stage = [&]<bool FULL>(int k) {
        read.template operator()<0>(k, buf);
        if (FULL || k + 2 < stages) {
            fetch.template operator()<0, FULL>(k + 2, free);
            fetch.template operator()<1, FULL>(k + 2, free);
            if constexpr (HALF == 3)
                fetch.template operator()<2, FULL>(k + 2, free);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        barrier();
        multiply.template operator()<0>();
        barrier();
        read.template operator()<1>(k, buf);
        if (FULL || k + 2 < stages) {
            fetch.template operator()<HALF, FULL>(k + 2, free);
            fetch.template operator()<HALF + 1, FULL>(k + 2, free);
            if constexpr (HALF == 3)
                fetch.template operator()<5, FULL>(k + 2, free);
            // this wave's part of stage k + 1 has come
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(MT + 2) : "memory");
        } else {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        if ((k & 3) == 3 && (FULL || k + 1 < stages))
            stash_s(k + 1);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        barrier();
        if ((k & 3) == 1 && k + 3 < stages)
            fetch_s(k + 3);
        multiply.template operator()<1>();
        barrier();
        const int b = buf;
        buf = next;
        next = free;
        free = b;
    };
    int k = 0;
#pragma unroll 1
    for (; 4 * (k + 3) <= nb; ++k)
        stage.template operator()<true>(k);
#pragma unroll 1
    for (; k < stages; ++k)
        stage.template operator()<false>(k);
    if (!wm)
        barrier();
}

}  // namespace awq
