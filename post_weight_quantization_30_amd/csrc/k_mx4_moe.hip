// k_mx4_moe.hip -- a mixture-of-experts layer on MXFP4 experts, few tokens.
//
//   l = X R^T;  the top_k largest l of a token (ties: lowest expert), p = softmax(l)
//   there (renorm: divided by their sum);  h_e = silu(Wg_e x) * (Wu_e x);
//   y = sum_e p_e Wd_e h_e.
//
// A few tokens read every routed expert's weights once and do little else:
// the layer is bound by HBM. Three launches: the routing; gate and up of each
// routed expert, writing p_e h_e; down, where the sum over experts is one
// more stretch of the contraction. The list of routed experts is found by
// every block from the routing's ids (at most 64 x 16 of them).
#include "mx4.h"

namespace awq {

namespace {

constexpr int kMaxTok = AWQ_MX4_MOE_MAX_TOKENS, kMaxE = AWQ_MX4_MOE_MAX_EXPERTS;

// ---- routing --------------------------------------------------------------
// Block: 16 tokens, 16 waves splitting the columns in steps of 32 (one
// 16x16x32 step per 16 experts); then wave w ranks token w's logits.
constexpr int kRouteWaves = 16;
constexpr int kRouteET = 4;        // expert tiles of 16 summed at a time

__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u)
        return 0;                                          // NaN ranks lowest
    const uint32_t z = (u << 1) == 0 ? 0 : u;              // -0 ties with +0
    return z & 0x80000000u ? ~z : z | 0x80000000u;
}

template <typename TX>
__global__ __launch_bounds__(64 * kRouteWaves) void k_mx4_moe_route(const TX *__restrict__ X, int M, int hidden,
                                                                    const TX *__restrict__ router, int E, int top_k,
                                                                    int renorm, int32_t *__restrict__ ids,
                                                                    float *__restrict__ weights)
{
    typedef typename Vec8<TX>::type vec;
    __shared__ f32x4 red[kRouteWaves * kRouteET * 64];     // 64 KB
    __shared__ float logits[16][kMaxE];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, c = lane >> 4;
    const int m0 = blockIdx.x * 16;
    const TX *x = X + (int64_t)(m0 + r < M ? m0 + r : M - 1) * hidden + 8 * c;
    const int steps = hidden / 32;
    for (int e0 = 0; e0 < E; e0 += 16 * kRouteET) {
        const TX *w[kRouteET];
#pragma unroll
        for (int t = 0; t < kRouteET; ++t) {
            const int e = e0 + 16 * t + r;
            w[t] = router + (int64_t)(e < E ? e : E - 1) * hidden + 8 * c;
        }
        f32x4 acc[kRouteET];
#pragma unroll
        for (int t = 0; t < kRouteET; ++t)
            acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int s = wave; s < steps; s += kRouteWaves) {
            const vec xv = load8(x + s * 32);
#pragma unroll
            for (int t = 0; t < kRouteET; ++t)
                acc[t] = mx4_mfma(xv, load8(w[t] + s * 32), acc[t]);
        }
#pragma unroll
        for (int t = 0; t < kRouteET; ++t)
            red[(wave * kRouteET + t) * 64 + lane] = acc[t];
        __syncthreads();
        for (int idx = threadIdx.x; idx < kRouteET * 64; idx += 64 * kRouteWaves) {
            f32x4 sum = red[idx];
#pragma unroll
            for (int k = 1; k < kRouteWaves; ++k)
                sum += red[k * kRouteET * 64 + idx];
            const int l = idx & 63, e = e0 + 16 * (idx / 64) + (l & 15);
            if (e < E)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    logits[4 * (l >> 4) + i][e] = sum[i];
        }
        __syncthreads();
    }
    const int m = m0 + wave;
    if (m >= M)
        return;
    // lane l ranks experts l, l + 64, ...: the largest (value, lowest index)
    // wins a round and leaves
    float l[kMaxE / 64];
    uint64_t key[kMaxE / 64];
#pragma unroll
    for (int q = 0; q < kMaxE / 64; ++q) {
        const int e = lane + 64 * q;
        l[q] = e < E ? logits[wave][e] : 0.f;
        key[q] = e < E ? (uint64_t)ordered(l[q]) << 32 | (uint32_t)(0xFFFF - e) : 0;
    }
    float top = 0.f, sum = 0.f, mine = 0.f;
    int my_id = 0;
    for (int k = 0; k < top_k; ++k) {
        uint64_t best = 0;
#pragma unroll
        for (int q = 0; q < kMaxE / 64; ++q)
            best = key[q] > best ? key[q] : best;
        for (int off = 32; off > 0; off >>= 1) {
            const uint64_t o = __shfl_xor(best, off);
            best = o > best ? o : best;
        }
        const int e = 0xFFFF - (int)(uint32_t)best;
#pragma unroll
        for (int q = 0; q < kMaxE / 64; ++q)
            if (key[q] == best)
                key[q] = 0;
        const float v = logits[wave][e];
        if (k == 0)
            top = v;
        const float p = expf(v - top);
        if (renorm)
            sum += p;
        if (lane == k) {
            mine = p;
            my_id = e;
        }
    }
    if (!renorm) {
#pragma unroll
        for (int q = 0; q < kMaxE / 64; ++q)
            sum += lane + 64 * q < E ? expf(l[q] - top) : 0.f;
        for (int off = 32; off > 0; off >>= 1)
            sum += __shfl_xor(sum, off);
    }
    if (lane < top_k) {
        ids[m * top_k + lane] = my_id;
        weights[m * top_k + lane] = mine / sum;
    }
}

// The routed experts as bits, from all ids (every thread of the block calls it).
__device__ __forceinline__ void routed_bits(const int32_t *ids, int pairs, uint32_t (&bits)[kMaxE / 32])
{
    if (threadIdx.x < kMaxE / 32)
        bits[threadIdx.x] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += blockDim.x)
        atomicOr(&bits[ids[p] >> 5], 1u << (ids[p] & 31));
    __syncthreads();
}

// ---- gate and up ------------------------------------------------------------
// Block: 16 columns of one expert's intermediate (a tile of gate rows and one
// of up rows), all tokens routed to it, the hidden columns split over 8 waves.
constexpr int kUpWaves = 8;

template <typename TX, int MT, int U>
__device__ __forceinline__ void up_tokens(const TX *__restrict__ X, int nb, const uint8_t *const (&w)[2],
                                          const uint8_t *const (&ws)[2], const uint16_t *list, int count, int top_k,
                                          const float *__restrict__ weights, int inter, int col0, f32x4 *red,
                                          TX *__restrict__ h, int lane, int wave)
{
    const int r = lane & 15, c = lane >> 4;
    Mx4Rows<TX, MT, 2> rows;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
        rows.w[nt] = w[nt];
        rows.ws[nt] = ws[nt];
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int t = 16 * mt + r;
        rows.x[mt] = X + (int64_t)(list[t < count ? t : count - 1] / top_k) * nb * 32;
        rows.xs[mt] = nullptr;
    }
    f32x4 acc[MT][2];
    mx4_wave<TX, MT, 2, U>(rows, acc, wave * (4 * U), kUpWaves * (4 * U), nb, c);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        __syncthreads();           // the previous tile's sums are read
        red[(wave * 2 + 0) * 64 + lane] = acc[mt][0];
        red[(wave * 2 + 1) * 64 + lane] = acc[mt][1];
        __syncthreads();
        // one thread per (token, column): f32 k of lane l is token 4 (l / 16) + k
        if (threadIdx.x < 256) {
            const int col = threadIdx.x & 15, t = threadIdx.x >> 4;
            const float *g = reinterpret_cast<const float *>(red) + ((t >> 2) * 16 + col) * 4 + (t & 3);
            float gate = 0.f, up = 0.f;
#pragma unroll
            for (int k = 0; k < kUpWaves; ++k) {
                gate += g[k * 512];
                up += g[k * 512 + 256];
            }
            const int tok = 16 * mt + t;
            if (tok < count) {
                const int pair = list[tok];
                const float v = gate / (1.0f + expf(-gate)) * up * weights[pair];
                h[(int64_t)pair * inter + col0 + col] = static_cast<TX>(v);
            }
        }
    }
}

template <typename TX>
__global__ __launch_bounds__(64 * kUpWaves) void k_mx4_moe_up(const TX *__restrict__ X, int pairs, int hidden,
                                                              int inter, int top_k, const int32_t *__restrict__ ids,
                                                              const float *__restrict__ weights,
                                                              const uint8_t *__restrict__ codes,
                                                              const uint8_t *__restrict__ scales, TX *__restrict__ h)
{
    __shared__ uint32_t bits[kMaxE / 32];
    __shared__ uint16_t list[kMaxTok];
    __shared__ int s_count;
    __shared__ f32x4 red[kUpWaves * 2 * 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    routed_bits(ids, pairs, bits);
    int e = -1, skip = blockIdx.y;
    for (int q = 0; q < kMaxE / 32 && e < 0; ++q) {
        uint32_t b = bits[q];
        const int n = __popc(b);
        if (skip >= n) {
            skip -= n;
            continue;
        }
        for (; skip > 0; --skip)
            b &= b - 1;
        e = 32 * q + __ffs(b) - 1;
    }
    if (e < 0)
        return;                    // fewer routed experts than blocks: the whole block leaves
    if (wave == 0) {               // this expert's pairs in ascending order (a token has it once at most)
        int n = 0;
        for (int p0 = 0; p0 < pairs; p0 += 64) {
            const bool in = p0 + lane < pairs && ids[p0 + lane] == e;
            const uint64_t mask = __ballot(in);
            if (in)
                list[n + __popcll(mask & ((1ull << lane) - 1))] = (uint16_t)(p0 + lane);
            n += __popcll(mask);
        }
        if (lane == 0)
            s_count = n;
    }
    __syncthreads();
    const int count = s_count, nb = hidden / kMxBlock, col0 = blockIdx.x * 16, r = lane & 15;
    const int64_t row = (int64_t)e * 2 * inter + col0 + r;
    const uint8_t *const w[2] = {codes + row * nb * 16, codes + (row + inter) * nb * 16};
    const uint8_t *const ws[2] = {scales + row * nb, scales + (row + inter) * nb};
    if (count <= 16)
        up_tokens<TX, 1, 2>(X, nb, w, ws, list, count, top_k, weights, inter, col0, red, h, lane, wave);
    else if (count <= 32)
        up_tokens<TX, 2, 1>(X, nb, w, ws, list, count, top_k, weights, inter, col0, red, h, lane, wave);
    else
        up_tokens<TX, 4, 1>(X, nb, w, ws, list, count, top_k, weights, inter, col0, red, h, lane, wave);
}

// ---- down -------------------------------------------------------------------
// Block: 16 hidden columns, all tokens; the waves split (routed expert, 128 U
// columns of it) items. A token that an expert does not serve multiplies some
// other row and drops the result: a NaN scale of an expert reaches its own
// tokens only.
constexpr int kDownWaves = 8;

template <typename TX, int MT, int U>
__global__ __launch_bounds__(64 * kDownWaves) void k_mx4_moe_down(const TX *__restrict__ h, int M, int hidden, int inter,
                                                                  int top_k, const int32_t *__restrict__ ids,
                                                                  const uint8_t *__restrict__ codes,
                                                                  const uint8_t *__restrict__ scales,
                                                                  TX *__restrict__ Y)
{
    __shared__ uint32_t bits[kMaxE / 32];
    __shared__ uint8_t expert[kMaxE];
    __shared__ __align__(8) int16_t pair_of[kMaxE][16 * MT];       // (routed expert, token) -> pair or -1
    __shared__ f32x4 red[kDownWaves * MT * 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, c = lane >> 4, pairs = M * top_k;
    routed_bits(ids, pairs, bits);
    int active = 0;
#pragma unroll
    for (int q = 0; q < kMaxE / 32; ++q)
        active += __popc(bits[q]);
    for (int idx = threadIdx.x; idx < active * 16 * MT; idx += blockDim.x)
        pair_of[idx / (16 * MT)][idx % (16 * MT)] = -1;
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += blockDim.x) {
        const int e = ids[p];
        int a = __popc(bits[e >> 5] & ((1u << (e & 31)) - 1));
        for (int q = 0; q < e >> 5; ++q)
            a += __popc(bits[q]);
        expert[a] = (uint8_t)e;                                    // the same value from every pair of e
        pair_of[a][p / top_k] = (int16_t)p;
    }
    __syncthreads();

    const int nb = inter / kMxBlock, per = (nb + 4 * U - 1) / (4 * U), items = active * per;
    const int n = blockIdx.x * 16 + r;
    f32x4 acc[MT][1];
    bool bad = false;
    mx4_zero(acc);

    auto load = [&](Mx4Item<TX, MT, 1, U> &it, int i) {
        const int a = i / per, b0 = (i - a * per) * 4 * U;
        const int64_t row = (int64_t)expert[a] * hidden + n;
        Mx4Rows<TX, MT, 1> rows;
        rows.w[0] = codes + row * nb * 16;
        rows.ws[0] = scales + row * nb;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int p = pair_of[a][16 * mt + r];
            rows.x[mt] = h + (int64_t)(p < 0 ? 0 : p) * inter;
            rows.xs[mt] = nullptr;
        }
        mx4_load(it, rows, b0, nb, c);
    };
    auto compute = [&]<bool WIDE>(Mx4Item<TX, MT, 1, U> &it, int i) {
        const int a = i / per, b0 = (i - a * per) * 4 * U;
        f32x4 part[MT][1];
        mx4_zero(part);
        mx4_compute<WIDE>(it, part, b0, nb, c, bad);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (pair_of[a][16 * mt + 4 * c + k] >= 0)
                    acc[mt][0][k] += part[mt][0][k];
    };
    Mx4Item<TX, MT, 1, U> A, B;
    int i = wave;
    if (i < items) {
        load(A, i);
        while (true) {
            if (i + kDownWaves < items)
                load(B, i + kDownWaves);
            compute.template operator()<false>(A, i);
            i += kDownWaves;
            if (i >= items)
                break;
            if (i + kDownWaves < items)
                load(A, i + kDownWaves);
            compute.template operator()<false>(B, i);
            i += kDownWaves;
            if (i >= items)
                break;
        }
        if constexpr (std::is_same<TX, f16>::value) {
            if (__any(bad)) {          // scales that fp16 cannot hold: once more in the wide form
                mx4_zero(acc);
#pragma unroll 1
                for (i = wave; i < items; i += kDownWaves) {
                    load(A, i);
                    compute.template operator()<true>(A, i);
                }
            }
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        red[(wave * MT + mt) * 64 + lane] = acc[mt][0];
    __syncthreads();
    for (int idx = threadIdx.x; idx < MT * 64; idx += 64 * kDownWaves) {
        f32x4 sum = red[idx];
#pragma unroll
        for (int w = 1; w < kDownWaves; ++w)
            sum += red[w * MT * 64 + idx];
        const int l = idx & 63, m = 16 * (idx / 64) + 4 * (l >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (m + k < M)
                Y[(int64_t)(m + k) * hidden + blockIdx.x * 16 + (l & 15)] = static_cast<TX>(sum[k]);
    }
}

template <typename TX>
hipError_t moe(const void *X, int M, int hidden, int inter, int E, int top_k, int renorm, const void *router,
               const uint8_t *gu, const uint8_t *gus, const uint8_t *dn, const uint8_t *dns, void *Y, char *ws,
               hipStream_t st)
{
    const Mx4MoeWs lay = mx4_moe_ws_layout(M, inter, top_k);
    int32_t *ids = (int32_t *)(ws + lay.ids_off);
    float *weights = (float *)(ws + lay.w_off);
    TX *h = (TX *)(ws + lay.h_off);
    const int pairs = M * top_k;
    k_mx4_moe_route<TX><<<dim3((M + 15) / 16), 64 * kRouteWaves, 0, st>>>(
        (const TX *)X, M, hidden, (const TX *)router, E, top_k, renorm, ids, weights);
    k_mx4_moe_up<TX><<<dim3(inter / 16, pairs < E ? pairs : E), 64 * kUpWaves, 0, st>>>(
        (const TX *)X, pairs, hidden, inter, top_k, ids, weights, gu, gus, h);
    const dim3 grid(hidden / 16), block(64 * kDownWaves);
    if (M <= 16)
        k_mx4_moe_down<TX, 1, 4><<<grid, block, 0, st>>>(h, M, hidden, inter, top_k, ids, dn, dns, (TX *)Y);
    else if (M <= 32)
        k_mx4_moe_down<TX, 2, 2><<<grid, block, 0, st>>>(h, M, hidden, inter, top_k, ids, dn, dns, (TX *)Y);
    else
        k_mx4_moe_down<TX, 4, 1><<<grid, block, 0, st>>>(h, M, hidden, inter, top_k, ids, dn, dns, (TX *)Y);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx4_moe(const void *X, int dtype, int M, int hidden, int inter, int experts, int top_k, int renorm,
                          const void *router, const uint8_t *gu_codes, const uint8_t *gu_scales,
                          const uint8_t *dn_codes, const uint8_t *dn_scales, void *Y, void *ws, hipStream_t st)
{
    if (dtype == AWQ_F16)
        return moe<f16>(X, M, hidden, inter, experts, top_k, renorm, router, gu_codes, gu_scales, dn_codes, dn_scales,
                        Y, (char *)ws, st);
    return moe<bf16>(X, M, hidden, inter, experts, top_k, renorm, router, gu_codes, gu_scales, dn_codes, dn_scales, Y,
                     (char *)ws, st);
}

}  // namespace awq
