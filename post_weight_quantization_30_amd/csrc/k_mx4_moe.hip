// k_mx4_moe.hip -- a mixture-of-experts layer on MXFP4 experts, few tokens.
//
//   l = X R^T;  the top_k largest l of a token (ties: lowest expert), p = softmax(l)
//   there (renorm: divided by their sum);  h_e = silu(Wg_e x) * (Wu_e x);
//   y = sum_e p_e Wd_e h_e.
//
// A few tokens read every routed expert's weights once and do little else:
// the layer is bound by HBM, and the smallest calls by their launches. Launches:
// the logits; the routing, unless the next one does it; gate and up of each
// routed expert, writing p_e h_e; down, where the sum over experts is one more
// stretch of the contraction; the sum of down's parts, if it has any. The list
// of routed experts is found by every block from the routing's ids (at most 64 x
// 16 of them).
//
//   1 token, 8 of 64 experts of 2048x1024     26.5 us (27 MB): logits 2.7, up
//                                             14.0 with the routing, down 10.3
//   8 tokens, 2 of 8 of 4096x14336, 7 hit     170 us (655 MB, 3.8 TB/s): up 102
//                                             (4.3 TB/s), down 58 (3.8)
//   33 tokens, 4 of 48 of 1056x1408, 44 hit   61 us (105 MB): logits 4.0, routing
//                                             3.6, up 31, down 20, sum 4.7
//   1 token, 8 of 256 of 4096x512             26 us
// (medians, the layers as graph replays, the launches from a kernel trace; experts
// of 600 MB and more in turn.)
#include "mx4.h"

namespace awq {

namespace {

constexpr int kMaxTok = AWQ_MX4_MOE_MAX_TOKENS, kMaxK = AWQ_MX4_MOE_MAX_TOPK, kMaxE = AWQ_MX4_MOE_MAX_EXPERTS;

// ---- routing ----------------------------------------------------------------
// Logits: a block per expert and TOK tokens, its four waves and their lanes
// along the columns. (A router row is read in whole kilobytes: 16 rows of 64
// bytes, as a matrix tile would read them, keep a load unit busy twice as long.)
// Bound by latency: 2.7 us for 1 token, 64 experts of 2048 columns; one block
// for all experts of 16 tokens took 11.
template <typename TX, int TOK>
__global__ __launch_bounds__(256) void k_mx4_moe_logits(const TX *__restrict__ X, int M, int hidden,
                                                        const TX *__restrict__ router, int E,
                                                        float *__restrict__ logits)
{
    typedef typename Vec8<TX>::type vec;
    __shared__ float part[4][TOK];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = blockIdx.x, m0 = blockIdx.y * TOK;
    const TX *const w = router + (int64_t)e * hidden;
    const TX *x[TOK];
    float acc[TOK];
#pragma unroll
    for (int t = 0; t < TOK; ++t) {                    // past the last token: that one again
        x[t] = X + (int64_t)(m0 + t < M ? m0 + t : M - 1) * hidden;
        acc[t] = 0.f;
    }
    for (int j = threadIdx.x * 8; j < hidden; j += 2048) {
        const vec wv = load8(w + j);
        vec xv[TOK];
#pragma unroll
        for (int t = 0; t < TOK; ++t)
            xv[t] = load8(x[t] + j);
        float wf[8];
        widen8<TX>(wv, wf);
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
            float xf[8];
            widen8<TX>(xv[t], xf);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc[t] = fmaf(xf[i], wf[i], acc[t]);
        }
    }
    // lanes of the two halves keep one half of the tokens each, and so on: then
    // lane l holds token l / (64 / TOK)
#pragma unroll
    for (int n = TOK / 2, off = 32; off > 0; off >>= 1, n /= 2) {
        if (n > 0) {
            const bool up = lane & off;
#pragma unroll
            for (int t = 0; t < n; ++t) {
                const float give = up ? acc[t] : acc[t + n];
                acc[t] = (up ? acc[t + n] : acc[t]) + __shfl_xor(give, off);
            }
        } else {
            acc[0] += __shfl_xor(acc[0], off);
        }
    }
    if ((lane & (64 / TOK - 1)) == 0)
        part[wave][lane / (64 / TOK)] = acc[0];
    __syncthreads();
    const int t = threadIdx.x;
    if (t < TOK && m0 + t < M)
        logits[(int64_t)(m0 + t) * E + e] = (part[0][t] + part[1][t]) + (part[2][t] + part[3][t]);
}

// Larger logits have larger keys; NaN the lowest, -0 ties with +0, and 0 is below all.
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u)
        return 1;
    const uint32_t z = (u << 1) == 0 ? 0 : u;
    return z & 0x80000000u ? ~z : z | 0x80000000u;
}

// The largest x of the wave.
__device__ __forceinline__ uint32_t wave_max(uint32_t x)
{
    auto with = [&](uint32_t o) { x = x > o ? x : o; };
    with(__builtin_amdgcn_update_dpp(x, x, 0x111, 0xF, 0xF, false));   // lanes 1, 2, 4, 8 below, within rows of 16
    with(__builtin_amdgcn_update_dpp(x, x, 0x112, 0xF, 0xF, false));
    with(__builtin_amdgcn_update_dpp(x, x, 0x114, 0xF, 0xF, false));
    with(__builtin_amdgcn_update_dpp(x, x, 0x118, 0xF, 0xF, false));
    with(__builtin_amdgcn_update_dpp(x, x, 0x142, 0xA, 0xF, false));   // lane 15 of the row below
    with(__builtin_amdgcn_update_dpp(x, x, 0x143, 0xC, 0xF, false));   // lane 31
    return __builtin_amdgcn_readlane(x, 63);
}

// Routes a token, by one wave: lane k < top_k gets the k-th expert and its
// weight. Each is the maximum of the keys that are left, found in 6 steps
// across the lanes: 16 experts of 256 take a microsecond, where counting the
// experts ahead of each one takes 8.
__device__ __forceinline__ void choose(const float *logits, int E, int top_k, int renorm, int lane, int &id,
                                       float &weight)
{
    constexpr int Q = kMaxE / 64;
    float l[Q], logit = 0.f, top = 0.f;
    uint32_t keys[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q)
        l[q] = 64 * q + lane < E ? logits[64 * q + lane] : 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q)
        keys[q] = 64 * q + lane < E ? ordered(l[q]) : 0;
    for (int k = 0; k < top_k; ++k) {
        uint32_t best = keys[0];
#pragma unroll
        for (int q = 1; q < Q; ++q)
            best = best > keys[q] ? best : keys[q];
        best = wave_max(best);
        int e = 0;
#pragma unroll
        for (int q = Q - 1; q >= 0; --q) {             // of equals the lowest
            const uint64_t at = __ballot(keys[q] == best);
            e = at ? 64 * q + __builtin_ctzll(at) : e;
        }
        float v = 0.f;
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (e >> 6 == q) {
                v = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, l[q]), e & 63));
                keys[q] = lane == (e & 63) ? 0 : keys[q];
            }
        top = k == 0 ? v : top;
        logit = lane == k ? v : logit;
        id = lane == k ? e : id;
    }
    const float own = expf(logit - top);
    float total = 0.f;
    if (renorm) {
        for (int k = 0; k < top_k; ++k)
            total += __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, own), k));
    } else {
#pragma unroll
        for (int q = 0; q < Q; ++q)
            total += 64 * q + lane < E ? expf(l[q] - top) : 0.f;
        for (int off = 32; off > 0; off >>= 1)
            total += __shfl_xor(total, off);
    }
    weight = own / total;
}

// A wave per token.
__global__ __launch_bounds__(64) void k_mx4_moe_topk(const float *__restrict__ logits, int E, int top_k, int renorm,
                                                     int32_t *__restrict__ ids, float *__restrict__ weights)
{
    const int lane = threadIdx.x;
    const int64_t m = blockIdx.x;
    int id = 0;
    float weight;
    choose(logits + m * E, E, top_k, renorm, lane, id, weight);
    if (lane < top_k) {
        ids[m * top_k + lane] = id;
        weights[m * top_k + lane] = weight;
    }
}

// What a block of `up` or `down` makes of the routing's ids: the (token, slot)
// pairs by expert and token, cut into groups of one expert's 16 at most.
constexpr int kMaxPairs = kMaxTok * kMaxK, kMaxGroups = kMaxE + kMaxPairs / 16;

struct Routed {
    uint64_t tokens[kMaxE];                            // of every expert, as bits
    uint32_t sums[kMaxE / 64];
    uint16_t first[kMaxE];                             // an expert's first place in `pairs`
    uint16_t pairs[kMaxPairs], group_of[kMaxPairs];    // group_of: by place
    uint16_t begin[kMaxGroups + 1];                    // a group's first place; begin[groups] = all pairs
    uint8_t expert[kMaxGroups];
    int groups;
    // uniform: a group's size
    __device__ __forceinline__ int size(int g) const
    {
        return __builtin_amdgcn_readfirstlane(begin[g + 1] - begin[g]);
    }
};

__device__ __forceinline__ void read_routing(Routed &rt, const int32_t *ids, int pairs, int top_k)
{
    const int t = threadIdx.x, lane = t & 63;
    if (t < kMaxE)
        rt.tokens[t] = 0;
    __syncthreads();
    for (int p = t; p < pairs; p += blockDim.x)
        atomicOr((unsigned long long *)&rt.tokens[ids[p]], 1ull << (p / top_k));   // any order gives the same bits
    __syncthreads();
    // prefix sums over the experts, one a thread: pairs below 65536, groups above
    uint32_t own = 0, sum = 0;
    if (t < kMaxE) {
        const uint32_t n = __popcll(rt.tokens[t]);
        own = sum = (n + 15) / 16 << 16 | n;
        for (int off = 1; off < 64; off <<= 1) {
            const uint32_t o = __shfl_up(sum, off);
            sum += lane >= off ? o : 0;
        }
        if (lane == 63)
            rt.sums[t >> 6] = sum;
    }
    __syncthreads();
    if (t < kMaxE) {
        for (int q = 0; q < t >> 6; ++q)
            sum += rt.sums[q];
        const uint32_t before = sum - own;
        rt.first[t] = (uint16_t)before;
        for (uint32_t k = 0; k < own >> 16; ++k) {
            rt.expert[(before >> 16) + k] = (uint8_t)t;
            rt.begin[(before >> 16) + k] = (uint16_t)(before + 16 * k);
        }
        if (t == kMaxE - 1) {
            rt.groups = (int)(sum >> 16);
            rt.begin[sum >> 16] = (uint16_t)sum;
        }
    }
    __syncthreads();
    for (int p = t; p < pairs; p += blockDim.x) {
        const int e = ids[p], nth = (int)__popcll(rt.tokens[e] & ((1ull << (p / top_k)) - 1));
        rt.pairs[rt.first[e] + nth] = (uint16_t)p;
    }
    for (int g = t; g < rt.groups; g += blockDim.x)
        for (int k = rt.begin[g]; k < rt.begin[g + 1]; ++k)
            rt.group_of[k] = (uint16_t)g;
    __syncthreads();
}

// ---- gate and up ------------------------------------------------------------
// Block: a group's tokens, 8 / S tiles of 16 columns of its expert's
// intermediate (16 gate rows and 16 up rows each), S waves a tile splitting the
// hidden columns. The tokens' activations lie in LDS by chunks of kc blocks;
// every wave streams its weights (see StreamItem). ROUTE: every block routes all
// tokens, a wave each, from the logits, and the first leaves `ids` for `down`.
// 8 tokens, 7 experts of 4096x14336: 102 us, 437 MB at 4.3 TB/s. Small experts
// lose by their starts: a block reads routing, tokens and first weights one
// after another (33 tokens, 44 experts of 1056x1408: 31 us, 70 MB at 2.3 TB/s).
// The fp16 form spills 7 to 8 registers a lane (its second pass, as in the
// products: one block below 2^-11 in one row of 64 takes that layer from 64 to 96 us).
constexpr int kUpWaves = 8;

template <typename TX, int S, bool ROUTE>
__global__ __launch_bounds__(64 * kUpWaves, 4) void k_mx4_moe_up(const TX *__restrict__ X, int pairs, int hidden,
                                                                 int inter, int top_k,
                                                                 const float *__restrict__ logits, int E, int renorm,
                                                                 int32_t *__restrict__ ids,
                                                                 const float *__restrict__ weights,
                                                                 const uint8_t *__restrict__ codes,
                                                                 const uint8_t *__restrict__ scales,
                                                                 bf16 *__restrict__ h)
{
    __shared__ Routed rt;
    __shared__ __align__(16) uint8_t lds[kStreamLds + 16 * 16];
    __shared__ int32_t own_ids[ROUTE ? kUpWaves * kMaxK : 1];
    __shared__ float own_weights[ROUTE ? kUpWaves * kMaxK : 1];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if constexpr (ROUTE) {
        if (wave * top_k < pairs) {
            int id = 0;
            float weight;
            choose(logits + wave * E, E, top_k, renorm, lane, id, weight);
            if (lane < top_k) {
                own_ids[wave * top_k + lane] = id;
                own_weights[wave * top_k + lane] = weight;
                if (blockIdx.x == 0 && blockIdx.y == 0)
                    ids[wave * top_k + lane] = id;
            }
        }
        __syncthreads();
        read_routing(rt, own_ids, pairs, top_k);
    } else {
        read_routing(rt, ids, pairs, top_k);
    }
    const int group = (int)blockIdx.y;
    if (group >= rt.groups)
        return;                    // fewer groups than blocks: the whole block leaves
    const int e = __builtin_amdgcn_readfirstlane(rt.expert[group]);
    const int nb = hidden / kMxBlock, r = lane & 15, c = lane >> 4, part = wave % S;
    const int col0 = ((int)blockIdx.x * (kUpWaves / S) + wave / S) * 16;
    const int64_t row = (int64_t)e * 2 * inter + (col0 < inter ? col0 : 0);          // past the end: not stored
    StreamRows<2> rows = {{codes + row * nb * 16, codes + (row + inter) * nb * 16},
                          {scales + row * nb, scales + (row + inter) * nb}};
    rows.lane(r, c, nb);
    const int items = (nb + kStreamBlocks - 1) / kStreamBlocks;

    const uint16_t *const list = rt.pairs + rt.begin[group];
    const int count = rt.size(group);
    const int kc = stream_chunk(count, nb), stride = kc * 64 + 16, per = kc / kStreamBlocks;
    const int xrow = (r < count ? r : count - 1) * stride + c * 16;
    F16Range range;
    f32x4 acc[1][2];
    auto contract = [&]<bool WIDE>() {
        mx4_zero(acc);
        StreamItem<2> a, b;
        int i = part;                              // the wave's items: part, part + S, ...
        bool in_a = true;                          // item i is in a
        if (i < items)
            stream_load(a, rows, i * kStreamBlocks, nb, c);
        for (int i0 = 0; i0 < items; i0 += per) {
            __syncthreads();                       // the LDS is free
            const int b0 = i0 * kStreamBlocks, len = (b0 + kc < nb ? kc : nb - b0) * 4;
            for (int m = wave; m < count; m += kUpWaves) {
                const TX *const x = X + ((int64_t)(list[m] / top_k) * nb + b0) * 32;
                for (int j = lane; j < len; j += 64)
                    *reinterpret_cast<u32x4 *>(lds + m * stride + j * 16) =
                        *reinterpret_cast<const u32x4 *>(x + j * 8);
            }
            __syncthreads();
            const int end = i0 + per < items ? i0 + per : items;
            auto one = [&](StreamItem<2> &cur, StreamItem<2> &next) {
                if (i + S < items)
                    stream_load(next, rows, (i + S) * kStreamBlocks, nb, c);
                const TX *const x[1] = {(const TX *)(lds + xrow + (i - i0) * kStreamBlocks * 64)};
                stream_compute<WIDE, false>(cur, x, acc, nb - i * kStreamBlocks, rows, -1, nb, c, range);
                i += S;
            };
            while (i < end) {
                if (in_a) {
                    one(a, b);
                    in_a = false;
                    if (i >= end)
                        break;
                }
                one(b, a);
                in_a = true;
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
        red[threadIdx.x * 2] = acc[0][0];
        red[threadIdx.x * 2 + 1] = acc[0][1];
        __syncthreads();
        if (part == 0) {
#pragma unroll
            for (int k = 1; k < S; ++k) {
                acc[0][0] += red[(threadIdx.x + 64 * k) * 2];
                acc[0][1] += red[(threadIdx.x + 64 * k) * 2 + 1];
            }
        }
    }
    if (part == 0 && col0 < inter) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (4 * c + k < count) {
                const int pair = list[4 * c + k];
                const float gate = acc[0][0][k], up = acc[0][1][k];
                const float v = gate / (1.0f + expf(-gate)) * up * (ROUTE ? own_weights : weights)[pair];
                // Two bf16 parts: 16 significant bits (an infinity stays in the first).
                // Of Y that costs 5e-6 (2-norm, 8 tokens, 2 of 8 experts of
                // 4096x14336), a three-hundredth of a bf16 Y's rounding; a third
                // part would be half as much again to read and multiply in `down`.
                const float hi = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & 0xFFFF0000u);
                bf16 *const out = h + (int64_t)pair * 2 * inter + col0 + r;
                out[0] = static_cast<bf16>(hi);
                out[inter] = static_cast<bf16>(v == hi ? 0.0f : v - hi);
            }
        }
    }
}

// ---- down -------------------------------------------------------------------
// The contraction is a list of units, 512 columns of one group's expert each, by
// group and column. A unit's activations are one row (1 KB of each part) for
// each of the group's tokens; a stage is as many units as have ROWS rows at
// most, in one of two LDS buffers. A stage's rows are on their way to registers
// while the one before it is multiplied, and so are every wave's next weights,
// across the stages' barriers. A unit's results, one row for each of its
// tokens, go to the wave's own sums of all tokens in LDS: an expert's NaN
// reaches its own tokens only, and the order of all additions is fixed. The
// units are shared out over gridDim.y blocks, whose fp32 sums k_mx4_moe_sum
// adds (`sums`: (gridDim.y, M, hidden)).
//
// Two ways to use a block's waves:
//   narrow: 16 hidden columns, the waves take a stage's units in turn. Nothing
//     is read ahead of need and every block starts with all of its loads, which
//     suits the smallest calls.
//   wide: 16 hidden columns a wave, each wave all units: the staged rows serve
//     all waves, which is what counts once tokens have more bytes than weights
//     (64 tokens x 8 experts of 4096x14336: 332 us narrow, 100 wide).
// 8 tokens, 7 experts of 4096x14336: 58 us, 218 MB at 3.8 TB/s.
constexpr int kPartBytes = 64 * kStreamBlocks, kRowBytes = 2 * kPartBytes + 16;    // in LDS, padded (see stream_chunk)

// Rows in unit order: group g's begin at per * begin[g], unit i's at + i *
// size. A stage: units u0 ... u0 + units - 1, rows r0 ... r0 + rows - 1.
struct Stage {                                         // uniform
    int u0, units, r0, rows;
};

template <int ROWS, int WAVES> struct DownRows {
    static constexpr int kRegs = (ROWS + WAVES - 1) / WAVES;       // rows a wave moves in a stage, at WAVES or more
    const Routed &rt;
    const bf16 *const h;
    const int nb, per, groups, end_unit, waves, wave, lane;
    u32x4 pre[kRegs][2];

    __device__ __forceinline__ void open(Stage &s, int u0) const
    {
        s.u0 = u0;
        s.units = s.rows = s.r0 = 0;
        if (u0 >= end_unit)
            return;
        const int g = u0 / per, i = u0 - g * per, count = rt.size(g);
        s.r0 = per * __builtin_amdgcn_readfirstlane(rt.begin[g]) + i * count;
        const int left = per - i, fit = ROWS / count;
        if (fit < left) {                              // ends inside this group
            s.units = fit < end_unit - u0 ? fit : end_unit - u0;
            s.rows = s.units * count;
            return;
        }
        // lane l: whether the stage holds all of the groups up to g + l
        const int end = per * rt.begin[g + lane < groups ? g + lane + 1 : groups] - s.r0;
        const int n = (int)__popcll(__ballot(g + lane < groups && end <= ROWS));   // a run from lane 0 on: ends grow
        s.rows = __builtin_amdgcn_readfirstlane(__shfl(end, n - 1));
        s.units = left + (n - 1) * per;
        if (g + n < groups) {                          // and some units of the next
            const int size = rt.size(g + n), more = (ROWS - s.rows) / size;
            s.units += more < per ? more : per - 1;
            s.rows += (more < per ? more : per - 1) * size;
        }
        if (s.units > end_unit - u0)                   // the rows past the last unit are moved, not used
            s.units = end_unit - u0;
    }
    __device__ __forceinline__ void fetch(const Stage &s)
    {
#pragma unroll
        for (int q = 0; q < kRegs; ++q)
            if (wave + q * waves < s.rows) {
                const int R = s.r0 + wave + q * waves, at = R / per;           // `at` lies among the group's pairs
                const int g = __builtin_amdgcn_readfirstlane(rt.group_of[at]), size = rt.size(g);
                const int begin = __builtin_amdgcn_readfirstlane(rt.begin[g]);
                const int local = R - per * begin, i = local / size;
                const int p = __builtin_amdgcn_readfirstlane(rt.pairs[begin + local - i * size]);
                const bf16 *const src = h + ((int64_t)p * 2 * nb + i * kStreamBlocks) * 32 + lane * 8;
                if (lane < (nb - i * kStreamBlocks) * 4) {
                    pre[q][0] = *reinterpret_cast<const u32x4 *>(src);
                    pre[q][1] = *reinterpret_cast<const u32x4 *>(src + nb * 32);
                }
            }
    }
    __device__ __forceinline__ void stash(const Stage &s, uint8_t *buf) const
    {                                                  // lanes past a row's end store what nothing reads
#pragma unroll
        for (int q = 0; q < kRegs; ++q)
            if (wave + q * waves < s.rows)
#pragma unroll
                for (int part = 0; part < 2; ++part)
                    *reinterpret_cast<u32x4 *>(buf + (wave + q * waves) * kRowBytes + part * kPartBytes + lane * 16) =
                        pre[q][part];
    }
};

template <typename TY, int TOK, int ROWS, bool WIDE>
__global__ __launch_bounds__(1024) void k_mx4_moe_down(const bf16 *__restrict__ h, int M, int hidden, int inter,
                                                       int top_k, const int32_t *__restrict__ ids,
                                                       const uint8_t *__restrict__ codes,
                                                       const uint8_t *__restrict__ scales, TY *__restrict__ Y,
                                                       float *__restrict__ sums)
{
    constexpr int kWaves = 16;                         // wide: at most, and 8 at least
    __shared__ __align__(16) uint8_t bufs[2][ROWS * kRowBytes];
    __shared__ float out[kWaves][TOK * 16];
    __shared__ Routed rt;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, c = lane >> 4, waves = WIDE ? (int)(blockDim.x >> 6) : kWaves;
    read_routing(rt, ids, M * top_k, top_k);
    const int groups = __builtin_amdgcn_readfirstlane(rt.groups);
    const int nb = inter / kMxBlock, per = (nb + kStreamBlocks - 1) / kStreamBlocks;   // units of a group
    const int first_unit = (int)((int64_t)per * groups * blockIdx.y / gridDim.y);
    const int end_unit = (int)((int64_t)per * groups * (blockIdx.y + 1) / gridDim.y);
    DownRows<ROWS, WIDE ? 8 : kWaves> act{rt, h, nb, per, groups, end_unit, waves, wave, lane, {}};

    const int tiles = hidden / 16;
    int tile = WIDE ? (int)blockIdx.x * waves + wave : (int)blockIdx.x;
    const bool idle = tile >= tiles;                   // wide: no columns left for this wave
    tile = idle ? tiles - 1 : tile;
    StreamRows<1> rows;
    rows.lane(r, c, nb);
    auto aim = [&](int u) -> int {                     // rows of the unit's expert; the unit's first block
        const int g = u / per;
        const int64_t row = (int64_t)__builtin_amdgcn_readfirstlane(rt.expert[g]) * hidden + tile * 16;
        rows.w[0] = codes + row * nb * 16;
        rows.s[0] = scales + row * nb;
        return (u - g * per) * kStreamBlocks;
    };

    for (int k = lane; k < TOK * 16; k += 64)
        out[wave][k] = 0.f;
    const int first = WIDE ? 0 : wave, step = WIDE ? 1 : kWaves;   // of a stage's units, this wave's
    Stage cur, nxt;
    act.open(cur, first_unit);
    act.fetch(cur);
    StreamItem<1> it;                                  // the wave's next unit, if `loaded`
    bool loaded = first < cur.units;
    if (loaded)
        stream_load(it, rows, aim(first_unit + first), nb, c);
    act.stash(cur, bufs[0]);
    act.open(nxt, cur.u0 + cur.units);
    act.fetch(nxt);
    __syncthreads();
    uint8_t *now = bufs[0], *then = bufs[1];
#pragma unroll 1
    while (cur.units) {
#pragma unroll 1
        for (int j = first; j < cur.units; j += step) {
            const int u = cur.u0 + j, g = u / per, i = u - g * per;
            const int count = rt.size(g), begin = __builtin_amdgcn_readfirstlane(rt.begin[g]);
            const int row0 = per * begin + i * count - cur.r0;
            const uint8_t *const row = now + (row0 + (r < count ? r : count - 1)) * kRowBytes + c * 16;
            const bf16 *const x[2] = {(const bf16 *)row, (const bf16 *)(row + kPartBytes)};
            const int ahead = j + step < cur.units ? u + step : first < nxt.units ? nxt.u0 + first : -1;
            loaded = ahead >= 0;
            const int next_b0 = loaded ? aim(ahead) : -1;
            f32x4 part[2][1];
            F16Range range;                            // of fp16 operands only
            mx4_zero(part);
            stream_compute<false, true>(it, x, part, nb - i * kStreamBlocks, rows, next_b0, nb, c, range);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (4 * c + k < count) {
                    const int tok = rt.pairs[begin + 4 * c + k] / top_k;
                    out[wave][tok * 16 + r] += part[0][0][k] + part[1][0][k];
                }
            // another lane may add to the same place next time
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
        if (!loaded && first < nxt.units) {            // nothing was left for it in this stage
            loaded = true;
            stream_load(it, rows, aim(nxt.u0 + first), nb, c);
        }
        act.stash(nxt, then);
        cur = nxt;
        act.open(nxt, cur.u0 + cur.units);
        act.fetch(nxt);
        __syncthreads();
        uint8_t *const t = now;
        now = then;
        then = t;
    }

    const int64_t part0 = blockIdx.y * (int64_t)M * hidden;
    if constexpr (WIDE) {
        if (!idle)
            for (int k = lane; k < M * 16; k += 64) {
                const int64_t at = (int64_t)(k >> 4) * hidden + tile * 16 + (k & 15);
                if (gridDim.y > 1)
                    sums[part0 + at] = out[wave][k];
                else
                    Y[at] = static_cast<TY>(out[wave][k]);
            }
    } else {
        __syncthreads();
        for (int k = threadIdx.x; k < M * 16; k += 64 * kWaves) {
            float sum = out[0][k];
#pragma unroll
            for (int w = 1; w < kWaves; ++w)
                sum += out[w][k];
            const int64_t at = (int64_t)(k >> 4) * hidden + tile * 16 + (k & 15);
            if (gridDim.y > 1)
                sums[part0 + at] = sum;
            else
                Y[at] = static_cast<TY>(sum);
        }
    }
}

// Y = the sum of Z parts of n fp32 values, in order.
template <typename TX>
__global__ __launch_bounds__(256) void k_mx4_moe_sum(const float *__restrict__ sums, int n, int Z, TX *__restrict__ Y)
{
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= n)
        return;
    float v = 0.f;
    int z = 0;
    for (; z + 8 <= Z; z += 8) {                       // eight loads in flight, added in order
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[k] = sums[(int64_t)(z + k) * n + i];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v += x[k];
    }
    for (; z < Z; ++z)
        v += sums[(int64_t)z * n + i];
    Y[i] = static_cast<TX>(v);
}

template <typename TX, int TOK>
void logits(const TX *X, int M, int hidden, const TX *router, int E, float *out, hipStream_t st)
{
    k_mx4_moe_logits<TX, TOK><<<dim3(E, (M + TOK - 1) / TOK), 256, 0, st>>>(X, M, hidden, router, E, out);
}

template <typename TX, int S, bool ROUTE = false>
void up(const TX *X, int pairs, int most, int hidden, int inter, int top_k, const float *logits, int E, int renorm,
        int32_t *ids, const float *weights, const uint8_t *gu, const uint8_t *gus, bf16 *h, hipStream_t st)
{
    const int tiles = inter / 16, per = kUpWaves / S;
    k_mx4_moe_up<TX, S, ROUTE><<<dim3((tiles + per - 1) / per, most), 64 * kUpWaves, 0, st>>>(
        X, pairs, hidden, inter, top_k, logits, E, renorm, ids, weights, gu, gus, h);
}

template <typename TY, int TOK, int ROWS, bool WIDE>
void down(const Mx4DownPlan &plan, const bf16 *h, int M, int hidden, int inter, int top_k, const int32_t *ids,
          const uint8_t *dn, const uint8_t *dns, TY *Y, float *sums, hipStream_t st)
{
    k_mx4_moe_down<TY, TOK, ROWS, WIDE><<<dim3(plan.blocks, plan.parts), 64 * plan.waves, 0, st>>>(
        h, M, hidden, inter, top_k, ids, dn, dns, Y, sums);
}

template <typename TX>
hipError_t moe(const void *X, int M, int hidden, int inter, int E, int top_k, int renorm, const void *router,
               const uint8_t *gu, const uint8_t *gus, const uint8_t *dn, const uint8_t *dns, void *Y, char *ws,
               hipStream_t st)
{
    const Mx4MoeWs lay = mx4_moe_ws_layout(M, hidden, inter, top_k);
    int32_t *const ids = (int32_t *)(ws + lay.ids_off);
    float *const weights = (float *)(ws + lay.w_off), *const lg = (float *)(ws + lay.logits_off);
    float *const sums = (float *)(ws + lay.sums_off);
    bf16 *const h = (bf16 *)(ws + lay.h_off);
    const TX *const x = (const TX *)X, *const rw = (const TX *)router;
    const int pairs = M * top_k, most = (pairs < E ? pairs : E) + (M > 16 ? pairs / 16 : 0);   // groups at most
    // Tokens a block: as many as still leave about a block a unit (a layer of 5
    // tokens, 8 experts of 1024x1024: one a block 22.5 us, four 23.2, eight 23.9).
    if (E * M <= 256)
        logits<TX, 1>(x, M, hidden, rw, E, lg, st);
    else if (M <= 4 || E * ((M + 7) / 8) <= 256)
        logits<TX, 4>(x, M, hidden, rw, E, lg, st);
    else
        logits<TX, 8>(x, M, hidden, rw, E, lg, st);
    // Waves a tile: as few as leave about two blocks a unit, since every block
    // reads the routing and its tokens first; with many columns to a wave two at
    // least (microseconds of a whole layer for S = 1, 2, 4, 8: 33 tokens, 4 of 48
    // experts of 1056x1408, 4928 tiles 60.9, 64.5, 71.2, 89.4; 16 tokens, 8 of 64 of
    // 2048x1024, 4096 tiles 65.3, 67.2, 74.5, 87.1; 2 tokens, 2 of 8 of 4096x14336,
    // 3584 tiles 99.7, 94.1, 98.6, 119; 4 tokens, 8 of 128 of 4096x1536, somewhat
    // fewer 96.5, 88.1, 91.7, 119; 1 token, 8 of 64 of 2048x1024, 512 tiles 30.7, 26.1,
    // 24.1, 24.1: waves beyond the items of 512 columns cost nothing there).
    const int64_t tiles = (int64_t)(inter / 16) * most;
    const int S = tiles >= 2048 && hidden < 4096 ? 1 : tiles >= 1536 ? 2 : tiles >= 768 ? 4 : 8;
    // With a wave for every token and blocks for about one round (S = 8), a launch
    // less: the blocks route for themselves.
    const bool route = S == 8 && M <= kUpWaves;
    if (!route)
        k_mx4_moe_topk<<<dim3(M), 64, 0, st>>>(lg, E, top_k, renorm, ids, weights);
    auto *const launch_up = S == 1 ? up<TX, 1> : S == 2 ? up<TX, 2> : S == 4 ? up<TX, 4>
                                 : route ? up<TX, 8, true> : up<TX, 8>;
    launch_up(x, pairs, most, hidden, inter, top_k, lg, E, renorm, ids, weights, gu, gus, h, st);
    const Mx4DownPlan plan = mx4_down_plan(M, hidden, inter, most);
    TX *const y = (TX *)Y;
    if (!plan.wide)
        down<TX, 16, 32, false>(plan, h, M, hidden, inter, top_k, ids, dn, dns, y, sums, st);
    else if (M <= 16)
        down<TX, 16, 32, true>(plan, h, M, hidden, inter, top_k, ids, dn, dns, y, sums, st);
    else
        down<TX, kMaxTok, 20, true>(plan, h, M, hidden, inter, top_k, ids, dn, dns, y, sums, st);
    if (plan.parts > 1)
        k_mx4_moe_sum<TX><<<dim3((M * hidden + 255) / 256), 256, 0, st>>>(sums, M * hidden, plan.parts, y);
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
