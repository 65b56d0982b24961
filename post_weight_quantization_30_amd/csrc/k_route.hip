// k_route.hip -- the choice of experts from router logits.
//
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e));  rank_e = s_e + b_e, or l_e without b
//   groups: the `top` groups whose `best` largest (s_e + b_e) have the largest sum stay;
//   ids: the top_k largest ranks there;  w = s there [/ their sum] * scale.
//
// A wave a token; expert e is register e / 64 of lane e % 64. Scores in 64 bits: the
// choice goes by differences that 32 bits lose (a sigmoid near 1, a bias much larger
// than the score). Bound by the issue of vector instructions, some 1000 a wave of 256
// experts in 8 groups: 8192 tokens 20.4 us, about half of it for the scores (64-bit exponentials
// and divisions of every expert) and half for the rounds of maxima (without groups 15.1, with
// one choice 10.8; 64 experts 8.8). 33 tokens of 48 3.5, a launch.
#include "awq_internal.h"

namespace awq {

namespace {

constexpr int kWaves = 4;                              // tokens a block

// Order of the ranks as whole numbers: -inf (masked) is 0, NaN below every number.
__device__ __forceinline__ uint64_t rank_key(double v)
{
    if (v != v)
        return 1;
    if (v == -__builtin_inf())
        return 0;
    v += 0.0;                                          // -0 and +0 are equal
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

// op over all lanes, in every lane: exchanges within 16 lanes by data-parallel moves, then
// of rows of 16 and of half waves. (By LDS permutes, six times two for each of a dozen
// maxima a token, they took most of the kernel: 8192 tokens, 256 experts, 8 groups 28 us.)
template <typename Op> __device__ __forceinline__ uint32_t over_wave(uint32_t v, Op op)
{
    v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));       // quad: 1 0 3 2
    v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));       // quad: 2 3 0 1
    v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));      // eight lanes mirrored
    v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true));      // sixteen mirrored
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = op(a[0], a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return op(b[0], b[1]);
}
template <typename Op> __device__ __forceinline__ double over_wave(double v, Op op)
{
    typedef uint32_t pair __attribute__((ext_vector_type(2)));
    auto moved = [&]<int CTRL>() {
        const pair w = __builtin_bit_cast(pair, v);
        return __builtin_bit_cast(double, pair{(uint32_t)__builtin_amdgcn_mov_dpp((int)w[0], CTRL, 0xF, 0xF, true),
                                               (uint32_t)__builtin_amdgcn_mov_dpp((int)w[1], CTRL, 0xF, 0xF, true)});
    };
    v = op(v, moved.template operator()<0xB1>());
    v = op(v, moved.template operator()<0x4E>());
    v = op(v, moved.template operator()<0x141>());
    v = op(v, moved.template operator()<0x140>());
    pair w = __builtin_bit_cast(pair, v);
    const auto a = __builtin_amdgcn_permlane16_swap(w[0], w[0], false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(w[1], w[1], false, false);
    v = op(__builtin_bit_cast(double, pair{a[0], b[0]}), __builtin_bit_cast(double, pair{a[1], b[1]}));
    w = __builtin_bit_cast(pair, v);
    const auto c = __builtin_amdgcn_permlane32_swap(w[0], w[0], false, false);
    const auto d = __builtin_amdgcn_permlane32_swap(w[1], w[1], false, false);
    return op(__builtin_bit_cast(double, pair{c[0], d[0]}), __builtin_bit_cast(double, pair{c[1], d[1]}));
}
__device__ __forceinline__ double wave_sum(double v)
{
    return over_wave(v, [](double a, double b) { return a + b; });
}

// Register and lane of the largest key of the wave, the lowest ones of equal keys; false
// where all keys are 0. The upper halves decide but for near ties.
template <int R> __device__ __forceinline__ bool largest(const uint64_t (&key)[R], int &reg, int &lane)
{
    auto most = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    uint32_t h = 0;
#pragma unroll
    for (int i = 0; i < R; ++i)
        h = most(h, (uint32_t)(key[i] >> 32));
    h = (uint32_t)__builtin_amdgcn_readfirstlane((int)over_wave(h, most));
    uint64_t has[R];
    int n = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        has[i] = __ballot((uint32_t)(key[i] >> 32) == h);
        n += __popcll(has[i]);
    }
    if (n > 1) {
        uint32_t l = 0;
#pragma unroll
        for (int i = 0; i < R; ++i)
            l = most(l, (uint32_t)(key[i] >> 32) == h ? (uint32_t)key[i] : 0u);
        l = (uint32_t)__builtin_amdgcn_readfirstlane((int)over_wave(l, most));
        if (h == 0 && l == 0)
            return false;
#pragma unroll
        for (int i = 0; i < R; ++i)
            has[i] = __ballot((uint32_t)(key[i] >> 32) == h && (uint32_t)key[i] == l);
    }
    reg = 0;
#pragma unroll
    for (int i = R - 1; i >= 0; --i)
        if (has[i]) {
            reg = i;
            lane = __ffsll((unsigned long long)has[i]) - 1;
        }
    return true;
}

// The two largest of (a, b) and (c, d), a >= b, c >= d.
__device__ __forceinline__ void merge2(double &a, double &b, double c, double d)
{
    b = a > c ? (b > c ? b : c) : (a > d ? a : d);
    a = a > c ? a : c;
}

template <typename T, int R>
__global__ __launch_bounds__(64 * kWaves) void k_route(const T *__restrict__ logits, int64_t M, int E,
                                                       const float *__restrict__ bias, int sigmoid, int groups,
                                                       int top, int best, int k, int renorm, float scale,
                                                       int32_t *__restrict__ ids, float *__restrict__ weights)
{
    __shared__ double ranks[kWaves][64 * R];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t m = (int64_t)blockIdx.x * kWaves + wave;
    if (m >= M)
        return;
    const T *const l = logits + m * E;
    double s[R], rank[R];
    double most = -__builtin_inf();
    bool nan = false;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int e = 64 * i + lane;
        s[i] = e < E ? static_cast<double>(static_cast<float>(l[e])) : -__builtin_inf();
        nan |= s[i] != s[i];
        most = fmax(most, s[i]);                       // a NaN is left out
    }
    nan = __any(nan);
    most = over_wave(most, [](double a, double b) { return a > b ? a : b; });
    double total = 0.0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const double x = s[i];
        rank[i] = x;
        if (sigmoid) {
            s[i] = 1.0 / (1.0 + exp(-x));
        } else {
            s[i] = x == most && x > -__builtin_inf() ? 1.0 : x == -__builtin_inf() ? 0.0 : exp(x - most);
            total += x != x ? 0.0 : s[i];
        }
    }
    if (!sigmoid) {
        total = wave_sum(total);
        if (total > 0.0)
#pragma unroll
            for (int i = 0; i < R; ++i)
                s[i] /= total;
    }
    // the scores that groups go by, and the ranks
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int e = 64 * i + lane;
        const double b = bias && e < E ? static_cast<double>(bias[e]) : 0.0;
        const bool masked = rank[i] == -__builtin_inf() || b == -__builtin_inf();
        const double sb = masked ? -__builtin_inf() : s[i] + b;
        ranks[wave][e] = sb;
        if (bias)
            rank[i] = sb;
    }
    if (groups > 1) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const int per = E / groups;
        uint64_t mine = 0;                             // lane `share` g: key of group g
        // `share` lanes a group, a power of two
        const int log_share = 31 - __clz(64 / groups), share = 1 << log_share, g = lane >> log_share;
        double a = -__builtin_inf(), b = a;
        for (int i = lane & (share - 1); i < per && g < groups; i += share) {
            double v = ranks[wave][g * per + i];
            v = v != v ? -1e300 : v;
            merge2(a, b, v, -__builtin_inf());
        }
        for (int off = 1; off < share; off <<= 1)
            merge2(a, b, __shfl_xor(a, off), __shfl_xor(b, off));
        // a second that is masked counts nothing; a group of masked experts ranks last
        if (g < groups && (lane & (share - 1)) == 0)
            mine = rank_key(best > 1 && b > -__builtin_inf() ? a + b : a) + 1;
        uint64_t keep = 0;
        for (int t = 0; t < top; ++t) {
            const uint64_t keys[1] = {mine};
            int reg, at = 0;
            largest<1>(keys, reg, at);                 // `groups` keys are not 0
            keep |= 1ull << (at >> log_share);
            if (lane == at)
                mine = 0;
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int e = 64 * i + lane;
            if (e < E && !(keep >> (e / per) & 1))
                rank[i] = -__builtin_inf();
        }
    }
    uint64_t key[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        key[i] = rank_key(rank[i]);
    int id = -1;                                       // lane j: choice j
    double w = 0.0;
    for (int j = 0; j < k; ++j) {
        int reg, at = 0;
        if (!largest<R>(key, reg, at))
            break;                                     // only masked experts are left
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (i == reg) {
                const uint64_t sv = __builtin_bit_cast(uint64_t, s[i]);
                const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)sv, at);
                const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(sv >> 32), at);
                if (lane == j) {
                    id = 64 * i + at;
                    w = __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
                }
                if (lane == at)
                    key[i] = 0;
            }
    }
    if (renorm) {
        const double sum = wave_sum(lane < k ? w : 0.0);
        if (sum > 0.0)
            w /= sum;
    }
    if (lane < k) {
        ids[m * k + lane] = id;
        weights[m * k + lane] = nan ? __builtin_nanf("") : static_cast<float>(w * static_cast<double>(scale));
    }
}

}  // namespace

hipError_t launch_route(const void *logits, int dtype, int64_t M, int E, const float *bias, int sigmoid, int groups,
                        int top, int best, int k, int renorm, float scale, int32_t *ids, float *weights, hipStream_t st)
{
    const uint32_t blocks = (uint32_t)((M + kWaves - 1) / kWaves);
    auto run = [&](auto *l) {
        typedef typename std::remove_const<typename std::remove_pointer<decltype(l)>::type>::type T;
#define ROUTE(R) k_route<T, R><<<blocks, 64 * kWaves, 0, st>>>(l, M, E, bias, sigmoid, groups, top, best, k, renorm, scale, ids, weights)
        if (E <= 64)
            ROUTE(1);
        else if (E <= 128)
            ROUTE(2);
        else if (E <= 256)
            ROUTE(4);
        else
            ROUTE(8);
#undef ROUTE
    };
    if (dtype == AWQ_F32)
        run((const float *)logits);
    else if (dtype == AWQ_F16)
        run((const f16 *)logits);
    else
        run((const bf16 *)logits);
    return hipGetLastError();
}

}  // namespace awq
