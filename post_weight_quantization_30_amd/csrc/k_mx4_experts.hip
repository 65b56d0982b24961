// k_mx4_experts.hip -- the experts of a given routing, MXFP8 activations, MXFP4 experts, any number of tokens.
//
//   g, u = Wg_e x, Wu_e x;  h = MXFP8(silu(g) u);  y = sum_j w_j Wd_{e_j} h_j
//
// A pair is a token and one of its choices. Launches: the pairs sorted by expert,
// and tiles of pairs of one expert; gate and up of the tiles, writing h; down, writing
// Wd h_j of every pair in fp32; the sum over a token's pairs in their order. A pair's
// results do not depend on the tile that it is in, so the order of an expert's pairs
// may differ from call to call, and results repeat bitwise. Up to 16 pairs, 8 of wide
// experts, go unsorted, in two launches.
// (us: 1 token, 8 of 64 experts of 2048x1024 17; 8, 2 of 8 of 4096x14336 164, bound by the
// weights of the seven that are hit, 4.0 TB/s; 203, 4 of 48 of 1056x1408 69: sort 5, up 39,
// down 20, sum 5; 2048, 8 of 64 of 2048x1024 267-288: sort 11, up 145-166, down 62, sum 29 for 134 MB
// of fp32 each way. One block sorts: 16384 pairs, which its registers hold, 10.6; 16392 17;
// 32768 32; 131072 119 of 1700; 2^20, of experts of 256x128, 1290 of 3130.)
#include "mx8_stream.h"
#include "mx8_tile.h"

namespace awq {

namespace {

constexpr int kMaxE = AWQ_MX4_EXPERTS_MAX_EXPERTS;

constexpr int kSmall = 16;                             // pairs of a tile where experts have few
constexpr int kSortKeep = 16;                          // pairs a thread of the sort keeps in registers

// Tiles of n pairs of one expert: LARGE of 256, what is left in one more of these, or if it
// is at most 128 pairs, in one that is done as 128.
template <bool LARGE> __device__ __forceinline__ int first_tiles(int n)
{
    return LARGE ? (n + 127) / 256 : (n + kSmall - 1) / kSmall;
}

// One block: pairs by expert into `list`, their places there into `place` (-1: no expert), tiles
// (expert, first place, pairs) into `tiles`, count[0] of them; LARGE: those of at most 128
// pairs last, so that the shorter ones fill the chip's last round. A pair's place among its
// expert's is the order in which the LDS counters were reached.
template <bool LARGE>
__global__ __launch_bounds__(1024) void k_experts_sort(const int32_t *__restrict__ ids, int64_t pairs, int E,
                                                       int32_t *__restrict__ list, int32_t *__restrict__ place,
                                                       int32_t *__restrict__ count, int4 *__restrict__ tiles)
{
    __shared__ int n[kMaxE], start[kMaxE], tile[kMaxE], last[kMaxE];
    const bool keep = pairs <= 1024 * kSortKeep;
    int expert[kSortKeep], rank[kSortKeep];
    for (int e = threadIdx.x; e < E; e += 1024)
        n[e] = 0;
    __syncthreads();
    if (keep) {
#pragma unroll
        for (int j = 0; j < kSortKeep; ++j) {
            const int64_t p = threadIdx.x + 1024 * j;
            expert[j] = p < pairs ? ids[p] : -1;
        }
#pragma unroll
        for (int j = 0; j < kSortKeep; ++j) {
            rank[j] = -1;
            if (expert[j] >= 0 && expert[j] < E)
                rank[j] = atomicAdd(&n[expert[j]], 1);
        }
    } else {
        for (int64_t p = threadIdx.x; p < pairs; p += 1024) {
            const int e = ids[p];
            if (e >= 0 && e < E)
                atomicAdd(&n[e], 1);
        }
    }
    __syncthreads();
    if (threadIdx.x < 64) {                            // sums over the experts before, 64 at a time
        int s = 0, t = 0, l = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int e = e0 + threadIdx.x, own = e < E ? n[e] : 0, own_t = first_tiles<LARGE>(own);
            const int own_l = LARGE && own > 256 * own_t;
            int a = own, b = own_t, c = own_l;
            for (int off = 1; off < 64; off <<= 1) {
                const int x = __shfl_up(a, off), y = __shfl_up(b, off), z = __shfl_up(c, off);
                if ((int)threadIdx.x >= off) {
                    a += x;
                    b += y;
                    c += z;
                }
            }
            if (e < E) {
                start[e] = s + a - own;
                tile[e] = t + b - own_t;
                last[e] = l + c - own_l;
            }
            s += __shfl(a, 63);
            t += __shfl(b, 63);
            l += __shfl(c, 63);
        }
        if (threadIdx.x == 0) {
            count[0] = t + l;
            count[1] = t;
        }
    }
    __syncthreads();
    const int firsts = tile[E - 1] + first_tiles<LARGE>(n[E - 1]);
    for (int e = threadIdx.x; e < E; e += 1024) {
        constexpr int size = LARGE ? 256 : kSmall;
        const int own_t = first_tiles<LARGE>(n[e]);
        int left = n[e], at = start[e];
        for (int i = 0; i < own_t; ++i, left -= size, at += size)
            tiles[tile[e] + i] = make_int4(e, at, left < size ? left : size, 0);
        if (left > 0)
            tiles[firsts + last[e]] = make_int4(e, at, left, 0);
    }
    if (keep) {
#pragma unroll
        for (int j = 0; j < kSortKeep; ++j) {
            const int64_t p = threadIdx.x + 1024 * j;
            if (p < pairs) {
                const int at = rank[j] < 0 ? -1 : start[expert[j]] + rank[j];
                if (at >= 0)
                    list[at] = (int)p;
                place[p] = at;
            }
        }
        return;
    }
    __syncthreads();
    for (int64_t p = threadIdx.x; p < pairs; p += 1024) {
        const int e = ids[p];
        int at = -1;
        if (e >= 0 && e < E) {
            at = atomicAdd(&start[e], 1);
            list[at] = (int)p;
        }
        place[p] = at;
    }
}

// Tile and column tile of this block. The blocks of one XCD (every eighth) take units of a
// tile and up to COLS column tiles, one after another, and the XCDs take the units in turn:
// each has its share of the shorter tiles at the end.
template <int COLS>
__device__ __forceinline__ bool tile_of_experts(int tiles, int columns, int &t, int &c)
{
    const int groups = (columns + COLS - 1) / COLS, i = blockIdx.x >> 3, unit = (i / COLS) * 8 + (blockIdx.x & 7);
    t = unit / groups;
    c = unit % groups * COLS + i % COLS;
    return t < tiles && c < columns;
}
template <int COLS> inline uint32_t experts_grid(int64_t tiles, int64_t columns)
{
    return (uint32_t)((tiles * tiles_of(columns, COLS) + 7) / 8 * 8 * COLS);
}

// Tile i, in scalar registers.
__device__ __forceinline__ int4 read_tile(const int4 *tiles, int i)
{
    const int4 t = tiles[i];
    return make_int4(__builtin_amdgcn_readfirstlane(t.x), __builtin_amdgcn_readfirstlane(t.y),
                     __builtin_amdgcn_readfirstlane(t.z), 0);
}

// h of 32 tokens (lanes r) and 32 columns, of which lane (r, half) has 8 (i / 4) + 4 half +
// i % 4 in register i: MXFP8 blocks, 16 bytes a lane.
__device__ __forceinline__ void store_h(const f32x16 &gate, const f32x16 &up, int half, bool there, uint8_t *codes,
                                        uint8_t *scale)
{
    float v[16];
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        v[i] = gate[i] / (1.0f + expf(-gate[i])) * up[i];
        a = umax(a, mx8_abs(v[i]));
    }
    a = umax(a, (uint32_t)__shfl_xor((int)a, 32));
    const uint32_t byte = mx8_byte(a);
    uint32_t d[4] = {0, 0, 0, 0};
    if (byte != 255) {
        const float s = mx8_factor(byte);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            d[j] = mx8_codes4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3], s);
    }
    // words 0, 2, 4, 6 | 1, 3, 5, 7 of the block to 0, 1, 2, 3 | 4, 5, 6, 7
    typedef uint32_t pair __attribute__((ext_vector_type(2)));
    const pair p = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
    const pair q = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
    if (there) {
        *reinterpret_cast<u32x4 *>(codes + 16 * half) = u32x4{p[0], p[1], q[0], q[1]};
        if (half == 0)
            *scale = (uint8_t)byte;
    }
}

// ---- many pairs an expert: large tiles (see mx8_tile.h) --------------------------------

// A tile of pairs x 128 columns of h: wave tiles of 32 gate rows and their 32 up rows.
// Products of eight columns exactly, as in k_experts_up: h is the same whatever the number of
// pairs and the type of Y. (What the matrix cores cut off would move an h next to a border
// to another 8-bit value, and all of an h where large products cancel: 2-norm of the error of Y
// 4.8e-4 where fp16's own is 2.1e-4, 1.8e-3 beside bf16's 1.7e-3.)
template <int MT>
__device__ __forceinline__ void up_tile(Tile8<MT> &lds, const int4 &t, int c0, const uint8_t *xc, const uint8_t *xs,
                                        int top_k, int nb, int inter, const int32_t *list, const uint8_t *gu,
                                        const uint8_t *gus, uint8_t *hc, uint8_t *hs)
{
    constexpr int BM = Tile8<MT>::BM;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    auto xrow = [&](int m) { return (int64_t)(list[t.y + (m < t.z ? m : t.z - 1)] / top_k); };
    const int64_t w0 = (int64_t)t.x * 2 * inter;
    // weight row n of the tile: wave column n / 64, gate or up, column n % 32
    auto wrow = [&](int n) {
        const int col = c0 + (n >> 6) * 32 + (n & 31);
        return (n >> 5 & 1) * inter + (col < inter ? col : inter - 1);
    };
    uint32_t xo[MT], wo[2];                            // M hidden and 2 inter hidden / 2: below 2^32
#pragma unroll
    for (int i = 0; i < MT; ++i)
        xo[i] = (uint32_t)xrow(tile8_xrow() + 64 * i) * (uint32_t)nb * 32 + tile8_xchunk() * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        wo[i] = (uint32_t)wrow(tile8_wrow() + 128 * i) * (uint32_t)nb * 16 + tile8_wchunk() * 16;
    const uint8_t *const sp = tid < BM ? xs + xrow(tid) * nb : gus + (w0 + wrow((tid - BM) & 255)) * nb;
    const bool words = (((uintptr_t)xs | (uintptr_t)gus | (uintptr_t)nb) & 3) == 0;
    f32x16 acc[MT][2];
    tile8_contract<true, true, MT>(lds, acc, xc, xo, gu + w0 * nb * 16, wo, sp, words, nb);
    const int r = lane & 31, h = lane >> 5, col = c0 + 32 * (wave & 3);
    if (col >= inter)
        return;
#pragma unroll
    for (int a = 0; a < MT; ++a) {
        const int m = 32 * MT * (wave >> 2) + 32 * a + r;
        const int64_t row = t.y + m;
        store_h(acc[a][0], acc[a][1], h, m < t.z, hc + row * inter + col, hs + row * (inter / 32) + col / 32);
    }
}

__global__ __launch_bounds__(512, 2) void k_experts_up_tile(const uint8_t *__restrict__ xc,
                                                            const uint8_t *__restrict__ xs, int top_k, int nb,
                                                            int inter, const int32_t *__restrict__ list,
                                                            const int32_t *__restrict__ count,
                                                            const int4 *__restrict__ tiles,
                                                            const uint8_t *__restrict__ gu,
                                                            const uint8_t *__restrict__ gus, uint8_t *__restrict__ hc,
                                                            uint8_t *__restrict__ hs)
{
    __shared__ __align__(16) union { Tile8<4> four; Tile8<2> two; } lds;
    int ti, ci;
    if (!tile_of_experts<4>(__builtin_amdgcn_readfirstlane(count[0]), (inter + 127) / 128, ti, ci))
        return;
    const int4 t = read_tile(tiles, ti);
    if (t.z > 128)
        up_tile<4>(lds.four, t, ci * 128, xc, xs, top_k, nb, inter, list, gu, gus, hc, hs);
    else
        up_tile<2>(lds.two, t, ci * 128, xc, xs, top_k, nb, inter, list, gu, gus, hc, hs);
}

// A tile of pairs x 256 rows of down. EXACT, here and in the other forms of down: products of
// eight columns exactly too, for an fp32 Y.
template <bool EXACT, int MT>
__device__ __forceinline__ void down_tile(Tile8<MT> &lds, const int4 &t, int n0, const uint8_t *hc, const uint8_t *hs,
                                          int nb, int hidden, const uint8_t *dn, const uint8_t *dns, float *part)
{
    constexpr int BM = Tile8<MT>::BM;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    auto xrow = [&](int m) { return m < t.z ? m : t.z - 1; };
    auto wrow = [&](int n) { return n0 + n < hidden ? n0 + n : hidden - 1; };
    const int64_t w0 = (int64_t)t.x * hidden;
    uint32_t xo[MT], wo[2];
    hc += (int64_t)t.y * nb * 32;
    hs += (int64_t)t.y * nb;
#pragma unroll
    for (int i = 0; i < MT; ++i)
        xo[i] = (uint32_t)xrow(tile8_xrow() + 64 * i) * (uint32_t)nb * 32 + tile8_xchunk() * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        wo[i] = (uint32_t)wrow(tile8_wrow() + 128 * i) * (uint32_t)nb * 16 + tile8_wchunk() * 16;
    const uint8_t *const sp = tid < BM ? hs + (int64_t)xrow(tid) * nb : dns + (w0 + wrow((tid - BM) & 255)) * nb;
    const bool words = (((uintptr_t)hs | (uintptr_t)dns | (uintptr_t)nb) & 3) == 0;
    f32x16 acc[MT][2];
    tile8_contract<false, EXACT, MT>(lds, acc, hc, xo, dn + w0 * nb * 16, wo, sp, words, nb);
    store_tiles<float, MT>(part + (int64_t)t.y * hidden, acc, reinterpret_cast<float *>(lds.x) + 2048 * wave,
                           32 * MT * (wave >> 2), n0 + 64 * (wave & 3), t.z, hidden, tid & 63);
}

template <bool EXACT>
__global__ __launch_bounds__(512, 2) void k_experts_down_tile(const uint8_t *__restrict__ hc,
                                                              const uint8_t *__restrict__ hs, int nb, int hidden,
                                                              const int32_t *__restrict__ count,
                                                              const int4 *__restrict__ tiles,
                                                              const uint8_t *__restrict__ dn,
                                                              const uint8_t *__restrict__ dns,
                                                              float *__restrict__ part)
{
    __shared__ __align__(16) union { Tile8<4> four; Tile8<2> two; } lds;
    int ti, ci;
    if (!tile_of_experts<4>(__builtin_amdgcn_readfirstlane(count[0]), (hidden + 255) / 256, ti, ci))
        return;
    const int4 t = read_tile(tiles, ti);
    if (t.z > 128)
        down_tile<EXACT, 4>(lds.four, t, ci * 256, hc, hs, nb, hidden, dn, dns, part);
    else
        down_tile<EXACT, 2>(lds.two, t, ci * 256, hc, hs, nb, hidden, dn, dns, part);
}

// ---- few pairs an expert: weights as a stream (see mx8_stream.h) --------------------------

// Up to kDirect pairs are not sorted: the pairs of an expert are a tile, which the first of
// them stands for, and every wave finds them for itself.
constexpr int kDirect = 16;
struct DirectPairs {
    int id, rank;                                      // lane l: pair l's expert (-1: none), rank among its pairs
    uint64_t first;                                    // the pairs that stand for a tile
    __device__ __forceinline__ DirectPairs(const int32_t *ids, int pairs, int E)
    {
        const int lane = threadIdx.x & 63;
        id = lane < pairs ? ids[lane] : -1;
        id = id < E ? id : -1;
        rank = 0;
        for (int i = 0; i < pairs; ++i)
            rank += i < lane && __builtin_amdgcn_readlane(id, i) == id;
        first = __ballot(id >= 0 && rank == 0);
    }
    // Pair p's tile: its expert and the number of its pairs, which go to `list`.
    __device__ __forceinline__ int4 tile(int p, int *list) const
    {
        const int e = __builtin_amdgcn_readlane(id, p);
        const bool mine = id == e;
        if (mine)
            list[rank] = threadIdx.x & 63;
        return make_int4(e, 0, __popcll(__ballot(mine)), 0);
    }
};

// A tile of up to 16 pairs and 64 / S columns of h, S waves a row tile: of every 32 columns
// two tiles of gate rows, two of up rows. Products of eight columns exactly: an h off by what
// the matrix cores cut off is rounded to another 8-bit value now and then. DIRECT: a block
// for each pair that begins a tile, h by the pair's number.
template <int S, bool DIRECT>
__global__ __launch_bounds__(512, 4) void k_experts_up(const uint8_t *__restrict__ xc, const uint8_t *__restrict__ xs,
                                                       int top_k, int nb, int inter, const int32_t *__restrict__ ids,
                                                       int pairs, int E, const int32_t *__restrict__ list,
                                                       const int32_t *__restrict__ count,
                                                       const int4 *__restrict__ tiles,
                                                       const uint8_t *__restrict__ gu,
                                                       const uint8_t *__restrict__ gus, uint8_t *__restrict__ hc,
                                                       uint8_t *__restrict__ hs)
{
    __shared__ __align__(16) union { StreamLds in; f32x4 red[8][64]; } lds;
    __shared__ float sums[8 / S][16][17];              // row tile, pair, row
    __shared__ int own[16];                            // the tile's pairs
    int ti, ci;
    if (!tile_of_experts<1>(DIRECT ? pairs : __builtin_amdgcn_readfirstlane(count[0]), (inter + 64 / S - 1) / (64 / S), ti,
                            ci))
        return;
    int4 t;
    if constexpr (DIRECT) {
        const DirectPairs all(ids, pairs, E);
        if (!(all.first >> ti & 1))
            return;
        t = all.tile(ti, own);                         // all waves write the same
    } else {
        t = read_tile(tiles, ti);
        if ((int)threadIdx.x < t.z)
            own[threadIdx.x] = list[t.y + threadIdx.x];
    }
    __syncthreads();
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, c = lane >> 4;
    const int rt = wave / S, col = ci * (64 / S) + (rt >> 2) * 32 + (rt & 1) * 16 + r;
    const int64_t n = (int64_t)t.x * 2 * inter + (rt >> 1 & 1) * inter + (col < inter ? col : inter - 1);
    f32x4 acc;
    stream_contract<true, S>(acc, lds.in, xc, xs, [&](int m) { return own[m] / top_k; }, t.z, gu + n * nb * 16,
                             gus + n * nb, wave % S, nb);
    if constexpr (S > 1) {                             // the waves' sums in wave order
        __syncthreads();
        lds.red[wave][lane] = acc;
        __syncthreads();
        if (wave % S == 0)
#pragma unroll
            for (int k = 1; k < S; ++k)
                acc += lds.red[wave + k][lane];
    }
    if (wave % S == 0)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sums[rt][4 * c + i][r] = acc[i];
    __syncthreads();
    // 8 columns of a pair a thread, 32 over four neighbours
    const int m = threadIdx.x >> 2 & 15, q = threadIdx.x & 3, g = threadIdx.x >> 6, first = ci * (64 / S) + 32 * g;
    if (g >= 2 / S || m >= t.z || first >= inter)
        return;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float gate = sums[4 * g + (q >> 1)][m][8 * (q & 1) + i], up = sums[4 * g + 2 + (q >> 1)][m][8 * (q & 1) + i];
        v[i] = gate / (1.0f + expf(-gate)) * up;
    }
    mx8_quantize8(v, hc, hs, (int64_t)(DIRECT ? own[m] : t.y + m) * (inter / 8) + first / 8 + q);
}

// Up to kDirect pairs: down of all of them and the sum over a token's. A block 16 rows; its
// waves take the tiles, each in `parts` of its items of 512 columns so that there are eight
// to sixteen of them, weights and h straight from memory. A pair's sums meet in
// LDS and are added up in the order of the parts and of the token's choices.
template <typename TY>
__global__ __launch_bounds__(512, 4) void k_experts_down_direct(const uint8_t *__restrict__ hc,
                                                                const uint8_t *__restrict__ hs, int nb, int hidden,
                                                                int M, int top_k, const int32_t *__restrict__ ids,
                                                                const float *__restrict__ weights, int E,
                                                                const uint8_t *__restrict__ dn,
                                                                const uint8_t *__restrict__ dns, TY *__restrict__ Y)
{
    constexpr bool EXACT = std::is_same<TY, float>::value;
    __shared__ float sums[8 * kDirect][17];            // part and pair, row
    __shared__ int own[8][16];
    const int pairs = M * top_k, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, c = lane >> 4, items = (nb + kItem - 1) / kItem, n0 = blockIdx.x * 16;
    const DirectPairs all(ids, pairs, E);
    const int tiles = __popcll(all.first);
    int parts = tiles > 2 ? 16 / tiles : 8;
    parts = parts < items ? parts : items;
    for (int u = wave; u < tiles * parts; u += 8) {
        uint64_t left = all.first;
        for (int i = u / parts; i > 0; --i)
            left &= left - 1;
        const int4 t = all.tile(__ffsll((unsigned long long)left) - 1, own[wave]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const int64_t n = (int64_t)t.x * hidden + n0 + r, m = own[wave][r < t.z ? r : t.z - 1];
        const uint8_t *const x = hc + m * nb * 32, *const xs = hs + m * nb, *const w = dn + n * nb * 16, *const ws = dns + n * nb;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        for (int i = u % parts; i < items; i += parts) {
            const int b = kItem * i + 4 * c, bx = kItem * i + 4 * (c >> 1);      // h as in mx8_stream.h
            u32x4 wr[4], x0[4], x1[4];
            const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                wr[k] = *reinterpret_cast<const u32x4 *>(w + (int64_t)(b + k < nb ? b + k : nb - 1) * 16);
                x0[k] = bx + k < nb ? *reinterpret_cast<const u32x4 *>(x + (int64_t)(bx + k) * 32 + 16 * (c & 1)) : zero;
                x1[k] = bx + 8 + k < nb ? *reinterpret_cast<const u32x4 *>(x + (int64_t)(bx + 8 + k) * 32 + 16 * (c & 1)) : zero;
            }
            const uint32_t sx = mx4_scales4(xs, b, nb), sw = mx4_scales4(ws, b, nb);
            auto step = [&]<int U>() {
                i32x8 high = join(x0[U], x1[U]), low;
                if constexpr (EXACT)
                    mx8_parts(join(x0[U], x1[U]), high, low);
                acc = mfma16_a8<U>(high, sx, wr[U], sw, acc);
                if constexpr (EXACT)
                    acc = mfma16_a8<U>(low, sx, wr[U], sw, acc);
            };
            step.template operator()<0>();
            step.template operator()<1>();
            step.template operator()<2>();
            step.template operator()<3>();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (4 * c + i < t.z)
                sums[(u % parts) * kDirect + own[wave][4 * c + i]][r] = acc[i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    for (int m = threadIdx.x >> 4; m < M; m += 32) {
        const int row = threadIdx.x & 15;
        float y = 0.f;
        for (int j = 0; j < top_k; ++j) {
            const int p = m * top_k + j, e = ids[p];
            if (e < 0 || e >= E)
                continue;
            float s = sums[p][row];
            for (int k = 1; k < parts; ++k)
                s += sums[k * kDirect + p][row];
            y += weights[p] * s;
        }
        Y[(int64_t)m * hidden + n0 + row] = static_cast<TY>(y);
    }
}

// A tile and 128 / S rows of down, S waves a row tile.
template <int S, bool EXACT>
__global__ __launch_bounds__(512, 4) void k_experts_down(const uint8_t *__restrict__ hc, const uint8_t *__restrict__ hs,
                                                         int nb, int hidden, const int32_t *__restrict__ count,
                                                         const int4 *__restrict__ tiles,
                                                         const uint8_t *__restrict__ dn,
                                                         const uint8_t *__restrict__ dns, float *__restrict__ part)
{
    __shared__ __align__(16) union { StreamLds in; f32x4 red[8][64]; } lds;
    int ti, ci;
    if (!tile_of_experts<1>(__builtin_amdgcn_readfirstlane(count[0]), (hidden + 128 / S - 1) / (128 / S), ti, ci))
        return;
    const int4 t = read_tile(tiles, ti);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, c = lane >> 4;
    const int n0 = ci * (128 / S) + wave / S * 16 + r;
    const int64_t n = (int64_t)t.x * hidden + (n0 < hidden ? n0 : hidden - 1);
    f32x4 acc;
    stream_contract<EXACT, S>(acc, lds.in, hc, hs, [&](int m) { return t.y + m; }, t.z, dn + n * nb * 16, dns + n * nb,
                              wave % S, nb);
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
        if (4 * c + i < t.z && n0 < hidden)
            part[(int64_t)(t.y + 4 * c + i) * hidden + n0] = acc[i];
}

// y = sum_j w_j (Wd h_j) in the order of j; pairs without an expert are left out.
template <typename TY>
__global__ __launch_bounds__(256) void k_experts_sum(const float *__restrict__ part, const int32_t *__restrict__ place,
                                                     const float *__restrict__ weights, int64_t M, int top_k,
                                                     int hidden, TY *__restrict__ Y)
{
    typedef TY piece __attribute__((ext_vector_type(4)));
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, m = at / (hidden / 4);
    if (m >= M)
        return;
    const int64_t col = at % (hidden / 4) * 4;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int j = 0; j < top_k; ++j) {
        const int p = place[m * top_k + j];
        const float w = weights[m * top_k + j];
        if (p >= 0)
            s += w * *reinterpret_cast<const f32x4 *>(part + (int64_t)p * hidden + col);
    }
    piece y;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        y[i] = static_cast<TY>(s[i]);
    *reinterpret_cast<piece *>(Y + m * hidden + col) = y;
}

}  // namespace

hipError_t launch_mx4_experts(const uint8_t *xc, const uint8_t *xs, int64_t M, int hidden, int inter, int experts,
                              int top_k, const int32_t *ids, const float *weights, const uint8_t *gu,
                              const uint8_t *gus, const uint8_t *dn, const uint8_t *dns, void *Y, int y_dtype, void *ws,
                              hipStream_t st)
{
    const Mx4ExpertsWs l = mx4_experts_ws_layout(M, hidden, inter, experts, top_k);
    char *const base = (char *)ws;
    int32_t *const list = (int32_t *)(base + l.list_off), *const count = (int32_t *)(base + l.count_off);
    int32_t *const place = (int32_t *)(base + l.place_off);
    int4 *const tiles = (int4 *)(base + l.tiles_off);
    uint8_t *const hc = (uint8_t *)(base + l.hc_off), *const hs = (uint8_t *)(base + l.hs_off);
    float *const part = (float *)(base + l.part_off);
    const int64_t pairs = M * top_k, hit = pairs < experts ? pairs : experts;
    if (pairs <= (inter >= 4096 ? kDirect / 2 : kDirect)) {
        // Two launches instead of four (us unsorted and sorted, 1 token, 8 of 64 experts of
        // 2048x1024 17, 25; 2 tokens 23, 29; 8 of 16 experts with hidden 4096, 1 token and 2: inter 2048
        // 33, 40 and 57, 64; inter 4096 57, 66 and 95, 105, where the rule is early; inter 8192 105, 110 and
        // 179, 170). Long streams of many pairs hide the sort: 2 of 8 experts of
        // 4096x14336, 1 token 44, 47; 4 tokens 126, 126; 8 tokens 176, 164.
        k_experts_up<2, true><<<experts_grid<1>(pairs, inter / 32), 512, 0, st>>>(
            xc, xs, top_k, hidden / 32, inter, ids, (int)pairs, experts, nullptr, nullptr, nullptr, gu, gus, hc, hs);
        auto down = [&](auto *y) {
            k_experts_down_direct<<<(uint32_t)(hidden / 16), 512, 0, st>>>(hc, hs, inter / 32, hidden, (int)M, top_k, ids,
                                                                          weights, experts, dn, dns, y);
        };
        if (y_dtype == AWQ_F32)
            down((float *)Y);
        else if (y_dtype == AWQ_F16)
            down((f16 *)Y);
        else
            down((bf16 *)Y);
        return hipGetLastError();
    }
    // Large tiles from 24 pairs an expert on (us by tiles and by streams, 8 of 64 experts of
    // 2048x1024: 64 tokens, 8 pairs an expert, 102, 78; 100 tokens 103, 83; 150 tokens, 19 pairs,
    // 104, 98; 200 tokens, 25 pairs, 105, 112; 300 tokens 104, 142; 4 of 48 of 1056x1408, which
    // would rather have it later: 17 pairs an expert 104, 69; 25 pairs 105, 83; 33 pairs 106, 94).
    // The host does not know how many experts are hit: few of many with all pairs stream.
    if (pairs >= 24 * (int64_t)experts) {
        const int64_t most = pairs / 256 + hit;
        k_experts_sort<true><<<1, 1024, 0, st>>>(ids, pairs, experts, list, place, count, tiles);
        k_experts_up_tile<<<experts_grid<4>(most, tiles_of(inter, 128)), 512, 0, st>>>(
            xc, xs, top_k, hidden / 32, inter, list, count, tiles, gu, gus, hc, hs);
        auto down = [&](auto exact) {
            k_experts_down_tile<exact.value><<<experts_grid<4>(most, tiles_of(hidden, 256)), 512, 0, st>>>(
                hc, hs, inter / 32, hidden, count, tiles, dn, dns, part);
        };
        if (y_dtype == AWQ_F32)
            down(std::true_type());
        else
            down(std::false_type());
    } else {
        const int64_t most = pairs / kSmall + hit;
        k_experts_sort<false><<<1, 1024, 0, st>>>(ids, pairs, experts, list, place, count, tiles);
        k_experts_up<1, false><<<experts_grid<1>(most, tiles_of(inter, 64)), 512, 0, st>>>(
            xc, xs, top_k, hidden / 32, inter, ids, (int)pairs, experts, list, count, tiles, gu, gus, hc, hs);
        // (us a layer by one, two, four waves a row tile: 203 tokens, 4 of 48 experts of 1056x1408 72,
        // 69.5, 71; 64, 8 of 64 of 2048x1024 78.5, 78.5, 88; 16, 4 of 16 of 4096x2048 68, 68, 70, of
        // 4096x8192 205, 199, 201; 8, 2 of 8 of 4096x14336 163, 166, 164)
        auto down = [&]<int S, bool EXACT>() {
            k_experts_down<S, EXACT><<<experts_grid<1>(most, tiles_of(hidden, 128 / S)), 512, 0, st>>>(
                hc, hs, inter / 32, hidden, count, tiles, dn, dns, part);
        };
        if (inter >= 4096 && y_dtype == AWQ_F32)
            down.template operator()<4, true>();
        else if (inter >= 4096)
            down.template operator()<4, false>();
        else if (y_dtype == AWQ_F32)
            down.template operator()<2, true>();
        else
            down.template operator()<2, false>();
    }
    const uint32_t blocks = (uint32_t)((M * (hidden / 4) + 255) / 256);
    if (y_dtype == AWQ_F32)
        k_experts_sum<<<blocks, 256, 0, st>>>(part, place, weights, M, top_k, hidden, (float *)Y);
    else if (y_dtype == AWQ_F16)
        k_experts_sum<<<blocks, 256, 0, st>>>(part, place, weights, M, top_k, hidden, (f16 *)Y);
    else
        k_experts_sum<<<blocks, 256, 0, st>>>(part, place, weights, M, top_k, hidden, (bf16 *)Y);
    return hipGetLastError();
}

}  // namespace awq
