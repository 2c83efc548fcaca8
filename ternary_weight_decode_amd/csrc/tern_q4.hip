// tern_q4.hip — 4-bit weights with group scales: load-time packing and the
// GEMV / small-M GEMM (bf16 or int8 activations) on the matrix cores.
//
//   y[m][n] = sum_g scale[n][g] sum_{k in g} t[n][k] x[m][k],  t in [-8, 7]
//
// Layout (include/tern.h): 16-row tiles; a 128-k block of a tile is 1 KiB in
// which lane (r, g) of a matrix-core operand has its 32 weights side by side,
// a word for each 32 k: k = 32c + 8g + i of word c.  Any 32 neighbours of k are
// one step of the matrix cores, so every group size sums its own products.
#include "tern_device.h"
#include "tern_launch.h"

namespace tern {

typedef _Float16 q4_f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 q4_f16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 q4_mfma(u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(q4_f16x8, a), __builtin_bit_cast(q4_f16x8, b), c,
                                                  0, 0, 0);
}

// Eight weights of a word to fp16, exact: the low byte of 1024 + v is v, and
// t + 8 = (t & 15) ^ 8; the nibbles at bit 4 stand for 16 (t + 8) there.  (Whole
// numbers put into the mantissa of a constant, the known way from packed bits to
// fp16: Kim, Henry, Fahim, Awadalla, "Who Says Elephants Can't Run", 2022.)
__device__ __forceinline__ u32x4 q4_decode(uint32_t w)
{
    const q4_f16x2 off = {(_Float16)1032.0f, (_Float16)1032.0f};
    const q4_f16x2 by = {(_Float16)0.0625f, (_Float16)0.0625f}, off16 = {(_Float16)72.0f, (_Float16)72.0f};
    const uint32_t v = w >> 8;
    const uint32_t x0 = (w & 0x000F000Fu) ^ 0x64086408u, x1 = (w & 0x00F000F0u) ^ 0x64806480u;
    const uint32_t x2 = (v & 0x000F000Fu) ^ 0x64086408u, x3 = (v & 0x00F000F0u) ^ 0x64806480u;
    const auto low = [&](uint32_t x) {
        return __builtin_bit_cast(uint32_t, (q4_f16x2)(__builtin_bit_cast(q4_f16x2, x) - off));
    };
    const auto high = [&](uint32_t x) {
        return __builtin_bit_cast(
            uint32_t, (q4_f16x2)__builtin_elementwise_fma(__builtin_bit_cast(q4_f16x2, x), by, -off16));
    };
    return u32x4{low(x0), high(x1), low(x2), high(x3)};
}

// ------------------------------------------------------------------ pack

// One thread per word: its eight weights, and for the first word of a group's
// row its scale.  Rows from N on are padding, written as zeros.
__global__ void q4_pack_kernel(const int8_t* __restrict__ t, const uint16_t* __restrict__ scale, int64_t N, int64_t K,
                               int group, uint32_t* __restrict__ words, uint16_t* __restrict__ scales)
{
    const int64_t nb = K / 128, total = npad16(N) * K / 8;
    for (int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; id < total;
         id += (int64_t)gridDim.x * blockDim.x) {
        const int c = (int)(id & 3), r = (int)(id >> 2 & 15), g = (int)(id >> 6 & 3);
        const int64_t tile = id >> 8, rt = tile / nb, b = tile - rt * nb, n = rt * 16 + r;
        const int64_t k = b * 128 + 32 * c + 8 * g;
        uint32_t w = 0;
        if (n < N) {
            const u32x2 x = *(const u32x2*)(t + n * K + k);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                int v = (int8_t)(x[i >> 2] >> 8 * (i & 3));
                v = v < -8 ? -8 : v > 7 ? 7 : v;
                w |= (uint32_t)(v & 15) << (16 * (i & 1) + 4 * (i >> 1));
            }
        }
        words[id] = w;
        if (g == 0 && k % group == 0) {
            const int64_t kt = b >> 2, bq = b & 3, nbq = nb - 4 * kt < 4 ? nb - 4 * kt : 4, per = 128 / group;
            scales[((rt * nb + 4 * kt) * 16 + r * nbq + bq) * per + 32 * c / group] =
                n < N ? scale[n * (K / group) + k / group] : 0;
        }
    }
}

// ------------------------------------------------------------------ GEMV

// A unit is BLK blocks (128 k) of a row tile.  Wave w of a workgroup has the
// units w, w + waves, ... along K, each for the R row tiles of the workgroup.
// The weights of up to four of these are under way at once; meanwhile the wave
// turns its own slice of x into matrix-core operands, which stay in registers
// for all row tiles (no other wave is waited for).  The waves meet once, in LDS,
// where their sums are added in order of K.
//
// x: a slice of a row is divided by a power of two that takes its largest value
// to [2^14, 2^15) and rounded to fp16: exact down to 2^-29 of the largest (bf16
// has 8 bits, fp16 11), and to 2^-39 of it below.  fp16 because eight weights
// become operands in nine instructions there; exact bf16 ones would take 14.
// int8 weights are the nibbles where they stand, times 16: three instructions.
//
// What bounds it: the weights' bytes and a launch (in a graph of calls over weights
// out of memory; 24576 x 4096, groups of 128, 52 MB: one row in int8 10.2 us, 5.1
// TB/s with the 1.9 us of an empty launch in it, in bf16 11.1; 16 rows 12.0 and
// 13.6).  A long K with many rows: x, which every workgroup reads (4096 x 12288,
// groups of 64, 27 MB, int8: one row 6.3 us, 7 rows 7.7, 16 rows 10.2, bf16 7.6,
// 11.8 and 16.5).

// operand of one step of 32 k: 8 activations
template <bool I8>
struct Q4Op {
    typedef u32x4 type;
    type v;
};
template <>
struct Q4Op<true> {
    typedef u32x2 type;
    type v;
};

// 8 activations of bf16, times 2^(14 - ex)
__device__ __forceinline__ u32x4 q4_half(u32x4 x, float up)
{
    u32x4 h;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const q4_f16x2 v = {(_Float16)(__builtin_bit_cast(float, x[e] << 16) * up),
                            (_Float16)(__builtin_bit_cast(float, x[e] & 0xFFFF0000u) * up)};
        h[e] = __builtin_bit_cast(uint32_t, v);
    }
    return h;
}

// largest of two bf16 magnitudes each in two 16-bit halves
typedef uint16_t q4_u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t q4_most(uint32_t top, uint32_t x)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(q4_u16x2, top),
                                                                  __builtin_bit_cast(q4_u16x2, x & 0x7FFF7FFFu)));
}

// powers of two into fp16's range and back, from the bf16 bits of a slice's
// largest value; slices below 2^-112 stay below, an infinity or a NaN stays one
__device__ __forceinline__ void q4_range(uint32_t top, float& up, float& down)
{
    int ex = (int)(top >> 7) - 127;
    ex = ex > 127 ? 14 : ex < -112 ? -112 : ex;
    up = __builtin_bit_cast(float, (uint32_t)(127 + 14 - ex) << 23);
    down = __builtin_bit_cast(float, (uint32_t)(127 + ex - 14) << 23);
}

// the largest over rows of 16 lanes, and over 2 or 4 such rows
template <int CTRL>
__device__ __forceinline__ uint32_t q4_dpp_max(uint32_t v)
{
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
    return o > v ? o : v;
}
template <int LANES>
__device__ __forceinline__ uint32_t q4_max(uint32_t v)
{
    static_assert(LANES == 16 || LANES == 32, "rows of a slice");
    v = q4_dpp_max<0xB1>(v);           // lanes 1 apart, 2 apart, mirrored in 8 and in 16
    v = q4_dpp_max<0x4E>(v);
    v = q4_dpp_max<0x141>(v);
    v = q4_dpp_max<0x140>(v);
    if constexpr (LANES == 32) {
        const auto o = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = o[0] > o[1] ? o[0] : o[1];
    }
    return v;
}
// over the four lanes of a row r
__device__ __forceinline__ uint32_t q4_max_rows(uint32_t v)
{
    const auto o = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = o[0] > o[1] ? o[0] : o[1];
    const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return p[0] > p[1] ? p[0] : p[1];
}

// eight int8 activations in the order of the decoded weights (0, 4, 1, 5, 2, 6, 3, 7)
__device__ __forceinline__ u32x2 q4_order(u32x2 q)
{
    return u32x2{__builtin_amdgcn_perm(q[1], q[0], 0x05010400u), __builtin_amdgcn_perm(q[1], q[0], 0x07030602u)};
}

// Rows of x that go through LDS, 0: none.  There a slice is loaded row by row,
// as it lies; straight into the operands' order every load touches all rows and
// a part of a line of each.  int8 always (4096 x 12288, 16 rows: 10.4 us, 15.2
// straight); bf16 finds a row's largest value in the 16 loads that are one lane's
// own when straight, so many rows go that way (16 rows 17.0 us, through LDS 17.8),
// and 5 to 8 where few row tiles use what is loaded (12.2, straight 14.5; 24576 x
// 4096, six row tiles, 14.2 and 12.5).
template <bool I8, int MT, int R>
constexpr int q4_staged() { return I8 || MT <= 4 || (MT == 8 && R <= 2) ? MT : 0; }

constexpr int kQ4Ahead = 4;

template <bool I8, int MT, int PER, int BLK, int R>
__global__ __launch_bounds__(1024) void q4_gemv_kernel(const uint8_t* __restrict__ packed, int64_t N, int64_t K,
                                                       const void* __restrict__ x, const float* __restrict__ s_x,
                                                       int M, float* __restrict__ y)
{
    constexpr int NI = MT < 4 ? MT : 4, C = 4 * BLK;       // live values of a lane's sums; steps of a unit
    constexpr int kLanes = MT <= 4 ? 16 : 4 * MT;          // lanes that hold sums
    constexpr int kStage = q4_staged<I8, MT, R>();            // rows of x that go through LDS
    constexpr int P = R < kQ4Ahead ? R : kQ4Ahead;         // row tiles whose weights are under way
    constexpr int kPass = 4 / BLK, kLoads = kStage > 0 ? (kStage + kPass - 1) / kPass : C;
    extern __shared__ __align__(16) uint8_t smem[];        // slices [waves][16 BLK][rows], then sums
    typedef typename Q4Op<I8>::type Op;
    const int nw = blockDim.x >> 6, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int nb = (int)(K >> 7), nu = (nb + BLK - 1) / BLK;
    const int64_t nrt = (N + 15) >> 4;
    Op* const stage = (Op*)smem + wave * (16 * BLK * kStage);
    float* const red = (float*)(smem + (size_t)nw * 16 * BLK * kStage * sizeof(Op));   // [R][waves][NI][kLanes]
    const TERN_GLOBAL uint8_t* codes = (const TERN_GLOBAL uint8_t*)packed;
    const TERN_GLOBAL uint8_t* scales = codes + q4_code_bytes(N, K);

    for (int u = wave; u < nu; u += nw) {
        const int valid = (int)K - u * (128 * BLK);        // k of this unit that are there; the rest counts as 0
        // x, then the weights
        Op raw[kLoads];
#pragma unroll
        for (int c = 0; c < kLoads; ++c) {
            int m = kStage > 0 ? kPass * c + lane / (16 * BLK) : r, k = kStage > 0 ? lane % (16 * BLK) * 8 : 32 * c + 8 * g;
            m = m < M ? m : M - 1;
            k = k < valid ? k : valid - 8;
            raw[c] = *(const TERN_GLOBAL Op*)((const TERN_GLOBAL uint8_t*)x +
                                              ((int64_t)m * K + u * (128 * BLK) + k) * (sizeof(Op) / 8));
        }
        __builtin_amdgcn_sched_barrier(0);
        u32x4 w[P][BLK];
        uint32_t sc[P][(BLK * PER + 1) / 2];
        const int kt = u * BLK >> 2, bq = u * BLK & 3, nbq = nb - 4 * kt < 4 ? nb - 4 * kt : 4;
        const auto load = [&](int i) {
            int64_t rt = (int64_t)blockIdx.x * R + i;
            rt = rt < nrt ? rt : nrt - 1;
            const TERN_GLOBAL uint8_t* base = codes + (rt * nb + u * BLK) * 1024 + lane * 16;
#pragma unroll
            for (int b = 0; b < BLK; ++b) w[i % P][b] = ld_nt16(base + (b * 128 < valid ? b : 0) * 1024);
            const TERN_GLOBAL uint8_t* s = scales + ((rt * nb + 4 * kt) * 16 + r * nbq + bq) * (2 * PER);
            constexpr int kWords = (BLK * PER + 1) / 2;
            if constexpr (BLK * PER == 1) {
                sc[i % P][0] = *(const TERN_GLOBAL uint16_t*)s;
            } else if (BLK == 1 || nbq % 2 == 0) {         // a unit's scales side by side
                typedef uint32_t vec __attribute__((ext_vector_type(kWords)));
                const vec v = *(const TERN_GLOBAL vec*)s;
#pragma unroll
                for (int j = 0; j < kWords; ++j) sc[i % P][j] = v[j];
            } else {                                       // the last blocks of an odd number
                const bool two = valid > 128;
                if constexpr (PER == 1) {
                    sc[i % P][0] = ((const TERN_GLOBAL uint16_t*)s)[0] |
                                   (two ? ((const TERN_GLOBAL uint16_t*)s)[1] << 16 : 0);
                } else {
#pragma unroll
                    for (int j = 0; j < kWords; ++j)
                        sc[i % P][j] = two || j < kWords / 2 ? ((const TERN_GLOBAL uint32_t*)s)[j] : 0;
                }
            }
        };
#pragma unroll
        for (int i = 0; i < P; ++i) load(i);
        __builtin_amdgcn_sched_barrier(0);

        Op a[C];
        float back[NI];
        if constexpr (kStage > 0) {
            // a slot's rows side by side; lanes that write one row of many slots, and
            // lanes that read all rows of a few, meet all banks
            constexpr int kSpan = 256 / (int)sizeof(Op) / kStage;
            const auto place = [](int slot, int m) { return slot * kStage + (m ^ (slot / kSpan & (kStage - 1))); };
            const int slot = lane % (16 * BLK);
            const bool in = slot * 8 < valid;
#pragma unroll
            for (int c = 0; c < kLoads; ++c) {
                const int m = kPass * c + lane / (16 * BLK);
                Op o = in ? raw[c] : Op{};
                if constexpr (I8) {
                    o = q4_order(o);
                } else {
                    uint32_t top = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = q4_most(top, o[e]);
                    top = q4_max<16 * BLK>(top >> 16 > (top & 0xFFFFu) ? top >> 16 : top & 0xFFFFu);
                    float up, down;
                    q4_range(top, up, down);
                    o = q4_half(o, up);
                    // the lane's own sums are rows 4 g + e
#pragma unroll
                    for (int e = 0; e < NI; ++e)
#pragma unroll
                        for (int q = 0; 4 * q + e < MT; ++q)
                            if ((4 * q + e) / kPass == c) {
                                const float f = __builtin_bit_cast(
                                    float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, down),
                                                                     (4 * q + e) % kPass * 16 * BLK));
                                back[e] = q == 0 || g == q ? f : back[e];
                            }
                }
                if (m < kStage) stage[place(slot, m)] = o;
            }
            __builtin_amdgcn_wave_barrier();               // a slice is its wave's own
            const int m = r < kStage ? r : kStage - 1;
#pragma unroll
            for (int c = 0; c < C; ++c) a[c] = stage[place(c * 4 + g, m)];
        } else if constexpr (I8) {
#pragma unroll
            for (int c = 0; c < C; ++c) a[c] = 32 * c < valid ? q4_order(raw[c]) : Op{};
        } else {
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (32 * c >= valid) raw[c] = Op{};
#pragma unroll
                for (int e = 0; e < 4; ++e) top = q4_most(top, raw[c][e]);
            }
            top = q4_max_rows(top >> 16 > (top & 0xFFFFu) ? top >> 16 : top & 0xFFFFu);
            float up, down;
            q4_range(top, up, down);
#pragma unroll
            for (int c = 0; c < C; ++c) a[c] = q4_half(raw[c], up);
#pragma unroll
            for (int e = 0; e < NI; ++e) back[e] = __shfl(down, 4 * g + e);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float sum[NI];
#pragma unroll
            for (int e = 0; e < NI; ++e) sum[e] = 0.0f;
#pragma unroll
            for (int b = 0; b < BLK; ++b) {
                const auto fold = [&](int p, float d0, float d1, float d2, float d3) {
                    const int at = b * PER + p;
                    const float f = half_bits_to_float(sc[i % P][at / 2] >> 16 * (at & 1) & 0xFFFFu);
                    const float d[4] = {d0, d1, d2, d3};
#pragma unroll
                    for (int e = 0; e < NI; ++e) sum[e] = fmaf(d[e], f, sum[e]);
                };
                const u32x4 ww = w[i % P][b];
                if constexpr (I8) {
                    i32x4 d[PER];                          // of bytes 16 t
#pragma unroll
                    for (int p = 0; p < PER; ++p) d[p] = i32x4{0, 0, 0, 0};
                    if constexpr (PER == 4) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            d[c] = __builtin_amdgcn_mfma_i32_16x16x32_i8(
                                __builtin_bit_cast(long, a[4 * b + c]),
                                __builtin_bit_cast(long, u32x2{ww[c] << 4 & 0xF0F0F0F0u, ww[c] & 0xF0F0F0F0u}), d[c], 0,
                                0, 0);
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; c += 2) {
                            const u32x2 a0 = a[4 * b + c], a1 = a[4 * b + c + 1];
                            d[c * PER / 4] = mfma_i8(u32x4{a0[0], a0[1], a1[0], a1[1]},
                                                     u32x4{ww[c] << 4 & 0xF0F0F0F0u, ww[c] & 0xF0F0F0F0u,
                                                           ww[c + 1] << 4 & 0xF0F0F0F0u, ww[c + 1] & 0xF0F0F0F0u},
                                                     d[c * PER / 4]);
                        }
                    }
#pragma unroll
                    for (int p = 0; p < PER; ++p)
                        fold(p, (float)d[p][0], (float)d[p][1], (float)d[p][2], (float)d[p][3]);
                } else {
                    f32x4 d[PER];
#pragma unroll
                    for (int p = 0; p < PER; ++p) d[p] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int c = 0; c < 4; ++c) d[c * PER / 4] = q4_mfma(a[4 * b + c], q4_decode(ww[c]), d[c * PER / 4]);
#pragma unroll
                    for (int p = 0; p < PER; ++p) fold(p, d[p][0], d[p][1], d[p][2], d[p][3]);
                }
            }
            if (i + P < R) {
                __builtin_amdgcn_sched_barrier(0);
                load(i + P);
            }
            if (lane < kLanes) {
                float* const mine = red + (i * nw + wave) * (NI * kLanes) + lane;
                if (!I8)
#pragma unroll
                    for (int e = 0; e < NI; ++e) sum[e] *= back[e];
                if (u > wave)
#pragma unroll
                    for (int e = 0; e < NI; ++e) sum[e] += mine[e * kLanes];
#pragma unroll
                for (int e = 0; e < NI; ++e) mine[e * kLanes] = sum[e];
            }
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < R * NI * kLanes; j += blockDim.x) {
        const int l = j % kLanes, e = j / kLanes % NI, i = j / (kLanes * NI), m = 4 * (l >> 4) + e;
        const int64_t n = ((int64_t)blockIdx.x * R + i) * 16 + (l & 15);
        if (m >= M || n >= N) continue;
        float sum = 0;
        for (int v = 0; v < nw; ++v) sum += red[(i * nw + v) * (NI * kLanes) + e * kLanes + l];
        y[m * N + n] = I8 ? s_x[m] * (0.0625f * sum) : sum;      // s_x may be fp32's smallest number
    }
}

// ------------------------------------------------------------------ launch

hipError_t launch_q4_pack(const int8_t* t, const uint16_t* scale, int64_t N, int64_t K, int group, uint8_t* packed,
                          hipStream_t stream)
{
    const int64_t blocks = (npad16(N) * K / 8 + 255) / 256;
    q4_pack_kernel<<<(unsigned)(blocks < 65536 ? blocks : 65536), 256, 0, stream>>>(
        t, scale, N, K, group, (uint32_t*)packed, (uint16_t*)(packed + q4_code_bytes(N, K)));
    return hipGetLastError();
}

// How a product is cut: blocks of a unit, waves along K, row tiles of a workgroup.
struct Q4Config {
    int blk, R, nw;
    int64_t grid;
};

// One block a unit while that fills 16 waves or fewer, so that small matrices
// wait for the shortest chain (in a graph, weights in the last-level cache, 4096 x
// 1024, one row in bf16: 3.0 us, with two blocks 0.1 more; four rows 3.3 and 0.6 more;
// 40000 x 2048 in 16 waves of one block 11.4, in 8 of two 10.4).
// Row tiles: a workgroup with R of them pays for its x and its meeting once, and
// 16 waves a CU run at once; the fewest (rounds) x (R + 1) is taken.  24576 x
// 4096, one and sixteen rows in bf16: R = 6, one round, 11.4 and 13.4 us; 3, two
// rounds, 12.7 and 17.4; 4, half of the second round idle, 14.7 and 18.7.
// 12288 x 4096: R = 3 7.6 and 9.5, 2 9.0 and 15.1.
// `most`: what registers hold (groups of 32 have four scales a block; 24576 x
// 4096, seven rows in bf16: R = 6 21.0, 3 16.2; one row 12.1 and 13.8).
static Q4Config q4_config(int64_t N, int64_t K, int most)
{
    const int64_t nb = K / 128, nrt = (N + 15) / 16;
    Q4Config c{};
    c.blk = nb < 16 ? 1 : 2;
    const int64_t nu = (nb + c.blk - 1) / c.blk;
    c.nw = (int)(nu < 16 ? nu : 16);
    const int64_t slots = device_cus() * (int64_t)(16 / c.nw);
    int64_t best = INT64_MAX;
    for (int R : {1, 2, 3, 4, 6}) {
        if (R > most || (c.blk == 1 && (R == 3 || R == 6))) continue;
        const int64_t grid = (nrt + R - 1) / R, path = (grid + slots - 1) / slots * (R + 1);
        if (path < best) {
            best = path;
            c.R = R;
            c.grid = grid;
        }
    }
    return c;
}

template <bool I8, int MT, int PER>
static hipError_t q4_gemv(const uint8_t* packed, int64_t N, int64_t K, const void* x, const float* s_x, int M,
                          float* y, hipStream_t stream)
{
    constexpr int kMost = PER == 4 && MT > (I8 ? 4 : 1) ? 3 : 6;
    const Q4Config c = q4_config(N, K, kMost);
#define Q4_CASE(B, RR)                                                                                          \
    if (c.blk == B && c.R == RR) {                                                                              \
        const size_t lds = (size_t)c.nw * 16 * B * q4_staged<I8, MT, RR>() * (I8 ? 8 : 16) +                    \
                           (size_t)RR * c.nw * (MT < 4 ? MT : 4) * (MT <= 4 ? 16 : 4 * MT) * 4;                 \
        q4_gemv_kernel<I8, MT, PER, B, RR>                                                                      \
            <<<(unsigned)c.grid, 64 * c.nw, lds, stream>>>(packed, N, K, x, s_x, M, y);                         \
        return hipGetLastError();                                                                               \
    }
    Q4_CASE(1, 1) Q4_CASE(1, 2) Q4_CASE(2, 1) Q4_CASE(2, 2) Q4_CASE(2, 3)
    if constexpr (kMost > 3) {
        Q4_CASE(1, 4) Q4_CASE(2, 4) Q4_CASE(2, 6)
    }
#undef Q4_CASE
    return hipErrorInvalidValue;
}

template <bool I8, int PER>
static hipError_t q4_gemv_rows(const uint8_t* packed, int64_t N, int64_t K, const void* x, const float* s_x, int64_t M,
                               float* y, hipStream_t stream)
{
    if (M == 1) return q4_gemv<I8, 1, PER>(packed, N, K, x, s_x, (int)M, y, stream);
    if (M <= 4) return q4_gemv<I8, 4, PER>(packed, N, K, x, s_x, (int)M, y, stream);
    if (M <= 8) return q4_gemv<I8, 8, PER>(packed, N, K, x, s_x, (int)M, y, stream);
    return q4_gemv<I8, 16, PER>(packed, N, K, x, s_x, (int)M, y, stream);
}

template <bool I8>
static hipError_t q4_gemv_group(const uint8_t* packed, int64_t N, int64_t K, int group, const void* x,
                                const float* s_x, int64_t M, float* y, hipStream_t stream)
{
    if (group == 128) return q4_gemv_rows<I8, 1>(packed, N, K, x, s_x, M, y, stream);
    if (group == 64) return q4_gemv_rows<I8, 2>(packed, N, K, x, s_x, M, y, stream);
    return q4_gemv_rows<I8, 4>(packed, N, K, x, s_x, M, y, stream);
}

hipError_t launch_q4_gemv_bf16(const uint8_t* packed, int64_t N, int64_t K, int group, const uint16_t* x, int64_t M,
                               float* y, hipStream_t stream)
{
    return q4_gemv_group<false>(packed, N, K, group, x, nullptr, M, y, stream);
}

hipError_t launch_q4_gemv_i8(const uint8_t* packed, int64_t N, int64_t K, int group, const int8_t* q,
                             const float* s_x, int64_t M, float* y, hipStream_t stream)
{
    return q4_gemv_group<true>(packed, N, K, group, q, s_x, M, y, stream);
}

}  // namespace tern
