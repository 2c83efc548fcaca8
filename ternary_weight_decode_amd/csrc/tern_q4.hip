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
// t + 8 = (t & 15) ^ 8; the nibbles at bit 4 stand for 16 (t + 8) there.
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

// One workgroup per row tile, its waves take the blocks in turn, x straight
// from memory; a block's 128 activations of a row share the power of two that
// takes them into fp16.
template <bool I8, int PER>
__global__ __launch_bounds__(512) void q4_gemv_kernel(const uint8_t* __restrict__ packed, int64_t N, int64_t K,
                                                      const void* __restrict__ x, const float* __restrict__ s_x, int M,
                                                      float* __restrict__ y)
{
    __shared__ float red[8][4][64];
    const int nw = blockDim.x >> 6, wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int64_t rt = blockIdx.x;
    const int nb = (int)(K / 128);
    const uint32_t* words = (const uint32_t*)packed + rt * nb * 256;
    const uint16_t* scales = (const uint16_t*)(packed + q4_code_bytes(N, K));
    const int m = r < M ? r : M - 1;
    f32x4 acc = {0, 0, 0, 0};
    for (int b = wave; b < nb; b += nw) {
        const u32x4 w = *(const u32x4*)(words + b * 256 + lane * 4);
        const int kt = b >> 2, bq = b & 3, nbq = nb - 4 * kt < 4 ? nb - 4 * kt : 4;
        const uint16_t* sc = scales + ((rt * nb + 4 * kt) * 16 + r * nbq + bq) * PER;
        f32x4 part[PER];
        float back[4] = {1, 1, 1, 1};
        if constexpr (I8) {
            const int8_t* q = (const int8_t*)x + m * K + b * 128 + 8 * g;
            i32x4 d[PER];
#pragma unroll
            for (int p = 0; p < PER; ++p) d[p] = i32x4{0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const u32x2 a = *(const u32x2*)(q + 32 * c);
                // bytes 16 t of weights 0, 4, 1, 5 and 2, 6, 3, 7
                const uint64_t bb = (uint64_t)(w[c] & 0xF0F0F0F0u) << 32 | (w[c] << 4 & 0xF0F0F0F0u);
                const uint64_t aa = (uint64_t)__builtin_amdgcn_perm(a[1], a[0], 0x07030602u) << 32 |
                                    __builtin_amdgcn_perm(a[1], a[0], 0x05010400u);
                d[c * PER / 4] = __builtin_amdgcn_mfma_i32_16x16x32_i8((long)aa, (long)bb, d[c * PER / 4], 0, 0, 0);
            }
#pragma unroll
            for (int p = 0; p < PER; ++p)
#pragma unroll
                for (int e = 0; e < 4; ++e) part[p][e] = (float)d[p][e] * 0.0625f;
        } else {
            const uint16_t* xr = (const uint16_t*)x + m * K + b * 128 + 8 * g;
            u32x4 a[4];
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                a[c] = *(const u32x4*)(xr + 32 * c);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t lo = a[c][e] << 16 & 0x7FFF0000u, hi = a[c][e] & 0x7FFF0000u;
                    top = lo > top ? lo : top;
                    top = hi > top ? hi : top;
                }
            }
            for (int off = 16; off < 64; off <<= 1) {
                const uint32_t o = (uint32_t)__shfl_xor((int)top, off);
                top = o > top ? o : top;
            }
            // 2^14 <= largest < 2^15 (a row of values below 2^-112 stays below); an
            // infinity or a NaN stays one
            int ex = (int)(top >> 23) - 127;
            ex = ex > 127 ? 14 : ex < -112 ? -112 : ex;
            const float up = ldexpf(1.0f, 14 - ex), down = ldexpf(1.0f, ex - 14);
#pragma unroll
            for (int e = 0; e < 4; ++e) back[e] = __shfl(down, 4 * g + e);
            f32x4 d[PER];
#pragma unroll
            for (int p = 0; p < PER; ++p) d[p] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                u32x4 h;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const q4_f16x2 v = {(_Float16)(__builtin_bit_cast(float, a[c][e] << 16) * up),
                                        (_Float16)(__builtin_bit_cast(float, a[c][e] & 0xFFFF0000u) * up)};
                    h[e] = __builtin_bit_cast(uint32_t, v);
                }
                d[c * PER / 4] = q4_mfma(h, q4_decode(w[c]), d[c * PER / 4]);
            }
#pragma unroll
            for (int p = 0; p < PER; ++p) part[p] = d[p];
        }
        f32x4 sum = {0, 0, 0, 0};
#pragma unroll
        for (int p = 0; p < PER; ++p) sum += part[p] * half_bits_to_float(sc[p]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = fmaf(sum[e], back[e], acc[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave][e][lane] = acc[e];
    __syncthreads();
    for (int i = threadIdx.x; i < 256; i += blockDim.x) {
        const int l = i & 63, e = i >> 6, mm = 4 * (l >> 4) + e;
        const int64_t n = rt * 16 + (l & 15);
        if (mm >= M || n >= N) continue;
        float sum = 0;
        for (int v = 0; v < nw; ++v) sum += red[v][e][l];
        y[mm * N + n] = I8 ? s_x[mm] * sum : sum;
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

template <bool I8>
static hipError_t q4_gemv(const uint8_t* packed, int64_t N, int64_t K, int group, const void* x, const float* s_x,
                          int64_t M, float* y, hipStream_t stream)
{
    const int64_t nb = K / 128;
    const unsigned grid = (unsigned)((N + 15) / 16), threads = 64 * (unsigned)(nb < 8 ? nb : 8);
    if (group == 128) q4_gemv_kernel<I8, 1><<<grid, threads, 0, stream>>>(packed, N, K, x, s_x, (int)M, y);
    else if (group == 64) q4_gemv_kernel<I8, 2><<<grid, threads, 0, stream>>>(packed, N, K, x, s_x, (int)M, y);
    else q4_gemv_kernel<I8, 4><<<grid, threads, 0, stream>>>(packed, N, K, x, s_x, (int)M, y);
    return hipGetLastError();
}

hipError_t launch_q4_gemv_bf16(const uint8_t* packed, int64_t N, int64_t K, int group, const uint16_t* x, int64_t M,
                               float* y, hipStream_t stream)
{
    return q4_gemv<false>(packed, N, K, group, x, nullptr, M, y, stream);
}

hipError_t launch_q4_gemv_i8(const uint8_t* packed, int64_t N, int64_t K, int group, const int8_t* q,
                             const float* s_x, int64_t M, float* y, hipStream_t stream)
{
    return q4_gemv<true>(packed, N, K, group, q, s_x, M, y, stream);
}

}  // namespace tern
