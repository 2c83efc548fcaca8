// tern_attend.h — what the attention kernels share: the tile of columns that a
// workgroup works on, the int8 path's kernel over a stretch of its blocks, and
// the fp16 paths' operands.
#pragma once

#include "tern_device.h"
#include "tern_kv.h"
#include "tern_launch.h"

namespace tern {

typedef short s16x2 __attribute__((ext_vector_type(2)));

constexpr int kAttWaves = 4;
constexpr float kPlane = 32512.0f;          // 127 * 256: hi stays within int8
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// two planes of four values in [-1, 1] * kPlane / 32767: hi and lo bytes of
// x = 256 hi + lo, lo signed
__device__ __forceinline__ void planes(float a, float b, float c, float d, uint32_t& hi, uint32_t& lo)
{
    const uint32_t ab = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pknorm_i16(a, b));
    const uint32_t cd = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pknorm_i16(c, d));
    const s16x2 half = {128, 128};
    const uint32_t abh = __builtin_bit_cast(uint32_t, (s16x2)(__builtin_bit_cast(s16x2, ab) + half));
    const uint32_t cdh = __builtin_bit_cast(uint32_t, (s16x2)(__builtin_bit_cast(s16x2, cd) + half));
    hi = __builtin_amdgcn_perm(cdh, abh, 0x07050301u);
    lo = __builtin_amdgcn_perm(cd, ab, 0x06040200u);
}

// waves that take the blocks of a tile of COLS columns in turn
template <int COLS>
constexpr int att_turn() { return COLS <= 16 * kAttWaves ? 16 * kAttWaves / COLS : 1; }

// The tile of columns a workgroup or a joining row works on.
struct AttTile {
    KvSeq s;
    int col0, cols;            // first column, live columns
    int b0;                    // first block any of them sees
    int nblk;                  // blocks from there to the last one seen
};

__device__ __forceinline__ int att_first(int pos, int window)
{
    return window > 0 && pos >= window ? pos - window + 1 : 0;
}

__device__ __forceinline__ int att_limit(const KvBatch& b) { return (int)((int64_t)b.table_width * kKvBlock - 1); }

__device__ __forceinline__ int att_last(int pos, int limit) { return pos < limit ? pos : limit; }

// columns [COLS * number, + COLS) of a.s
template <int COLS>
__device__ __forceinline__ bool att_tile(const KvBatch& b, int number, int G, int window, AttTile& a)
{
    const int64_t total = (int64_t)a.s.n * G, col0 = (int64_t)number * COLS;
    if (col0 >= total || col0 > INT32_MAX - COLS) return false;
    a.col0 = (int)col0;
    a.cols = (int)(total - col0 < COLS ? total - col0 : COLS);
    const int lo = att_first(a.s.p0 + a.col0 / G, window);
    const int hi = att_last(a.s.p0 + (a.col0 + a.cols - 1) / G, att_limit(b));
    a.b0 = lo / kKvBlock;
    a.nblk = hi < lo ? 0 : hi / kKvBlock - a.b0 + 1;
    return true;
}

struct AttArgs {
    const uint16_t* q;
    uint16_t* out;
    float* part;               // [workgroups][2][COLS][D] unnormalised sums, then their (max, sum)
    float2* stat;
    uint32_t* start;           // [nseq] where each sequence starts in the line, then the total (trees: further on)
    int64_t q_stride;
    int window;
    float scale;
    int G;
    int groups;                // workgroups that share the line; 0: one workgroup for each unit
    int min_cols, max_cols;    // the sequences of this launch, by their columns
    int by_sequence;           // the joining kernel goes by sequences and columns, not by rows
    // TREE, behind what the causal kernels read: in front of it they were built with
    // their scalars in other places (a prompt of 4096 rows beside 1024 behind 15000
    // 432 us, 437.5 so)
    const uint64_t* mask;      // [T][words], the newest rows that a row sees
    int words;
};

// Values equal in all lanes of a wave, held in scalar registers.
__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ void att_uniform(AttTile& a)
{
    a.s.i = uni(a.s.i);
    a.s.t0 = uni(a.s.t0);
    a.s.n = uni(a.s.n);
    a.s.p0 = uni(a.s.p0);
    a.col0 = uni(a.col0);
    a.cols = uni(a.cols);
    a.b0 = uni(a.b0);
    a.nblk = uni(a.nblk);
}

// A row's tree: the words of its mask in LDS, behind them the position of the
// tree's first row.  The 64 bits of the tokens from `at` on that a row sees
// whose last token is `last`: all in front of the tree, of the tree those of
// the mask.
__device__ __forceinline__ uint64_t tree_bits(const uint64_t* row, int words, int p0, int at, int last)
{
    const int o = at - p0, w = o >> 6, sh = o & 63;
    const uint64_t lo = w >= 0 && w < words ? row[w] : 0, hi = w + 1 >= 0 && w + 1 < words ? row[w + 1] : 0;
    uint64_t bits = sh ? lo >> sh | hi << (64 - sh) : lo;
    if (o < 0) bits |= o > -64 ? (1ull << -o) - 1 : ~0ull;
    const int most = last - at;
    return most >= 63 ? bits : most < 0 ? 0 : bits & ((2ull << most) - 1);
}

// x where bit k is set, else -inf: two instructions
__device__ __forceinline__ float tree_sees(uint32_t bits, int k, float x)
{
    const uint32_t sees = (uint32_t)((int32_t)(bits << (31 - k)) >> 31);
    return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, x) & sees) | (0xFF800000u & ~sees));
}

// bits 0, N, 2 N, ...
template <int N>
constexpr uint64_t every()
{
    uint64_t m = 0;
    for (int i = 0; i < 64; i += N) m |= 1ull << i;
    return m;
}

// blocks [begin, end) of one unit; whole: the result is written, else it is
// part `slot` of the unit.  STREAM: codes are read past the caches.  TREE: of
// the newest rows a row sees those of its mask.
template <int D, int X, bool STREAM, bool TREE>
__device__ __forceinline__ void attend_blocks(const KvCache& c, const KvBatch& b, const AttArgs& a,
                                              const AttTile& tile, int h, int begin, int end, bool whole,
                                              uint32_t slot)
{
    constexpr int S = D / 64, U = D / 16, COLS = 16 * X, kTurn = att_turn<COLS>();
    constexpr int kPad = D + 4;
    __shared__ float sacc[kAttWaves][16][kPad];
    __shared__ float2 sstat[kAttWaves][16];
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;

    // this lane's columns: q as planes, the factor of its scores, the keys it sees
    const int limit = att_limit(b);
    const int group = wave % X;
    u32x4 qhi[S], qlo[S];
    float rowf;
    int first, last;
    // a wave's own columns' masks: no other wave waits for them
    __shared__ uint64_t smask[TREE ? kAttWaves : 1][16][TREE ? kTreeWords + 1 : 1];
    {
        const int col = 16 * group + n;
        const bool live = col < tile.cols;
        const int cc = tile.col0 + (live ? col : 0);
        const int j = cc / a.G;
        const uint16_t* row = a.q + (int64_t)(tile.s.t0 + j) * a.q_stride + (int64_t)(h * a.G + cc - j * a.G) * D;
        const int pos = tile.s.p0 + j;
        first = live ? att_first(pos, a.window) : 0;
        last = live ? att_last(pos, limit) : INT32_MAX;
        if constexpr (TREE) {
            const uint64_t* words = a.mask + (int64_t)(tile.s.t0 + j) * a.words;
            for (int w = g; w < a.words; w += 4) smask[wave][n][w] = words[w];
            __builtin_amdgcn_wave_barrier();         // read by the column's other lanes
        }
        u32x4 raw[S][2];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            raw[s][0] = *(const u32x4*)(row + 64 * s + 16 * g);
            raw[s][1] = *(const u32x4*)(row + 64 * s + 16 * g + 8);
        }
        uint32_t top = 0;              // bits of max |q|, an infinity above every number, a NaN above that
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t w = raw[s][e >> 2][e & 3];
                const uint32_t x0 = (w << 16) & 0x7FFF0000u, x1 = w & 0x7FFF0000u;
                top = x0 > top ? x0 : top;
                top = x1 > top ? x1 : top;
            }
        for (int off = 16; off < 64; off <<= 1) {
            const uint32_t o = (uint32_t)__shfl_xor((int)top, off);
            top = o > top ? o : top;
        }
        const float amax = __builtin_bit_cast(float, top);
        // rows of nothing but zeros (or less than 2^-100) score 0; a row that
        // is not finite scores 0 * amax = NaN
        const float inv = live && amax >= 0x1p-100f && top < 0x7F800000u ? kPlane / 32767.0f / amax : 0.0f;
        rowf = amax * (a.scale * kLog2e / kPlane);
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t w0 = raw[s][e >> 1][2 * (e & 1)], w1 = raw[s][e >> 1][2 * (e & 1) + 1];
                uint32_t hi, lo;
                planes(__builtin_bit_cast(float, w0 << 16) * inv, __builtin_bit_cast(float, w0 & 0xFFFF0000u) * inv,
                       __builtin_bit_cast(float, w1 << 16) * inv, __builtin_bit_cast(float, w1 & 0xFFFF0000u) * inv,
                       hi, lo);
                qhi[s][e] = inv == 0.0f ? 0u : hi;
                qlo[s][e] = inv == 0.0f ? 0u : lo;
            }
    }

    float m = -INFINITY, l = 0.0f;
    f32x4 acc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) acc[u] = f32x4{0, 0, 0, 0};

    for (int seg = begin; seg < end; seg += 64) {
        // lane i looks up block seg + i: its place and scales
        const int count = end - seg < 64 ? end - seg : 64;
        int mine = -1;
        float2 sc = make_float2(0.0f, 0.0f);
        if (lane < count) {
            mine = kv_block(b, c, tile.s.i, tile.b0 + seg + lane);
            if (mine >= 0) sc = *(const float2*)(c.scales + ((int64_t)mine * c.heads + h) * 2);
        }
        // this wave's blocks among those that are there (none for a group without columns)
        uint64_t todo = 16 * group < tile.cols ? __ballot(mine >= 0) & (every<kTurn>() << (wave / X)) : 0;
        const auto codes = [&](int i) {
            const int64_t phys = __builtin_amdgcn_readlane(mine, i);
            return c.codes + (phys * c.heads + h) * 2 * (kKvBlock * D);
        };
        // the lane's 16 bytes of a KiB behind a scalar address
        const uint32_t own = lane * 16;
        const auto load = [&](const int8_t* p, int byte) {
            return STREAM ? ld_nt16(p + byte + own) : *(const u32x4*)(p + byte + own);
        };
        u32x4 kr[4][S], vr[U];
        if (todo) {
            const int8_t* p = codes(__builtin_ctzll(todo));
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int s = 0; s < S; ++s) kr[t][s] = load(p, 1024 * (t * S + s));
            __builtin_amdgcn_sched_barrier(0);           // keys first: they are waited for first
#pragma unroll
            for (int u = 0; u < U; ++u) vr[u] = load(p, 1024 * (U + u));
        }
        while (todo) {
            const int i = __builtin_ctzll(todo);
            todo &= todo - 1;
            const float sk = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sc.x), i));
            const float sv = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sc.y), i));
            // The next block's keys are asked for before this one's softmax, its
            // values behind this one's; never behind a branch, or the waits
            // would be for all of them.  Without a next block one KiB of this
            // one is read 16 times.
            const int8_t* next = codes(todo ? __builtin_ctzll(todo) : i);
            const int kib = todo ? 1024 : 0;
            const int at = (tile.b0 + seg + i) * kKvBlock;
            float x[16];
            const float f = rowf * sk;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                i32x4 hi = {0, 0, 0, 0}, lo = {0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    hi = mfma_i8(kr[t][s], qhi[s], hi);
                    lo = mfma_i8(kr[t][s], qlo[s], lo);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * t + e] = (float)(hi[e] * 256 + lo[e]) * f;
                asm volatile("" : "+v"(x[4 * t]), "+v"(x[4 * t + 1]), "+v"(x[4 * t + 2]), "+v"(x[4 * t + 3]));
            }
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int s = 0; s < S; ++s) kr[t][s] = load(next, kib * (t * S + s));
            bool sees;
            if constexpr (TREE) {
                sees = true;
                if (at + 63 >= tile.s.p0) {
                    const uint64_t bits = tree_bits(smask[wave][n], a.words, tile.s.p0, at, last);
                    sees = bits != 0;
                    const uint64_t mine = bits >> 4 * g;
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        x[e] = tree_sees(e < 8 ? (uint32_t)mine : (uint32_t)(mine >> 32), 16 * (e >> 2 & 1) + (e & 3), x[e]);
                }
            } else {
                sees = first <= at + 63 && last >= at;
            }
            if (!TREE && __any(first > at || last < at + 63)) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int p = at + 16 * (e >> 2) + 4 * g + (e & 3);
                    x[e] = p >= first && p <= last ? x[e] : -INFINITY;
                }
            }
            float top = x[0];
#pragma unroll
            for (int e = 1; e < 16; ++e) top = fmaxf(top, x[e]);
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            // weights relative to the block's largest, in units of kPlane / 32767
            const float base = (top == -INFINITY ? 0.0f : top) + 0x1.715664p-7f;   // log2(32767 / 32512)
            float sum = 0.0f;
            u32x4 phi, plo;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = exp2_fast(x[4 * t + e] - base);
                    sum += w[e];
                }
                uint32_t hi, lo;
                planes(w[0], w[1], w[2], w[3], hi, lo);
                phi[t] = hi;
                plo[t] = lo;
            }
            const float mn = fmaxf(m, top);
            const float keep = m == mn ? 1.0f : exp2_fast(m - mn);
            const float join = top == -INFINITY ? 0.0f : exp2_fast(top - mn);
            const float fv = sees ? join * sv * (1.0f / 32767.0f) : 0.0f;
            m = mn;
            l = l * keep + sum * join;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const i32x4 zero = {0, 0, 0, 0};
                const i32x4 hi = mfma_i8(vr[u], phi, zero), lo = mfma_i8(vr[u], plo, zero);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[u][e] = fmaf((float)(hi[e] * 256 + lo[e]), fv, acc[u][e] * keep);
                // in this order: or all sums wait in registers behind the loads below
                asm volatile("" : "+v"(acc[u]));
            }
#pragma unroll
            for (int u = 0; u < U; ++u) vr[u] = load(next, kib * (U + u));
        }
    }

    // a group's waves meet: common maximum, scaled sums
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g == 0) sstat[wave][n] = make_float2(m, l);
    __syncthreads();
    {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kTurn; ++w) top = fmaxf(top, sstat[group + X * w][n].x);
        const float f = m == top ? 1.0f : exp2_fast(m - top);
#pragma unroll
        for (int u = 0; u < U; ++u) *(f32x4*)&sacc[wave][n][16 * u + 4 * g] = acc[u] * f;
    }
    __syncthreads();
    constexpr int kPer = D / 4;                     // threads per column, four dims each
    for (int i = threadIdx.x; i < tile.cols * kPer; i += 64 * kAttWaves) {
        const int col = i / kPer, d = i % kPer * 4;
        float top = -INFINITY, sum = 0.0f;
        f32x4 o = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kTurn; ++w) top = fmaxf(top, sstat[(col >> 4) + X * w][col & 15].x);
#pragma unroll
        for (int w = 0; w < kTurn; ++w) {
            const float2 st = sstat[(col >> 4) + X * w][col & 15];
            sum += st.y * (st.x == top ? 1.0f : exp2_fast(st.x - top));
            o += *(const f32x4*)&sacc[(col >> 4) + X * w][col & 15][d];
        }
        if (!whole) {
            const uint32_t at = slot * COLS + col;
            *(f32x4*)(a.part + (int64_t)at * D + d) = o;
            if (d == 0) a.stat[at] = make_float2(top, sum);
        } else {
            const int cc = tile.col0 + col;
            uint16_t* dst = a.out + ((int64_t)(tile.s.t0 + cc / a.G) * c.heads * a.G + h * a.G + cc % a.G) * D + d;
            const float r = sum == 0.0f ? 0.0f : 1.0f / sum;
            typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
            u16x4 y;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = f32_to_bf16(sum == 0.0f ? 0.0f : o[e] * r);
            *(u16x4*)dst = y;
        }
    }
}

// ---- fp16 operands ----
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kF16Up = 9.0f, kF16Most = 32768.0f, kF16Top = 15.0f;
// A smaller scale of values than 2^-80, 0 among them, stands for that, so that
// its logarithm and what takes it out of the sum of weights stay in range;
// results below what the largest code makes of it are 0.
constexpr float kF16Least = 0x1p-80f, kF16None = 0x1p-73f;
constexpr int kAhead = 4;                    // LDS operands under way to the matrix cores

__device__ __forceinline__ f32x16 mfma_f16(u32x4 a, u32x4 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}

// four codes to fp16: 1024 + (code + 128) as bits, minus 1152
__device__ __forceinline__ u32x2 codes_f16(uint32_t x)
{
    const uint32_t u = x ^ 0x80808080u;
    const f16x2 off = {(_Float16)1152.0f, (_Float16)1152.0f};
    u32x2 r;
    r[0] = __builtin_bit_cast(
        uint32_t, (f16x2)(__builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) - off));
    r[1] = __builtin_bit_cast(
        uint32_t, (f16x2)(__builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) - off));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b)
{
    const f16x2 h = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, h);
}

// a result of the fp16 path (NaN kept)
template <bool F16>
__device__ __forceinline__ float none_below(float y)
{
    return F16 && fabsf(y) < kF16None ? 0.0f : y;
}

}  // namespace tern
