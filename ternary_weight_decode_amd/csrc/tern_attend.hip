// tern_attend.hip — attention over the paged int8 cache.
//
//   out = sum_p w_p V[p] / sum_p w_p,  w_p = exp(scale * q . K[p])
//
// The rows of one key/value head are columns here: column c of a sequence is
// row c / G under query head h*G + c % G, so a group's G query heads share one
// pass over the cached bytes.
//
// The int8 path: 16 columns per wave, for single tokens and drafts, bound by
// the cache's bytes.  The four waves of a workgroup are X groups of 16 columns
// that read the same blocks (from memory once, then from the caches), and
// 4 / X of each that take blocks in turn.  The codes go from memory to the int8
// matrix cores as they are:
//   S^T = K Q^T    A = K (16 tokens x 64 dims, one 16-byte load per lane),
//                  B = q as two int8 planes, x = 256 hi + lo of
//                  rint(q / max|q| * 32512): 2^-16 of the row's largest value;
//                  exact int32 sums, one fp32 factor for row and block.
//   softmax        lane (column c, g) holds tokens 16t + 4g + i of a block.
//   O^T = V^T P^T  A = V^T (16 dims x 64 tokens), whose bytes the cache holds
//                  in the order in which the lane has its weights, so a
//                  weight never leaves its lane; B = the weights as two int8
//                  planes relative to the largest of their own block (2^-16
//                  of it: a flat tail behind one large weight elsewhere keeps
//                  its digits); int32 sums, scaled into the fp32 accumulator
//                  once a block.
// Every wave walks its own blocks with a running maximum and sum; the waves
// of a group meet in LDS at the end.
//
// Long sequences are split.  Only the device knows the lengths (a captured
// graph follows them), so it also makes the split: the blocks of all units
// (tile of columns, head) stand in one line, each unit padded to whole turns
// of a group's waves, and every workgroup takes an equal stretch of it.
// A unit that lies in one stretch is written at once, the parts of the others
// are joined by a second kernel.
//
// What bounds it, 32:8 heads of 128, the two kernels of a call: long contexts
// the cache's bytes (64 streams up to 16000, 482 MB: 87 to 91 + 5 us, 5.4 TB/s;
// one of 40960, 84 MB, out of the last-level cache: 18.5 + 5 us); a short one
// the chain from cu over the table to the scales, the codes and the waves'
// meeting (513 tokens 8 us whole, of which 2 are an empty launch; 0.28 us more
// per block of the longest unit); drafts the same chain until their tiles fill
// the card, then 0.8 to 1.2 ns per (16 columns, block).
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
    uint32_t* start;           // [nseq] where each sequence starts in the line, then the total
    int64_t q_stride;
    int window;
    float scale;
    int G;
    int groups;                // workgroups that share the line; 0: one workgroup for each unit
    int min_cols, max_cols;    // the sequences of this launch, by their columns
    int by_sequence;           // the joining kernel goes by sequences and columns, not by rows
};

// A sequence's share of the line: its tiles, and the blocks that each of its
// units takes there (padded; no tile of the sequence sees more).  None for a
// sequence without rows or of another launch; s.n < 0 where cu descends.
struct AttShare {
    uint32_t tiles, len;
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

template <int COLS>
__device__ __forceinline__ AttShare att_share(const KvBatch& b, int i, const AttArgs& a, KvSeq& s)
{
    s.i = i;
    s.t0 = b.cu[i];
    const int t1 = b.cu[i + 1];
    s.n = t1 < s.t0 ? -1 : t1 - s.t0;
    s.p0 = kv_length(b, i) - s.n;
    constexpr uint32_t kTurn = att_turn<COLS>();
    AttShare r = {0, kTurn};
    if (s.t0 < 0 || t1 > b.T || s.n <= 0) return r;
    const int64_t cols = (int64_t)s.n * a.G;
    if (cols < a.min_cols || cols > a.max_cols) return r;
    r.tiles = (uint32_t)((cols + COLS - 1) / COLS);
    const int last = att_last(s.p0 + s.n - 1, att_limit(b));
    uint32_t blocks = last < 0 ? 1 : last / kKvBlock + 1;
    if (a.window > 0) {        // a tile spans window + its rows - 1 keys
        const uint32_t most = ((uint32_t)a.window + COLS / a.G + 1) / kKvBlock + 2;
        blocks = blocks < most ? blocks : most;
    }
    r.len = (blocks + kTurn - 1) / kTurn * kTurn;
    return r;
}

// blocks of the line for each of `groups` workgroups
template <int COLS>
__device__ __forceinline__ uint32_t att_stretch(uint32_t total, int groups)
{
    constexpr uint32_t kTurn = att_turn<COLS>();
    const uint32_t turn = (uint32_t)groups * kTurn;
    return (total + turn - 1) / turn * kTurn;
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
// part `slot` of the unit.  STREAM: codes are read past the caches.
template <int D, int X, bool STREAM>
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
    {
        const int col = 16 * group + n;
        const bool live = col < tile.cols;
        const int cc = tile.col0 + (live ? col : 0);
        const int j = cc / a.G;
        const uint16_t* row = a.q + (int64_t)(tile.s.t0 + j) * a.q_stride + (int64_t)(h * a.G + cc - j * a.G) * D;
        const int pos = tile.s.p0 + j;
        first = live ? att_first(pos, a.window) : 0;
        last = live ? att_last(pos, limit) : INT32_MAX;
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
            const bool sees = first <= at + 63 && last >= at;
            if (__any(first > at || last < at + 63)) {
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

// The fp16 tile: 256 columns per workgroup, 32 for each of eight waves, for
// prompts.  A block's codes are turned into fp16 once for all waves, on their
// way into LDS (exact: |code| <= 127); the sums stay in the fp32 accumulators
// of the fp16 matrix cores, so the vector units are left with about eight
// operations per score instead of sixteen.
//   S^T = K Q^T   32 tokens x 32 columns x 16 dims; q divided by the power of
//                 two below its row's largest value, exact to 2^-25 of that.
//   weights       2^(9 + x + log2 s_V - m) in fp16: the values' scale rides in
//                 the exponent and leaves the sum of weights again with one
//                 product a block.  m, the row's own largest x + log2 s_V so
//                 far (what a row does not see has no say in it), moves only
//                 when a lane's weights sum to more than 2^15.  fp16 holds
//                 2^-11 of a weight, and 2^-34 of the row's largest product of
//                 weight and scale where that is more.
//   O^T = V^T P^T the lane's weights are the B operand as they stand; V lies
//                 in LDS in their order.
// The matrix cores and the vector units are kept busy at once by the two waves
// of each SIMD taking turns: while waves 0-3 run one block's products
// (P V of the block before, then K Q), waves 4-7 run their softmax, then the
// other way round; a barrier ends every half turn.  Waves 0-3 fill LDS with V,
// waves 4-7 with K, in their vector half.  In half turns, block j's K is
// written in 2j - 2 and read in 2j and 2j + 1, its V written in 2j + 1 and read
// in 2j + 2 and 2j + 3: two buffers of each are enough.
// Bound by the matrix cores' half turns and, with all CUs busy, by the rate the
// card sustains: a block of 256 columns takes 1.67 us where half of the CUs
// work and 2.1 where all do.  16384 tokens from nothing run at 1010 to 1115 TFLOP/s (a
// library's product of 8192^3 in fp16 at 1165 here), 4096 behind 15000 at 1056,
// 4096 from nothing beside 1024 behind 15000 in 415 to 444 us by the card, 960 to 897.
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kF16Up = 9.0f, kF16Most = 32768.0f;
// A smaller scale of values than 2^-80, 0 among them, stands for that, so that
// its logarithm and what takes it out of the sum of weights stay in range;
// results below what the largest code makes of it are 0.
constexpr float kF16Least = 0x1p-80f, kF16None = 0x1p-73f;
constexpr int kTileWaves = 8;
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
template <int COLS>
__device__ __forceinline__ float none_below(float y)
{
    return COLS == 256 && fabsf(y) < kF16None ? 0.0f : y;
}

__device__ __forceinline__ void half_turn()
{
    __builtin_amdgcn_sched_barrier(0);
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
}

template <int D>
__device__ __forceinline__ void attend_tile_f16(const KvCache& c, const KvBatch& b, const AttArgs& a,
                                                const AttTile& tile, int h, int begin, int end, bool whole,
                                                uint32_t slot)
{
    constexpr int S = D / 64, ST = D / 16, DT = D / 32, COLS = 32 * kTileWaves;
    __shared__ u32x4 kbuf[2][kKvBlock * D / 8], vbuf[2][kKvBlock * D / 8];
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const int half = lane >> 5;
    const bool second = wave >= kTileWaves / 2;      // waves i and i + 4 share a SIMD
    const int tid = threadIdx.x & 255;

    // this lane's column
    const int col = 32 * wave + (lane & 31);
    const bool works = 32 * wave < tile.cols;         // a wave without columns only fills LDS
    const bool live = col < tile.cols;
    const int cc = tile.col0 + (live ? col : 0), j = cc / a.G;
    const uint16_t* row = a.q + (int64_t)(tile.s.t0 + j) * a.q_stride + (int64_t)(h * a.G + cc - j * a.G) * D;
    const int pos = tile.s.p0 + j;
    const int first = live ? att_first(pos, a.window) : 0;
    const int last = live ? att_last(pos, att_limit(b)) : INT32_MAX;
    int all_first = first, all_last = last;           // keys that every column sees
    for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_xor(all_first, off), y = __shfl_xor(all_last, off);
        all_first = x > all_first ? x : all_first;
        all_last = y < all_last ? y : all_last;
    }
    all_first = uni(all_first);
    all_last = uni(all_last);
    // step 4 s + e, half: dims 64 s + 16 half + 4 e .. + 3 and 32 further on
    u32x4 q[ST];
    uint32_t qtop = 0;
#pragma unroll
    for (int s = 0; s < ST; ++s) {
        const uint16_t* p = row + 64 * (s >> 2) + 16 * half + 4 * (s & 3);
        const u32x2 x = *(const u32x2*)p, y = *(const u32x2*)(p + 32);
        q[s] = u32x4{x[0], x[1], y[0], y[1]};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t x0 = (q[s][e] << 16) & 0x7FFF0000u, x1 = q[s][e] & 0x7FFF0000u;
            qtop = x0 > qtop ? x0 : qtop;
            qtop = x1 > qtop ? x1 : qtop;
        }
    }
    const uint32_t other = (uint32_t)__shfl_xor((int)qtop, 32);
    qtop = other > qtop ? other : qtop;
    const bool scored = live && qtop >= 0x0D800000u && qtop < 0x7F800000u;    // 2^-100 <= max |q| < inf
    // the power of two below max |q| and its inverse; the sign of the scale goes into q
    const float size = __builtin_bit_cast(float, qtop >= 0x7F800000u ? qtop : qtop & 0x7F800000u);
    const float inv =
        scored ? copysignf(fmaxf(__builtin_bit_cast(float, 0x7F000000u - (qtop & 0x7F800000u)), 0x1p-127f), a.scale)
               : 0.0f;
    const float rowf = size * (fabsf(a.scale) * kLog2e);
#pragma unroll
    for (int s = 0; s < ST; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t w = q[s][e];
            const uint32_t p = pack_f16(__builtin_bit_cast(float, w << 16) * inv,
                                        __builtin_bit_cast(float, w & 0xFFFF0000u) * inv);
            q[s][e] = scored ? p : 0u;
        }

    // This thread's two chunks of 16 bytes of a block's K (waves 4-7) or V
    // (waves 0-3), groups g and g + 2 of one token and 64 dims, or of one dim:
    // their e-th words, side by side, are what lane half g reads in step e.
    const bool fills = tid < 2 * D;
    const int item = fills ? tid : 0, fr = item & 15, fg = (item >> 4) & 1, fu = item >> 5;
    const int from = (second ? 0 : kKvBlock * D) + ((fu * 4 + fg) * 16 + fr) * 16;
    // K: fu = 16-token tile and 64 dims, V: fu = 16 dims
    const int step = second ? ((fu / S >> 1) * ST + fu % S * 4) * 64 + (fu / S & 1) * 16 : (fu >> 1) * 256 + (fu & 1) * 16;
    u32x4* const to = (second ? kbuf[0] : vbuf[0]) + step + fg * 32 + fr;

    float m = -INFINITY, l = 0.0f;
    f32x16 acc[DT];
#pragma unroll
    for (int u = 0; u < DT; ++u)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[u][e] = 0.0f;

    for (int seg = begin; seg < end; seg += 64) {
        // lane i looks up block seg + i; the blocks that are there move to the front
        const int count = end - seg < 64 ? end - seg : 64;
        int mine = -1;
        float2 sc = make_float2(0.0f, 0.0f);
        if (lane < count) {
            mine = kv_block(b, c, tile.s.i, tile.b0 + seg + lane);
            if (mine >= 0) sc = *(const float2*)(c.scales + ((int64_t)mine * c.heads + h) * 2);
        }
        const uint64_t there = __ballot(mine >= 0), below = (1ull << lane) - 1;
        const int blocks = __popcll(there);
        if (blocks == 0) continue;
        const int dest = (mine >= 0 ? __popcll(there & below) : blocks + __popcll(~there & below)) * 4;
        mine = __builtin_amdgcn_ds_permute(dest, mine);
        const int number = __builtin_amdgcn_ds_permute(dest, tile.b0 + seg + lane);
        const float sk = __builtin_bit_cast(float, __builtin_amdgcn_ds_permute(dest, __builtin_bit_cast(int, sc.x)));
        const float sv = __builtin_bit_cast(float, __builtin_amdgcn_ds_permute(dest, __builtin_bit_cast(int, sc.y)));
        // the values' scales as exponents, and what takes them out of the sum of weights
        const float lv = sv < INFINITY ? __log2f(fmaxf(sv, kF16Least)) : NAN, back = exp2_fast(-lv);
        const auto pick = [](float v, int i) {
            return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), i));
        };

        u32x4 raw[2];
        const auto fetch = [&](int i) {
            const int64_t phys = __builtin_amdgcn_readlane(mine, i < blocks ? i : blocks - 1);
            const int8_t* p = c.codes + (phys * c.heads + h) * 2 * (kKvBlock * D);
            raw[0] = *(const u32x4*)(p + from);
            raw[1] = *(const u32x4*)(p + from + 512);
        };
        const auto fill = [&](int buf) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const u32x2 x0 = codes_f16(raw[0][e]), x1 = codes_f16(raw[1][e]);
                if (D == 128 || fills) to[buf * (kKvBlock * D / 8) + 64 * e] = u32x4{x0[0], x0[1], x1[0], x1[1]};
            }
        };
        f32x16 x[2];
        u32x4 w[4];                  // the weights: B operands of 16 tokens each
        u32x4 ahead[kAhead];
        // Four operands ahead of the matrix cores (alone, the compiler reads one
        // at a time and waits for it), neighbouring products independent.
        const auto scores = [&](int buf) {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[0][e] = x[1][e] = 0.0f;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) ahead[k] = kbuf[buf][((k & 1) * ST + (k >> 1)) * 64 + lane];
#pragma unroll
            for (int k = 0; k < 2 * ST; ++k) {
                x[k & 1] = mfma_f16(ahead[k % kAhead], q[k >> 1], x[k & 1]);
                const int o = k + kAhead;
                if (o < 2 * ST) ahead[k % kAhead] = kbuf[buf][((o & 1) * ST + (o >> 1)) * 64 + lane];
            }
            __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
            for (int k = 0; k < 2 * ST - kAhead; ++k) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
        };
        const auto values = [&](int buf) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) ahead[k] = vbuf[buf][((k % DT) * 4 + k / DT) * 64 + lane];
#pragma unroll
            for (int k = 0; k < 4 * DT; ++k) {
                acc[k % DT] = mfma_f16(ahead[k % kAhead], w[k / DT], acc[k % DT]);
                const int o = k + kAhead;
                if (o < 4 * DT) ahead[k % kAhead] = vbuf[buf][((o % DT) * 4 + o / DT) * 64 + lane];
            }
            __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 1);
#pragma unroll
            for (int k = 0; k < 4 * DT - kAhead; ++k) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 1);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 1);
            }
            __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 1);
        };
        const auto softmax = [&](int i) {
            // read with every lane active: a lane's value must not be computed behind a mask
            const float f = rowf * pick(sk, i), lvi = pick(lv, i), backi = pick(back, i);
            const int at = __builtin_amdgcn_readlane(number, i) * kKvBlock;
            // exponents against the maximum so far; token of x[t][e]:
            // at + 32 t + 8 (e / 4) + 4 half + e % 4
            const float m0 = m == -INFINITY ? 0.0f : m, base = kF16Up + lvi - m0;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e) x[t][e] = fmaf(x[t][e], f, base);
            if (all_first > at || all_last < at + 63) {
                const int lo = first - at - 4 * half, hi = last - at - 4 * half;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int p = 32 * t + 8 * (e >> 2) + (e & 3);
                        x[t][e] = p >= lo && p <= hi ? x[t][e] : -INFINITY;
                    }
            }
            float sum;
            const auto weigh = [&](float by) {
                float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float w0 = exp2_fast(x[t][e] - by), w1 = exp2_fast(x[t][e + 1] - by);
                        sum0 += w0;
                        sum1 += w1;
                        w[2 * t + (e >> 3)][(e >> 1) & 3] = pack_f16(w0, w1);
                    }
                sum = sum0 + sum1;
            };
            // The maximum is looked at only when the weights say so: while a
            // lane's sum stays below 2^15 no weight has left fp16's range.
            weigh(0.0f);
            if (__any(sum > kF16Most || m == -INFINITY)) {
                float top = fmaxf(x[0][0], x[1][0]);
#pragma unroll
                for (int e = 1; e < 16; ++e) top = fmaxf(top, fmaxf(x[0][e], x[1][e]));
                top = fmaxf(top, __shfl_xor(top, 32));
                const float over = top - kF16Up;
                const bool grow = m == -INFINITY ? over > -INFINITY : over > 0.0f;
                const float by = grow ? over : 0.0f;
                const float keep = m == -INFINITY ? 0.0f : exp2_fast(-by);
                m = grow ? m0 + by : m;
                l *= keep;
#pragma unroll
                for (int u = 0; u < DT; ++u)
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[u][e] *= keep;
                weigh(by);
            }
            // a row that sees nothing here is spared a scale that is not finite
            l += sum == 0.0f ? 0.0f : sum * backi;
        };

        if (second) {
            fetch(0);
            fill(0);
            fetch(1);
        } else {
            fetch(0);
        }
        half_turn();
        if (second) {
            fill(1);
            fetch(2);
            half_turn();
        }
        for (int i = 0; i < blocks; ++i) {
            if (works) {
                if (i > 0) values((i - 1) & 1);
                scores(i & 1);
            }
            half_turn();
            if (works) softmax(i);
            fill(i & 1);             // V of block i, or K of block i + 2
            fetch(second ? i + 3 : i + 1);
            half_turn();
        }
        if (works) values((blocks - 1) & 1);
        if (!second) half_turn();
        half_turn();                 // before the next blocks, or the next unit, use LDS
    }
    l += __shfl_xor(l, 32);
    if (!live) return;
    const bool none = l == 0.0f;
    if (whole) {
        typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
        const float r = none ? 0.0f : 1.0f / l;
        uint16_t* dst =
            a.out + ((int64_t)(tile.s.t0 + j) * c.heads * a.G + h * a.G + cc - j * a.G) * D + 4 * half;
#pragma unroll
        for (int u = 0; u < DT; ++u)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                u16x4 y;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    y[k] = none ? (uint16_t)0 : f32_to_bf16(none_below<COLS>(acc[u][e + k] * r));
                *(u16x4*)(dst + 32 * u + 2 * e) = y;
            }
    } else {
        const uint32_t place = slot * COLS + col;
        float* part = a.part + (int64_t)place * D + 4 * half;
        if (half == 0) a.stat[place] = make_float2(m, l);
#pragma unroll
        for (int u = 0; u < DT; ++u)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                f32x4 o;
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] = acc[u][e + k];
                *(f32x4*)(part + 32 * u + 2 * e) = o;
            }
    }
}

// COLS 16, 32 and 64: the int8 path, 256: the fp16 path
template <int COLS>
constexpr int att_threads() { return COLS <= 64 ? 64 * kAttWaves : 64 * kTileWaves; }

template <int D, int COLS, bool STREAM>
__global__ __launch_bounds__(att_threads<COLS>(), COLS <= 64 ? 3 : 2) void kv_attend_kernel(KvCache c, KvBatch b,
                                                                                            AttArgs a)
{
    const int lane = threadIdx.x & 63;
    AttTile tile;
    AttShare r = {0, 1};
    uint32_t x = 0, x0 = 0, x1 = 1, at = 0;
    int i = 0;
    if (a.groups > 0) {
        // the line: every lane sums the shares of a run of sequences, up to the
        // first descent of cu (so that no rows are counted twice, and the sums
        // stay in the bits that the launcher has checked)
        const int run = (b.nseq + 63) / 64;
        uint32_t mine = 0;
        bool falls = false;
        for (int k = lane * run; k < lane * run + run && k < b.nseq && !falls; ++k) {
            r = att_share<COLS>(b, k, a, tile.s);
            falls = tile.s.n < 0;
            mine += r.tiles * c.heads * r.len;
        }
        const uint64_t fell = __ballot(falls);
        const int lanes = fell ? __builtin_ctzll(fell) : 63;  // the last that counts
        if (lane > lanes) mine = 0;
        uint32_t upto = mine;
        if (b.nseq > 1)
            for (int off = 1; off < 64; off <<= 1) {
                const uint32_t o = __shfl(upto, lane - off);
                if (lane >= off) upto += o;
            }
        const uint32_t total = __builtin_amdgcn_readlane(upto, b.nseq > 1 ? 63 : 0);
        if (blockIdx.x == 0 && threadIdx.x < 64) {           // for the joining kernel
            uint32_t from = upto - mine;
            bool counts = lane <= lanes;
            for (int k = lane * run; k < lane * run + run && k < b.nseq; ++k) {
                KvSeq s;
                const AttShare o = att_share<COLS>(b, k, a, s);
                counts = counts && s.n >= 0;
                a.start[k] = counts ? from : total;
                from += o.tiles * c.heads * o.len;
            }
            if (lane == 0) a.start[b.nseq] = total;
        }
        // per <= total (both whole turns), so x passes total, below 2^31, by less than a turn of all workgroups
        const uint32_t per = att_stretch<COLS>(total, a.groups);
        x0 = x = blockIdx.x * per;
        x1 = x > total || total - x < per ? total : x + per;
        if (x >= x1) return;
        // the lane whose run holds x, then the sequence inside the run
        const int owner = b.nseq > 1 ? __popcll(__ballot(upto <= x)) : 0;
        at = __builtin_amdgcn_readlane(upto - mine, owner);
        i = uni(owner * run);
        r = att_share<COLS>(b, i, a, tile.s);
        r = {(uint32_t)uni(r.tiles), (uint32_t)uni(r.len)};
    }
    while (true) {
        int h, number, begin = 0, end = INT32_MAX;
        bool whole = true, any;
        uint32_t slot = 0;
        if (a.groups == 0) {
            // heads fastest (a head's workgroups meet in one XCD's L2 where heads are a
            // multiple of 8), the last tiles, with the most to see, first
            const uint32_t item = (gridDim.x - 1 - blockIdx.x) / c.heads;
            int64_t local;
            any = kv_find(b, item, a.G, COLS, 1, tile.s, local);
            const int64_t cols = any ? (int64_t)tile.s.n * a.G : 0;
            any = any && cols >= a.min_cols && cols <= a.max_cols;
            number = any ? uni((int)local) : 0;
            h = gridDim.x - 1 - blockIdx.x - item * c.heads;
            x = x1;
        } else {
            while (x - at >= r.tiles * c.heads * r.len) {     // ends: x < total
                at += r.tiles * c.heads * r.len;
                r = att_share<COLS>(b, ++i, a, tile.s);
                r = {(uint32_t)uni(r.tiles), (uint32_t)uni(r.len)};
            }
            const uint32_t unit = (x - at) / r.len, from = x - at - unit * r.len;
            const uint32_t len = r.len - from < x1 - x ? r.len - from : x1 - x;
            h = (int)(unit / r.tiles);
            number = (int)(unit - h * r.tiles);
            begin = (int)from;
            end = (int)(from + len);
            whole = len == r.len;
            slot = blockIdx.x * 2 + (x > x0);
            x += len;
            any = true;
        }
        if (any && att_tile<COLS>(b, number, a.G, a.window, tile)) {
            att_uniform(tile);
            end = end < tile.nblk ? end : tile.nblk;
            if (begin < end || begin == 0) {
                if constexpr (COLS <= 64) attend_blocks<D, COLS / 16, STREAM>(c, b, a, tile, h, begin, end, whole, slot);
                else attend_tile_f16<D>(c, b, a, tile, h, begin, end, whole, slot);
            }
        }
        if (x >= x1) break;
        __syncthreads();                                      // LDS is used again
    }
}

// Joins the parts of every row and query head that lie in more than one
// stretch.  JW waves take one row's parts in turn, eight loads each in
// flight; with one wave a workgroup holds four rows.
template <int D, int COLS, int JW>
__global__ __launch_bounds__(JW == 1 ? 256 : 64 * JW) void kv_attend_join_kernel(KvCache c, KvBatch b, AttArgs a)
{
    constexpr int kRows = JW == 1 ? 4 : 1;
    __shared__ float so[JW][D];
    const int lane = threadIdx.x & 63, wave = JW == 1 ? 0 : threadIdx.x >> 6;
    const uint32_t Hq = c.heads * a.G, id = blockIdx.x * kRows + (JW == 1 ? threadIdx.x >> 6 : 0);
    AttTile tile;
    AttShare r;
    int64_t cc;                // column of the sequence
    int h;
    if (a.by_sequence) {       // id: sequence, head, column
        const uint32_t i = id / (c.heads * a.max_cols), rest = id - i * c.heads * a.max_cols;
        if (i >= (uint32_t)b.nseq) return;
        r = att_share<COLS>(b, i, a, tile.s);
        h = rest / a.max_cols;
        cc = rest - h * a.max_cols;
        if (cc >= (int64_t)tile.s.n * a.G) return;
    } else {                   // id: row, query head
        const uint32_t t = id / Hq;
        const int hq = id - t * Hq;
        int64_t j;
        if (t >= (uint32_t)b.T || !kv_find(b, t, 1, 1, 0, tile.s, j) || j >= tile.s.n) return;
        r = att_share<COLS>(b, tile.s.i, a, tile.s);
        h = hq / a.G;
        cc = j * a.G + (hq - h * a.G);
    }
    if (r.tiles == 0) return;
    const bool alone = b.nseq == 1;          // one load's latency less
    const uint32_t total = alone ? r.tiles * c.heads * r.len : a.start[b.nseq], start = alone ? 0 : a.start[tile.s.i];
    if (start >= total) return;              // behind a descent of cu
    const int number = (int)(cc / COLS), col = (int)(cc % COLS);
    if (!att_tile<COLS>(b, number, a.G, a.window, tile)) return;
    const uint32_t per = att_stretch<COLS>(total, a.groups);
    const uint32_t u0 = start + (h * r.tiles + number) * r.len, w0 = u0 / per;
    if ((u0 + r.len - 1) / per == w0) return;                       // whole: written already
    const int used = (int)((u0 + (tile.nblk > 0 ? tile.nblk : 1) - 1) / per - w0) + 1;   // parts with blocks seen
    // part s > 0 starts its stretch, part 0 may start inside one
    const auto place = [&](int s) { return (2 * (w0 + s) + (s == 0 && u0 > w0 * per)) * COLS + col; };
    float top = -INFINITY, sum = 0.0f, o[D / 64] = {};
    for (int seg = 0; seg < used; seg += 8 * JW) {
        float x[8][D / 64];
        float2 st[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {               // behind the last part its values are read again, unused
            const int s = seg + wave + JW * k;
            const uint32_t at = place(s < used ? s : used - 1);
            st[k] = a.stat[at];
            if (s >= used) st[k] = make_float2(-INFINITY, 0.0f);
#pragma unroll
            for (int u = 0; u < D / 64; ++u) x[k][u] = a.part[(int64_t)at * D + u * 64 + lane];
        }
        float now = top;
#pragma unroll
        for (int k = 0; k < 8; ++k) now = fmaxf(now, st[k].x);
        const float keep = top == now ? 1.0f : exp2_fast(top - now);
        top = now;
        sum *= keep;
#pragma unroll
        for (int u = 0; u < D / 64; ++u) o[u] *= keep;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float f = st[k].x == top ? 1.0f : exp2_fast(st[k].x - top);
            sum = fmaf(st[k].y, f, sum);
#pragma unroll
            for (int u = 0; u < D / 64; ++u) o[u] = seg + wave + JW * k < used ? fmaf(x[k][u], f, o[u]) : o[u];
        }
    }
    const int row = (int)(cc / a.G);
    uint16_t* dst = a.out + ((int64_t)(tile.s.t0 + row) * Hq + h * a.G + (cc - (int64_t)row * a.G)) * D;
    if constexpr (JW == 1) {
#pragma unroll
        for (int u = 0; u < D / 64; ++u)
            dst[u * 64 + lane] = f32_to_bf16(sum == 0.0f ? 0.0f : none_below<COLS>(o[u] / sum));
    } else {
        __shared__ float2 sst[JW];
        if (lane == 0) sst[wave] = make_float2(top, sum);
#pragma unroll
        for (int u = 0; u < D / 64; ++u) so[wave][u * 64 + lane] = o[u];
        __syncthreads();
        const int d = threadIdx.x;
        if (d >= D) return;
        float y = 0.0f;
        sum = 0.0f;
#pragma unroll
        for (int w = 0; w < JW; ++w) top = fmaxf(top, sst[w].x);
#pragma unroll
        for (int w = 0; w < JW; ++w) {
            const float f = sst[w].x == top ? 1.0f : exp2_fast(sst[w].x - top);
            y = fmaf(so[w][d], f, y);
            sum = fmaf(sst[w].y, f, sum);
        }
        dst[d] = f32_to_bf16(sum == 0.0f ? 0.0f : none_below<COLS>(y / sum));
    }
}

// How a launch is cut: columns per workgroup, tiles at most, workgroups that
// share the line (0: one for each unit, no second kernel), which sequences.
struct AttPart {
    int cols, groups, min_cols, max_cols;
    bool streams;
    int64_t items;
    int64_t part_floats, stats, starts;
    int64_t bytes() const { return part_floats * 4 + stats * 8 + (starts + 3) / 4 * 16; }
};

// A call is one launch, or two where a batch may hold prompts beside single
// tokens: only the device knows the rows of each sequence.
struct AttPlan {
    AttPart part[2];
    int parts;
    int64_t bytes() const { return part[0].bytes() + (parts > 1 ? part[1].bytes() : 0); }
};

constexpr int64_t kAttGroups = 768;          // three workgroups a CU: what registers allow on the int8 path
constexpr int64_t kTileGroups = 256;         // one a CU on the fp16 path

// The choice of path.  A unit (tile of columns, head) whole in one workgroup
// needs no second kernel, and the tiles of a head run side by side and share
// its blocks in L2; split, a long unit does not wait for one workgroup.
// Measured on caches used in turn, 32:8 heads of 128, lengths evenly spread up
// to the one given (16 columns whole / 16 split / 64 split / 256 fp16, us):
//   1 x 1 row up to 1500     10.9 / 11.3 /   -  /   -      up to 3000  17.4 / 12.0 /   -  /   -
//   16 x 1 up to 3000        20.9 / 22.2 /   -  /   -      up to 4500  29.5 / 27.7 /   -  /   -
//   64 x 1 up to 3000        42.6 / 45.2 /   -  /   -      up to 16000  194 /  178 /   -  /   -
//   16 x 7 up to 3000        21.4 / 33.0 / 30.4 / 52.6     up to 4500  29.7 / 39.7 / 36.4 /   -
//   16 x 16 up to 3000       24.8 / 49.1 / 39.5 / 59.1     up to 12000 80.8 /   -  / 81.9 / 105
//   1 x 48 up to 3000        18.5 / 22.0 / 27.1 / 34.3     up to 12000 55.7 / 39.5 / 36.6 / 41.8
//   8 x 64 up to 3000        32.6 / 79.1 / 51.7 / 54.9     up to 12000  112 /   -  / 122  / 94.2
//   32 x 128 up to 1500       127 /  -   /  -   / 86.8     up to 12000  672 /   -  /   -  / 447
// (32 x 128 up to 600: 82.5 with 16 columns, 60.4 with 32, 49.9 with 64.)
constexpr int64_t kAttWhole = 22;            // blocks up to which a lone unit stays whole
// one long sequence among many short ones is waited for alone: 64 x 16 rows over 500, one of them over 12000,
// 110 us whole and 55 split, over 6000 62 and 65; more than 64 columns are several tiles, split or not, and
// gain more where all are long (32 x 24 rows up to 12000 167 whole, 250 split)
constexpr int64_t kAttWholeMost = 128;
constexpr int64_t kAttShared = 4096;         // (block, head) pairs from which split tiles of one head share their reads
constexpr int64_t kAttPair = 2048, kAttQuad = 4096;   // units from which two or four whole tiles share theirs
constexpr int64_t kAttTileCols = 128;        // columns a sequence from which 256-column tiles are looked at
constexpr int64_t kAttSmall = 24576;         // (unit of 16 columns, block) pairs up to which split ones do not pay off
constexpr int64_t kAttMixed = 512;           // columns that one of several sequences may have: then both paths

// Caches that pass the last-level cache (256 MB) are read past it: 64 streams
// up to 16000 (2.1 GB at most, 483 MB) 95 us against 107; below, the plain
// loads are faster, one stream over 40960 (84 MB) 23.8 us against 25.2.  Not
// where several waves or tiles read a block (16 x 48 rows up to 12000 217 us
// against 151, 64 x 16 up to 12000 split 386 against 265).
constexpr double kAttStream = 256 << 20;

static void att_cut(AttPart& p, int64_t cols, int64_t heads, int64_t D, int64_t nseq, int64_t blocks, bool whole)
{
    p.items = cols / p.cols + nseq;
    p.streams = cols <= 16 * nseq && (double)(nseq * heads * blocks) * (2 * kKvBlock * D) > kAttStream;
    if (whole) return;
    const int64_t units = p.items * heads, groups = p.cols == 256 ? kTileGroups : kAttGroups;
    const int64_t turn = p.cols <= 64 ? 64 / p.cols : 1, turns = (blocks + turn - 1) / turn;
    p.groups = (int)(units > groups / turns ? groups : units * turns);
    p.stats = (int64_t)p.groups * 2 * p.cols;
    p.part_floats = p.stats * D;
    p.starts = nseq + 1;
}

static AttPlan att_plan(int64_t T, int64_t Hq, int64_t heads, int64_t D, int64_t nseq, int64_t max_len,
                        int64_t max_rows, int64_t window)
{
    AttPlan p{};
    AttPart &first = p.part[0], &second = p.part[1];
    // blocks that a unit has at most
    const int64_t G = Hq / heads, cols = T * G, all = (max_len + kKvBlock - 1) / kKvBlock;
    const int64_t seen = window > 0 ? window / kKvBlock + 256 / kKvBlock + 2 : all;
    const bool windowed = seen < all;
    const int64_t blocks = windowed ? seen : all;
    const bool small = (cols / 16 + nseq) * heads * blocks <= kAttSmall;
    // the most columns that a sequence may have; not told, a batch of few rows
    // each is taken for one of drafts
    const int64_t rows = nseq == 1 ? T : max_rows > 0 ? max_rows : T > 16 * nseq ? T - nseq + 1 : 16;
    const int64_t most = (rows < T ? rows : T) * G;
    const auto units = [&](int64_t c) {
        const int64_t n = (cols + c - 1) / c;
        return (n > nseq ? n : nseq) * heads;
    };
    const int64_t u16 = units(16), u256 = units(256);
    // estimates in us from the table's kind of measurements: the longest unit,
    // and (unit, block) pairs over the card; rows of one sequence see all but
    // half of themselves; the lengths of several lie between all alike and evenly
    // spread from none (0.5 of the longest on average)
    const double mean = windowed    ? (double)blocks
                        : nseq == 1 ? (double)(blocks - (T < max_len ? T : max_len) / (2 * kKvBlock))
                                    : 0.75 * blocks;
    const auto either = [](double a, double b) { return a > b ? a : b; };
    const double rounds = (double)((u256 + kTileGroups - 1) / kTileGroups);
    const double int8 = either(5 + 0.28 * blocks, 5 + 0.95e-3 * u16 * mean);
    const double tile = 1.15 * either(13 + 1.45 * blocks, 5 + 8 * rounds + 7.5e-3 * u256 * mean);
    const double tile_split = 25 + 1.5e-3 * T * Hq + 8e-3 * u256 * mean;
    p.parts = 1;
    first.max_cols = second.max_cols = INT32_MAX;
    bool whole = (blocks <= kAttWhole + u16 / (cols > 16 * nseq ? 2 : 8) || u16 >= 2 * kAttGroups) &&
                 blocks <= (cols > 64 * nseq ? 2 : 1) * kAttWholeMost;
    if (nseq > 1 && most > kAttMixed && cols < most * nseq) {
        // only the prompts' work goes to the tiles, whoever has the longest length
        const double u = (double)((cols + 255) / 256 * heads);
        if (!small && int8 > 15 + 8 * (double)(int64_t)(u / kTileGroups + 1) + 8.6e-3 * u * mean) {
            p.parts = 2;
            first.cols = 256;
            first.min_cols = kAttTileCols + 1;
            second.cols = 16;
            second.max_cols = kAttTileCols;
            att_cut(first, cols, heads, D, nseq, blocks, blocks <= 16 || (cols / 256 + nseq) * heads >= kTileGroups);
            // always split: a grid by units would be idle in a batch of prompts
            att_cut(second, cols, heads, D, nseq, blocks, false);
            return p;
        }
        whole = whole || !small;
    } else if (cols > kAttTileCols * nseq && most > kAttTileCols) {
        const double best = tile < tile_split ? tile : tile_split;
        whole = int8 <= best && (whole || !small);
        if (!whole && !small) {
            first.cols = 256;
            att_cut(first, cols, heads, D, nseq, blocks, tile <= tile_split);
            return p;
        }
    }
    if (whole) {
        const bool pair = u16 >= kAttPair || (u16 >= kAttPair / 2 && blocks <= 16);
        first.cols = cols > 32 * nseq && u16 >= kAttQuad ? 64 : cols > 16 * nseq && pair ? 32 : 16;
    } else {
        first.cols = cols <= 16 * nseq || nseq * heads * blocks < kAttShared ? 16 : cols <= 32 * nseq ? 32 : 64;
    }
    att_cut(first, cols, heads, D, nseq, blocks, whole);
    return p;
}

int64_t kv_attend_workspace_bytes(int64_t T, int64_t Hq, int64_t heads, int64_t D, int64_t nseq, int64_t max_len,
                                  int64_t max_rows)
{
    const AttPlan p = att_plan(T, Hq, heads, D, nseq, max_len, max_rows, 0);
    return p.bytes();
}

template <int D, int COLS>
static hipError_t attend(const KvCache& c, const KvBatch& b, const AttArgs& a, int64_t items, bool streams,
                         hipStream_t stream)
{
    const int64_t grid = a.groups ? a.groups : items * c.heads;
    if (COLS == 16 && streams)
        kv_attend_kernel<D, COLS, COLS == 16><<<(unsigned)grid, att_threads<COLS>(), 0, stream>>>(c, b, a);
    else
        kv_attend_kernel<D, COLS, false><<<(unsigned)grid, att_threads<COLS>(), 0, stream>>>(c, b, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.groups == 0) return e;
    int64_t rows = (int64_t)b.T * c.heads * a.G;
    if (a.by_sequence) rows = (int64_t)b.nseq * c.heads * a.max_cols;
    // few rows: their parts to many waves
    if (rows <= 256)
        kv_attend_join_kernel<D, COLS, 12><<<(unsigned)rows, 768, 0, stream>>>(c, b, a);
    else if (rows <= 2048 && (int64_t)b.nseq * c.heads * 8 < a.groups)
        kv_attend_join_kernel<D, COLS, 4><<<(unsigned)rows, 256, 0, stream>>>(c, b, a);
    else
        kv_attend_join_kernel<D, COLS, 1><<<(unsigned)((rows + 3) / 4), 256, 0, stream>>>(c, b, a);
    return hipGetLastError();
}

template <int D>
static hipError_t attend_part(const KvCache& c, const KvBatch& b, const AttArgs& a, const AttPart& p,
                              hipStream_t stream)
{
    switch (p.cols) {
    case 16: return attend<D, 16>(c, b, a, p.items, p.streams, stream);
    case 32: return attend<D, 32>(c, b, a, p.items, p.streams, stream);
    case 64: return attend<D, 64>(c, b, a, p.items, p.streams, stream);
    default: return attend<D, 256>(c, b, a, p.items, p.streams, stream);
    }
}

// the plan of one call
static AttPlan att_choose(int64_t T, int64_t Hq, int64_t heads, int64_t D, int64_t nseq, int64_t table_width,
                          int64_t window, int64_t max_len, int64_t max_rows)
{
    AttPlan plan = att_plan(T, Hq, heads, D, nseq, max_len, max_rows, 0);
    if (window > 0) {
        // what a window leaves to see is often short enough for whole units (64 x 7 rows up to 12000, window
        // 512: 26 us instead of 42), but the workspace was sized for any window
        const AttPlan near = att_plan(T, Hq, heads, D, nseq, max_len, max_rows, window);
        if (near.bytes() <= plan.bytes()) plan = near;
    }
    for (int i = 0; i < plan.parts; ++i) {
        // the line is counted in 32 bits; a batch that could pass that has units enough
        const int64_t line = plan.part[i].items * heads * (table_width + kAttWaves);
        if (line >= (1ll << 31)) plan.part[i].groups = 0;
    }
    return plan;
}

int kv_attend_config(int64_t T, int64_t Hq, int64_t heads, int64_t D, int64_t nseq, int64_t table_width,
                     int64_t window, int64_t max_len, int64_t max_rows, int64_t* out)
{
    const AttPlan plan = att_choose(T, Hq, heads, D, nseq, table_width, window, max_len, max_rows);
    for (int i = 0; i < plan.parts; ++i) {
        const AttPart& p = plan.part[i];
        *out++ = p.cols;
        *out++ = p.groups;
        *out++ = p.groups ? p.groups : p.items * heads;
        *out++ = p.min_cols;
        *out++ = p.max_cols;
        *out++ = p.cols == 16 && p.streams;
    }
    return plan.parts;
}

hipError_t launch_kv_attend(const KvCache& c, const KvBatch& b, int64_t D, const uint16_t* q, int64_t Hq,
                            int64_t q_stride, float scale, int64_t window, int64_t max_len, int64_t max_rows,
                            uint16_t* out, void* workspace, hipStream_t stream)
{
    const AttPlan plan = att_choose(b.T, Hq, c.heads, D, b.nseq, b.table_width, window, max_len, max_rows);
    uint8_t* ws = (uint8_t*)workspace;
    for (int i = 0; i < plan.parts; ++i) {
        const AttPart& p = plan.part[i];
        AttArgs a{};
        a.q = q;
        a.out = out;
        a.part = (float*)ws;
        a.stat = (float2*)(a.part + p.part_floats);
        a.start = (uint32_t*)(a.stat + p.stats);
        ws += p.bytes();
        a.q_stride = q_stride;
        a.window = window < INT32_MAX ? (int)window : 0;      // one that nothing is as far as
        a.scale = scale;
        a.G = (int)(Hq / c.heads);
        a.min_cols = p.min_cols;
        a.max_cols = p.max_cols;
        a.by_sequence = p.max_cols < INT32_MAX && (int64_t)b.nseq * p.max_cols < (int64_t)b.T * a.G;
        a.groups = p.groups;
        const hipError_t e = D == 128 ? attend_part<128>(c, b, a, p, stream) : attend_part<64>(c, b, a, p, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace tern
