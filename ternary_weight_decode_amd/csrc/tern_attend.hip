// tern_attend.hip — attention over the paged int8 cache.
//
//   out = sum_p w_p V[p] / sum_p w_p,  w_p = exp(scale * q . K[p])
//
// The rows of one key/value head are columns here: column c of a sequence is
// row c / G under query head h*G + c % G, so a group's G query heads share one
// pass over the cached bytes.
//
// kv_attend_i8_kernel: 16 * CT columns per workgroup, for single tokens and
// drafts, bound by the cache's bytes.  The codes go from memory to the int8
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
// of a workgroup meet in LDS at the end, the parts of a long sequence in a
// second kernel.
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

// The tile of columns a workgroup or a combining row works on.
struct AttTile {
    KvSeq s;
    int col0, cols;            // first column, live columns
    int64_t b0;                // first block any of them sees
    int64_t nblk;              // blocks from there to the last one seen
};

__device__ __forceinline__ int64_t att_first(int64_t pos, int64_t window)
{
    return window > 0 && pos >= window ? pos - window + 1 : 0;
}

__device__ __forceinline__ int64_t att_last(int64_t pos, int64_t limit) { return pos < limit ? pos : limit; }

// columns [COLS * tile, + COLS) of the sequence that owns `item`
template <int COLS>
__device__ __forceinline__ bool att_tile(const KvBatch& b, int64_t item, int G, int64_t window, AttTile& a)
{
    int64_t local;
    if (!kv_find(b, item, G, COLS, 1, a.s, local)) return false;
    const int64_t total = (int64_t)a.s.n * G;
    if (local * COLS >= total) return false;
    a.col0 = (int)(local * COLS);
    a.cols = (int)(total - a.col0 < COLS ? total - a.col0 : COLS);
    const int64_t limit = b.table_width * kKvBlock - 1;
    const int64_t lo = att_first(a.s.p0 + a.col0 / G, window);
    const int64_t hi = att_last(a.s.p0 + (a.col0 + a.cols - 1) / G, limit);
    a.b0 = lo / kKvBlock;
    a.nblk = hi < lo ? 0 : hi / kKvBlock - a.b0 + 1;
    return true;
}

struct AttArgs {
    const uint16_t* q;
    uint16_t* out;
    float* part;               // [items][heads][slots][COLS][D] unnormalised sums, then their (max, sum)
    float2* stat;
    int64_t q_stride;
    int64_t window;
    float scale;
    int G;
    int chunk, slots;          // blocks per workgroup, workgroups along a sequence
};

template <int D, int CT>
__global__ __launch_bounds__(64 * kAttWaves) void kv_attend_i8_kernel(KvCache c, KvBatch b, AttArgs a)
{
    constexpr int S = D / 64, U = D / 16, COLS = 16 * CT;
    constexpr int kPad = D + 4;
    __shared__ float sacc[kAttWaves][COLS][kPad];
    __shared__ float2 sstat[kAttWaves][COLS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = lane & 15, g = lane >> 4;
    // slots fastest: neighbouring workgroups read neighbouring parts of one sequence
    const int slot = blockIdx.x % a.slots;
    const int h = blockIdx.x / a.slots % c.heads;
    const int64_t item = blockIdx.x / a.slots / c.heads;
    AttTile tile;
    if (!att_tile<COLS>(b, item, a.G, a.window, tile)) return;
    const int64_t begin = (int64_t)slot * a.chunk;
    // the last slot takes what is left (lengths above the caller's bound)
    const int64_t end = slot == a.slots - 1 || begin + a.chunk > tile.nblk ? tile.nblk : begin + a.chunk;
    if (begin >= end && slot > 0) return;

    // this lane's columns: q as planes, the factor of its scores, the keys it sees
    const int64_t limit = b.table_width * kKvBlock - 1;
    u32x4 qhi[CT][S], qlo[CT][S];
    float rowf[CT];
    int64_t first[CT], last[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const int col = 16 * ct + n;
        const bool live = col < tile.cols;
        const int cc = tile.col0 + (live ? col : 0);
        const int j = cc / a.G;
        const uint16_t* row = a.q + (tile.s.t0 + j) * a.q_stride + (int64_t)(h * a.G + cc % a.G) * D;
        const int64_t pos = tile.s.p0 + j;
        first[ct] = live ? att_first(pos, a.window) : 0;
        last[ct] = live ? att_last(pos, limit) : INT64_MAX;
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
        rowf[ct] = amax * (a.scale * kLog2e / kPlane);
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t w0 = raw[s][e >> 1][2 * (e & 1)], w1 = raw[s][e >> 1][2 * (e & 1) + 1];
                uint32_t hi, lo;
                planes(__builtin_bit_cast(float, w0 << 16) * inv, __builtin_bit_cast(float, w0 & 0xFFFF0000u) * inv,
                       __builtin_bit_cast(float, w1 << 16) * inv, __builtin_bit_cast(float, w1 & 0xFFFF0000u) * inv,
                       hi, lo);
                qhi[ct][s][e] = inv == 0.0f ? 0u : hi;
                qlo[ct][s][e] = inv == 0.0f ? 0u : lo;
            }
    }

    float m[CT], l[CT];
    f32x4 acc[CT][U];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        m[ct] = -INFINITY;
        l[ct] = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) acc[ct][u] = f32x4{0, 0, 0, 0};
    }

    for (int64_t seg = begin; seg < end; seg += 64) {
        // lane i looks up block seg + i: its place and scales
        const int count = (int)(end - seg < 64 ? end - seg : 64);
        int mine = -1;
        float2 sc = make_float2(0.0f, 0.0f);
        if (lane < count) {
            mine = (int)kv_block(b, c, tile.s.i, tile.b0 + seg + lane);
            if (mine >= 0) sc = *(const float2*)(c.scales + ((int64_t)mine * c.heads + h) * 2);
        }
        for (int i = wave; i < count; i += kAttWaves) {
            const int phys = __builtin_amdgcn_readlane(mine, i);
            if (phys < 0) continue;
            const float sk = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sc.x), i));
            const float sv = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sc.y), i));
            const int8_t* kc = c.codes + ((int64_t)phys * c.heads + h) * 2 * (kKvBlock * D);
            const u32x4* kp = (const u32x4*)kc + lane;
            const u32x4* vp = (const u32x4*)(kc + kKvBlock * D) + lane;
            u32x4 kr[4][S], vr[U];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int s = 0; s < S; ++s) kr[t][s] = kp[64 * (t * S + s)];
#pragma unroll
            for (int u = 0; u < U; ++u) vr[u] = vp[64 * u];
            const int64_t at = (tile.b0 + seg + i) * kKvBlock;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                float x[16];
                const float f = rowf[ct] * sk;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    i32x4 hi = {0, 0, 0, 0}, lo = {0, 0, 0, 0};
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        hi = mfma_i8(kr[t][s], qhi[ct][s], hi);
                        lo = mfma_i8(kr[t][s], qlo[ct][s], lo);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[4 * t + e] = (float)(hi[e] * 256 + lo[e]) * f;
                }
                const bool sees = first[ct] <= at + 63 && last[ct] >= at;
                if (__any(first[ct] > at || last[ct] < at + 63)) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int64_t p = at + 16 * (e >> 2) + 4 * g + (e & 3);
                        x[e] = p >= first[ct] && p <= last[ct] ? x[e] : -INFINITY;
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
                const float mn = fmaxf(m[ct], top);
                const float keep = m[ct] == mn ? 1.0f : exp2_fast(m[ct] - mn);
                const float join = top == -INFINITY ? 0.0f : exp2_fast(top - mn);
                const float fv = sees ? join * sv * (1.0f / 32767.0f) : 0.0f;
                m[ct] = mn;
                l[ct] = l[ct] * keep + sum * join;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const i32x4 zero = {0, 0, 0, 0};
                    const i32x4 hi = mfma_i8(vr[u], phi, zero), lo = mfma_i8(vr[u], plo, zero);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[ct][u][e] = fmaf((float)(hi[e] * 256 + lo[e]), fv, acc[ct][u][e] * keep);
                }
            }
        }
    }

    // the waves meet: common maximum, scaled sums
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        l[ct] += __shfl_xor(l[ct], 16);
        l[ct] += __shfl_xor(l[ct], 32);
        if (g == 0) sstat[wave][16 * ct + n] = make_float2(m[ct], l[ct]);
    }
    __syncthreads();
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kAttWaves; ++w) top = fmaxf(top, sstat[w][16 * ct + n].x);
        const float f = m[ct] == top ? 1.0f : exp2_fast(m[ct] - top);
#pragma unroll
        for (int u = 0; u < U; ++u) *(f32x4*)&sacc[wave][16 * ct + n][16 * u + 4 * g] = acc[ct][u] * f;
    }
    __syncthreads();
    constexpr int kPer = D / 4;                     // threads per column, four dims each
    for (int i = threadIdx.x; i < tile.cols * kPer; i += 64 * kAttWaves) {
        const int col = i / kPer, d = i % kPer * 4;
        float top = -INFINITY, sum = 0.0f;
        f32x4 o = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kAttWaves; ++w) top = fmaxf(top, sstat[w][col].x);
#pragma unroll
        for (int w = 0; w < kAttWaves; ++w) {
            const float2 st = sstat[w][col];
            sum += st.y * (st.x == top ? 1.0f : exp2_fast(st.x - top));
            o += *(const f32x4*)&sacc[w][col][d];
        }
        if (a.slots > 1) {
            const int64_t at = ((item * c.heads + h) * a.slots + slot) * COLS + col;
            *(f32x4*)(a.part + at * D + d) = o;
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

// Joins the parts of every column: one workgroup per column, its waves take
// the parts in turn.
constexpr int kJoinWaves = 8;

template <int D, int COLS>
__global__ __launch_bounds__(64 * kJoinWaves) void kv_attend_join_kernel(KvCache c, KvBatch b, AttArgs a)
{
    __shared__ float so[kJoinWaves][D], sf[kJoinWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = blockIdx.x % COLS, h = blockIdx.x / COLS % c.heads;
    const int64_t item = blockIdx.x / COLS / c.heads;
    AttTile tile;
    if (!att_tile<COLS>(b, item, a.G, a.window, tile) || col >= tile.cols) return;
    int64_t used = (tile.nblk + a.chunk - 1) / a.chunk;
    used = used < 1 ? 1 : used > a.slots ? a.slots : used;
    const int64_t at = (item * c.heads + h) * a.slots * COLS + col;
    const float2* stat = a.stat + at;
    const float* part = a.part + at * D + lane;
    float top = -INFINITY;
    for (int64_t s = lane; s < used; s += 64) top = fmaxf(top, stat[s * COLS].x);
    for (int off = 1; off < 64; off <<= 1) top = fmaxf(top, __shfl_xor(top, off));
    float sum = 0.0f, o[D / 64] = {};
    for (int64_t seg = 0; seg < used; seg += 64) {
        const int count = (int)(used - seg < 64 ? used - seg : 64);
        float f = 0.0f;
        if (lane < count) {
            const float2 st = stat[(seg + lane) * COLS];
            f = st.x == top ? 1.0f : exp2_fast(st.x - top);
            sum += st.y * f;
        }
        sf[wave][lane] = f;              // 0 behind the last part
        __builtin_amdgcn_wave_barrier();
        // eight loads in flight; behind the last part its values are read again and weigh 0
#pragma unroll
        for (int r = 0; r < 64 / kJoinWaves; ++r) {
            const int i = wave + kJoinWaves * r, ic = i < count ? i : count - 1;
            const float fi = sf[wave][i];
#pragma unroll
            for (int u = 0; u < D / 64; ++u) {
                const float x = part[(seg + ic) * COLS * D + u * 64];
                o[u] = i < count ? fmaf(x, fi, o[u]) : o[u];
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
    for (int off = 1; off < 64; off <<= 1) sum += __shfl_xor(sum, off);
#pragma unroll
    for (int u = 0; u < D / 64; ++u) so[wave][u * 64 + lane] = o[u];
    __syncthreads();
    const int d = threadIdx.x;
    if (d >= D) return;
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWaves; ++w) y += so[w][d];
    const int cc = tile.col0 + col;
    a.out[((int64_t)(tile.s.t0 + cc / a.G) * c.heads * a.G + h * a.G + cc % a.G) * D + d] =
        f32_to_bf16(sum == 0.0f ? 0.0f : y / sum);
}

// How a call is cut: columns per workgroup, blocks per workgroup, workgroups
// along a sequence.
struct AttPlan {
    int cols, chunk, slots;
    int64_t items;
    int64_t part_floats, stats;
};

static AttPlan att_plan(int64_t T, int64_t Hq, int64_t heads, int64_t D, int64_t nseq, int64_t max_len)
{
    AttPlan p;
    const int64_t G = Hq / heads;
    p.cols = T * G <= 16 * nseq ? 16 : 32;
    p.items = T * G / p.cols + nseq;
    const int64_t blocks = (max_len + kKvBlock - 1) / kKvBlock, base = p.items * heads;
    int64_t slots = blocks * base / 1024 < 32 ? 1024 / base : (blocks + 31) / 32;
    const int64_t most = 8192 / base, useful = (blocks + kAttWaves - 1) / kAttWaves;
    slots = slots > most ? most : slots;
    slots = slots > useful ? useful : slots;
    slots = slots < 1 ? 1 : slots;
    const int64_t chunk = (blocks + slots - 1) / slots;
    p.chunk = (int)((chunk + kAttWaves - 1) / kAttWaves * kAttWaves);
    p.slots = (int)((blocks + p.chunk - 1) / p.chunk);
    const int64_t n = p.slots > 1 ? p.items * heads * p.slots * p.cols : 0;
    p.part_floats = n * D;
    p.stats = n;
    return p;
}

int64_t kv_attend_workspace_bytes(int64_t T, int64_t Hq, int64_t heads, int64_t D, int64_t nseq, int64_t max_len)
{
    const AttPlan p = att_plan(T, Hq, heads, D, nseq, max_len);
    return p.part_floats * 4 + p.stats * 8;
}

template <int D, int CT>
static hipError_t attend_i8(const KvCache& c, const KvBatch& b, const AttArgs& a, const AttPlan& p,
                            hipStream_t stream)
{
    const int64_t grid = p.items * c.heads * p.slots;
    kv_attend_i8_kernel<D, CT><<<(unsigned)grid, 64 * kAttWaves, 0, stream>>>(c, b, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.slots == 1) return e;
    kv_attend_join_kernel<D, 16 * CT>
        <<<(unsigned)(p.items * c.heads * 16 * CT), 64 * kJoinWaves, 0, stream>>>(c, b, a);
    return hipGetLastError();
}

hipError_t launch_kv_attend(const KvCache& c, const KvBatch& b, int64_t D, const uint16_t* q, int64_t Hq,
                            int64_t q_stride, float scale, int64_t window, int64_t max_len, uint16_t* out,
                            void* workspace, hipStream_t stream)
{
    const AttPlan p = att_plan(b.T, Hq, c.heads, D, b.nseq, max_len);
    AttArgs a{};
    a.q = q;
    a.out = out;
    a.part = (float*)workspace;
    a.stat = (float2*)((float*)workspace + p.part_floats);
    a.q_stride = q_stride;
    a.window = window;
    a.scale = scale;
    a.G = (int)(Hq / c.heads);
    a.chunk = p.chunk;
    a.slots = p.slots;
    if (D == 128) return p.cols == 16 ? attend_i8<128, 1>(c, b, a, p, stream) : attend_i8<128, 2>(c, b, a, p, stream);
    return p.cols == 16 ? attend_i8<64, 1>(c, b, a, p, stream) : attend_i8<64, 2>(c, b, a, p, stream);
}

}  // namespace tern
