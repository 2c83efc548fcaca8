// tern_kv.hip — query/key norm with rotation, and the paged int8 cache's
// append and read.
//
// A head vector of D elements belongs to 16 lanes (four vectors per wave).
// Lane j holds two runs of E = D/32 elements, from dim E*j and from
// D/2 + E*j, so that both members of a rotation pair are its own in the
// half-split style (j, j + D/2) as well as in the interleaved one (2j, 2j+1),
// loads are 16 bytes (fp32, D = 128) and sums of squares and maxima need four
// lane exchanges.
#include "tern_device.h"
#include "tern_kv.h"
#include "tern_launch.h"

namespace tern {

// E contiguous elements of a head vector
template <int E, typename TI>
__device__ __forceinline__ void load_run(const TI* p, float* x)
{
    if constexpr (sizeof(TI) == 4) {
        typedef float vec __attribute__((ext_vector_type(E)));
        const vec v = *(const vec*)p;
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = v[i];
    } else {
        typedef uint16_t vec __attribute__((ext_vector_type(E)));
        const vec v = *(const vec*)p;
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = bf16_to_f32(v[i]);
    }
}

template <int E, typename TO>
__device__ __forceinline__ void store_run(TO* p, const float* x)
{
    typedef TO vec __attribute__((ext_vector_type(E)));
    vec v;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        if constexpr (sizeof(TO) == 4) v[i] = x[i];
        else v[i] = f32_to_bf16(x[i]);
    }
    *(vec*)p = v;
}

// cos and sin of pos * inv_freq: the angle in revolutions in fp64 (off by at
// most pos * 2^-52 of a revolution), its fraction in fp32
__device__ __forceinline__ void turn(int pos, double inv_freq, float& c, float& s)
{
    constexpr double kPerRev = 0.15915494309189533577;   // 1 / (2 pi)
    const double rev = (double)pos * (inv_freq * kPerRev);
    const float half_turns = (float)(2.0 * (rev - rint(rev)));
    sincospif(half_turns, &s, &c);
}

// index into [D/2] angles of the pair that element i of run `run` (0, 1) starts or joins
template <int D>
__device__ __forceinline__ int pair_of(int j, int run, int i, bool interleaved)
{
    constexpr int E = D / 32;
    return interleaved ? (run * (D / 2) + E * j + i) / 2 : E * j + i;
}

// RMS norm over the 16 lanes' vector, both runs in x[0..E) and x[E..2E)
template <int D>
__device__ __forceinline__ void norm(float* x, const float* gain, float eps, int j)
{
    constexpr int E = D / 32;
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 2 * E; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) ss += __shfl_xor(ss, off);
    const float r = __fdiv_rn(1.0f, __fsqrt_rn(fmaf(ss, 1.0f / D, eps)));
    float g[2 * E];
    load_run<E>(gain + E * j, g);
    load_run<E>(gain + D / 2 + E * j, g + E);
#pragma unroll
    for (int i = 0; i < 2 * E; ++i) x[i] = x[i] * r * g[i];
}

// rotation of a pair, its roundings fixed so that every kernel gives the same bits
__device__ __forceinline__ void rotate_pair(float& a, float& b, float2 w)
{
    const float x = fmaf(a, w.x, -__fmul_rn(b, w.y)), y = fmaf(b, w.x, __fmul_rn(a, w.y));
    a = x;
    b = y;
}

// rotation of a lane's pairs with (cos, sin) = cs(pair)
template <int D, typename CS>
__device__ __forceinline__ void rotate(float* x, int j, bool interleaved, CS cs)
{
    constexpr int E = D / 32;
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 2 * E; i += 2) rotate_pair(x[i], x[i + 1], cs(pair_of<D>(j, i / E, i % E, true)));
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) rotate_pair(x[i], x[i + E], cs(pair_of<D>(j, 0, i, false)));
    }
}

// ---- norm + rotation -------------------------------------------------------
// One workgroup per token and 16 heads; the token's D/2 angles are computed
// once per workgroup.  One token of 32:8 heads takes 2.7 us, an empty kernel
// 1.95; bound by the rows from a few hundred tokens on: 4096 tokens, fp32 in
// and bf16 out (126 MB), 20 us, 6.3 TB/s (the rows just written come in part
// from the last-level cache; a plain copy of as many bytes reaches 4.9).
template <int D, typename TI, typename TO>
__global__ __launch_bounds__(256) void norm_rope_kernel(QkTransform f, const TI* q, int Hq, int64_t q_stride,
                                                        const TI* k, int Hk, int64_t k_stride, const int32_t* pos,
                                                        TO* q_out, TO* k_out, int parts)
{
    constexpr int E = D / 32;
    __shared__ float2 cs[D / 2];
    const int64_t t = blockIdx.x / parts;
    const int part = blockIdx.x % parts;
    if (f.inv_freq) {
        if (threadIdx.x < D / 2) {
            float c, s;
            turn(pos[t], f.inv_freq[threadIdx.x], c, s);
            cs[threadIdx.x] = make_float2(c, s);
        }
        __syncthreads();
    }
    const int j = threadIdx.x & 15;
    const int h = part * 16 + (threadIdx.x >> 4);
    if (h >= Hq + Hk) return;          // a whole group of 16 lanes
    const bool is_q = h < Hq;
    const TI* src = is_q ? q + t * q_stride + (int64_t)h * D : k + t * k_stride + (int64_t)(h - Hq) * D;
    TO* dst = is_q ? q_out + (t * Hq + h) * D : k_out + (t * Hk + h - Hq) * D;
    const float* gain = is_q ? f.q_gain : f.k_gain;
    float x[2 * E];
    load_run<E>(src + E * j, x);
    load_run<E>(src + D / 2 + E * j, x + E);
    if (gain) norm<D>(x, gain, f.eps, j);
    if (f.inv_freq) rotate<D>(x, j, f.interleaved != 0, [&](int p) { return cs[p]; });
    store_run<E>(dst + E * j, x);
    store_run<E>(dst + D / 2 + E * j, x + E);
}

// ---- append ----------------------------------------------------------------
// For every (sequence, touched block, key/value head) one workgroup has K and V
// of all the block's new tokens (the block's scale needs the maximum over them,
// and nothing else writes the block); the queries of their rows are its too where
// tokens are few, have a workgroup of their own where those are too few for the
// card, and four in prompts (figures at the launcher).  Loads are issued before
// the tokens' angles are computed, once per workgroup, into LDS; up to four K and
// four V vectors (or four queries) of each 16-lane group wait in registers.
// Single tokens are bound by the chain cu -> table -> rows -> scale -> codes: 5.7
// us for one, calls one behind another in a graph, 7.2 for 48, an empty kernel
// 1.95.  Prompts are bound by the rows read: 4131 tokens of 32:8 heads of 128
// (144 MB) take 36 us, 4.0 TB/s (35 in a kernel trace), where a plain copy of
// those bytes takes 29.

// the scale after values of magnitude `top` (bits, so that inf < NaN) join;
// shift: doublings that the old codes have to follow, 31 where they vanish
__device__ __forceinline__ float join_scale(float old, uint32_t top_bits, bool first, int& shift)
{
    const float top = __builtin_bit_cast(float, top_bits);
    shift = 0;
    if (first || old == 0.0f) return top_bits >= 0x7F800000u ? top : __fdiv_rn(top, 127.0f);
    if (!(fabsf(old) < INFINITY)) {
        shift = 31;
        return old;
    }
    if (top_bits >= 0x7F800000u) {
        shift = 31;
        return top;
    }
    const float room = 127.0f * old;
    if (!(top > room)) return old;
    // least g with top <= room * 2^g: exact, both sides scaled by powers of two
    int et, er;
    const float mt = frexpf(top, &et), mr = frexpf(room, &er);
    shift = et - er + (mt > mr ? 1 : 0);
    return ldexpf(old, shift);
}

__device__ __forceinline__ uint32_t quantise(float x, float scale)
{
    if (!(scale > 0.0f && scale < INFINITY)) return 0;
    return (uint32_t)(int)fminf(fmaxf(__builtin_rintf(__fdiv_rn(x, scale)), -127.0f), 127.0f) & 0xFFu;
}

// rint(code / 2^shift) of the four codes of a word
__device__ __forceinline__ uint32_t shift_codes(uint32_t w, int shift)
{
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float c = (float)(int8_t)(w >> 8 * i);
        r |= (shift >= 9 ? 0u : (uint32_t)(int)__builtin_rintf(ldexpf(c, -shift)) & 0xFFu) << 8 * i;
    }
    return r;
}

// the first n bytes of a word
__device__ __forceinline__ void store_bytes(int8_t* p, uint32_t w, int n)
{
    if (n >= 4) {
        *(uint32_t*)p = w;
        return;
    }
    for (int i = 0; i < n; ++i) p[i] = (int8_t)(w >> 8 * i);
}

// angles of n tokens into cs[n][D/2]; thread i always has pair i % (D/2)
template <int D>
__device__ __forceinline__ void angles(float2* cs, int n, const double* inv_freq, const int32_t* pos, int first)
{
    const int p = threadIdx.x % (D / 2);
    const double f = inv_freq[p];
    for (int t = threadIdx.x / (D / 2); t < n; t += 256 / (D / 2)) {
        float c, s;
        turn(pos ? pos[t] : first + t, f, c, s);
        cs[t * (D / 2) + p] = make_float2(c, s);
    }
}

template <int D, typename TI>
__global__ __launch_bounds__(256) void kv_append_kernel(KvCache c, KvBatch b, QkTransform f, const TI* q, int G,
                                                        int64_t q_stride, const TI* k, int64_t k_stride, const TI* v,
                                                        int64_t v_stride, const int32_t* pos, uint16_t* q_out,
                                                        int roles)
{
    constexpr int E = D / 32;
    __shared__ float2 cs[kKvBlock * D / 2];
    __shared__ uint32_t tops[2][4];
    // keys and values, with the most to do, start first (the prompt above takes
    // 40 us with a block's roles side by side)
    const uint32_t items = gridDim.x / roles, role = blockIdx.x / items, item = blockIdx.x - role * items;
    const int h = item % c.heads;
    KvSeq s;
    int64_t local;
    KvSpan w;
    if (!kv_find(b, item / c.heads, 1, kKvBlock, 2, s, local) || !kv_span(s, local, w)) return;
    const int j = threadIdx.x & 15, grp = threadIdx.x >> 4;
    const int at = w.block * kKvBlock + w.slot;                    // position of the first token
    const bool inter = f.interleaved != 0;

    // K and V: group grp has slots grp, grp + 16, grp + 32, grp + 48 of the
    // block, so a wave's four groups are four tokens whose V codes share words
    const int o = w.slot, end = o + w.n;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, quad = lane >> 4;
    // whether any of the wave's four slots 16 r + 4 wave .. + 3 is new
    const auto busy = [&](int r) { return 16 * r + 4 * wave + 3 >= o && 16 * r + 4 * wave < end; };
    const int64_t phys = role == 0 ? kv_block(b, c, s.i, w.block) : -1;
    float* const scales = c.scales + (phys * c.heads + h) * 2;
    float xk[4][2 * E], xv[4][2 * E], old_k = 0.0f, old_v = 0.0f;
    if (phys >= 0) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (!busy(r)) continue;
            const int t = 16 * r + grp - o;
            if (t < 0 || t >= w.n) continue;
            const TI* ks = k + (w.row + t) * k_stride + (int64_t)h * D;
            const TI* vs = v + (w.row + t) * v_stride + (int64_t)h * D;
            load_run<E>(ks + E * j, xk[r]);
            load_run<E>(ks + D / 2 + E * j, xk[r] + E);
            load_run<E>(vs + E * j, xv[r]);
            load_run<E>(vs + D / 2 + E * j, xv[r] + E);
        }
        if (o) {
            old_k = scales[0];
            old_v = scales[1];
        }
    }

    // queries: tokens [from, from + nt) of the block's rows, heads [qh, qh + qn)
    // of each: G heads of all tokens, or in prompts all heads of a slice of the
    // tokens, so that their angles are computed once for all query heads
    const bool sliced = roles > 2;
    const int slices = sliced ? (roles - 1) * c.heads : 1, slice = sliced ? h * (roles - 1) + (int)role - 1 : 0;
    const int from = role > 0 ? w.n * slice / slices : 0;
    const int nt = (role > 0 ? w.n * (slice + 1) / slices : w.n) - from;
    const int qh = sliced ? 0 : h * G, qn = sliced ? G * c.heads : G;
    const int count = role > 0 || roles == 1 ? nt * qn : 0;
    const int64_t row = w.row + from;
    const auto query = [&](int i, auto use) {
        const int t = i / qn;
        const int64_t hq = qh + i - t * qn;
        use(t, q + (row + t) * q_stride + hq * D, q_out + ((row + t) * ((int64_t)c.heads * G) + hq) * D);
    };
    float x[4][2 * E];
    const auto load_queries = [&](int base) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (base + 16 * r + grp < count)
                query(base + 16 * r + grp, [&](int, const TI* src, uint16_t*) {
                    load_run<E>(src + E * j, x[r]);
                    load_run<E>(src + D / 2 + E * j, x[r] + E);
                });
    };
    load_queries(0);
    if (f.inv_freq) {
        angles<D>(cs, nt, f.inv_freq, pos ? pos + row : nullptr, at + from);
        __syncthreads();
    }
    for (int base = 0; base < count; base += 64) {
        if (base) load_queries(base);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (base + 16 * r + grp < count)
                query(base + 16 * r + grp, [&](int t, const TI*, uint16_t* dst) {
                    if (f.q_gain) norm<D>(x[r], f.q_gain, f.eps, j);
                    if (f.inv_freq) rotate<D>(x[r], j, inter, [&](int p) { return cs[t * (D / 2) + p]; });
                    store_run<E>(dst + E * j, x[r]);
                    store_run<E>(dst + D / 2 + E * j, x[r] + E);
                });
    }
    if (phys < 0) return;

    uint32_t mk = 0, mv = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (!busy(r)) continue;
        const int t = 16 * r + grp - o;
        if (t < 0 || t >= w.n) continue;
        if (f.k_gain) norm<D>(xk[r], f.k_gain, f.eps, j);
        if (f.inv_freq) rotate<D>(xk[r], j, inter, [&](int p) { return cs[t * (D / 2) + p]; });
#pragma unroll
        for (int i = 0; i < 2 * E; ++i) {
            const uint32_t a = __builtin_bit_cast(uint32_t, xk[r][i]) & 0x7FFFFFFFu;
            const uint32_t e = __builtin_bit_cast(uint32_t, xv[r][i]) & 0x7FFFFFFFu;
            mk = a > mk ? a : mk;
            mv = e > mv ? e : mv;
        }
    }
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t a = __shfl_xor(mk, off), e = __shfl_xor(mv, off);
        mk = a > mk ? a : mk;
        mv = e > mv ? e : mv;
    }
    if (lane == 0) {
        tops[0][wave] = mk;
        tops[1][wave] = mv;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        mk = tops[0][i] > mk ? tops[0][i] : mk;
        mv = tops[1][i] > mv ? tops[1][i] : mv;
    }
    int shift_k, shift_v;
    const float sk = join_scale(old_k, mk, o == 0, shift_k), sv = join_scale(old_v, mv, o == 0, shift_v);
    if (threadIdx.x == 0) {
        scales[0] = sk;
        scales[1] = sv;
    }
    int8_t* kc = c.codes + (phys * c.heads + h) * 2 * (kKvBlock * D);
    int8_t* vc = kc + kKvBlock * D;
    // Old codes follow a doubled scale, 16 bytes a thread: K of one token, V of
    // one dim and 16 tokens.  No byte written here is written below.
    if (shift_k)
        for (int i = threadIdx.x; i < kKvBlock * D / 16; i += 256) {
            const int token = i / D * 16 + (i & 15);
            if (token >= o) continue;
            u32x4 x = *(const u32x4*)(kc + i * 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = shift_codes(x[e], shift_k);
            *(u32x4*)(kc + i * 16) = x;
        }
    if (shift_v)
        for (int i = threadIdx.x; i < kKvBlock * D / 16; i += 256) {
            const u32x4 x = *(const u32x4*)(vc + i * 16);
            const int g = i >> 4 & 3;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int old = o - (16 * e + 4 * g);              // tokens of this word that are old
                if (old > 0) store_bytes(vc + i * 16 + 4 * e, shift_codes(x[e], shift_v), old);
            }
        }
    // the new codes.  K: a lane's E dims of a token are neighbours.  V: four
    // lanes, 16 apart, have four tokens of the same dims; they exchange them
    // so that each has one dim of all four (a word), for all of a lane's four
    // slots a whole chunk of 16 bytes.
    constexpr int kWords = E == 4 ? 2 : 1;
    uint32_t vw[kWords][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (!busy(r)) continue;
        const int slot = 16 * r + grp;
        const bool mine = slot >= o && slot < end;
        uint32_t kq[2] = {0, 0}, vq[2] = {0, 0};
        if (mine) {
#pragma unroll
            for (int i = 0; i < 2 * E; ++i) {
                kq[i / E] |= quantise(xk[r][i], sk) << 8 * (i % E);
                vq[i / E] |= quantise(xv[r][i], sv) << 8 * (i % E);
            }
#pragma unroll
            for (int run = 0; run < 2; ++run) {
                int8_t* p = kc + kv_k_byte<D>(slot, run * (D / 2) + E * j);
                if constexpr (E == 4) *(uint32_t*)p = kq[run];
                else *(uint16_t*)p = (uint16_t)kq[run];
            }
        }
        if constexpr (E == 2) vq[0] |= vq[1] << 16;
#pragma unroll
        for (int n = 0; n < kWords; ++n) {
            // bytes are dims; after both exchanges lane `quad` has dim `quad`, bytes are tokens
            const uint32_t x = vq[n], y = __shfl_xor(x, 16);
            const uint32_t z = quad & 1 ? __builtin_amdgcn_perm(x, y, 0x07030501u)
                                        : __builtin_amdgcn_perm(y, x, 0x06020400u);
            const uint32_t u = __shfl_xor(z, 32);
            vw[n][r] = quad & 2 ? __builtin_amdgcn_perm(z, u, 0x07060302u) : __builtin_amdgcn_perm(u, z, 0x05040100u);
        }
    }
#pragma unroll
    for (int n = 0; n < kWords; ++n) {
        const int d = E == 4 ? n * (D / 2) + E * j + quad : (quad >> 1) * (D / 2) + E * j + (quad & 1);
        int8_t* p = vc + kv_v_byte(4 * wave, d);
        if (o == 0 && end == kKvBlock) {
            *(u32x4*)p = u32x4{vw[n][0], vw[n][1], vw[n][2], vw[n][3]};
            continue;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (!busy(r)) continue;
            const int slot = 16 * r + 4 * wave;
            if (slot >= o && slot + 4 <= end) {
                *(uint32_t*)(p + 4 * r) = vw[n][r];
            } else {
                for (int i = 0; i < 4; ++i)
                    if (slot + i >= o && slot + i < end) p[4 * r + i] = (int8_t)(vw[n][r] >> 8 * i);
            }
        }
    }
}

// ---- read ------------------------------------------------------------------
// One workgroup per (sequence, block, head); 16 bytes a thread.  A chunk of K
// is 16 dims of one token; a chunk of V is one dim of 16 tokens, and four
// neighbouring lanes exchange theirs so that each has four dims of four
// tokens.  Bound by what it writes: eight contexts of 2500 to 9000 tokens, 8
// heads of 128, to bf16 (254 MB, two thirds of them written) take 43 us, 5.9
// TB/s; 777 tokens 4.6 us.

// 4 N codes as values, in stores of 16 bytes where there are as many
template <int N, typename TO>
__device__ __forceinline__ void store_codes(TO* p, const uint32_t* w, float scale)
{
    constexpr int kAt = sizeof(TO) == 2 && N > 1 ? 8 : 4;
    float x[4 * N];
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) x[i] = (float)(int8_t)(w[i / 4] >> 8 * (i % 4)) * scale;
#pragma unroll
    for (int i = 0; i < 4 * N; i += kAt) store_run<kAt>(p + i, x + i);
}

template <int D, typename TO>
__global__ __launch_bounds__(256) void kv_read_kernel(KvCache c, KvBatch b, TO* k_out, TO* v_out)
{
    constexpr int S = D / 64;                                      // chunks of each side per thread
    const int h = blockIdx.x % c.heads;
    KvSeq s;
    int64_t local;
    KvSpan w;
    if (!kv_find(b, blockIdx.x / c.heads, 1, kKvBlock, 2, s, local) || !kv_span(s, local, w)) return;
    const int64_t phys = kv_block(b, c, s.i, w.block);
    const bool there = phys >= 0;
    const int64_t unit = (there ? phys : 0) * c.heads + h;
    const float sk = there ? c.scales[unit * 2] : 0.0f, sv = there ? c.scales[unit * 2 + 1] : 0.0f;
    const u32x4* kc = (const u32x4*)(c.codes + unit * 2 * (kKvBlock * D));
    const int64_t stride = (int64_t)c.heads * D;
    TO* const k_row = k_out + w.row * stride + (int64_t)h * D;     // of the block's slot w.slot
    TO* const v_row = v_out + w.row * stride + (int64_t)h * D;
    // K: a wave has 64 dims of 16 tokens; V: 64 dims of a quarter of the tokens
    // (16 t + 4 wave + i), so that either stores 64 dims of a row side by side
    const int wave = threadIdx.x >> 6, r = threadIdx.x & 15, quarter = threadIdx.x >> 4 & 3, quad = threadIdx.x & 3;
    u32x4 kx[S], vx[S];
#pragma unroll
    for (int n = 0; n < S; ++n) {
        kx[n] = vx[n] = u32x4{0, 0, 0, 0};
        if (there) {
            kx[n] = kc[threadIdx.x + 256 * n];
            vx[n] = kc[kKvBlock * D / 16 + ((4 * n + quarter) * 4 + wave) * 16 + r];
        }
    }
#pragma unroll
    for (int n = 0; n < S; ++n) {
        const int hi = wave + 4 * n, kt = hi / S * 16 + r - w.slot;
        if (kt >= 0 && kt < w.n) {
            const uint32_t x[4] = {kx[n][0], kx[n][1], kx[n][2], kx[n][3]};
            store_codes<4>(k_row + kt * stride + hi % S * 64 + quarter * 16, x, sk);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            // bytes are tokens; after both exchanges lane `quad` has token `quad`, bytes are dims
            const uint32_t x = vx[n][t], y = __shfl_xor(x, 1);
            const uint32_t z = quad & 1 ? __builtin_amdgcn_perm(x, y, 0x07030501u)
                                        : __builtin_amdgcn_perm(y, x, 0x06020400u);
            const uint32_t u = __shfl_xor(z, 2);
            const uint32_t word = quad & 2 ? __builtin_amdgcn_perm(z, u, 0x07060302u)
                                           : __builtin_amdgcn_perm(u, z, 0x05040100u);
            const int vt = 16 * t + 4 * wave + quad - w.slot;
            if (vt >= 0 && vt < w.n)
                store_codes<1>(v_row + vt * stride + (4 * n + quarter) * 16 + (r & ~3), &word, sv);
        }
    }
}

// ---- keep ------------------------------------------------------------------
// The accepted branch of a tree moves up: slot p0 + k takes the token of slot
// p0 + path[k].  One workgroup per (sequence, head, side).  The last 64 tokens of
// the path or fewer go to two blocks at most and are taken at once; while more
// follow, those of one block are, up to its end, so that every block is scaled
// once, by all tokens that come into it.  A path ascends, so they come from these
// blocks or from others behind, whose bytes are as they were: all tokens are in
// LDS before anything is written.
// A branch is a few tokens: bound by the launch and the chain from cu over the
// table to scales and codes.
template <int D>
__global__ __launch_bounds__(256) void kv_keep_kernel(KvCache c, KvBatch b, const int32_t* paths, int width,
                                                      int32_t* lens_out)
{
    __shared__ __align__(16) int8_t code[kKvBlock][D];
    __shared__ int64_t from[kKvBlock];                 // unit (block and head) of a token's source, -1: none
    __shared__ float its[kKvBlock];                    // the source's scale
    __shared__ int slot[kKvBlock];
    __shared__ int tokens, more;
    __shared__ int64_t place[2];                       // the units that tokens go to, -1: none, or nothing moves
    __shared__ uint32_t tops[2][4];
    const int side = blockIdx.x & 1, h = (blockIdx.x >> 1) % c.heads, i = (blockIdx.x >> 1) / c.heads;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int32_t* path = paths + (int64_t)i * width;
    int r = wave == 0 && lane < width ? path[lane] : -1;
    KvSeq s;
    const bool any = kv_seq(b, i, s);
    const int rows = any ? (s.n < kTreeRows ? s.n : kTreeRows) : 0, most = width < rows ? width : rows;
    int kept = 0;
    for (int k0 = 0; k0 < most;) {
        const int base = (s.p0 + k0) & 63;
        if (wave == 0) {
            const int k = k0 + lane;
            if (k0 > 0) r = k < most ? path[k] : -1;
            int before = __shfl(r, lane - 1);
            if (lane == 0) before = k0 > 0 ? path[k0 - 1] : -1;
            const uint64_t end = __ballot(!(k < most && r > before && r >= 0 && r < rows));
            const bool on = end == 0 && k0 + kKvBlock < most;
            const int n = on ? kKvBlock - base : end ? __builtin_ctzll(end) : kKvBlock;
            const bool mine = lane < n;
            // tokens in front of position 0 are not there (their block is below 0)
            const int p = s.p0 + r, source = mine ? kv_block(b, c, s.i, p >> 6) : -1;
            const int to = mine ? kv_block(b, c, s.i, (s.p0 + k) >> 6) : -1, second = base + lane >= kKvBlock;
            const int64_t unit = (int64_t)source * c.heads + h;
            from[lane] = source < 0 ? -1 : unit;
            its[lane] = source >= 0 ? c.scales[unit * 2 + side] : 0.0f;
            slot[lane] = p & 63;
            const bool moves = mine && r != k && source >= 0 && to >= 0;
            const uint64_t m0 = __ballot(moves && !second), m1 = __ballot(moves && second);
            if (lane == 0) {
                tokens = n;
                more = on;
                place[0] = place[1] = -1;
            }
            __builtin_amdgcn_wave_barrier();
            if (mine && to >= 0 && (second ? m1 : m0)) place[second] = (int64_t)to * c.heads + h;
        }
        __syncthreads();
        const int n = tokens;
        const bool on = more;
        kept += n;
        k0 += n;
        const int64_t unit[2] = {place[0], place[1]};
        if (unit[0] >= 0 || unit[1] >= 0) {
            const float before[2] = {unit[0] >= 0 ? c.scales[unit[0] * 2 + side] : 0.0f,
                                     unit[1] >= 0 ? c.scales[unit[1] * 2 + side] : 0.0f};
            // the tokens to LDS, and the largest value that comes from another block
            uint32_t top[2] = {0, 0};
            const auto sized = [&](int t, int largest) {
                const int w = base + t >= kKvBlock;
                if (from[t] != unit[w]) {
                    // of a scale that is not finite, itself (not 0 times it)
                    const float scale = fabsf(its[t]), value = scale < INFINITY ? (float)largest * scale : scale;
                    const uint32_t x = __builtin_bit_cast(uint32_t, value);
                    top[0] = w == 0 && x > top[0] ? x : top[0];
                    top[1] = w == 1 && x > top[1] ? x : top[1];
                }
            };
            if (side == 0) {
                for (int e = threadIdx.x; e < n * (D / 16); e += 256) {
                    const int t = e / (D / 16), d = e % (D / 16) * 16;
                    if (from[t] < 0) continue;
                    const u32x4 x = *(const u32x4*)(c.codes + from[t] * 2 * (kKvBlock * D) + kv_k_byte<D>(slot[t], d));
                    *(u32x4*)&code[t][d] = x;
                    int largest = 0;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int v = (int8_t)(x[j >> 2] >> 8 * (j & 3));
                        largest = v > largest ? v : -v > largest ? -v : largest;
                    }
                    sized(t, largest);
                }
            } else {
                // eight bytes a thread under way: a branch of 16 tokens waits once
                for (int e0 = threadIdx.x; e0 < n * D; e0 += 256 * 8) {
                    int8_t x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int e = e0 + 256 * j < n * D ? e0 + 256 * j : e0, t = e / D;
                        const int64_t of = from[t] < 0 ? 0 : from[t];
                        x[j] = c.codes[(of * 2 + 1) * (kKvBlock * D) + kv_v_byte(slot[t], e % D)];
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int e = e0 + 256 * j, t = e / D;
                        if (e >= n * D || from[t] < 0) continue;
                        code[t][e % D] = x[j];
                        sized(t, x[j] < 0 ? -x[j] : x[j]);
                    }
                }
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                for (int off = 1; off < 64; off <<= 1) {
                    const uint32_t x = __shfl_xor(top[w], off);
                    top[w] = x > top[w] ? x : top[w];
                }
                if (lane == 0) tops[w][wave] = top[w];
            }
            __syncthreads();                           // code and tops are there, the old scales read
            float scale[2];
            int shift[2];
#pragma unroll
            for (int w = 0; w < 2; ++w) {
#pragma unroll
                for (int v = 0; v < 4; ++v) top[w] = tops[w][v] > top[w] ? tops[w][v] : top[w];
                scale[w] = before[w];
                shift[w] = 0;
                if (unit[w] < 0 || top[w] == 0) continue;
                scale[w] = join_scale(before[w], top[w], false, shift[w]);
                if (before[w] == 0.0f) shift[w] = 31;
                if (threadIdx.x == 0) c.scales[unit[w] * 2 + side] = scale[w];
            }
            if (shift[0] || shift[1]) {                // every code follows a doubled scale, 16 bytes a thread
#pragma unroll 1
                for (int w = 0; w < 2; ++w) {
                    const int by = w ? shift[1] : shift[0];
                    int8_t* const codes = c.codes + ((w ? unit[1] : unit[0]) * 2 + side) * (kKvBlock * D);
                    if (by)
#pragma unroll 1
                        for (int e = threadIdx.x; e < kKvBlock * D / 16; e += 256) {
                            u32x4 x = *(const u32x4*)(codes + 16 * e);
#pragma unroll
                            for (int j = 0; j < 4; ++j) x[j] = shift_codes(x[j], by);
                            *(u32x4*)(codes + 16 * e) = x;
                        }
                }
                __syncthreads();                       // before the tokens are written over them
            }
            // tokens at their places: K 16 dims a thread, V one
            const int per = side == 0 ? D / 16 : D;
#pragma unroll 1
            for (int e = threadIdx.x; e < n * per; e += 256) {
                const int t = e / per, d = e % per, w = base + t >= kKvBlock, at = (base + t) & 63;
                const int64_t of = from[t], to = w ? unit[1] : unit[0];
                if (of < 0 || to < 0) continue;
                const bool far = of != to;
                const float by = its[t], sc = w ? scale[1] : scale[0];
                const int sh = w ? shift[1] : shift[0];
                int8_t* const codes = c.codes + (to * 2 + side) * (kKvBlock * D);
                if (side == 0) {
                    u32x4 x = *(const u32x4*)&code[t][16 * d];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (far) {
                            uint32_t y = 0;
#pragma unroll
                            for (int q = 0; q < 4; ++q) y |= quantise((float)(int8_t)(x[j] >> 8 * q) * by, sc) << 8 * q;
                            x[j] = y;
                        } else if (sh) {
                            x[j] = shift_codes(x[j], sh);
                        }
                    }
                    *(u32x4*)(codes + kv_k_byte<D>(at, 16 * d)) = x;
                } else {
                    uint32_t x = (uint8_t)code[t][d];
                    if (far) x = quantise((float)(int8_t)x * by, sc);
                    else if (sh) x = shift_codes(x, sh);
                    codes[kv_v_byte(at, d)] = (int8_t)x;
                }
            }
        }
        if (!on) break;
        __syncthreads();                               // LDS is used again
    }
    if (lens_out && side == 0 && h == 0 && threadIdx.x == 0) {
        const int len = s.p0 + kept;                   // without rows: the length as it is
        lens_out[i] = len > 0 ? len : 0;
    }
}

// ---- launchers -------------------------------------------------------------
template <int D, typename TI, typename TO>
static hipError_t norm_rope(const QkTransform& f, int64_t T, const void* q, int64_t Hq, int64_t q_stride,
                            const void* k, int64_t Hk, int64_t k_stride, const int32_t* pos, void* q_out,
                            void* k_out, hipStream_t stream)
{
    const int parts = (int)((Hq + Hk + 15) / 16);
    norm_rope_kernel<D, TI, TO><<<(unsigned)(T * parts), 256, 0, stream>>>(
        f, (const TI*)q, (int)Hq, q_stride, (const TI*)k, (int)Hk, k_stride, pos, (TO*)q_out, (TO*)k_out, parts);
    return hipGetLastError();
}

hipError_t launch_qk_norm_rope(const QkTransform& f, int64_t T, int64_t D, const void* q, int64_t Hq,
                               int64_t q_stride, const void* k, int64_t Hk, int64_t k_stride, bool in_bf16,
                               const int32_t* pos, void* q_out, void* k_out, bool out_bf16, hipStream_t stream)
{
#define TERN_NR(DD, TI, TO) \
    norm_rope<DD, TI, TO>(f, T, q, Hq, q_stride, k, Hk, k_stride, pos, q_out, k_out, stream)
    if (D == 128)
        return in_bf16 ? (out_bf16 ? TERN_NR(128, uint16_t, uint16_t) : TERN_NR(128, uint16_t, float))
                       : (out_bf16 ? TERN_NR(128, float, uint16_t) : TERN_NR(128, float, float));
    return in_bf16 ? (out_bf16 ? TERN_NR(64, uint16_t, uint16_t) : TERN_NR(64, uint16_t, float))
                   : (out_bf16 ? TERN_NR(64, float, uint16_t) : TERN_NR(64, float, float));
#undef TERN_NR
}

// workgroups of the append and the read: every sequence's touched blocks, for each head
static unsigned block_items(const KvCache& c, const KvBatch& b)
{
    return (unsigned)(((int64_t)b.T / kKvBlock + 2 * (int64_t)b.nseq) * c.heads);
}

hipError_t launch_kv_append(const KvCache& c, const KvBatch& b, int64_t D, const QkTransform& f, const void* q,
                            int64_t Hq, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, bool in_bf16, const int32_t* pos, uint16_t* q_out, hipStream_t stream)
{
    const int G = (int)(Hq / c.heads);
    // Workgroups for a block and head: one for K and V and four for the queries
    // in prompts, one and one for few streams, else one for all.  Calls one
    // behind another in a graph, 32:8 heads of 128 (one for all / one and one /
    // one and four, us):
    //   4131 rows of two sequences  46.0 / 46.1 / 36.2    16 x 16 rows  9.5 /  7.2 /  7.1
    //   1 token  5.9 / 5.7 / 5.7    16 streams  6.3 / 6.1 / 6.4    24  6.5 /  6.3 /  9.2
    //   48 streams  7.2 / 9.0 / 14.2    128  15.9 / 18.6 / 33.9    64 x 8 rows  10.0 / 11.8 / 16.0
    const int roles = G == 0 ? 1 : (int64_t)b.T >= 16 * (int64_t)b.nseq ? kKvRoles : block_items(c, b) <= 256 ? 2 : 1;
#define TERN_AP(DD, TI)                                                                                      \
    kv_append_kernel<DD, TI><<<block_items(c, b) * roles, 256, 0, stream>>>(                                 \
        c, b, f, (const TI*)q, G, q_stride, (const TI*)k, k_stride, (const TI*)v, v_stride, pos, q_out, roles)
    if (D == 128) {
        if (in_bf16) TERN_AP(128, uint16_t);
        else TERN_AP(128, float);
    } else {
        if (in_bf16) TERN_AP(64, uint16_t);
        else TERN_AP(64, float);
    }
#undef TERN_AP
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvCache& c, const KvBatch& b, int64_t D, void* k_out, void* v_out, bool out_bf16,
                          hipStream_t stream)
{
#define TERN_RD(DD, TO) kv_read_kernel<DD, TO><<<block_items(c, b), 256, 0, stream>>>(c, b, (TO*)k_out, (TO*)v_out)
    if (D == 128) {
        if (out_bf16) TERN_RD(128, uint16_t);
        else TERN_RD(128, float);
    } else {
        if (out_bf16) TERN_RD(64, uint16_t);
        else TERN_RD(64, float);
    }
#undef TERN_RD
    return hipGetLastError();
}

hipError_t launch_kv_keep(const KvCache& c, const KvBatch& b, int64_t D, const int32_t* path, int width,
                          int32_t* lens_out, hipStream_t stream)
{
    const unsigned grid = (unsigned)((int64_t)b.nseq * c.heads * 2);
    if (D == 128) kv_keep_kernel<128><<<grid, 256, 0, stream>>>(c, b, path, width, lens_out);
    else kv_keep_kernel<64><<<grid, 256, 0, stream>>>(c, b, path, width, lens_out);
    return hipGetLastError();
}

}  // namespace tern
