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
// once per workgroup.
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
// One workgroup per (sequence, touched block, key/value head): the block's
// scale needs the maximum over all its new tokens, and nothing else writes
// the block.  Up to four K and four V vectors of each 16-lane group stay in
// registers from the maximum to the quantisation.

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

__device__ __forceinline__ int quantise(float x, float scale)
{
    if (!(scale > 0.0f && scale < INFINITY)) return 0;
    return (int)fminf(fmaxf(__builtin_rintf(__fdiv_rn(x, scale)), -127.0f), 127.0f);
}

// rint(code / 2^shift)
__device__ __forceinline__ uint32_t shift_code(uint32_t byte, int shift)
{
    const float c = (float)(int8_t)byte;
    return shift >= 9 ? 0u : (uint32_t)(int)__builtin_rintf(ldexpf(c, -shift)) & 0xFFu;
}

template <int D, typename TI>
__global__ __launch_bounds__(256) void kv_append_kernel(KvCache c, KvBatch b, QkTransform f, const TI* q, int G,
                                                        int64_t q_stride, const TI* k, int64_t k_stride, const TI* v,
                                                        int64_t v_stride, const int32_t* pos, uint16_t* q_out)
{
    constexpr int E = D / 32;
    __shared__ float2 cs[kKvBlock * D / 2];
    __shared__ uint32_t top[2];
    const int h = blockIdx.x % c.heads;
    KvSeq s;
    int64_t local;
    if (!kv_find(b, blockIdx.x / c.heads, 1, kKvBlock, 2, s, local)) return;
    KvSpan w;
    if (!kv_span(s, local, w)) return;
    const int nt = w.n, o = w.slot;
    const int64_t t0 = w.row;
    const int64_t phys = kv_block(b, c, s.i, w.block);

    if (threadIdx.x < 2) top[threadIdx.x] = 0;
    if (f.inv_freq)
        for (int i = threadIdx.x; i < nt * (D / 2); i += 256) {
            const int t = i / (D / 2), p = i % (D / 2);
            float cc, ss;
            turn(pos ? pos[t0 + t] : w.block * kKvBlock + o + t, f.inv_freq[p], cc, ss);
            cs[i] = make_float2(cc, ss);
        }
    __syncthreads();
    const int j = threadIdx.x & 15, grp = threadIdx.x >> 4;

    // queries: G heads of every token
    for (int i = grp; i < nt * G; i += 16) {
        const int t = i / G;
        const int64_t head = (int64_t)h * G + i % G;
        const TI* src = q + (t0 + t) * q_stride + head * D;
        float x[2 * E];
        load_run<E>(src + E * j, x);
        load_run<E>(src + D / 2 + E * j, x + E);
        if (f.q_gain) norm<D>(x, f.q_gain, f.eps, j);
        if (f.inv_freq) rotate<D>(x, j, f.interleaved != 0, [&](int p) { return cs[t * (D / 2) + p]; });
        uint16_t* dst = q_out + ((t0 + t) * ((int64_t)c.heads * G) + head) * D;
        store_run<E>(dst + E * j, x);
        store_run<E>(dst + D / 2 + E * j, x + E);
    }
    if (phys < 0) return;

    float xk[4][2 * E], xv[4][2 * E];
    uint32_t mk = 0, mv = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int t = grp + 16 * r;
        if (t >= nt) break;
        const TI* ks = k + (t0 + t) * k_stride + (int64_t)h * D;
        const TI* vs = v + (t0 + t) * v_stride + (int64_t)h * D;
        load_run<E>(ks + E * j, xk[r]);
        load_run<E>(ks + D / 2 + E * j, xk[r] + E);
        load_run<E>(vs + E * j, xv[r]);
        load_run<E>(vs + D / 2 + E * j, xv[r] + E);
        if (f.k_gain) norm<D>(xk[r], f.k_gain, f.eps, j);
        if (f.inv_freq) rotate<D>(xk[r], j, f.interleaved != 0, [&](int p) { return cs[t * (D / 2) + p]; });
#pragma unroll
        for (int i = 0; i < 2 * E; ++i) {
            const uint32_t a = __builtin_bit_cast(uint32_t, xk[r][i]) & 0x7FFFFFFFu;
            const uint32_t e = __builtin_bit_cast(uint32_t, xv[r][i]) & 0x7FFFFFFFu;
            mk = a > mk ? a : mk;
            mv = e > mv ? e : mv;
        }
    }
    float* scales = c.scales + (phys * c.heads + h) * 2;
    const float old_k = o ? scales[0] : 0.0f, old_v = o ? scales[1] : 0.0f;
    if (mk) atomicMax(&top[0], mk);
    if (mv) atomicMax(&top[1], mv);
    __syncthreads();
    int shift_k, shift_v;
    const float sk = join_scale(old_k, top[0], o == 0, shift_k), sv = join_scale(old_v, top[1], o == 0, shift_v);
    if (threadIdx.x == 0) {
        scales[0] = sk;
        scales[1] = sv;
    }
    int8_t* kc = c.codes + (phys * c.heads + h) * 2 * (kKvBlock * D);
    int8_t* vc = kc + kKvBlock * D;
    // old codes follow the doubled scale; a byte is changed by one thread here
    // and never by the stores of new tokens below
    if (shift_k)
        for (int i = threadIdx.x; i < o * D; i += 256) {
            int8_t* p = kc + kv_k_byte<D>(i / D, i % D);
            *p = (int8_t)shift_code((uint8_t)*p, shift_k);
        }
    if (shift_v)
        for (int i = threadIdx.x; i < o * D; i += 256) {
            int8_t* p = vc + kv_v_byte(i / D, i % D);
            *p = (int8_t)shift_code((uint8_t)*p, shift_v);
        }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int t = grp + 16 * r;
        if (t >= nt) break;
#pragma unroll
        for (int run = 0; run < 2; ++run) {
            const int d = run * (D / 2) + E * j;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                kc[kv_k_byte<D>(o + t, d + i)] = (int8_t)quantise(xk[r][run * E + i], sk);
                vc[kv_v_byte(o + t, d + i)] = (int8_t)quantise(xv[r][run * E + i], sv);
            }
        }
    }
}

// ---- read ------------------------------------------------------------------
template <int D, typename TO>
__global__ __launch_bounds__(256) void kv_read_kernel(KvCache c, KvBatch b, TO* k_out, TO* v_out)
{
    const int h = blockIdx.x % c.heads;
    KvSeq s;
    int64_t local;
    if (!kv_find(b, blockIdx.x / c.heads, 1, kKvBlock, 2, s, local)) return;
    KvSpan w;
    if (!kv_span(s, local, w)) return;
    const int nt = w.n, o = w.slot;
    const int64_t t0 = w.row;
    const int64_t phys = kv_block(b, c, s.i, w.block);
    const float* scales = c.scales + (phys * c.heads + h) * 2;
    const int8_t* kc = c.codes + (phys * c.heads + h) * 2 * (kKvBlock * D);
    const int8_t* vc = kc + kKvBlock * D;
    for (int i = threadIdx.x; i < nt * D; i += 256) {
        const int t = i / D, d = i % D;
        float kx = 0.0f, vx = 0.0f;
        if (phys >= 0) {
            kx = (float)kc[kv_k_byte<D>(o + t, d)] * scales[0];
            vx = (float)vc[kv_v_byte(o + t, d)] * scales[1];
        }
        const int64_t at = ((t0 + t) * c.heads + h) * D + d;
        store_run<1>(k_out + at, &kx);
        store_run<1>(v_out + at, &vx);
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
#define TERN_AP(DD, TI)                                                                                      \
    kv_append_kernel<DD, TI><<<block_items(c, b), 256, 0, stream>>>(c, b, f, (const TI*)q, G, q_stride,      \
                                                                    (const TI*)k, k_stride, (const TI*)v,    \
                                                                    v_stride, pos, q_out)
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

}  // namespace tern
