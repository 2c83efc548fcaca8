// tern_attend.hip — attention over the paged int8 cache.
//
//   out = sum_p w_p V[p] / sum_p w_p,  w_p = exp(scale * q . K[p])
//
// One wave per row and query head walks the row's blocks of 64 tokens with a
// running maximum and sum: lane = token for the scores, lane = dim for the
// values.
#include "tern_device.h"
#include "tern_kv.h"
#include "tern_launch.h"

namespace tern {

template <int D>
__global__ __launch_bounds__(64) void kv_attend_kernel(KvCache c, KvBatch b, const uint16_t* q, int Hq,
                                                       int64_t q_stride, float scale, int64_t window, uint16_t* out)
{
    __shared__ float qs[D], ps[64];
    const int64_t t = blockIdx.x / Hq;
    const int hq = blockIdx.x % Hq, h = hq / (Hq / c.heads), lane = threadIdx.x;
    KvSeq s;
    int64_t local;
    if (!kv_find(b, t, 1, 1, 0, s, local) || local >= s.n) return;
    const int64_t pos = s.p0 + local;
    for (int d = lane; d < D; d += 64) qs[d] = bf16_to_f32(q[t * q_stride + (int64_t)hq * D + d]);
    __syncthreads();
    float m = -INFINITY, l = 0.0f, acc[D / 64] = {};
    const int64_t first = window > 0 && pos - window + 1 > 0 ? pos - window + 1 : 0;
    int64_t last = b.table_width * kKvBlock - 1;
    if (pos < last) last = pos;
    for (int64_t blk = first / kKvBlock; blk * kKvBlock <= last; ++blk) {
        const int64_t phys = kv_block(b, c, s.i, blk);
        if (phys < 0) continue;
        const float* scales = c.scales + (phys * c.heads + h) * 2;
        const int8_t* kc = c.codes + (phys * c.heads + h) * 2 * (kKvBlock * D);
        const int8_t* vc = kc + kKvBlock * D;
        const int64_t at = blk * kKvBlock + lane;
        float dot = 0.0f;
        for (int d = 0; d < D; ++d) dot = fmaf(qs[d], (float)kc[kv_k_byte<D>(lane, d)], dot);
        const bool seen = at >= first && at <= last;
        const float x = seen ? dot * (scales[0] * scale) : -INFINITY;
        float top = x;
        for (int off = 32; off; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
        const float mn = fmaxf(m, top);
        if (mn == -INFINITY && !__any(seen && x != x)) continue;
        const float p = seen ? expf(x - mn) : 0.0f;
        const float keep = m == -INFINITY ? 0.0f : expf(m - mn);
        float sum = p;
        for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off);
        l = l * keep + sum;
        m = mn;
        ps[lane] = p;
        __syncthreads();
        const int from = (int)(first > blk * kKvBlock ? first - blk * kKvBlock : 0);
        const int upto = (int)(last < blk * kKvBlock + 63 ? last - blk * kKvBlock : 63);
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
            float part = 0.0f;
            for (int i = from; i <= upto; ++i) part = fmaf(ps[i], (float)vc[kv_v_byte(i, u * 64 + lane)], part);
            acc[u] = acc[u] * keep + part * scales[1];
        }
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < D / 64; ++u)
        out[(t * Hq + hq) * D + u * 64 + lane] = f32_to_bf16(l == 0.0f ? 0.0f : acc[u] / l);
}

int64_t kv_attend_workspace_bytes(int64_t T, int64_t Hq, int64_t heads, int64_t D, int64_t nseq, int64_t max_len)
{
    return 0;
}

hipError_t launch_kv_attend(const KvCache& c, const KvBatch& b, int64_t D, const uint16_t* q, int64_t Hq,
                            int64_t q_stride, float scale, int64_t window, int64_t max_len, uint16_t* out,
                            void* workspace, hipStream_t stream)
{
    const unsigned grid = (unsigned)((int64_t)b.T * Hq);
    if (D == 128)
        kv_attend_kernel<128><<<grid, 64, 0, stream>>>(c, b, q, (int)Hq, q_stride, scale, window, out);
    else
        kv_attend_kernel<64><<<grid, 64, 0, stream>>>(c, b, q, (int)Hq, q_stride, scale, window, out);
    return hipGetLastError();
}

}  // namespace tern
