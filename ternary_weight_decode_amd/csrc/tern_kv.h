// tern_kv.h — the paged int8 key/value cache: layout, batch lookup and the
// arguments that the append, read and attention kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tern {

constexpr int kKvBlock = 64;   // tokens per cache block: one scale for each block, head and side
constexpr int kKvRoles = 5;    // workgroups of an append for each touched block and head, at most

struct KvCache {
    int8_t* codes;             // [blocks][heads][2][64*D]
    float* scales;             // [blocks][heads][2]
    int64_t blocks;
    int heads;
};

struct KvBatch {
    const int32_t* cu;
    const int32_t* lens;
    const int32_t* table;
    int nseq;
    int table_width;           // at most 2^31 / 64: positions are 32-bit
    int64_t table_stride;
    int T;                     // rows of the per-token tensors
};

struct QkTransform {
    const float* q_gain;
    const float* k_gain;
    const double* inv_freq;
    float eps;
    int interleaved;
};

// byte of a code inside its (block, head, side): the order of include/tern.h
template <int D>
__device__ __forceinline__ int kv_k_byte(int token, int d)
{
    return ((((token >> 4) * (D / 64) + (d >> 6)) * 4 + ((d >> 4) & 3)) * 16 + (token & 15)) * 16 + (d & 15);
}

__device__ __forceinline__ int kv_v_byte(int token, int d)
{
    return (((d >> 4) * 4 + ((token >> 2) & 3)) * 16 + (d & 15)) * 16 + ((token >> 4) << 2) + (token & 3);
}

// One sequence of a batch: its rows [t0, t0 + n) and the position of row t0.
struct KvSeq {
    int i, t0, n, p0;
};

// a negative length is one of 0
__device__ __forceinline__ int kv_length(const KvBatch& b, int i) { return b.lens[i] > 0 ? b.lens[i] : 0; }

// Work items of a batch whose row counts only the device knows: sequence i
// owns the items from cu[i] * mul / div + i * extra on, which leaves it at
// least ceil(n * mul / div) + extra - 1 items (floor(a + b) - floor(a) >=
// floor(b)).  Finds the owner of `item` and the item's number inside it; all
// lanes of a wave call it together (64 entries of cu at a time, so the lookup
// is one load's latency for up to 64 sequences).  False: no such sequence, or
// rows outside the tensors.  Sequences from the first descent of cu on own
// nothing: an item of theirs falls to the one in front, past its end.
__device__ __forceinline__ bool kv_find(const KvBatch& b, int64_t item, int mul, int div, int extra, KvSeq& s,
                                        int64_t& local)
{
    const int lane = threadIdx.x & 63;
    int owners = 0, cu0 = 0, cu1 = 0, len = 0;
    for (int c = 0; c < b.nseq; c += 64) {
        const int i = c + lane < b.nseq ? c + lane : b.nseq - 1;
        const int r0 = b.cu[i], r1 = b.cu[i + 1], r2 = kv_length(b, i);
        const bool in = c + lane < b.nseq && r1 >= r0 && (int64_t)r0 * mul / div + (int64_t)i * extra <= item;
        const uint64_t out = ~__ballot(in);
        const int got = out ? __builtin_ctzll(out) : 64;
        if (got == 0) break;
        owners += got;
        cu0 = __builtin_amdgcn_readlane(r0, got - 1);
        cu1 = __builtin_amdgcn_readlane(r1, got - 1);
        len = __builtin_amdgcn_readlane(r2, got - 1);
        if (got < 64) break;
    }
    if (owners == 0) return false;
    s.i = owners - 1;
    s.t0 = cu0;
    s.n = cu1 - cu0;
    if (s.t0 < 0 || cu1 > b.T || s.n <= 0) return false;
    s.p0 = len - s.n;
    local = item - ((int64_t)s.t0 * mul / div + (int64_t)s.i * extra);
    return local >= 0;
}

// Physical block of a sequence's block, -1 where there is none.
__device__ __forceinline__ int kv_block(const KvBatch& b, const KvCache& c, int seq, int block)
{
    if (block < 0 || block >= b.table_width) return -1;
    const int phys = b.table[(int64_t)seq * b.table_stride + block];
    return phys >= 0 && phys < c.blocks ? phys : -1;
}

// The rows of a sequence that fall into its `local`-th touched block.
struct KvSpan {
    int block;                 // the block's number in the sequence, below 0 in front of it
    int slot, n;               // first slot, rows
    int64_t row;               // first row
};

__device__ __forceinline__ bool kv_span(const KvSeq& s, int64_t local, KvSpan& w)
{
    const int64_t block = (s.p0 >> 6) + local;                     // floor: p0 may be negative
    const int64_t from = block * kKvBlock, end = (int64_t)s.p0 + s.n;
    const int64_t lo = s.p0 > from ? s.p0 : from, hi = end < from + kKvBlock ? end : from + kKvBlock;
    if (lo >= hi) return false;
    w.block = (int)block;
    w.slot = (int)(lo - from);
    w.n = (int)(hi - lo);
    w.row = s.t0 + (lo - s.p0);
    return true;
}

__device__ __forceinline__ float bf16_to_f32(uint16_t h) { return __builtin_bit_cast(float, (uint32_t)h << 16); }

// nearest-even, NaN kept
__device__ __forceinline__ uint16_t f32_to_bf16(float f)
{
    return __builtin_bit_cast(uint16_t, (__bf16)f);
}

}  // namespace tern
