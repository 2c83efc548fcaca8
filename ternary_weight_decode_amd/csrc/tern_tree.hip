// tern_tree.hip — trees of drafted tokens: who descends from whom, and the
// branch that the target's own tokens take.
//
// Both calls read a few bytes a row and are bound by their launch and one chain
// of dependent loads (cu, then the rows); the walks themselves run in LDS.  One
// workgroup per sequence.
#include "tern_device.h"
#include "tern_kv.h"
#include "tern_launch.h"

namespace tern {

// parent of row r as the calls take it: an earlier row, or -1
__device__ __forceinline__ int tree_parent(int p, int r) { return p >= 0 && p < r ? p : -1; }

// mask[r] = mask[parent[r]] | 1 << r.  Every row walks up its branch, a load
// from LDS a step, which ends a tree of ordinary depth; the bits go to LDS on the
// side.  From there on by doubling, for chains: a row's mask holds the branch from
// the row down to before `jump`, and takes in that row's mask and jump.  A mask
// that is read while its owner adds to it holds rows of the branch either way;
// the jumps change between barriers.  (48 trees of up to 512 rows 20 deep: by
// doubling alone 8.7 us.)  One thread per row of 64 * words.
constexpr int kTreeWalk = 24;

__global__ __launch_bounds__(kTreeRows) void tree_mask_kernel(KvBatch b, const int32_t* parent, int words,
                                                              uint64_t* mask, int32_t* pos)
{
    __shared__ uint64_t rows[kTreeRows][kTreeWords + 1];
    __shared__ int jump[kTreeRows];
    KvSeq s;
    if (!kv_seq(b, blockIdx.x, s)) return;
    const int r = threadIdx.x, n = s.n < 64 * words ? s.n : 64 * words;
    int j = r < n ? tree_parent(parent[s.t0 + r], r) : -1;
#pragma unroll
    for (int w = 0; w < kTreeWords; ++w)
        if (w < words) rows[r][w] = r < n && w == r >> 6 ? 1ull << (r & 63) : 0;
    jump[r] = j;
    __syncthreads();
    for (int k = 0; k < kTreeWalk && __any(j >= 0); ++k)
        if (j >= 0) {
            atomicOr((unsigned long long*)&rows[r][j >> 6], 1ull << (j & 63));
            j = jump[j];
        }
    while (__syncthreads_or(j >= 0)) {
        jump[r] = j;
        __syncthreads();
        int next = -1;
        uint64_t m[kTreeWords];
        if (j >= 0) {
            next = jump[j];
#pragma unroll
            for (int w = 0; w < kTreeWords; ++w)
                if (w < words) m[w] = rows[j][w];
#pragma unroll
            for (int w = 0; w < kTreeWords; ++w)
                if (w < words) rows[r][w] |= m[w];
        }
        j = next;
    }
    int depth = -1;
#pragma unroll
    for (int w = 0; w < kTreeWords; ++w) {
        if (w >= words || r >= n) continue;
        const uint64_t m = rows[r][w];
        mask[(int64_t)(s.t0 + r) * words + w] = m;
        depth += __popcll(m);
    }
    if (pos && r < n) pos[s.t0 + r] = s.p0 + depth;
    // rows that no mask has a bit for
    for (int k = 64 * words + r; k < s.n; k += 64 * words) {
        for (int w = 0; w < words; ++w) mask[(int64_t)(s.t0 + k) * words + w] = 0;
        if (pos) pos[s.t0 + k] = s.p0 + k;
    }
}

// A wave walks one tree: every lane holds rows lane, lane + 64, ... and says
// whether they continue the current row with the target's token.
__global__ __launch_bounds__(64) void tree_accept_kernel(KvBatch b, const int32_t* parent, const int32_t* token,
                                                         const int32_t* target, int width, int32_t* path,
                                                         int32_t* count, int32_t* next)
{
    __shared__ int answer[kTreeRows];
    const int lane = threadIdx.x, i = blockIdx.x;
    int32_t* const mine = path + (int64_t)i * width;
    KvSeq s;
    int taken = 0, last = -1;
    if (kv_seq(b, i, s)) {
        const int n = s.n < kTreeRows ? s.n : kTreeRows;
        int from[kTreeWords], says[kTreeWords];
#pragma unroll
        for (int w = 0; w < kTreeWords; ++w) {
            const int r = 64 * w + lane;
            from[w] = -2;
            if (r >= n) continue;
            from[w] = tree_parent(parent[s.t0 + r], r);
            says[w] = token[s.t0 + r];
            answer[r] = target[s.t0 + r];
        }
        __syncthreads();
        int current = 0;
        while (true) {
            if (lane == 0) mine[taken] = current;
            ++taken;
            last = answer[current];
            if (taken == width) break;
            int child = -1;
#pragma unroll
            for (int w = 0; w < kTreeWords; ++w) {
                if (64 * w >= n) break;
                const uint64_t hit = __ballot(from[w] == current && says[w] == last);
                if (hit && child < 0) child = 64 * w + __builtin_ctzll(hit);
            }
            if (child < 0) break;             // ends: a child is a later row
            current = child;
        }
    }
    for (int k = taken + lane; k < width; k += 64) mine[k] = -1;
    if (lane == 0) {
        if (count) count[i] = taken;
        if (next) next[i] = last;
    }
}

hipError_t launch_tree_mask(const KvBatch& b, const int32_t* parent, int words, uint64_t* mask, int32_t* pos,
                            hipStream_t stream)
{
    tree_mask_kernel<<<(unsigned)b.nseq, 64 * words, 0, stream>>>(b, parent, words, mask, pos);
    return hipGetLastError();
}

hipError_t launch_tree_accept(const KvBatch& b, const int32_t* parent, const int32_t* token, const int32_t* target,
                              int width, int32_t* path, int32_t* count, int32_t* next, hipStream_t stream)
{
    tree_accept_kernel<<<(unsigned)b.nseq, 64, 0, stream>>>(b, parent, token, target, width, path, count, next);
    return hipGetLastError();
}

}  // namespace tern
