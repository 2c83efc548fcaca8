// tern_attend_tree.hip — attention for the rows of trees of drafted tokens over
// the paged int8 cache: a row sees what stands in front of its tree and, of the
// tree, the rows of its mask.
//
//   out = sum_p w_p V[p] / sum_p w_p,  w_p = exp(scale * q . K[p])
//
// As in the causal kernels the rows of one key/value head are columns: column c
// of a sequence is row c / G under query head h*G + c % G.  Few columns or short
// contexts: the int8 path, in tiles of 16, as single tokens and drafts take it.
// Long work of many columns: the fp16 path below, in tiles of 128.  Only the blocks
// that hold rows of the tree look at masks.
//
// Work: a unit is a tile of columns and a head.  Long units are cut into chunks
// of blocks, one for each workgroup; only the device knows the lengths (a
// captured graph follows them), so every workgroup works out how long a chunk
// is for the chunks of all units to fill the card once, and which is its own.
// Chunks of one head are a multiple of the heads apart, tile beside tile: the
// tiles of a chunk run at the same time, where heads are a multiple of 8 on one
// XCD, and share its reads in L2.  The parts of a cut unit are joined by a second
// kernel.
//
// Measured, us, medians of the kernel and the join in a trace (MI355X, 32:8 heads of
// 128, caches of 600 MB used in turn; 10% between cards):
//   64 rows over 12338 tokens                  30.6 + 6.6    (26 MB, 16 of parts)
//   32 trees of 9 to 33 rows over 200 to 8000  74.3 + 10.5   (154 MB, 21 of parts; at best 65.6 + 9.2)
//   500 rows over 4001, 130 over 900           63.9 + 8.0    (37.9e6 matrix-core cycles: 28% of them)
//   8 rows over 512, 16:8 heads                 8.8
// What bounds the second and third: chunks of unlike length (with all blocks alike
// and sequences in order the last ended at 65 us, the median at 44 to 46).  Equal
// stretches of a line of all units, cut anywhere, were built: 63 and 63 us, but more
// parts, 12.6 and 9.8 us to join, and the first 32: tiles of a head no longer side by
// side.  Loads a block further ahead changed nothing.
#include "tern_attend.h"

namespace tern {

typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

// where a tile's column is written to
__device__ __forceinline__ uint16_t* tree_row(const AttArgs& a, const AttTile& tile, int h, int col, int heads, int D)
{
    const int cc = tile.col0 + col, j = cc / a.G;
    return a.out + ((int64_t)(tile.s.t0 + j) * heads * a.G + h * a.G + cc - j * a.G) * D;
}

__device__ __forceinline__ u16x4 tree_result(f32x4 o, float sum, float r)
{
    u16x4 y;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = sum == 0.0f ? (uint16_t)0 : f32_to_bf16(none_below<true>(o[e] * r));
    return y;
}

// ---- the fp16 path ----------------------------------------------------------
// Tiles of 128 CG columns, four waves with CG groups of 32 columns each.  A block's
// codes are turned into fp16 once for all of them on their way into LDS.
//   S^T = K Q^T   32 tokens x 32 columns x 16 dims; q divided by the power of
//                 two below its row's largest value, exact to 2^-25 of that.
//   weights       2^(9 + x + log2 s_V - m) in fp16, the values' scale in the
//                 exponent; m, the row's largest x + log2 s_V so far, moves only
//                 when a weight would pass 2^15.
//   O^T = V^T P^T the lane's weights are the B operand as they stand; V lies in
//                 LDS in their order.
// A block's step has two stretches without a branch: the next block's scores on the
// matrix cores beside this one's weights, then this one's values beside the codes
// of later blocks on their way into LDS.  So each wave by itself keeps both the
// matrix cores and the vector units busy; the order is written out, piece by piece
// behind every matrix instruction.  What needs a branch stands in front of them:
// masks, in the blocks that hold rows of the tree, and a maximum that moves.
// A block takes a lone workgroup of a CU 2400 cycles, two together 3150 for a block
// of each (scores 1090, values 1350, barrier 290 of them); 4900 a pair before the
// order was written out.  The matrix cores need 1024 for each, the vector units
// about 1400: those are the bound while many blocks are left, the way to the first
// one (8 us: cu, table, codes, each behind the other) while few are.
template <int D>
__device__ __forceinline__ void attend_tree_f16(const KvCache& c, const KvBatch& b, const AttArgs& a,
                                                const AttTile& tile, int h, int begin, int end, bool whole,
                                                uint32_t slot)
{
    constexpr int S = D / 64, ST = D / 16, U = D / 32, COLS = 32 * kAttWaves;
    constexpr int kHalf = kKvBlock * D / 8;          // fp16 operands of a block's keys, or of its values
    __shared__ u32x4 kbuf[2 * kHalf], vbuf[2 * kHalf];
    __shared__ uint64_t smask[kAttWaves][32][kTreeWords + 1];
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6), half = lane >> 5;
    // lane i looks up block seg + i; the first look-up is under way before all else
    const auto find = [&](int seg) {
        return lane < end - seg ? kv_block(b, c, tile.s.i, tile.b0 + seg + lane) : -1;
    };
    int mine = find(begin);
    __builtin_amdgcn_sched_barrier(0);

    const bool works = 32 * wave < tile.cols;        // a wave without columns only fills LDS
    const int col = 32 * wave + (lane & 31);
    const bool live = col < tile.cols;
    const int cc = tile.col0 + (live ? col : 0), j = cc / a.G;
    const uint16_t* row = a.q + (int64_t)(tile.s.t0 + j) * a.q_stride + (int64_t)(h * a.G + cc - j * a.G) * D;
    const int last = live ? att_last(tile.s.p0 + j, att_limit(b)) : INT32_MAX;
    // a wave's own columns' masks: no other wave waits for them
    const uint64_t* words = a.mask + (int64_t)(tile.s.t0 + j) * a.words;
    const uint64_t word0 = half < a.words ? words[half] : 0;
    // step 4 s + e, half: dims 64 s + 16 half + 4 e .. + 3 and 32 further on
    u32x4 q[ST];
#pragma unroll
    for (int s = 0; s < ST; ++s) {
        const uint16_t* p = row + 64 * (s >> 2) + 16 * half + 4 * (s & 3);
        const u32x2 x = *(const u32x2*)p, y = *(const u32x2*)(p + 32);
        q[s] = u32x4{x[0], x[1], y[0], y[1]};
    }
    // This thread's two chunks of 16 bytes of a block's K and of its V: groups g
    // and g + 2 of one token and 64 dims, or of one dim.
    const int tid = threadIdx.x;
    const bool fills = tid < 2 * D;
    const int item = fills ? tid : 0, fr = item & 15, fg = (item >> 4) & 1, fu = item >> 5;
    const int from = ((fu * 4 + fg) * 16 + fr) * 16;
    u32x4* const k_to = kbuf + ((fu / S >> 1) * ST + fu % S * 4) * 64 + (fu / S & 1) * 16 + fg * 32 + fr;
    u32x4* const v_to = vbuf + (fu >> 1) * 256 + (fu & 1) * 16 + fg * 32 + fr;

    // the blocks that are there move to the front, and the first are asked for
    typedef u32x4 Raw[2];
    int blocks, number;
    float sk, lv, back;
    Raw k0, v0, k1, rk, rv;              // blocks 0 and 1; then keys two blocks ahead, values one
    const auto fetch = [&](int i, int side, Raw& raw) {
        const int64_t phys = __builtin_amdgcn_readlane(mine, i < blocks ? i : blocks - 1);
        const int8_t* p = c.codes + ((phys * c.heads + h) * 2 + side) * (kKvBlock * D) + from;
        raw[0] = *(const u32x4*)p;
        raw[1] = *(const u32x4*)(p + 512);
    };
    const auto look = [&](int seg) {
        float2 sc = make_float2(0.0f, 0.0f);
        const uint64_t there = __ballot(mine >= 0), below = (1ull << lane) - 1;
        if (mine >= 0) sc = *(const float2*)(c.scales + ((int64_t)mine * c.heads + h) * 2);
        blocks = __popcll(there);
        if (blocks == 0) return;
        const int dest = (mine >= 0 ? __popcll(there & below) : blocks + __popcll(~there & below)) * 4;
        mine = __builtin_amdgcn_ds_permute(dest, mine);
        number = __builtin_amdgcn_ds_permute(dest, tile.b0 + seg + lane);
        fetch(0, 0, k0);
        fetch(0, 1, v0);
        fetch(1, 0, k1);
        fetch(1, 1, rv);
        fetch(2, 0, rk);
        sk = __builtin_bit_cast(float, __builtin_amdgcn_ds_permute(dest, __builtin_bit_cast(int, sc.x)));
        const float sv = __builtin_bit_cast(float, __builtin_amdgcn_ds_permute(dest, __builtin_bit_cast(int, sc.y)));
        // the values' scales as exponents, and what takes them out of the sum of weights
        lv = sv < INFINITY ? __log2f(fmaxf(sv, kF16Least)) : NAN;
        back = exp2_fast(-lv);
    };
    const auto pick = [](float v, int i) {
        return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), i));
    };
    look(begin);
    __builtin_amdgcn_sched_barrier(0);               // all of it is under way before the queries are waited for
    if (half < a.words) smask[wave][lane & 31][half] = word0;
    for (int w = half + 2; w < a.words; w += 2) smask[wave][lane & 31][w] = words[w];
    uint32_t qtop = 0;
#pragma unroll
    for (int s = 0; s < ST; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t x0 = (q[s][e] << 16) & 0x7FFF0000u, x1 = q[s][e] & 0x7FFF0000u;
            qtop = x0 > qtop ? x0 : qtop;
            qtop = x1 > qtop ? x1 : qtop;
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
    __builtin_amdgcn_wave_barrier();                 // masks are read by the column's other lane

    const auto fill = [&](u32x4* to, int buf, const Raw& raw) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const u32x2 x0 = codes_f16(raw[0][e]), x1 = codes_f16(raw[1][e]);
            if (D == 128 || fills) to[buf * kHalf + 64 * e] = u32x4{x0[0], x0[1], x1[0], x1[1]};
        }
    };
    float m = -INFINITY, l = 0.0f, top = 0.0f;         // top: the lane's largest score of the block that a step weighs
    f32x16 acc[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[u][e] = 0.0f;
    // Operands of a block's keys and of its values, and the pieces of other work that
    // go behind each of their matrix instructions.
    constexpr int kScore = 2 * ST, kValue = 4 * U, kPairs = 16 / kScore, kWords = 16 / kValue;
    u32x4 ahead[kAhead];                             // operands on their way from LDS
    const auto key = [&](int buf, int k) { return kbuf[buf * kHalf + (k % 2 * ST + k / 2) * 64 + lane]; };

    // One block: its scores are in x, the next block's go to nx.  Token of x[t][e]:
    // 32 t + 8 (e / 4) + 4 half + e % 4.
    const auto step = [&](int i, f32x16 (&x)[2], f32x16 (&nx)[2]) {
        __syncthreads();                 // keys up to block i + 1 and values up to i are in LDS
        // read with every lane active: a lane's value must not be computed behind a mask
        float f = rowf * pick(sk, i);
        const float lvi = pick(lv, i), backi = pick(back, i);
        const int at = __builtin_amdgcn_readlane(number, i) * kKvBlock;
        float base = kF16Up + lvi - (m == -INFINITY ? 0.0f : m);
        const bool own = at + 63 >= tile.s.p0;
        const uint64_t moves = __ballot((m == -INFINITY) | (fmaf(top, f, base) > kF16Top));
        if (__builtin_expect((moves != 0) | own, 0)) {            // one branch, seldom taken
            const uint64_t bits =
                own ? tree_bits(smask[wave][lane & 31], a.words, tile.s.p0, at, last) >> 4 * half : ~0ull;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    x[t][e] = tree_sees((uint32_t)(bits >> 32 * t), 8 * (e >> 2) + (e & 3), fmaf(x[t][e], f, base));
            f = 1.0f;                    // exponents already, all but a maximum that moves
            base = 0.0f;
            if (moves) {                 // also where only hidden scores are large: then by is 0
                top = x[0][0];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 16; ++e) top = fmaxf(top, x[t][e]);
                top = fmaxf(top, __shfl_xor(top, 32));
                const float over = top - kF16Up;
                const bool first = m == -INFINITY, grow = first ? over > -INFINITY : over > 0.0f;
                const float by = grow ? over : 0.0f;
                m = grow ? (first ? 0.0f : m) + by : m;
                if (__any(grow && !first)) {         // what has been summed so far is of the old maximum
                    const float keep = first ? 1.0f : exp2_fast(-by);
                    l *= keep;
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[u][e] *= keep;
                }
                base = -by;
            }
        }
        u32x4 w[4];                      // the weights: B operands of 16 tokens each
        float sum0 = 0.0f, sum1 = 0.0f, w0 = 0.0f, w1 = 0.0f;
        const auto finish = [&](int p) {
            sum0 += w0;
            sum1 += w1;
            w[p >> 2][p & 3] = pack_f16(w0, w1);
        };
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) ahead[k] = key((i + 1) & 1, k);
#pragma unroll
        for (int k = 0; k < kScore; ++k) {
            nx[k % 2] = mfma_f16(ahead[k % kAhead], q[k / 2], k < 2 ? f32x16{} : nx[k % 2]);
            if (k + kAhead < kScore) ahead[k % kAhead] = key((i + 1) & 1, k + kAhead);
#pragma unroll
            for (int p = k * kPairs; p < (k + 1) * kPairs; ++p) {
                const float y0 = fmaf(x[p >> 3][2 * p & 15], f, base), y1 = fmaf(x[p >> 3][(2 * p & 15) + 1], f, base);
                if (p > 0) finish(p - 1);
                w0 = exp2_fast(y0);
                w1 = exp2_fast(y1);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        finish(15);
        const float sum = sum0 + sum1;
        // a row that sees nothing here is spared a scale that is not finite
        l += sum == 0.0f ? 0.0f : sum * backi;
        top = nx[0][0];
        const auto value = [&](int k) { return vbuf[(i & 1) * kHalf + (k % U * 4 + k / U) * 64 + lane]; };
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) ahead[k] = value(k);
        u32x4 wide;
#pragma unroll
        for (int k = 0; k < kValue; ++k) {
            acc[k % U] = mfma_f16(ahead[k % kAhead], w[k / U], acc[k % U]);
            if (k + kAhead < kValue) ahead[k % kAhead] = value(k + kAhead);
#pragma unroll
            for (int p = k * kWords; p < (k + 1) * kWords; ++p)
                top = fmaxf(fmaxf(top, nx[p >> 3][2 * p & 15]), nx[p >> 3][(2 * p & 15) + 1]);
#pragma unroll
            for (int n = k * kWords; n < (k + 1) * kWords; ++n) {
                const int e = n / 2 % 4, chunk = n % 2;
                const u32x2 two = codes_f16((n < 8 ? rk : rv)[chunk][e]);
                wide[2 * chunk] = two[0];
                wide[2 * chunk + 1] = two[1];
                if (chunk == 1 && (D == 128 || fills))
                    (n < 8 ? k_to + (i & 1) * kHalf : v_to + ((i + 1) & 1) * kHalf)[64 * e] = wide;
                if (n == 7) fetch(i + 3, 0, rk);
                if (n == 15) fetch(i + 2, 1, rv);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    for (int seg = begin; seg < end; seg += 64) {
        if (seg > begin) {
            mine = find(seg);
            look(seg);
        }
        if (blocks == 0) continue;
        fill(k_to, 0, k0);
        fill(v_to, 0, v0);
        fill(k_to, 1, k1);
        __syncthreads();
        f32x16 x0[2], x1[2];
        if (works) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) ahead[k] = key(0, k);
#pragma unroll
            for (int k = 0; k < kScore; ++k) {
                x0[k % 2] = mfma_f16(ahead[k % kAhead], q[k / 2], k < 2 ? f32x16{} : x0[k % 2]);
                if (k + kAhead < kScore) ahead[k % kAhead] = key(0, k + kAhead);
            }
            // As a step does for the next block; before the first one m is -inf and top not looked at
            // (64 rows over 12338 tokens 33.4 us in a graph, 33.7 with it there too).
            if (seg > begin) {
                top = x0[0][0];
#pragma unroll
                for (int p = 0; p < 16; ++p)
                    top = fmaxf(fmaxf(top, x0[p >> 3][2 * p & 15]), x0[p >> 3][(2 * p & 15) + 1]);
            }
            for (int i = 0;;) {          // the scores change places: no copies
                step(i, x0, x1);
                if (++i == blocks) break;
                step(i, x1, x0);
                if (++i == blocks) break;
            }
        } else {
            for (int i = 0; i < blocks; ++i) {
                __syncthreads();         // as in step
                fill(k_to, i & 1, rk);
                fill(v_to, (i + 1) & 1, rv);
                fetch(i + 3, 0, rk);
                fetch(i + 2, 1, rv);
            }
        }
        __syncthreads();                 // before the next blocks use LDS
    }

    // dim of acc[u][e]: 32 u + 8 (e / 4) + 4 half + e % 4; parts stay in this order
    if (!works) return;
    const float sum = l + __shfl_xor(l, 32);
    if (!whole) {
        float* to = a.part + ((int64_t)slot * kAttWaves + wave) * (32 * D) + lane * 4;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                *(f32x4*)(to + (4 * u + e / 4) * 256) = f32x4{acc[u][e], acc[u][e + 1], acc[u][e + 2], acc[u][e + 3]};
        if (half == 0) a.stat[slot * COLS + col] = make_float2(m, sum);
    } else if (live) {
        const float r = sum == 0.0f ? 0.0f : 1.0f / sum;
        uint16_t* to = tree_row(a, tile, h, col, c.heads, D) + 4 * half;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                *(u16x4*)(to + 32 * u + 2 * e) =
                    tree_result(f32x4{acc[u][e], acc[u][e + 1], acc[u][e + 2], acc[u][e + 3]}, sum, r);
    }
}

// ---- work --------------------------------------------------------------------

// A sequence's tiles and what each of its units costs at most, in blocks; none for a
// sequence without rows, s.n < 0 where cu descends.  On the fp16 path one of the last
// blocks, those that hold rows of the tree and look at masks, counts as two where
// they are more than two (500 rows over 4001 tokens, 130 over 900: 69.3 us with all
// blocks alike, 64.5 so; 32 trees of 9 to 33 rows 70.4 and 73.2).
struct TreeShare {
    uint32_t tiles, cost, plain;             // plain: the blocks in front of the tree's
};

// of a sequence whose rows are its own and inside the tensors
template <int COLS>
__device__ __forceinline__ TreeShare tree_share_of(const KvBatch& b, int G, const KvSeq& s)
{
    const int last = att_last(s.p0 + s.n - 1, att_limit(b));
    const uint32_t blocks = last < 0 ? 1 : (uint32_t)last / kKvBlock + 1;
    const uint32_t front = s.p0 > 0 ? (uint32_t)s.p0 / kKvBlock : 0;
    const uint32_t plain = COLS == 16 || front + 2 >= blocks ? blocks : front;
    return {(uint32_t)(((int64_t)s.n * G + COLS - 1) / COLS), 2 * blocks - plain, plain};
}

// the block at a place of a unit's cost, and the first place of a block
__device__ __forceinline__ uint32_t tree_block(const TreeShare& r, uint32_t at)
{
    return at <= r.plain ? at : r.plain + (at - r.plain + 1) / 2;
}

__device__ __forceinline__ uint32_t tree_place(const TreeShare& r, uint32_t block)
{
    return block <= r.plain ? block : 2 * block - r.plain - 1;
}

template <int COLS>
__device__ __forceinline__ TreeShare tree_share(const KvBatch& b, int i, int G, KvSeq& s)
{
    s.i = i;
    s.t0 = b.cu[i];
    const int t1 = b.cu[i + 1], len = kv_length(b, i);
    s.n = t1 < s.t0 ? -1 : t1 - s.t0;
    s.p0 = len - s.n;
    if (s.t0 < 0 || t1 > b.T || s.n <= 0) return {0, 1, 1};
    return tree_share_of<COLS>(b, G, s);
}

// chunks of a unit of this cost, `most` of it each at most (0: any), and the cost of
// each: the waves of the int8 path take blocks in turn
template <int COLS>
__device__ __forceinline__ uint32_t tree_chunks(uint32_t cost, uint32_t most, uint32_t& each)
{
    constexpr uint32_t kTurn = COLS < 64 ? att_turn<COLS>() : 1;
    if (most == 0 || cost <= most) {
        each = cost;
        return 1;
    }
    const uint32_t n = (cost + most - 1) / most;
    each = ((cost + n - 1) / n + kTurn - 1) / kTurn * kTurn;
    return n;
}

constexpr uint32_t kTreeLeast = 4;           // blocks of a chunk
constexpr int kTreeTries = 16;
// Sequences a lane up to which whole units are counted without gaps, so that each CU
// gets as many; more are found 64 at a time (512 trees of 4 rows over 500 tokens
// 175 us and 153, 1024 of 2 over 300 382 and 172; 16 of 8 over 3000 26 and 31).
constexpr int kTreeRun = 4;

// sums over the lanes up to each
__device__ __forceinline__ uint32_t scan(uint32_t v)
{
#define TREE_STEP(ctrl, rows) v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xF, false)
    TREE_STEP(0x111, 0xF);                   // a row of 16 lanes: by 1, 2, 4, 8
    TREE_STEP(0x112, 0xF);
    TREE_STEP(0x114, 0xF);
    TREE_STEP(0x118, 0xF);
    TREE_STEP(0x142, 0xA);                   // rows 0 and 2 into the next, then the lower half into the upper
    TREE_STEP(0x143, 0xC);
#undef TREE_STEP
    return v;
}

template <int D, int COLS>
__global__ __launch_bounds__(64 * kAttWaves, COLS == 16 ? 3 : 2) void kv_attend_tree_kernel(KvCache c, KvBatch b,
                                                                                            AttArgs a)
{
    const int lane = threadIdx.x & 63, run = (b.nseq + 63) / 64;
    const uint32_t x = blockIdx.x;
    AttTile tile;
    uint32_t number, h, parts = 1;
    int begin = 0, end = INT32_MAX;
    if (a.groups == 0 && run > kTreeRun) {
        int64_t local;
        if (!kv_find(b, x / c.heads, a.G, COLS, 1, tile.s, local)) return;
        number = (uint32_t)local;
        h = x % c.heads;
    } else {
        // every lane has a run of sequences, up to the first descent of cu
        TreeShare r = {0, 1, 1};
        uint32_t work = 0;
        bool falls = false;
        for (int k = lane * run; k < lane * run + run && k < b.nseq && !falls; ++k) {
            r = tree_share<COLS>(b, k, a.G, tile.s);
            falls = tile.s.n < 0;
            work += r.tiles * r.cost;
        }
        const uint64_t fell = __ballot(falls);
        const int lanes = fell ? __builtin_ctzll(fell) : 63;      // the last that counts
        // a lane's chunks, `most` blocks each at most
        const auto chunks = [&](uint32_t most) {
            uint32_t n = 0, each;
            if (lane > lanes) return n;
            if (run == 1) return r.tiles * c.heads * tree_chunks<COLS>(r.cost, most, each);
            KvSeq s;
            for (int k = lane * run; k < lane * run + run && k < b.nseq; ++k) {
                const TreeShare o = tree_share<COLS>(b, k, a.G, s);
                if (s.n < 0) break;
                n += o.tiles * c.heads * tree_chunks<COLS>(o.cost, most, each);
            }
            return n;
        };
        // chunks as short as the card holds at one time, to within a sixteenth
        uint32_t most = 0, mine = 0, base = 0, sum = 0, each = 0;
        if (a.groups > 0) {
            const uint32_t all = __builtin_amdgcn_readlane(scan(lane > lanes ? 0 : work), 63) * c.heads;
            most = (all + a.groups - 1) / a.groups;
            most = most < kTreeLeast ? kTreeLeast : most;
        }
        for (int tries = 0;; ++tries) {
            mine = chunks(most);
            base = scan(mine);
            sum = __builtin_amdgcn_readlane(base, 63);
            base -= mine;
            if (most == 0 || sum <= (uint32_t)a.groups || tries == kTreeTries) break;
            most += 1 + most / 16;
        }
        // The longest chunks first, so that the last to run are short (48 trees of 20 to
        // 32 rows over 200 to 16000 tokens, at random, 309 us in order, 291 so, 32 of 9 to
        // 33 over 200 to 8000 73.0 and 71.3; for up to 64 sequences, one a lane); of whole
        // units the order costs more than it gives (60 of 4 to 8 rows over 200 to 2000 38.5
        // and 42.6).
        if (a.groups > 0 && run == 1) {
            tree_chunks<COLS>(r.cost, most, each);
            base = 0;
            for (int k = 0; k < b.nseq; ++k) {
                const uint32_t other = __builtin_amdgcn_readlane(each, k), count = __builtin_amdgcn_readlane(mine, k);
                base += other > each || (other == each && k < lane) ? count : 0;
            }
        }
        if (a.groups > 0 && blockIdx.x == 0 && threadIdx.x < 64) {   // for the joining kernel
            uint32_t from = base;
            for (int k = lane * run; k < lane * run + run && k < b.nseq; ++k) {
                KvSeq s;
                const TreeShare o = tree_share<COLS>(b, k, a.G, s);
                a.start[k] = lane <= lanes && s.n >= 0 ? from : sum;
                from += o.tiles * c.heads * tree_chunks<COLS>(o.cost, most, each);
                if (s.n < 0) from = sum;
            }
            if (lane == 0) {
                a.start[b.nseq] = sum;
                a.start[b.nseq + 1] = most;
            }
        }
        if (x >= sum) return;
        // the lane whose run holds x, then the sequence inside the run
        const int owner = __builtin_ctzll(__ballot(x - base < mine));
        uint32_t at = __builtin_amdgcn_readlane(base, owner);
        int i = owner * run;
        while (true) {
            r = tree_share<COLS>(b, i, a.G, tile.s);
            parts = tree_chunks<COLS>(r.cost, most, each);
            const uint32_t here = r.tiles * c.heads * parts;
            if (x - at < here || i + 1 >= b.nseq) break;          // the first: x is below the run's end
            at += here;
            ++i;
        }
        const uint32_t rest = (x - at) / c.heads, chunk = rest / r.tiles;
        h = x - at - rest * c.heads;
        number = rest - chunk * r.tiles;
        begin = (int)tree_block(r, chunk * each);
        end = (int)tree_block(r, (chunk + 1) * each);
    }
    if (!att_tile<COLS>(b, (int)number, a.G, 0, tile)) return;
    att_uniform(tile);
    begin = uni(begin);
    if (begin > 0 && begin >= tile.nblk) return;              // the tile sees less than the sequence's last
    end = uni(end < tile.nblk ? end : tile.nblk);
    if constexpr (COLS < 64) attend_blocks<D, COLS / 16, false, true>(c, b, a, tile, h, begin, end, parts == 1, x);
    else attend_tree_f16<D>(c, b, a, tile, h, begin, end, parts == 1, x);
}

// Joins the parts of the cut units.  A job is 32 columns and 8 dims of a unit (fp16
// path: 1 KiB of each part in the order in which the lanes held it), or a column
// (int8 path).  Few units: the waves of a workgroup take one job's parts in turn, JW
// = 4.  Many: a wave has JOBS jobs of one unit, all their loads in flight at once
// (32 trees 12.2 us one after another).
template <int D, int COLS, int JW, int JOBS>
__global__ __launch_bounds__(64 * kAttWaves) void kv_attend_tree_join_kernel(KvCache c, KvBatch b, AttArgs a)
{
    constexpr bool F16 = COLS >= 64;
    constexpr int kAll = F16 ? COLS / 32 * (D / 8) : COLS, kDims = F16 ? 4 : D / 64;
    constexpr int kEach = JOBS * kAttWaves / JW, kLoads = JW == 1 ? 4 : 8;
    const int lane = threadIdx.x & 63, own = uni(threadIdx.x >> 6), wave = JW == 1 ? 0 : own;
    const uint32_t unit = blockIdx.x / (kAll / kEach);
    const int first = (blockIdx.x - unit * (kAll / kEach)) * kEach + (JW == 1 ? own * JOBS : 0);
    const uint32_t tiles = unit / c.heads, h = unit - tiles * c.heads;
    const uint32_t all = a.start[b.nseq], most = a.start[b.nseq + 1];
    const uint32_t starts = a.start[lane < b.nseq ? lane : 0];
    AttTile tile;
    int64_t number;
    if (!kv_find(b, tiles, a.G, COLS, 1, tile.s, number) || !att_tile<COLS>(b, (int)number, a.G, 0, tile)) return;
    att_uniform(tile);
    const uint32_t start = tile.s.i < 64 ? __builtin_amdgcn_readlane(starts, tile.s.i) : a.start[tile.s.i];
    const TreeShare r = tree_share_of<COLS>(b, a.G, tile.s);
    uint32_t each;
    if (start >= all || tree_chunks<COLS>(r.cost, most, each) == 1) return;     // written already
    // parts that have blocks
    const int used = tile.nblk > 0 ? (int)((tree_place(r, tile.nblk) + each - 1) / each) : 1;
    // a wave's jobs are of the same columns (fp16), or of the columns from `first` on
    const int col0 = F16 ? first / (D / 8) * 32 : first;
    if (col0 >= tile.cols) return;
    const auto column = [&](int f) { return F16 ? col0 + (lane & 31) : first + f; };
    float top[JOBS], sum[JOBS], o[JOBS][kDims];
#pragma unroll
    for (int f = 0; f < JOBS; ++f) {
        top[f] = -INFINITY;
        sum[f] = 0.0f;
#pragma unroll
        for (int u = 0; u < kDims; ++u) o[f][u] = 0.0f;
    }
    for (int seg = 0; seg < used; seg += kLoads * JW) {
        float x[kLoads][JOBS][kDims];
        float2 st[kLoads][JOBS];
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {          // behind the last part its values are read again, unused
            const int s = seg + wave + JW * k;
            const int64_t at = start + ((uint32_t)(s < used ? s : used - 1) * r.tiles + (uint32_t)number) * c.heads + h;
#pragma unroll
            for (int f = 0; f < JOBS; ++f) {
                st[k][f] = F16 && f > 0 ? st[k][0] : a.stat[at * COLS + column(f)];
                if (s >= used) st[k][f] = make_float2(-INFINITY, 0.0f);
                if constexpr (F16) {
                    const f32x4 v = *(const f32x4*)(a.part + at * (COLS * D) + (first + f) * 256 + lane * 4);
#pragma unroll
                    for (int u = 0; u < 4; ++u) x[k][f][u] = v[u];
                } else {
#pragma unroll
                    for (int u = 0; u < kDims; ++u) x[k][f][u] = a.part[(at * COLS + column(f)) * D + u * 64 + lane];
                }
            }
        }
#pragma unroll
        for (int f = 0; f < JOBS; ++f) {
            float now = top[f];
#pragma unroll
            for (int k = 0; k < kLoads; ++k) now = fmaxf(now, st[k][f].x);
            const float keep = top[f] == now ? 1.0f : exp2_fast(top[f] - now);
            top[f] = now;
            sum[f] *= keep;
#pragma unroll
            for (int u = 0; u < kDims; ++u) o[f][u] *= keep;
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const float w = st[k][f].x == now ? 1.0f : exp2_fast(st[k][f].x - now);
                sum[f] = fmaf(st[k][f].y, w, sum[f]);
#pragma unroll
                for (int u = 0; u < kDims; ++u)
                    o[f][u] = seg + wave + JW * k < used ? fmaf(x[k][f][u], w, o[f][u]) : o[f][u];
            }
        }
    }
    if constexpr (JW > 1) {
        static_assert(JOBS == 1);
        __shared__ float so[JW][kDims][64];
        __shared__ float2 sst[JW][64];
        sst[wave][lane] = make_float2(top[0], sum[0]);
#pragma unroll
        for (int u = 0; u < kDims; ++u) so[wave][u][lane] = o[0][u];
        __syncthreads();
        if (wave > 0) return;
        sum[0] = 0.0f;
#pragma unroll
        for (int w = 0; w < JW; ++w) top[0] = fmaxf(top[0], sst[w][lane].x);
#pragma unroll
        for (int u = 0; u < kDims; ++u) o[0][u] = 0.0f;
#pragma unroll
        for (int w = 0; w < JW; ++w) {
            const float f = sst[w][lane].x == top[0] ? 1.0f : exp2_fast(sst[w][lane].x - top[0]);
            sum[0] = fmaf(sst[w][lane].y, f, sum[0]);
#pragma unroll
            for (int u = 0; u < kDims; ++u) o[0][u] = fmaf(so[w][u][lane], f, o[0][u]);
        }
    }
#pragma unroll
    for (int f = 0; f < JOBS; ++f) {
        const int col = column(f);
        if (col >= tile.cols) continue;
        const float inv = sum[f] == 0.0f ? 0.0f : 1.0f / sum[f];
        uint16_t* to = tree_row(a, tile, h, col, c.heads, D);
        if constexpr (F16) {
            *(u16x4*)(to + (first + f) % (D / 8) * 8 + 4 * (lane >> 5)) =
                tree_result(f32x4{o[f][0], o[f][1], o[f][2], o[f][3]}, sum[f], inv);
        } else {
#pragma unroll
            for (int u = 0; u < kDims; ++u) to[u * 64 + lane] = f32_to_bf16(sum[f] == 0.0f ? 0.0f : o[f][u] * inv);
        }
    }
}

// ---- choice ------------------------------------------------------------------

// A call: columns of a tile; workgroups that chunks are to fill, one round of the
// card (0: every unit whole, one launch); workgroups at most.
struct TreePlan {
    int cols, groups;
    int64_t grid, part_floats, stats, starts;
    int64_t bytes() const { return part_floats * 4 + stats * 8 + (starts + 3) / 4 * 16; }
};

// what the parts of a cut call take
static void tree_space(TreePlan& p, int64_t D, int64_t nseq)
{
    p.stats = p.grid * p.cols;
    p.part_floats = p.stats * D;
    p.starts = nseq + 2;
}

constexpr int64_t kTreeUnits = 1024;             // of 128 columns that are cut, at most

// Estimates in us, fitted to 14 shapes of D 128 (1 to 64 trees of 8 to 500 rows
// over 500 to 40000 tokens, G 2 and 4, graphs of calls over caches used in turn).
// 16 columns whole: 0.27 us a block of the longest unit (four waves take blocks in
// turn), or 1050 blocks of all units a us and the starts of each round of the card;
// cut, nothing waits for the longest, but parts are written, read and joined.  128
// columns: 205 blocks a us, more where waves have no columns.  What decides, us (16
// whole, 16 cut, 128 cut):
//   64 rows over   1000 tokens     10.8   17.5   20.9
//   64 rows over   4000 tokens     22.3   24.6   27.1
//   16 rows over  12338 tokens     54.9   20.6   26.9
//   64 rows over  12338 tokens     56     40     35.7
//   16 x 64 rows over 3000        103    106     80
//   32 trees of 9 to 33 rows over 200 to 8000     85     92     76
// Held against all three at 65 further shapes (D 64 and 128, G 1, 4 and 8, 1 to 64
// trees of 8 to 500 rows over 200 to 40000): within 6% of the best at 61, at most
// 19% off (64 rows over 12338 tokens, D 64, G 8: 44 us, 16 cut 37).
// 128 columns, one workgroup a CU or two: two leave parts twice as many, and pay off
// where chunks are long or units many (us, 256 and 512 workgroups: 64 rows over 6000
// tokens 29.4 and 31.3, over 12338 33.7 and 35.9, over 30000 54.3 and 53.2; 32 trees
// of 9 to 33 rows 152 and 75).  Above 1024 units they are not cut: they fill the
// card, and parts would take gigabytes.
static TreePlan tree_plan(int64_t T, int64_t Hq, int64_t heads, int64_t D, int64_t nseq, int64_t table_width,
                          int64_t max_len)
{
    const int64_t cols = T * (Hq / heads), blocks = (max_len + kKvBlock - 1) / kKvBlock;
    const auto units = [&](int c) { return (cols / c + nseq) * heads; };                      // at most
    const auto alike = [&](int c) { return (double)(nseq * heads * ((cols + nseq * c - 1) / (nseq * c))); };
    // lengths lie between all alike and evenly spread from none
    const double mean = (nseq > 1 ? 0.75 : 1.0) * blocks, u16 = alike(16);
    const double all16 = u16 * mean / 1050, longest = 0.27 * blocks;
    const double all128 = (0.45 * alike(128) + 0.55 * heads * cols / 128) * mean / 205;
    const double starts = 6 * (u16 > 768 ? u16 / 768 : 1), whole16 = starts + (longest > all16 ? longest : all16);
    const double cut16 = starts + 11 + all16, cut128 = 22 + all128;
    TreePlan p{};
    const bool wide = cut128 < whole16 && cut128 < cut16;
    p.cols = wide ? 128 : 16;
    const double u128 = alike(128);
    const int lone = u128 <= 64 && u128 * mean <= 256 * 28 ? 256 : 512;
    p.groups = wide ? (units(128) <= kTreeUnits ? lone : 0) : cut16 < whole16 ? 768 : 0;
    // the line of blocks is counted in 32 bits
    if (units(p.cols) * 2 * (table_width + kTreeTries) > INT32_MAX) p.groups = 0;
    p.grid = units(p.cols) + p.groups;
    if (p.groups > 0) tree_space(p, D, nseq);
    return p;
}

int64_t kv_attend_tree_workspace_bytes(int64_t T, int64_t Hq, int64_t heads, int64_t D, int64_t nseq, int64_t max_len)
{
    return tree_plan(T, Hq, heads, D, nseq, 0, max_len).bytes();
}

// The most that a call of up to these rows and sequences takes.  16 columns are cut
// where 0.27 us a block come to more than 11 us and 1050 blocks of all units a us,
// three quarters of the longest on average: below 0.27 * 1050 / 0.75 = 378 units of
// sequences alike, or 756 as they are counted for the workspace.
int64_t kv_attend_tree_workspace_limit(int64_t T, int64_t Hq, int64_t heads, int64_t D, int64_t nseq)
{
    int64_t most = 0;
    for (int cols : {16, 128}) {
        const int64_t units = (T * (Hq / heads) / cols + nseq) * heads, cut = cols == 16 ? 756 : kTreeUnits;
        TreePlan p{};
        p.cols = cols;
        p.grid = (units < cut ? units : cut) + (cols == 16 ? 768 : 512);
        tree_space(p, D, nseq < cut ? nseq : cut);       // a unit for each sequence at least
        most = p.bytes() > most ? p.bytes() : most;
    }
    return most;
}

void kv_attend_tree_config(int64_t T, int64_t Hq, int64_t heads, int64_t D, int64_t nseq, int64_t table_width,
                           int64_t max_len, int64_t* out)
{
    const TreePlan p = tree_plan(T, Hq, heads, D, nseq, table_width, max_len);
    out[0] = p.cols;
    out[1] = p.groups;
    out[2] = p.grid;
}

template <int D, int COLS>
static hipError_t attend_tree(const KvCache& c, const KvBatch& b, const AttArgs& a, const TreePlan& p,
                              hipStream_t stream)
{
    kv_attend_tree_kernel<D, COLS><<<(unsigned)p.grid, 64 * kAttWaves, 0, stream>>>(c, b, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.groups == 0) return e;
    const int64_t jobs = (p.grid - p.groups) * (COLS >= 64 ? COLS / 32 * (D / 8) : COLS);
    if (jobs <= 4096) kv_attend_tree_join_kernel<D, COLS, 4, 1><<<(unsigned)jobs, 256, 0, stream>>>(c, b, a);
    else kv_attend_tree_join_kernel<D, COLS, 1, 4><<<(unsigned)(jobs / 16), 256, 0, stream>>>(c, b, a);
    return hipGetLastError();
}

hipError_t launch_kv_attend_tree(const KvCache& c, const KvBatch& b, int64_t D, const uint16_t* q, int64_t Hq,
                                 int64_t q_stride, float scale, const uint64_t* mask, int words, int64_t max_len,
                                 uint16_t* out, void* workspace, hipStream_t stream)
{
    const TreePlan p = tree_plan(b.T, Hq, c.heads, D, b.nseq, b.table_width, max_len);
    AttArgs a{};
    a.q = q;
    a.out = out;
    a.part = (float*)workspace;
    a.stat = (float2*)(a.part + p.part_floats);
    a.start = (uint32_t*)(a.stat + p.stats);
    a.q_stride = q_stride;
    a.mask = mask;
    a.words = words;
    a.scale = scale;
    a.G = (int)(Hq / c.heads);
    a.groups = p.groups;
    if (p.cols == 16) return D == 128 ? attend_tree<128, 16>(c, b, a, p, stream) : attend_tree<64, 16>(c, b, a, p, stream);
    return D == 128 ? attend_tree<128, 128>(c, b, a, p, stream) : attend_tree<64, 128>(c, b, a, p, stream);
}

}  // namespace tern
