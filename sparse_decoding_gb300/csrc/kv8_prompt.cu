// kv8_prompt.cu -- attention of many queries over the 8-bit paged cache (prompts), on
// the 5th-generation tensor cores.
//
// For one sequence and kv head the rows are its new tokens times the query heads that
// share the kv head. A CTA works on a pair of 128-row tiles at a time and walks the
// tokens they see in blocks of 128:
//
//   S = (Qh + Ql) codes(K)^T   tcgen05.mma kind::f8f6f4, both operands in shared memory, S in tensor memory
//   P = 2^(S r s_K + e - m + 6)  one row per thread, written back to tensor memory as fp16
//   O += P codes(V) 2^-d       tcgen05.mma kind::f16, P from tensor memory, V^T in shared memory
//
// Each row of q is scaled by a power of two and split into an e4m3 and an e5m2 part, whose sum it is (exactly,
// down to 2^-13 of the row's largest): K's codes are an operand as they are stored, at the 8-bit rate, and no thread
// has to make them fp16. S carries the fp32 rounding of the sums, as in the kernel for few rows.
// The scales are powers of two of each cell (16 tokens). K's multiplies the scores in the softmax. V's codes are
// made fp16 and brought to one scale for the block, 2^e, a 128th of the largest of its eight (which keeps them below
// 448 * 2^7, in fp16's range; d: how many binary places a cell's scale is below it), which is an exponent of the weights; the
// sums of the weights are freed of it a block at a time. A row may see only tokens whose scales are far below that of a later
// one: codes are exact down to 2^-22 of the block's largest scale, and off by at most 2^-32 of it beyond.
//
// Roles (16 warps): two softmax warpgroups, one per tile (a thread owns a row: no
// reductions across threads; it also loads and splits its row of Q, rescales and
// stores its row of O); a warpgroup that copies the codes of K and V to shared memory, two blocks ahead, and makes V^T (both
// tiles use them); one warp that issues the MMAs; one that lists the pieces of work. While one tile is in its
// softmax, the other's MMAs run. The running maximum is raised only when a score passes it by 2^8, so O is rarely
// rescaled.
//
// What bounds it: the softmax warpgroups' instructions and their fetch. The exponentials alone (16 a clock and SM)
// take 230 us of the case below, its products 273 us at the measured bf16 rate, and the roles' loops together have to
// stay in the instruction caches, so they are rolled. One sequence of 8192 new tokens, 32 query heads on 8 (0.55
// TFLOP): K made fp16 beside V by 640 threads 705 us; K as an 8-bit operand 521; one copy of the MMA
// step and masks written back once 502, 1.1 PFLOP/s. Not kept: the softmax unrolled 740, its maximum in steps of 64
// columns 537, P passed on in halves 547.
//
// The blocks of all (sequence, kv head, pair) segments are one line, on which a
// segment takes kOver blocks more (what starting and ending a piece costs), cut evenly
// over one CTA per SM; a segment that was cut is joined, row by row, by the last
// CTAs to arrive of groups of its parts and then of the groups, in CTA order.
//
// All waits are bounded; one that runs out sets NM_ERR_TIMEOUT. Its thread's later waits
// poll once and its warp takes no more pieces, so the others run out in turn, the MMAs
// in flight end, and the kernel frees its tensor memory and returns.
#include "kv8.cuh"
#include "kv_ops.cuh"

namespace nm {
namespace {

constexpr int kSoft = 256;      // softmax threads: two tiles of 128 rows
constexpr int kUnpack = 128;    // unpacking threads
constexpr int kMmaWarp = 12;    // of its warpgroup, the next one lists the pieces and two idle
constexpr int kThreads = 512;
// Registers of a thread: at launch (what 512 threads can have), and in each role.
constexpr int kLaunchRegs = 128, kSoftRegs = 184, kUnpackRegs = 104, kMmaRegs = 40;
static_assert(kSoftRegs >= kLaunchRegs && kUnpackRegs <= kLaunchRegs && kMmaRegs <= kLaunchRegs &&
                  kSoft * kSoftRegs + kUnpack * kUnpackRegs + 128 * kMmaRegs <= kThreads * kLaunchRegs,
              "a role that takes registers waits until others have given them back");
constexpr int kSeqCache = 512;  // sequences whose descriptors are kept in shared memory
constexpr int kBlock = 128;    // tokens of a block
constexpr int kMinShare = 2;   // blocks of a CTA at least
constexpr float kShift = 6.0f, kSlack = 8.0f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int D> struct Cfg {
    static constexpr int kK = 128 * D;      // one part of a tile of Q, a stage of K, of V's codes
    static constexpr int kV = 2 * D * 128;  // a stage of V^T: two halves of 64 tokens
    static constexpr int kOffK = 4 * kK, kOffV = kOffK + 2 * kK, kOffRaw = kOffV + 2 * kV, kTiles = kOffRaw + 2 * kK;
    static constexpr int kPart = 128 * (D + 2); // floats of a tile's part
    // where in a row of D bytes (under the D-byte swizzle) its c-th 16 bytes are
    static __device__ __forceinline__ uint32_t piece(int row, int c) { return (c ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4; }
};

// The scales of a block, in shared memory: K's of each cell (1 where there is none), the exponent of
// V's one and 2^-that, and which cells are not there.
struct BlockScales {
    float k[8];
    float ev, iv;
    uint32_t gaps, pad;
};
// Two codes as fp16, times a power of two of at most 2^7: V's scale in its cell over the block's one. Exact
// down to 2^-15 of that; beyond, it is rounded to 2^-24 of it.
__device__ __forceinline__ uint32_t decode_by(uint32_t two, __half2 by) { return as_u32(__hmul2(as_half2(kv8_decode(two)), by)); }
// V's one scale of a block: a 128th of the largest that lanes 0 .. 7 have (0: none; 1 if all are).
__device__ __forceinline__ float common_scale(float v)
{
#pragma unroll
    for (int o = 1; o < 8; o <<= 1)
        v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
    return v > 0.0f ? v * 0x1p-7f : 1.0f;
}
__device__ __forceinline__ float pow2_inverse(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

// The codes of a block go to shared memory 16 bytes at a time: K to its rows, V as they are, where piece
// (cell, four channels, t) is the t ^ (cell % 4)th of its four. where: lane z < 8's, the address of cell z
// (0: it is not there, and reads as zeros).
template <int D> __device__ __forceinline__ void copy_block(uint64_t where, const void *pool, uint32_t ks, uint32_t raw, int u)
{
    // of K piece [2 halves][D / 64][8 tokens][4] of a cell, of V piece [D / 4][4]; at D = 64 two cells at once
    const int first = D == 128 ? 0 : u >> 6, piece = u & (D - 1);
    const int g = (piece >> 2) & 7, c = D == 128 ? ((piece >> 5) & 1) * 4 + (piece & 3) : piece & 3, row = (piece / (D / 2)) * 8 + g;
    const uint32_t to_k = ks + row * D + Cfg<D>::piece(row, c), to_v = raw + (piece >> 2) * 64;
#pragma unroll 2
    for (int i = 0; i < D / 16; ++i) {
        const int z = D == 128 ? i : 2 * i + first;
        const uint64_t cell = __shfl_sync(~0u, where, z);
        const uint8_t *const from = cell ? (const uint8_t *)cell + piece * 16 : (const uint8_t *)pool;
        async_copy16(to_k + z * 16 * D, from, cell != 0);
        async_copy16(to_v + z * 16 * D + (((piece & 3) ^ (z & 3)) << 4), cell ? from + Kv8Cell<D>::kV : from, cell != 0);
    }
}
// V^T as fp16 from V's codes: a thread takes four channels of a cell at a time, 16 tokens of each.
// by: lane z < 8's, the factor of cell z. left: tokens of the sequence from the block's first on; past them V is 0,
// whatever is there.
template <int D> __device__ __forceinline__ void unpack_v(uint32_t raw, uint32_t vs, float by, int u, int left)
{
    // lanes that store together differ in the cell (of four) and in the channels' parity, and
    // then in which half of the cell's tokens they store first: no two in one bank
    const int odd = u & 1;
#pragma unroll 1
    for (int i = 0; i < D / 64; ++i) {
        const int four = odd + 2 * ((u >> 3) & 3) + 8 * ((u >> 5) & (D / 32 - 1)); // channels 4 four ..
        const int cell = ((u >> 1) & 3) + 4 * (D == 128 ? i : u >> 6);
        const __half2 f = __float2half2_rn(__shfl_sync(~0u, by, cell));
        uint32_t w[4][4]; // [t][channel]
#pragma unroll
        for (int t = 0; t < 4; ++t)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[t][0]), "=r"(w[t][1]), "=r"(w[t][2]), "=r"(w[t][3])
                         : "r"(raw + cell * 16 * D + four * 64 + ((t ^ (cell & 3)) << 4)));
        const int end = left - cell * 16;
        if (end < 16) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint32_t keep = (2 * t < end ? 0xFFu : 0u) | (2 * t + 1 < end ? 0xFF00u : 0u) |
                                      (2 * t + 8 < end ? 0xFF0000u : 0u) | (2 * t + 9 < end ? 0xFF000000u : 0u);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    w[t][c] &= keep;
            }
        }
        const uint32_t rows = vs + (cell >> 2) * (D * 128) + four * 512;
#pragma unroll 1
        for (int p = 0; p < 2; ++p) {
            const int half = p ^ odd; // tokens 8 half ..
#pragma unroll
            for (int c = 0; c < 4; ++c)
                sts128(rows + c * 128 + (((2 * (cell & 3) + half) ^ (4 * odd + c)) << 4), decode_by(w[0][c] >> (16 * half), f),
                       decode_by(w[1][c] >> (16 * half), f), decode_by(w[2][c] >> (16 * half), f), decode_by(w[3][c] >> (16 * half), f));
        }
    }
}

struct PromptArgs {
    int layer, ratio, n_q_heads;
    const uint16_t *q;
    int64_t q_stride;
    float scale;
    uint16_t *out;
    int64_t out_stride;
    float *lse;
    uint32_t *counters;
    float *partials;
};

// Tokens that tile `tile` of a sequence sees at most (its last row's), 0 for a
// tile without tokens; tt: tokens of a tile.
__device__ __forceinline__ int tile_limit(const Kv4Seq &s, int tile, int tt)
{
    if (tile * tt >= s.n_new)
        return 0;
    const int last = (tile + 1) * tt < s.n_new ? (tile + 1) * tt : s.n_new;
    const int n = s.len - s.n_new + last;
    return n > 0 ? n : 0;
}
__device__ __forceinline__ int blocks_of(int tokens) { return (tokens + kBlock - 1) / kBlock; }
// Blocks of a pair of tiles (one at least, so that rows that see nothing are answered).
__device__ __forceinline__ int pair_blocks(const Kv4Seq &s, int pair, int tt)
{
    const int a = tile_limit(s, 2 * pair, tt), b = tile_limit(s, 2 * pair + 1, tt);
    const int n = blocks_of(a > b ? a : b);
    return n > 0 ? n : 1;
}
__device__ __forceinline__ int pairs_of(const Kv4Seq &s, int tt) { return (s.n_new + 2 * tt - 1) / (2 * tt); }

// A segment takes its blocks and kOver more on the line: what starting and ending a
// piece costs. A step before the first block of a segment is in those.
constexpr int kOver = 3;

// One piece of a CTA's work: blocks [b0, b0 + nblk) of the total of a (sequence, kv
// head, pair); nblk = 0 ends the work.
struct Piece {
    int row, len, n_new, first; // the sequence (Kv4Seq)
    int head, pair, b0, nblk, total;
    int n0, n1;                 // blocks that each tile takes
    int cta0, cta1;             // the CTAs that share the segment
};
constexpr int kRing = 4;        // pieces known ahead

struct Shared {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], raw_full[2];
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2], met[2], scales_full[4];
    uint32_t tmem;
    uint32_t last[2];
    uint64_t piece_full[kRing], piece_empty[kRing];
    Piece piece[kRing];
    BlockScales scales[4]; // of the last blocks: block n's are overwritten by n + 4's, when n + 1 is done
    int64_t total, share;
    int seq, head, pair, step; // where the CTA's part of the line starts
    bool rest;                 // some rows belong to no sequence
};

// A part of a tile: m and l of its 128 rows, then O, four channels of the rows side by side.
__device__ __forceinline__ int part_column(int row, int ch)
{
    return 256 + (ch / 4) * 512 + row * 4;
}

__device__ __forceinline__ float lse_of(float m, float l)
{
    return l == 0.0f ? -INFINITY : (m - kShift + log2f(l)) * kLn2;
}

// 16 channels of a row, times inv, as bf16.
__device__ __forceinline__ void store_row(uint16_t *out, const float (&x)[16], float inv)
{
#pragma unroll
    for (int e = 0; e < 16; e += 8) {
        uint32_t y[4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
            y[n] = f32_to_bf16_rn(x[e + 2 * n] * inv) | ((uint32_t)f32_to_bf16_rn(x[e + 2 * n + 1] * inv) << 16);
        *(uint4 *)(out + e) = make_uint4(y[0], y[1], y[2], y[3]);
    }
}

// Joins a row of the parts of n CTAs of a segment, z, z + step, ... (parts: this tile's slot 0 of
// CTA 0; cta0: the segment's first), into the first of them (final: into out and lse, where they
// are given). Four parts at a time, so that their loads are in flight together. Not inlined: beside
// the softmax loop its registers cost that loop 4% (8192 tokens 548 -> 570 us).
template <int D>
__device__ __noinline__ void join(float *parts, int cta0, int z, int step, int n, int row, bool final, uint16_t *out,
                                      float *lse)
{
    const auto of = [&](int i) {
        const int cta = z + (i < n ? i : n - 1) * step;
        return parts + ((int64_t)cta * 2 + (cta > cta0 ? 0 : 1)) * 2 * Cfg<D>::kPart;
    };
    float m = -INFINITY, l = 0.0f;
#pragma unroll 1
    for (int i = 0; i < n; i += 8) {
        float mz[8], lz[8], top = m;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const float *part = of(i + u);
            mz[u] = __ldcg(part + row);
            lz[u] = __ldcg(part + 128 + row);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            top = fmaxf(top, mz[u]);
        l *= m == top ? 1.0f : exp2_approx(m - top);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (i + u < n)
                l = fmaf(mz[u] == top ? 1.0f : exp2_approx(mz[u] - top), lz[u], l);
        m = top;
    }
    if (lse)
        *lse = lse_of(m, l);
    if (final && !out)
        return;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
    for (int h = 0; h < D / 16; ++h) {
        float x[16] = {};
#pragma unroll 1
        for (int i = 0; i < n; i += 4) {
            float mz[4];
            float4 y[4][4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float *part = of(i + u);
                mz[u] = __ldcg(part + row);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[u][e] = __ldcg((const float4 *)(part + part_column(row, 16 * h + 4 * e)));
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (i + u >= n)
                    break;
                const float f = mz[u] == m ? 1.0f : exp2_approx(mz[u] - m);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[4 * e] = fmaf(f, y[u][e].x, x[4 * e]);
                    x[4 * e + 1] = fmaf(f, y[u][e].y, x[4 * e + 1]);
                    x[4 * e + 2] = fmaf(f, y[u][e].z, x[4 * e + 2]);
                    x[4 * e + 3] = fmaf(f, y[u][e].w, x[4 * e + 3]);
                }
            }
        }
        if (final) {
            store_row(out + 16 * h, x, inv);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *(float4 *)(of(0) + part_column(row, 16 * h + 4 * e)) =
                    make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        }
    }
    if (!final) {
        of(0)[row] = m;
        of(0)[128 + row] = l;
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv8_prompt_kernel(const Kv4 c, const Kv4Batch b, const PromptArgs a)
{
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t dsmem[];
    __shared__ Shared sh;
    uint8_t *const base = dsmem + ((1024u - (smem_addr(dsmem) & 1023u)) & 1023u);
    const uint32_t tiles = smem_addr(base);
    int64_t *const pre = (int64_t *)base;                // [n_seqs + 1], before the tiles are filled
    Kv4Seq *const seqs = (Kv4Seq *)(base + C::kTiles);   // [min(n_seqs, kSeqCache)]
    const auto seq_at = [&](int i) { return b.n_seqs <= kSeqCache ? seqs[i] : kv4_seq(c, b, i, false); };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tt = 128 / a.ratio; // tokens of a tile

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sh.k_full[i]), kUnpack);
            mbar_init(smem_addr(&sh.raw_full[i]), kUnpack);
            mbar_init(smem_addr(&sh.v_full[i]), kUnpack);
            mbar_init(smem_addr(&sh.k_empty[i]), 1);
            mbar_init(smem_addr(&sh.v_empty[i]), 1);
            mbar_init(smem_addr(&sh.q_full[i]), 128);
            mbar_init(smem_addr(&sh.p_full[i]), 128);
            mbar_init(smem_addr(&sh.met[i]), 128);
            mbar_init(smem_addr(&sh.s_full[i]), 1);
            mbar_init(smem_addr(&sh.o_full[i]), 1);
        }
        for (int i = 0; i < 4; ++i)
            mbar_init(smem_addr(&sh.scales_full[i]), 1);
        for (int i = 0; i < kRing; ++i) {
            mbar_init(smem_addr(&sh.piece_full[i]), 1);
            mbar_init(smem_addr(&sh.piece_empty[i]), kMmaWarp + 1); // a lane of each warp that takes pieces
        }
        fence_mbar_init();
    }
    if (warp == kMmaWarp)
        tmem_alloc(smem_addr(&sh.tmem), 512);

    // blocks of each sequence (a warp to a sequence), then where each starts on the line
    for (int i = warp; i < b.n_seqs; i += kThreads / 32) {
        const Kv4Seq s = kv4_seq(c, b, i, blockIdx.x == 0 && lane == 0);
        if (lane == 0 && b.n_seqs <= kSeqCache)
            seqs[i] = s;
        int64_t n = 0;
        for (int j = lane; j < pairs_of(s, tt); j += 32)
            n += pair_blocks(s, j, tt) + kOver;
        for (int o = 16; o; o >>= 1)
            n += __shfl_xor_sync(~0u, n, o);
        if (lane == 0)
            pre[i + 1] = s.first < 0 ? -1 : n * c.n_kv_heads; // -1: starts out of range, no blocks
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 0) {
        int64_t sum = 0;
        bool rest = !kv4_ends(b);
        for (int i0 = 0; i0 < b.n_seqs; i0 += 32) {
            int64_t x = i0 + lane < b.n_seqs ? pre[i0 + lane + 1] : 0;
            rest |= x < 0;
            x = x < 0 ? 0 : x;
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(~0u, x, o);
                if (lane >= o)
                    x += y;
            }
            if (i0 + lane < b.n_seqs)
                pre[i0 + lane + 1] = sum + x;
            sum += __shfl_sync(~0u, x, 31);
        }
        if (lane == 0)
            pre[0] = 0;
        __syncwarp();
        const int64_t total = sum;
        int64_t share = (total + gridDim.x - 1) / gridDim.x;
        share = share < kMinShare + kOver ? kMinShare + kOver : share;
        const int64_t pos = (int64_t)blockIdx.x * share;
        int seq = 0, head = 0, pair = 0, step = 0;
        if (pos < total) {
            int h = b.n_seqs;
            while (h - seq > 1) {
                const int m = (seq + h) >> 1;
                if (pre[m] <= pos)
                    seq = m;
                else
                    h = m;
            }
            const Kv4Seq s = seq_at(seq);
            const int64_t per = (pre[seq + 1] - pre[seq]) / c.n_kv_heads;
            head = (int)((pos - pre[seq]) / per);
            int64_t left = (pos - pre[seq]) % per;
            // the pair that holds step `left` of the head's line
            const int pairs = pairs_of(s, tt);
#pragma unroll 1
            for (int j0 = 0;; j0 += 32) {
                const int n = j0 + lane < pairs ? pair_blocks(s, j0 + lane, tt) + kOver : 0;
                int x = n; // 32 pairs of fewer than 2^24 blocks
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(~0u, x, o);
                    if (lane >= o)
                        x += y;
                }
                const uint32_t in = __ballot_sync(~0u, left < x);
                if (in || j0 + 32 >= pairs) {
                    const int who = in ? __ffs(in) - 1 : 0;
                    pair = j0 + who;
                    step = (int)(left - (__shfl_sync(~0u, x, who) - __shfl_sync(~0u, n, who)));
                    break;
                }
                left -= __shfl_sync(~0u, x, 31);
            }
        }
        rest = __any_sync(~0u, rest);
        if (lane == 0) {
            sh.rest = rest;
            sh.total = total;
            sh.share = share;
            sh.seq = seq;
            sh.head = head;
            sh.pair = pair;
            sh.step = step;
        }
    }
    __syncthreads();
    const uint32_t tmem = sh.tmem;
    if (sh.rest)
        kv4_answer_uncovered(b, a.out, a.out_stride, a.n_q_heads * D, a.lse, a.n_q_heads,
                             (int64_t)blockIdx.x * (kThreads / 32) + warp, (int64_t)gridDim.x * (kThreads / 32));
    bool dead = false;
    const auto wait = [&](uint64_t &bar, uint32_t parity) {
        kv4_wait(smem_addr(&bar), parity & 1u, c.status, dead);
    };
    // Piece number p of the CTA, for a whole warp. After a wait that ran out there are no more:
    // what stands in the ring may be no piece, or half of one.
    const auto get_piece = [&](uint32_t p) {
        wait(sh.piece_full[p % kRing], p / kRing);
        dead = __any_sync(~0u, dead);
        Piece w = sh.piece[p % kRing];
        if (dead)
            w.nblk = w.n0 = w.n1 = 0;
        __syncwarp();
        if (lane == 0)
            kv4_arrive(smem_addr(&sh.piece_empty[p % kRing]));
        return w;
    };

    if (warp < 8) {
        // ---- softmax: a row per thread ----
        setmaxnreg_inc<kSoftRegs>();
        const int k = warp >> 2; // the tile
        const int row = tid & 127;
        const int row_token = row / a.ratio, row_head = row % a.ratio;
        const uint32_t q_tile = tiles + 2 * k * C::kK;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + k * 128, t_o = tmem + lanes + 256 + k * 128;
        const auto count = [&](const Piece &w) { return k ? w.n1 : w.n0; };
        const auto token_of = [&](const Piece &w) { return (2 * w.pair + k) * tt + row_token; };
        const auto valid_in = [&](const Piece &w) { return row < tt * a.ratio && token_of(w) < w.n_new; };
        uint32_t n_s = 0, n_o = 0; // blocks and pieces of this tile so far
        uint32_t n_first = 0;      // blocks of the CTA before the piece

        // The row of Q in its two parts. Returns the factor of the scores.
        const auto load_q = [&](const Piece &w) {
            constexpr int N = D / 8; // 16-byte pieces of a row
            const bool valid = valid_in(w);
            const uint16_t *q = a.q + (int64_t)(w.first + token_of(w)) * a.q_stride + ((int64_t)w.head * a.ratio + row_head) * D;
            uint4 x[N];
#pragma unroll
            for (int i = 0; i < N; ++i)
                x[i] = valid ? ldg_nc128(q + 8 * i) : make_uint4(0, 0, 0, 0);
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < N; ++i)
                top = max(top, kv8_magnitude(x[i]));
            const Kv8Row of = kv8_row(top, a.scale, w.len - w.n_new + token_of(w) >= 0);
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                uint2 hi[2], lo[2]; // of 16 channels
                kv8_split(x[i], of.down, hi[0], lo[0]);
                kv8_split(x[i + 1], of.down, hi[1], lo[1]);
                const uint32_t at = q_tile + row * D + C::piece(row, i / 2);
                sts128(at, hi[0].x, hi[0].y, hi[1].x, hi[1].y);
                sts128(at + C::kK, lo[0].x, lo[0].y, lo[1].x, lo[1].y);
            }
            fence_proxy_async_smem();
            kv4_arrive(smem_addr(&sh.q_full[k]));
            return of.factor;
        };

        // The rows of O of a piece.
        const auto finish = [&](const Piece &done, int nk, float m, float l) {
            if (l == 0.0f)
                m = -INFINITY; // nothing seen
            if (nk > 0) {
                wait(sh.o_full[k], n_o);
                ++n_o;
                fence_after();
            }
            const int64_t token = done.first + token_of(done);
            const int head = done.head * a.ratio + row_head;
            const bool valid = valid_in(done);
            const bool whole = done.nblk == done.total;
            uint16_t *out = a.out + token * a.out_stride + (int64_t)head * D;
            float *lse = a.lse && valid ? a.lse + token * a.n_q_heads + head : nullptr;
            // a part: m, l of the rows, then O, four channels of the rows side by side. A CTA has at
            // most one piece that goes on from another's (slot 0) and one that another goes on from.
            const auto part_at = [&](int cta, int slot) {
                return a.partials + (((int64_t)cta * 2 + slot) * 2 + k) * C::kPart;
            };
            if (!whole) {
                float *part = part_at(blockIdx.x, done.b0 > 0 ? 0 : 1);
                part[row] = m;
                part[128 + row] = l;
#pragma unroll 1
                for (int h = 0; h < D / 16; ++h) {
                    uint32_t o[16] = {};
                    if (nk > 0) {
                        ld16(t_o + 16 * h, o);
                        wait_ld();
                        tie<16>(o);
                    }
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *(uint4 *)(part + part_column(row, 16 * h + e)) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
                // The parts of this tile are joined by the last CTA to arrive, in CTA order: of many,
                // first in groups of g (at most 16 to a join), then the groups (32 new tokens after
                // 32768 by one join of 32 parts: 77 us). The tile's threads meet on an mbarrier, whose
                // wait is bounded: after one that ran out, warps may be missing.
                const auto meet = [&]() { kv4_meet(smem_addr(&sh.met[k]), c.status, dead); };
                const auto last_of = [&](uint32_t *counter, int n) {
                    meet();
                    if (row == 0) {
                        const uint32_t before = n > 1 ? atom_add_acq_rel_gpu(counter, 1u) : 0;
                        sh.last[k] = before == (uint32_t)n - 1;
                        if (n > 1 && sh.last[k])
                            *counter = 0; // for the next launch
                    }
                    meet();
                    dead = __any_sync(~0u, dead);
                    return !dead && sh.last[k] != 0;
                };
                const int n = done.cta1 - done.cta0 + 1;
                const int g = n <= 8 ? n : n <= 16 ? 4 : n <= 64 ? 8 : n <= 144 ? 12 : (n + 15) / 16;
                const int z = (int)blockIdx.x - (int)(blockIdx.x - done.cta0) % g; // the group's first
                const int in = g < done.cta1 - z + 1 ? g : done.cta1 - z + 1, groups = (n + g - 1) / g;
                // a group of one has no counter: its CTA may be the first of the next segment
                bool all = last_of(a.counters + 2 * z + k, in);
                if (all && groups > 1) {
                    if (in > 1)
                        join<D>(part_at(0, 0), done.cta0, z, 1, in, row, false, nullptr, nullptr);
                    all = last_of(a.counters + kKv4Counters / 2 + 2 * done.cta0 + k, groups);
                }
                if (all)
                    join<D>(part_at(0, 0), done.cta0, done.cta0, groups > 1 ? g : 1, groups > 1 ? groups : n, row, true,
                                valid ? out : nullptr, lse);
                fence_before(); // the next MMAs on O follow this thread's next arrival
                return;
            }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            if (lse)
                *lse = lse_of(m, l);
#pragma unroll 1
            for (int h = 0; h < D / 16; ++h) {
                uint32_t o[16] = {};
                if (nk > 0) {
                    ld16(t_o + 16 * h, o);
                    wait_ld();
                    tie<16>(o);
                }
                float x[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    x[e] = __uint_as_float(o[e]);
                if (valid)
                    store_row(out + 16 * h, x, inv);
            }
            fence_before();
        };

        // Q of a piece is loaded while the last MMAs of the one before run. Pieces stay in the ring until they
        // are finished, and are read there: in registers they would be held across the softmax.
        float rs = 1.0f, m = 0.0f, l = 0.0f;
        int nk = 0;
#pragma unroll 1
        for (uint32_t piece = 0;; ++piece) {
            wait(sh.piece_full[piece % kRing], piece / kRing);
            dead = __any_sync(~0u, dead);
            const Piece &w = sh.piece[piece % kRing];
            const bool none = dead || w.nblk == 0; // as in get_piece
            const int n_done = nk;
            nk = none ? 0 : count(w);
            if (nk > 0)
                rs = load_q(w);
            if (piece > 0) {
                finish(sh.piece[(piece - 1) % kRing], n_done, m, l);
                __syncwarp();
                if (lane == 0)
                    kv4_arrive(smem_addr(&sh.piece_empty[(piece - 1) % kRing]));
            }
            if (none)
                break;
            const int limit = valid_in(w) ? w.len - w.n_new + token_of(w) + 1 : 0;
            // rows that see nothing of the piece need no maximum
            m = limit > w.b0 * kBlock ? -INFINITY : 0.0f;
            l = 0.0f;
#pragma unroll 1
            for (int i = 0; i < nk; ++i, ++n_s) {
                const uint32_t n_blk = n_first + i;
                wait(sh.s_full[k], n_s);
                wait(sh.scales_full[n_blk & 3], n_blk >> 2); // they are there: their K was unpacked
                fence_after();
                const int vis = limit - (w.b0 + i) * kBlock; // columns this row sees
                const BlockScales &bs = sh.scales[n_blk & 3];
                const float ev = bs.ev;
                const uint32_t gaps = bs.gaps;
                // Only the last blocks of a row are masked, as a rule, and blocks with cells that are not there.
                const bool masked = !__all_sync(~0u, vis >= kBlock && gaps == 0);
                uint32_t r[32];
                const auto read = [&](int h) { // columns 32 h ..
                    ld32(t_s + 32 * h, r);
                    wait_ld();
                    tie<32>(r);
                };
                // S is read twice, 32 columns at a time: for the maximum, which is raised when a score passes
                // it by more than the slack, and for the weights. Loops, so that the code stays in the
                // instruction caches beside the other roles'.
                float mx = -INFINITY;
#pragma unroll 1
                for (int h = 0; h < 4; ++h) {
                    read(h);
                    if (masked) { // once: they are written back
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const int end = gaps >> (2 * h + z) & 1u ? 0 : vis - 32 * h - 16 * z;
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                r[16 * z + e] = e < end ? r[16 * z + e] : 0xFF800000u;
                            st16(t_s + 32 * h + 16 * z, r + 16 * z);
                        }
                        wait_st();
                    }
                    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        top[e / 16] = fmaxf(fmaxf(top[e / 16], __uint_as_float(r[e])), __uint_as_float(r[e + 1]));
                    mx = fmaxf(mx, fmaxf(top[0] * bs.k[2 * h], top[1] * bs.k[2 * h + 1]));
                }
                mx = fmaf(mx, rs, ev);
                if (__any_sync(~0u, mx > m + kSlack)) {
                    const float mn = fmaxf(m, mx);
                    const float f = mn == m ? 1.0f : exp2_approx(m - mn);
                    m = mn;
                    l *= f;
                    if (i > 0) {
#pragma unroll 1
                        for (int h = 0; h < D / 16; ++h) {
                            uint32_t o[16];
                            ld16(t_o + 16 * h, o);
                            wait_ld();
                            tie<16>(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            st16(t_o + 16 * h, o);
                        }
                    }
                }
                const float off = kShift - (m == -INFINITY ? 0.0f : m) + ev;
                const uint64_t off2 = pair(off, off);
                uint64_t sum2[2] = {0, 0};
#pragma unroll 1
                for (int h = 0; h < 4; ++h) {
                    const float f[2] = {rs * bs.k[2 * h], rs * bs.k[2 * h + 1]};
                    read(h);
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float x, y;
                        unpair(fma2(pair(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), pair(f[e / 16], f[e / 16]), off2), x, y);
                        x = exp2_approx(x);
                        y = exp2_approx(y);
                        sum2[(e / 2) & 1] = add2(sum2[(e / 2) & 1], pair(x, y));
                        p[e / 2] = pack_half2(x, y);
                    }
                    st16(t_s + 16 * h, p);
                }
                float x, y;
                unpair(add2(sum2[0], sum2[1]), x, y);
                l = fmaf(x + y, bs.iv, l);
                wait_st();
                fence_before();
                kv4_arrive(smem_addr(&sh.p_full[k]));
            }

            n_first += w.nblk;
        }
    } else if (warp < kMmaWarp) {
        setmaxnreg_dec<kUnpackRegs>();
        // ---- the codes: block n's are asked for, and block n - 1's V^T made, a round ----
        const int u = tid - kSoft;
        const int in_page = c.page_shift - 4;
        uint32_t piece = 0, n = 0; // n: blocks asked for
        Piece w{};
        int i = -1, page = -2; // the block to ask for next, and its pages (lane z < 8's: that of cell z; -2: none)
        int left = 0;    // tokens of the last one's sequence from its first on
        float by = 0.0f; // lane z < 8: its cell z's factor of V
        bool more;
#pragma unroll 1
        do {
            more = w.nblk > 0 && i >= 0;
            uint64_t where = 0;
            if (page >= 0 && page < c.n_pages)
                where = (uint64_t)(c.pool + kv8_head_offset<D>(c, page, a.layer, w.head) +
                                   (((w.b0 + i) * 8 + (lane & 7)) & ((1 << in_page) - 1)) * Kv8Cell<D>::kBytes);
            else if (page != -2 && u < 8)
                kv4_bad(c);
            // 0: the cell is not there
            const float2 scales =
                where ? __ldg((const float2 *)((const uint8_t *)where + Kv8Cell<D>::kScales)) : make_float2(0.0f, 0.0f);
            const int now_left = w.len - (w.b0 + i) * kBlock;
            // the pages of the next block are asked for before this one is worked on
            if (++i == w.nblk) { // at first there is no piece
                i = 0;
                w = get_piece(piece++);
            }
            page = -2;
            const int next = (w.b0 + i) * 8 + (lane & 7);
            if (w.nblk > 0 && next * kKv4Cell < w.len)
                page = max(c.tables[(int64_t)w.row * c.max_pages + (next >> in_page)], -1);
            const uint32_t st = n & 1;
            float next_by = 0.0f;
            if (more) {
                // K's place is free when S has been computed of block n - 2, V's when all have made its V^T
                if (n >= 2) {
                    wait(sh.k_empty[st], (n >> 1) - 1);
                    wait(sh.v_full[st], (n >> 1) - 1);
                }
                copy_block<D>(where, c.pool, tiles + C::kOffK + st * C::kK, tiles + C::kOffRaw + st * C::kK, u);
                async_copies_arrive(smem_addr(&sh.k_full[st]));
                async_copies_arrive(smem_addr(&sh.raw_full[st]));
                const float v = common_scale(scales.y);
                if (u < 32) {
                    BlockScales &bs = sh.scales[n & 3];
                    const uint32_t gaps = __ballot_sync(~0u, scales.x == 0.0f) & 0xFFu;
                    if (u < 8)
                        bs.k[u] = scales.x == 0.0f ? 1.0f : scales.x;
                    __syncwarp();
                    if (u == 0) {
                        bs.ev = (float)((int)(__float_as_uint(v) >> 23) - 127);
                        bs.iv = pow2_inverse(v);
                        bs.gaps = gaps;
                        kv4_arrive(smem_addr(&sh.scales_full[n & 3]));
                    }
                }
                next_by = scales.y * pow2_inverse(v);
            }
            if (n >= 1 && (more || w.nblk == 0)) {
                const uint32_t was = st ^ 1;
                wait(sh.raw_full[was], (n - 1) >> 1);
                if (n >= 3)
                    wait(sh.v_empty[was], ((n - 1) >> 1) - 1);
                unpack_v<D>(tiles + C::kOffRaw + was * C::kK, tiles + C::kOffV + was * C::kV, by, u, left);
                fence_proxy_async_smem();
                kv4_arrive(smem_addr(&sh.v_full[was]));
            }
            if (more) {
                by = next_by;
                left = now_left;
                ++n;
            }
        } while (w.nblk > 0 || more);
        async_copies_wait(); // there are some in flight only after a wait that ran out
    } else {
        // one instruction for the warpgroup: its warps have to meet in the same one
        setmaxnreg_dec<kMmaRegs>();
        if (warp == kMmaWarp + 1) {
            // ---- the pieces, one lane ----
            if (lane == 0) {
                const int64_t share = sh.share;
                int64_t pos = (int64_t)blockIdx.x * share;
                const int64_t hi = pos + share < sh.total ? pos + share : sh.total;
                int seq = sh.seq, head = sh.head, pair = sh.pair, step = sh.step;
                Kv4Seq s = pos < hi ? seq_at(seq) : Kv4Seq{};
#pragma unroll 1
                for (uint32_t p = 0;; ++p) {
                    Piece w{};
                    if (pos < hi) {
                        w.row = s.row;
                        w.len = s.len;
                        w.n_new = s.n_new;
                        w.first = s.first;
                        w.head = head;
                        w.pair = pair;
                        w.total = pair_blocks(s, pair, tt);
                        const int64_t seg = pos - step + kOver; // the place of the segment's first block
                        const int all = w.total + kOver - step;
                        const int steps = hi - pos < all ? (int)(hi - pos) : all;
                        w.b0 = step > kOver ? step - kOver : 0;
                        const int b1 = step + steps - kOver;
                        w.nblk = b1 > w.b0 ? b1 - w.b0 : 0; // 0: the CTA's part ends before the first block
                        const int n0 = blocks_of(tile_limit(s, 2 * pair, tt)) - w.b0;
                        const int n1 = blocks_of(tile_limit(s, 2 * pair + 1, tt)) - w.b0;
                        w.n0 = n0 < 0 ? 0 : n0 > w.nblk ? w.nblk : n0;
                        w.n1 = n1 < 0 ? 0 : n1 > w.nblk ? w.nblk : n1;
                        w.cta0 = (int)(seg / share);
                        w.cta1 = (int)((seg + w.total - 1) / share);
                        pos += steps;
                        step = 0;
                        if (pos < hi && ++pair == pairs_of(s, tt)) {
                            pair = 0;
                            if (++head == c.n_kv_heads) {
                                head = 0;
                                do
                                    s = seq_at(++seq);
                                while (s.n_new == 0); // pos < hi: there is one
                            }
                        }
                    }
                    if (p >= kRing)
                        wait(sh.piece_empty[p % kRing], p / kRing - 1);
                    if (dead)
                        break; // the place may still be read
                    sh.piece[p % kRing] = w;
                    kv4_arrive(smem_addr(&sh.piece_full[p % kRing]));
                    if (w.nblk == 0)
                        break;
                }
            }
        } else if (warp == kMmaWarp) {
            // ---- the MMAs: every lane follows, one issues ----
            const uint32_t one = elect();
            constexpr uint32_t tmem = 0; // all 512 columns are this kernel's: they start at 0

            uint32_t n = 0, n_p0 = 0, n_p1 = 0, n_q0 = 0, n_q1 = 0;
            const uint32_t desc0 = kDescLo | (tiles >> 4);
            const auto scores = [&](int k, int stage) { // S of tile k, K in `stage`
                const uint32_t q = desc0 + k * (2 * C::kK >> 4), kk = desc0 + (C::kOffK >> 4) + stage * (C::kK >> 4);
                const uint32_t d = tmem + k * 128;
#pragma unroll 1
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int x = 0; x < D / 32; ++x)
                        mma_ss_f8<D>(d, q + ((part * C::kK + 32 * x) >> 4), kk + ((32 * x) >> 4),
                                     kIdesc<128> | (part ? kE5m2A : 0u), part + x, one);
                commit(smem_addr(&sh.s_full[k]), one);
            };
            const auto values = [&](int k, int stage, uint32_t accumulate) { // O of tile k, V in `stage`
                const uint32_t v = desc0 + (C::kOffV >> 4) + stage * (C::kV >> 4);
                const uint32_t d = tmem + 256 + k * 128, p = tmem + k * 128;
#pragma unroll 1
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        mma_ts(d, p + 32 * h + 8 * x, v + ((h * (D * 128) + 32 * x) >> 4), kIdesc<D>,
                               h + x > 0 ? 1u : accumulate, one);
            };
            // O of block i of a piece (block n - 1 of the CTA), then S of block i + 1 (block n), tile by
            // tile: one copy of this for both (two, and two of each for the stages: 521 against 502 us at 8192 tokens).
            int nblk, n0, n1;
            const auto step = [&](int i) {
                const int nxt = __shfl_sync(~0u, n & 1, 0), cur = nxt ^ 1;
                const bool more = i + 1 < nblk;
                if (i >= 0)
                    wait(sh.v_full[cur], (n - 1) >> 1);
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {
                    const int nk = k ? n1 : n0;
                    if (i >= 0 && i < nk) {
                        wait(sh.p_full[k], k ? n_p1 : n_p0);
                        n_p0 += 1 - k;
                        n_p1 += k;
                        fence_after();
                        values(k, cur, i > 0);
                        if (i == nk - 1)
                            commit(smem_addr(&sh.o_full[k]), one);
                    }
                    if (more) {
                        if (k == 0) {
                            wait(sh.k_full[nxt], n >> 1);
                            fence_proxy_async_smem(); // copies wrote K: the threads that asked for them have gone on
                        }
                        if (i + 1 < nk) {
                            if (i < 0) {
                                wait(sh.q_full[k], k ? n_q1 : n_q0);
                                n_q0 += 1 - k;
                                n_q1 += k;
                            }
                            fence_after();
                            scores(k, nxt);
                        }
                    }
                }
                if (i >= 0)
                    commit(smem_addr(&sh.v_empty[cur]), one);
                if (more) {
                    commit(smem_addr(&sh.k_empty[nxt]), one);
                    ++n;
                }
            };
            uint32_t piece = 0;
#pragma unroll 1
            for (;;) {
                wait(sh.piece_full[piece % kRing], piece / kRing);
                dead = __any_sync(~0u, dead);
                nblk = dead ? 0 : sh.piece[piece % kRing].nblk; // as in get_piece
                n0 = sh.piece[piece % kRing].n0;
                n1 = sh.piece[piece % kRing].n1;
                __syncwarp();
                if (one)
                    kv4_arrive(smem_addr(&sh.piece_empty[piece % kRing]));
                ++piece;
                if (nblk == 0)
                    break;
#pragma unroll 1
                for (int i = -1; i < nblk; ++i) {
                    step(i);
                }
            }
            // before leaving, the MMAs in flight end (bounded, after a wait that ran out too): the last
            // stages are released
            if (n > 0) {
                dead = false;
                wait(sh.k_empty[(n - 1) & 1], (n - 1) >> 1);
                wait(sh.v_empty[(n - 1) & 1], (n - 1) >> 1);
            }
        }
    }
    fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        __syncwarp();
        tmem_dealloc(tmem, 512);
    }
}

template <int D> nm_status launch(const Kv4 &c, const Kv4Batch &b, const PromptArgs &a, const Kv4Work &w, cudaStream_t st)
{
    constexpr size_t kMax = Cfg<D>::kTiles + 1024 + kSeqCache * sizeof(Kv4Seq);
    static_assert(kMax + sizeof(Shared) <= 227 * 1024, "shared memory");
    static OncePerDevice once;
    if (!once(w.device, [] {
            return cudaFuncSetAttribute(kv8_prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMax) ==
                   cudaSuccess;
        }))
        return NM_ERR_CUDA;
    const size_t smem =
        Cfg<D>::kTiles + 1024 + (size_t)(b.n_seqs < kSeqCache ? b.n_seqs : kSeqCache) * sizeof(Kv4Seq);
    const int grid = w.num_sms < kKv4PromptCtas ? w.num_sms : kKv4PromptCtas;
    kv8_prompt_kernel<D><<<grid, kThreads, smem, st>>>(c, b, a);
    return cudaGetLastError() == cudaSuccess ? NM_OK : NM_ERR_CUDA;
}

} // namespace

size_t kv8_prompt_partial_bytes(int head_dim) { return (size_t)kKv4PromptCtas * 4 * 128 * (head_dim + 2) * 4; }

nm_status kv8_launch_prompt(const Kv4 &c, const Kv4Batch &b, const Kv4Attn &at, const Kv4Work &w, cudaStream_t st)
{
    const PromptArgs a{at.layer, at.n_q_heads / c.n_kv_heads, at.n_q_heads, (const uint16_t *)at.q, at.q_stride,
                       at.scale, (uint16_t *)at.out, at.out_stride, at.lse, w.counters, w.partials};
    return c.head_dim == 128 ? launch<128>(c, b, a, w, st) : launch<64>(c, b, a, w, st);
}

} // namespace nm
