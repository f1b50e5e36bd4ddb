// kv8_prompt.cu -- attention of many queries over the 8-bit paged cache (prompts), on
// the 5th-generation tensor cores.
//
// For one sequence and kv head the rows are its new tokens times the query heads that
// share the kv head. A CTA works on a pair of 128-row tiles at a time and walks the
// tokens they see in blocks of 128:
//
//   S = Q codes(K)^T    tcgen05.mma, Q and K in shared memory, S in tensor memory
//   P = 2^(S r s_K + e - m + 6)  one row per thread, written back to tensor memory as fp16
//   O += P codes(V)     tcgen05.mma, P from tensor memory, V^T in shared memory
//
// Both operands of S are exact in fp16: the codes, and q scaled by a power of two per row.
// The scales are powers of two of each cell (16 tokens): K's multiplies the scores in the
// softmax, V's (2^e) is an exponent of the weights, and the sums of the weights are freed of it
// again, sixteen columns at a time. Scores carry fp32 rounding only, as in the kernel for few rows.
//
// Roles (20 warps): two softmax warpgroups, one per tile (a thread owns a row: no
// reductions across threads; it also loads and scales its row of Q, rescales and
// stores its row of O); two warpgroups that make the codes fp16 in two stages of K
// and of V^T (both tiles use them); one warp that issues the MMAs; one that lists
// the pieces of work. While one tile is in its softmax, the other's MMAs run. The
// running maximum is raised only when a score passes it by 2^8, so O is rarely
// rescaled. The next block's bytes are in the unpacking threads' registers before
// the current one is written.
//
// The blocks of all (sequence, kv head, pair) segments are one line, on which a
// segment takes kOver blocks more (what starting and ending a piece costs), cut evenly
// over one CTA per SM; a segment that was cut is joined, row by row, by the last
// CTAs to arrive of groups of its parts and then of the groups, in CTA order.
//
// All waits are bounded; one that runs out sets NM_ERR_TIMEOUT. Its thread's later waits
// poll once and its warp takes no more pieces, so the others run out in turn, the MMAs
// in flight end, and the kernel frees its tensor memory and returns.
#include <type_traits>

#include "kv8.cuh"
#include "kv_ops.cuh"

namespace nm {
namespace {

constexpr int kSoft = 256;      // softmax threads: two tiles of 128 rows
constexpr int kUnpack = 256;    // unpacking threads
constexpr int kMmaWarp = 16;    // of its warpgroup, the next one lists the pieces and two idle
constexpr int kThreads = 640;
// Registers of a thread: at launch (what 640 threads can have), and in each role.
constexpr int kLaunchRegs = 96, kSoftRegs = 160, kUnpackRegs = 64, kMmaRegs = 32;
static_assert(kSoftRegs >= kLaunchRegs && kUnpackRegs <= kLaunchRegs && kMmaRegs <= kLaunchRegs &&
                  kSoft * kSoftRegs + kUnpack * kUnpackRegs + 128 * kMmaRegs <= kThreads * kLaunchRegs,
              "a role that takes registers waits until others have given them back");
constexpr int kSeqCache = 512;  // sequences whose descriptors are kept in shared memory
constexpr int kBlock = 128;    // tokens of a block
constexpr int kMinShare = 2;   // blocks of a CTA at least
constexpr int kSub = 128 * 128; // bytes of 128 rows of 64 fp16
constexpr float kShift = 6.0f, kSlack = 8.0f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int D> struct Cfg {
    static constexpr int G = D / 64;
    static constexpr int kQ = G * kSub;          // a tile of Q, and a stage of K
    static constexpr int kV = 2 * D * 128;       // a stage of V^T: two halves of 64 tokens
    static constexpr int kOffK = 2 * kQ, kOffV = kOffK + 2 * kQ, kTiles = kOffV + 2 * kV;
    static constexpr int kPart = 128 * (D + 2);  // floats of a tile's part
};

// What an unpacking thread u holds of a block. K: 64 channels of row u / G (at D = 64 of the first 128
// threads). V: the cell u / (D / 4), channels 4 (u % (D / 4)) .. of its 16 tokens (at D = 64, of the first
// 128 threads too). Both are 64 bytes side by side.
struct Codes {
    uint4 w[4];
};
// The scales of a block's cells, in shared memory: of K, V's exponent, and 2^-that. Cells that are not
// there have the factor -1.
struct CellScales {
    float k, ev, iv, pad;
};
template <int D> __device__ __forceinline__ bool unpacks(int u) { return u < 128 * Cfg<D>::G; }
template <int D> __device__ __forceinline__ void load_k(Codes &r, uint64_t where, int u)
{
    constexpr int G = Cfg<D>::G;
    const int row = u / G, j = u % G;
    const uint64_t cell = __shfl_sync(~0u, where, (row >> 4) & 7);
    const uint8_t *const src = (const uint8_t *)cell + ((row >> 3) & 1) * 8 * D + j * 512 + (row & 7) * 64;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r.w[i] = cell && unpacks<D>(u) ? ldg_nc128(src + 16 * i) : make_uint4(0, 0, 0, 0);
}
template <int D> __device__ __forceinline__ void unpack_k(const Codes &r, uint32_t ks, int u)
{
    constexpr int G = Cfg<D>::G;
    if (!unpacks<D>(u))
        return;
    const int row = u / G, j = u % G;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
        for (int f = 0; f < 2; ++f)
            sts128(ks + j * kSub + row * 128 + (((2 * i + f) ^ (row & 7)) << 4), kv8_decode(w[2 * f]),
                   kv8_decode(w[2 * f] >> 16), kv8_decode(w[2 * f + 1]), kv8_decode(w[2 * f + 1] >> 16));
    }
}
template <int D> __device__ __forceinline__ void load_v(Codes &r, uint64_t where, int u)
{
    const uint64_t cell = __shfl_sync(~0u, where, (u / (D / 4)) & 7);
    const uint8_t *const src = (const uint8_t *)cell + Kv8Cell<D>::kV + (u % (D / 4)) * 64;
#pragma unroll
    for (int t = 0; t < 4; ++t)
        r.w[t] = cell && unpacks<D>(u) ? ldg_nc128(src + 16 * t) : make_uint4(0, 0, 0, 0);
}
// left: tokens of the sequence from the block's first on; past them V is 0, whatever is there.
template <int D> __device__ __forceinline__ void unpack_v(const Codes &r, uint32_t vs, int u, int left)
{
    if (!unpacks<D>(u))
        return;
    const int cell = u / (D / 4), ch0 = 4 * (u % (D / 4)), tok = cell * 16;
    const uint32_t dst = vs + (cell >> 2) * (D * 128) + ch0 * 128;
    uint32_t keep[4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
        keep[t] = tok + 16 <= left ? ~0u
                                   : (tok + 2 * t < left ? 0xFFu : 0u) | (tok + 2 * t + 1 < left ? 0xFF00u : 0u) |
                                         (tok + 2 * t + 8 < left ? 0xFF0000u : 0u) | (tok + 2 * t + 9 < left ? 0xFF000000u : 0u);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int ch = ch0 + c; // of its row's 16-byte pieces (8 tokens), 2 (cell % 4) + p
        uint32_t w[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
            w[t] = (c == 0 ? r.w[t].x : c == 1 ? r.w[t].y : c == 2 ? r.w[t].z : r.w[t].w) & keep[t];
#pragma unroll
        for (int p = 0; p < 2; ++p)
            sts128(dst + c * 128 + (((2 * (cell & 3) + p) ^ (ch & 7)) << 4), kv8_decode(w[0] >> (16 * p)),
                   kv8_decode(w[1] >> (16 * p)), kv8_decode(w[2] >> (16 * p)), kv8_decode(w[3] >> (16 * p)));
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
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2], met[2], scales_full[4];
    uint32_t tmem;
    uint32_t last[2];
    uint64_t piece_full[kRing], piece_empty[kRing];
    Piece piece[kRing];
    CellScales scales[4][8]; // of the last blocks' cells: block n's are overwritten by n + 4's, when n + 1 is done
    bool gaps[4];            // whether some of a block's cells are not there
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
    constexpr int G = C::G;
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
        const uint32_t q_tile = tiles + k * C::kQ;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + k * 128, t_o = tmem + lanes + 256 + k * 128;
        const auto count = [&](const Piece &w) { return k ? w.n1 : w.n0; };
        const auto token_of = [&](const Piece &w) { return (2 * w.pair + k) * tt + row_token; };
        const auto valid_in = [&](const Piece &w) { return row < tt * a.ratio && token_of(w) < w.n_new; };
        uint32_t n_s = 0, n_o = 0; // blocks and pieces of this tile so far
        uint32_t n_first = 0;      // blocks of the CTA before the piece

        // The row of Q, scaled by a power of two. Returns the factor of the scores.
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
            for (int i = 0; i < N; ++i) {
                const uint32_t ws[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    top = max(top, max(ws[n] & 0x7FFF0000u, (ws[n] << 16) & 0x7FFF0000u));
            }
            uint32_t e2 = top >> 23;
            e2 = e2 == 0xFFu || e2 == 0 ? 127u : e2 > 253u ? 253u : e2;
            const float up = __uint_as_float(e2 << 23);
            const float down = a.scale < 0.0f ? -__uint_as_float((254u - e2) << 23) : __uint_as_float((254u - e2) << 23);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t ws[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                uint32_t y[4];
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    y[n] = pack_half2(bf16lo_to_f32(ws[n]) * down, bf16hi_to_f32(ws[n]) * down);
                sts128(q_tile + (i >> 3) * kSub + row * 128 + (((i & 7) ^ (row & 7)) << 4), y[0], y[1], y[2], y[3]);
            }
            fence_proxy_async_smem();
            kv4_arrive(smem_addr(&sh.q_full[k]));
            return fmaxf(up * (fabsf(a.scale) * kLog2e), 1e-30f); // above 0, so that masked scores stay -inf
        };

        // The rows of O of a piece.
        const auto finish = [&](const Piece &done, float m, float l) {
            const int nk = count(done);
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

        // Q of a piece is loaded while the last MMAs of the one before run
        float rs = 1.0f, m = 0.0f, l = 0.0f;
        Piece done{};
#pragma unroll 1
        for (uint32_t piece = 0;; ++piece) {
            const Piece w = get_piece(piece);
            if (count(w) > 0)
                rs = load_q(w);
            if (piece > 0)
                finish(done, m, l);
            if (w.nblk == 0)
                break;
            const int nk = count(w);
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
                const CellScales *const cells = sh.scales[n_blk & 3];
                // only the last blocks of a row are masked, and blocks with cells that are not there
                const bool masked = !__all_sync(~0u, vis >= kBlock) || sh.gaps[n_blk & 3];
                const auto mask = [&](uint32_t *r, int h) { // columns 32 h ..
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const int end = cells[2 * h + z].k < 0.0f ? 0 : vis - 32 * h - 16 * z;
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            r[16 * z + e] = e < end ? r[16 * z + e] : 0xFF800000u;
                    }
                };
                // S is read twice, 64 columns at a time: for the maximum, then for the weights. The maximum is
                // raised when a score passes it by more than the slack.
                uint32_t r[2][32];
                const auto read = [&](int h) { // columns 32 h .. 32 h + 63
                    ld32(t_s + 32 * h, r[0]);
                    ld32(t_s + 32 * h + 32, r[1]);
                    wait_ld();
                    tie<32>(r[0]);
                    tie<32>(r[1]);
                    if (masked) {
                        mask(r[0], h);
                        mask(r[1], h + 1);
                    }
                };
                float mx = -INFINITY;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    if (h % 2 == 0)
                        read(h);
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const uint32_t *const x = r[h & 1] + 16 * z;
                        float top[2] = {__uint_as_float(x[0]), __uint_as_float(x[1])};
#pragma unroll
                        for (int e = 2; e < 14; e += 4) {
                            top[0] = fmaxf(fmaxf(top[0], __uint_as_float(x[e])), __uint_as_float(x[e + 1]));
                            top[1] = fmaxf(fmaxf(top[1], __uint_as_float(x[e + 2])), __uint_as_float(x[e + 3]));
                        }
                        top[0] = fmaxf(fmaxf(top[0], __uint_as_float(x[14])), __uint_as_float(x[15]));
                        const CellScales &cs = cells[2 * h + z];
                        mx = fmaxf(mx, fmaf(fmaxf(top[0], top[1]), rs * fabsf(cs.k), cs.ev));
                    }
                }
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
                const float off = kShift - (m == -INFINITY ? 0.0f : m);
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    if (h % 2 == 0)
                        read(h);
                    uint32_t p[16];
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const uint32_t *const s = r[h & 1] + 16 * z;
                        const CellScales cs = cells[2 * h + z];
                        const float rk = rs * fabsf(cs.k), at = off + cs.ev;
                        const uint64_t rk2 = pair(rk, rk), at2 = pair(at, at);
                        uint64_t sum2[2] = {0, 0};
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            float x, y;
                            unpair(fma2(pair(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), rk2, at2), x, y);
                            x = exp2_approx(x);
                            y = exp2_approx(y);
                            sum2[(e / 2) & 1] = add2(sum2[(e / 2) & 1], pair(x, y));
                            p[8 * z + e / 2] = pack_half2(x, y);
                        }
                        float x, y;
                        unpair(add2(sum2[0], sum2[1]), x, y);
                        l = fmaf(x + y, cs.iv, l);
                    }
                    st16(t_s + 16 * h, p);
                }
                wait_st();
                fence_before();
                kv4_arrive(smem_addr(&sh.p_full[k]));
            }

            n_first += w.nblk;
            done = w;
        }
    } else if (warp < kMmaWarp) {
        setmaxnreg_dec<kUnpackRegs>();
        // ---- unpacking: 256 threads fill K and V^T of a block ----
        const int u = tid - kSoft;
        const int in_page = c.page_shift - 4;
        Codes rk, rv;
        float2 scales = make_float2(-1.0f, 1.0f); // lane z < 8 of the first warp: cell z's
        uint32_t piece = 0;
        Piece w = get_piece(piece);
        int i = 0;        // the block to fetch: b0 + i of piece w
        int left = 0;     // tokens of the fetched block's sequence from its first on
        uint32_t n = ~0u; // the number of the fetched block; none yet
        bool more = w.nblk > 0;
#pragma unroll 1
        for (;;) {
            // Block n (fetched before) is unpacked, and the next one fetched, K and V in turn:
            // each one's registers are free as soon as it is in shared memory. Lane z < 8 asks
            // for the page of cell z first, and finds where it is (0: nowhere).
            const int cell = (w.b0 + i) * 8 + (lane & 7);
            const bool inside = more && cell * kKv4Cell < w.len;
            const int32_t page = inside ? c.tables[(int64_t)w.row * c.max_pages + (cell >> in_page)] : -1;
            const int st = n & 1;
            if (n != ~0u) {
                if (n >= 2)
                    wait(sh.k_empty[st], (n >> 1) - 1);
                unpack_k<D>(rk, tiles + C::kOffK + st * C::kQ, u);
                if (u < 32) {
                    if (u < 8) {
                        const uint32_t e = __float_as_uint(scales.y);
                        sh.scales[n & 3][u] = CellScales{scales.x, (float)((int)(e >> 23) - 127), __uint_as_float((254u << 23) - e), 0.0f};
                    }
                    const bool gaps = __any_sync(~0u, u < 8 && scales.x < 0.0f);
                    __syncwarp();
                    if (u == 0) {
                        sh.gaps[n & 3] = gaps;
                        kv4_arrive(smem_addr(&sh.scales_full[n & 3]));
                    }
                }
                fence_proxy_async_smem();
                kv4_arrive(smem_addr(&sh.k_full[st]));
            }
            uint64_t where = 0;
            if (more) {
                if (page >= 0 && page < c.n_pages)
                    where = (uint64_t)(c.pool + kv8_head_offset<D>(c, page, a.layer, w.head) +
                                       (cell & ((1 << in_page) - 1)) * Kv8Cell<D>::kBytes);
                else if (inside && u < 8)
                    kv4_bad(c);
                scales = where ? __ldg((const float2 *)((const uint8_t *)where + Kv8Cell<D>::kScales)) : make_float2(-1.0f, 1.0f);
                load_k<D>(rk, where, u);
            }
            if (n != ~0u) {
                if (n >= 2)
                    wait(sh.v_empty[st], (n >> 1) - 1);
                unpack_v<D>(rv, tiles + C::kOffV + st * C::kV, u, left);
                fence_proxy_async_smem();
                kv4_arrive(smem_addr(&sh.v_full[st]));
            }
            if (!more)
                break;
            load_v<D>(rv, where, u);
            left = w.len - (w.b0 + i) * kBlock;
            ++n;
            if (++i == w.nblk) {
                i = 0;
                w = get_piece(++piece);
                more = w.nblk > 0;
            }
        }
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
                const uint32_t q = desc0 + k * (C::kQ >> 4), kk = desc0 + (C::kOffK >> 4) + stage * (C::kQ >> 4);
                const uint32_t d = tmem + k * 128;
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        mma_ss<128>(d, q + ((g * kSub + 32 * x) >> 4), kk + ((g * kSub + 32 * x) >> 4), kIdesc<128>, g + x,
                                    one);
                commit(smem_addr(&sh.s_full[k]), one);
            };
            const auto values = [&](int k, int stage, uint32_t accumulate) { // O of tile k, V in `stage`
                const uint32_t v = desc0 + (C::kOffV >> 4) + stage * (C::kV >> 4);
                const uint32_t d = tmem + 256 + k * 128, p = tmem + k * 128;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        mma_ts(d, p + 32 * h + 8 * x, v + ((h * (D * 128) + 32 * x) >> 4), kIdesc<D>,
                               h + x > 0 ? 1u : accumulate, one);
            };
            // O of block i of a piece (block n - 1 of the CTA), then S of block i + 1 (block n), tile by
            // tile. The stages are constants of two copies of this, so that all descriptors are uniform.
            int nblk, n0, n1;
            const auto step = [&](auto parity, int i) {
                constexpr int nxt = decltype(parity)::value, cur = nxt ^ 1; // n & 1, (n - 1) & 1
                const bool more = i + 1 < nblk;
                if (i >= 0) {
                    wait(sh.v_full[cur], (n - 1) >> 1);
                    if (i < n0) {
                        wait(sh.p_full[0], n_p0++);
                        fence_after();
                        values(0, cur, i > 0);
                        if (i == n0 - 1)
                            commit(smem_addr(&sh.o_full[0]), one);
                    }
                }
                if (more) {
                    wait(sh.k_full[nxt], n >> 1);
                    if (i + 1 < n0) {
                        if (i < 0)
                            wait(sh.q_full[0], n_q0++);
                        fence_after();
                        scores(0, nxt);
                    }
                }
                if (i >= 0) {
                    if (i < n1) {
                        wait(sh.p_full[1], n_p1++);
                        fence_after();
                        values(1, cur, i > 0);
                        if (i == n1 - 1)
                            commit(smem_addr(&sh.o_full[1]), one);
                    }
                    commit(smem_addr(&sh.v_empty[cur]), one);
                }
                if (more) {
                    if (i + 1 < n1) {
                        if (i < 0)
                            wait(sh.q_full[1], n_q1++);
                        fence_after();
                        scores(1, nxt);
                    }
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
                    if (n & 1)
                        step(std::integral_constant<int, 1>{}, i);
                    else
                        step(std::integral_constant<int, 0>{}, i);
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
