// kv8_attn.cu -- attention of few queries over the 8-bit paged cache (decode steps and
// drafted tokens), and of any queries over the pages that were selected for each.
//
// For one sequence and kv head, the rows are its queries times the query heads that share the kv
// head (with lists of pages: one query's); a tile holds 8 NT of them. A warp takes the cache a
// cell (16 tokens) at a time:
//
//   S^T [16 tokens][rows] = codes(K) Q^T      m16n8k16, the codes and q as fp16
//   s = scale_K S^T                           fp32
//   p = 2^(s + e - m + 6)                     2^e: V's scale; m: the row's running maximum of s + e
//   O^T [channels][rows] += codes(V)^T P^T    m16n8k16, P as fp16
//   l += 2^-e p
//
// The codes are exact in fp16, q is made so by a power of two per row, so scores carry fp32
// rounding only. V's scale is a power of two too: as an exponent of the weights it costs an addition,
// V's codes are exact operands, and only the weights are rounded (2^-11). m is raised only when a
// score passes it by 2^8: the warp votes instead of reducing.
//
// The layout of a cell is the operands' own: lane l reads 16 bytes at 16 l, so K and V need no
// transposition on the way to the registers, and an instruction makes two codes fp16.
//
// A (sequence, kv head, tile) is a segment. Each CTA gets one piece of one where that can be
// balanced, else an even part of the line of all segments. A CTA's warps take the cells of a piece
// in turn and are joined in shared memory. A segment that was cut is joined by the last of its
// CTAs, in CTA order, from the workspace.
#include "kv8.cuh"
#include "kv_ops.cuh"

namespace nm {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int64_t kMinShare = 8;  // cells of a CTA at least: one for each warp
constexpr int kWhole = 32;        // when none has more cells than this, no segment is cut
constexpr float kMoreUnits = 24.0f; // a second piece costs about as many cells
constexpr int kOver = 32;         // cells that starting and ending a piece costs as much as (4 x 5 tokens: 42.4 us, with 16 44.1)
constexpr float kShift = 6.0f;    // p = 2^(s + e - m + kShift)
constexpr float kSlack = 8.0f;    // a score may pass m by this much
constexpr float kNone = 1e38f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnArgs {
    int layer, ratio; // ratio: query heads of one kv head
    int n_q_heads;
    const uint16_t *q;
    int64_t q_stride;
    float scale;
    uint16_t *out;
    int64_t out_stride;
    float *lse;
    uint32_t *counters;
    float *partials;
    const int32_t *pages; // of a selection: [n_tokens][n_kv_heads][n_list]
    int n_list;
};

// Floats of one part in the workspace: m and l of each row, then O.
template <int D, int NT> constexpr int part_floats() { return 8 * NT * (D + 2); }

// What the scores of a row need: its factor, and how many tokens it attends.
struct RowInfo {
    float scale;
    int limit;
};

template <int D, int NT> struct Smem {
    static constexpr int kRows = 8 * NT;
    static constexpr int kPitch = D + 4;
    static constexpr int kStage = Kv8Cell<D>::kBytes;
    // cells of a warp in flight or in use: what two CTAs (up to 16 rows) or one leave room for
    static constexpr int kStages = D == 128 ? (NT <= 2 ? 3 : 5) : (NT <= 2 ? 5 : 8);
    static constexpr int kSteps = D / 16;
    // the warps' rings; when a piece is done, the warps' parts (m, l, O) in their place
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kMerge = kWarps * kRows * (2 + kPitch) * 4;
    static constexpr int kJoin = (kKv4Counters / 4 * kRows + 2 * kRows) * 4; // weights of the parts of a segment
    static constexpr int kMost = kRing > kMerge ? (kRing > kJoin ? kRing : kJoin) : (kMerge > kJoin ? kMerge : kJoin);
    static constexpr int kBig = (kMost + 127) / 128 * 128;
    // Q in B fragments: [n-tile][k-step][lane][2], then the rows' RowInfo, the rings' barriers and the
    // first tokens of their cells
    static constexpr int kQ = kBig, kInfo = kQ + NT * kSteps * 256, kBars = kInfo + kRows * 8;
    static constexpr int kFirst = kBars + kWarps * kStages * 8, kSeqs = kFirst + (kWarps * kStages * 4 + 15) / 16 * 16;
};

// The last i with pre[i] <= x, of n entries that do not fall; -1: none.
__device__ __forceinline__ int find(const int64_t *pre, int n, int64_t x)
{
    int lo = -1, hi = n;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (pre[m] <= x)
            lo = m;
        else
            hi = m;
    }
    return lo;
}

// Which entries of a list count: the first -1 ends it; before that, those that are pages of the sequence (of `most`
// tokens) and above all that count before them. Others before the end are passed over and reported.
__device__ __forceinline__ bool is_page(const Kv4 &c, int index, int most)
{
    return index >= 0 && (int64_t)index << c.page_shift < most;
}
// Entry j (`index`) is as it should be behind an entry (`before`) that is. If all up to j are, j counts unless it is -1.
__device__ __forceinline__ bool in_order(const Kv4 &c, int j, int before, int index, int most)
{
    return index == -1 || (is_page(c, index, most) && (j == 0 || (before >= 0 && before < index)));
}
// Whether entry j counts (another j in each lane of a warp, up to `last`), of a list that need not be in order: it is followed from
// entry `from` on, behind entries of which `top` is the last one that counts (-1: none, kEnded: the list has ended).
constexpr int kEnded = 0x7FFFFFFF;
__device__ __forceinline__ bool follow(const Kv4 &c, const int32_t *list, int from, int &top, int j, int last, int most)
{
    const int lane = threadIdx.x & 31;
    bool yes = false;
#pragma unroll 1
    for (int b = from; b <= last; b += 32) {
        const int index = list[min(b + lane, last)];
        const uint32_t ends = __ballot_sync(~0u, index == -1);
        const bool open = b + lane <= last && top != kEnded && lane < (ends ? __ffs(ends) - 1 : 32);
        int upto = open && is_page(c, index, most) ? index : -1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(~0u, upto, o);
            upto = lane >= o ? max(upto, x) : upto;
        }
        const int x = __shfl_up_sync(~0u, upto, 1), before = lane > 0 ? max(top, x) : top;
        const bool counts = open && index > before && is_page(c, index, most);
        if (open && !counts)
            kv4_bad(c);
        const uint32_t all = __ballot_sync(~0u, counts);
        yes = j >= b && j < b + 32 ? (all >> (j - b) & 1u) != 0 : yes;
        const int most_here = __shfl_sync(~0u, upto, 31);
        top = ends ? kEnded : max(top, most_here);
    }
    return yes;
}

// The cell that entry x of a list's cells names, in its entry `index`, which counts: its address, or 0, and the position it
// begins at. What is listed beyond the query is not seen.
template <int D>
__device__ __forceinline__ uint64_t listed_cell(const Kv4 &c, int row, const uint8_t *heads, int x, int index, int limit,
                                                int *begins)
{
    const int cell = x & ((1 << (c.page_shift - 4)) - 1);
    *begins = (index << c.page_shift) + (cell << 4);
    if (*begins >= limit)
        return 0;
    const int page = kv4_page(c, row, index);
    if (page < 0) {
        kv4_bad(c);
        return 0;
    }
    return (uint64_t)(heads + page * c.page_bytes + cell * Kv8Cell<D>::kBytes);
}

// A row of q as the B operand: the lane's channels 64 e + 16 t .. are words of four k-steps (put(step, word)).
// Returns the factor of the row's scores. sees: whether the row sees any token, which something that is not finite
// in it then meets.
template <int D, class F>
__device__ __forceinline__ float split_q(const uint4 (&qw)[D / 64][2], float scale, bool sees, const F &put)
{
    constexpr int G = D / 64;
    float x[G][16];
    uint32_t top = 0; // the largest magnitude, as fp32 bits
#pragma unroll
    for (int e = 0; e < G; ++e)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            top = max(top, kv8_magnitude(qw[e][f]));
            const uint32_t ws[4] = {qw[e][f].x, qw[e][f].y, qw[e][f].z, qw[e][f].w};
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                x[e][8 * f + 2 * n] = bf16lo_to_f32(ws[n]);
                x[e][8 * f + 2 * n + 1] = bf16hi_to_f32(ws[n]);
            }
        }
    top = max(top, __shfl_xor_sync(~0u, top, 1));
    top = max(top, __shfl_xor_sync(~0u, top, 2));
    // 2^-e brings the row's largest magnitude into [1, 2): what is at least 2^-17 of it is
    // exact in fp16 (eight bits above 2^-24), the rest is rounded to 2^-24
    const uint32_t field = top >> 23, e2 = field == 0xFFu || field == 0 ? 127u : field > 253u ? 253u : field;
    const float up = __uint_as_float(e2 << 23); // the sign of the scale goes with q
    const float down = scale < 0.0f ? -__uint_as_float((254u - e2) << 23) : __uint_as_float((254u - e2) << 23);
#pragma unroll
    for (int e = 0; e < G; ++e)
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            const float *const y = &x[e][4 * f];
            put(4 * e + f, make_uint2(pack_half2(y[0] * down, y[1] * down), pack_half2(y[2] * down, y[3] * down)));
        }
    // above 0, so that masked scores stay -inf; finite, so that scores of 0 stay 0
    return field == 0xFFu && sees ? __uint_as_float(0x7FC00000u)
                                  : fminf(fmaxf(up * (fabsf(scale) * kLog2e), 1e-30f), 0x1.fffffep127f);
}

// What a warp keeps of its rows (lane (g, t): rows 8 j + 2 t + n), and a cell's part in it.
template <int D, int NT> struct Rows {
    float o[NT][D / 16][4]; // [n-tile][m-tile][fragment]
    float mo[NT][2];        // kShift - m, m the running maximum; before the first score so large that any raises m
    float l[NT][2], scale[NT][2];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int z = 0; z < D / 16; ++z)
#pragma unroll
                for (int f = 0; f < 4; ++f)
                    o[j][z][f] = 0.0f;
            mo[j][0] = mo[j][1] = kNone, l[j][0] = l[j][1] = 0.0f;
        }
    }
    // channels 32 q + 4 g .. of row 8 j + 2 t + n
    __device__ __forceinline__ float4 four(int j, int n, int q) const
    {
        return make_float4(o[j][2 * q][n], o[j][2 * q][n + 2], o[j][2 * q + 1][n], o[j][2 * q + 1][n + 2]);
    }
    // C cells in shared memory, one behind the other, whose tokens begin at positions tok. all: positions that every row
    // sees; end: positions that hold tokens (a cell that begins there or beyond may hold anything); q(j, z): B operands;
    // limit(j, n): positions that a row sees.
    template <int C, class Q, class L>
    __device__ __forceinline__ void take(const uint8_t *cells, const int (&tok)[C], int all, int end, int lane, const Q &qop,
                                         const L &limit)
    {
        constexpr int G = D / 64;
        const int g = lane >> 2, t = lane & 3;
        float ks[C], ev[C], iv[C];
        bool part = false;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float2 scales = *(const float2 *)(cells + c * Kv8Cell<D>::kBytes + Kv8Cell<D>::kScales);
            if (C > 1 && tok[c] >= end)
                scales = make_float2(1.0f, 1.0f);
            ks[c] = scales.x;
            // V's scale goes with the weights, as an exponent; the sums are freed of it again
            ev[c] = (float)((int)(__float_as_uint(scales.y) >> 23) - 127);
            iv[c] = __uint_as_float((254u << 23) - __float_as_uint(scales.y));
            part |= tok[c] + kKv4Cell > all;
        }

        // scores
        float sc[C][NT][4];
        {
            float acc[C][G][NT][4] = {};
#pragma unroll
            for (int e = 0; e < G; ++e) {
                uint4 x0[C], x1[C];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    x0[c] = *((const uint4 *)(cells + c * Kv8Cell<D>::kBytes + e * 512) + lane);
                    x1[c] = *((const uint4 *)(cells + c * Kv8Cell<D>::kBytes + 8 * D + e * 512) + lane);
                }
#pragma unroll
                for (int f = 0; f < 4; ++f)
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const uint32_t w0 = f == 0 ? x0[c].x : f == 1 ? x0[c].y : f == 2 ? x0[c].z : x0[c].w;
                        const uint32_t w1 = f == 0 ? x1[c].x : f == 1 ? x1[c].y : f == 2 ? x1[c].z : x1[c].w;
                        const uint32_t af[4] = {kv8_decode(w0), kv8_decode(w1), kv8_decode(w0 >> 16), kv8_decode(w1 >> 16)};
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            const uint2 q = qop(j, 4 * e + f);
                            mma16816(acc[c][e][j], af, q.x, q.y);
                        }
                    }
            }
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int f = 0; f < 4; ++f) // token g + 8 (f / 2), row 2 t + f % 2
                        sc[c][j][f] = (G == 2 ? acc[c][0][j][f] + acc[c][G - 1][j][f] : acc[c][0][j][f]) * ks[c];
        }
        // a row may see only part of a cell
        if (part) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int f = 0; f < 4; ++f)
                        sc[c][j][f] = tok[c] + g + 8 * (f >> 1) < limit(j, f & 1) ? sc[c][j][f] : -INFINITY;
        }
        float top = -INFINITY;
        float y[C][NT][4];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    y[c][j][f] = fmaf(sc[c][j][f], scale[j][f & 1], mo[j][f & 1] + ev[c]);
                    top = fmaxf(top, y[c][j][f]);
                }
        if (__any_sync(~0u, top > kShift + kSlack)) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    float z = -INFINITY;
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        z = fmaxf(z, fmaf(fmaxf(sc[c][j][n], sc[c][j][n + 2]), scale[j][n], ev[c]));
                    z = fmaxf(z, __shfl_xor_sync(~0u, z, 4));
                    z = fmaxf(z, __shfl_xor_sync(~0u, z, 8));
                    z = fmaxf(z, __shfl_xor_sync(~0u, z, 16));
                    const float was = mo[j][n], now = z == -INFINITY ? was : fminf(was, kShift - z);
                    const float by = was == now ? 1.0f : exp2_approx(now - was);
                    mo[j][n] = now;
                    l[j][n] *= by;
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        y[c][j][n] = fmaf(sc[c][j][n], scale[j][n], now + ev[c]);
                        y[c][j][n + 2] = fmaf(sc[c][j][n + 2], scale[j][n], now + ev[c]);
                    }
#pragma unroll
                    for (int z4 = 0; z4 < D / 16; ++z4) {
                        o[j][z4][n] *= by;
                        o[j][z4][n + 2] *= by;
                    }
                }
        }
        uint32_t pb[C][NT][2];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float p[4];
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    p[f] = exp2_approx(y[c][j][f]);
                    l[j][f & 1] = fmaf(p[f], iv[c], l[j][f & 1]);
                }
                pb[c][j][0] = transpose8x8(pack_half2(p[0], p[1]));
                pb[c][j][1] = transpose8x8(pack_half2(p[2], p[3]));
            }

        // O^T += V^T P^T; tokens past the last that is seen hold anything: their V is taken as 0
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int left = end - tok[c];
            uint32_t keep = ~0u;
            if (left < kKv4Cell)
                keep = (2 * t < left ? 0xFFu : 0u) | (2 * t + 1 < left ? 0xFF00u : 0u) | (2 * t + 8 < left ? 0xFF0000u : 0u) |
                       (2 * t + 9 < left ? 0xFF000000u : 0u);
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
                const uint4 x4 = *((const uint4 *)(cells + c * Kv8Cell<D>::kBytes + Kv8Cell<D>::kV + q * 512) + lane);
                const uint32_t w[4] = {x4.x & keep, x4.y & keep, x4.z & keep, x4.w & keep};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t af[4] = {kv8_decode(w[2 * h]), kv8_decode(w[2 * h + 1]), kv8_decode(w[2 * h] >> 16),
                                            kv8_decode(w[2 * h + 1] >> 16)};
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        mma16816(o[j][2 * q + h], af, pb[c][j][0], pb[c][j][1]);
                }
            }
        }
    }
};

// Pieces of a segment that is cut every `chunk` units.
__device__ __forceinline__ int pieces_of(int units, int chunk) { return (int)((uint32_t)(units + chunk - 1) / (uint32_t)chunk); }
__device__ __forceinline__ int units_of(int len) { return len > 0 ? (len + kKv4Cell - 1) / kKv4Cell : 1; }

template <int D, int NT, bool kListed>
__global__ void __launch_bounds__(kThreads, NT <= 2 ? 2 : 1)
    kv8_rows_kernel(const Kv4 c, const Kv4Batch b, const AttnArgs a)
{
    constexpr int G = D / 64;
    constexpr int RT = 8 * NT;
    constexpr int KS = 4 * G; // k-steps of 16 channels
    using SM = Smem<D, NT>;
    constexpr int S = SM::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    float *const sm_m = (float *)smem, *const sm_l = sm_m + kWarps * RT, *const sm_o = sm_l + kWarps * RT;
    uint2 *const sm_q = (uint2 *)(smem + SM::kQ);
    RowInfo *const sm_info = (RowInfo *)(smem + SM::kInfo);
    int64_t *const pre = (int64_t *)(smem + SM::kSeqs);      // [n_seqs + 1]
    Kv4Seq *const seqs = (Kv4Seq *)(pre + b.n_seqs + 1);     // [n_seqs]
    __shared__ uint32_t s_last;
    __shared__ int s_chunk;
    __shared__ bool s_rest; // some rows belong to no sequence
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    uint8_t *const ring = smem + warp * S * SM::kStage;
    int *const sm_first = (int *)(smem + SM::kFirst) + warp * S;
    const uint32_t rings = smem_addr(ring), bars = smem_addr(smem + SM::kBars) + warp * S * 8;

    // the segments of each sequence, and where they start on the line of units
    if (lane == 0)
        for (int i = 0; i < S; ++i)
            mbar_init(bars + 8 * i, 1);
    fence_mbar_init();
    int longest = 0;
    for (int i = tid; i < b.n_seqs; i += kThreads) {
        const Kv4Seq s = kv4_seq(c, b, i, blockIdx.x == 0);
        seqs[i] = s;
        if (kListed) {
            pre[i] = b.starts ? b.starts[i] : i;
            continue;
        }
        longest = max(longest, s.n_new == 0 ? 0 : units_of(s.len));
        pre[i + 1] = (int64_t)((uint32_t)(s.n_new * a.ratio + RT - 1) / RT) * c.n_kv_heads; // segments
    }
    const bool is_long = __syncthreads_or(longest > kWhole);
    // Lists: a token, kv head and tile is a segment, all of one length
    const int list_tiles = (a.ratio + RT - 1) / RT, list_units = a.n_list << (c.page_shift - 4);
    const int64_t list_segments = kListed ? b.n_tokens * c.n_kv_heads * list_tiles : 0;
    if constexpr (kListed) {
        if (tid == 0) {
            int z = 0; // an even cut of the line, as below
            if (list_units <= kWhole || list_segments >= 4 * (int64_t)gridDim.x)
                z = 1 << 30;
            else if (list_segments <= gridDim.x)
                z = (int)ceil_div(ceil_div(list_units, gridDim.x / list_segments), kWarps) * kWarps;
            s_chunk = z;
            s_rest = false;
        }
    } else if (warp == 0) {
        // How the segments are cut:
        //   chunk > 0: into pieces of so many units (a multiple of the warps), each a step of the
        //     line; the least chunk with which all pieces fit the CTAs of one wave,
        //   chunk = 0: the line has a step for each unit and kOver more for each segment, and is cut
        //     evenly. Taken when there are more segments than CTAs, or when one chunk for all lengths
        //     is over an even cut by more than a second piece costs a CTA.
        const auto total_of = [&](const auto &f) { // counts, each cut off far above the grid
            uint32_t x = 0;
            for (int i = lane; i < b.n_seqs; i += 32) {
                const int64_t y = f(i);
                x += y < 65536 ? (uint32_t)y : 65536u;
            }
            return __reduce_add_sync(~0u, x);
        };
        int chunk = 0;
        if (!is_long) {
            chunk = 1 << 30;
        } else if (total_of([&](int i) { return pre[i + 1]; }) <= gridDim.x) {
            float work = 0.0f;
            for (int i = lane; i < b.n_seqs; i += 32)
                work += (float)pre[i + 1] * (float)units_of(seqs[i].len);
            for (int z = 16; z; z >>= 1)
                work += __shfl_xor_sync(~0u, work, z);
            const float even = work / (float)gridDim.x;
            const int step = (int)(even / (8 * kWarps)) * kWarps + kWarps;
            for (int z = (int)(even / kWarps) * kWarps + kWarps; (float)z <= even + kMoreUnits; z += step) {
                if (total_of([&](int i) { return pre[i + 1] * pieces_of(units_of(seqs[i].len), z); }) <= gridDim.x) {
                    chunk = z;
                    break;
                }
            }
        }
        int64_t sum = 0;
        bool rest = !kv4_ends(b);
        for (int i0 = 0; i0 < b.n_seqs; i0 += 32) {
            int64_t x = 0;
            if (i0 + lane < b.n_seqs) {
                rest |= seqs[i0 + lane].first < 0;
                const int units = units_of(seqs[i0 + lane].len);
                x = pre[i0 + lane + 1] * (chunk ? pieces_of(units, chunk) : kOver + units);
            }
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(~0u, x, o);
                if (lane >= o)
                    x += y;
            }
            __syncwarp();
            if (i0 + lane < b.n_seqs)
                pre[i0 + lane + 1] = sum + x;
            sum += __shfl_sync(~0u, x, 31);
        }
        rest = __any_sync(~0u, rest);
        if (lane == 0) {
            pre[0] = 0;
            s_chunk = chunk;
            s_rest = rest;
        }
    }
    __syncthreads();
    const int chunk = s_chunk;
    const int list_per = chunk ? pieces_of(list_units, chunk) : kOver + list_units;
    const int64_t total = kListed ? list_segments * list_per : pre[b.n_seqs];
    int64_t share = ceil_div(total, gridDim.x);
    if (!chunk && share < kMinShare + kOver)
        share = kMinShare + kOver;
    const int64_t lo = (int64_t)blockIdx.x * share, hi = lo + share < total ? lo + share : total;
    const int shift = c.page_shift - 4;
    uint32_t used = 0; // cells of this warp so far: the next takes stage used % S
    bool dead = false;

    for (int64_t pos = lo; pos < hi;) {
        int most = 0; // (lists) tokens of the sequence
        int i, units, per, head, row0;
        int64_t seg_lo, list = 0;
        Kv4Seq s{};
        if (kListed) {
            const int64_t seg = quotient(pos, list_per), token = quotient(seg, c.n_kv_heads * list_tiles);
            const int rest = (int)(seg - token * c.n_kv_heads * list_tiles);
            head = rest / list_tiles;
            row0 = rest % list_tiles * RT;
            units = list_units;
            per = list_per;
            seg_lo = seg * list_per;
            list = (token * c.n_kv_heads + head) * a.n_list;
            i = find(pre, b.n_seqs, token);
            if (i >= 0)
                s = seqs[i];
            // the token's own position is the last that it sees; a row of no sequence sees nothing
            const int64_t seen = i >= 0 && s.first >= 0 && token - s.first < s.n_new ? s.len - s.n_new + (token - s.first) + 1 : 0;
            most = s.len;
            s.len = seen > 0 && s.len > 0 ? (int)seen : 0;
            s.first = (int)token;
            s.n_new = 1;
        } else {
            i = find(pre, b.n_seqs, pos);
            s = seqs[i];
            units = units_of(s.len);
            per = chunk ? pieces_of(units, chunk) : kOver + units; // steps of the segment
            const int64_t seg = quotient(pos - pre[i], per);
            seg_lo = pre[i] + seg * per;
            const int tiles = (s.n_new * a.ratio + RT - 1) / RT;
            head = (int)quotient(seg, tiles);
            row0 = (int)(seg - (int64_t)head * tiles) * RT; // first row of the tile
        }
        const int over = chunk ? 0 : kOver;
        const int64_t seg_hi = seg_lo + per;
        int steps, c0, c1;
        if (chunk) {
            steps = 1;
            c0 = (int)(pos - seg_lo) * (per > 1 ? chunk : 0);
            c1 = per > 1 && units - c0 > chunk ? c0 + chunk : units;
        } else {
            steps = (int)((hi < seg_hi ? hi : seg_hi) - pos);
            const int from = (int)(pos - seg_lo) - over;
            c0 = from > 0 ? from : 0;
            c1 = from + steps;
            if (c1 <= c0)
                break; // the CTA's part of the line ends before the segment's first unit
        }
        const int rows = s.n_new * a.ratio; // rows of the sequence and kv head
        const int tile_first = s.len - s.n_new + row0 / a.ratio + 1; // tokens that its first row attends

        // Q: warp j takes n-tile j: row g, channels 64 e + 16 t ..
        uint4 qw[G][2];
        const int qrow = row0 + 8 * warp + g;
        const bool real = warp < NT && qrow < rows;
        if (warp < NT) {
            const uint16_t *q = a.q + (int64_t)(s.first + qrow / a.ratio) * a.q_stride +
                                ((int64_t)head * a.ratio + qrow % a.ratio) * D + 16 * t;
#pragma unroll
            for (int e = 0; e < G; ++e)
#pragma unroll
                for (int f = 0; f < 2; ++f)
                    qw[e][f] = real ? ldg_nc128(q + 64 * e + 8 * f) : make_uint4(0, 0, 0, 0);
        }

        // The warp's cells are c0 + warp, + kWarps, ... Lane n holds the address of every 32nd (0: its page
        // is none of the pool's, or it is past the tokens that are seen) and the position it begins at;
        // `have` has a bit for each stage that was filled.
        int mine = !dead && s.len > 0 && c1 - c0 > warp ? (c1 - c0 - warp + kWarps - 1) / kWarps : 0;
        const uint8_t *const heads = c.pool + kv8_head_offset<D>(c, 0, a.layer, head);
        uint64_t where = 0;
        int begins = 0;
        uint32_t have = 0;
        // (lists) Of the entries up to the piece's last one: of a few each warp looks at all of them, more are shared by the
        // CTA, four at a time to a thread (one at a time: a token of 4096 pages of 16 took 33.8 us, now 30.8; of 32768 pages
        // 99, now 68, of which this is 12).
        bool ordered = true;
        if constexpr (kListed) {
            constexpr int kAsk = 4; // entries of a thread that are asked for together
            const int n = s.len > 0 ? ((c1 - 1) >> shift) + 1 : 0, step = n > 32 ? kThreads : 32;
            const int32_t *const l = a.pages + list;
            bool odd = false;
            if (n > step) {
#pragma unroll 1
                for (int j0 = tid; j0 < n; j0 += kAsk * kThreads) {
                    int index[kAsk], before[kAsk];
#pragma unroll
                    for (int u = 0; u < kAsk; ++u) {
                        const int j = min(j0 + u * kThreads, n - 1);
                        index[u] = l[j];
                        before[u] = l[max(j - 1, 0)];
                    }
#pragma unroll
                    for (int u = 0; u < kAsk; ++u)
                        odd |= !in_order(c, min(j0 + u * kThreads, n - 1), before[u], index[u], most);
                }
            } else {
                const int j = tid & (step - 1);
                if (j < n)
                    odd = !in_order(c, j, l[max(j - 1, 0)], l[j], most);
            }
            ordered = !(n > 32 ? __syncthreads_or(odd) : __any_sync(~0u, odd));
        }
        const auto fetch = [&](int x) {
            if ((x & 31) == 0) {
                const int cell = c0 + warp + (x + lane) * kWarps;
                where = 0;
                if constexpr (kListed) {
                    const int32_t *const l = a.pages + list;
                    bool counts = x + lane < mine;
                    const int j = counts ? cell >> shift : 0, index = l[j];
                    counts &= index != -1;
                    if (!ordered) {
                        int top = -1;
                        counts &= follow(c, l, 0, top, j, __reduce_max_sync(~0u, j), most);
                    }
                    if (counts)
                        where = listed_cell<D>(c, s.row, heads, cell, index, s.len, &begins);
                } else if (x + lane < mine) {
                    if (cell * kKv4Cell < s.len) {
                        begins = cell * kKv4Cell;
                        const int page = kv4_page(c, s.row, cell >> shift);
                        if (page >= 0)
                            where = (uint64_t)(heads + page * c.page_bytes + (cell & ((1 << shift) - 1)) * Kv8Cell<D>::kBytes);
                        else
                            kv4_bad(c);
                    }
                }
            }
            const uint64_t src = __shfl_sync(~0u, where, x & 31);
            const int first = __shfl_sync(~0u, begins, x & 31);
            const uint32_t st = (used + x) % S, bar = bars + 8 * st;
            have = (have & ~(1u << st)) | (uint32_t)(src != 0) << st;
            if (lane == 0) {
                sm_first[st] = first;
                mbar_arrive_expect_tx(bar, src ? Kv8Cell<D>::kBytes : 0u);
                if (src)
                    bulk_load(rings + st * SM::kStage, (const void *)src, Kv8Cell<D>::kBytes, bar);
            }
            __syncwarp();
        };
        for (int x = 0; x < S - 1 && x < mine; ++x)
            fetch(x);

        // Q as the B operand
        if (warp < NT) {
            const int limit = real ? s.len - s.n_new + qrow / a.ratio + 1 : 0;
            const float factor = split_q<D>(qw, a.scale, limit > 0, [&](int z, uint2 v) { sm_q[(warp * KS + z) * 32 + lane] = v; });
            if (t == 0)
                sm_info[8 * warp + g] = RowInfo{factor, limit};
        }
        __syncthreads();
        // with one n-tile Q stays in registers
        constexpr bool kKeepQ = NT == 1;
        uint2 qb[kKeepQ ? KS : 1];
        Rows<D, NT> r;
        if (kKeepQ) {
#pragma unroll
            for (int x = 0; x < KS; ++x)
                qb[x % (kKeepQ ? KS : 1)] = sm_q[x * 32 + lane];
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            r.scale[j][0] = sm_info[8 * j + 2 * t].scale;
            r.scale[j][1] = sm_info[8 * j + 2 * t + 1].scale;
        }

        r.clear();

#pragma unroll 1
        for (int x = 0; x < mine; ++x) {
            if (x + S - 1 < mine) {
                __syncwarp(); // the stage that is filled now was read by all lanes
                fetch(x + S - 1);
            }
            const uint32_t st = (used + x) % S;
            kv4_wait(bars + 8 * st, ((used + x) / S) & 1, c.status, dead);
            if (__any_sync(~0u, dead)) {
                // Ran out: the warp asks for no more cells, in this piece or the next, and the copies in
                // flight end (bounded) before the parts take the rings' place.
                for (int z = x; z < x + S && z < mine; ++z) {
                    dead = false;
                    kv4_wait(bars + 8 * ((used + z) % S), ((used + z) / S) & 1, c.status, dead);
                }
                dead = true;
                mine = x;
                break;
            }
            if (have >> st & 1u)
                r.template take<1>(ring + st * SM::kStage, {sm_first[st]}, tile_first, s.len, lane,
                       [&](int j, int z) { return kKeepQ ? qb[z % (kKeepQ ? KS : 1)] : sm_q[(j * KS + z) * 32 + lane]; },
                       [&](int j, int n) { return sm_info[8 * j + 2 * t + n].limit; });
        }
        used += mine;
        __syncthreads(); // the rings are read: the parts take their place

        // the warp's part to shared memory: rows 2 t, 2 t + 1, channels 32 q + 4 g ..
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                float x = r.l[j][n];
                x += __shfl_xor_sync(~0u, x, 4);
                x += __shfl_xor_sync(~0u, x, 8);
                x += __shfl_xor_sync(~0u, x, 16);
                const int row = 8 * j + 2 * t + n;
                if (g == 0) {
                    sm_m[warp * RT + row] = r.mo[j][n] == kNone ? -INFINITY : kShift - r.mo[j][n];
                    sm_l[warp * RT + row] = x;
                }
                float *dst = sm_o + (warp * RT + row) * SM::kPitch + 4 * g;
#pragma unroll
                for (int q = 0; q < D / 32; ++q)
                    *(float4 *)(dst + 32 * q) = r.four(j, n, q);
            }
        __syncthreads();

        // joined over the warps; four channels of a row to a thread
        const auto store = [&](int row, int ch, const float4 &x, float M, float L) {
            const int r = row0 + row;
            if (r >= rows)
                return;
            const int64_t token = s.first + r / a.ratio, h = (int64_t)head * a.ratio + r % a.ratio;
            const float inv = L == 0.0f ? 0.0f : 1.0f / L;
            uint2 w;
            w.x = f32_to_bf16_rn(x.x * inv) | ((uint32_t)f32_to_bf16_rn(x.y * inv) << 16);
            w.y = f32_to_bf16_rn(x.z * inv) | ((uint32_t)f32_to_bf16_rn(x.w * inv) << 16);
            *(uint2 *)(a.out + token * a.out_stride + h * D + ch) = w;
            if (a.lse && ch == 0)
                a.lse[token * a.n_q_heads + h] = L == 0.0f ? -INFINITY : (M - kShift + log2f(L)) * kLn2;
        };
        const bool whole = c0 == 0 && c1 == units;
        float *part = nullptr;
        if (!whole)
            part = a.partials + ((int64_t)blockIdx.x * 2 + (c0 > 0 ? 0 : 1)) * part_floats<D, NT>();
        for (int x = tid; x < RT * (D / 4); x += kThreads) {
            const int row = x / (D / 4), ch = (x % (D / 4)) * 4;
            float M = -INFINITY, L = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                M = fmaxf(M, sm_m[w * RT + row]);
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = sm_m[w * RT + row];
                const float f = mw == M ? 1.0f : exp2_approx(mw - M);
                const float4 z = *(const float4 *)(sm_o + (w * RT + row) * SM::kPitch + ch);
                L = fmaf(f, sm_l[w * RT + row], L);
                y.x = fmaf(f, z.x, y.x);
                y.y = fmaf(f, z.y, y.y);
                y.z = fmaf(f, z.z, y.z);
                y.w = fmaf(f, z.w, y.w);
            }
            if (whole) {
                store(row, ch, y, M, L);
            } else {
                if (ch == 0) {
                    part[row] = M;
                    part[RT + row] = L;
                }
                *(float4 *)(part + 2 * RT + row * D + ch) = y;
            }
        }
        if (!whole) {
            // the segment's CTAs are first .. last; the last one to arrive joins their parts in order
            const int first = (int)quotient(seg_lo + over, share), last = (int)quotient(seg_hi - 1, share);
            __syncthreads();
            if (tid == 0) {
                const uint32_t n = (uint32_t)(last - first);
                s_last = atom_add_acq_rel_gpu(a.counters + first, 1u) == n;
                if (s_last)
                    a.counters[first] = 0; // for the next launch
            }
            __syncthreads();
            if (s_last) {
                // weights of the parts first (a warp to a row), then their O: independent loads in a row
                const int n = last - first + 1;
                float *const weight = (float *)smem; // [n][RT], then [RT] M, [RT] L
                float *const sum_m = weight + n * RT, *const sum_l = sum_m + RT;
                const auto at = [&](int k) {
                    return a.partials + ((int64_t)(first + k) * 2 + (k > 0 ? 0 : 1)) * part_floats<D, NT>();
                };
                // O of the first parts is asked for before the weights, 16 parts at a time (8 at a time and after the weights:
                // 131071 tokens, 38 parts 55.0 us, now 54.5; one token of 32 pages 21.2, 19.8 with its selection)
                constexpr int kBatch = 16;
                float4 z[kBatch];
                const auto ask = [&](int x, int k0) {
                    const int row = x / (D / 4), ch = (x % (D / 4)) * 4;
#pragma unroll
                    for (int k = 0; k < kBatch; ++k)
                        z[k] = k0 + k < n ? __ldcg((const float4 *)(at(k0 + k) + 2 * RT + row * D + ch))
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
                };
                if (tid < RT * (D / 4))
                    ask(tid, 0);
                for (int row = warp; row < RT; row += kWarps) {
                    float mk[2], lk[2], M = -INFINITY, L = 0.0f;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int k = lane + 32 * u;
                        mk[u] = k < n ? ldcg_f32(at(k) + row) : -INFINITY;
                        lk[u] = k < n ? ldcg_f32(at(k) + RT + row) : 0.0f;
                        M = fmaxf(M, mk[u]);
                    }
                    for (int k = lane + 64; k < n; k += 32)
                        M = fmaxf(M, ldcg_f32(at(k) + row));
                    for (int z = 16; z; z >>= 1)
                        M = fmaxf(M, __shfl_xor_sync(~0u, M, z));
                    const auto weigh = [&](int k, float m, float l) {
                        const float f = m == M ? 1.0f : exp2_approx(m - M);
                        weight[k * RT + row] = f;
                        L = fmaf(f, l, L);
                    };
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        if (lane + 32 * u < n)
                            weigh(lane + 32 * u, mk[u], lk[u]);
                    for (int k = lane + 64; k < n; k += 32)
                        weigh(k, ldcg_f32(at(k) + row), ldcg_f32(at(k) + RT + row));
                    for (int z = 16; z; z >>= 1)
                        L += __shfl_xor_sync(~0u, L, z);
                    if (lane == 0) {
                        sum_m[row] = M;
                        sum_l[row] = L;
                    }
                }
                __syncthreads();
                for (int x = tid; x < RT * (D / 4); x += kThreads) {
                    const int row = x / (D / 4), ch = (x % (D / 4)) * 4;
                    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int k0 = 0; k0 < n; k0 += kBatch) {
                        if (x != tid || k0 > 0)
                            ask(x, k0);
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) {
                            const float f = k0 + k < n ? weight[(k0 + k) * RT + row] : 0.0f;
                            y.x = fmaf(f, z[k].x, y.x);
                            y.y = fmaf(f, z[k].y, y.y);
                            y.z = fmaf(f, z[k].z, y.z);
                            y.w = fmaf(f, z[k].w, y.w);
                        }
                    }
                    store(row, ch, y, sum_m[row], sum_l[row]);
                }
            }
        }
        // the next piece's copies overwrite the parts: they are read, and the reads come first
        fence_proxy_async_smem();
        __syncthreads();
        pos += steps;
    }
    if (!kListed && s_rest)
        kv4_answer_uncovered(b, a.out, a.out_stride, a.n_q_heads * D, a.lse, a.n_q_heads,
                             (int64_t)blockIdx.x * kWarps + warp, (int64_t)gridDim.x * kWarps);
}

// With lists and many of them: a warp takes a token's kv head by itself, all of its list, so that no threads
// meet, two cells at a time, whose chains of instructions overlap: 12 warps of two cells have as much under way as 24 of
// one, for whose registers and rings there is no room. Q is in its registers, and a lane has two rows' output of four
// channels in 32. Lists are dealt over the SMs before their warps, so that a last round is spread evenly. 512 tokens
// of 16 pages of 64 tokens, 32 heads on 8: 116 us (a cell at a time by 16 warps 123), 9.3 TB/s of cells, most of them
// from L2; what bounds it is the latency of a warp's chain: it issues an instruction in 60% of the cycles.
template <int D, int NT> struct Lists {
    static constexpr int kWarps = NT == 1 ? 12 : 8, kThreads = 32 * kWarps;
    static constexpr int kCells = 2; // of a stage: those of one copy, which a cell of its own page is not part of
    static constexpr int kStages = (NT == 1 ? 2 : 3) * (128 / D), kStage = kCells * Kv8Cell<D>::kBytes;
    static constexpr int kBytes = kWarps * kStages * kStage;
    static_assert(kBytes <= 200 * 1024, "shared memory");
};
constexpr int kAbsent = 0x7FFFFF00; // the first token of a cell that is not there: seen by no row

template <int D, int NT>
__global__ void __launch_bounds__(Lists<D, NT>::kThreads, 1) kv8_lists_kernel(const Kv4 c, const Kv4Batch b, const AttnArgs a)
{
    using LS = Lists<D, NT>;
    constexpr int kWarps = LS::kWarps, kThreads = LS::kThreads, S = LS::kStages, C = LS::kCells;
    constexpr int G = D / 64, KS = 4 * G;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t s_bars[kWarps * S];
    __shared__ int s_first[kWarps * S][C];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    uint8_t *const ring = smem + warp * S * LS::kStage;
    int(*const first_of)[C] = s_first + warp * S;
    const uint32_t rings = smem_addr(ring), bars = smem_addr(s_bars) + warp * S * 8;
    if (lane == 0)
        for (int i = 0; i < S; ++i)
            mbar_init(bars + 8 * i, 1);
    fence_mbar_init();
    __syncwarp();
    if (blockIdx.x == 0)
        for (int i = tid; i < b.n_seqs; i += kThreads)
            kv4_seq(c, b, i, true);
    const int shift = c.page_shift - 4, mask = (1 << shift) - 1;
    const int64_t segments = b.n_tokens * c.n_kv_heads;
    uint32_t used = 0;
    bool dead = false;
#pragma unroll 1
    for (int64_t seg = (int64_t)warp * gridDim.x + blockIdx.x; seg < segments; seg += (int64_t)gridDim.x * kWarps) {
        const int64_t token = quotient(seg, c.n_kv_heads);
        const int head = (int)(seg - token * c.n_kv_heads);
        // the rows of Q: row 8 j + g, channels 64 e + 16 t ..
        uint4 qw[NT][G][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const bool real = 8 * j + g < a.ratio;
            const uint16_t *q = a.q + token * a.q_stride + ((int64_t)head * a.ratio + 8 * j + g) * D + 16 * t;
#pragma unroll
            for (int e = 0; e < G; ++e)
#pragma unroll
                for (int f = 0; f < 2; ++f)
                    qw[j][e][f] = real ? ldg_nc128(q + 64 * e + 8 * f) : make_uint4(0, 0, 0, 0);
        }
        const int i = kv4_find(b, token);
        Kv4Seq s{};
        if (i >= 0)
            s = kv4_seq(c, b, i, false);
        const int64_t seen = i >= 0 && s.first >= 0 && token - s.first < s.n_new ? s.len - s.n_new + (token - s.first) + 1 : 0;
        const int most = s.len, limit = seen > 0 && s.len > 0 ? (int)seen : 0;
        const int32_t *const list = a.pages + seg * a.n_list;
        const int cells = a.n_list << shift;
        int mine = dead || limit == 0 ? 0 : (cells + C - 1) / C; // stages
        const uint8_t *const heads = c.pool + kv8_head_offset<D>(c, 0, a.layer, head);
        uint64_t where = 0;
        int begins = kAbsent;
        uint32_t have = 0;
        int top = -1;        // of a list that is not in order, the last entry so far that counts
        bool ordered = true; // the list's entries so far
        const auto fetch = [&](int x) {
            const int z = C * x;
            if ((z & 31) == 0) {
                where = 0;
                begins = kAbsent;
                const int j = min(z + lane, cells - 1) >> shift, index = list[j], before = list[max(j - 1, 0)];
                bool counts = z + lane < cells && index != -1;
                const bool odd = __any_sync(~0u, !in_order(c, j, before, index, most));
                if (odd || !ordered) {
                    const int from = z >> shift, last = __shfl_sync(~0u, j, 31);
                    if (ordered && from > 0) { // up to here it is in order
                        top = __shfl_sync(~0u, before, 0);
                        top = top == -1 ? kEnded : top;
                    }
                    ordered = false;
                    counts &= follow(c, list, from, top, j, last, most);
                }
                if (counts)
                    where = listed_cell<D>(c, s.row, heads, z + lane, index, limit, &begins);
                if (where == 0)
                    begins = kAbsent;
                // nothing is listed from here on
                if (x > 0 && !__any_sync(~0u, where != 0)) {
                    const bool rest = z + lane < cells && list[(z + lane) >> shift] != -1;
                    if (!__any_sync(~0u, rest))
                        mine = x;
                }
            }
            if (x >= mine)
                return;
            const uint32_t st = (used + x) % S, bar = bars + 8 * st;
            const uint32_t there = __ballot_sync(~0u, where != 0) >> (z & 31) & ((1u << C) - 1);
            have = (have & ~(1u << st)) | (uint32_t)(there != 0) << st;
            // the lanes of the stage's cells; of cells side by side the first one copies both
            static_assert(C == 2, "the second lane tells whether they are");
            const int who = lane - (z & 31);
            const uint64_t before = __shfl_up_sync(~0u, where, 1);
            const bool joined = where != 0 && who == 1 && where == before + Kv8Cell<D>::kBytes && before != 0;
            const uint32_t pair = __ballot_sync(~0u, joined);
            if (lane == 0)
                mbar_arrive_expect_tx(bar, __popc(there) * Kv8Cell<D>::kBytes);
            __syncwarp();
            if (who >= 0 && who < C) {
                first_of[st][who] = begins;
                if (where != 0 && !joined)
                    bulk_load(rings + st * LS::kStage + who * Kv8Cell<D>::kBytes, (const void *)where,
                              Kv8Cell<D>::kBytes << (who == 0 && pair != 0), bar);
            }
            __syncwarp();
        };
        for (int x = 0; x < S - 1 && x < mine; ++x)
            fetch(x);

        uint2 qb[NT][KS];
        float factor[NT]; // of row 8 j + g
        Rows<D, NT> r;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            factor[j] = split_q<D>(qw[j], a.scale, true, [&](int z, uint2 v) { qb[j][z] = v; });
            r.scale[j][0] = __shfl_sync(~0u, factor[j], 8 * t);
            r.scale[j][1] = __shfl_sync(~0u, factor[j], 8 * t + 4);
        }
        r.clear();
#pragma unroll 1
        for (int x = 0; x < mine; ++x) {
            if (x + S - 1 < mine) {
                __syncwarp(); // the stage that is filled now was read by all lanes
                fetch(x + S - 1);
            }
            const uint32_t st = (used + x) % S;
            kv4_wait(bars + 8 * st, ((used + x) / S) & 1, c.status, dead);
            if (__any_sync(~0u, dead)) { // as in kv8_rows_kernel
                for (int z = x; z < x + S && z < mine; ++z) {
                    dead = false;
                    kv4_wait(bars + 8 * ((used + z) % S), ((used + z) / S) & 1, c.status, dead);
                }
                dead = true;
                mine = x;
                break;
            }
            if (have >> st & 1u)
                r.template take<C>(ring + st * LS::kStage, {first_of[st][0], first_of[st][1]}, limit, limit, lane,
                                   [&](int j, int z) { return qb[j][z]; }, [&](int, int) { return limit; });
        }
        used += mine;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                float l = r.l[j][n];
                l += __shfl_xor_sync(~0u, l, 4);
                l += __shfl_xor_sync(~0u, l, 8);
                l += __shfl_xor_sync(~0u, l, 16);
                const int row = 8 * j + 2 * t + n;
                if (row >= a.ratio)
                    continue;
                const int64_t h = (int64_t)head * a.ratio + row;
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                uint16_t *const out = a.out + token * a.out_stride + h * D + 4 * g;
#pragma unroll
                for (int q = 0; q < D / 32; ++q) {
                    const float4 y = r.four(j, n, q);
                    *(uint2 *)(out + 32 * q) = make_uint2(f32_to_bf16_rn(y.x * inv) | ((uint32_t)f32_to_bf16_rn(y.y * inv) << 16),
                                                          f32_to_bf16_rn(y.z * inv) | ((uint32_t)f32_to_bf16_rn(y.w * inv) << 16));
                }
                if (a.lse && g == 0)
                    a.lse[token * a.n_q_heads + h] = l == 0.0f ? -INFINITY : (log2f(l) - r.mo[j][n]) * kLn2;
            }
        __syncwarp(); // the stages are read before the next list's cells overwrite them
    }
}

template <int D, int NT, bool kListed>
nm_status launch(const Kv4 &c, const Kv4Batch &b, const AttnArgs &a, const Kv4Work &w, cudaStream_t st)
{
    constexpr size_t kMost = Smem<D, NT>::kSeqs + kKv4MaxSeqs * 24 + 8;
    static_assert(kMost + 1024 <= 227 * 1024, "shared memory");
    static OncePerDevice once;
    if (!once(w.device, [] {
            return cudaFuncSetAttribute(kv8_rows_kernel<D, NT, kListed>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost) ==
                   cudaSuccess;
        }))
        return NM_ERR_CUDA;
    const size_t smem = Smem<D, NT>::kSeqs + (size_t)(b.n_seqs + 1) * 8 + (size_t)b.n_seqs * sizeof(Kv4Seq);
    const unsigned grid = (unsigned)(w.num_sms * (NT <= 2 ? 2 : 1)); // at most kKv4Counters / 4
    kv8_rows_kernel<D, NT, kListed><<<grid, kThreads, smem, st>>>(c, b, a);
    return cudaGetLastError() == cudaSuccess ? NM_OK : NM_ERR_CUDA;
}

template <int D, int NT>
nm_status launch_lists(const Kv4 &c, const Kv4Batch &b, const AttnArgs &a, const Kv4Work &w, cudaStream_t st)
{
    using LS = Lists<D, NT>;
    static OncePerDevice once;
    if (!once(w.device, [] {
            return cudaFuncSetAttribute(kv8_lists_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, LS::kBytes) ==
                   cudaSuccess;
        }))
        return NM_ERR_CUDA;
    kv8_lists_kernel<D, NT><<<(unsigned)w.num_sms, LS::kThreads, LS::kBytes, st>>>(c, b, a);
    return cudaGetLastError() == cudaSuccess ? NM_OK : NM_ERR_CUDA;
}

} // namespace

// Two parts of a CTA: of two CTAs to an SM with up to 16 rows, or of one with up to 32; here for 32 rows
// and as many CTAs as the counters could serve.
size_t kv8_partial_bytes(int head_dim)
{
    const size_t rows = (size_t)kKv4Counters / 2 * 2 * 32 * (head_dim + 2) * 4;
    const size_t prompt = kv8_prompt_partial_bytes(head_dim);
    return rows > prompt ? rows : prompt;
}

nm_status kv8_launch_attention(const Kv4 &c, const Kv4Batch &b, const Kv4Attn &at, int64_t max_new, const int32_t *pages,
                               int n_list, const Kv4Work &w, cudaStream_t st)
{
    const AttnArgs a{at.layer, at.n_q_heads / c.n_kv_heads, at.n_q_heads, (const uint16_t *)at.q, at.q_stride,
                     at.scale, (uint16_t *)at.out, at.out_stride, at.lse, w.counters, w.partials, pages, n_list};
    // Figures: head size 128, 8 kv heads, us.
    if (pages) {
        // 16 pages of 64 tokens, a CTA per piece of a list against a warp per list. 32 heads: 20 tokens 14 against 23; 80: 35,
        // 37; 112: 44, 37; 160: 61, 44; 512: 164, 113. 128 heads: 40 tokens 32 against 36; 96: 56, 47; 112: 65, 48; 512: 234, 172.
        // Head size 64, 32 heads: 80 tokens 32 against 30; 112: 41, 30; 512: 145, 91. Other lists of 32 heads at 112 tokens: 8 pages
        // of 16 tokens 16 against 9; 64 of 16 46, 38; 4 of 64 19, 13; 8 of 128 44, 36; where half of the lists have two pages of
        // 16, at 160 tokens 59, 44. Lists of more than a hundred cells would stay with CTAs a little longer: 64 pages of 64 tokens
        // at 112 tokens 114 against 136; 160: 178, 162; 512: 494, 427; of 128 heads 160: 239, 301; 512: 665, 648.
        // More than 16 query heads to a kv head are several tiles, which that kernel does not cut (512 tokens of 256 heads:
        // 9, 16, 64 pages of 64 tokens 333, 450, 1282).
        const int rows = a.ratio;
        if (rows <= 16 && b.n_tokens * c.n_kv_heads >= 5 * (int64_t)w.num_sms) {
            if (c.head_dim == 64)
                return rows <= 8 ? launch_lists<64, 1>(c, b, a, w, st) : launch_lists<64, 2>(c, b, a, w, st);
            return rows <= 8 ? launch_lists<128, 1>(c, b, a, w, st) : launch_lists<128, 2>(c, b, a, w, st);
        }
        if (c.head_dim == 64)
            return rows <= 8 ? launch<64, 1, true>(c, b, a, w, st) : launch<64, 2, true>(c, b, a, w, st);
        return rows <= 8 ? launch<128, 1, true>(c, b, a, w, st) : launch<128, 2, true>(c, b, a, w, st);
    }
    // A sequence's rows and this kernel with 1, 2, 3 n-tiles, kv8_prompt.cu:
    //   4 x 2 new tokens of 32 heads (8 rows), after 12288:    22, 28, 37,  77
    //   4 x 4 of 32 heads (16 rows), after 12288:              33, 28, 38,  77
    //   4 x 5 of 32 heads (20 rows), after 12288:              42, 41, 38,  76
    //   8 x 3 of 64 heads (24 rows), after 8192:               55, 52, 46,  93
    //   4 x 5 of 40 heads (25 rows), after 12288:              53, 42, 57,  78
    //   1 x 16 of 32 heads (64 rows), after 32768:             65, 50, 55,  69
    //   4 x 24 of 32 heads (96 rows), after 8192:              93, 68, 70,  61
    //   4 x 64 of 32 heads (256 rows), after 8192:            231, 155, 167, 59
    //   2 x 20 of 32 heads (80 rows), 1024 in all:             18, 17, 17,  30
    //   1 x 32 of 32 heads (128 rows), 1032 in all:            14, 17, 17,  28, but after 32768 118, 83, 94, 63
    // Lengths are on the device: a few rows of one sequence, which may be short, stay here.
    const int64_t rows = (max_new < 65 ? max_new : 65) * a.ratio;
    if (rows > 64 && b.n_tokens * at.n_q_heads > 1024)
        return kv8_launch_prompt(c, b, at, w, st);
    if (c.head_dim == 64)
        return rows <= 8                 ? launch<64, 1, false>(c, b, a, w, st)
               : rows > 16 && rows <= 24 ? launch<64, 3, false>(c, b, a, w, st)
                                         : launch<64, 2, false>(c, b, a, w, st);
    return rows <= 8                 ? launch<128, 1, false>(c, b, a, w, st)
           : rows > 16 && rows <= 24 ? launch<128, 3, false>(c, b, a, w, st)
                                     : launch<128, 2, false>(c, b, a, w, st);
}

} // namespace nm
