// kv4_attn.cu -- attention of few queries over the 4-bit paged cache (decode
// steps and drafted tokens).
//
// For one sequence and kv head, the rows are its queries times the query heads
// that share the kv head; a tile holds 8 NT of them. A warp takes the cache two
// cells (16 tokens each) at a time:
//
//   S^T [16 tokens][rows] = codes(K) Q^T      m16n8k16, A = codes - 8 as fp16
//   s = scale_t S^T + mid_t sum(q) over the groups of 64 channels, in fp32 (the
//                                   middles as one more product, of k = 8)
//   p = 2^(s - m + 6)                         m: the row's running maximum
//   O^T [channels][rows] += V^T P^T           A = V as fp16, B = P as fp16
//
// The codes are exact in fp16, q is made so by a power of two per row, and the
// scale is applied in fp32, so scores carry fp32 rounding only. V's values are
// rounded once to fp16 (2^-11), like the weights p. m is raised only when a score
// passes it by 2^8 (p <= 2^14 stays inside fp16, and weights down to 2^-30 of
// the largest keep a digit): the warp votes instead of reducing.
//
// The layout of a cell is the operands' own: lane l reads 16 bytes at 16 l, so K
// and V need no transposition on the way to the registers.
//
// A (sequence, kv head, tile) is a segment. Each CTA gets one piece of one where that
// can be balanced, else an even part of the line of all segments (see the kernel's
// beginning): a piece costs about 5 us before and after its cells, as much as eight
// units (pairs of cells) of each warp. A CTA's warps take the units of a piece in
// turn and are joined in shared memory. A segment that was cut is joined by the
// last of its CTAs, in CTA order, from the workspace.
//
// Measured (one GB300, D = 128): 131071 tokens, 64 query heads over 8: 43 us, 3.5 TB/s
// (0.52 of the measured copy rate; the cache is read once). What bounds it is a unit's
// chain in its warp, scores, weights, values, with four warps a scheduler to hide it:
// 345 instructions a cell issue at 0.56 a cycle and scheduler, and a warp waits most for
// results of fixed latency, then for the tensor pipe (active 22%); 8 us are start and
// joins. Eight sequences of 1 to 8191 tokens 19 us, four times five drafted tokens (25
// rows) at 9001 to 16385 tokens 47 us (248 registers leave two warps a scheduler), 20
// rows of four sequences of 12288 tokens 40 us, 129 tokens 8.9 us. Steps on the way for the
// first: 67 us with loads straight to registers; 62 by bulk copies; 50.6 with masks at
// the end only and addresses a round ahead; 43.9 two cells at a time and a join of
// independent loads.
#include <type_traits>

#include "kv4.cuh"

namespace nm {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 2;          // cells that a warp takes at a time
constexpr int kTokens = kUnit * kKv4Cell;
constexpr int64_t kMinShare = 8;  // units of a CTA at least: one for each warp
constexpr int kWhole = 16;        // when none has more units than this, no segment is cut
constexpr float kMoreUnits = 12.0f; // of about 0.3 us in a full CTA; a second piece costs about 4 us
constexpr int kOver = 8;          // units that starting and ending a piece costs as much as
constexpr float kShift = 6.0f;    // p = 2^(s - m + kShift)
constexpr float kSlack = 8.0f;    // a score may pass m by this much
constexpr float kNone = 1e38f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma1688(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b)
{
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(b));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ float exp2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *(__half2 *)&x; }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *(uint32_t *)&x; }

// Nibble N (0..3) of both halves of w, minus `bias`, as two fp16 numbers: the
// bits under an exponent of 2^10 are 1024 + n (or 1024 + 16 n), so the result is
// exact.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
template <int N> __device__ __forceinline__ __half2 nibble(uint32_t w, float bias)
{
    const uint32_t x = N >= 2 ? w >> 8 : w;
    if (N % 2 == 0)
        return __hadd2(as_half2(and_or(x, 0x000F000Fu, 0x64006400u)), __float2half2_rn(-1024.0f - bias));
    return __hfma2(as_half2(and_or(x, 0x00F000F0u, 0x64006400u)), __float2half2_rn(0.0625f),
                   __float2half2_rn(-64.0f - bias));
}

// A cell's parts in a lane's registers, from the cell in shared memory.
template <int D> struct CellK {
    static constexpr int G = Kv4Cell<D>::G;
    uint32_t w[2][2 * G]; // tokens g, g + 8: 16 channels of each group
    uint32_t p[2][G];     // (s, mid)
};
template <int D> struct CellV {
    static constexpr int G = Kv4Cell<D>::G;
    uint32_t w[G][4];     // (quad 0, pair 0), (quad 1, pair 0), (quad 0, pair 1), (quad 1, pair 1)
    uint32_t p[2][2 * G]; // token pairs t, t + 4: per group (s, s), (mid, mid)
};
template <int D> __device__ __forceinline__ void lds_k(CellK<D> &r, const uint8_t *cell, int lane)
{
    using C = Kv4Cell<D>;
    const int g = lane >> 2;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (D == 128) {
            const uint4 x = *(const uint4 *)(cell + e * 512 + lane * 16);
            r.w[e][0] = x.x;
            r.w[e][1] = x.y;
            r.w[e][2 * C::G - 2] = x.z;
            r.w[e][2 * C::G - 1] = x.w;
            const uint2 p = *(const uint2 *)(cell + C::kKp + (g + 8 * e) * 8);
            r.p[e][0] = p.x;
            r.p[e][C::G - 1] = p.y;
        } else {
            const uint2 x = *(const uint2 *)(cell + e * 256 + lane * 8);
            r.w[e][0] = x.x;
            r.w[e][1] = x.y;
            r.p[e][0] = *(const uint32_t *)(cell + C::kKp + (g + 8 * e) * 4);
        }
    }
}
template <int D> __device__ __forceinline__ void lds_v(CellV<D> &r, const uint8_t *cell, int lane)
{
    using C = Kv4Cell<D>;
    const int t = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (D == 128) {
            const uint4 q = *(const uint4 *)(cell + C::kVp + (t + 4 * e) * 16);
            r.p[e][0] = q.x;
            r.p[e][1] = q.y;
            r.p[e][2 * C::G - 2] = q.z;
            r.p[e][2 * C::G - 1] = q.w;
        } else {
            const uint2 q = *(const uint2 *)(cell + C::kVp + (t + 4 * e) * 8);
            r.p[e][0] = q.x;
            r.p[e][1] = q.y;
        }
    }
#pragma unroll
    for (int e = 0; e < C::G; ++e) {
        const uint4 x = *(const uint4 *)(cell + C::kV + e * 512 + lane * 16);
        r.w[e][0] = x.x;
        r.w[e][1] = x.y;
        r.w[e][2] = x.z;
        r.w[e][3] = x.w;
    }
}

// A copy of n bytes (a multiple of 16, 16-byte aligned ends) to shared memory,
// counted on an mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t n, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(n), "r"(bar)
                 : "memory");
}

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
    static constexpr int kStages = NT <= 2 ? 2 : 4; // units of a warp in flight or in use
    static constexpr int kStage = kUnit * Kv4Cell<D>::kBytes;
    // Rows of one n-tile leave room for both cells of a unit at once; otherwise one after the other.
    static constexpr int kAtOnce = NT == 1 ? 2 : 1;
    static constexpr int kSteps = D / 16;
    // the warps' rings; when a piece is done, the warps' parts (m, l, O) in their place
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kMerge = kWarps * kRows * (2 + kPitch) * 4;
    static constexpr int kJoin = (kKv4Counters / 4 * kRows + 2 * kRows) * 4; // weights of the parts of a segment
    static constexpr int kBig = kRing > kMerge ? (kRing > kJoin ? kRing : kJoin) : (kMerge > kJoin ? kMerge : kJoin);
    // Q in B fragments: [n-tile][k-step][lane][2], the sums of q as one more (of k = 8), then the rows' RowInfo
    static constexpr int kQ = kBig, kSums = kQ + NT * kSteps * 256, kInfo = kSums + NT * 128, kBars = kInfo + kRows * 8;
    static constexpr int kSeqs = kBars + kWarps * kStages * 8;
};

// Pieces of a segment that is cut every `chunk` units.
__device__ __forceinline__ int pieces_of(int units, int chunk) { return (int)((uint32_t)(units + chunk - 1) / (uint32_t)chunk); }
__device__ __forceinline__ int units_of(int len) { return len > 0 ? (len + kTokens - 1) / kTokens : 1; }
// a / b of numbers that fit 32 bits as a rule (a 64-bit division takes ten times as long).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
__device__ __forceinline__ int64_t ceil_div(int64_t a, int64_t b) { return quotient(a + b - 1, b); }

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, NT <= 2 ? 2 : 1)
    attn_rows_kernel(const Kv4 c, const Kv4Batch b, const AttnArgs a)
{
    constexpr int G = Kv4Cell<D>::G;
    constexpr int RT = 8 * NT;
    constexpr int KS = 4 * G; // k-steps of 16 channels
    using SM = Smem<D, NT>;
    constexpr int S = SM::kStages, U = SM::kAtOnce;
    extern __shared__ __align__(128) uint8_t smem[];
    float *const sm_m = (float *)smem, *const sm_l = sm_m + kWarps * RT, *const sm_o = sm_l + kWarps * RT;
    uint2 *const sm_q = (uint2 *)(smem + SM::kQ);
    uint32_t *const sm_sums = (uint32_t *)(smem + SM::kSums);
    RowInfo *const sm_info = (RowInfo *)(smem + SM::kInfo);
    int64_t *const pre = (int64_t *)(smem + SM::kSeqs);      // [n_seqs + 1]
    Kv4Seq *const seqs = (Kv4Seq *)(pre + b.n_seqs + 1);     // [n_seqs]
    __shared__ uint32_t s_last;
    __shared__ int s_chunk;
    __shared__ bool s_rest; // some rows belong to no sequence
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    uint8_t *const ring = smem + warp * S * SM::kStage;
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
        longest = max(longest, s.n_new == 0 ? 0 : units_of(s.len));
        pre[i + 1] = (int64_t)((uint32_t)(s.n_new * a.ratio + RT - 1) / RT) * c.n_kv_heads; // segments
    }
    const bool is_long = __syncthreads_or(longest > kWhole);
    if (warp == 0) {
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
    const int64_t total = pre[b.n_seqs];
    int64_t share = ceil_div(total, gridDim.x);
    if (!chunk && share < kMinShare + kOver)
        share = kMinShare + kOver;
    const int64_t lo = (int64_t)blockIdx.x * share, hi = lo + share < total ? lo + share : total;
    const int shift = c.page_shift - 4;
    uint32_t used = 0; // cells of this warp so far: the next takes stage used % S
    bool dead = false;

    for (int64_t pos = lo; pos < hi;) {
        int i;
        {
            int l = 0, h = b.n_seqs; // pre[l] <= pos < pre[h]
            while (h - l > 1) {
                const int m = (l + h) >> 1;
                if (pre[m] <= pos)
                    l = m;
                else
                    h = m;
            }
            i = l;
        }
        const Kv4Seq s = seqs[i];
        const int units = units_of(s.len);
        const int over = chunk ? 0 : kOver, per = chunk ? pieces_of(units, chunk) : kOver + units; // steps of the segment
        const int64_t seg = quotient(pos - pre[i], per);
        const int64_t seg_lo = pre[i] + seg * per, seg_hi = seg_lo + per;
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
        const int tiles = (rows + RT - 1) / RT;
        const int head = (int)quotient(seg, tiles);
        const int row0 = (int)(seg - (int64_t)head * tiles) * RT; // first row of the tile
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

        // The warp's units are c0 + warp, + kWarps, ... Lanes 2 n, 2 n + 1 hold the addresses of the
        // cells of every 16th (0: its page is none of the pool's, or it is past the sequence's end);
        // `have` has a bit for each cell of a stage that was filled.
        int mine = !dead && s.len > 0 && c1 - c0 > warp ? (c1 - c0 - warp + kWarps - 1) / kWarps : 0;
        const uint8_t *const heads = c.pool + kv4_cell_offset<D>(c, 0, a.layer, head, 0);
        uint64_t where = 0;
        uint32_t have = 0;
        const auto fetch = [&](int x) {
            if ((x & 15) == 0) {
                const int cell = kUnit * (c0 + warp + (x + (lane >> 1)) * kWarps) + (lane & 1);
                where = 0;
                if (x + (lane >> 1) < mine && cell * kKv4Cell < s.len) {
                    const int page = kv4_page(c, s.row, cell >> shift);
                    if (page >= 0)
                        where = (uint64_t)(heads + page * c.page_bytes + (cell & ((1 << shift) - 1)) * Kv4Cell<D>::kBytes);
                    else
                        kv4_bad(c);
                }
            }
            const uint64_t src = __shfl_sync(~0u, where, 2 * (x & 15) + (lane & 1));
            const uint32_t st = (used + x) % S, bar = bars + 8 * st;
            const uint32_t both = __ballot_sync(~0u, src != 0) & 3u;
            have = (have & ~(3u << (2 * st))) | both << (2 * st);
            if (lane == 0)
                mbar_arrive_expect_tx(bar, __popc(both) * Kv4Cell<D>::kBytes);
            __syncwarp();
            if (lane < kUnit && src)
                bulk_load(rings + st * SM::kStage + lane * Kv4Cell<D>::kBytes, (const void *)src, Kv4Cell<D>::kBytes, bar);
        };
        for (int x = 0; x < (S > 2 ? S - 1 : S) && x < mine; ++x)
            fetch(x);

        // Q as the B operand
        if (warp < NT) {
            const int j = warp;
            float x[G][16];
            float top = 0.0f;
#pragma unroll
            for (int e = 0; e < G; ++e)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const uint32_t ws[4] = {qw[e][f].x, qw[e][f].y, qw[e][f].z, qw[e][f].w};
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        x[e][8 * f + 2 * n] = bf16lo_to_f32(ws[n]);
                        x[e][8 * f + 2 * n + 1] = bf16hi_to_f32(ws[n]);
                    }
                }
#pragma unroll
            for (int e = 0; e < G; ++e)
#pragma unroll
                for (int n = 0; n < 16; ++n)
                    top = fmaxf(top, fabsf(x[e][n]));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
            // 2^-e brings the row's largest magnitude into [1, 2): what is at least 2^-17 of it is
            // exact in fp16 (eight bits above 2^-24), the rest is rounded to 2^-24
            uint32_t e2 = (__float_as_uint(top) >> 23) & 0xFFu;
            e2 = e2 == 0xFFu || e2 == 0 ? 127u : e2 > 253u ? 253u : e2;
            const float up = __uint_as_float(e2 << 23); // the sign of the scale goes with q
            const float down = a.scale < 0.0f ? -__uint_as_float((254u - e2) << 23) : __uint_as_float((254u - e2) << 23);
            float sums[G];
#pragma unroll
            for (int e = 0; e < G; ++e) {
                sums[e] = 0.0f;
#pragma unroll
                for (int n = 0; n < 16; ++n) {
                    x[e][n] = __half2float(__float2half_rn(x[e][n] * down));
                    sums[e] += x[e][n];
                }
                sums[e] += __shfl_xor_sync(~0u, sums[e], 1);
                sums[e] += __shfl_xor_sync(~0u, sums[e], 2);
                // word f of 8 channels: nibble pairs (0,4),(1,5) and (2,6),(3,7) are two k-steps
#pragma unroll
                for (int f = 0; f < 2; ++f)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float *y = &x[e][8 * f + 2 * h];
                        sm_q[(j * KS + 4 * e + 2 * f + h) * 32 + lane] =
                            make_uint2(pack_half2(y[0], y[4]), pack_half2(y[1], y[5]));
                    }
            }
            // the middles of the groups meet the sums of q, in two fp16 parts: k = 0, 1 and k = 2, 3
            const float h0 = __half2float(__float2half_rn(sums[0]));
            const float h1 = G == 2 ? __half2float(__float2half_rn(sums[G - 1])) : 0.0f;
            const float l1 = G == 2 ? sums[G - 1] - h1 : 0.0f;
            sm_sums[32 * j + lane] = t == 0 ? pack_half2(h0, h1) : t == 1 ? pack_half2(sums[0] - h0, l1) : 0u;
            if (t == 0)
                sm_info[8 * j + g] = RowInfo{fmaxf(up * (fabsf(a.scale) * kLog2e), 1e-30f),
                                             real ? s.len - s.n_new + qrow / a.ratio + 1 : 0};
        }
        __syncthreads();
        // with one n-tile Q stays in registers
        constexpr bool kKeepQ = NT == 1;
        uint2 qb[kKeepQ ? KS : 1];
        uint32_t qs[NT];
        float scale[NT][2];
        if (kKeepQ) {
#pragma unroll
            for (int x = 0; x < KS; ++x)
                qb[x % (kKeepQ ? KS : 1)] = sm_q[x * 32 + lane];
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            qs[j] = sm_sums[32 * j + lane];
            scale[j][0] = sm_info[8 * j + 2 * t].scale;
            scale[j][1] = sm_info[8 * j + 2 * t + 1].scale;
        }

        float o[NT][G][4][4] = {}; // [n-tile][group][m-tile][fragment]
        // mo = kShift - m, the running maximum; before the first score so large that any raises m
        float mo[NT][2], l[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j)
            mo[j][0] = mo[j][1] = kNone, l[j][0] = l[j][1] = 0.0f;

#pragma unroll 1
        for (int x = 0; x < mine; ++x) {
            if (S > 2 && x + S - 1 < mine) {
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
            const uint32_t filled = have >> (2 * st) & 3u;
#pragma unroll 1
            for (int v0 = 0; v0 < kUnit; v0 += U) {
                const uint8_t *const cell_at = ring + st * SM::kStage + v0 * Kv4Cell<D>::kBytes;
                const int tok = (c0 + warp + x * kWarps) * kTokens + v0 * kKv4Cell;

                // scores
                float sc[U][NT][4];
#pragma unroll
                for (int v = 0; v < U; ++v) {
                    CellK<D> r;
                    lds_k<D>(r, cell_at + v * Kv4Cell<D>::kBytes, lane);
                    const uint32_t mid0 = G == 2 ? __byte_perm(r.p[0][0], r.p[0][G - 1], 0x7632) : r.p[0][0] >> 16;
                    const uint32_t mid1 = G == 2 ? __byte_perm(r.p[1][0], r.p[1][G - 1], 0x7632) : r.p[1][0] >> 16;
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        sc[v][j][0] = sc[v][j][1] = sc[v][j][2] = sc[v][j][3] = 0.0f;
                        mma1688(sc[v][j], mid0, mid1, qs[j]);
                    }
#pragma unroll
                    for (int e = 0; e < G; ++e) {
                        float acc[NT][4] = {};
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            uint32_t af[2][4];
                            const uint32_t w0 = r.w[0][2 * e + f], w1 = r.w[1][2 * e + f];
                            af[0][0] = as_u32(nibble<0>(w0, 8.0f));
                            af[0][1] = as_u32(nibble<0>(w1, 8.0f));
                            af[0][2] = as_u32(nibble<1>(w0, 8.0f));
                            af[0][3] = as_u32(nibble<1>(w1, 8.0f));
                            af[1][0] = as_u32(nibble<2>(w0, 8.0f));
                            af[1][1] = as_u32(nibble<2>(w1, 8.0f));
                            af[1][2] = as_u32(nibble<3>(w0, 8.0f));
                            af[1][3] = as_u32(nibble<3>(w1, 8.0f));
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int j = 0; j < NT; ++j) {
                                    const int z = 4 * e + 2 * f + h;
                                    const uint2 q = kKeepQ ? qb[z % (kKeepQ ? KS : 1)] : sm_q[(j * KS + z) * 32 + lane];
                                    mma16816(acc[j], af[h], q.x, q.y);
                                }
                        }
                        const float k0 = __low2float(as_half2(r.p[0][e])), k1 = __low2float(as_half2(r.p[1][e]));
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int f = 0; f < 4; ++f) // token g + 8 (f / 2), row 2 t + f % 2
                                sc[v][j][f] = fmaf(f < 2 ? k0 : k1, acc[j][f], sc[v][j][f]);
                    }
                }
                // a row may see only part of the cells, or a cell may not be there
                if (tok + U * kKv4Cell > tile_first || filled != 3u) {
#pragma unroll
                    for (int v = 0; v < U; ++v)
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int f = 0; f < 4; ++f) {
                                const int limit = sm_info[8 * j + 2 * t + (f & 1)].limit;
                                const bool sees = tok + v * kKv4Cell + g + 8 * (f >> 1) < limit && filled >> (v0 + v) & 1;
                                sc[v][j][f] = sees ? sc[v][j][f] : -INFINITY;
                            }
                }
                float top = -INFINITY;
                float y[U][NT][4];
#pragma unroll
                for (int v = 0; v < U; ++v)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            y[v][j][f] = fmaf(sc[v][j][f], scale[j][f & 1], mo[j][f & 1]);
                            top = fmaxf(top, y[v][j][f]);
                        }
                if (__any_sync(~0u, top > kShift + kSlack)) {
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            float z = -INFINITY;
#pragma unroll
                            for (int v = 0; v < U; ++v)
                                z = fmaxf(z, fmaxf(sc[v][j][n], sc[v][j][n + 2]));
                            z = fmaxf(z, __shfl_xor_sync(~0u, z, 4));
                            z = fmaxf(z, __shfl_xor_sync(~0u, z, 8));
                            z = fmaxf(z, __shfl_xor_sync(~0u, z, 16)) * scale[j][n];
                            const float was = mo[j][n], now = z == -INFINITY ? was : fminf(was, kShift - z);
                            const float by = was == now ? 1.0f : exp2_approx(now - was);
                            mo[j][n] = now;
                            l[j][n] *= by;
#pragma unroll
                            for (int v = 0; v < U; ++v) {
                                y[v][j][n] = fmaf(sc[v][j][n], scale[j][n], now);
                                y[v][j][n + 2] = fmaf(sc[v][j][n + 2], scale[j][n], now);
                            }
#pragma unroll
                            for (int e = 0; e < G; ++e)
#pragma unroll
                                for (int i4 = 0; i4 < 4; ++i4) {
                                    o[j][e][i4][n] *= by;
                                    o[j][e][i4][n + 2] *= by;
                                }
                        }
                }
                uint32_t pb[U][NT][2];
#pragma unroll
                for (int v = 0; v < U; ++v)
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        float p[4];
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            p[f] = exp2_approx(y[v][j][f]);
                            l[j][f & 1] += p[f];
                        }
                        pb[v][j][0] = transpose8x8(pack_half2(p[0], p[1]));
                        pb[v][j][1] = transpose8x8(pack_half2(p[2], p[3]));
                    }

                // O^T += V^T P^T; tokens past the sequence's end, and cells that are not there, hold
                // anything: their V is taken as 0
#pragma unroll
                for (int v = 0; v < U; ++v) {
                    CellV<D> r;
                    lds_v<D>(r, cell_at + v * Kv4Cell<D>::kBytes, lane);
                    const int end = filled >> (v0 + v) & 1 ? s.len - (tok + v * kKv4Cell) : 0; // tokens of the cell
                    if (end < kKv4Cell) {
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int first = 8 * u + 2 * t;
                            const uint32_t keep = (first < end ? 0x0000FFFFu : 0u) | (first + 1 < end ? 0xFFFF0000u : 0u);
#pragma unroll
                            for (int e = 0; e < 2 * G; ++e)
                                r.p[u][e] &= keep;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < G; ++e) {
                        const __half2 s0 = as_half2(r.p[0][2 * e]), m0 = as_half2(r.p[0][2 * e + 1]);
                        const __half2 s1 = as_half2(r.p[1][2 * e]), m1 = as_half2(r.p[1][2 * e + 1]);
                        const auto tile = [&](auto nib) {
                            constexpr int N = decltype(nib)::value;
                            uint32_t af[4];
                            af[0] = as_u32(__hfma2(nibble<N>(r.w[e][0], 8.0f), s0, m0));
                            af[1] = as_u32(__hfma2(nibble<N>(r.w[e][1], 8.0f), s0, m0));
                            af[2] = as_u32(__hfma2(nibble<N>(r.w[e][2], 8.0f), s1, m1));
                            af[3] = as_u32(__hfma2(nibble<N>(r.w[e][3], 8.0f), s1, m1));
#pragma unroll
                            for (int j = 0; j < NT; ++j)
                                mma16816(o[j][e][N], af, pb[v][j][0], pb[v][j][1]);
                        };
                        tile(std::integral_constant<int, 0>{});
                        tile(std::integral_constant<int, 1>{});
                        tile(std::integral_constant<int, 2>{});
                        tile(std::integral_constant<int, 3>{});
                    }
                }
            }
            if (S == 2 && x + S < mine) {
                __syncwarp(); // every lane has read the stage that is filled again
                fetch(x + S);
            }
        }
        used += mine;
        __syncthreads(); // the rings are read: the parts take their place

        // the warp's part to shared memory: rows 2 t, 2 t + 1, channels 64 e + 8 g ..
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                float x = l[j][n];
                x += __shfl_xor_sync(~0u, x, 4);
                x += __shfl_xor_sync(~0u, x, 8);
                x += __shfl_xor_sync(~0u, x, 16);
                const int row = 8 * j + 2 * t + n;
                if (g == 0) {
                    sm_m[warp * RT + row] = mo[j][n] == kNone ? -INFINITY : kShift - mo[j][n];
                    sm_l[warp * RT + row] = x;
                }
                float *dst = sm_o + (warp * RT + row) * SM::kPitch + 8 * g;
#pragma unroll
                for (int e = 0; e < G; ++e) {
                    *(float4 *)(dst + 64 * e) =
                        make_float4(o[j][e][0][n], o[j][e][1][n], o[j][e][2][n], o[j][e][3][n]);
                    *(float4 *)(dst + 64 * e + 4) =
                        make_float4(o[j][e][0][n + 2], o[j][e][1][n + 2], o[j][e][2][n + 2], o[j][e][3][n + 2]);
                }
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
                for (int row = warp; row < RT; row += kWarps) {
                    float M = -INFINITY, L = 0.0f;
                    for (int k = lane; k < n; k += 32)
                        M = fmaxf(M, ldcg_f32(at(k) + row));
                    for (int z = 16; z; z >>= 1)
                        M = fmaxf(M, __shfl_xor_sync(~0u, M, z));
                    for (int k = lane; k < n; k += 32) {
                        const float mk = ldcg_f32(at(k) + row);
                        const float f = mk == M ? 1.0f : exp2_approx(mk - M);
                        weight[k * RT + row] = f;
                        L = fmaf(f, ldcg_f32(at(k) + RT + row), L);
                    }
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
                    for (int k0 = 0; k0 < n; k0 += 8) {
                        float4 z[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            z[k] = k0 + k < n ? __ldcg((const float4 *)(at(k0 + k) + 2 * RT + row * D + ch))
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
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
    if (s_rest)
        kv4_answer_uncovered(b, a.out, a.out_stride, a.n_q_heads * D, a.lse, a.n_q_heads,
                             (int64_t)blockIdx.x * kWarps + warp, (int64_t)gridDim.x * kWarps);
}

template <int D, int NT>
nm_status launch_rows(const Kv4 &c, const Kv4Batch &b, const AttnArgs &a, const Kv4Work &w, cudaStream_t st)
{
    constexpr size_t kMost = Smem<D, NT>::kSeqs + kKv4MaxSeqs * 24 + 8;
    static_assert(kMost + 1024 <= 227 * 1024, "shared memory");
    static OncePerDevice once;
    if (!once(w.device, [] {
            return cudaFuncSetAttribute(attn_rows_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost) ==
                   cudaSuccess;
        }))
        return NM_ERR_CUDA;
    const size_t smem = Smem<D, NT>::kSeqs + (size_t)(b.n_seqs + 1) * 8 + (size_t)b.n_seqs * sizeof(Kv4Seq);
    const unsigned grid = (unsigned)(w.num_sms * (NT <= 2 ? 2 : 1)); // at most kKv4Counters / 4
    attn_rows_kernel<D, NT><<<grid, kThreads, smem, st>>>(c, b, a);
    return cudaGetLastError() == cudaSuccess ? NM_OK : NM_ERR_CUDA;
}

} // namespace

// Two parts of a CTA: of two CTAs to an SM with up to 16 rows, or of one with up to 32; here for 32 rows
// and as many CTAs as the counters could serve, which is still less than the prompt kernel's parts.
size_t kv4_partial_bytes(int head_dim)
{
    const size_t rows = (size_t)kKv4Counters / 2 * 2 * 32 * (head_dim + 2) * 4;
    const size_t prompt = kv4_prompt_partial_bytes(head_dim);
    return rows > prompt ? rows : prompt;
}

nm_status kv4_launch_attention(const Kv4 &c, const Kv4Batch &b, const Kv4Attn &at, int64_t max_new, const Kv4Work &w,
                               cudaStream_t st)
{
    const AttnArgs a{at.layer, at.n_q_heads / c.n_kv_heads, at.n_q_heads, (const uint16_t *)at.q, at.q_stride,
                     at.scale, (uint16_t *)at.out, at.out_stride, at.lse, w.counters, w.partials};
    // By the rows of a kv head. Measured, in us, with 8 kv heads (sequences x new tokens of 4 query
    // heads, tokens in the cache; k: 1024):
    //   D = 128                  NT = 1    2      3      4    prompt
    //    8 rows (4 x 2, 12k)     23.5   31.6   39.8   45.5    68.5
    //   12 rows (4 x 3, 12k)     35.2   31.4   39.8   45.7    68.3
    //   16 rows (4 x 4, 12k)     35.2   31.6   39.8   45.7    68.5   (1 x 4, 32k: 27.3 29.3 31.4 35.5 66.2)
    //   20 rows (4 x 5, 12k)     43.7   47.5   39.8   46.0    68.5   (1 x 5, 32k: 33.7 36.8 31.6 35.7 66.5)
    //   32 rows (4 x 8, 12k)     55.5   47.8   58.3   46.0    68.5
    //   48 rows (4 x 12, 12k)    74.4   60.1   58.3   66.7    68.5   (1 x 12, 32k: 53.9 47.3 46.8 53.9 65.7)
    //   64 rows (4 x 16, 12k)    94.9   76.5   78.5   67.0    69.5   (1 x 16, 32k: 67.5 57.8 58.3 54.2 66.0)
    //   96 rows (4 x 24, 8k)     95.9   76.7   72.6   68.3    56.2
    //  128 rows (1 x 32, 32k)   119.7   93.3   96.9   80.6    63.4   (8 x 32, 512: 35.0 27.3 31.1 25.5 37.8)
    //  256 rows (4 x 64, 8k)    232.9  174.0  168.9  144.0    58.3
    //   D = 64
    //    8 rows (4 x 2, 12k)     18.9   23.2   31.1   34.0    56.2
    //   16 rows (4 x 4, 12k)     26.5   23.2   31.1   33.7    56.2
    //   20 rows (4 x 5, 12k)     30.4   33.4   31.4   34.7    56.2
    //   32 rows (4 x 8, 12k)     39.3   33.7   43.7   34.7    56.2
    //   48 rows (4 x 12, 12k)    51.4   39.8   43.7   49.8    56.0
    //   64 rows (4 x 16, 8k)     47.8   39.3   43.7   39.6    45.7
    //  128 rows (4 x 32, 8k)     82.4   64.2   70.8   60.3    41.6
    // Of all tokens' query heads together, the prompt kernel's 20 to 50 us of start, and join, against
    // tiles that read the cache again (one sequence, 32 heads, D = 128; tokens in the cache before):
    //                               0     1000     8000    32000    40000
    //   24 new,  768    few      12.4     19.1     31.4     66.2     76.4
    //                   prompt   19.6     31.1     46.5     76.4     72.4
    //   32 new, 1024    few      12.4     22.2     35.5     80.5     94.9
    //                   prompt   21.2     31.4     47.8     73.6     68.5
    //   64 new, 2048    few      12.5     23.2     51.9    135.8    164.8
    //                   prompt   25.2     36.0     50.8     78.5     73.1
    // The lengths are on the device, so the choice cannot go by them: up to 1024 rows short contexts
    // gain up to a quarter, and from some 30000 tokens on the other kernel would.
    const int64_t rows = (max_new < 65 ? max_new : 65) * a.ratio;
    if (rows > 64 && b.n_tokens * at.n_q_heads > 1024)
        return kv4_launch_prompt(c, b, at, w, st);
    if (c.head_dim == 64)
        return rows <= 8                 ? launch_rows<64, 1>(c, b, a, w, st)
               : rows > 16 && rows <= 24 ? launch_rows<64, 3>(c, b, a, w, st)
                                         : launch_rows<64, 2>(c, b, a, w, st);
    return rows <= 8    ? launch_rows<128, 1>(c, b, a, w, st)
           : rows <= 16 ? launch_rows<128, 2>(c, b, a, w, st)
           : rows <= 24 ? launch_rows<128, 3>(c, b, a, w, st)
           : rows <= 32 ? launch_rows<128, 4>(c, b, a, w, st)
           : rows <= 48 ? launch_rows<128, 3>(c, b, a, w, st)
                        : launch_rows<128, 4>(c, b, a, w, st);
}

} // namespace nm
