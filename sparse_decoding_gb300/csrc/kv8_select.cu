// kv8_select.cu -- which pages of the 8-bit cache a query attends: the best by a bound on
// its scores.
//
// A full page keeps, per kv head and channel, the greatest and the least of its keys as whole
// numbers of one power of two (kv8.cu). For a query vector q the sum over the channels of
// max(q_d hi_d, q_d lo_d) = max(q_d, 0) hi_d + min(q_d, 0) lo_d bounds q.k of every key of the page. The
// query heads of a kv head share their pages, so their bounds are added: first the heads'
// positive and negative parts (fp32, in order), then one product of 2 D whole numbers for all of
// them. Both sums are rounded to whole numbers up to 127 times a power of two, so a score is a whole
// number below 2^23 times the page's step: exact in fp32 in any order, and two programs that
// compute it select the same pages.
//
// A CTA takes one token and kv head, or, of prompts, a tile of eight tokens of a sequence, whose
// bounds it then reads once: eight lanes share a page, 16 bytes of each bound to a lane, four products to an
// instruction. With few tokens and many pages the CTAs of a cluster share the pages and write the
// scores to the first one's shared memory. There the want-th largest is found by counting the
// scores in bins of their range (2048 bins, of a tile 256 for each token), then of the bin that it lies
// in, until a bin is one number; the pages above it, with the lowest of those equal to it, are
// written in order.
//
// What bounds it: latencies. One token, 8 kv heads, 2048 pages (4.5 MB of bounds): 10 us, of them 3 until the bounds
// are there and 3 for two or three rounds of bins. Prompts: 512 tokens of 256 pages 27 us, where the bounds come from L2
// and issue slots are half used (products, then sums over lanes, for 1 M scores).
#include "kv8.cuh"

namespace nm {
namespace {

constexpr int kTile = 8;  // tokens of a tile of prompts

struct SelectArgs {
    int layer, ratio, want, first, last;
    const uint16_t *q;
    int64_t q_stride;
    int32_t *pages;
    int64_t units; // tiles (at most) times the kv heads
    int cluster;
};

// The two halves of cluster_sync, apart.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// An order of fp32 numbers as unsigned ones.
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t b = __float_as_uint(x);
    return b ^ (b >> 31 ? ~0u : 0x80000000u);
}

// Sums of eight values over the eight lanes of a group: lane n of it gets value n's.
__device__ __forceinline__ int sum_across(int (&x)[8], int n)
{
#pragma unroll
    for (int o = 4; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const int mine = n & o ? x[i + o] : x[i], other = n & o ? x[i] : x[i + o];
            x[i] = mine + __shfl_xor_sync(~0u, other, o);
        }
    return x[0];
}

// The sums of the positive and of the negative parts of a token's query heads, as whole numbers: D
// bytes each to shared memory. What is not finite counts as 0, what is above 2^100 as that. A warp.
template <int D> __device__ __forceinline__ void query_sums(const SelectArgs &a, const uint16_t *q, int8_t *up, int8_t *down)
{
    constexpr int E = D / 32; // channels of a lane
    const int lane = threadIdx.x & 31;
    float p[E] = {}, m[E] = {};
#pragma unroll 4
    for (int h = 0; h < a.ratio; ++h) {
        uint32_t w[2] = {0, 0};
        if (E == 4) {
            const uint2 x = __ldg((const uint2 *)(q + (int64_t)h * D) + lane);
            w[0] = x.x;
            w[1] = x.y;
        } else {
            w[0] = __ldg((const uint32_t *)(q + (int64_t)h * D) + lane);
        }
#pragma unroll
        for (int n = 0; n < E; ++n) {
            const uint32_t b = n & 1 ? w[n / 2] & 0xFFFF0000u : w[n / 2] << 16;
            float x = (b & 0x7FFFFFFFu) < 0x7F800000u ? __uint_as_float(b) : 0.0f;
            x = fminf(fmaxf(x, -0x1p100f), 0x1p100f);
            p[n] = __fadd_rn(p[n], fmaxf(x, 0.0f));
            m[n] = __fadd_rn(m[n], fminf(x, 0.0f));
        }
    }
    uint32_t most = 0;
#pragma unroll
    for (int n = 0; n < E; ++n)
        most = max(most, max(__float_as_uint(p[n]), __float_as_uint(m[n]) & 0x7FFFFFFFu));
    most = __reduce_max_sync(~0u, most);
    // 2^-e for the least e with most <= 127 2^e, at least -100
    int e = (int)((most + 0x01FFFFu) >> 23) - 127 - 6;
    e = e < -100 ? -100 : e;
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    uint32_t u = 0, d = 0;
#pragma unroll
    for (int n = 0; n < E; ++n) {
        u |= ((uint32_t)__float2int_rn(p[n] * inv) & 0xFFu) << (8 * n);
        d |= ((uint32_t)__float2int_rn(m[n] * inv) & 0xFFu) << (8 * n);
    }
    if (E == 4) {
        ((uint32_t *)up)[lane] = u;
        ((uint32_t *)down)[lane] = d;
    } else {
        ((uint16_t *)up)[lane] = (uint16_t)u;
        ((uint16_t *)down)[lane] = (uint16_t)d;
    }
}

// D / 8 bytes as whole words
template <int D> struct Words {
    int w[D / 32];
};
template <int D> __device__ __forceinline__ Words<D> words_at(const void *p)
{
    Words<D> r;
    if (D == 128) {
        const uint4 x = *(const uint4 *)p;
        r.w[0] = (int)x.x;
        r.w[1] = (int)x.y;
        r.w[D / 32 - 2] = (int)x.z;
        r.w[D / 32 - 1] = (int)x.w;
    } else {
        const uint2 x = *(const uint2 *)p;
        r.w[0] = (int)x.x;
        r.w[1] = (int)x.y;
    }
    return r;
}

// A group of W warps that chooses the pages of one query: the CTA, or a warp. Of few warps, since what takes
// the time is the shuffles (with 32 warps to the CTA choosing took 8000 cycles).
template <int W> struct Group {
    static constexpr int kThreads = 32 * W, kEach = 8, kBins = kThreads * kEach, kBits = W == 1 ? 8 : 11;
    static_assert(kBins == 1 << kBits, "bins");
    uint32_t *bins;   // [kBins] of shared memory
    uint32_t *parts;  // [2][32]: the warps' sums, in turn
    uint32_t *found;  // [2]
    int turn = 0;
    __device__ int thread() const { return W == 1 ? threadIdx.x & 31 : threadIdx.x; }
    __device__ void sync()
    {
        if (W == 1)
            __syncwarp();
        else
            __syncthreads();
    }
    // Sum over the threads before this one, and over all; x is the warp's scan already (its lanes up to this one).
    __device__ uint32_t before(uint32_t upto, uint32_t x, uint32_t *total)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (W == 1) {
            *total = __shfl_sync(~0u, upto, 31);
            return upto - x;
        }
        uint32_t *const part = parts + 32 * turn;
        turn ^= 1;
        if (lane == 31)
            part[warp] = upto;
        __syncthreads();
        const uint32_t all = scan32(lane < W ? part[lane] : 0u);
        *total = __shfl_sync(~0u, all, 31);
        const uint32_t prior = __shfl_sync(~0u, all, warp > 0 ? warp - 1 : 0);
        return (warp > 0 ? prior : 0u) + upto - x;
    }
    static __device__ uint32_t scan32(uint32_t x)
    {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t z = __shfl_up_sync(~0u, x, o);
            if ((int)(threadIdx.x & 31) >= o)
                x += z;
        }
        return x;
    }
};

// The least and the greatest over a warp.
__device__ __forceinline__ void range_of(uint32_t &least, uint32_t &most)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        least = min(least, __shfl_xor_sync(~0u, least, o));
        most = max(most, __shfl_xor_sync(~0u, most, o));
    }
}

// The list of one query: the first and last pages, and of the others those with the largest keys, which are
// within least .. most.
template <int W>
__device__ __forceinline__ void choose(const SelectArgs &a, Group<W> &g, const uint32_t *keys, int count, uint32_t least,
                                       uint32_t most, int32_t *out)
{
    using G = Group<W>;
    const int me = g.thread();
    if (count <= a.want) {
        for (int j = me; j < a.want; j += G::kThreads)
            out[j] = j < count ? j : -1;
        return;
    }
    const int lo = a.first, hi = count - a.last; // the others: lo < hi, since first + last <= want < count
    uint32_t need = (uint32_t)(a.want - a.first - a.last); // of the keys within the border's bin still to take
    // each thread's keys lie side by side, four to a load
    const int per = ((count + G::kThreads - 1) / G::kThreads + 3) / 4 * 4;
    const int from = min(me * per, count), to = min(from + per, count);
    const auto each = [&](const auto &f) {
        for (int z = from; z < to; z += 4) {
            const uint4 k = *(const uint4 *)(keys + z);
            f(z, k.x);
            f(z + 1, k.y);
            f(z + 2, k.z);
            f(z + 3, k.w);
        }
    };
    // The border: keys above it are taken, and of those equal to it the lowest pages. The range of
    // the keys is divided into bins, then the bin that the need-th largest lies in, until a bin is one number.
    uint32_t border = ~0u;
    if (need) {
        uint32_t width = most - least; // the keys in question: least .. least + width
#pragma unroll 1
        while (width) {
            const int shift = max(0, 32 - __clz(width) - G::kBits);
            uint4 *const mine = (uint4 *)(g.bins + 8 * (G::kThreads - 1 - me)); // thread 0 has the largest
            mine[0] = mine[1] = make_uint4(0, 0, 0, 0);
            g.sync();
            each([&](int z, uint32_t k) {
                if (z >= lo && z < hi && k - least <= width)
                    atomicAdd(g.bins + ((k - least) >> shift), 1u);
            });
            g.sync();
            const uint4 x = mine[1], y = mine[0];
            const uint32_t n[8] = {x.w, x.z, x.y, x.x, y.w, y.z, y.y, y.x};
            const uint32_t sum = x.x + x.y + x.z + x.w + y.x + y.y + y.z + y.w;
            uint32_t total, above = g.before(G::scan32(sum), sum, &total);
            if (above < need && above + sum >= need) {
                int b = 0;
                bool there = false;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    there = there || above + n[i] >= need;
                    above += there ? 0 : n[i];
                    b += there ? 0 : 1;
                }
                g.found[0] = (uint32_t)(8 * (G::kThreads - 1 - me) + 7 - b);
                g.found[1] = need - above;
            }
            g.sync();
            const uint32_t bin = g.found[0] << shift;
            need = g.found[1];
            least += bin;
            width = min(width - bin, (1u << shift) - 1);
        }
        border = least;
    }
    const auto is_over = [&](int z, uint32_t k) {
        return z < count && (z < lo || z >= hi || (need && k > border));
    };
    const auto is_tie = [&](int z, uint32_t k) { return z >= lo && z < hi && need && k == border; };
    uint32_t mine = 0, total; // keys above the border, and (times 65536) equal to it
    each([&](int z, uint32_t k) { mine += is_over(z, k) ? 1u : is_tie(z, k) ? 65536u : 0u; });
    const uint32_t before = g.before(G::scan32(mine), mine, &total);
    uint32_t n_over = before & 0xFFFFu, n_tie = before >> 16;
    if (mine)
        each([&](int z, uint32_t k) {
            const bool over = is_over(z, k), tie = is_tie(z, k);
            if (over || (tie && n_tie < need))
                out[n_over + min(n_tie, need)] = z;
            n_over += over;
            n_tie += tie;
        });
}

// T tokens of a sequence and one kv head; W warps choose the pages of one token.
template <int D, int T, int W>
__global__ void __launch_bounds__(T == 1 ? 32 * W : 32 * T, T == 1 ? 1 : 3) select_kernel(const Kv4 c, const Kv4Batch b, const SelectArgs a)
{
    constexpr int kThreads = T == 1 ? 32 * W : 32 * T;
    extern __shared__ __align__(16) uint32_t keys[]; // [T][the table's width]
    __shared__ __align__(16) int8_t sq[T][2][D];
    constexpr int kGroups = T == 1 ? 1 : T;
    __shared__ __align__(16) uint32_t bins[kGroups * Group<T == 1 ? W : 1>::kBins];
    __shared__ uint32_t parts[64], found[kGroups][2];
    // the ranges of the keys that the warps scored: of every CTA's of a cluster (in its first CTA), or of each token
    constexpr int kWarps = kThreads / 32, kRanges = T == 1 ? 8 * kWarps : kWarps * T;
    __shared__ uint32_t ranges[kRanges][2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t unit = blockIdx.x / a.cluster;
    const int rank = (int)(blockIdx.x - unit * a.cluster);
    if (a.cluster > 1)
        cluster_arrive();

    if (b.starts) { // rows that belong to no sequence: no pages
        bool rest = !kv4_ends(b);
        for (int x = tid; x < b.n_seqs; x += kThreads)
            rest |= kv4_seq(c, b, x, blockIdx.x == 0).first < 0;
        if (__syncthreads_or(rest)) {
            const int64_t n = (int64_t)c.n_kv_heads * a.want;
            kv4_uncovered(b, (int64_t)blockIdx.x * (kThreads / 32) + warp, (int64_t)gridDim.x * (kThreads / 32), [&](int64_t row) {
                for (int64_t i = lane; i < n; i += 32)
                    a.pages[row * n + i] = -1;
            });
        }
    }

    // the tile: sequence i has the slots from starts[i] / T + i on
    const int head = (int)(unit % c.n_kv_heads);
    const int64_t slot = unit / c.n_kv_heads;
    int i = (int)slot, nth = 0;
    if (b.starts) {
        int lo = 0, hi = b.n_seqs;
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if ((int64_t)(b.starts[m] / T) + m <= slot)
                lo = m;
            else
                hi = m;
        }
        i = lo;
        nth = (int)(slot - ((int64_t)(b.starts[i] / T) + i));
    }
    if (a.cluster > 1)
        cluster_wait(); // the first CTA's shared memory is there from here on
    if (unit >= a.units || i >= b.n_seqs || nth < 0)
        return; // with the whole cluster
    const Kv4Seq s = kv4_seq(c, b, i, !b.starts && head == 0 && rank == 0 && tid == 0);
    const int t0 = nth * T, nt = min(T, s.n_new - t0);
    if (nt <= 0)
        return;
    const auto count_of = [&](int t) { // pages up to the query's own
        const int pos = s.len - s.n_new + t0 + t;
        return pos < 0 ? 0 : (pos >> c.page_shift) + 1;
    };
    const int most = count_of(nt - 1);
    const int width = (c.max_pages + 3) / 4 * 4;

    if (most > a.want) {
        // Pages up to the last query's own (which needs no score) are full. A group of eight lanes
        // asks for the bounds of kAhead of them together, the first ones before the queries' sums.
        constexpr int kAhead = T == 1 ? 8 : 2, kStride = kThreads / 8;
        const int per = (most - 1 + a.cluster - 1) / a.cluster;
        const int z0 = rank * per, z1 = min(most - 1, z0 + per);
        const int n = lane & 7, group = tid >> 3;
        const uint8_t *const tails = c.pool + kv8_head_offset<D>(c, 0, a.layer, head) +
                                     ((int64_t)Kv8Cell<D>::kBytes << (c.page_shift - 4)) + n * (D / 8);
        Words<D> hi[kAhead], lo[kAhead];
        float step[kAhead];
        const auto ask = [&](int z) {
            int page[kAhead];
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                const bool in = z + x * kStride < z1;
                page[x] = in ? kv4_page(c, s.row, z + x * kStride) : -1;
                if (in && page[x] < 0)
                    kv4_bad(c);
            }
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                hi[x] = Words<D>{};
                lo[x] = Words<D>{};
                step[x] = -INFINITY; // a page that is none of the pool's is the last choice
                if (page[x] >= 0) {
                    const uint8_t *const at = tails + page[x] * c.page_bytes;
                    hi[x] = words_at<D>(at);
                    lo[x] = words_at<D>(at + Kv8Cell<D>::kLower);
                    step[x] = *(const float *)(at + Kv8Cell<D>::kStep - n * (D / 8));
                }
            }
        };
        ask(z0 + group);
        if (warp < nt)
            query_sums<D>(a, a.q + (int64_t)(s.first + t0 + warp) * a.q_stride + (int64_t)head * a.ratio * D, sq[warp % T][0],
                          sq[warp % T][1]);
        __syncthreads();
        uint32_t to = smem_addr(keys), to_range = smem_addr(ranges);
        if (a.cluster > 1) {
            to = cluster_map(to, 0);
            to_range = cluster_map(to_range, 0);
        }
        uint32_t least = ~0u, largest = 0;
#pragma unroll 1
        for (int z = z0 + group; z - group < z1; z += kAhead * kStride) {
            if (z != z0 + group)
                ask(z);
            int sum[kAhead][8];
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const Words<D> up = words_at<D>(&sq[t][0][n * (D / 8)]), down = words_at<D>(&sq[t][1][n * (D / 8)]);
#pragma unroll
                for (int x = 0; x < kAhead; ++x) {
                    sum[x][t] = 0;
#pragma unroll
                    for (int w = 0; w < D / 32; ++w)
                        sum[x][t] = __dp4a(up.w[w], hi[x].w[w], __dp4a(down.w[w], lo[x].w[w], sum[x][t]));
                }
            }
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                int mine = sum[x][0];
                if (T == 1) {
#pragma unroll
                    for (int o = 4; o; o >>= 1)
                        mine += __shfl_xor_sync(~0u, mine, o);
                } else {
                    mine = sum_across(sum[x], n);
                }
                const int zx = z + x * kStride;
                if (zx < z1 && n < T) {
                    const uint32_t key = key_of(step[x] == -INFINITY ? -INFINITY : (float)mine * step[x]);
                    st_cluster_f32(to + 4 * (n * width + zx), __uint_as_float(key));
                    least = min(least, key);
                    largest = max(largest, key);
                }
            }
        }
        // over the four groups of a warp (each lane of a group has a token's, or the first has all)
#pragma unroll
        for (int o = 8; o < 32; o <<= 1) {
            least = min(least, __shfl_xor_sync(~0u, least, o));
            largest = max(largest, __shfl_xor_sync(~0u, largest, o));
        }
        if (lane < T) {
            const uint32_t at = to_range + 8 * (T == 1 ? rank * kWarps + warp : warp * T + lane);
            st_cluster_f32(at, __uint_as_float(least));
            st_cluster_f32(at + 4, __uint_as_float(largest));
        }
    }
    if (a.cluster > 1) {
        cluster_sync();
        if (rank > 0)
            return;
    } else {
        __syncthreads();
    }
    const auto out_of = [&](int t) { return a.pages + ((int64_t)(s.first + t0 + t) * c.n_kv_heads + head) * a.want; };
    if (T == 1) {
        Group<W> g{bins, parts, found[0]};
        uint32_t least = ~0u, largest = 0;
        if (most > a.want) {
            for (int x = lane; x < a.cluster * kWarps; x += 32) {
                least = min(least, ranges[x][0]);
                largest = max(largest, ranges[x][1]);
            }
            range_of(least, largest);
        }
        choose(a, g, keys, most, least, largest, out_of(0));
    } else if (warp < nt) {
        Group<1> g{bins + warp % kGroups * Group<1>::kBins, nullptr, found[warp % kGroups]};
        uint32_t least = ~0u, largest = 0;
        if (most > a.want && lane < kWarps) {
            least = ranges[(lane % kWarps) * T + warp % T][0];
            largest = ranges[(lane % kWarps) * T + warp % T][1];
        }
        range_of(least, largest);
        choose(a, g, keys + warp * width, count_of(warp), least, largest, out_of(warp));
    }
}

template <int D, int T, int W>
nm_status launch(const Kv4 &c, const Kv4Batch &b, SelectArgs a, int cluster, const Kv4Work &w, cudaStream_t st)
{
    static OncePerDevice once;
    if (!once(w.device, [] {
            return cudaFuncSetAttribute(select_kernel<D, T, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        kKv8SelectPages * 4) == cudaSuccess;
        }))
        return NM_ERR_CUDA;
    const int64_t tiles = b.starts && b.n_seqs > 0 ? b.n_tokens / T + b.n_seqs : b.n_seqs;
    a.units = tiles * c.n_kv_heads;
    a.cluster = cluster;
    // no sequence is listed: one CTA answers the rows
    const int64_t grid = (a.units > 0 ? a.units : 1) * cluster;
    if (grid > 0x7FFFFFFF)
        return NM_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(T == 1 ? 32 * W : 32 * T);
    cfg.dynamicSmemBytes = (size_t)T * ((c.max_pages + 3) / 4 * 4) * 4;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, select_kernel<D, T, W>, c, b, a) == cudaSuccess ? NM_OK : NM_ERR_CUDA;
}

} // namespace

nm_status kv8_launch_select(const Kv4 &c, const Kv4Batch &b, const Kv8Select &x, const Kv4Work &w, cudaStream_t st)
{
    const SelectArgs a{x.layer, x.n_q_heads / c.n_kv_heads, x.count, x.first, x.last, (const uint16_t *)x.q, x.q_stride, x.pages, 0, 1};
    // Tiles of tokens when there are two tokens and kv heads to an SM, and their scores fit. A CTA each against tiles, us,
    // 8 kv heads: 20 tokens (256 pages) 9.8, 12.2; 4 x 5 tokens (up to 512) 14.7, 17.5; 40 tokens (256) 15.8, 12.1; 8 x 5 (32)
    // 15.1, 8.8. The scores of a tile stand in shared memory by the table's width, not the lengths: 512 tokens of 264 pages take
    // 27 us in tables of up to 3200, 43 from there (one CTA an SM) and 121 above 6141 pages, where there are no tiles; of 6000 pages
    // 522 in a table of 6141, 1112 in one of 6142.
    if (b.starts && b.n_tokens * c.n_kv_heads >= 2 * (int64_t)w.num_sms && (int64_t)kTile * (c.max_pages + 3) <= kKv8SelectPages)
        return c.head_dim == 128 ? launch<128, kTile, 1>(c, b, a, 1, w, st) : launch<64, kTile, 1>(c, b, a, 1, w, st);
    // The CTAs of a cluster share a token's pages while they are at most two to an SM and have 128 pages each. At most one to
    // an SM and at most two: 5 tokens of 1024 pages 14.1 us, 11.9; of 4096 pages 33.4, 25.1; 8 tokens of up to 1024 pages
    // with their attention 23.1, 20.6.
    int cluster = 1;
    while (cluster < 8 && cluster * b.n_tokens * c.n_kv_heads <= w.num_sms && c.max_pages >= 256 * cluster)
        cluster *= 2;
    return c.head_dim == 128 ? launch<128, 1, 8>(c, b, a, cluster, w, st) : launch<64, 1, 8>(c, b, a, cluster, w, st);
}

} // namespace nm
