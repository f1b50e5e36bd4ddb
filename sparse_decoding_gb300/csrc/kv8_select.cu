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
// scores to the first one's shared memory. There the want-th largest is found two bits at a time
// (counts of three borders in a pass over the scores), and the pages above it, with the lowest of
// those equal to it, are written in order.
#include "kv8.cuh"

namespace nm {
namespace {

constexpr int kTile = 8;  // tokens of a tile of prompts
constexpr int kAhead = 4; // pages whose bounds a group of lanes asks for together

struct SelectArgs {
    int layer, ratio, want, first, last;
    const uint16_t *q;
    int64_t q_stride;
    int32_t *pages;
    int64_t units; // tiles (at most) times the kv heads
    int cluster;
};

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

// A group of W warps (the CTA, or one): sums of a thread's numbers over the group.
template <int W> struct Group {
    uint32_t (*part)[2][32]; // (W > 1) two buffers in shared memory, used in turn
    int turn = 0;
    __device__ int thread() const { return W == 1 ? threadIdx.x & 31 : threadIdx.x; }
    __device__ void sums(uint32_t &x, uint32_t &y)
    {
        x = __reduce_add_sync(~0u, x);
        y = __reduce_add_sync(~0u, y);
        if (W == 1)
            return;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0) {
            part[turn][0][warp] = x;
            part[turn][1][warp] = y;
        }
        __syncthreads();
        x = __reduce_add_sync(~0u, lane < W ? part[turn][0][lane] : 0u);
        y = __reduce_add_sync(~0u, lane < W ? part[turn][1][lane] : 0u);
        turn ^= 1;
    }
    // Sum over the threads before this one, and over all.
    __device__ uint32_t scan(uint32_t x, uint32_t *total)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        uint32_t y = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t z = __shfl_up_sync(~0u, y, o);
            if (lane >= o)
                y += z;
        }
        if (W == 1) {
            *total = __shfl_sync(~0u, y, 31);
            return y - x;
        }
        if (lane == 31)
            part[turn][0][warp] = y;
        __syncthreads();
        const uint32_t s = lane < W ? part[turn][0][lane] : 0u;
        *total = __reduce_add_sync(~0u, s);
        const uint32_t before = __reduce_add_sync(~0u, lane < warp ? s : 0u);
        turn ^= 1;
        return before + y - x;
    }
};

// The list of one query: the first and last pages, and of the others those with the largest keys.
template <int W> __device__ __forceinline__ void choose(const SelectArgs &a, Group<W> &g, const uint32_t *keys, int count, int32_t *out)
{
    const int me = g.thread();
    constexpr int kThreads = 32 * W;
    if (count <= a.want) {
        for (int j = me; j < a.want; j += kThreads)
            out[j] = j < count ? j : -1;
        return;
    }
    const int lo = a.first, hi = count - a.last; // the others: lo < hi, since first + last <= want < count
    const uint32_t need = (uint32_t)(a.want - a.first - a.last);
    // the largest border with at least `need` keys at or above it
    uint32_t border = need ? 0u : ~0u, above = 0; // above: keys over it
    if (need) {
#pragma unroll 1
        for (int bit = 30; bit >= 0; bit -= 2) {
            const uint32_t step = 1u << bit;
            uint32_t n12 = 0, n3 = 0; // counts of at most 2^16 - 1
            for (int z = lo + me; z < hi; z += kThreads) {
                const uint32_t k = keys[z];
                n12 += (k >= border + step ? 1u : 0u) + (k >= border + 2 * step ? 65536u : 0u);
                n3 += k >= border + 3 * step ? 1u : 0u;
            }
            g.sums(n12, n3);
            const uint32_t n1 = n12 & 0xFFFFu, n2 = n12 >> 16;
            if (n3 >= need)
                border += 3 * step;
            else if (n2 >= need)
                border += 2 * step, above = n3;
            else if (n1 >= need)
                border += step, above = n2;
            else
                above = n1;
        }
    }
    const uint32_t ties = need - above; // of the keys equal to the border, the lowest pages
    uint32_t done = 0;                  // above the border, and (times 65536) equal to it
    for (int z0 = 0; z0 < count; z0 += kThreads) {
        const int z = z0 + me;
        const bool forced = z < lo || (z >= hi && z < count), other = z >= lo && z < hi;
        const uint32_t k = other ? keys[z] : 0u;
        const bool over = forced || (other && need && k > border), tie = other && need && k == border;
        uint32_t total;
        const uint32_t before = done + g.scan((over ? 1u : 0u) + (tie ? 65536u : 0u), &total);
        const uint32_t n_over = before & 0xFFFFu, n_tie = before >> 16;
        if (over || (tie && n_tie < ties))
            out[n_over + (n_tie < ties ? n_tie : ties)] = z;
        done += total;
    }
}

// T tokens of a sequence and one kv head; W warps choose the pages of one token.
template <int D, int T, int W>
__global__ void __launch_bounds__(T == 1 ? 32 * W : 32 * T) select_kernel(const Kv4 c, const Kv4Batch b, const SelectArgs a)
{
    constexpr int kThreads = T == 1 ? 32 * W : 32 * T;
    extern __shared__ __align__(16) uint32_t keys[]; // [T][the table's width]
    __shared__ __align__(16) int8_t sq[T][2][D];
    __shared__ uint32_t parts[2][2][32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t unit = blockIdx.x / a.cluster;
    const int rank = (int)(blockIdx.x - unit * a.cluster);

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
    const int width = c.max_pages;

    if (most > a.want) {
        if (warp < nt)
            query_sums<D>(a, a.q + (int64_t)(s.first + t0 + warp) * a.q_stride + (int64_t)head * a.ratio * D, sq[warp % T][0],
                          sq[warp % T][1]);
        __syncthreads();
        const int n = lane & 7, group = tid >> 3;
        Words<D> up[T], down[T];
#pragma unroll
        for (int t = 0; t < T; ++t) {
            up[t] = words_at<D>(&sq[t][0][n * (D / 8)]);
            down[t] = words_at<D>(&sq[t][1][n * (D / 8)]);
        }
        // pages up to the last query's own (which needs no score) are full
        const int per = (most - 1 + a.cluster - 1) / a.cluster;
        const int z0 = rank * per, z1 = min(most - 1, z0 + per);
        const uint8_t *const tails = c.pool + kv8_head_offset<D>(c, 0, a.layer, head) + ((int64_t)Kv8Cell<D>::kBytes << (c.page_shift - 4));
        uint32_t to = smem_addr(keys);
        if (a.cluster > 1) {
            to = cluster_map(to, 0);
            cluster_sync(); // the first CTA's shared memory is there from here on
        }
#pragma unroll 1
        for (int z = z0 + group; z - group < z1; z += kAhead * (kThreads / 8)) {
            Words<D> hi[kAhead], lo[kAhead];
            float step[kAhead];
            const uint8_t *at[kAhead];
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                const int zx = z + x * (kThreads / 8);
                const int page = zx < z1 ? kv4_page(c, s.row, zx) : -1;
                at[x] = page < 0 ? nullptr : tails + page * c.page_bytes;
                if (zx < z1 && page < 0)
                    kv4_bad(c);
            }
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                hi[x] = Words<D>{};
                lo[x] = Words<D>{};
                step[x] = -INFINITY; // a page that is none of the pool's is the last choice
                if (at[x]) {
                    hi[x] = words_at<D>(at[x] + n * (D / 8));
                    lo[x] = words_at<D>(at[x] + Kv8Cell<D>::kLower + n * (D / 8));
                    step[x] = *(const float *)(at[x] + Kv8Cell<D>::kStep);
                }
            }
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                int sum[8];
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    sum[t] = 0;
#pragma unroll
                    for (int w = 0; w < D / 32; ++w)
                        sum[t] = __dp4a(up[t].w[w], hi[x].w[w], __dp4a(down[t].w[w], lo[x].w[w], sum[t]));
                }
                int mine = sum[0];
                if (T == 1) {
#pragma unroll
                    for (int o = 4; o; o >>= 1)
                        mine += __shfl_xor_sync(~0u, mine, o);
                } else {
                    mine = sum_across(sum, n);
                }
                const int zx = z + x * (kThreads / 8);
                if (zx < z1 && n < T) {
                    const uint32_t key = key_of(at[x] ? (float)mine * step[x] : -INFINITY);
                    st_cluster_f32(to + 4 * (n * width + zx), __uint_as_float(key));
                }
            }
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
        Group<W> g{parts};
        choose(a, g, keys, most, out_of(0));
    } else if (warp < nt) {
        Group<1> g{parts};
        choose(a, g, keys + warp * width, count_of(warp), out_of(warp));
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
    cfg.dynamicSmemBytes = (size_t)T * c.max_pages * 4;
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
    // tiles of tokens when there are several for each SM, and their scores fit
    if (b.starts && b.n_tokens * c.n_kv_heads >= 4 * (int64_t)w.num_sms && (int64_t)kTile * c.max_pages <= kKv8SelectPages)
        return c.head_dim == 128 ? launch<128, kTile, 1>(c, b, a, 1, w, st) : launch<64, kTile, 1>(c, b, a, 1, w, st);
    int cluster = 1;
    while (cluster < 8 && 2 * cluster * b.n_tokens * c.n_kv_heads <= w.num_sms && c.max_pages >= 256 * cluster)
        cluster *= 2;
    return c.head_dim == 128 ? launch<128, 1, 32>(c, b, a, cluster, w, st) : launch<64, 1, 32>(c, b, a, cluster, w, st);
}

} // namespace nm
