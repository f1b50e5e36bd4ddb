// kv4_pages.cu -- the bookkeeping of the paged cache: reserving, forking and
// freeing sequences' pages, compacting the pool, copying pages.
//
// The tables live in device memory and change there, so a decode loop that is a
// CUDA graph needs no host round trip. One CTA changes them (they are small: a
// call touches a few entries per sequence and scans the reference counts until it
// has the free pages it needs); a second kernel, over all SMs, moves what page
// contents have to move, from the list that the first one left.
//
// Measured (one GB300): moving 128 pages of 2.36 MB 87 us (604 MB, 6.9 TB/s, the measured
// copy rate); the table kernels take 5 to 8 us, which is the latency of their few
// dependent loads, and the seven copies of a beam step (14 MB, from L2) 8 us.
#include "kv4.cuh"

namespace nm {
namespace {

constexpr int kT = 1024;

// Exclusive prefix sum over the CTA of kT threads; *total gets the sum.
__device__ int block_scan(int x, int *warp_sums, int *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int y = x;
    for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(~0u, y, o);
        if (lane >= o)
            y += z;
    }
    __syncthreads(); // warp_sums may still be read from the last scan
    if (lane == 31)
        warp_sums[warp] = y;
    __syncthreads();
    int s = warp_sums[lane];
    for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(~0u, s, o);
        if (lane >= o)
            s += z;
    }
    *total = __shfl_sync(~0u, s, 31);
    const int before = __shfl_sync(~0u, s, warp > 0 ? warp - 1 : 0);
    return y - x + (warp > 0 ? before : 0);
}

// Four reference counts from page 4 i on; beyond the last page they read as used.
__device__ __forceinline__ int4 refs4(const Kv4 &c, int64_t i)
{
    if (4 * i + 3 < c.n_pages)
        return *(const int4 *)(c.refs + 4 * i);
    int4 r = make_int4(1, 1, 1, 1);
    int *p = (int *)&r;
    for (int k = 0; k < 4; ++k)
        if (4 * i + k < c.n_pages)
            p[k] = c.refs[4 * i + k];
    return r;
}

// The `want` lowest free pages, in order, to out; false when there are fewer.
__device__ bool find_free(const Kv4 &c, int want, int32_t *out, int *warp_sums)
{
    int have = 0;
    for (int64_t base = 0; have < want && 4 * base < c.n_pages; base += kT) {
        const int4 r = refs4(c, base + threadIdx.x);
        const int n = (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
        int total;
        int at = have + block_scan(n, warp_sums, &total);
        const int32_t page = (int32_t)(4 * (base + threadIdx.x));
        if (r.x == 0 && at++ < want)
            out[at - 1] = page;
        if (r.y == 0 && at++ < want)
            out[at - 1] = page + 1;
        if (r.z == 0 && at++ < want)
            out[at - 1] = page + 2;
        if (r.w == 0 && at++ < want)
            out[at - 1] = page + 3;
        have += total;
    }
    __syncthreads();
    return have >= want;
}

__device__ __forceinline__ int pages_of(const Kv4 &c, int64_t len) { return (int)((len + c.page_tokens - 1) >> c.page_shift); }
__device__ __forceinline__ bool len_ok(const Kv4 &c, int len) { return len >= 0 && len <= (int64_t)c.max_pages << c.page_shift; }

__global__ void __launch_bounds__(kT)
    reserve_kernel(const Kv4 c, const int32_t *seqs, const int32_t *starts, int n, int32_t *list)
{
    __shared__ int ids[kKv4MaxSeqs], off[kKv4MaxSeqs], warp_sums[32];
    const int i = threadIdx.x;
    int id = -1, len = 0, need = 0, old = 0;
    int64_t grown = 0;
    bool bad = false;
    if (i < n) {
        id = seqs ? seqs[i] : i;
        const int64_t n_new = starts ? (int64_t)starts[i + 1] - starts[i] : 1;
        bad = id < 0 || id >= c.max_seqs || n_new < 0;
        if (!bad) {
            len = c.lens[id];
            grown = len + n_new;
            bad = !len_ok(c, len) || grown > (int64_t)c.max_pages << c.page_shift;
            if (!bad) {
                old = pages_of(c, len);
                need = pages_of(c, grown) - old;
            }
        }
        ids[i] = id;
    }
    __syncthreads();
    for (int j = 0; j < i && i < n; ++j)
        bad |= ids[j] == id;
    if (__syncthreads_or(bad)) {
        if (i == 0)
            c.info[1] = -1;
        return;
    }
    int total;
    const int at = block_scan(need, warp_sums, &total);
    if (i < n)
        off[i] = at;
    const int free_pages = c.info[0];
    int32_t *pages = list + 64;
    if (total > free_pages || !find_free(c, total, pages, warp_sums)) {
        if (i == 0)
            c.info[1] = total > free_pages ? total - free_pages : total;
        return;
    }
    // page k goes to the last sequence whose first page number is at most k
    for (int k = i; k < total; k += kT) {
        int lo = 0, hi = n;
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if (off[m] <= k)
                lo = m;
            else
                hi = m;
        }
        const int s = ids[lo];
        c.tables[(int64_t)s * c.max_pages + pages_of(c, c.lens[s]) + (k - off[lo])] = pages[k];
        c.refs[pages[k]] = 1;
    }
    __syncthreads(); // the lengths above are read before they grow
    if (i < n)
        c.lens[id] = (int)grown;
    if (i == 0) {
        c.info[0] = free_pages - total;
        c.info[1] = 0;
    }
}

// list: [0] copies; [64 + k] their destination pages, [64 + n_pages + k] their
// sources, [64 + 2 n_pages + k] the cells to copy in each layer and head.
__global__ void __launch_bounds__(kT)
    fork_kernel(const Kv4 c, const int32_t *src, const int32_t *dst, int n, int32_t *list)
{
    __shared__ int from[kKv4MaxSeqs], to[kKv4MaxSeqs], warp_sums[32];
    const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
    int a = -1, d = -1, len = 0, need = 0;
    bool bad = false;
    if (i < n) {
        a = src[i];
        d = dst[i];
        bad = a < 0 || a >= c.max_seqs || d < 0 || d >= c.max_seqs;
        if (!bad) {
            len = c.lens[a];
            bad = !len_ok(c, len) || c.lens[d] != 0;
            need = (len & (c.page_tokens - 1)) != 0;
        }
        from[i] = a;
        to[i] = d;
    }
    if (i == 0)
        list[0] = 0;
    __syncthreads();
    for (int j = 0; j < n && i < n; ++j)
        bad |= d == from[j] || (j < i && d == to[j]);
    if (__syncthreads_or(bad)) {
        if (i == 0)
            c.info[1] = -1;
        return;
    }
    int total;
    const int at = block_scan(need, warp_sums, &total);
    const int free_pages = c.info[0];
    int32_t *pages = list + 64;
    if (total > free_pages || !find_free(c, total, pages, warp_sums)) {
        if (i == 0)
            c.info[1] = total > free_pages ? total - free_pages : total;
        return;
    }
    for (int j = warp; j < n; j += kT / 32) { // the full pages, shared
        const int full = c.lens[from[j]] >> c.page_shift;
        const int32_t *f = c.tables + (int64_t)from[j] * c.max_pages;
        int32_t *t = c.tables + (int64_t)to[j] * c.max_pages;
        for (int k = lane; k < full; k += 32) {
            const int32_t p = f[k];
            t[k] = p;
            if (p >= 0 && p < c.n_pages)
                atomicAdd(c.refs + p, 1);
            else
                kv4_bad(c);
        }
    }
    if (need) {
        const int full = len >> c.page_shift;
        const int32_t p = c.tables[(int64_t)a * c.max_pages + full];
        const bool ok = p >= 0 && p < c.n_pages;
        if (!ok)
            kv4_bad(c);
        c.tables[(int64_t)d * c.max_pages + full] = pages[at];
        c.refs[pages[at]] = 1;
        list[64 + c.n_pages + at] = p;
        list[64 + 2 * c.n_pages + at] = ok ? ((len & (c.page_tokens - 1)) + kKv4Cell - 1) / kKv4Cell : 0;
    }
    if (i < n)
        c.lens[d] = len;
    if (i == 0) {
        list[0] = total;
        c.info[0] = free_pages - total;
        c.info[1] = 0;
    }
}

__global__ void __launch_bounds__(kT) free_kernel(const Kv4 c, const int32_t *seqs, int n)
{
    __shared__ int ids[kKv4MaxSeqs];
    __shared__ int freed;
    const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
    if (i == 0)
        freed = 0;
    if (i < n) {
        const int id = seqs ? seqs[i] : i;
        const bool ok = id >= 0 && id < c.max_seqs && len_ok(c, c.lens[id]);
        if (!ok)
            kv4_bad(c);
        ids[i] = ok ? id : -1;
    }
    __syncthreads();
    bool again = false;
    for (int j = 0; j < i && i < n; ++j)
        again |= ids[j] == ids[i];
    __syncthreads();
    if (i < n && again)
        ids[i] = -1;
    __syncthreads();
    for (int j = warp; j < n; j += kT / 32) {
        if (ids[j] < 0)
            continue;
        int32_t *t = c.tables + (int64_t)ids[j] * c.max_pages;
        const int np = pages_of(c, c.lens[ids[j]]);
        int mine = 0;
        for (int k = lane; k < np; k += 32) {
            const int32_t p = t[k];
            t[k] = -1;
            if (p < 0 || p >= c.n_pages)
                kv4_bad(c);
            else
                mine += atomicSub(c.refs + p, 1) == 1;
        }
        mine = __reduce_add_sync(~0u, mine);
        if (lane == 0) {
            c.lens[ids[j]] = 0;
            if (mine)
                atomicAdd(&freed, mine);
        }
    }
    __syncthreads();
    if (i == 0)
        c.info[0] += freed;
}

// list: [0] moves, [1] pages in use; [64 + k] the free pages below that count
// (destinations), [64 + n_pages + k] the used pages from it on, both ascending.
__global__ void __launch_bounds__(kT) compact_kernel(const Kv4 c, int32_t *list)
{
    __shared__ int warp_sums[32];
    const int64_t quads = (c.n_pages + 3) / 4;
    int used = 0;
    for (int64_t q = threadIdx.x; q < quads; q += kT) {
        const int4 r = refs4(c, q);
        used += (r.x != 0) + (r.y != 0) + (r.z != 0) + (r.w != 0);
    }
    int total;
    block_scan(used, warp_sums, &total);
    const int live = total - (int)(4 * quads - c.n_pages); // pages beyond the last read as used
    int32_t *holes = list + 64, *movers = list + 64 + c.n_pages;
    int nh = 0, nm = 0;
    for (int64_t base = 0; base < quads; base += kT) {
        const int64_t q = base + threadIdx.x;
        int4 r = make_int4(1, 1, 1, 1);
        if (q < quads)
            r = refs4(c, q);
        const int *p = (const int *)&r;
        int h = 0, m = 0;
        for (int k = 0; k < 4; ++k) {
            const int64_t page = 4 * q + k;
            h += page < live && p[k] == 0;
            m += page >= live && page < c.n_pages && p[k] != 0;
        }
        int th, tm;
        int ah = nh + block_scan(h, warp_sums, &th), am = nm + block_scan(m, warp_sums, &tm);
        for (int k = 0; k < 4; ++k) {
            const int64_t page = 4 * q + k;
            if (page < live && p[k] == 0)
                holes[ah++] = (int32_t)page;
            if (page >= live && page < c.n_pages && p[k] != 0)
                movers[am++] = (int32_t)page;
        }
        nh += th;
        nm += tm;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < nh; k += kT) { // nh == nm
        c.refs[holes[k]] = c.refs[movers[k]];
        c.refs[movers[k]] = 0;
    }
    if (threadIdx.x == 0) {
        list[0] = nh;
        list[1] = live;
        c.info[0] = (int)(c.n_pages - live);
        c.info[2] = nh;
    }
}

// n bytes (a multiple of 16) by the CTA's threads, four loads in flight.
__device__ __forceinline__ void copy_bytes(uint8_t *dst, const uint8_t *src, int64_t n)
{
    const int64_t v = n / 16;
    const uint4 *s = (const uint4 *)src;
    uint4 *d = (uint4 *)dst;
    int64_t i = threadIdx.x;
    for (; i + 3 * (int64_t)blockDim.x < v; i += 4 * (int64_t)blockDim.x) {
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            x[k] = __ldcs(s + i + k * blockDim.x);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            __stcs(d + i + k * blockDim.x, x[k]);
    }
    for (; i < v; i += blockDim.x)
        d[i] = s[i];
}

constexpr int64_t kChunk = 32768; // bytes of a page that a CTA copies at a time

// The copies of a fork: the first cells of every layer and head of a page.
__global__ void __launch_bounds__(256) fork_copy_kernel(const Kv4 c, const int32_t *list, int cell_bytes)
{
    const int heads = c.n_layers * c.n_kv_heads;
    const int64_t head_bytes = c.page_bytes / heads;
    const int64_t items = (int64_t)list[0] * heads;
    for (int64_t x = blockIdx.x; x < items; x += gridDim.x) {
        const int k = (int)(x / heads), h = (int)(x % heads);
        const int64_t d = list[64 + k], s = list[64 + c.n_pages + k];
        const int cells = list[64 + 2 * c.n_pages + k];
        copy_bytes(c.pool + d * c.page_bytes + h * head_bytes, c.pool + s * c.page_bytes + h * head_bytes,
                   (int64_t)cells * cell_bytes);
    }
}

// The moves of a compaction, and the tables that name the moved pages.
__global__ void __launch_bounds__(256) compact_move_kernel(const Kv4 c, const int32_t *list)
{
    const int moves = list[0], live = list[1];
    if (moves == 0)
        return;
    const int32_t *holes = list + 64, *movers = list + 64 + c.n_pages;
    const int64_t entries = (int64_t)c.max_seqs * c.max_pages;
    for (int64_t x = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; x < entries; x += (int64_t)gridDim.x * blockDim.x) {
        const int32_t p = c.tables[x];
        if (p < live)
            continue;
        int lo = 0, hi = moves; // movers[lo] <= p < movers[hi]
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if (movers[m] <= p)
                lo = m;
            else
                hi = m;
        }
        if (movers[lo] == p)
            c.tables[x] = holes[lo];
    }
    const int64_t chunks = (c.page_bytes + kChunk - 1) / kChunk;
    for (int64_t x = blockIdx.x; x < moves * chunks; x += gridDim.x) {
        const int64_t k = x / chunks, at = (x % chunks) * kChunk;
        const int64_t n = c.page_bytes - at < kChunk ? c.page_bytes - at : kChunk;
        copy_bytes(c.pool + (int64_t)holes[k] * c.page_bytes + at, c.pool + (int64_t)movers[k] * c.page_bytes + at, n);
    }
}

__global__ void __launch_bounds__(256)
    copy_pages_kernel(const uint8_t *src, int64_t src_n, const int32_t *src_pages, uint8_t *dst, int64_t dst_n,
                      const int32_t *dst_pages, int64_t page_bytes, int64_t n, uint32_t *status)
{
    const int64_t chunks = (page_bytes + kChunk - 1) / kChunk;
    for (int64_t x = blockIdx.x; x < n * chunks; x += gridDim.x) {
        const int64_t k = x / chunks, at = (x % chunks) * kChunk;
        const int64_t s = src_pages[k], d = dst_pages[k];
        if (s < 0 || s >= src_n || d < 0 || d >= dst_n) {
            if (threadIdx.x == 0)
                atomicOr(status, 1u << NM_ERR_BOUNDS);
            continue;
        }
        const int64_t m = page_bytes - at < kChunk ? page_bytes - at : kChunk;
        copy_bytes(dst + d * page_bytes + at, src + s * page_bytes + at, m);
    }
}

nm_status done() { return cudaGetLastError() == cudaSuccess ? NM_OK : NM_ERR_CUDA; }

} // namespace

nm_status kv4_launch_reserve(const Kv4 &c, const int32_t *seqs, const int32_t *starts, int n, const Kv4Work &w,
                             cudaStream_t st)
{
    reserve_kernel<<<1, kT, 0, st>>>(c, seqs, starts, n, w.list);
    return done();
}

nm_status kv4_launch_fork(const Kv4 &c, const int32_t *src, const int32_t *dst, int n, const Kv4Work &w, int num_sms,
                          cudaStream_t st)
{
    fork_kernel<<<1, kT, 0, st>>>(c, src, dst, n, w.list);
    fork_copy_kernel<<<num_sms * 8, 256, 0, st>>>(c, w.list, 16 * c.head_dim + c.head_dim * 2);
    return done();
}

nm_status kv4_launch_free(const Kv4 &c, const int32_t *seqs, int n, cudaStream_t st)
{
    free_kernel<<<1, kT, 0, st>>>(c, seqs, n);
    return done();
}

nm_status kv4_launch_compact(const Kv4 &c, const Kv4Work &w, int num_sms, cudaStream_t st)
{
    compact_kernel<<<1, kT, 0, st>>>(c, w.list);
    compact_move_kernel<<<num_sms * 8, 256, 0, st>>>(c, w.list);
    return done();
}

nm_status kv4_launch_copy(const uint8_t *src, int64_t src_n, const int32_t *src_pages, uint8_t *dst, int64_t dst_n,
                          const int32_t *dst_pages, int64_t page_bytes, int64_t n, uint32_t *status, int num_sms,
                          cudaStream_t st)
{
    copy_pages_kernel<<<num_sms * 8, 256, 0, st>>>(src, src_n, src_pages, dst, dst_n, dst_pages, page_bytes, n, status);
    return done();
}

} // namespace nm
