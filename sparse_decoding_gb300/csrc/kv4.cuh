// kv4.cuh -- the 4-bit paged KV cache: its layout on the device and what its
// kernels share. The format is described in nmspmv.h.
#pragma once

#include <cuda_fp16.h>

#include "kernels.h"
#include "nm_common.cuh"
#include "per_device.h"

namespace nm {

constexpr int kKv4Cell = 16;       // tokens of a cell
constexpr int kKv4Group = 64;      // channels that share a scale
constexpr int kKv4MaxSeqs = 1024;  // sequences of one call
constexpr float kKv4Limit = 32768.0f;

// Bytes of the parts of a cell.
template <int D> struct Kv4Cell {
    static constexpr int G = D / kKv4Group;
    static constexpr int kCodes = kKv4Cell * D / 2;     // of K, and of V
    static constexpr int kParams = kKv4Cell * G * 4;    // of K, and of V
    static constexpr int kV = kCodes;
    static constexpr int kKp = 2 * kCodes;
    static constexpr int kVp = 2 * kCodes + kParams;
    static constexpr int kBytes = 2 * (kCodes + kParams);
};

// A cache as the kernels see it.
struct Kv4 {
    uint8_t *pool;
    int64_t n_pages;
    int64_t page_bytes;
    int page_tokens, page_shift; // page_tokens = 1 << page_shift
    int n_layers, n_kv_heads, head_dim;
    int max_seqs, max_pages;
    int32_t *info, *lens, *refs, *tables;
    uint32_t *status;            // the library's status word
};

// The new tokens of one call.
struct Kv4Batch {
    const int32_t *seqs;   // NULL: the identity
    const int32_t *starts; // NULL: one token each
    int n_seqs;
    int64_t n_tokens;
};

__device__ __forceinline__ void kv4_bad(const Kv4 &c) { atomicOr(c.status, 1u << NM_ERR_BOUNDS); }

// One listed sequence: its row of the tables, its length, and its new tokens
// [first, first + n_new) of the token arrays. Anything out of range is reported
// and leaves it without tokens: len 0, but its rows, where starts names rows of
// the arrays, are still there to be answered with zeros; where it does not, n_new
// is 0 and first -1.
struct Kv4Seq {
    int row, len, first, n_new;
};

__device__ __forceinline__ Kv4Seq kv4_seq(const Kv4 &c, const Kv4Batch &b, int i, bool report)
{
    Kv4Seq s;
    int64_t a = i, e = i + 1;
    if (b.starts) {
        a = b.starts[i];
        e = b.starts[i + 1];
    }
    bool ok = a >= 0 && e >= a && e <= b.n_tokens;
    s.first = ok ? (int)a : -1;
    s.n_new = ok ? (int)(e - a) : 0;
    s.row = b.seqs ? b.seqs[i] : i;
    s.len = 0;
    if (s.row >= 0 && s.row < c.max_seqs) {
        s.len = c.lens[s.row];
        if (s.len < 0 || s.len > (int64_t)c.max_pages << c.page_shift) {
            s.len = 0;
            ok = false;
        }
    } else {
        s.row = 0;
        ok = false;
    }
    if (!ok && report)
        kv4_bad(c);
    return s;
}

// The listed sequence that token i belongs to, -1 for none (starts that do not
// cover it). starts is nondecreasing; any values end the search.
__device__ __forceinline__ int kv4_find(const Kv4Batch &b, int64_t i)
{
    if (!b.starts || b.n_seqs == 0)
        return i < b.n_seqs ? (int)i : -1;
    int lo = 0, hi = b.n_seqs; // starts[lo] <= i < starts[hi], if it is covered at all
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (b.starts[m] <= i)
            lo = m;
        else
            hi = m;
    }
    return (i >= b.starts[lo] && i < b.starts[lo + 1]) ? lo : -1;
}

// Rows of the token arrays that no sequence covers: before starts[0], past the last end (padding), or
// left by starts that are out of range. There are none when the starts rise from 0 to the number of
// tokens, that is when all sequences are in range (no first is -1) and kv4_ends holds.
__device__ __forceinline__ bool kv4_ends(const Kv4Batch &b)
{
    return !b.starts || (b.starts[0] == 0 && b.starts[b.n_seqs] == b.n_tokens);
}
// f(row) for those rows, a warp to each.
template <class F>
__device__ __forceinline__ void kv4_uncovered(const Kv4Batch &b, int64_t warp, int64_t warps, const F &f)
{
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int64_t row = warp; row < b.n_tokens; row += warps) {
        bool covered = false;
#pragma unroll 1
        for (int i = lane; i < b.n_seqs; i += 32) {
            const int64_t a = b.starts[i], e = b.starts[i + 1];
            covered |= a >= 0 && a <= row && row < e && e <= b.n_tokens;
        }
        if (!__any_sync(~0u, covered))
            f(row);
    }
}
// What attention answers there: width channels of out 0, lse -inf.
__device__ __forceinline__ void kv4_answer_uncovered(const Kv4Batch &b, uint16_t *out, int64_t out_stride, int width,
                                                     float *lse, int n_q_heads, int64_t warp, int64_t warps)
{
    kv4_uncovered(b, warp, warps, [&](int64_t row) {
        for (int i = threadIdx.x & 31; i < width / 8; i += 32)
            *(uint4 *)(out + row * out_stride + 8 * i) = make_uint4(0, 0, 0, 0);
        for (int h = threadIdx.x & 31; lse && h < n_q_heads; h += 32)
            lse[row * n_q_heads + h] = -INFINITY;
    });
}

// The cell that holds position `pos` of table row `row`, for one layer and kv
// head; NULL (reported) when the table names no page of the pool there.
__device__ __forceinline__ int kv4_page(const Kv4 &c, int row, int index)
{
    const int32_t p = c.tables[(int64_t)row * c.max_pages + index];
    return (p >= 0 && p < c.n_pages) ? p : -1;
}
template <int D>
__device__ __forceinline__ int64_t kv4_cell_offset(const Kv4 &c, int page, int layer, int head, int cell)
{
    return (int64_t)page * c.page_bytes +
           ((((int64_t)layer * c.n_kv_heads + head) << (c.page_shift - 4)) + cell) * Kv4Cell<D>::kBytes;
}

// A bounded wait (about a second, then NM_ERR_TIMEOUT; `dead` threads poll once). The
// clock is read only after some polls: reading it takes longer than most waits.
template <class F> __device__ __forceinline__ void kv4_until(const F &there, uint32_t *status, bool &dead)
{
    uint64_t t0 = 0;
    uint32_t polls = 0;
#pragma unroll 1
    while (!there()) {
        if (dead)
            return;
        if (++polls < 64)
            continue;
        const uint64_t t = globaltimer_ns();
        if (t0 == 0)
            t0 = t;
        if (t - t0 > kWaitLimitNs) {
            atomicOr(status, 1u << NM_ERR_TIMEOUT);
            dead = true;
            return;
        }
    }
}
__device__ __forceinline__ void kv4_wait(uint32_t bar, uint32_t parity, uint32_t *status, bool &dead)
{
    kv4_until([&]() { return mbar_try_wait(bar, parity); }, status, dead);
}

__device__ __forceinline__ void kv4_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Arrives and waits for the others of the barrier's count: a __syncthreads() of some threads that is
// bounded as above.
__device__ __forceinline__ void kv4_meet(uint32_t bar, uint32_t *status, bool &dead)
{
    uint64_t phase;
    asm volatile("mbarrier.arrive.shared::cta.b64 %0, [%1];" : "=l"(phase) : "r"(bar) : "memory");
    kv4_until([&]() {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(bar), "l"(phase)
                     : "memory");
        return ok != 0;
    }, status, dead);
}

// 16 bytes of read-only data
__device__ __forceinline__ uint4 ldg_nc128(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// ---- internal launch interface ------------------------------------------------

constexpr size_t kKv4Counters = 2048;  // join counters at the workspace's start

struct Kv4Work {
    uint32_t *counters;  // [kKv4Counters], zero between launches
    int32_t *list;       // [64 + 2 n_pages]: page lists of the table calls
    float *partials;     // attention parts
    int device, num_sms;
};
size_t kv4_partial_bytes(int head_dim);

nm_status kv4_launch_append(const Kv4 &c, const Kv4Batch &b, int layer, const void *k, int64_t k_stride,
                            const void *v, int64_t v_stride, const void *q, int64_t q_stride, int n_q_heads,
                            void *q_out, int64_t q_out_stride, const float *rope, int64_t rope_rows, cudaStream_t st);
nm_status kv4_launch_read(const Kv4 &c, const Kv4Batch &b, int layer, void *k, void *v, bool f32, cudaStream_t st);

struct Kv4Attn {
    int layer;
    const void *q;
    int64_t q_stride;
    int n_q_heads;
    float scale;
    void *out;
    int64_t out_stride;
    float *lse;
};
constexpr int kKv4PromptCtas = 160; // CTAs of the prompt kernel at most
size_t kv4_prompt_partial_bytes(int head_dim);
nm_status kv4_launch_prompt(const Kv4 &c, const Kv4Batch &b, const Kv4Attn &a, const Kv4Work &w, cudaStream_t st);
nm_status kv4_launch_attention(const Kv4 &c, const Kv4Batch &b, const Kv4Attn &a, int64_t max_new, const Kv4Work &w,
                               cudaStream_t st);

nm_status kv4_launch_reserve(const Kv4 &c, const int32_t *seqs, const int32_t *starts, int n, const Kv4Work &w,
                             cudaStream_t st);
nm_status kv4_launch_fork(const Kv4 &c, const int32_t *src, const int32_t *dst, int n, const Kv4Work &w, int num_sms,
                          cudaStream_t st);
nm_status kv4_launch_free(const Kv4 &c, const int32_t *seqs, int n, cudaStream_t st);
nm_status kv4_launch_compact(const Kv4 &c, const Kv4Work &w, int num_sms, cudaStream_t st);
nm_status kv4_launch_copy(const uint8_t *src, int64_t src_pages_n, const int32_t *src_pages, uint8_t *dst,
                          int64_t dst_pages_n, const int32_t *dst_pages, int64_t page_bytes, int64_t n,
                          uint32_t *status, int num_sms, cudaStream_t st);

} // namespace nm
