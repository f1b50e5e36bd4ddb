// kv8.cuh -- the 8-bit paged KV cache: its layout on the device and what its
// kernels share. The format is described in nmspmv.h; tables, lengths and calls'
// tokens are those of the 4-bit cache (kv4.cuh).
#pragma once

#include "kv4.cuh"

namespace nm {

constexpr int kKv8MinExp = -24, kKv8MaxExp = 7; // of a block's scales: 448 * 2^7 holds kKv4Limit
constexpr int kKv8MinStep = -30;                // exponent of the bounds' step at least
constexpr int kKv8SelectPages = 49152;          // pages of a sequence that a selection takes at most

// Bytes of a cell: K [2][D / 64][8 tokens][64], V [D / 32][8][4][4 channels][4 tokens], the
// scales of K and V and eight bytes more; then of a kv head's bounds behind its cells.
template <int D> struct Kv8Cell {
    static constexpr int kV = kKv4Cell * D;
    static constexpr int kScales = 2 * kKv4Cell * D;
    static constexpr int kBytes = kScales + 16;
    static constexpr int kLower = D, kStep = 2 * D; // behind the upper bounds
    static constexpr int kTail = 2 * D + 16;
};

// One kv head's share of a page.
template <int D> __device__ __forceinline__ int64_t kv8_head_bytes(const Kv4 &c)
{
    return ((int64_t)Kv8Cell<D>::kBytes << (c.page_shift - 4)) + Kv8Cell<D>::kTail;
}
template <int D> __device__ __forceinline__ int64_t kv8_head_offset(const Kv4 &c, int page, int layer, int head)
{
    return (int64_t)page * c.page_bytes + ((int64_t)layer * c.n_kv_heads + head) * kv8_head_bytes<D>(c);
}

// Two codes as fp16, exactly (a NaN code as NaN).
__device__ __forceinline__ uint32_t kv8_decode(uint32_t two)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}

// A selection: count pages of each token and kv head, the first and last of them always.
struct Kv8Select {
    int layer, n_q_heads, count, first, last;
    const void *q;
    int64_t q_stride;
    int32_t *pages;
};

size_t kv8_partial_bytes(int head_dim);
size_t kv8_prompt_partial_bytes(int head_dim);

nm_status kv8_launch_append(const Kv4 &c, const Kv4Batch &b, int layer, const void *k, int64_t k_stride,
                            const void *v, int64_t v_stride, const void *q, int64_t q_stride, int n_q_heads,
                            void *q_out, int64_t q_out_stride, const float *rope, int64_t rope_rows, cudaStream_t st);
nm_status kv8_launch_read(const Kv4 &c, const Kv4Batch &b, int layer, void *k, void *v, bool f32, cudaStream_t st);
nm_status kv8_launch_prompt(const Kv4 &c, const Kv4Batch &b, const Kv4Attn &a, const Kv4Work &w, cudaStream_t st);
// pages: NULL, or the lists [n_tokens][n_kv_heads][n_list] of a selection
nm_status kv8_launch_attention(const Kv4 &c, const Kv4Batch &b, const Kv4Attn &a, int64_t max_new, const int32_t *pages,
                               int n_list, const Kv4Work &w, cudaStream_t st);
nm_status kv8_launch_select(const Kv4 &c, const Kv4Batch &b, const Kv8Select &a, const Kv4Work &w, cudaStream_t st);

} // namespace nm
