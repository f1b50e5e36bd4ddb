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

// q in 8-bit floats (for prompts). A row is scaled by a power of two that brings its largest magnitude into [2^7, 2^8), and
// a bf16 number (eight significant bits) is split into its first four (e4m3, nearest) and what is left: at most
// eight units of the last place, which e5m2 holds exactly. That is so down to 2^-6, 2^-13 of the row's
// largest at least. Below, the first part is a multiple of 2^-9 and what is left is rounded: by at most 2^-14,
// 2^-21 of the row's largest.
__device__ __forceinline__ uint32_t kv8_magnitude(const uint4 &x) // the largest of eight, as fp32 bits
{
    const uint32_t ws[4] = {x.x, x.y, x.z, x.w};
    uint32_t top = 0;
#pragma unroll
    for (int n = 0; n < 4; ++n)
        top = max(top, max(ws[n] & 0x7FFF0000u, (ws[n] << 16) & 0x7FFF0000u));
    return top;
}
struct Kv8Row {
    float down, factor; // of q, with the sign of the scale; of the scores, to the base 2
};
// sees: whether the row sees any token: something that is not finite then makes its result NaN.
__device__ __forceinline__ Kv8Row kv8_row(uint32_t top, float scale, bool sees)
{
    const uint32_t field = top >> 23;
    const uint32_t e = field == 0xFFu || field == 0 ? 127u : field < 8u ? 8u : field;
    const float up = __uint_as_float((e - 7u) << 23), down = __uint_as_float((261u - e) << 23);
    Kv8Row r;
    r.down = scale < 0.0f ? -down : down;
    // above 0, so that masked scores stay -inf; finite, K's scale of up to 2^7 with it, so that scores of 0 stay 0
    r.factor = field == 0xFFu && sees ? __uint_as_float(0x7FC00000u)
                                      : fminf(fmaxf(up * (fabsf(scale) * 1.4426950408889634f), 1e-30f), 0x1.fffffep120f);
    return r;
}
// Eight channels: two words of each part.
__device__ __forceinline__ void kv8_split(const uint4 &x, float down, uint2 &hi, uint2 &lo)
{
    const uint32_t ws[4] = {x.x, x.y, x.z, x.w};
    uint32_t h[4], l[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        uint32_t y, z;
        uint16_t p, r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(bf16hi_to_f32(ws[n]) * down), "f"(bf16lo_to_f32(ws[n]) * down));
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(p) : "r"(y));
        const uint32_t back = kv8_decode(p);
        const __half2 left = __hsub2(*(const __half2 *)&y, *(const __half2 *)&back);
        z = *(const uint32_t *)&left;
        asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(z));
        h[n] = p;
        l[n] = r;
    }
    hi = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    lo = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
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
