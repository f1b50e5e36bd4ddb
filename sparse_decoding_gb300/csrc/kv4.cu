// kv4.cu -- writing tokens to the 4-bit paged KV cache (with the rotary
// positions of q and k) and reading the values it holds back.
#include "kv4.cuh"

namespace nm {
namespace {

// Channels of a lane, where a warp holds one head's vector: 2 l, 2 l + 1 and
// D/2 + 2 l, + 1 (the two halves that a rotation turns together), l < D / 4.
template <int D> struct Lane4 {
    float v[4];
};
template <int D> __device__ __forceinline__ int lane_channel(int lane, int half) { return half * (D / 2) + 2 * lane; }

template <int D> __device__ __forceinline__ Lane4<D> load_vec(const uint16_t *p, int lane)
{
    Lane4<D> r;
    const uint32_t a = *(const uint32_t *)(p + lane_channel<D>(lane, 0));
    const uint32_t b = *(const uint32_t *)(p + lane_channel<D>(lane, 1));
    r.v[0] = bf16lo_to_f32(a);
    r.v[1] = bf16hi_to_f32(a);
    r.v[2] = bf16lo_to_f32(b);
    r.v[3] = bf16hi_to_f32(b);
    return r;
}

// (a cos - b sin, b cos + a sin), each operation rounded.
template <int D> __device__ __forceinline__ void rotate(Lane4<D> &x, const float *row, int lane)
{
    const float2 c = *(const float2 *)(row + 2 * lane), s = *(const float2 *)(row + D / 2 + 2 * lane);
    const float a0 = x.v[0], a1 = x.v[1], b0 = x.v[2], b1 = x.v[3];
    x.v[0] = __fsub_rn(__fmul_rn(a0, c.x), __fmul_rn(b0, s.x));
    x.v[1] = __fsub_rn(__fmul_rn(a1, c.y), __fmul_rn(b1, s.y));
    x.v[2] = __fadd_rn(__fmul_rn(b0, c.x), __fmul_rn(a0, s.x));
    x.v[3] = __fadd_rn(__fmul_rn(b1, c.y), __fmul_rn(a1, s.y));
}

__device__ __forceinline__ bool finite_f32(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }
__device__ __forceinline__ float saturate(float x)
{
    return x != x ? 0.0f : fminf(fmaxf(x, -kKv4Limit), kKv4Limit);
}

// Scale and middle of a group with least and greatest value lo and hi, as the
// cache holds them, and the code of one value.
__device__ __forceinline__ void group_params(float lo, float hi, __half &s, __half &mid)
{
    const uint16_t sb = f32_to_bf16_rn(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f));
    s = __float2half_rn(bf16_to_f32(sb));
    mid = __float2half_rn(__fadd_rn(lo, __fmul_rn(__half2float(s), 8.0f)));
}
__device__ __forceinline__ uint32_t code_of(float x, float s, float mid)
{
    const float u = s > 0.0f ? rintf(__fdiv_rn(__fsub_rn(x, mid), s)) : 0.0f;
    return (uint32_t)(int)(fminf(fmaxf(u, -8.0f), 7.0f) + 8.0f);
}

__device__ __forceinline__ float warp_min(float x)
{
    for (int o = 16; o; o >>= 1)
        x = fminf(x, __shfl_xor_sync(~0u, x, o));
    return x;
}
__device__ __forceinline__ float warp_max(float x)
{
    for (int o = 16; o; o >>= 1)
        x = fmaxf(x, __shfl_xor_sync(~0u, x, o));
    return x;
}

// The byte in a cell that holds the codes of channels ch, ch + 1 (ch even) of
// token `slot`: of K, and of V.
template <int D> __device__ __forceinline__ int k_byte(int slot, int ch)
{
    constexpr int G = Kv4Cell<D>::G;
    const int g = ch / kKv4Group, x = ch % kKv4Group;
    return slot * (D / 2) + (x / 16) * (8 * G) + g * 8 + (x % 16) / 2;
}
template <int D> __device__ __forceinline__ int v_byte(int slot, int ch)
{
    const int g = ch / kKv4Group, x = ch % kKv4Group;
    return Kv4Cell<D>::kV + g * 512 + ((x / 8) * 4 + (slot / 2) % 4) * 16 + (slot / 8) * 8 + ((x / 4) % 2) * 4 +
           (slot % 2) * 2 + (x % 4) / 2;
}

struct AppendArgs {
    int layer, n_q_heads;
    const uint16_t *k, *v, *q;
    uint16_t *q_out;
    int64_t k_stride, v_stride, q_stride, q_out_stride;
    const float *rope;
    int64_t rope_rows;
};

// One warp per (token, head): the kv heads are rotated, quantised and written,
// the q heads rotated.
template <int D> __global__ void __launch_bounds__(256) append_kernel(const Kv4 c, const Kv4Batch b, const AppendArgs a)
{
    constexpr int G = Kv4Cell<D>::G;
    const int lane = threadIdx.x & 31;
    const int jobs = c.n_kv_heads + (a.q ? a.n_q_heads : 0);
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t token = w / jobs;
    const int job = (int)(w % jobs);
    if (token >= b.n_tokens)
        return;
    const int i = kv4_find(b, token);
    Kv4Seq s{};
    int pos = -1;
    if (i >= 0) {
        s = kv4_seq(c, b, i, lane == 0);
        pos = s.len - s.n_new + (int)(token - s.first);
    }
    bool ok = pos >= 0 && pos < s.len && (!a.rope || pos < a.rope_rows);
    const bool mine = lane < D / 4;
    const float *row = a.rope && ok ? a.rope + (int64_t)pos * D : nullptr;

    if (job >= c.n_kv_heads) { // a q head
        const int h = job - c.n_kv_heads;
        if (!mine)
            return;
        Lane4<D> x = load_vec<D>(a.q + token * a.q_stride + (int64_t)h * D, lane);
        if (row)
            rotate<D>(x, row, lane);
        uint16_t *o = a.q_out + token * a.q_out_stride + (int64_t)h * D;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t p = f32_to_bf16_rn(x.v[2 * e]) | ((uint32_t)f32_to_bf16_rn(x.v[2 * e + 1]) << 16);
            *(uint32_t *)(o + lane_channel<D>(lane, e)) = ok ? p : 0u;
        }
        return;
    }
    const int page = ok ? kv4_page(c, s.row, pos >> c.page_shift) : -1;
    if (page < 0) {
        if (lane == 0)
            kv4_bad(c);
        return;
    }
    const int slot = pos % kKv4Cell, cell = (pos & (c.page_tokens - 1)) / kKv4Cell;
    uint8_t *dst = c.pool + kv4_cell_offset<D>(c, page, a.layer, job, cell);
    Lane4<D> kx{}, vx{};
    if (mine) {
        kx = load_vec<D>(a.k + token * a.k_stride + (int64_t)job * D, lane);
        vx = load_vec<D>(a.v + token * a.v_stride + (int64_t)job * D, lane);
        if (row)
            rotate<D>(kx, row, lane);
    }
    bool fine = true;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        fine = fine && finite_f32(kx.v[e]) && finite_f32(vx.v[e]);
    fine = __all_sync(~0u, fine);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        Lane4<D> &x = kv ? vx : kx;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            x.v[e] = saturate(x.v[e]);
        __half sc[2], md[2];
        float lo[2], hi[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) { // the lane's two halves
            lo[e] = mine ? fminf(x.v[2 * e], x.v[2 * e + 1]) : INFINITY;
            hi[e] = mine ? fmaxf(x.v[2 * e], x.v[2 * e + 1]) : -INFINITY;
        }
        if (G == 1) {
            lo[0] = lo[1] = fminf(lo[0], lo[1]);
            hi[0] = hi[1] = fmaxf(hi[0], hi[1]);
        }
#pragma unroll
        for (int e = 0; e < G; ++e) {
            lo[e] = warp_min(lo[e]);
            hi[e] = warp_max(hi[e]);
            group_params(lo[e], hi[e], sc[e], md[e]);
        }
        if (G == 1) {
            sc[1] = sc[0];
            md[1] = md[0];
        }
        if (mine) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float fs = __half2float(sc[e]), fm = __half2float(md[e]);
                uint32_t byte = code_of(x.v[2 * e], fs, fm) | (code_of(x.v[2 * e + 1], fs, fm) << 4);
                const int ch = lane_channel<D>(lane, e);
                if (!kv && !fine)
                    byte = 0x88;
                dst[kv ? v_byte<D>(slot, ch) : k_byte<D>(slot, ch)] = (uint8_t)byte;
            }
        }
        if (lane < G) {
            const __half ss = lane ? sc[G - 1] : sc[0], mm = lane ? md[G - 1] : md[0];
            if (!kv) {
                const __half nan = __ushort_as_half(0x7E00);
                *(__half2 *)(dst + Kv4Cell<D>::kKp + (slot * G + lane) * 4) =
                    fine ? __halves2half2(ss, mm) : __halves2half2(nan, nan);
            } else {
                __half *p = (__half *)(dst + Kv4Cell<D>::kVp + ((slot / 2) * G + lane) * 8 + (slot % 2) * 2);
                p[0] = ss;
                p[2] = mm;
            }
        }
    }
}

// One warp per (token, kv head).
template <int D, bool F32>
__global__ void __launch_bounds__(256) read_kernel(const Kv4 c, const Kv4Batch b, int layer, void *k, void *v)
{
    constexpr int G = Kv4Cell<D>::G;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t token = w / c.n_kv_heads;
    const int head = (int)(w % c.n_kv_heads);
    if (token >= b.n_tokens)
        return;
    const int i = kv4_find(b, token);
    Kv4Seq s{};
    int pos = -1;
    if (i >= 0) {
        s = kv4_seq(c, b, i, lane == 0);
        pos = s.len - s.n_new + (int)(token - s.first);
    }
    const int page = pos >= 0 && pos < s.len ? kv4_page(c, s.row, pos >> c.page_shift) : -1;
    if (page < 0 && lane == 0)
        kv4_bad(c);
    if (lane >= D / 4)
        return;
    const int slot = pos % kKv4Cell, cell = (pos & (c.page_tokens - 1)) / kKv4Cell;
    const uint8_t *src = page < 0 ? nullptr : c.pool + kv4_cell_offset<D>(c, page, layer, head, cell);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        void *out = kv ? v : k;
        if (!out)
            continue;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int ch = lane_channel<D>(lane, e), g = ch / kKv4Group;
            float x0 = 0.0f, x1 = 0.0f;
            if (src) {
                float sc, md;
                if (!kv) {
                    const __half2 p = *(const __half2 *)(src + Kv4Cell<D>::kKp + (slot * G + g) * 4);
                    sc = __low2float(p);
                    md = __high2float(p);
                } else {
                    const __half *p = (const __half *)(src + Kv4Cell<D>::kVp + ((slot / 2) * G + g) * 8 + (slot % 2) * 2);
                    sc = __half2float(p[0]);
                    md = __half2float(p[2]);
                }
                const uint32_t by = src[kv ? v_byte<D>(slot, ch) : k_byte<D>(slot, ch)];
                x0 = __fadd_rn(__fmul_rn((float)(int)(by & 15u) - 8.0f, sc), md);
                x1 = __fadd_rn(__fmul_rn((float)(int)(by >> 4) - 8.0f, sc), md);
            }
            const int64_t at = (token * c.n_kv_heads + head) * D + ch;
            if (F32)
                *(float2 *)((float *)out + at) = make_float2(x0, x1);
            else
                *(uint32_t *)((uint16_t *)out + at) = f32_to_bf16_rn(x0) | ((uint32_t)f32_to_bf16_rn(x1) << 16);
        }
    }
}

nm_status grid_of(int64_t warps, unsigned *grid)
{
    const int64_t g = (warps + 7) / 8;
    if (g > 0x7FFFFFFF)
        return NM_ERR_SHAPE;
    *grid = (unsigned)g;
    return NM_OK;
}

} // namespace

nm_status kv4_launch_append(const Kv4 &c, const Kv4Batch &b, int layer, const void *k, int64_t k_stride,
                            const void *v, int64_t v_stride, const void *q, int64_t q_stride, int n_q_heads,
                            void *q_out, int64_t q_out_stride, const float *rope, int64_t rope_rows, cudaStream_t st)
{
    const AppendArgs a{layer, n_q_heads, (const uint16_t *)k, (const uint16_t *)v, (const uint16_t *)q,
                       (uint16_t *)q_out, k_stride, v_stride, q_stride, q_out_stride, rope, rope_rows};
    unsigned grid;
    nm_status s = grid_of(b.n_tokens * (c.n_kv_heads + (q ? n_q_heads : 0)), &grid);
    if (s != NM_OK)
        return s;
    if (c.head_dim == 128)
        append_kernel<128><<<grid, 256, 0, st>>>(c, b, a);
    else
        append_kernel<64><<<grid, 256, 0, st>>>(c, b, a);
    return cudaGetLastError() == cudaSuccess ? NM_OK : NM_ERR_CUDA;
}

nm_status kv4_launch_read(const Kv4 &c, const Kv4Batch &b, int layer, void *k, void *v, bool f32, cudaStream_t st)
{
    unsigned grid;
    nm_status s = grid_of(b.n_tokens * c.n_kv_heads, &grid);
    if (s != NM_OK)
        return s;
    if (c.head_dim == 128) {
        if (f32)
            read_kernel<128, true><<<grid, 256, 0, st>>>(c, b, layer, k, v);
        else
            read_kernel<128, false><<<grid, 256, 0, st>>>(c, b, layer, k, v);
    } else {
        if (f32)
            read_kernel<64, true><<<grid, 256, 0, st>>>(c, b, layer, k, v);
        else
            read_kernel<64, false><<<grid, 256, 0, st>>>(c, b, layer, k, v);
    }
    return cudaGetLastError() == cudaSuccess ? NM_OK : NM_ERR_CUDA;
}

} // namespace nm
