// kv8.cu -- writing tokens to the 8-bit paged KV cache (with the rotary positions of q
// and k) and reading the values it holds back.
//
// A warp takes one block (16 tokens) of one kv head, four tokens at a time with eight
// lanes each: lane i of a token holds channels i D/16 .. of each half of the vector, the
// two halves that a rotation turns together. The four tokens are 2 t, 2 t + 1, 2 t + 8,
// 2 t + 9 for t = 0 .. 3: together they fill the 4-byte words of V's codes, so their
// lanes exchange words and store 16 bytes each.
//
// A block's scale is a power of two, so a value is its code exactly, and a token that
// needs a larger one moves the codes held there by whole exponents: they are rounded
// again only where they leave the codes' normal range. The greatest magnitude of the
// new tokens decides before any is written.
//
// The warps of a page's blocks stand side by side in a CTA. When a call fills a page its
// keys' bounds are taken from the codes just written and those held before.
#include "kv8.cuh"

namespace nm {
namespace {

// N = D / 16 channels of each half of a vector, as bf16 pairs and in fp32.
template <int N> struct Raw {
    uint32_t w[2][N / 2];
};
template <int N> struct Vec {
    float x[2][N];
};
// kOwn: of memory that the kernel may write too (q in place), not by the read-only path.
template <int N, bool kOwn> __device__ __forceinline__ Raw<N> load_raw(const uint16_t *p, int i, int half)
{
    Raw<N> r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint16_t *const at = p + h * half + N * i;
        if (N == 8) {
            const uint4 v = kOwn ? *(const uint4 *)at : __ldg((const uint4 *)at);
            r.w[h][0] = v.x;
            r.w[h][1] = v.y;
            r.w[h][N / 2 - 2] = v.z;
            r.w[h][N / 2 - 1] = v.w;
        } else {
            const uint2 v = kOwn ? *(const uint2 *)at : __ldg((const uint2 *)at);
            r.w[h][0] = v.x;
            r.w[h][1] = v.y;
        }
    }
    return r;
}
template <int N> __device__ __forceinline__ Vec<N> unpack(const Raw<N> &r)
{
    Vec<N> v;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < N / 2; ++n) {
            v.x[h][2 * n] = bf16lo_to_f32(r.w[h][n]);
            v.x[h][2 * n + 1] = bf16hi_to_f32(r.w[h][n]);
        }
    return v;
}
// (a cos - b sin, b cos + a sin) with the position's row of the table, each operation rounded.
template <int N> __device__ __forceinline__ void rotate(Vec<N> &v, const float *row, int i)
{
#pragma unroll
    for (int n = 0; n < N; n += 4) {
        const float4 c4 = __ldg((const float4 *)(row + N * i + n)), s4 = __ldg((const float4 *)(row + 8 * N + N * i + n));
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float a = v.x[0][n + m], b = v.x[1][n + m];
            v.x[0][n + m] = __fsub_rn(__fmul_rn(a, c[m]), __fmul_rn(b, s[m]));
            v.x[1][n + m] = __fadd_rn(__fmul_rn(b, c[m]), __fmul_rn(a, s[m]));
        }
    }
}

// 2^e for the least e with most <= m 2^e, m = (1 + limit / 2^23) 2^base: an exponent field.
__device__ __forceinline__ float pow2_over(uint32_t most, uint32_t limit, int base, int least, int largest)
{
    int e = (int)((most + (0x7FFFFFu - limit)) >> 23) - 127 - base;
    e = most == 0 || e < least ? least : e > largest ? largest : e;
    return __uint_as_float((uint32_t)(e + 127) << 23);
}
// Of a block: 448 = 1.75 * 2^8 is the largest code. Of bounds: 127 = 1.984375 * 2^6.
__device__ __forceinline__ float block_scale(uint32_t most) { return pow2_over(most, 0x600000u, 8, kKv8MinExp, kKv8MaxExp); }
__device__ __forceinline__ float bounds_step(uint32_t most) { return pow2_over(most, 0x7E0000u, 6, kKv8MinStep, 127); }
// 1 / s for a power of two
__device__ __forceinline__ float pow2_inverse(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

__device__ __forceinline__ uint32_t encode2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// large: some value of the block is above kKv4Limit
__device__ __forceinline__ uint32_t encode4(const float *x, float inv, bool large)
{
    float y[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        y[n] = x[n];
        if (large)
            y[n] = fminf(fmaxf(y[n], -kKv4Limit), kKv4Limit);
        y[n] *= inv;
    }
    return encode2(y[0], y[1]) | encode2(y[2], y[3]) << 16;
}
// Four codes times `by` (a power of two of at most 1), rounded again.
__device__ __forceinline__ uint32_t again4(uint32_t codes, __half2 by)
{
    uint16_t r[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t two = kv8_decode(codes >> (16 * h));
        const __half2 x = __hmul2(*(const __half2 *)&two, by);
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r[h]) : "r"(*(const uint32_t *)&x));
    }
    return r[0] | (uint32_t)r[1] << 16;
}

// Words of the four lanes of a part of a token (8 lanes apart): lane `part` gives its word p to
// lane p and gets word `part` of each: out[p] comes from lane p.
__device__ __forceinline__ void swap_words(uint32_t (&a)[4], int part)
{
    const auto swap = [](uint32_t &x, uint32_t &y, bool yes) {
        const uint32_t z = yes ? y : x;
        y = yes ? x : y;
        x = z;
    };
    swap(a[0], a[1], part & 1);
    swap(a[2], a[3], part & 1);
    swap(a[0], a[2], part & 2);
    swap(a[1], a[3], part & 2);
}
__device__ __forceinline__ void exchange(uint32_t (&a)[4], int part)
{
    swap_words(a, part); // a[x]: the word for lane part ^ x
#pragma unroll
    for (int x = 1; x < 4; ++x)
        a[x] = __shfl_xor_sync(~0u, a[x], 8 * x);
    swap_words(a, part);
}
// Byte b of word a becomes byte a of word b.
__device__ __forceinline__ void transpose_bytes(uint32_t (&a)[4])
{
    const uint32_t x = __byte_perm(a[0], a[1], 0x5140), y = __byte_perm(a[2], a[3], 0x5140);
    const uint32_t z = __byte_perm(a[0], a[1], 0x7362), w = __byte_perm(a[2], a[3], 0x7362);
    a[0] = __byte_perm(x, y, 0x5410);
    a[1] = __byte_perm(x, y, 0x7632);
    a[2] = __byte_perm(z, w, 0x5410);
    a[3] = __byte_perm(z, w, 0x7632);
}
// Where in a cell word p of lane i stands in K (slot's row) and where its four channels stand in V.
template <int D> __device__ __forceinline__ int channel_of(int p, int i)
{
    return D == 128 ? (p >> 1) * 64 + 8 * i + 4 * (p & 1) : p * 32 + 4 * i;
}
template <int D> __device__ __forceinline__ int k_at(int slot, int ch)
{
    return (slot >> 3) * 8 * D + (ch >> 6) * 512 + (slot & 7) * 64 + (ch & 63);
}
template <int D> __device__ __forceinline__ int v_at(int t, int ch) // of a multiple of 4
{
    return Kv8Cell<D>::kV + ch * 16 + t * 16;
}
__device__ __forceinline__ int slot_of(int t, int part) { return 2 * t + (part & 1) + 8 * (part >> 1); }

// The stretch of 2^shift positions (a block or a page) that slot x of a call's work stands for.
// Sequence i has the slots from (starts[i] >> shift) + 2 i on: at least as many as the stretches
// that its new tokens lie in.
struct Job {
    Kv4Seq s;
    int nth, from, to; // the stretch's number; positions [from, to) of it are the call's
    int missing;       // (first slot) the first so many new tokens are at no position: len < n_new
};
__device__ __forceinline__ bool job_of(const Kv4 &c, const Kv4Batch &b, int64_t x, int shift, bool report, Job *j)
{
    int i;
    int64_t first = x;
    j->missing = 0;
    if (!b.starts) {
        i = (int)x;
        if (i >= b.n_seqs)
            return false;
    } else {
        int lo = 0, hi = b.n_seqs;
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if ((int64_t)(b.starts[m] >> shift) + 2 * m <= x)
                lo = m;
            else
                hi = m;
        }
        i = lo;
        first = (int64_t)(b.starts[i] >> shift) + 2 * i;
    }
    const int64_t nth = x - first;
    if (nth < 0)
        return false;
    j->s = kv4_seq(c, b, i, report && nth == 0);
    int begin = j->s.len - j->s.n_new;
    if (begin < 0) {
        if (nth == 0) {
            j->missing = -begin;
            if (report)
                kv4_bad(c);
        }
        begin = 0;
    }
    if (j->s.n_new == 0 || j->s.len == 0 || nth > ((j->s.len - 1) >> shift) - (begin >> shift))
        return false;
    j->nth = (begin >> shift) + (int)nth;
    j->from = max(begin, j->nth << shift);
    j->to = (int)min((int64_t)j->s.len, ((int64_t)j->nth + 1) << shift);
    return true;
}
// Slots of the stretches of a call.
int64_t slots_of(const Kv4Batch &b, int shift)
{
    return b.starts && b.n_seqs > 0 ? (b.n_tokens >> shift) + 2 * (int64_t)b.n_seqs : b.n_seqs;
}

constexpr int kFours = 4; // fours of heads that a warp turns at most
struct AppendArgs {
    int layer, n_q_heads;
    const uint16_t *k, *v, *q;
    uint16_t *q_out;
    int64_t k_stride, v_stride, q_stride, q_out_stride;
    const float *rope;
    int64_t rope_rows;
    int64_t units;      // page slots times the kv heads
    int64_t unit_ctas;  // the CTAs that hold their warps
    int64_t q_ctas;     // and the ones that turn q
    int q_warps, q_each; // warps of a token's q heads, and how many fours of heads each turns
};

// Tokens at positions [from, to) of the block that begins at `base`, to its cell.
template <int D>
__device__ __forceinline__ void append_block(const AppendArgs &a, const Kv4Seq &s, int head, uint8_t *cell, int base,
                                             int from, int to)
{
    constexpr int N = D / 16;
    using C = Kv8Cell<D>;
    const int lane = threadIdx.x & 31, i = lane & 7, part = lane >> 3;
    // The four tokens t of the lanes: K rotated, V as it came. The tokens are read twice, for the scale and for the
    // codes (the second time from L1): held in registers they leave room for half as many warps.
    const auto token_at = [&](int t, Vec<N> *k, Raw<N> *v) {
        const int pos = base + slot_of(t, part);
        const bool ok = pos >= from && pos < to;
        Raw<N> rk{};
        *v = Raw<N>{};
        if (ok) {
            const int64_t token = (int64_t)s.first + (pos - (s.len - s.n_new));
            rk = load_raw<N, false>(a.k + token * a.k_stride + (int64_t)head * D, i, D / 2);
            *v = load_raw<N, false>(a.v + token * a.v_stride + (int64_t)head * D, i, D / 2);
        }
        *k = unpack<N>(rk);
        if (a.rope && ok)
            rotate<N>(*k, a.rope + (int64_t)pos * D, i);
        return ok;
    };
    uint32_t most_k = 0, most_v = 0, bad_bits = 0;
    // not unrolled: a decode step's one token runs a quarter of the code
#pragma unroll 1
    for (int t = 0; t < 4; ++t) {
        const int first = base + 2 * t;
        if (first + 9 < from || first >= to)
            continue; // none of the four is the call's
        Vec<N> k;
        Raw<N> v;
        token_at(t, &k, &v);
        const Vec<N> w = unpack<N>(v);
        uint32_t mk = 0, mv = 0; // magnitudes as whole numbers: what is not finite is at least 0x7F800000
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < N; ++n) {
                mk = max(mk, __float_as_uint(k.x[h][n]) & 0x7FFFFFFFu);
                mv = max(mv, __float_as_uint(w.x[h][n]) & 0x7FFFFFFFu);
            }
        const uint32_t votes = __ballot_sync(~0u, max(mk, mv) < 0x7F800000u);
        if (((votes >> (8 * part)) & 0xFFu) != 0xFFu) { // one of the token's eight lanes
            bad_bits |= 1u << t;
        } else {
            most_k = max(most_k, mk);
            most_v = max(most_v, mv);
        }
    }
    most_k = __reduce_max_sync(~0u, most_k);
    most_v = __reduce_max_sync(~0u, most_v);
    float sk = block_scale(most_k), sv = block_scale(most_v);
    if (from > base) { // codes of earlier tokens: the scales may only grow
        const float2 old = *(const float2 *)(cell + C::kScales);
        const auto grow = [&](float &now, float was, uint8_t *codes) {
            if (now <= was) {
                now = was;
                return;
            }
            // (2^-20 brings every code below half the least one, as any smaller factor does)
            const float by = fmaxf(was * pow2_inverse(now), 9.5367431640625e-07f);
            const __half2 by2 = __float2half2_rn(by);
#pragma unroll
            for (int n = 0; n < D / 32; ++n) {
                uint4 *const p = (uint4 *)(codes + n * 512) + lane;
                uint4 x = *p;
                x.x = again4(x.x, by2);
                x.y = again4(x.y, by2);
                x.z = again4(x.z, by2);
                x.w = again4(x.w, by2);
                *p = x;
            }
        };
        grow(sk, old.x, cell);
        grow(sv, old.y, cell + C::kV);
        __syncwarp(); // before the new tokens' codes
    }
    if (lane == 0)
        *(float2 *)(cell + C::kScales) = make_float2(sk, sv);
    const float ik = pow2_inverse(sk), iv = pow2_inverse(sv);
    const bool large = max(most_k, most_v) > __float_as_uint(kKv4Limit);
#pragma unroll 1
    for (int t = 0; t < 4; ++t) {
        const int first = base + 2 * t;
        if (first + 9 < from || first >= to)
            continue;
        Vec<N> k;
        Raw<N> v;
        const bool ok = token_at(t, &k, &v), bad = bad_bits >> t & 1u;
        const uint32_t votes = __ballot_sync(~0u, ok);
        const Vec<N> w = unpack<N>(v);
        uint32_t cv[4] = {0, 0, 0, 0};
#pragma unroll
        for (int p = 0; p < N / 2; ++p) {
            const int h = p / (N / 4), n = 4 * (p % (N / 4));
            const uint32_t ck = bad ? 0x7F7F7F7Fu : encode4(&k.x[h][n], ik, large); // a NaN for each query
            if (ok)
                *(uint32_t *)(cell + k_at<D>(slot_of(t, part), channel_of<D>(p, i))) = ck;
            cv[p] = bad ? 0u : encode4(&w.x[h][n], iv, large);
        }
        exchange(cv, part);
        transpose_bytes(cv);
        if (part < N / 2) {
            uint4 *const at = (uint4 *)(cell + v_at<D>(t, channel_of<D>(part, i)));
            const uint32_t keep = (votes & 1u ? 0u : 0xFFu) | (votes & 0x100u ? 0u : 0xFF00u) |
                                  (votes & 0x10000u ? 0u : 0xFF0000u) | (votes & 0x1000000u ? 0u : 0xFF000000u);
            uint4 x = make_uint4(cv[0], cv[1], cv[2], cv[3]);
            if (keep) {
                const uint4 was = *at;
                x = make_uint4((x.x & ~keep) | (was.x & keep), (x.y & ~keep) | (was.y & keep),
                               (x.z & ~keep) | (was.z & keep), (x.w & ~keep) | (was.w & keep));
            }
            *at = x;
        }
    }
}

// Per channel the greatest and the least key of a block's 16 tokens, to shared memory. NaN keys do
// not count (a channel of nothing else gives NaN).
template <int D> __device__ __forceinline__ void block_bounds(const uint8_t *cell, float *upper, float *lower)
{
    using C = Kv8Cell<D>;
    const int lane = threadIdx.x & 31;
    const float s = *(const float *)(cell + C::kScales);
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
        __half2 hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint4 x = *((const uint4 *)(cell + e * 8 * D + j * 512) + lane);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                const uint32_t two = kv8_decode(w[n / 2] >> (16 * (n & 1)));
                const __half2 y = *(const __half2 *)&two;
                hi[n] = e ? __hmax2(hi[n], y) : y;
                lo[n] = e ? __hmin2(lo[n], y) : y;
            }
        }
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                hi[n] = __hmax2(hi[n], __shfl_xor_sync(~0u, hi[n], o));
                lo[n] = __hmin2(lo[n], __shfl_xor_sync(~0u, lo[n], o));
            }
        if (lane < 4) {
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                const int ch = 64 * j + 16 * lane + 2 * n;
                *(float2 *)(upper + ch) = make_float2(__low2float(hi[n]) * s, __high2float(hi[n]) * s);
                *(float2 *)(lower + ch) = make_float2(__low2float(lo[n]) * s, __high2float(lo[n]) * s);
            }
        }
    }
}

// The bounds of a page, from those of its blocks (rows of D floats in shared memory), by one warp.
template <int D>
__device__ __forceinline__ void page_bounds(const float *upper, const float *lower, int blocks, uint8_t *tail)
{
    using C = Kv8Cell<D>;
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    float hi[E], lo[E];
    uint32_t most = 0;
#pragma unroll
    for (int n = 0; n < E; ++n) {
        hi[n] = upper[E * lane + n];
        lo[n] = lower[E * lane + n];
        for (int x = 1; x < blocks; ++x) {
            hi[n] = fmaxf(hi[n], upper[x * D + E * lane + n]);
            lo[n] = fminf(lo[n], lower[x * D + E * lane + n]);
        }
        if (hi[n] != hi[n])
            hi[n] = lo[n] = 0.0f;
        most = max(most, max(__float_as_uint(hi[n]) & 0x7FFFFFFFu, __float_as_uint(lo[n]) & 0x7FFFFFFFu));
    }
    const float step = bounds_step(__reduce_max_sync(~0u, most)), inv = pow2_inverse(step);
    uint32_t up = 0, down = 0;
#pragma unroll
    for (int n = 0; n < E; ++n) {
        up |= ((uint32_t)(int)ceilf(hi[n] * inv) & 0xFFu) << (8 * n);
        down |= ((uint32_t)(int)floorf(lo[n] * inv) & 0xFFu) << (8 * n);
    }
    if (E == 4) {
        *(uint32_t *)(tail + 4 * lane) = up;
        *(uint32_t *)(tail + C::kLower + 4 * lane) = down;
    } else {
        *(uint16_t *)(tail + 2 * lane) = (uint16_t)up;
        *(uint16_t *)(tail + C::kLower + 2 * lane) = (uint16_t)down;
    }
    if (lane == 0)
        *(float *)(tail + C::kStep) = step;
}

template <int D> __device__ __forceinline__ void append_pages(const Kv4 &c, const Kv4Batch &b, const AppendArgs &a)
{
    __shared__ __align__(16) float upper[8 * D], lower[8 * D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int shift = c.page_shift - 4, blocks = 1 << shift, nth = warp & (blocks - 1);
    const int64_t unit = (int64_t)blockIdx.x * (8 >> shift) + (warp >> shift);
    Job j;
    const int head = (int)(unit % c.n_kv_heads);
    const bool report = lane == 0 && nth == 0;
    bool have = unit < a.units && job_of(c, b, unit / c.n_kv_heads, c.page_shift, report && head == 0, &j);
    uint8_t *at = nullptr;
    if (have) {
        const int page = kv4_page(c, j.s.row, j.nth);
        // A page that another sequence reads is not written: tokens fall there only when reserve did
        // not make room for them.
        have = page >= 0 && c.refs[page] <= 1;
        if (!have && report)
            kv4_bad(c);
        if (have && a.rope && j.to > a.rope_rows) {
            if (report)
                kv4_bad(c);
            j.to = (int)a.rope_rows;
        }
        if (have)
            at = c.pool + kv8_head_offset<D>(c, page, a.layer, head);
    }
    const bool full = have && j.from < j.to && j.to == (j.nth + 1) << c.page_shift;
    if (have) {
        const int base = (j.nth << c.page_shift) + nth * kKv4Cell;
        const int from = max(j.from, base), to = min(j.to, base + kKv4Cell);
        uint8_t *const cell = at + nth * Kv8Cell<D>::kBytes;
        if (from < to)
            append_block<D>(a, j.s, head, cell, base, from, to);
        if (full) {
            __syncwarp(); // the codes are read by other lanes than wrote them
            block_bounds<D>(cell, upper + warp * D, lower + warp * D);
        }
    }
    __syncthreads();
    if (full && nth == 0)
        page_bounds<D>(upper + warp * D, lower + warp * D, blocks, at + blocks * Kv8Cell<D>::kBytes);
}

template <int D> __device__ __forceinline__ void append_q(const Kv4 &c, const Kv4Batch &b, const AppendArgs &a, int64_t w)
{
    constexpr int N = D / 16;
    const int lane = threadIdx.x & 31, i = lane & 7;
    const int64_t token = w / a.q_warps;
    if (token >= b.n_tokens)
        return;
    const int at = kv4_find(b, token);
    int pos = -1, len = 0;
    if (at >= 0) {
        const Kv4Seq s = kv4_seq(c, b, at, false); // the warps of the pages report
        len = s.len;
        pos = s.len - s.n_new + (int)(token - s.first);
    }
    const bool ok = pos >= 0 && pos < len && (!a.rope || pos < a.rope_rows);
    const int h0 = (int)(w % a.q_warps) * a.q_each * 4 + (lane >> 3);
    // all of the warp's heads are asked for before the first is written
    Raw<N> raw[kFours];
#pragma unroll
    for (int n = 0; n < kFours; ++n)
        if (n < a.q_each && h0 + 4 * n < a.n_q_heads)
            raw[n] = load_raw<N, true>(a.q + token * a.q_stride + (int64_t)(h0 + 4 * n) * D, i, D / 2);
#pragma unroll
    for (int n = 0; n < kFours; ++n) {
        const int h = h0 + 4 * n;
        if (n >= a.q_each || h >= a.n_q_heads)
            break;
        Vec<N> v = unpack<N>(raw[n]);
        if (a.rope && ok)
            rotate<N>(v, a.rope + (int64_t)pos * D, i);
        uint16_t *const o = a.q_out + token * a.q_out_stride + (int64_t)h * D;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t y[N / 2];
#pragma unroll
            for (int m = 0; m < N / 2; ++m)
                y[m] = ok ? f32_to_bf16_rn(v.x[half][2 * m]) | ((uint32_t)f32_to_bf16_rn(v.x[half][2 * m + 1]) << 16) : 0u;
            if (N == 8)
                *(uint4 *)(o + half * (D / 2) + 8 * i) = make_uint4(y[0], y[1], y[N / 2 - 2], y[N / 2 - 1]);
            else
                *(uint2 *)(o + half * (D / 2) + 4 * i) = make_uint2(y[0], y[1]);
        }
    }
}

template <int D> __global__ void __launch_bounds__(256, 4) append_kernel(const Kv4 c, const Kv4Batch b, const AppendArgs a)
{
    if (blockIdx.x < a.unit_ctas) {
        append_pages<D>(c, b, a);
    } else if (blockIdx.x < a.unit_ctas + a.q_ctas) {
        append_q<D>(c, b, a, (int64_t)(blockIdx.x - a.unit_ctas) * 8 + (threadIdx.x >> 5));
    } else { // starts out of range need not have a page of their own: one CTA looks at all of them
        for (int i = threadIdx.x; i < b.n_seqs; i += blockDim.x)
            kv4_seq(c, b, i, true);
    }
}

// One row of read's results (n bytes of each) becomes zeros, a warp to it.
__device__ __forceinline__ void zero_row(void *k, void *v, int64_t row, int64_t n)
{
    for (int64_t i = threadIdx.x & 31; i < n / 16; i += 32) {
        if (k)
            ((uint4 *)((uint8_t *)k + row * n))[i] = make_uint4(0, 0, 0, 0);
        if (v)
            ((uint4 *)((uint8_t *)v + row * n))[i] = make_uint4(0, 0, 0, 0);
    }
}

constexpr int kRestCtas = 16; // CTAs that look for rows of no sequence: there are few as a rule

// One warp per (block, kv head); the last CTAs see to the rows that belong to no sequence.
template <int D, bool F32>
__global__ void __launch_bounds__(256)
    read_kernel(const Kv4 c, const Kv4Batch b, int layer, void *k, void *v, int64_t slots, int64_t block_ctas)
{
    constexpr int N = D / 16;
    using C = Kv8Cell<D>;
    const int lane = threadIdx.x & 31, i = lane & 7, part = lane >> 3;
    const int64_t row_bytes = (int64_t)c.n_kv_heads * D * (F32 ? 4 : 2);
    if (blockIdx.x >= block_ctas) {
        bool rest = !kv4_ends(b);
        for (int x = threadIdx.x; x < b.n_seqs; x += blockDim.x)
            rest |= kv4_seq(c, b, x, blockIdx.x == block_ctas).first < 0;
        if (__syncthreads_or(rest))
            kv4_uncovered(b, (blockIdx.x - block_ctas) * 8 + (threadIdx.x >> 5), kRestCtas * 8,
                          [&](int64_t row) { zero_row(k, v, row, row_bytes); });
        return;
    }
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (w >= slots)
        return;
    const int head = (int)(w % c.n_kv_heads);
    Job j;
    const bool have = job_of(c, b, w / c.n_kv_heads, 4, head == 0 && lane == 0, &j);
    for (int z = 0; z < j.missing; ++z) { // rows of tokens that the sequence does not have
        const int64_t at = ((int64_t)(j.s.first + z) * c.n_kv_heads + head) * D;
        for (int n = lane; n < D * (F32 ? 2 : 1); n += 32) {
            if (k)
                ((uint16_t *)k + at * (F32 ? 2 : 1))[n] = 0;
            if (v)
                ((uint16_t *)v + at * (F32 ? 2 : 1))[n] = 0;
        }
    }
    if (!have)
        return;
    const int page = kv4_page(c, j.s.row, j.nth >> (c.page_shift - 4));
    if (page < 0 && lane == 0)
        kv4_bad(c);
    const uint8_t *cell = nullptr;
    float2 scales = make_float2(0.0f, 0.0f);
    if (page >= 0) {
        cell = c.pool + kv8_head_offset<D>(c, page, layer, head) +
               (j.nth & ((1 << (c.page_shift - 4)) - 1)) * C::kBytes;
        scales = *(const float2 *)(cell + C::kScales);
    }
    // K and V codes of the lane's words, all asked for first
    uint32_t ck[4][N / 2], cv[4][4] = {};
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int p = 0; p < N / 2; ++p)
            ck[t][p] = cell ? *(const uint32_t *)(cell + k_at<D>(slot_of(t, part), channel_of<D>(p, i))) : 0u;
        if (cell && part < N / 2) {
            const uint4 x = *(const uint4 *)(cell + v_at<D>(t, channel_of<D>(part, i)));
            cv[t][0] = x.x, cv[t][1] = x.y, cv[t][2] = x.z, cv[t][3] = x.w;
        }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        transpose_bytes(cv[t]);
        exchange(cv[t], part);
        const int pos = j.nth * kKv4Cell + slot_of(t, part);
        if (pos < j.from || pos >= j.to)
            continue;
        const int64_t token = (int64_t)j.s.first + (pos - (j.s.len - j.s.n_new));
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            void *const out = kv ? v : k;
            if (!out)
                continue;
            const float s = kv ? scales.y : scales.x;
#pragma unroll
            for (int p = 0; p < N / 2; ++p) {
                const uint32_t code = kv ? cv[t][p] : ck[t][p];
                const uint32_t a2 = kv8_decode(code), b2 = kv8_decode(code >> 16);
                const __half2 x = *(const __half2 *)&a2, y = *(const __half2 *)&b2;
                const float4 f = make_float4(__low2float(x) * s, __high2float(x) * s, __low2float(y) * s, __high2float(y) * s);
                const int64_t o = (token * c.n_kv_heads + head) * D + channel_of<D>(p, i);
                if (F32)
                    *(float4 *)((float *)out + o) = f;
                else
                    *(uint2 *)((uint16_t *)out + o) =
                        make_uint2(f32_to_bf16_rn(f.x) | ((uint32_t)f32_to_bf16_rn(f.y) << 16),
                                   f32_to_bf16_rn(f.z) | ((uint32_t)f32_to_bf16_rn(f.w) << 16));
            }
        }
    }
}

} // namespace

nm_status kv8_launch_append(const Kv4 &c, const Kv4Batch &b, int layer, const void *k, int64_t k_stride,
                            const void *v, int64_t v_stride, const void *q, int64_t q_stride, int n_q_heads,
                            void *q_out, int64_t q_out_stride, const float *rope, int64_t rope_rows, cudaStream_t st)
{
    AppendArgs a{layer, n_q_heads, (const uint16_t *)k, (const uint16_t *)v, (const uint16_t *)q,
                 (uint16_t *)q_out, k_stride, v_stride, q_stride, q_out_stride, rope, rope_rows, 0, 0, 0, 1, 1};
    const int per_cta = 8 >> (c.page_shift - 4);
    a.units = slots_of(b, c.page_shift) * c.n_kv_heads;
    a.unit_ctas = (a.units + per_cta - 1) / per_cta;
    if (q) {
        // With many tokens a warp turns up to four fours of a token's heads, so that its angles are read once. A four and up to
        // four to a warp, us, head size 128, 8 kv heads: 32 query heads, 2048 tokens 16.0, 16.7; 4096 24.9, 20.5; 8192 55, 43;
        // 16384 109, 82. 128 heads: 512 tokens 13.9, 14.2; 1024 18.0, 16.7; 2048 39, 31; 16384 304, 197.
        const int fours = (n_q_heads + 3) / 4;
        a.q_each = b.n_tokens * fours >= 65536 ? (fours < kFours ? fours : kFours) : 1;
        a.q_warps = (fours + a.q_each - 1) / a.q_each;
        a.q_ctas = (b.n_tokens * a.q_warps + 7) / 8;
    }
    const int64_t grid = a.unit_ctas + a.q_ctas + (b.starts ? 1 : 0);
    if (grid > 0x7FFFFFFF)
        return NM_ERR_SHAPE;
    if (c.head_dim == 128)
        append_kernel<128><<<(unsigned)grid, 256, 0, st>>>(c, b, a);
    else
        append_kernel<64><<<(unsigned)grid, 256, 0, st>>>(c, b, a);
    return cudaGetLastError() == cudaSuccess ? NM_OK : NM_ERR_CUDA;
}

nm_status kv8_launch_read(const Kv4 &c, const Kv4Batch &b, int layer, void *k, void *v, bool f32, cudaStream_t st)
{
    const int64_t slots = slots_of(b, 4) * c.n_kv_heads, ctas = (slots + 7) / 8;
    const int64_t grid = ctas + (b.starts ? kRestCtas : 0);
    if (grid > 0x7FFFFFFF)
        return NM_ERR_SHAPE;
    const auto go = [&](auto kernel) { kernel<<<(unsigned)grid, 256, 0, st>>>(c, b, layer, k, v, slots, ctas); };
    if (c.head_dim == 128)
        f32 ? go(read_kernel<128, true>) : go(read_kernel<128, false>);
    else
        f32 ? go(read_kernel<64, true>) : go(read_kernel<64, false>);
    return cudaGetLastError() == cudaSuccess ? NM_OK : NM_ERR_CUDA;
}

} // namespace nm
