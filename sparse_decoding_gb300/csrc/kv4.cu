// kv4.cu -- writing tokens to the 4-bit paged KV cache (with the rotary
// positions of q and k) and reading the values it holds back.
//
// A warp takes one cell (16 tokens) of one kv head, four tokens at a time with
// eight lanes each: lane i of a token holds channels i D/16 .. of each half of the
// vector, the two halves that a rotation turns together, so a rotation stays in the
// lane and a group's least and greatest values take three shuffles. The four tokens
// are 2 t, 2 t + 1, 2 t + 8, 2 t + 9 for t = 0 .. 3: together they fill 16 bytes of
// V's codes, so a cell is written in full sectors. The q heads are turned by other warps of the same launch, four heads of a
// token at a time with the token's angles in registers.
//
// Bytes should bound it: k, v, q and q_out once, the angles once per SM and token.
// Measured (one GB300; 16384 tokens, 32 and 8 heads, D = 128): append 80 us (362 MB,
// 0.67 of the measured copy rate; 101000 instructions a scheduler, half of them the
// quantisation, waiting for each cell's loads), 86 while a warp asked for its q heads one
// by one; read 22 us, of which its 86 MB take 13: it waits for one token's codes and
// parameters at a time. A warp per token and head with a division for each value took 138 us.
#include "kv4.cuh"

namespace nm {
namespace {

__device__ __forceinline__ float saturate(float x)
{
    return x != x ? 0.0f : fminf(fmaxf(x, -kKv4Limit), kKv4Limit);
}

// N = D / 16 channels of each half of a vector, as bf16 pairs and in fp32.
template <int N> struct Raw {
    uint32_t w[2][N / 2];
};
template <int N> struct Vec {
    float x[2][N];
};
template <int N> __device__ __forceinline__ Raw<N> load_raw(const uint16_t *p, int i, int half)
{
    Raw<N> r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (N == 8) {
            const uint4 v = ldg_nc128(p + h * half + 8 * i);
            r.w[h][0] = v.x;
            r.w[h][1] = v.y;
            r.w[h][N / 2 - 2] = v.z;
            r.w[h][N / 2 - 1] = v.w;
        } else {
            const uint2 v = __ldg((const uint2 *)(p + h * half + 4 * i));
            r.w[h][0] = v.x;
            r.w[h][1] = v.y;
        }
    }
    return r;
}
// The same of memory that the kernel may write too (q in place): not by the read-only path.
template <int N> __device__ __forceinline__ Raw<N> load_own(const uint16_t *p, int i, int half)
{
    Raw<N> r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (N == 8) {
            const uint4 v = *(const uint4 *)(p + h * half + 8 * i);
            r.w[h][0] = v.x;
            r.w[h][1] = v.y;
            r.w[h][N / 2 - 2] = v.z;
            r.w[h][N / 2 - 1] = v.w;
        } else {
            const uint2 v = *(const uint2 *)(p + h * half + 4 * i);
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
// A token's cos and sin of the lane's angles.
template <int N> struct Turn {
    float c[N], s[N];
};
template <int N> __device__ __forceinline__ Turn<N> load_turn(const float *row, int i)
{
    Turn<N> t;
#pragma unroll
    for (int n = 0; n < N; n += 4) {
        const float4 c = __ldg((const float4 *)(row + N * i + n)), s = __ldg((const float4 *)(row + 8 * N + N * i + n));
        t.c[n] = c.x, t.c[n + 1] = c.y, t.c[n + 2] = c.z, t.c[n + 3] = c.w;
        t.s[n] = s.x, t.s[n + 1] = s.y, t.s[n + 2] = s.z, t.s[n + 3] = s.w;
    }
    return t;
}
// (a cos - b sin, b cos + a sin), each operation rounded.
template <int N> __device__ __forceinline__ void rotate(Vec<N> &v, const Turn<N> &t)
{
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const float a = v.x[0][n], b = v.x[1][n];
        v.x[0][n] = __fsub_rn(__fmul_rn(a, t.c[n]), __fmul_rn(b, t.s[n]));
        v.x[1][n] = __fadd_rn(__fmul_rn(b, t.c[n]), __fmul_rn(a, t.s[n]));
    }
}

// The codes of N values of a group, value n in bits 4 n ..: rint((x - mid) / s), the
// quotient rounded as fp32 division rounds it. x * (1 / s) is off by under 1e-5 here
// (|quotient| < 16), so it decides unless it is that near to the middle between two
// codes; then the division does.
template <int N> __device__ __forceinline__ uint32_t codes_of(const float *x, float s, float mid)
{
    constexpr float kMagic = 12582912.0f; // 1.5 * 2^23: adding it rounds to a whole number, ties to even
    const float inv = s > 0.0f ? 1.0f / s : 0.0f;
    float whole[N], far = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const float t = fminf(fmaxf(__fsub_rn(x[n], mid) * inv, -8.0f), 7.0f);
        whole[n] = (t + kMagic) - kMagic;
        far = fmaxf(far, fabsf(t - whole[n]));
    }
    if (far > 0.4999f) {
#pragma unroll 1
        for (int n = 0; n < N; ++n) {
            float y = x[0];
#pragma unroll
            for (int m = 1; m < N; ++m)
                y = m == n ? x[m] : y;
            const float w = rintf(fminf(fmaxf(__fdiv_rn(__fsub_rn(y, mid), s), -8.0f), 7.0f));
#pragma unroll
            for (int m = 0; m < N; ++m)
                whole[m] = m == n ? w : whole[m];
        }
    }
    // four codes to a number below 2^16: sums of code * 16^k are exact
    uint32_t r = 0;
#pragma unroll
    for (int n = 0; n < N; n += 4) {
        const float four = fmaf(whole[n + 3], 4096.0f, fmaf(whole[n + 2], 256.0f, fmaf(whole[n + 1], 16.0f, whole[n] + 34952.0f)));
        r |= (__float_as_uint(four + 8388608.0f) & 0xFFFFu) << (4 * n); // 34952 = 8 * 0x1111
    }
    return r;
}

// One group's parameters, from the least and greatest of its values.
__device__ __forceinline__ __half2 params_of(float lo, float hi)
{
    const float s = __half2float(__float2half_rn(bf16_to_f32(f32_to_bf16_rn(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f)))));
    return __halves2half2(__float2half_rn(s), __float2half_rn(__fadd_rn(lo, __fmul_rn(s, 8.0f))));
}

// A token of a warp's cell, as its eight lanes hold it: K's and V's codes of the two
// halves (8 or 4 of them each) and the parameters of the groups.
template <int D> struct Coded {
    uint32_t code[2][2];
    __half2 par[2][D / 64];
};
template <int D> __device__ __forceinline__ Coded<D> encode(Vec<D / 16> &k, Vec<D / 16> &v)
{
    constexpr int N = D / 16, G = D / 64;
    Coded<D> r;
    float lo[2][2], hi[2][2], none = 0.0f; // [K, V][half]; 0 * x is NaN for what is not finite
    const auto bounds = [&]() {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float *z = kv ? v.x[h] : k.x[h];
                lo[kv][h] = hi[kv][h] = z[0];
#pragma unroll
                for (int n = 1; n < N; ++n) {
                    lo[kv][h] = fminf(lo[kv][h], z[n]);
                    hi[kv][h] = fmaxf(hi[kv][h], z[n]);
                }
            }
    };
    bounds();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < N; ++n)
            none = fmaf(v.x[h][n], 0.0f, fmaf(k.x[h][n], 0.0f, none));
    bool fine = none == 0.0f;
    const float least = fminf(fminf(lo[0][0], lo[0][1]), fminf(lo[1][0], lo[1][1]));
    const float most = fmaxf(fmaxf(hi[0][0], hi[0][1]), fmaxf(hi[1][0], hi[1][1]));
    const uint32_t votes = __ballot_sync(~0u, fine);
    if (__any_sync(~0u, !fine || least < -kKv4Limit || most > kKv4Limit)) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < N; ++n) {
                k.x[h][n] = saturate(k.x[h][n]);
                v.x[h][n] = saturate(v.x[h][n]);
            }
        bounds();
    }
    fine = ((votes >> (threadIdx.x & 24)) & 0xFFu) == 0xFFu; // all eight lanes of the token
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        Vec<N> &z = kv ? v : k;
        if (G == 1) {
            lo[kv][0] = fminf(lo[kv][0], lo[kv][1]);
            hi[kv][0] = fmaxf(hi[kv][0], hi[kv][1]);
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                lo[kv][g] = fminf(lo[kv][g], __shfl_xor_sync(~0u, lo[kv][g], o));
                hi[kv][g] = fmaxf(hi[kv][g], __shfl_xor_sync(~0u, hi[kv][g], o));
            }
            r.par[kv][g] = params_of(lo[kv][g], hi[kv][g]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const __half2 p = r.par[kv][G == 2 ? h : 0];
            r.code[kv][h] = codes_of<N>(z.x[h], __low2float(p), __high2float(p));
        }
    }
    if (!fine) { // K poisoned, V kept finite
        r.code[0][0] = r.code[0][1] = 0x88888888u;
#pragma unroll
        for (int g = 0; g < G; ++g)
            r.par[0][g] = __halves2half2(__ushort_as_half(0x7E00), __ushort_as_half(0x7E00));
    }
    return r;
}

// The cell that slot x of a call's work stands for. Sequence i has the slots from
// starts[i] / 16 + 2 i on: at least as many as the cells that its new tokens lie in.
struct CellJob {
    Kv4Seq s;
    int cell, from, to; // positions [from, to) of the cell's are the call's
    int missing;        // (first slot) the first so many new tokens are at no position: len < n_new
};
__device__ __forceinline__ bool cell_job(const Kv4 &c, const Kv4Batch &b, int64_t x, bool report, CellJob *j)
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
            if ((int64_t)(b.starts[m] >> 4) + 2 * m <= x)
                lo = m;
            else
                hi = m;
        }
        i = lo;
        first = (int64_t)(b.starts[i] >> 4) + 2 * i;
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
    if (j->s.n_new == 0 || j->s.len == 0 || nth > (j->s.len - 1) / kKv4Cell - begin / kKv4Cell)
        return false;
    j->cell = begin / kKv4Cell + (int)nth;
    j->from = max(begin, j->cell * kKv4Cell);
    j->to = min(j->s.len, (j->cell + 1) * kKv4Cell);
    return true;
}

constexpr int kFours = 4; // fours of heads that a warp turns at most
struct AppendArgs {
    int layer, n_q_heads;
    const uint16_t *k, *v, *q;
    uint16_t *q_out;
    int64_t k_stride, v_stride, q_stride, q_out_stride;
    const float *rope;
    int64_t rope_rows;
    int64_t slots;      // of cells, times the kv heads: warps that write the cache
    int64_t cell_ctas;  // the CTAs that hold those warps
    int64_t q_ctas;     // and the ones that turn q
    int q_warps, q_each; // warps of a token's q heads, and how many fours of heads each turns
};

template <int D> __device__ __forceinline__ void append_cell(const Kv4 &c, const Kv4Batch &b, const AppendArgs &a, int64_t w)
{
    constexpr int N = D / 16, G = D / 64;
    using C = Kv4Cell<D>;
    const int lane = threadIdx.x & 31, i = lane & 7, part = lane >> 3; // part: r + 2 p of the token
    const int head = (int)(w % c.n_kv_heads);
    CellJob j;
    if (!cell_job(c, b, w / c.n_kv_heads, head == 0 && lane == 0, &j))
        return;
    const int page = kv4_page(c, j.s.row, (j.cell * kKv4Cell) >> c.page_shift);
    // A page that another sequence reads is not written: tokens fall there only when reserve did not make
    // room for them.
    if (page < 0 || c.refs[page] > 1) {
        if (lane == 0)
            kv4_bad(c);
        return;
    }
    if (a.rope && j.to > a.rope_rows) {
        if (lane == 0)
            kv4_bad(c);
        j.to = (int)a.rope_rows;
    }
    uint8_t *const dst = c.pool + kv4_cell_offset<D>(c, page, a.layer, head, j.cell & ((c.page_tokens >> 4) - 1));
    const int base = j.cell * kKv4Cell;
    const auto slot_of = [&](int t) { return 2 * t + (part & 1) + 8 * (part >> 1); };
    // not unrolled: a decode step's one token runs a quarter of the code, and more warps fit an SM
#pragma unroll 1
    for (int t = 0; t < 4; ++t) {
        const int slot = slot_of(t);
        const bool ok = base + slot >= j.from && base + slot < j.to;
        if (!__any_sync(~0u, ok))
            continue;
        const int64_t token = (int64_t)j.s.first + (base + slot - (j.s.len - j.s.n_new));
        Raw<N> rk{}, rv{};
        Turn<N> turn{};
        if (ok) {
            rk = load_raw<N>(a.k + token * a.k_stride + (int64_t)head * D, i, D / 2);
            rv = load_raw<N>(a.v + token * a.v_stride + (int64_t)head * D, i, D / 2);
            if (a.rope)
                turn = load_turn<N>(a.rope + (int64_t)(base + slot) * D, i);
        }
        Vec<N> k = unpack<N>(rk), v = unpack<N>(rv);
        if (a.rope)
            rotate<N>(k, turn);
        const Coded<D> e = encode<D>(k, v);
        // K: the token's row; half h of lane i: channels h D/2 + i N ..
        if (ok) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (D == 128)
                    *(uint32_t *)(dst + slot * 64 + (i >> 1) * 16 + h * 8 + (i & 1) * 4) = e.code[0][h];
                else // four codes: channels 32 h + 4 i of the one group
                    *(uint16_t *)(dst + slot * 32 + (2 * h + (i >> 2)) * 8 + (i & 3) * 2) = (uint16_t)e.code[0][h];
            }
            if (i < G)
                *(__half2 *)(dst + C::kKp + (slot * G + i) * 4) = i == 0 ? e.par[0][0] : e.par[0][G - 1];
        }
        // V: a token pair's fours of channels side by side: the even token's lane stores the pair's
        // first four of a half's channels, the odd one's the second (D = 128), or each half's (64)
        const bool both = __shfl_xor_sync(~0u, ok, 8) && ok;
        const int odd = part & 1;
        uint8_t *const at = dst + C::kV + t * 16 + (part >> 1) * 8; // + group * 512 + e * 64 + f * 4 + r * 2
        const uint32_t p0 = __shfl_xor_sync(~0u, e.code[1][0], 8), p1 = __shfl_xor_sync(~0u, e.code[1][1], 8);
        if (D == 128) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t own = e.code[1][h], other = h ? p1 : p0;
                uint8_t *const q = at + h * 512 + i * 64;
                if (both)
                    *(uint32_t *)(q + odd * 4) = odd ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
                else if (ok) {
                    *(uint16_t *)(q + odd * 2) = (uint16_t)own;
                    *(uint16_t *)(q + 4 + odd * 2) = (uint16_t)(own >> 16);
                }
            }
        } else {
            // four channels 32 h + 4 i: e = 4 h + i / 2, f = i % 2; the even lane stores half 0, the odd half 1
            const auto place = [&](int h) { return at + (4 * h + (i >> 1)) * 64 + (i & 1) * 4; };
            if (both)
                *(uint32_t *)place(odd) = odd ? (p1 & 0xFFFFu) | e.code[1][1] << 16 : (e.code[1][0] & 0xFFFFu) | p0 << 16;
            else if (ok) {
                *(uint16_t *)(place(0) + odd * 2) = (uint16_t)e.code[1][0];
                *(uint16_t *)(place(1) + odd * 2) = (uint16_t)e.code[1][1];
            }
        }
        if (i < G && ok) {
            const __half2 m = i == 0 ? e.par[1][0] : e.par[1][G - 1];
            __half *p = (__half *)(dst + C::kVp + ((t + 4 * (part >> 1)) * G + i) * 8) + odd;
            p[0] = __low2half(m);
            p[2] = __high2half(m);
        }
    }
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
        const Kv4Seq s = kv4_seq(c, b, at, false); // the warps of the cells report
        len = s.len;
        pos = s.len - s.n_new + (int)(token - s.first);
    }
    const bool ok = pos >= 0 && pos < len && (!a.rope || pos < a.rope_rows);
    Turn<N> turn{};
    if (a.rope && ok)
        turn = load_turn<N>(a.rope + (int64_t)pos * D, i);
    const int h0 = (int)(w % a.q_warps) * a.q_each * 4 + (lane >> 3);
    // all of the warp's heads are asked for before the first is written
    Raw<N> raw[kFours];
#pragma unroll
    for (int n = 0; n < kFours; ++n)
        if (n < a.q_each && h0 + 4 * n < a.n_q_heads)
            raw[n] = load_own<N>(a.q + token * a.q_stride + (int64_t)(h0 + 4 * n) * D, i, D / 2);
#pragma unroll
    for (int n = 0; n < kFours; ++n) {
        const int h = h0 + 4 * n;
        if (n >= a.q_each || h >= a.n_q_heads)
            break;
        Vec<N> v = unpack<N>(raw[n]);
        if (a.rope)
            rotate<N>(v, turn);
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
    const int warp = threadIdx.x >> 5;
    if (blockIdx.x < a.cell_ctas) {
        const int64_t w = (int64_t)blockIdx.x * 8 + warp;
        if (w < a.slots)
            append_cell<D>(c, b, a, w);
    } else if (blockIdx.x < a.cell_ctas + a.q_ctas) {
        append_q<D>(c, b, a, (int64_t)(blockIdx.x - a.cell_ctas) * 8 + warp);
    } else { // starts out of range need not have a cell of their own: one CTA looks at all of them
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

// One warp per (cell, kv head), as append; the last CTAs see to the rows that belong to no sequence.
template <int D, bool F32>
__global__ void __launch_bounds__(256)
    read_kernel(const Kv4 c, const Kv4Batch b, int layer, void *k, void *v, int64_t slots, int64_t cell_ctas)
{
    constexpr int N = D / 16, G = D / 64;
    using C = Kv4Cell<D>;
    const int lane = threadIdx.x & 31, i = lane & 7, part = lane >> 3;
    if (blockIdx.x >= cell_ctas) {
        bool rest = !kv4_ends(b);
        for (int x = threadIdx.x; x < b.n_seqs; x += blockDim.x)
            rest |= kv4_seq(c, b, x, blockIdx.x == cell_ctas).first < 0;
        if (__syncthreads_or(rest))
            kv4_uncovered(b, (blockIdx.x - cell_ctas) * 8 + (threadIdx.x >> 5), kRestCtas * 8,
                          [&](int64_t row) { zero_row(k, v, row, (int64_t)c.n_kv_heads * D * (F32 ? 4 : 2)); });
        return;
    }
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (w >= slots)
        return;
    const int head = (int)(w % c.n_kv_heads);
    CellJob j;
    const bool have = cell_job(c, b, w / c.n_kv_heads, head == 0 && lane == 0, &j);
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
    const int page = kv4_page(c, j.s.row, (j.cell * kKv4Cell) >> c.page_shift);
    if (page < 0 && lane == 0)
        kv4_bad(c);
    const uint8_t *const src =
        page < 0 ? nullptr : c.pool + kv4_cell_offset<D>(c, page, layer, head, j.cell & ((c.page_tokens >> 4) - 1));
#pragma unroll 1
    for (int t = 0; t < 4; ++t) {
        const int slot = 2 * t + (part & 1) + 8 * (part >> 1), pos = j.cell * kKv4Cell + slot;
        if (pos < j.from || pos >= j.to)
            continue;
        const int64_t token = (int64_t)j.s.first + (pos - (j.s.len - j.s.n_new));
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            void *const out = kv ? v : k;
            if (!out)
                continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int g = G == 2 ? h : 0;
                uint32_t code = 0;
                float s = 0.0f, mid = 0.0f;
                if (src) {
                    if (kv == 0) {
                        const __half2 p = *(const __half2 *)(src + C::kKp + (slot * G + g) * 4);
                        s = __low2float(p);
                        mid = __high2float(p);
                        code = D == 128 ? *(const uint32_t *)(src + slot * 64 + (i >> 1) * 16 + h * 8 + (i & 1) * 4)
                                        : *(const uint16_t *)(src + slot * 32 + (2 * h + (i >> 2)) * 8 + (i & 3) * 2);
                    } else {
                        const __half *p = (const __half *)(src + C::kVp + ((t + 4 * (part >> 1)) * G + g) * 8) + (part & 1);
                        s = __half2float(p[0]);
                        mid = __half2float(p[2]);
                        const uint8_t *const at = src + C::kV + t * 16 + (part >> 1) * 8 + (part & 1) * 2;
                        if (D == 128) {
                            const uint8_t *const q = at + h * 512 + i * 64;
                            code = *(const uint16_t *)q | (uint32_t)*(const uint16_t *)(q + 4) << 16;
                        } else {
                            code = *(const uint16_t *)(at + (4 * h + (i >> 1)) * 64 + (i & 1) * 4);
                        }
                    }
                }
                float x[N];
#pragma unroll
                for (int n = 0; n < N; ++n)
                    x[n] = __fadd_rn(__fmul_rn((float)(int)((code >> (4 * n)) & 15u) - 8.0f, s), mid);
                const int64_t o = (token * c.n_kv_heads + head) * D + h * (D / 2) + N * i;
                if (!src) {
#pragma unroll
                    for (int n = 0; n < N; ++n)
                        x[n] = 0.0f;
                }
                if (F32) {
#pragma unroll
                    for (int n = 0; n < N; n += 4)
                        *(float4 *)((float *)out + o + n) = make_float4(x[n], x[n + 1], x[n + 2], x[n + 3]);
                } else {
                    uint32_t y[N / 2];
#pragma unroll
                    for (int n = 0; n < N / 2; ++n)
                        y[n] = f32_to_bf16_rn(x[2 * n]) | ((uint32_t)f32_to_bf16_rn(x[2 * n + 1]) << 16);
                    if (N == 8)
                        *(uint4 *)((uint16_t *)out + o) = make_uint4(y[0], y[1], y[N / 2 - 2], y[N / 2 - 1]);
                    else
                        *(uint2 *)((uint16_t *)out + o) = make_uint2(y[0], y[1]);
                }
            }
        }
    }
}

// Slots of cells for the new tokens of a call (see cell_job).
int64_t slots_of(const Kv4Batch &b)
{
    return b.starts && b.n_seqs > 0 ? b.n_tokens / kKv4Cell + 2 * (int64_t)b.n_seqs : b.n_seqs;
}

} // namespace

nm_status kv4_launch_append(const Kv4 &c, const Kv4Batch &b, int layer, const void *k, int64_t k_stride,
                            const void *v, int64_t v_stride, const void *q, int64_t q_stride, int n_q_heads,
                            void *q_out, int64_t q_out_stride, const float *rope, int64_t rope_rows, cudaStream_t st)
{
    AppendArgs a{layer, n_q_heads, (const uint16_t *)k, (const uint16_t *)v, (const uint16_t *)q,
                 (uint16_t *)q_out, k_stride, v_stride, q_stride, q_out_stride, rope, rope_rows, 0, 0, 0, 1, 1};
    a.slots = slots_of(b) * c.n_kv_heads;
    a.cell_ctas = (a.slots + 7) / 8;
    if (q) {
        // with many tokens a warp turns up to four fours of a token's heads, so that its angles are read once
        const int fours = (n_q_heads + 3) / 4;
        a.q_each = b.n_tokens * fours >= 65536 ? (fours < kFours ? fours : kFours) : 1;
        a.q_warps = (fours + a.q_each - 1) / a.q_each;
        a.q_ctas = (b.n_tokens * a.q_warps + 7) / 8;
    }
    const int64_t grid = a.cell_ctas + a.q_ctas + (b.starts ? 1 : 0);
    if (grid > 0x7FFFFFFF)
        return NM_ERR_SHAPE;
    if (c.head_dim == 128)
        append_kernel<128><<<(unsigned)grid, 256, 0, st>>>(c, b, a);
    else
        append_kernel<64><<<(unsigned)grid, 256, 0, st>>>(c, b, a);
    return cudaGetLastError() == cudaSuccess ? NM_OK : NM_ERR_CUDA;
}

nm_status kv4_launch_read(const Kv4 &c, const Kv4Batch &b, int layer, void *k, void *v, bool f32, cudaStream_t st)
{
    const int64_t slots = slots_of(b) * c.n_kv_heads, ctas = (slots + 7) / 8;
    const int64_t grid = ctas + (b.starts ? kRestCtas : 0);
    if (grid > 0x7FFFFFFF)
        return NM_ERR_SHAPE;
    if (c.head_dim == 128) {
        if (f32)
            read_kernel<128, true><<<(unsigned)grid, 256, 0, st>>>(c, b, layer, k, v, slots, ctas);
        else
            read_kernel<128, false><<<(unsigned)grid, 256, 0, st>>>(c, b, layer, k, v, slots, ctas);
    } else {
        if (f32)
            read_kernel<64, true><<<(unsigned)grid, 256, 0, st>>>(c, b, layer, k, v, slots, ctas);
        else
            read_kernel<64, false><<<(unsigned)grid, 256, 0, st>>>(c, b, layer, k, v, slots, ctas);
    }
    return cudaGetLastError() == cudaSuccess ? NM_OK : NM_ERR_CUDA;
}

} // namespace nm
